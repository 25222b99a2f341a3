// Forward of cross attention on the sm_103a tensor cores: O and the row log-sum-exp of
// queries over the keys of another sequence, with shared key heads, padded batches
// and splits of the key axis.
//
//   S = Q K_j^T (fp32, TMEM), m = running row maximum of S * scale * log2e,
//   P = exp2(S * scale * log2e - m), l += rowsum(P), O += P V_j;  O / l, m + log2 l
//
// A persistent grid: one CTA an SM takes units in a fixed stride. A unit is two 128-row
// tiles A and B of query rows that share a key head (of one head, or of several where
// queries are few) against the keys of one split. TMEM: S_A [0, 128), S_B [128, 256),
// O_A [256, 256 + d), O_B after it. One warp issues all MMAs, per key block
// O_A(j), S_A(j+1), O_B(j), S_B(j+1): while tile A's softmax warps turn S_A into P_A, the
// tensor cores run tile B. Eight softmax warps a tile: a row is split between two
// warps (the same TMEM lane), 64 keys of a block each, that exchange only whether a row's
// reference has to move a block (and then their halves' maxima) and their sums at the end. P
// goes back over the S columns it came from, per K step of 16 keys as 8 columns of 16-bit
// values and 8 of their rounding residuals, and the O MMAs read both from TMEM. The row's
// reference m moves only when a block's maximum exceeds it by more than 2^8.
//
// The residuals are half as many MMAs again. Rounded once, P moves an output about as much as
// the rounding of the output itself does (bf16, 2-norm error against 64 bits 2.3e-3 over 77 as
// over 16383 keys; 1.66e-3 with residuals, which is the output's own rounding). What they cost
// (us, with / without): 4x16 4096 over texts of 169 to 512 84 / 70, 2x16/4 4095 over 34 and 77,
// d = 64, 21.3 / 18.2, 1x16 64 over 16383 40 / 33, 1x32/8 8192 over 4096 518 / 397, d = 64 459 /
// 340. (In the form of one pass without them, which kept P's image in registers until both warps
// agreed on the reference, they spilled: 97 and 605.) Not only for tiles with large weights,
// as in fa_fwd: over a few hundred keys nearly every tile has some, and a branch in front of the
// residuals' MMAs took 25% by itself.
//
// Few keys a unit are the common case here (a text's 77 to 512), so a unit is short: steps,
// ring stages and barrier phases run on from unit to unit, the next unit's queries and
// first keys are loaded and its first S MMAs issued while the last block's softmax
// and the epilogue of this one run. Only the O accumulator is handed over: its next first
// MMA waits until the epilogue has loaded it (OFree).
//
// Masks. Keys from the split's end on get P = 0 by selects, so K's rows there may hold
// anything; V's rows there are zeroed in shared memory before the MMA (0 * NaN). Rows of
// Q that are not there give rows of S that nobody reads.
#include <algorithm>

#include "fa_cross.h"
#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kThreads = 576;  // TMA warp, MMA warp, 2 x 8 softmax warps
constexpr float kRescaleLog2 = 8.f;

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kPanel = 128 * 128;        // 16 KB: 128 rows x 64 elements
  static constexpr uint32_t kTile = kPanels * kPanel;  // one 128-row tile of Q, K or V
  static constexpr int kNK = D == 64 ? 4 : 2;          // K ring stages
  static constexpr int kNV = D == 64 ? 4 : 2;          // V ring stages
  static constexpr uint32_t oQ = 0;                    // [2 tiles]
  static constexpr uint32_t oK = 2 * kTile;
  static constexpr uint32_t oV = oK + kNK * kTile;
  static constexpr uint32_t oBar = oV + kNV * kTile;
  static constexpr int bQ = 0;                         // [2] a unit's Q tile landed
  static constexpr int bQFree = bQ + 2;                // [2] its last S MMA done
  static constexpr int bKFull = bQFree + 2;
  static constexpr int bKEmpty = bKFull + kNK;
  static constexpr int bVFull = bKEmpty + kNK;
  static constexpr int bVEmpty = bVFull + kNV;
  static constexpr int bSFull = bVEmpty + kNV;         // [2] S landed
  static constexpr int bPFull = bSFull + 2;            // [2] P image written
  static constexpr int bODone = bPFull + 2;            // [2] O MMA of a block done
  static constexpr int bOFree = bODone + 2;            // [2] the epilogue has read O
  static constexpr int bDrain = bOFree + 2;
  static constexpr int bXchg = bDrain + 1;             // [tile][lane quarter] row-maximum exchange
  static constexpr int bSum = bXchg + 8;              // [tile][lane quarter] final row-sum exchange
  static constexpr int bFast = bSum + 8;               // [tile][lane quarter] outcome of the one-pass form exchanged
  static constexpr int kBars = bFast + 8;
  static constexpr uint32_t oTmemSlot = oBar + kBars * 8;
  static constexpr uint32_t oAbort = oTmemSlot + 8;
  static constexpr uint32_t oFast = (oAbort + 8 + 15) & ~15u;    // [exchange parity][16 softmax warps] outcomes
  static constexpr uint32_t oUnits = oFast + 2 * 16 * 4;         // [kMostUnits]
  // row maxima [tile][exchange parity][half][128 rows], then the sums [tile][half][128 rows]
  static constexpr uint32_t oXchg = oUnits + kMostUnits * sizeof(CrossUnit);
  static constexpr uint32_t kSmem = oXchg + (2 * 2 * 2 + 2 * 2) * 128 * 4 + 1024;  // + slack for 1024-byte alignment
  static_assert(kSmem <= 227u * 1024u, "shared memory budget exceeded");
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CrossParams p, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  let_next_begin();
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::oAbort);
  auto bar = [&](int idx) -> uint32_t { return sb + C::oBar + 8u * idx; };
  const int mine = (cross_units<2>(p) - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // units of this block
  CrossUnit* const unit = reinterpret_cast<CrossUnit*>(smem + C::oUnits);
  // The first from the i-th on that has blocks to compute (mine: none).
  const auto next_work = [&](int i) {
    while (i < mine && unit[i].blocks == 0) ++i;
    return i;
  };

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(C::bQ + x), 1);
      mbar_init(bar(C::bQFree + x), 1);
      mbar_init(bar(C::bSFull + x), 1);
      mbar_init(bar(C::bPFull + x), 256);  // the tile's eight softmax warps
      mbar_init(bar(C::bODone + x), 1);
      mbar_init(bar(C::bOFree + x), 256);
    }
    for (int s = 0; s < C::kNK; ++s) {
      mbar_init(bar(C::bKFull + s), 1);
      mbar_init(bar(C::bKEmpty + s), 1);
    }
    for (int s = 0; s < C::kNV; ++s) {
      mbar_init(bar(C::bVFull + s), 1);
      mbar_init(bar(C::bVEmpty + s), 1);
    }
    mbar_init(bar(C::bDrain), 1);
    for (int x = 0; x < 8; ++x) {  // the two warps of a row quarter
      mbar_init(bar(C::bXchg + x), 64);
      mbar_init(bar(C::bSum + x), 64);
      mbar_init(bar(C::bFast + x), 64);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + C::oTmemSlot, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  wait_for_previous();
  if ((int)threadIdx.x < mine) {
    CrossUnit u;
    cross_unit<2>(p, blockIdx.x + threadIdx.x * gridDim.x, u);
    unit[threadIdx.x] = u;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::oTmemSlot);

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)C::kPanels * 128u << (p.plan.q_tile.q_log + p.plan.q_tile.h_log);
      int t = 0, nq[2] = {0, 0}, issuedK = 0, issuedV = 0;  // blocks and tiles loaded
      bool ok = true;
      for (int i = next_work(0); ok && i < mine; i = next_work(i + 1)) {
        const CrossUnit& u = unit[i];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || !u.live(x)) continue;
          if (nq[x] > 0 && !mbar_wait(bar(C::bQFree + x), (nq[x] - 1) & 1, abort_flag, p.status)) {
            ok = false;
            continue;
          }
          mbar_arrive_expect_tx(bar(C::bQ + x), q_bytes);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_4d(sb + C::oQ + x * C::kTile + pn * C::kPanel, &tmQ, bar(C::bQ + x), 64 * pn, u.q0[x], u.h0[x],
                        u.b);
          ++nq[x];
        }
        for (int j = 0; ok && j < u.blocks; ++j, ++t) {
          const int sk = t % C::kNK, sv = t % C::kNV, row = u.j_begin + 128 * j;
          if (!mbar_wait(bar(C::bKEmpty + sk), ((t / C::kNK) & 1) ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::bKFull + sk), C::kTile);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_4d(sb + C::oK + sk * C::kTile + pn * C::kPanel, &tmK, bar(C::bKFull + sk), 64 * pn, row, u.hk,
                        u.b);
          issuedK = t + 1;
          if (!mbar_wait(bar(C::bVEmpty + sv), ((t / C::kNV) & 1) ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::bVFull + sv), C::kTile);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_4d(sb + C::oV + sv * C::kTile + pn * C::kPanel, &tmV, bar(C::bVFull + sv), 64 * pn, row, u.hk,
                        u.b);
          issuedV = t + 1;
        }
      }
      if (*abort_flag) {
        // Let every copy this thread started land before the CTA exits.
        for (int x = 0; x < 2; ++x)
          if (nq[x] > 0) mbar_wait_drain(bar(C::bQ + x), (nq[x] - 1) & 1, p.status);
        for (int j = max(0, issuedK - C::kNK); j < issuedK; ++j)
          mbar_wait_drain(bar(C::bKFull + j % C::kNK), (j / C::kNK) & 1, p.status);
        for (int j = max(0, issuedV - C::kNV); j < issuedV; ++j)
          mbar_wait_drain(bar(C::bVFull + j % C::kNV), (j / C::kNV) & 1, p.status);
      }
    }
  } else if (warp == 1) {
    // ------------------------------- MMA issuer --------------------------------
    // S_X = Q_X K_j^T: M = 128 rows, N = 128 keys, K = d (both K-major). O_X += P_X V_j:
    // M = 128, N = d, K = 128 keys; A = the P image in TMEM, B = V_j read MN-major.
    constexpr uint32_t idS = make_idesc(128, 128, kBf16, false, false);
    constexpr uint32_t idO = make_idesc(128, D, kBf16, false, true);
    const uint64_t dQ0 = make_sdesc(sb + C::oQ, 16, 1024);
    const uint64_t dK0 = make_sdesc(sb + C::oK, 16, 1024);
    const uint64_t dV0 = make_sdesc(sb + C::oV, C::kPanel, 1024);
    int steps[2] = {0, 0}, tiles[2] = {0, 0};  // blocks and units a tile has been through
    bool ok = true;
    // S of tile x for block t of the CTA (K landed); last: the unit's last for this tile.
    auto issue_s = [&](int x, int t, bool last) {
      const uint64_t kd = desc_add(dK0, (t % C::kNK) * C::kTile), qd = desc_add(dQ0, x * C::kTile);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        tc_mma_ss_w(tmem + 128 * x, desc_add(qd, (k >> 2) * C::kPanel + (k & 3) * 32),
                    desc_add(kd, (k >> 2) * C::kPanel + (k & 3) * 32), idS, k > 0 ? 1u : 0u);
      tc_commit_w(bar(C::bSFull + x));
      if (last) tc_commit_w(bar(C::bQFree + x));
    };
    auto issue_o = [&](int x, int t, bool first) {
      const uint64_t vd = desc_add(dV0, (t % C::kNV) * C::kTile);
      const uint32_t tO = tmem + 256 + D * x, tP = tmem + 128 * x;
#pragma unroll
      for (int k = 0; k < 8; ++k)  // (a K step's image: 8 rounded columns, then 8 of their residuals)
        tc_mma_ts_w(tO, tP + 16 * k, desc_add(vd, 2048 * k), idO, k > 0 || !first ? 1u : 0u);
#pragma unroll
      for (int k = 0; k < 8; ++k) tc_mma_ts_w(tO, tP + 16 * k + 8, desc_add(vd, 2048 * k), idO, 1u);
      tc_commit_w(bar(C::bODone + x));
    };
    struct {
      int i, blocks, j_begin, j_end;
      bool live[2];
    } u, next;  // the unit at hand and the next one (i = mine: none)
    const auto read = [&](int i, auto& to) {
      to.i = uniform(next_work(i));
      const CrossUnit& from = unit[min(to.i, mine - 1)];
      to.blocks = uniform(from.blocks);
      to.j_begin = uniform(from.j_begin);
      to.j_end = uniform(from.j_end);
      const int has = uniform(from.has);
#pragma unroll
      for (int x = 0; x < 2; ++x) to.live[x] = to.i < mine && (has >> (2 + x) & 1);
    };
    int t = 0;
    read(0, u);
    if (u.i < mine) {
      ok = warp_wait<kIssuerPoll>(bar(C::bKFull), 0, abort_flag, p.status);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ok || !u.live[x]) continue;
        ok = warp_wait<kIssuerPoll>(bar(C::bQ + x), 0, abort_flag, p.status);
        if (!ok) continue;
        tc_fence_after();
        issue_s(x, 0, u.blocks == 1);
      }
      if (ok) tc_commit_w(bar(C::bKEmpty));
    }
    while (ok && u.i < mine) {
      read(u.i + 1, next);
      for (int j = 0; ok && j < u.blocks; ++j, ++t) {
        const int sv = t % C::kNV;
        const bool inside = j + 1 < u.blocks, more = inside || next.i < mine;
        if (!warp_wait<kIssuerPoll>(bar(C::bVFull + sv), (t / C::kNV) & 1, abort_flag, p.status) ||
            (more && !warp_wait<kIssuerPoll>(bar(C::bKFull + (t + 1) % C::kNK), ((t + 1) / C::kNK) & 1, abort_flag,
                                             p.status))) {
          ok = false;
          break;
        }
        // V's rows from the sequence's end on, as far as they are the tensor's (past it: zeros by TMA).
        const int from = u.j_end - u.j_begin - 128 * j, to = min(128, p.Nk - u.j_begin - 128 * j);
        if (from < to) zero_rows<C::kPanels>(sb + C::oV + sv * C::kTile, C::kPanel, from, to);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok) continue;
          if (u.live[x]) {
            if (!warp_wait<kIssuerPoll>(bar(C::bPFull + x), steps[x] & 1, abort_flag, p.status) ||
                (j == 0 && tiles[x] > 0 &&
                 !warp_wait<kIssuerPoll>(bar(C::bOFree + x), (tiles[x] - 1) & 1, abort_flag, p.status))) {
              ok = false;
              continue;
            }
            tc_fence_after();
            issue_o(x, t, j == 0);
            ++steps[x];
            if (!inside) ++tiles[x];
          }
          if (inside ? u.live[x] : next.live[x]) {
            if (!inside && !warp_wait<kIssuerPoll>(bar(C::bQ + x), tiles[x] & 1, abort_flag, p.status)) {
              ok = false;
              continue;
            }
            tc_fence_after();
            issue_s(x, t + 1, inside ? j + 2 == u.blocks : next.blocks == 1);
          }
        }
        if (!ok) break;
        tc_commit_w(bar(C::bVEmpty + sv));                             // V read by both O MMAs
        if (more) tc_commit_w(bar(C::bKEmpty + (t + 1) % C::kNK));  // the next K read by both S MMAs
      }
      u = next;
    }
    // Every MMA this warp issued is complete before the CTA frees TMEM and exits.
    tc_commit_w(bar(C::bDrain));
    if (lane == 0) mbar_wait_drain(bar(C::bDrain), 0, p.status);
    __syncwarp();
  } else {
    // ------------------------------ softmax warps ------------------------------
    // warps 2-17; a warp reaches TMEM lanes 32 (warp % 4) .. + 31
    const int x = (warp - 2) >> 3;           // tile
    const int half = ((warp - 2) >> 2) & 1;  // keys [64 half, 64 half + 64) of a block
    const int wq = warp & 3;
    const int il = wq * 32 + lane;  // row in the tile, TMEM lane
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + 128 * x + 64 * half;           // this warp's 64 S columns
    const uint32_t tO = tmem + lane_off + 256 + D * x + (D / 2) * half;  // and D/2 O columns
    float* xchg = reinterpret_cast<float*>(smem + C::oXchg);
    float* xl = xchg + 8 * 128 + (x * 2) * 128;
    const int pq = 4 * x + wq;  // the two warps holding rows 32 wq .. 32 wq + 31 of tile x
    const float c2 = p.scale_log2;
    const int row_q = il & (p.plan.q_tile.queries() - 1), row_h = il >> p.plan.q_tile.q_log;
    const bool row_in = row_h < p.plan.q_tile.heads();
    volatile int* fast = reinterpret_cast<volatile int*>(smem + C::oFast);
    int nx = 0, nf = 0;   // exchanges of maxima and of outcomes so far
    int n = 0, done = 0;  // blocks and units this tile has been through
    bool ok = true;
    // Waits block (the hardware suspends the warp): each tile's warps idle about half the
    // time, and spinning would take issue slots from the other tile's warps.
    for (int ui = 0; ok && ui < mine; ++ui) {
      const CrossUnit& u = unit[ui];
      if (!u.there(x)) continue;
      // this warp's real keys from the first block on; a real query's row: what else lies in the tile has no vote
      const int blocks = u.live(x) ? u.blocks : 0, left = u.j_end - u.j_begin - 64 * half;
      const bool real = row_in && u.q0[x] + row_q < u.nq;
      float mref = -INFINITY, lsum = 0.f;  // lsum: this half's part of the row sum
      for (int j = 0; j < blocks; ++j, ++n) {
        if (!warp_wait<false>(bar(C::bSFull + x), n & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int hi = left - 128 * j;  // columns 0 .. hi - 1
        // A row's first reference is the maximum of its first 16 scores, which both of its warps read.
        if (j == 0) {
          uint32_t cur[16];
          const int in = hi + 64 * half;
          tmem_ld16(tS - 64 * half, cur);
          tmem_ld_wait16(cur);
#pragma unroll
          for (int e = 0; e < 16; ++e) mref = e < in ? fmaxf(mref, __uint_as_float(cur[e])) : mref;
          mref *= c2;
        }
        // This half's maximum of S. Both warps of the rows move the reference where a row's maximum asks for it,
        // which it nearly never does after the first block: the outcomes are exchanged before the maxima.
        float hmax = -INFINITY;
        {
          uint32_t s0[32], s1[32];
          __syncwarp();
          tmem_ld32(tS, s0);
          tmem_ld32(tS + 32, s1);
          tmem_ld_wait2(s0, s1);
          if (hi >= 64) {
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              m0 = fmax3(m0, __uint_as_float(s0[e]), __uint_as_float(s0[e + 1]));
              m1 = fmax3(m1, __uint_as_float(s1[e]), __uint_as_float(s1[e + 1]));
            }
            hmax = fmaxf(m0, m1);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              hmax = (e < hi) ? fmaxf(hmax, __uint_as_float(s0[e])) : hmax;
              hmax = (32 + e < hi) ? fmaxf(hmax, __uint_as_float(s1[e])) : hmax;
            }
          }
        }
        const bool moves = __any_sync(0xffffffffu, real && hmax * c2 > mref + kRescaleLog2);
        if (lane == 0) fast[16 * (nf & 1) + (warp - 2)] = moves;
        warp_arrive(bar(C::bFast + pq));
        if (!warp_wait<false>(bar(C::bFast + pq), nf & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        const bool either = moves || fast[16 * (nf & 1) + ((warp - 2) ^ 4)] != 0;
        ++nf;
        if (either) {
          // The block maximum of the row: this half's and the other warp's (slots alternate
          // from exchange to exchange, so a slot is rewritten only after the partner has passed
          // the next one, i.e. has read it).
          float* xs = xchg + ((x * 2 + (nx & 1)) * 2) * 128;
          xs[half * 128 + il] = hmax;
          warp_arrive(bar(C::bXchg + pq));
          if (!warp_wait<false>(bar(C::bXchg + pq), nx & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          ++nx;
          const float bmax = fmaxf(hmax, xs[(half ^ 1) * 128 + il]) * c2;  // (scale > 0)
          // Lazy rescale. Both warps of a row take the same decision; each rescales its D/2 O columns.
          const bool mv = bmax > mref + kRescaleLog2;
          const float alpha = mv ? ex2_approx(mref - bmax) : 1.f;  // 0 when mref = -inf
          // (warp-wide decision: the wait and the TMEM accesses below are collective)
          if (j > 0 && __any_sync(0xffffffffu, mv && mref != -INFINITY)) {
            // this tile's O MMA of the block before is done before its rows are rescaled
            if (!warp_wait<false>(bar(C::bODone + x), (n - 1) & 1, abort_flag, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < D / 64; ++cc) {
              uint32_t r[32];
              tmem_ld32(tO + 32 * cc, r);
              tmem_ld_wait(r);
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
              tmem_st32(tO + 32 * cc, r);
            }
          }
          if (mv) {
            lsum *= alpha;
            mref = bmax;
          }
        }
        const float base = mref == -INFINITY ? 0.f : mref;  // (every score so far is -inf or NaN)
        // 32 keys at a time: P (0 past the end), this half's running sum, and the image.
        const uint64_t cc2 = f2_pack(c2, c2), nm2 = f2_pack(-base, -base);
        uint64_t sum2 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t cur[32], img[32];
          __syncwarp();
          tmem_ld32(tS + 32 * q, cur);
          tmem_ld_wait(cur);
          const auto weights = [&](auto masked) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float p0, p1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(cur[e]), __uint_as_float(cur[e + 1])), cc2, nm2), p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              if constexpr (decltype(masked)::value) {
                p0 = 32 * q + e < hi ? p0 : 0.f;
                p1 = 32 * q + e + 1 < hi ? p1 : 0.f;
              }
              sum2 = f2_add(sum2, f2_pack(p0, p1));
              uint32_t &top = img[16 * (e >> 4) + ((e & 15) >> 1)], &rest = img[16 * (e >> 4) + ((e & 15) >> 1) + 8];
              if constexpr (kBf16) {
                top = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
                float r0, r1;
                f2_unpack(f2_add(f2_pack(p0, p1), f2_pack(-__uint_as_float(__float_as_uint(p0) & 0xFFFF0000u),
                                                          -__uint_as_float(__float_as_uint(p1) & 0xFFFF0000u))),
                          r0, r1);
                rest = pack2<kBf16>(r0, r1);
              } else {
                top = pack2<kBf16>(p0, p1);
                rest = pack2_residual<kBf16>(p0, p1, top);
              }
            }
          };
          if (hi >= 64)
            weights(std::false_type{});
          else
            weights(std::true_type{});
          __syncwarp();
          tmem_st32(tS + 32 * q, img);
        }
        lsum += f2_sum(sum2);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(bar(C::bPFull + x));
      }
      if (!ok) break;
      // Epilogue: the row sum of both halves; this warp's D/2 columns of O / l, 32 at a time. The accumulator is
      // released (OFree) behind its last load.
      float ltot = 0.f;
      if (blocks > 0) {
        xl[half * 128 + il] = lsum;
        warp_arrive(bar(C::bSum + pq));
        if (!warp_wait<false>(bar(C::bSum + pq), done & 1, abort_flag, p.status) ||
            !warp_wait<false>(bar(C::bODone + x), (n - 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        ltot = lsum + xl[(half ^ 1) * 128 + il];
        tc_fence_after();
        ++done;
      }
      const int i = u.q0[x] + row_q, h = u.h0[x] + row_h, b = u.b, part = u.split;
      const bool in = row_in && i < p.Nq, has = blocks > 0 && i < u.nq && ltot != 0.f;  // (a NaN sum is there)
      const float inv = has ? 1.f / ltot : 0.f, lse2 = has ? mref + lg2(ltot) : -INFINITY;
      const long long at = ((long long)b * p.Hq + h) * p.Nq + i, rows = (long long)p.B * p.Nq * p.Hq;
      const bool parts = p.plan.k_splits > 1;
      if (in && half == 0) {
        if (parts)
          p.part_lse[part * rows + at] = lse2;
        else
          p.lse_out[at] = has ? lse2 * 0.6931471805599453f : -INFINITY;
      }
      // (rows without keys of the split: the join does not read their part)
      float* to_part = nullptr;
      uint16_t* to_out = nullptr;
      if (parts && in && has)
        to_part = p.part + (part * rows + ((long long)b * p.Nq + i) * p.Hq + h) * D + D / 2 * half;
      if (!parts && in)
        to_out = static_cast<uint16_t*>(p.out) + b * p.out_st.b + i * p.out_st.n + h * p.out_st.h + D / 2 * half;
#pragma unroll 1
      for (int cc = 0; cc < D / 64; ++cc) {
        uint32_t r[32];  // (set on every path: left undefined on one, values of the blocks' loop spilled)
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = 0u;
        __syncwarp();
        if (blocks > 0) {
          tmem_ld32(tO + 32 * cc, r);
          tmem_ld_wait(r);
          if (cc == D / 64 - 1) {
            tc_fence_before();
            warp_arrive(bar(C::bOFree + x));
          }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = has ? r[e] : 0u;
        store_columns32<kBf16>(r, inv, parts, to_part ? to_part + 32 * cc : nullptr,
                               to_out ? to_out + 32 * cc : nullptr);
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kBf16>
cudaError_t launch_t(const CrossParams& p, const CUtensorMap* maps, cudaStream_t st) {
  constexpr int bytes = (int)std::max(Cfg<D>::kSmem, kMinSmemOneCtaPerSm);
  constexpr auto kKernel = cross_fwd_kernel<D, kBf16>;
  const cudaError_t e = allow_smem<kKernel>(bytes);
  if (e != cudaSuccess) return e;
  const long long units = (long long)p.B * p.Hk * ((p.plan.q_tile.count(p.Nq, p.G) + 1) / 2) * p.plan.k_splits;
  const long long blocks = std::max(std::min(units, 152ll), (units + kMostUnits - 1) / kMostUnits);
  return launch_chained_maps(kKernel, dim3((unsigned)blocks), kThreads, bytes, st, p, maps[0], maps[1], maps[2]);
}

}  // namespace

cudaError_t launch_cross_fwd_tc(const CrossParams& p, bool bf16, const CUtensorMap* maps, cudaStream_t st) {
  if (p.d == 128) return bf16 ? launch_t<128, true>(p, maps, st) : launch_t<128, false>(p, maps, st);
  return bf16 ? launch_t<64, true>(p, maps, st) : launch_t<64, false>(p, maps, st);
}

}  // namespace fa
