// Backward of cross attention on the sm_103a tensor cores: two kinds of blocks over the
// same recomputed probabilities, one that holds keys and walks queries (dK, dV), one that
// holds queries and walks keys (dQ), so that every sum is formed on chip in a fixed order.
//
//   S = Q K^T, P = exp2(S * scale*log2e - L*log2e), dP = dO V^T, dS = P o (dP - D)
//   dV += P^T dO, dK += dS^T Q over the queries of all heads of a group; dQ += dS K
//
// dK/dV: keys on the 128 TMEM lanes, steps of 64 query rows (of one head of the group, or
// of several where queries are few; the steps run over all heads of the group, so shared
// key heads cost no extra sums), S^T and dP^T in double buffers, P^T and dS^T written back
// over them in 16 bits with their rounding residual, dV and dK in TMEM. dQ: 128 query rows on the
// lanes, steps of 128 keys, dS with its residual as well. Rounded once, P and dS move dV and dK by
// about as much as the rounding of the results (2-norm error against 64 bits 1.41 times that, 1.00
// with residuals), and dQ by more: a row's dS add up to 0, their roundings do not, and what is left
// of them is multiplied by the mean of the keys under P, which is not small where q and k have large
// channels (bf16 700 over 160 keys 1.46). Times, us, with all residuals / with those of dV and dK in
// tiles with a probability above 1/64 only, as in fa_bwd (1.0 to 1.4), whose vote costs some too:
// bf16 4x16 2048 over texts of 169 to 512 138 / 142, 1x32/8 8192x4096 with even scores 1722 / 1632,
// with large channels and the forward 2500 / 2445. D comes from the scores (kernels_cross_dot.cu).
// Warp 0 issues TMA loads, warps 1 and 3 the S and dP MMAs, warp 2 the accumulating
// ones, warps 4-19 do the row math.
//
// One CTA an SM. Both kinds are in one launch, dK/dV first. A block takes a few units (key
// tiles; query tiles) in a fixed stride, enough of them to outweigh its start; steps, ring
// stages and barrier phases run on from unit to unit, so that the next unit's loads and
// first MMAs overlap this one's end. Where there are few units for the GPU (few keys and
// many queries, or the other way round) the walked axis is cut into splits whose fp32 sums
// a second kernel adds in order.
//
// Masks. Query columns and key columns past their sequence's length get P = dS = 0 by
// selects (S and dP there may be NaN); the rows of Q, dO and K that such columns meet in the
// accumulating MMAs are zeroed in shared memory first (0 * NaN).
#include <algorithm>

#include "fa_cross.h"
#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kThreads = 640;  // 4 role warps + 4 row-math warpgroups
constexpr int kStep = 64;      // query rows of a step of the dK/dV kernel

// ------------------------------- dK and dV -------------------------------
template <int D>
struct KCfg {
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kKVPanel = 128 * 128;   // 16 KB: 128 rows x 64 elements
  static constexpr uint32_t kKVTile = kPanels * kKVPanel;
  static constexpr uint32_t kQPanel = kStep * 128;  // 8 KB: 64 rows x 64 elements
  static constexpr uint32_t kQTile = kPanels * kQPanel;
  static constexpr int kNS = 4;                     // Q/dO ring stages
  static constexpr uint32_t oK = 0;
  static constexpr uint32_t oV = oK + kKVTile;
  static constexpr uint32_t oQ = oV + kKVTile;
  static constexpr uint32_t oDO = oQ + kNS * kQTile;
  static constexpr uint32_t oL = oDO + kNS * kQTile;
  static constexpr uint32_t oD = oL + kNS * kStep * 4;
  static constexpr uint32_t oBar = oD + kNS * kStep * 4;
  static constexpr int bKV = 0;                     // K, V of a unit landed
  static constexpr int bQFull = 1;
  static constexpr int bQEmpty = bQFull + kNS;
  static constexpr int bSFull = bQEmpty + kNS;      // [2] S^T landed
  static constexpr int bDPFull = bSFull + 2;        // [2] dP^T landed
  static constexpr int bSEmpty = bDPFull + 2;       // [2] dV done with the P^T image
  static constexpr int bDPEmpty = bSEmpty + 2;      // [2] dK done with the dS^T image
  static constexpr int bPFull = bDPEmpty + 2;       // [2] P^T image written
  static constexpr int bDSFull = bPFull + 2;        // [2] dS^T image written
  // [2] a unit's dV, dK complete in TMEM: a barrier for each pair of row-math warpgroups, which waits for the units
  // whose epilogue it writes (on one barrier for both, a pair that skips the other's units could take the
  // phase before last for the one that it waits for)
  static constexpr int bAcc = bDSFull + 2;
  static constexpr int bDrain = bAcc + 2;           // one per MMA-issuing warp
  static constexpr int bKVFree = bDrain + 3;        // a unit's last reads of K, V done
  static constexpr int bAccFree = bKVFree + 1;      // the epilogue has read dV, dK
  static constexpr int kBars = bAccFree + 1;
  static constexpr uint32_t oTmemSlot = oBar + kBars * 8;
  static constexpr uint32_t oAbort = oTmemSlot + 8;
  static constexpr uint32_t oUnits = oAbort + 8;    // [kMostUnits]
  static constexpr uint32_t kSmem = oUnits + kMostUnits * 44 + 1024;  // + slack for 1024-byte alignment
  static_assert(kSmem <= 227u * 1024u, "shared memory budget exceeded");
};

// One key tile of a (batch, key head) against the query steps of one split.
struct KUnit {
  int b, hk, split, j0, nq, nk;
  int first, steps;  // steps first .. first + steps - 1 of the sequence's live ones (0: nothing to compute)
  int chunks, chunk;  // live chunks of a head's queries, the first step's
  int exp;            // fp16: dS is multiplied as dS * 2^exp (cross_exponent)
};
static_assert(sizeof(KUnit) == 44, "as KCfg::kSmem has it");

__device__ __forceinline__ int k_units(const CrossParams& p) {
  return p.B * p.Hk * ((p.Nk + 127) / 128) * p.plan.q_splits;
}

// idx: split fastest, then the tiles of a (batch, key head), which share its queries through L2.
__device__ __forceinline__ void k_unit(const CrossParams& p, int idx, KUnit& u) {
  const int tiles = (p.Nk + 127) / 128;
  const int rest = idx / p.plan.q_splits;
  u.split = idx - rest * p.plan.q_splits;
  const int bh = rest / tiles;
  u.j0 = (rest - bh * tiles) * 128;
  u.b = bh / p.Hk;
  u.hk = bh - u.b * p.Hk;
  u.nq = cross_q_len(p, u.b);
  u.nk = cross_k_len(p, u.b);
  u.chunks = p.plan.step.chunks(u.nq);
  const int total = u.chunks * (p.G >> p.plan.step.h_log), per = (total + p.plan.q_splits - 1) / p.plan.q_splits;
  u.first = u.split * per;
  u.steps = u.j0 < u.nk ? max(min(per, total - u.first), 0) : 0;
  u.chunk = u.first % max(u.chunks, 1);
}

// Head (of all) and first query of a live step.
__device__ __forceinline__ void k_step(const CrossParams& p, const KUnit& u, int it, int& h0, int& q0) {
  const int s = u.first + it, group = s / u.chunks;
  h0 = u.hk * p.G + (group << p.plan.step.h_log);
  q0 = (s - group * u.chunks) << p.plan.step.q_log;
}

// Columns 32 c .. 32 c + 31 of a step that hold a real query.
__device__ __forceinline__ uint32_t step_columns(const CrossTile& t, int c, int left) {
  const int q = t.queries(), rows = q << t.h_log;
  uint32_t m;
  if (q >= 32) {
    const int in = q == 64 ? 32 * c : 0;  // the chunk's first query
    m = bit_range(0, left - in);
  } else {
    m = bit_range(0, min(q, left));
    for (int s = q; s < 32; s <<= 1) m |= m << s;
  }
  return m & bit_range(0, rows - 32 * c);
}

// A block's share: the units first, first + stride, ...
template <int D, bool kBf16>
__device__ __forceinline__ void dkdv_block(const CrossParams& p, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                           const CUtensorMap& tmV, const CUtensorMap& tmDO, uint8_t* smem, int first,
                                           int stride) {
  using C = KCfg<D>;
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::oAbort);
  auto bar = [&](int idx) -> uint32_t { return sb + C::oBar + 8u * idx; };
  const int mine = (k_units(p) - first + stride - 1) / stride;  // units of this block
  KUnit* const unit = reinterpret_cast<KUnit*>(smem + C::oUnits);
  const int rows = 1 << (p.plan.step.q_log + p.plan.step.h_log);
  // The first unit from the i-th on that has steps (mine: none).
  const auto next_work = [&](int i) {
    while (i < mine && unit[i].steps == 0) ++i;
    return i;
  };

  if (threadIdx.x == 0) {
    mbar_init(bar(C::bKV), 1);
    for (int s = 0; s < C::kNS; ++s) {
      mbar_init(bar(C::bQFull + s), 1);
      mbar_init(bar(C::bQEmpty + s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(C::bSFull + x), 1);
      mbar_init(bar(C::bDPFull + x), 1);
      mbar_init(bar(C::bSEmpty + x), 1);
      mbar_init(bar(C::bDPEmpty + x), 1);
      mbar_init(bar(C::bPFull + x), 256);   // two warpgroups
      mbar_init(bar(C::bDSFull + x), 256);
      mbar_init(bar(C::bAcc + x), 1);
    }
    for (int x = 0; x < 3; ++x) mbar_init(bar(C::bDrain + x), 1);
    mbar_init(bar(C::bKVFree), 2);          // S^T and dP^T issuers
    mbar_init(bar(C::bAccFree), 8 * 32);    // the epilogue pair's row-math warps
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
    prefetch_tmap(&tmDO);
  }
  if (rows < kStep) {  // the rows that no copy reaches: the accumulating MMAs read them with weight 0
    for (int x = threadIdx.x; x < 2 * C::kNS * (int)C::kQTile / 16; x += kThreads)
      st_shared_v4(sb + C::oQ + 16 * x, 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  wait_for_previous();
  if ((int)threadIdx.x < mine) {
    KUnit u;
    k_unit(p, first + threadIdx.x * stride, u);
    u.exp = 0;
    if constexpr (!kBf16) {
      const int bh = u.b * p.Hk + u.hk;
      u.exp = cross_exponent(__uint_as_float(p.dout_most[bh]), cross_v_norm(p, bh));
    }
    unit[threadIdx.x] = u;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::oTmemSlot);
  const uint32_t tS = tmem, tdP = tmem + 128, tdV = tmem + 256, tdK = tmem + 256 + D;

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)(2 * C::kPanels * 128 + 2 * 4) * rows;
      int kl = 0, G = 0;  // units and steps loaded
      bool ok = true;
      for (int i = next_work(0); ok && i < mine; i = next_work(i + 1)) {
        const KUnit& u = unit[i];
        // K and V of this unit, once the previous unit's last reads of them are done
        if (kl > 0 && !mbar_wait(bar(C::bKVFree), (kl - 1) & 1, abort_flag, p.status)) break;
        mbar_arrive_expect_tx(bar(C::bKV), 2 * C::kKVTile);
        for (int pn = 0; pn < C::kPanels; ++pn) {
          tma_load_4d(sb + C::oK + pn * C::kKVPanel, &tmK, bar(C::bKV), 64 * pn, u.j0, u.hk, u.b);
          tma_load_4d(sb + C::oV + pn * C::kKVPanel, &tmV, bar(C::bKV), 64 * pn, u.j0, u.hk, u.b);
        }
        ++kl;
        for (int it = 0; it < u.steps; ++it, ++G) {
          const int s = G % C::kNS;
          if (!mbar_wait(bar(C::bQEmpty + s), ((G / C::kNS) & 1) ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          int h0, q0;
          k_step(p, u, it, h0, q0);
          mbar_arrive_expect_tx(bar(C::bQFull + s), q_bytes);
          for (int pn = 0; pn < C::kPanels; ++pn) {
            tma_load_4d(sb + C::oQ + s * C::kQTile + pn * C::kQPanel, &tmQ, bar(C::bQFull + s), 64 * pn, q0, h0, u.b);
            tma_load_4d(sb + C::oDO + s * C::kQTile + pn * C::kQPanel, &tmDO, bar(C::bQFull + s), 64 * pn, q0, h0,
                        u.b);
          }
          const int q = p.plan.step.queries();
          for (int h = 0; h < p.plan.step.heads(); ++h) {
            const long long at = ((long long)u.b * p.Hq + h0 + h) * p.nq_pad + q0;
            bulk_load(sb + C::oL + (s * kStep + h * q) * 4, p.nL2 + at, q * 4, bar(C::bQFull + s));
            bulk_load(sb + C::oD + (s * kStep + h * q) * 4, p.nD + at, q * 4, bar(C::bQFull + s));
          }
        }
      }
      if (*abort_flag) {
        // Let every copy this thread started land before the CTA exits.
        if (kl > 0) mbar_wait_drain(bar(C::bKV), (kl - 1) & 1, p.status);
        for (int x = max(0, G - C::kNS); x < G; ++x)
          mbar_wait_drain(bar(C::bQFull + x % C::kNS), (x / C::kNS) & 1, p.status);
      }
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------ S^T (warp 1) / dP^T (warp 3) MMA issuer ----------------
    // S^T = K Q^T or dP^T = V dO^T: M = 128 keys, N = 64 queries, K = d, both K-major.
    const bool isS = warp == 1;
    constexpr uint32_t idS = make_idesc(128, kStep, kBf16, false, false);
    const uint64_t dA0 = make_sdesc(sb + (isS ? C::oK : C::oV), 16, 1024),
                   dB0 = make_sdesc(sb + (isS ? C::oQ : C::oDO), 16, 1024);
    const uint32_t tD = isS ? tS : tdP;
    const int bF = isS ? C::bSFull : C::bDPFull, bE = isS ? C::bSEmpty : C::bDPEmpty;
    int kl = 0, G = 0;
    bool ok = true;
    for (int i = next_work(0); ok && i < mine; i = next_work(i + 1), ++kl) {
      i = uniform(i);
      const int steps = uniform(unit[i].steps);
      ok = warp_wait<kIssuerPoll>(bar(C::bKV), kl & 1, abort_flag, p.status);
      for (int it = 0; ok && it < steps; ++it, ++G) {
        const int s = G % C::kNS, bb = G & 1;
        if (!warp_wait<kIssuerPoll>(bar(C::bQFull + s), (G / C::kNS) & 1, abort_flag, p.status) ||
            !warp_wait<kIssuerPoll>(bar(bE + bb), ((G >> 1) & 1) ^ 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t bq = desc_add(dB0, s * C::kQTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss_w(tD + 64 * bb, desc_add(dA0, (kk >> 2) * C::kKVPanel + (kk & 3) * 32),
                      desc_add(bq, (kk >> 2) * C::kQPanel + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
        tc_commit_w(bar(bF + bb));
      }
      if (!ok) break;
      tc_commit_w(bar(C::bKVFree));  // this unit's last reads of K / V
    }
    // Every MMA this warp issued is complete before the CTA frees TMEM and exits.
    const int dr = isS ? 0 : 2;
    tc_commit_w(bar(C::bDrain + dr));
    if (lane == 0) mbar_wait_drain(bar(C::bDrain + dr), 0, p.status);
    __syncwarp();
  } else if (warp == 2) {
    // ----------------------------- dV / dK MMA issuer ----------------------------
    constexpr uint32_t idG = make_idesc(128, D, kBf16, false, true);
    const uint64_t mQ0 = make_sdesc(sb + C::oQ, C::kQPanel, 1024), mO0 = make_sdesc(sb + C::oDO, C::kQPanel, 1024);
    int kl = 0, G = 0;
    bool ok = true;
    for (int i = next_work(0); ok && i < mine; i = next_work(i + 1), ++kl) {
      i = uniform(i);
      const int steps = uniform(unit[i].steps), chunks = uniform(unit[i].chunks), nq = uniform(unit[i].nq);
      int chunk = uniform(unit[i].chunk);
      for (int it = 0; it < steps; ++it, ++G) {
        const int bt = G & 1, st = G % C::kNS;
        if (!warp_wait<kConsumerPoll>(bar(C::bPFull + bt), (G >> 1) & 1, abort_flag, p.status) ||
            // a unit's first MMAs overwrite the accumulators that the previous unit's epilogue reads
            (it == 0 && kl > 0 && !warp_wait<kConsumerPoll>(bar(C::bAccFree), (kl - 1) & 1, abort_flag, p.status))) {
          ok = false;
          break;
        }
        // Rows of queries past the sequence's end, as far as they are the tensors' (past them: zeros by
        // TMA). S^T is formed; dP^T may still read dO: its columns of these rows are not used.
        if (++chunk == chunks) {
          chunk = 0;
          const int q0 = (chunks - 1) << p.plan.step.q_log, q = p.plan.step.queries();
          const int from = nq - q0, to = min(q, p.Nq - q0);
          for (int h = 0; from < to && h < p.plan.step.heads(); ++h) {
            zero_rows<C::kPanels>(sb + C::oQ + st * C::kQTile, C::kQPanel, h * q + from, h * q + to);
            zero_rows<C::kPanels>(sb + C::oDO + st * C::kQTile, C::kQPanel, h * q + from, h * q + to);
          }
        }
        tc_fence_after();
        const uint32_t keep = it > 0 ? 1u : 0u;
        const uint64_t qd = desc_add(mQ0, st * C::kQTile), gd = desc_add(mO0, st * C::kQTile);
        // dV += P^T dO: K step kk reads the 8 rounded columns at 16kk of the P^T image and the 8 residual
        // columns at 16kk + 8.
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          tc_mma_ts_w(tdV, tS + 64 * bt + 16 * kk, desc_add(gd, 2048 * kk), idG, kk > 0 ? 1u : keep);
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          tc_mma_ts_w(tdV, tS + 64 * bt + 16 * kk + 8, desc_add(gd, 2048 * kk), idG, 1u);
        tc_commit_w(bar(C::bSEmpty + bt));
        // dK once the dS^T image is in place; dV above only needed P^T.
        if (!warp_wait<kConsumerPoll>(bar(C::bDSFull + bt), (G >> 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          tc_mma_ts_w(tdK, tdP + 64 * bt + 16 * kk, desc_add(qd, 2048 * kk), idG, kk > 0 ? 1u : keep);
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          tc_mma_ts_w(tdK, tdP + 64 * bt + 16 * kk + 8, desc_add(qd, 2048 * kk), idG, 1u);
        tc_commit_w(bar(C::bDPEmpty + bt));
        tc_commit_w(bar(C::bQEmpty + st));
      }
      if (!ok) break;
      tc_commit_w(bar(C::bAcc + ((G - 1) & 1)));  // (the pair that ran the last step)
    }
    tc_commit_w(bar(C::bDrain + 1));
    if (lane == 0) mbar_wait_drain(bar(C::bDrain + 1), 0, p.status);
    __syncwarp();
  } else {
    // ------------------------- row-math warpgroups --------------------------
    // rg = 0, 1 take the even steps (TMEM buffer 0) and rg = 2, 3 the odd ones, counted
    // across units; warpgroup rg & 1 takes query columns [32 (rg & 1), + 32). Two phases a
    // step: P^T from S^T (released to the dV MMA at once), then dS^T from dP^T and the kept
    // fp32 P. The pair that ran a unit's last step writes its epilogue; the other goes on.
    const int rg = (warp - 4) >> 2, wq = warp & 3, c = rg & 1, bb = rg >> 1;
    const int jl = wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tSc = tS + lane_off + 64 * bb + 32 * c, tdPc = tdP + lane_off + 64 * bb + 32 * c;
    const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
    int written = 0, G = 0;  // units whose epilogue this pair wrote, steps of all units
    bool ok = true;
    for (int ui = 0; ok && ui < mine; ++ui) {
      const KUnit& u = unit[ui];
      const int steps = u.steps, chunks = max(u.chunks, 1);
      int chunk = u.chunk + ((bb ^ G) & 1);
      chunk -= chunk >= chunks ? chunks : 0;
      // The columns with real queries of any step but a head's last (or last few heads') and of that one. (A lane
      // without a real key needs no mask: its row of P^T and dS^T reaches nothing but its own row of dV and dK, which
      // the epilogue drops.)
      const uint32_t full = step_columns(p.plan.step, c, kStep);
      const uint32_t tail = step_columns(p.plan.step, c, u.nq - ((chunks - 1) << p.plan.step.q_log));
      const float to_ds = kBf16 ? 1.f : power_of_2(u.exp - (int)kCrossPLog2<kBf16>);  // from P's power of 2 to dS's
      const uint64_t to_ds2 = f2_pack(to_ds, to_ds);
      for (int it = (bb ^ G) & 1; it < steps; it += 2) {
        const int gs = G + it, s = gs % C::kNS;
        const uint32_t allow = chunk == chunks - 1 ? tail : full;
        chunk += 2;
        chunk -= chunk >= chunks ? chunks : 0;
        chunk -= chunk >= chunks ? chunks : 0;  // (a head of one chunk)
        if (!warp_wait<kRowMathPoll>(bar(C::bQFull + s), (gs / C::kNS) & 1, abort_flag, p.status) ||
            !warp_wait<kRowMathPoll>(bar(C::bSFull + bb), (gs >> 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float4* L4 = reinterpret_cast<const float4*>(smem + C::oL + s * kStep * 4 + 128 * c);
        const float4* D4 = reinterpret_cast<const float4*>(smem + C::oD + s * kStep * 4 + 128 * c);
        float P[32];  // of this thread's 32 pairs (times kCrossPUnit), for the dS phase
        // ---- phase 1: the P^T image over the S^T columns ----
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t sr[16];
          __syncwarp();
          tmem_ld16(tSc + 16 * hh, sr);
          tmem_ld_wait16(sr);
          auto p_phase = [&](auto masked) {
#pragma unroll
            for (int x = 0; x < 16; x += 4) {
              const float4 l4 = L4[(16 * hh + x) >> 2];
              float pv[4];
              const uint64_t s01 = f2_pack(__uint_as_float(sr[x]), __uint_as_float(sr[x + 1]));
              const uint64_t s23 = f2_pack(__uint_as_float(sr[x + 2]), __uint_as_float(sr[x + 3]));
              f2_unpack(f2_fma(s01, c2, f2_pack(l4.x, l4.y)), pv[0], pv[1]);
              f2_unpack(f2_fma(s23, c2, f2_pack(l4.z, l4.w)), pv[2], pv[3]);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int bit = 16 * hh + x + y;
                pv[y] = ex2_approx(pv[y]);
                if constexpr (decltype(masked)::value) pv[y] = ((allow >> bit) & 1u) ? pv[y] : 0.f;
                P[bit] = pv[y];
              }
            }
          };
          if (allow == 0xFFFFFFFFu)  // (the same for the whole warp)
            p_phase(std::false_type{});
          else
            p_phase(std::true_type{});
          uint32_t hp[8], ep[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) hp[x] = pack2<kBf16>(P[16 * hh + 2 * x], P[16 * hh + 2 * x + 1]);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            ep[x] = pack2_residual<kBf16>(P[16 * hh + 2 * x], P[16 * hh + 2 * x + 1], hp[x]);
          __syncwarp();
          // this K step's image: 8 rounded columns, then 8 residual columns
          tmem_st8<0>(tSc + 16 * hh, hp);
          tmem_st8<0>(tSc + 16 * hh + 8, ep);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(bar(C::bPFull + bb));
        // ---- phase 2: dS^T = P o (dP^T + (-D)) ----
        if (!warp_wait<kRowMathPoll>(bar(C::bDPFull + bb), (gs >> 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t dr[16];
          __syncwarp();
          tmem_ld16(tdPc + 16 * hh, dr);
          tmem_ld_wait16(dr);
          float ds[16];
#pragma unroll
          for (int x = 0; x < 16; x += 4) {
            const float4 d4 = D4[(16 * hh + x) >> 2];
            const uint64_t d01 =
                f2_add(f2_pack(__uint_as_float(dr[x]), __uint_as_float(dr[x + 1])), f2_pack(d4.x, d4.y));
            const uint64_t d23 =
                f2_add(f2_pack(__uint_as_float(dr[x + 2]), __uint_as_float(dr[x + 3])), f2_pack(d4.z, d4.w));
            uint64_t p01 = f2_pack(P[16 * hh + x], P[16 * hh + x + 1]);
            uint64_t p23 = f2_pack(P[16 * hh + x + 2], P[16 * hh + x + 3]);
            if constexpr (!kBf16) {
              p01 = f2_mul(p01, to_ds2);
              p23 = f2_mul(p23, to_ds2);
            }
            f2_unpack(f2_mul(p01, d01), ds[x], ds[x + 1]);
            f2_unpack(f2_mul(p23, d23), ds[x + 2], ds[x + 3]);
          }
          if (allow != 0xFFFFFFFFu) {  // (dP^T of what is not there may be NaN)
#pragma unroll
            for (int x = 0; x < 16; ++x) ds[x] = ((allow >> (16 * hh + x)) & 1u) ? ds[x] : 0.f;
          }
          __syncwarp();
          uint32_t hd[8], ed[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) hd[x] = pack2<kBf16>(ds[2 * x], ds[2 * x + 1]);
#pragma unroll
          for (int x = 0; x < 8; ++x) ed[x] = pack2_residual<kBf16>(ds[2 * x], ds[2 * x + 1], hd[x]);
          tmem_st8<0>(tdPc + 16 * hh, hd);
          tmem_st8<0>(tdPc + 16 * hh + 8, ed);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(bar(C::bDSFull + bb));
      }
      if (!ok) break;
      // Epilogue, by the pair that ran the unit's last step: dV, then dK, each warpgroup half of the
      // columns; both accumulators are released (AccFree) behind the last load.
      const bool epi = steps > 0 ? bb == ((G + steps - 1) & 1) : bb == 0;
      if (epi) {
        if (steps > 0) {
          if (!warp_wait<kRowMathPoll>(bar(C::bAcc + bb), written & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          ++written;
        }
        const int b = u.b, hk = u.hk, j = u.j0 + jl, nk = u.nk;
        const long long size = (long long)p.B * p.Nk * p.Hk * D;
        const bool parts = p.plan.q_splits > 1;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {  // 32 columns of dV, then of dK
          const bool isK = cc >= D / 64;
          const int col = c * (D / 2) + 32 * (cc & (D / 64 - 1));
          uint32_t r[32];  // (set on every path: left undefined on one, 25 values of the steps' loop spilled)
#pragma unroll
          for (int x = 0; x < 32; ++x) r[x] = 0u;
          __syncwarp();
          if (steps > 0) {
            tmem_ld32((isK ? tdK : tdV) + lane_off + col, r);
            tmem_ld_wait(r);
            if (cc == D / 32 - 1) {
              tc_fence_before();
              warp_arrive(bar(C::bAccFree));
            }
          }
#pragma unroll
          for (int x = 0; x < 32; ++x) r[x] = j < nk ? r[x] : 0u;  // (0 * NaN of a real query's)
          float* to_part = parts && j < nk ? p.part_kv + 2 * u.split * size + (isK ? 0 : size) +
                                                 (((long long)b * p.Nk + j) * p.Hk + hk) * D + col
                                           : nullptr;
          const fa_strides& st = isK ? p.dk_st : p.dv_st;
          uint16_t* const grad = static_cast<uint16_t*>(isK ? p.dk : p.dv);
          uint16_t* to_out = !parts && j < p.Nk ? grad + b * st.b + j * st.n + hk * st.h + col : nullptr;
          float mul = isK && !parts ? p.scale : 1.f;
          if (!kBf16) mul *= isK ? power_of_2(-u.exp) : 1.f / kCrossPUnit<kBf16>;
          store_columns32<kBf16>(r, mul, parts, to_part, to_out);
        }
        __syncwarp();
      }
      G += steps;
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

// ---------------------------------- dQ -----------------------------------
template <int D>
struct QCfg {
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kPanel = 128 * 128;
  static constexpr uint32_t kTile = kPanels * kPanel;  // one 128-row tile of Q, dO, K or V
  static constexpr int kNV = 2;                        // V ring stages
  static constexpr int kNK = D == 64 ? 4 : 3;          // K ring stages (read by S and by dQ)
  static constexpr uint32_t oQ = 0;
  static constexpr uint32_t oDO = oQ + kTile;
  static constexpr uint32_t oV = oDO + kTile;
  static constexpr uint32_t oK = oV + kNV * kTile;
  static constexpr uint32_t oBar = oK + kNK * kTile;
  static constexpr int bRes = 0;                       // Q, dO of a unit landed
  static constexpr int bVFull = 1;
  static constexpr int bVEmpty = bVFull + kNV;
  static constexpr int bKFull = bVEmpty + kNV;
  static constexpr int bKEmpty = bKFull + kNK;
  static constexpr int bSFull = bKEmpty + kNK;         // [2] S and dP landed
  static constexpr int bSEmpty = bSFull + 2;           // [2] dQ MMA done with the image
  static constexpr int bDPEmpty = bSEmpty + 2;         // row math has read dP
  static constexpr int bPFull = bDPEmpty + 1;          // [2] dS image written
  // Accumulators, units in turn. With d = 64 there is room for two, and a unit's epilogue runs behind the next
  // unit's first step, so that its last dQ MMA and the next S and dP are under way meanwhile: with one key block a
  // unit (77 keys) 5.6 k cycles a unit before, 3.8 since (backward of 2x16/4 4095x77 57 -> 52 us). With one
  // accumulator the next unit's first MMA waited for the epilogue (4x16 2048x512 138 -> 139.5 us).
  static constexpr int kAcc = D == 64 ? 2 : 1;
  static constexpr int bAcc = bPFull + 2;              // [kAcc] dQ of a unit complete
  static constexpr int bDrain = bAcc + kAcc;           // one per MMA-issuing warp
  static constexpr int bResFree = bDrain + 3;          // a unit's last reads of Q and dO done
  static constexpr int bAccFree = bResFree + 1;        // [kAcc] the epilogue has read the accumulator
  static constexpr int kBars = bAccFree + kAcc;
  static constexpr uint32_t oTmemSlot = oBar + kBars * 8;
  static constexpr uint32_t oAbort = oTmemSlot + 8;
  static constexpr uint32_t oUnits = oAbort + 8;       // [kMostUnits]
  static constexpr uint32_t kSmem = oUnits + kMostUnits * sizeof(CrossUnit) + 1024;  // + slack for 1024-byte alignment
  static_assert(kSmem <= 227u * 1024u, "shared memory budget exceeded");
};

template <int D, bool kBf16>
__device__ __forceinline__ void dq_block(const CrossParams& p, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                         const CUtensorMap& tmV, const CUtensorMap& tmDO, uint8_t* smem, int first,
                                         int stride) {
  using C = QCfg<D>;
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::oAbort);
  auto bar = [&](int idx) -> uint32_t { return sb + C::oBar + 8u * idx; };
  const int mine = (cross_units<1>(p) - first + stride - 1) / stride;  // units of this block
  CrossUnit* const unit = reinterpret_cast<CrossUnit*>(smem + C::oUnits);
  const auto next_work = [&](int i) {
    while (i < mine && unit[i].blocks == 0) ++i;
    return i;
  };

  if (threadIdx.x == 0) {
    mbar_init(bar(C::bRes), 1);
    for (int s = 0; s < C::kNV; ++s) {
      mbar_init(bar(C::bVFull + s), 1);
      mbar_init(bar(C::bVEmpty + s), 1);
    }
    for (int s = 0; s < C::kNK; ++s) {
      mbar_init(bar(C::bKFull + s), 1);
      mbar_init(bar(C::bKEmpty + s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(C::bSFull + x), 2);
      mbar_init(bar(C::bSEmpty + x), 1);
      mbar_init(bar(C::bPFull + x), 512);
    }
    mbar_init(bar(C::bDPEmpty), 512);
    for (int x = 0; x < C::kAcc; ++x) {
      mbar_init(bar(C::bAcc + x), 1);
      mbar_init(bar(C::bAccFree + x), 512);  // every row-math warp
    }
    for (int x = 0; x < 3; ++x) mbar_init(bar(C::bDrain + x), 1);
    mbar_init(bar(C::bResFree), 2);    // S and dP issuers
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
    prefetch_tmap(&tmDO);
  }
  wait_for_previous();
  if ((int)threadIdx.x < mine) {
    CrossUnit u;
    cross_unit<1>(p, first + threadIdx.x * stride, u);
    u.v_norm = kBf16 ? 0.f : cross_v_norm(p, u.b * p.Hk + u.hk);
    unit[threadIdx.x] = u;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::oTmemSlot);
  const uint32_t tS = tmem, tdP = tmem + 256, tAcc = tmem + 384;

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (lane == 0) {
      const uint32_t q_bytes = 2u * C::kPanels * 128u << (p.plan.q_tile.q_log + p.plan.q_tile.h_log);
      int kl = 0, G = 0, issuedV = 0, issuedK = 0;
      bool ok = true;
      for (int i = next_work(0); ok && i < mine; i = next_work(i + 1)) {
        const CrossUnit& u = unit[i];
        if (kl > 0 && !mbar_wait(bar(C::bResFree), (kl - 1) & 1, abort_flag, p.status)) break;
        mbar_arrive_expect_tx(bar(C::bRes), q_bytes);
        for (int pn = 0; pn < C::kPanels; ++pn) {
          tma_load_4d(sb + C::oQ + pn * C::kPanel, &tmQ, bar(C::bRes), 64 * pn, u.q0[0], u.h0[0], u.b);
          tma_load_4d(sb + C::oDO + pn * C::kPanel, &tmDO, bar(C::bRes), 64 * pn, u.q0[0], u.h0[0], u.b);
        }
        ++kl;
        for (int it = 0; it < u.blocks; ++it, ++G) {
          const int row = u.j_begin + 128 * it, sv = G % C::kNV, sk = G % C::kNK;
          if (!mbar_wait(bar(C::bVEmpty + sv), ((G / C::kNV) & 1) ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::bVFull + sv), C::kTile);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_4d(sb + C::oV + sv * C::kTile + pn * C::kPanel, &tmV, bar(C::bVFull + sv), 64 * pn, row, u.hk,
                        u.b);
          issuedV = G + 1;
          if (!mbar_wait(bar(C::bKEmpty + sk), ((G / C::kNK) & 1) ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::bKFull + sk), C::kTile);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_4d(sb + C::oK + sk * C::kTile + pn * C::kPanel, &tmK, bar(C::bKFull + sk), 64 * pn, row, u.hk,
                        u.b);
          issuedK = G + 1;
        }
      }
      if (*abort_flag) {
        if (kl > 0) mbar_wait_drain(bar(C::bRes), (kl - 1) & 1, p.status);
        for (int x = max(0, issuedV - C::kNV); x < issuedV; ++x)
          mbar_wait_drain(bar(C::bVFull + x % C::kNV), (x / C::kNV) & 1, p.status);
        for (int x = max(0, issuedK - C::kNK); x < issuedK; ++x)
          mbar_wait_drain(bar(C::bKFull + x % C::kNK), (x / C::kNK) & 1, p.status);
      }
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------ S (warp 1) / dP (warp 3) MMA issuer -------------------
    const bool isS = warp == 1;
    constexpr uint32_t idS = make_idesc(128, 128, kBf16, false, false);
    const uint64_t dA0 = make_sdesc(sb + (isS ? C::oQ : C::oDO), 16, 1024),
                   dB0 = make_sdesc(sb + (isS ? C::oK : C::oV), 16, 1024);
    int kl = 0, G = 0;
    bool ok = true;
    for (int i = next_work(0); ok && i < mine; i = next_work(i + 1), ++kl) {
      i = uniform(i);
      const int blocks = uniform(unit[i].blocks);
      ok = warp_wait<kIssuerPoll>(bar(C::bRes), kl & 1, abort_flag, p.status);
      for (int it = 0; ok && it < blocks; ++it, ++G) {
        const int bb = G & 1, st = isS ? G % C::kNK : G % C::kNV;
        const bool landed = isS ? warp_wait<kIssuerPoll>(bar(C::bKFull + st), (G / C::kNK) & 1, abort_flag, p.status)
                                : warp_wait<kIssuerPoll>(bar(C::bVFull + st), (G / C::kNV) & 1, abort_flag, p.status);
        // S: its buffer's image is consumed; dP: the row math has read the step before's
        if (!landed ||
            (isS && !warp_wait<kIssuerPoll>(bar(C::bSEmpty + bb), ((G >> 1) & 1) ^ 1, abort_flag, p.status)) ||
            (!isS && G > 0 && !warp_wait<kIssuerPoll>(bar(C::bDPEmpty), (G - 1) & 1, abort_flag, p.status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t bd = desc_add(dB0, st * C::kTile);
        const uint32_t tD = isS ? tS + 128 * bb : tdP;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss_w(tD, desc_add(dA0, (kk >> 2) * C::kPanel + (kk & 3) * 32),
                      desc_add(bd, (kk >> 2) * C::kPanel + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
        tc_commit_w(bar(C::bSFull + bb));
        if (!isS) tc_commit_w(bar(C::bVEmpty + st));
      }
      if (!ok) break;
      tc_commit_w(bar(C::bResFree));  // this unit's last reads of Q / dO
    }
    const int dr = isS ? 0 : 2;
    tc_commit_w(bar(C::bDrain + dr));
    if (lane == 0) mbar_wait_drain(bar(C::bDrain + dr), 0, p.status);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------ dQ MMA issuer -----------------------------
    constexpr uint32_t idO = make_idesc(128, D, kBf16, false, true);
    const uint64_t b0 = make_sdesc(sb + C::oK, C::kPanel, 1024);
    int kl = 0, G = 0;
    bool ok = true;
    for (int i = next_work(0); ok && i < mine; i = next_work(i + 1), ++kl) {
      i = uniform(i);
      const int blocks = uniform(unit[i].blocks);
      const int j_begin = uniform(unit[i].j_begin), j_end = uniform(unit[i].j_end);
      const int x = kl % C::kAcc, turn = kl / C::kAcc;
      for (int it = 0; it < blocks; ++it, ++G) {
        const int bt = G & 1, sk = G % C::kNK;
        if (!warp_wait<kConsumerPoll>(bar(C::bPFull + bt), (G >> 1) & 1, abort_flag, p.status) ||
            (it == 0 && turn > 0 &&
             !warp_wait<kConsumerPoll>(bar(C::bAccFree + x), (turn - 1) & 1, abort_flag, p.status))) {
          ok = false;
          break;
        }
        // K's rows from the sequence's end on, as far as they are the tensor's (S, which read them, is formed)
        const int from = j_end - j_begin - 128 * it, to = min(128, p.Nk - j_begin - 128 * it);
        if (from < to) zero_rows<C::kPanels>(sb + C::oK + sk * C::kTile, C::kPanel, from, to);
        tc_fence_after();
        const uint64_t bop = desc_add(b0, sk * C::kTile);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc_mma_ts_w(tAcc + 64 * x, tS + 128 * bt + 16 * kk, desc_add(bop, 2048 * kk), idO,
                      kk > 0 || it > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc_mma_ts_w(tAcc + 64 * x, tS + 128 * bt + 16 * kk + 8, desc_add(bop, 2048 * kk), idO, 1u);
        tc_commit_w(bar(C::bSEmpty + bt));
        tc_commit_w(bar(C::bKEmpty + sk));
      }
      if (!ok) break;
      tc_commit_w(bar(C::bAcc + x));
    }
    tc_commit_w(bar(C::bDrain + 1));
    if (lane == 0) mbar_wait_drain(bar(C::bDrain + 1), 0, p.status);
    __syncwarp();
  } else {
    // ---------------- row-math warpgroups + epilogue ----------------------
    // Warpgroup c takes key columns [32c, 32c + 32) of every step, in halves of 16 (a K step of the dQ MMA: 8
    // rounded columns, then 8 residual ones), and a quarter of the epilogue's columns.
    const int c = (warp - 4) >> 2, wq = warp & 3;
    const int il = wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tdPc = tdP + lane_off + 32 * c;
    const int row_q = il & (p.plan.q_tile.queries() - 1), row_h = il >> p.plan.q_tile.q_log;
    const bool row_in = row_h < p.plan.q_tile.heads();
    const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
    int kl = 0, G = 0;
    bool ok = true;
    // The next unit's -L and -D of this row (-inf and 0 past the sequence) are on their way while one is worked on.
    // (fp16: -L with the row's exponent added, which makes P and dS 2^e times as large, and 2^-e)
    const auto row_of = [&](int ui, float& nl, float& nd, float& back) {
      nl = -INFINITY;
      nd = 0.f;
      back = 1.f;
      if (ui < mine && unit[ui].blocks > 0 && row_in) {
        const CrossUnit& u = unit[ui];
        const long long at = ((long long)u.b * p.Hq + u.h0[0] + row_h) * p.nq_pad + u.q0[0] + row_q;
        nl = p.nL2[at];
        nd = p.nD[at];
        if constexpr (!kBf16) {
          const int e = cross_exponent(p.dout_norm[at], u.v_norm);
          nl += (float)e - kCrossPLog2<kBf16>;
          back = power_of_2(-e);
        }
      }
    };
    float nL2, nD, back_now, nL2_next, nD_next, back_next, back_last = 1.f;
    row_of(0, nL2, nD, back_now);
    constexpr bool kLater = C::kAcc == 2;  // (see kAcc; the round of ui = mine then has an epilogue alone)
    for (int ui = 0; ok && ui < mine + kLater;
         ++ui, nL2 = nL2_next, nD = nD_next, back_last = back_now, back_now = back_next) {
      const CrossUnit& u = unit[min(ui, mine - 1)];
      // left: real keys from this warpgroup's first column on
      const int blocks = ui < mine ? u.blocks : 0, left = u.j_end - u.j_begin - 32 * c;
      if (!kLater) row_of(ui + 1, nL2_next, nD_next, back_next);
      const uint64_t l2 = f2_pack(nL2, nL2), d2 = f2_pack(nD, nD);
      int it = 0;
      do {
        if (it < blocks) {
          const int gs = G + it, bb = gs & 1;
          const uint32_t tSc = tS + lane_off + 128 * bb + 32 * c;
          const uint32_t allow = bit_range(0, left - 128 * it);
          if (!warp_wait<kRowMathPoll>(bar(C::bSFull + bb), (gs >> 1) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // both halves of dP come in with S, so the dP buffer is released before any arithmetic
          uint32_t sr[16], dr[2][16];
          __syncwarp();
          tmem_ld16(tSc, sr);
          tmem_ld16(tdPc, dr[0]);
          tmem_ld16(tdPc + 16, dr[1]);
          tmem_ld_wait16x3(sr, dr[0], dr[1]);
          tc_fence_before();
          warp_arrive(bar(C::bDPEmpty));
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            if (hh == 1) {
              __syncwarp();
              tmem_ld16(tSc + 16, sr);
              tmem_ld_wait16(sr);
            }
            float ds[16];
            auto elementwise = [&](auto masked) {
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                float p0, p1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), c2, l2), p0, p1);
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                const uint64_t dd = f2_add(f2_pack(__uint_as_float(dr[hh][e]), __uint_as_float(dr[hh][e + 1])), d2);
                f2_unpack(f2_mul(f2_pack(p0, p1), dd), ds[e], ds[e + 1]);
                if constexpr (decltype(masked)::value) {
                  const bool in0 = (allow >> (16 * hh + e)) & 1u, in1 = (allow >> (16 * hh + e + 1)) & 1u;
                  ds[e] = in0 ? ds[e] : 0.f;
                  ds[e + 1] = in1 ? ds[e + 1] : 0.f;
                }
              }
            };
            // (the mask is the same for the whole warp)
            if (allow == 0xFFFFFFFFu)
              elementwise(std::false_type{});
            else
              elementwise(std::true_type{});
            uint32_t hv[16];  // rounded, then the residuals
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              hv[x] = pack2<kBf16>(ds[2 * x], ds[2 * x + 1]);
              hv[8 + x] = pack2_residual<kBf16>(ds[2 * x], ds[2 * x + 1], hv[x]);
            }
            tmem_st16(tSc + 16 * hh, hv);
          }
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(bar(C::bPFull + bb));
        }
        if (kLater ? it > 0 : it + 1 < blocks) continue;
        if (kLater) row_of(ui + 1, nL2_next, nD_next, back_next);
        if (kLater && ui == 0) continue;
        // Epilogue: columns [c d / 4, (c + 1) d / 4). The accumulator is loaded and released
        // (AccFree) before the stores, so the next MMA into it can start meanwhile.
        const CrossUnit& to = unit[ui - kLater];
        uint32_t r[32];  // (D / 4 of them)
#pragma unroll
        for (int x = 0; x < 32; ++x) r[x] = 0u;
        if (to.blocks > 0) {
          const int x = kl % C::kAcc;
          if (!warp_wait<kRowMathPoll>(bar(C::bAcc + x), kl / C::kAcc & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t col0 = tAcc + 64 * x + lane_off + c * (D / 4);
          if constexpr (D == 128) {
            tmem_ld32(col0, r);
            tmem_ld_wait(r);
          } else {
            uint32_t half[16];
            tmem_ld16(col0, half);
            tmem_ld_wait16(half);
#pragma unroll
            for (int y = 0; y < 16; ++y) r[y] = half[y];
          }
          tc_fence_before();
          warp_arrive(bar(C::bAccFree + x));
          ++kl;
        }
        const int i = to.q0[0] + row_q, h = to.h0[0] + row_h, b = to.b, nq = to.nq;
        const bool parts = p.plan.k_splits > 1, in = row_in && i < (parts ? nq : p.Nq);
#pragma unroll
        for (int x = 0; x < 32; ++x) r[x] = i < nq ? r[x] : 0u;  // (rows that are not there may hold NaN)
        float* to_part = nullptr;
        uint16_t* to_out = nullptr;
        if (parts && in)
          to_part = p.part + ((((long long)to.split * p.B + b) * p.Nq + i) * p.Hq + h) * D + c * (D / 4);
        if (!parts && in)
          to_out = static_cast<uint16_t*>(p.out) + b * p.out_st.b + i * p.out_st.n + h * p.out_st.h + c * (D / 4);
        float mul = parts ? 1.f : p.scale;
        if (!kBf16) mul *= kLater ? back_last : back_now;
        if constexpr (D == 128)
          store_columns32<kBf16>(r, mul, parts, to_part, to_out);
        else
          store_columns16<kBf16>(r, mul, parts, to_part, to_out);
        __syncwarp();
      } while (ok && ++it < blocks);
      G += blocks;
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

// One launch for both: blocks [0, kv_blocks) take the units of dK/dV, the others those of dQ, so that they share
// the GPU and each other's tails (4x16 2048x512 77 + 50 us in two launches, 118 in one; 1x32/8 8192x4096 823 + 507
// and 1300).
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    cross_bwd_kernel(const __grid_constant__ CrossParams p, const __grid_constant__ CUtensorMap tmQStep,
                     const __grid_constant__ CUtensorMap tmDOStep, const __grid_constant__ CUtensorMap tmQTile,
                     const __grid_constant__ CUtensorMap tmDOTile, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
  extern __shared__ uint8_t smem_raw[];
  let_next_begin();
  const int kv = p.plan.kv_blocks;
  if ((int)blockIdx.x < kv)
    dkdv_block<D, kBf16>(p, tmQStep, tmK, tmV, tmDOStep, align1024(smem_raw), blockIdx.x, kv);
  else
    dq_block<D, kBf16>(p, tmQTile, tmK, tmV, tmDOTile, align1024(smem_raw), blockIdx.x - kv, gridDim.x - kv);
}

template <int D, bool kBf16>
cudaError_t launch_t(const CrossParams& p, const CUtensorMap* m, cudaStream_t st) {
  constexpr int bytes = (int)std::max(std::max(KCfg<D>::kSmem, QCfg<D>::kSmem), kMinSmemOneCtaPerSm);
  constexpr auto kKernel = cross_bwd_kernel<D, kBf16>;
  const cudaError_t e = allow_smem<kKernel>(bytes);
  if (e != cudaSuccess) return e;
  return launch_chained_maps(kKernel, dim3(p.plan.kv_blocks + p.plan.q_blocks), kThreads, bytes, st, p, m[0], m[1],
                             m[2], m[3], m[4], m[5]);
}

}  // namespace

cudaError_t launch_cross_bwd_tc(const CrossParams& p, bool bf16, const CUtensorMap* maps, cudaStream_t st) {
  if (p.d == 128) return bf16 ? launch_t<128, true>(p, maps, st) : launch_t<128, false>(p, maps, st);
  return bf16 ? launch_t<64, true>(p, maps, st) : launch_t<64, false>(p, maps, st);
}

}  // namespace fa
