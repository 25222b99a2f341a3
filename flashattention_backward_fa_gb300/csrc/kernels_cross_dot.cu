// What cross attention's backward needs of every query row before its products, 16-bit types:
//
//   D_i = sum_j P_ij dP_ij,  P = exp2(S * scale*log2e - L*log2e), S = Q K^T, dP = dO V^T,
//
// stored negated, with -L * log2(e) beside it (-inf and 0 for rows that are not there), and in
// fp16 |dO_i| and the largest of a key head's rows (cross_exponent).
//
// D is rowsum(dO o O) as well, for a read of O and dO, but O is there in 16 bits, and its rounding in
// D meets the keys' mean under P: dS_ij = P_ij (dP_ij - D_i) add up to 0 over j, with D_i off by e they add
// up to -e, and dQ_i is off by scale e sum_j P_ij K_j. Where q and k share large channels, or a few keys make up
// the row, that is more than everything else: error of dQ (bf16, 2-norm, in units of its own rounding) 1.05 to
// 2.4 over 128 to 4096 keys with none to three of four large channels shared, of dK 3 with q eight times as sharp
// over 200 keys. From the scores both are 1.0.
//
// Bound by its two products over long keys (bf16 1x32/8 8192x4096 306 us, 1.80 PFLOP/s), by the starts and ends of
// its units over few (4x16 2048 over texts of 169 to 512 32 us, fp16 2x16/4 4095 over 34 and 77 20, by themselves).
// Backward with it / with rowsum(dO o O): 1620 / 1388 us, 142 / 132, in bf16 55 / 55 for the last.
//
// A persistent grid: one CTA an SM takes units (128 query rows of a group against the keys of one split) in a
// fixed stride, as dQ's blocks do. Warp 0 loads, warps 1 and 3 issue the products into two buffers of S and dP (all
// of TMEM), warps 4-19 sum: a row is on four warps (one TMEM lane), 32 keys of a step each, which add their
// sums up through shared memory. Splits leave theirs in the workspace and a second kernel adds them in order.
#include <algorithm>

#include "fa_cross.h"
#include "fa_serve.h"
#include "rope_common.cuh"

namespace fa {

namespace {

constexpr int kThreads = 640;  // 4 role warps + 4 row-math warpgroups
constexpr int kSums = 4;       // units whose partial sums have places of their own

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kPanel = 128 * 128;
  static constexpr uint32_t kTile = kPanels * kPanel;  // one 128-row tile of Q, dO, K or V
  static constexpr int kRes = D == 64 ? 2 : 1;         // units whose Q and dO are there
  static constexpr int kNS = D == 64 ? 4 : 2;          // K and V ring stages
  static constexpr uint32_t oQ = 0;                    // [kRes] Q, dO
  static constexpr uint32_t oK = kRes * 2 * kTile;
  static constexpr uint32_t oV = oK + kNS * kTile;
  static constexpr uint32_t oBar = oV + kNS * kTile;
  static constexpr int bRes = 0;                       // [kRes] Q, dO of a unit landed
  static constexpr int bResFree = bRes + kRes;         // [kRes] a unit's last reads of them done
  static constexpr int bKFull = bResFree + kRes;
  static constexpr int bKEmpty = bKFull + kNS;
  static constexpr int bVFull = bKEmpty + kNS;
  static constexpr int bVEmpty = bVFull + kNS;
  static constexpr int bSFull = bVEmpty + kNS;         // [2] S and dP landed
  static constexpr int bSEmpty = bSFull + 2;           // [2] the row math has read them
  // [kSums] a unit's partial sums are there (on one barrier a warp that is a unit ahead would be counted for one
  // that is behind)
  static constexpr int bSum = bSEmpty + 2;
  static constexpr int bDrain = bSum + kSums;          // one per MMA-issuing warp
  static constexpr int kBars = bDrain + 2;
  static constexpr uint32_t oTmemSlot = oBar + kBars * 8;
  static constexpr uint32_t oAbort = oTmemSlot + 8;
  static constexpr uint32_t oUnits = oAbort + 8;       // [kMostUnits]
  // partial sums: [kSums][D, |dO|^2][warpgroup][128 rows]
  static constexpr uint32_t oSums = (oUnits + kMostUnits * sizeof(CrossUnit) + 15) & ~15u;
  static constexpr uint32_t kSmem = oSums + kSums * 2 * 4 * 128 * 4 + 1024;  // + slack for 1024-byte alignment
  static_assert(kSmem <= 227u * 1024u, "shared memory budget exceeded");
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    cross_dot_kernel(const __grid_constant__ CrossParams p, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmDO, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  let_next_begin();
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::oAbort);
  auto bar = [&](int idx) -> uint32_t { return sb + C::oBar + 8u * idx; };
  const int mine = (cross_units<1>(p) - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // units of this block
  CrossUnit* const unit = reinterpret_cast<CrossUnit*>(smem + C::oUnits);
  // The first from the i-th on that has blocks to compute (mine: none).
  const auto next_work = [&](int i) {
    while (i < mine && unit[i].blocks == 0) ++i;
    return i;
  };

  if (threadIdx.x == 0) {
    for (int x = 0; x < C::kRes; ++x) {
      mbar_init(bar(C::bRes + x), 1);
      mbar_init(bar(C::bResFree + x), 2);  // S and dP issuers
    }
    for (int s = 0; s < C::kNS; ++s) {
      mbar_init(bar(C::bKFull + s), 1);
      mbar_init(bar(C::bKEmpty + s), 1);
      mbar_init(bar(C::bVFull + s), 1);
      mbar_init(bar(C::bVEmpty + s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(C::bSFull + x), 2);
      mbar_init(bar(C::bSEmpty + x), 512);
      mbar_init(bar(C::bDrain + x), 1);
    }
    for (int x = 0; x < kSums; ++x) mbar_init(bar(C::bSum + x), 512);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + C::oTmemSlot, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmDO);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  wait_for_previous();
  if ((int)threadIdx.x < mine) {
    CrossUnit u;
    cross_unit<1>(p, blockIdx.x + threadIdx.x * gridDim.x, u);
    unit[threadIdx.x] = u;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::oTmemSlot);
  const uint32_t tS = tmem, tdP = tmem + 256;

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (lane == 0) {
      const uint32_t q_bytes = 2u * C::kPanels * 128u << (p.plan.q_tile.q_log + p.plan.q_tile.h_log);
      int kl = 0, issuedK = 0, issuedV = 0;  // units and blocks loaded
      bool ok = true;
      for (int i = next_work(0); ok && i < mine; i = next_work(i + 1)) {
        const CrossUnit& u = unit[i];
        const int x = kl % C::kRes, turn = kl / C::kRes;
        if (turn > 0 && !mbar_wait(bar(C::bResFree + x), (turn - 1) & 1, abort_flag, p.status)) break;
        mbar_arrive_expect_tx(bar(C::bRes + x), q_bytes);
        for (int pn = 0; pn < C::kPanels; ++pn) {
          const uint32_t to = sb + C::oQ + x * 2 * C::kTile + pn * C::kPanel;
          tma_load_4d(to, &tmQ, bar(C::bRes + x), 64 * pn, u.q0[0], u.h0[0], u.b);
          tma_load_4d(to + C::kTile, &tmDO, bar(C::bRes + x), 64 * pn, u.q0[0], u.h0[0], u.b);
        }
        ++kl;
        for (int it = 0; it < u.blocks; ++it) {
          const int row = u.j_begin + 128 * it, s = issuedK % C::kNS;
          const uint32_t phase = ((issuedK / C::kNS) & 1) ^ 1;
          if (!mbar_wait(bar(C::bKEmpty + s), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::bKFull + s), C::kTile);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_4d(sb + C::oK + s * C::kTile + pn * C::kPanel, &tmK, bar(C::bKFull + s), 64 * pn, row, u.hk, u.b);
          ++issuedK;
          if (!mbar_wait(bar(C::bVEmpty + s), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::bVFull + s), C::kTile);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_4d(sb + C::oV + s * C::kTile + pn * C::kPanel, &tmV, bar(C::bVFull + s), 64 * pn, row, u.hk, u.b);
          ++issuedV;
        }
      }
      if (*abort_flag) {
        // Let every copy this thread started land before the CTA exits.
        for (int j = max(0, kl - C::kRes); j < kl; ++j)
          mbar_wait_drain(bar(C::bRes + j % C::kRes), (j / C::kRes) & 1, p.status);
        for (int j = max(0, issuedK - C::kNS); j < issuedK; ++j)
          mbar_wait_drain(bar(C::bKFull + j % C::kNS), (j / C::kNS) & 1, p.status);
        for (int j = max(0, issuedV - C::kNS); j < issuedV; ++j)
          mbar_wait_drain(bar(C::bVFull + j % C::kNS), (j / C::kNS) & 1, p.status);
      }
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------ S (warp 1) / dP (warp 3) MMA issuer -------------------
    // S = Q K^T or dP = dO V^T: M = 128 rows, N = 128 keys, K = d, both K-major.
    const bool isS = warp == 1;
    constexpr uint32_t idS = make_idesc(128, 128, kBf16, false, false);
    const uint64_t dA0 = make_sdesc(sb + C::oQ + (isS ? 0u : C::kTile), 16, 1024),
                   dB0 = make_sdesc(sb + (isS ? C::oK : C::oV), 16, 1024);
    const uint32_t tD = isS ? tS : tdP;
    const int bF = isS ? C::bKFull : C::bVFull, bE = isS ? C::bKEmpty : C::bVEmpty;
    int kl = 0, G = 0;
    bool ok = true;
    for (int i = next_work(0); ok && i < mine; i = next_work(i + 1), ++kl) {
      i = uniform(i);
      const int blocks = uniform(unit[i].blocks), x = kl % C::kRes;
      const uint64_t ad = desc_add(dA0, x * 2 * C::kTile);
      ok = warp_wait<kIssuerPoll>(bar(C::bRes + x), (kl / C::kRes) & 1, abort_flag, p.status);
      for (int it = 0; ok && it < blocks; ++it, ++G) {
        const int bb = G & 1, s = G % C::kNS;
        if (!warp_wait<kIssuerPoll>(bar(bF + s), (G / C::kNS) & 1, abort_flag, p.status) ||
            !warp_wait<kIssuerPoll>(bar(C::bSEmpty + bb), ((G >> 1) & 1) ^ 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t bd = desc_add(dB0, s * C::kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss_w(tD + 128 * bb, desc_add(ad, (kk >> 2) * C::kPanel + (kk & 3) * 32),
                      desc_add(bd, (kk >> 2) * C::kPanel + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
        tc_commit_w(bar(C::bSFull + bb));
        tc_commit_w(bar(bE + s));
      }
      if (!ok) break;
      tc_commit_w(bar(C::bResFree + x));  // this unit's last reads of Q / dO
    }
    // Every MMA this warp issued is complete before the CTA frees TMEM and exits.
    tc_commit_w(bar(C::bDrain + (isS ? 0 : 1)));
    if (lane == 0) mbar_wait_drain(bar(C::bDrain + (isS ? 0 : 1)), 0, p.status);
    __syncwarp();
  } else if (warp >= 4) {
    // --------------------------- row-math warpgroups ---------------------------
    // Warpgroup c takes key columns [32c, 32c + 32) of every step, and a quarter of dO's row.
    const int c = (warp - 4) >> 2, wq = warp & 3;
    const int il = wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const int row_q = il & (p.plan.q_tile.queries() - 1), row_h = il >> p.plan.q_tile.q_log;
    const bool row_in = row_h < p.plan.q_tile.heads();
    const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
    float* const sums = reinterpret_cast<float*>(smem + C::oSums);
    int kl = 0, G = 0;
    bool ok = true;
    // -L of this row of a unit (-inf past the sequence); the next unit's is on its way while one is worked on.
    const auto row_of = [&](int ui) {
      if (ui >= mine || !row_in) return -INFINITY;
      const CrossUnit& u = unit[ui];
      const int i = u.q0[0] + row_q;
      return i < u.nq ? p.lse[((long long)u.b * p.Hq + u.h0[0] + row_h) * p.Nq + i] : -INFINITY;
    };
    float lse = row_of(0), lse_next;
    for (int ui = 0; ok && ui < mine; ++ui, lse = lse_next) {
      const CrossUnit& u = unit[ui];
      const int blocks = u.blocks, left = u.j_end - u.j_begin - 32 * c, i = u.q0[0] + row_q, h = u.h0[0] + row_h;
      const bool real = row_in && i < u.nq;
      lse_next = row_of(ui + 1);
      const float nl = lse == -INFINITY ? lse : -(lse * 1.4426950408889634f);
      const uint64_t l2 = f2_pack(nl, nl);
      float square = 0.f;  // of a quarter of dO's row
      if constexpr (!kBf16) {
        if (real && blocks > 0 && u.split == 0) {
          const __half* g = static_cast<const __half*>(p.dout) + u.b * p.do_st.b + i * p.do_st.n + h * p.do_st.h;
          Raw8<__half> rg[D / 32];
#pragma unroll
          for (int x = 0; x < D / 32; ++x) load8(rg[x], g + c * (D / 4) + 8 * x);
          uint64_t s1 = 0ull;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint64_t y[4];
            rg[x].unpack(y);
#pragma unroll
            for (int e = 0; e < 4; ++e) s1 = f2_fma(y[e], y[e], s1);
          }
          square = f2_sum(s1);
        }
      }
      uint64_t acc = 0ull;
      for (int it = 0; it < blocks; ++it, ++G) {
        const int bb = G & 1;
        const uint32_t allow = bit_range(0, left - 128 * it);
        if (!warp_wait<kRowMathPoll>(bar(C::bSFull + bb), (G >> 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[32], dr[32];
        __syncwarp();
        tmem_ld32(tS + lane_off + 128 * bb + 32 * c, sr);
        tmem_ld32(tdP + lane_off + 128 * bb + 32 * c, dr);
        tmem_ld_wait2(sr, dr);
        tc_fence_before();
        warp_arrive(bar(C::bSEmpty + bb));
        const auto add = [&](auto masked) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), c2, l2), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            float d0 = __uint_as_float(dr[e]), d1 = __uint_as_float(dr[e + 1]);
            if constexpr (decltype(masked)::value) {  // (S and dP of what is not there may be NaN)
              const bool in0 = (allow >> e) & 1u, in1 = (allow >> (e + 1)) & 1u;
              p0 = in0 ? p0 : 0.f;
              p1 = in1 ? p1 : 0.f;
              d0 = in0 ? d0 : 0.f;
              d1 = in1 ? d1 : 0.f;
            }
            acc = f2_fma(f2_pack(p0, p1), f2_pack(d0, d1), acc);
          }
        };
        if (allow == 0xFFFFFFFFu)  // (the same for the whole warp)
          add(std::false_type{});
        else
          add(std::true_type{});
      }
      if (!ok) break;
      float dot = 0.f;
      if (blocks > 0) {
        // The four warpgroups' sums. (A place and its barrier are taken again kSums units on, whose steps begin only
        // when warpgroup 0 has read the S of units that come after this one.)
        float* const at = sums + (kl % kSums) * (2 * 4 * 128) + il;
        at[128 * c] = f2_sum(acc);
        if constexpr (!kBf16) at[4 * 128 + 128 * c] = square;
        warp_arrive(bar(C::bSum + kl % kSums));
        if (c == 0) {
          if (!warp_wait<kRowMathPoll>(bar(C::bSum + kl % kSums), (kl / kSums) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          dot = (at[0] + at[128]) + (at[256] + at[384]);
          if constexpr (!kBf16) square = (at[512] + at[640]) + (at[768] + at[896]);
        }
        ++kl;
      }
      if (c != 0) continue;
      const long long row = ((long long)u.b * p.Hq + h) * p.nq_pad + i;
      if (row_in) {
        const float nd = real ? -dot : 0.f;
        if (p.plan.k_splits > 1)
          p.part[(long long)u.split * p.B * p.Hq * p.nq_pad + row] = nd;
        else
          p.nD[row] = nd;
      }
      if (u.split != 0) continue;
      if (row_in) p.nL2[row] = nl + kCrossPLog2<kBf16>;
      if constexpr (!kBf16) {
        const float norm = real ? sqrtf(square) : 0.f;
        if (row_in) p.dout_norm[row] = norm;
        // (fmaxf passes a NaN over: where dO has one, every gradient that this scales is NaN)
        const unsigned int most = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(norm, 0.f)));
        if (lane == 0 && most != 0u) atomicMax(&p.dout_most[u.b * p.Hk + u.hk], most);
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

// The splits' D in ascending order.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) cross_dot_join_kernel(const __grid_constant__ CrossParams p) {
  let_next_begin();
  wait_for_previous();
  const long long rows = (long long)p.B * p.Hq * p.nq_pad, apart = (long long)gridDim.x * kJoinThreads;
  for (long long row = (long long)blockIdx.x * kJoinThreads + threadIdx.x; row < rows; row += apart) {
    float sum = 0.f;
    for (int s = 0; s < p.plan.k_splits; ++s) sum += p.part[s * rows + row];
    p.nD[row] = sum;
  }
}

// fp16: maxima of |V_j|^2 over even shares of a (batch, key head)'s real keys, one a block, and zeros where the rows'
// largest |dO_i| goes. (A sum that is NaN is passed over: where V has one, every gradient that this scales is NaN.)
template <int D>
__global__ void __launch_bounds__(kJoinThreads) cross_value_norms_kernel(const __grid_constant__ CrossParams p) {
  constexpr int kLanes = D / 8, kApart = kJoinThreads / kLanes, kRowsEach = 4;
  __shared__ float tops[kJoinThreads / 32];
  let_next_begin();
  wait_for_previous();
  const int bh = blockIdx.x / p.v_norms, part = blockIdx.x - bh * p.v_norms, b = bh / p.Hk, h = bh - b * p.Hk;
  const int nk = cross_k_len(p, b), per = (nk + p.v_norms - 1) / p.v_norms, end = min(nk, (part + 1) * per);
  const __half* v = static_cast<const __half*>(p.v) + b * p.v_st.b + h * p.v_st.h + 8 * (threadIdx.x % kLanes);
  float top = 0.f;
  for (int first = part * per; first < end; first += kRowsEach * kApart) {
    Raw8<__half> rv[kRowsEach];
#pragma unroll
    for (int r = 0; r < kRowsEach; ++r) {
      const int j = first + r * kApart + threadIdx.x / kLanes;
      zero8(rv[r]);
      if (j < end) load8(rv[r], v + j * p.v_st.n);
    }
#pragma unroll
    for (int r = 0; r < kRowsEach; ++r) {
      uint64_t x[4], s0 = 0ull;
      rv[r].unpack(x);
#pragma unroll
      for (int e = 0; e < 4; ++e) s0 = f2_fma(x[e], x[e], s0);
      top = fmaxf(top, row_sum<kLanes>(f2_sum(s0)));
    }
  }
#pragma unroll
  for (int o = 16; o >= kLanes; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kJoinThreads / 32; ++w) top = fmaxf(top, tops[w]);
  p.v_norm[blockIdx.x] = top;
  if (part == 0) p.dout_most[bh] = 0u;
}

template <int D, bool kBf16>
cudaError_t launch_t(CrossParams p, const CUtensorMap* m, cudaStream_t st) {
  if constexpr (!kBf16) {
    const dim3 grid((unsigned)((long long)p.B * p.Hk * p.v_norms));
    const cudaError_t e = launch_chained(cross_value_norms_kernel<D>, grid, kJoinThreads, 0, 1, p, st);
    if (e != cudaSuccess) return e;
  }
  constexpr int bytes = (int)std::max(Cfg<D>::kSmem, kMinSmemOneCtaPerSm);
  constexpr auto kKernel = cross_dot_kernel<D, kBf16>;
  cudaError_t e = allow_smem<kKernel>(bytes);
  if (e != cudaSuccess) return e;
  // dQ's splits, each cut into two or four while that gives more blocks, of 8 key blocks at least (backward of 64
  // queries over 16383 keys, 16 heads, 154 -> 144 us). The sums fit where dQ's splits go (4 nq_pad <= Nq d).
  long long units = (long long)p.B * p.Hk * p.plan.q_tile.count(p.Nq, p.G) * p.plan.k_splits;
  if (p.plan.k_splits > 1)
    for (int i = 0; i < 2 && units * 2 <= 152 && p.Nk >= 128 * 8 * 2 * p.plan.k_splits; ++i, units *= 2)
      p.plan.k_splits *= 2;
  const long long blocks = std::max(std::min(units, 152ll), (units + kMostUnits - 1) / kMostUnits);
  e = launch_chained_maps(kKernel, dim3((unsigned)blocks), kThreads, bytes, st, p, m[0], m[1], m[2], m[3]);
  if (e != cudaSuccess || p.plan.k_splits == 1) return e;
  const long long joins = ((long long)p.B * p.Hq * p.nq_pad + kJoinThreads - 1) / kJoinThreads;
  return launch_chained(cross_dot_join_kernel, dim3((unsigned)std::min(joins, 152ll * 8)), kJoinThreads, 0, 1, p, st);
}

}  // namespace

cudaError_t launch_cross_dot(const CrossParams& p, bool bf16, const CUtensorMap* maps, cudaStream_t st) {
  if (p.d == 128) return bf16 ? launch_t<128, true>(p, maps, st) : launch_t<128, false>(p, maps, st);
  return bf16 ? launch_t<64, true>(p, maps, st) : launch_t<64, false>(p, maps, st);
}

}  // namespace fa
