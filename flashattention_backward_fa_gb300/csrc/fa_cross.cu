// C entry points of cross attention (fa_cross_*): argument checks, the plan of the
// splits, the workspaces' layouts and the launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "fa_cross.h"

namespace {

using fa::aligned_to;
using fa::CrossParams;
using fa::CrossPlan;

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// The sizes of a call.
int check_shape(const fa_cross_shape* s, fa_dtype dtype) {
  if (!s) return FA_ERR_INVALID_ARG;
  if (s->B < 1 || s->Nq < 1 || s->Nk < 1 || s->Hq < 1 || s->Hk < 1 || s->d < 1 || s->Hq % s->Hk)
    return FA_ERR_INVALID_ARG;
  if (dtype != FA_F32 && dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (dtype == FA_F32 ? s->d > 128 : (s->d != 64 && s->d != 128)) return FA_ERR_UNSUPPORTED;
  // batches and heads are grid extents; the kernels' units of work and their steps are counted in 31 bits
  if (s->B > 65535 || s->Hq > 65535 || s->Nq > (1 << 24) || s->Nk > (1 << 24)) return FA_ERR_UNSUPPORTED;
  if ((long long)s->B * s->Hq > (1 << 24) || (long long)s->Nq * (s->Hq / s->Hk) > (1 << 30)) return FA_ERR_UNSUPPORTED;
  const long long q_tiles = (long long)s->B * s->Hq * ((s->Nq + 31ll) / 32);
  const long long k_tiles = (long long)s->B * s->Hk * ((s->Nk + 31ll) / 32);
  if (q_tiles > (1 << 30) || k_tiles > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if (!aligned_to(s->q_lens, 4) || !aligned_to(s->k_lens, 4)) return FA_ERR_ALIGNMENT;
  return FA_OK;
}

int check_tensor(const void* ptr, fa_strides st, fa_dtype dtype) {
  if (!ptr || st.b < 1 || st.n < 1 || st.h < 1) return FA_ERR_INVALID_ARG;
  if (!aligned_to(ptr, 16)) return FA_ERR_ALIGNMENT;
  if (dtype != FA_F32 && ((st.b | st.n | st.h) & 7)) return FA_ERR_ALIGNMENT;
  return FA_OK;
}

int check_all(std::initializer_list<const void*> ptrs, std::initializer_list<fa_strides> st, fa_dtype dtype) {
  auto s = st.begin();
  for (const void* p : ptrs) {
    const int rc = check_tensor(p, *s++, dtype);
    if (rc) return rc;
  }
  return FA_OK;
}

int check_scale(float scale) { return scale > 0.f && std::isfinite(scale) ? FA_OK : FA_ERR_INVALID_ARG; }

int check_workspace(const void* ws, size_t have, size_t need) {
  return need && (!ws || !aligned_to(ws, 256) || have < need) ? FA_ERR_WORKSPACE : FA_OK;
}

// Query rows of a head in the backward's -L and -D: whole tiles of the kernels that read them (4 queries at least).
int padded_queries(const fa_cross_shape* s, const CrossPlan& c) {
  const int tile = std::max(c.q_tile.queries(), c.step.queries());
  return (s->Nq + tile - 1) / tile * tile;
}

void fill(CrossParams& p, const fa_cross_shape* s, const CrossPlan& plan, float scale) {
  std::memset(&p, 0, sizeof(p));
  p.B = s->B;
  p.Nq = s->Nq;
  p.Nk = s->Nk;
  p.Hq = s->Hq;
  p.Hk = s->Hk;
  p.G = s->Hq / s->Hk;
  p.d = s->d;
  p.q_lens = s->q_lens;
  p.k_lens = s->k_lens;
  p.nq_pad = padded_queries(s, plan);
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.plan = plan;
  p.few_cluster = plan.few_cluster;
}

long long div_up(long long a, long long b) { return (a + b - 1) / b; }

constexpr int kPlaces = 152;  // SMs, one block of the tensor-core kernels each

// Splits of an axis of `steps` for `units` independent pieces of work on `places` that run them round by
// round: the number that makes the rounds' steps fewest, where a unit costs `start` steps more than its
// own and the join `join` in all.
int best_splits(long long units, int steps, int places, int start, int join) {
  const long long most = std::min<long long>(steps, 4 * places / units + 1);
  int best = 1;
  long long least = div_up(units, places) * (steps + start);
  for (int s = 2; s <= most; ++s) {
    const long long cost = div_up(units * s, places) * (div_up(steps, s) + start) + join;
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return (int)div_up(steps, div_up(steps, best));
}

// Whether the forward's kernel of few rows takes a call: always up to 16 rows a key head, and up to 64 where
// the row tiles, which read the keys once each, are few and so are the keys. Measured against the kernel of
// 128-row tiles, us: 16 rows, 8 sequences of 16 heads d = 128 over 8192 keys 92 / 127; 64 rows, 1 x 16 d = 64
// over 500 keys 11.0 / 14.3, over 8192 keys 24 / 25, d = 128 over 16383 keys 70 / 45; 32 rows (256 row tiles),
// 8 x 16 over 8192 keys 129 / 128.
bool few_rows(long long groups, long long rows, int Nk) {
  return groups <= 65535 && (rows <= 16 || (rows <= 64 && groups * div_up(rows, 16) <= 64 && Nk <= 4096));
}

// Its shares of the keys: clusters of two to eight blocks while there are no more blocks than the GPU holds
// twice over and each has 128 keys (32 sequences x 8 heads of up to 4096 keys: 62 us; four times over 64, eight
// times 79); shares through the workspace where clusters of eight leave the GPU empty and their blocks would
// have over 2048 keys (16 heads, d = 64, 8192 keys: cluster 11.5 us, workspace 16.9).
void few_plan(long long units, int Nk, CrossPlan* c) {
  c->k_splits = c->few_cluster = 1;
  while (c->few_cluster < 8 && units * c->few_cluster * 2 <= 608 && c->few_cluster * 2 * 128 <= Nk + 127)
    c->few_cluster *= 2;
  if (units * 8 <= 152 && Nk > 8 * 2048) {
    c->few_cluster = 0;
    c->k_splits = (int)std::min<long long>(304 / units, Nk / 256);
  }
}

// The backward's splits and blocks. Splits: until dK/dV has 128 units or they are down to 16 query steps, dQ 64
// units or 8 key blocks. Blocks: as many as there are units, but not under 16 steps (8 key blocks) each while 128
// blocks remain. Measured, bf16 backward, us (dK/dV splits / blocks, dQ splits / blocks; * what this plan takes):
// 16 heads, 4095 queries over 77 keys, d = 64: *4 / 64, 1 / 128 38; 4 / 32, 1 / 104 57; 32 / 256, 1 / 512 55.
// Two sequences of 16/4 heads: *16 / 128, 1 / 128 56; 8 / 64, 1 / 128 66; 16 / 128, 1 / 512 61; 32 / 256, 1 / 128 65.
// 2 x 16/4 heads, 1024 over 1024: *2 / 128, 1 / 256 93; 1 / 64, 1 / 62 101; 4 / 256, 1 / 256 100.
// 16 heads, 64 queries over 16384 keys: *1 / 128, 4 / 64 136; 1 / 128, 1 / 16 268.
// 4 x 16 heads, 2048 over 512 keys (texts of 512, 227, 453 and 169): *1 / 256, 1 / 512 167 (143); 1 / 152, 1 / 304 166
// (147); 1 / 128, 1 / 256 175 (150); 1 / 152, 1 / 152 178 (158); 2 / 512, 1 / 512 220 (187).
void bwd_plan(const fa_cross_shape* s, long long groups, long long tiles, CrossPlan* c) {
  const int steps = c->step.count(s->Nq, s->Hq / s->Hk), blocks = (int)div_up(s->Nk, 128);
  const long long kv = groups * div_up(s->Nk, 128), q = groups * tiles;
  const auto splits = [](long long units, long long most, int n, int least) {  // of n steps a unit
    const long long want = std::min<long long>(div_up(most, units), std::max(1, n / least));
    return (int)div_up(n, div_up(n, want));
  };
  c->q_splits = splits(kv, 128, steps, 16);
  c->k_splits = splits(q, 64, blocks, 8);
  const auto share = [](long long units, int n, int least) {
    const long long each = std::max(1, least / n);  // units of a block
    return (int)std::max({div_up(units, each), std::min(units, 128ll), div_up(units, fa::kMostUnits)});
  };
  c->kv_blocks = share(kv * c->q_splits, (int)div_up(steps, c->q_splits), 16);
  c->q_blocks = share(q * c->k_splits, (int)div_up(blocks, c->k_splits), 8);
}

CrossPlan plan_of(const fa_cross_shape* s, fa_dtype dtype, bool backward) {
  CrossPlan c;
  const int G = s->Hq / s->Hk;
  c.q_tile = fa::cross_tile(s->Nq, G, 7, 0);
  c.step = fa::cross_tile(s->Nq, G, 6, 2);
  c.q_splits = 1;
  c.few_cluster = 0;
  c.few_sorted = false;
  c.few = !backward && dtype != FA_F32 && few_rows((long long)s->B * s->Hk, (long long)s->Nq * G, s->Nk);
  if (c.few) {
    const long long units = (long long)s->B * s->Hk * div_up((long long)s->Nq * G, 16);
    few_plan(units, s->Nk, &c);
    // By falling lengths where blocks come in several rounds and are long: 32 sequences x 8 heads of up to 4096
    // keys 61.9 -> 54.6 us, 64 x 8 of up to 2048 59.4 -> 50.5; 100 x 8 heads of 64 of up to 1000 keys 28.8 -> 32.5.
    const int shares = std::max(c.few_cluster, c.k_splits);
    c.few_sorted = s->k_lens && s->B > 1 && s->B <= 128 && units * shares > 304 &&
                   (long long)s->Nk * s->d / shares >= 1 << 17;
    return c;
  }
  const long long groups = (long long)s->B * s->Hk, rows = (long long)s->Nq * G;
  if (dtype == FA_F32) {
    c.k_splits = best_splits(groups * div_up(rows, 32), (int)div_up(s->Nk, 64), 304, 1, 3);
    if (backward) c.q_splits = best_splits(groups * div_up(s->Nk, 32), (int)div_up(rows, 64), 152, 1, 3);
    return c;
  }
  const long long tiles = c.q_tile.count(s->Nq, G);
  if (!backward) {
    c.k_splits = best_splits(groups * div_up(tiles, 2), (int)div_up(s->Nk, 128), kPlaces, 1, 4);
  } else {
    bwd_plan(s, groups, tiles, &c);
  }
  return c;
}

// TMA maps: of the rows of a query tile, and of 128 keys.
bool q_map(CUtensorMap* m, const CrossParams& p, const void* base, fa_strides st, fa::CrossTile t, fa_dtype dtype) {
  return fa::make_tensor_map(m, base, dtype == FA_BF16, p.B, p.Nq, p.Hq, p.d, st, t.queries(), t.heads());
}
bool k_map(CUtensorMap* m, const CrossParams& p, const void* base, fa_strides st, fa_dtype dtype) {
  return fa::make_tensor_map(m, base, dtype == FA_BF16, p.B, p.Nk, p.Hk, p.d, st, 128, 1);
}

// Forward: [outputs of the splits | their log-sum-exps], none without splits.
struct FwdLayout {
  size_t lse, total;
};
FwdLayout fwd_layout(const fa_cross_shape* s, const CrossPlan& c) {
  if (c.k_splits == 1) return {0, 0};
  const size_t rows = (size_t)c.k_splits * s->B * s->Nq * s->Hq;
  const size_t lse = round256(rows * s->d * 4);
  return {lse, lse + round256(rows * 4)};
}

// Backward: [-L * log2(e) | -D | fp16: |dO| | its maxima | norms of V | dQ of the splits (before it their D) | dK and
// dV of the splits].
struct BwdLayout {
  size_t nD, dout_norm, dout_most, v_norm, dq, dkdv, total;
};
int v_norms(const fa_cross_shape* s) { return (int)std::min<long long>(fa::kMostNorms, div_up(s->Nk, 128)); }
BwdLayout bwd_layout(const fa_cross_shape* s, const CrossPlan& c, fa_dtype dtype) {
  const size_t vec = round256((size_t)s->B * s->Hq * padded_queries(s, c) * 4);
  BwdLayout w;
  w.nD = vec;
  w.dout_norm = w.dout_most = w.v_norm = w.dq = 2 * vec;
  if (dtype == FA_F16) {
    const size_t heads = (size_t)s->B * s->Hk;
    w.dout_most = w.dout_norm + vec;
    w.v_norm = w.dout_most + round256(heads * 4);
    w.dq = w.v_norm + round256(heads * v_norms(s) * 4);
  }
  w.dkdv = w.dq + (c.k_splits > 1 ? round256((size_t)c.k_splits * s->B * s->Nq * s->Hq * s->d * 4) : 0);
  w.total = w.dkdv + (c.q_splits > 1 ? round256((size_t)c.q_splits * 2 * s->B * s->Nk * s->Hk * s->d * 4) : 0);
  return w;
}

}  // namespace

extern "C" {

size_t fa_cross_fwd_workspace_size(const fa_cross_shape* shape, fa_dtype dtype) {
  return check_shape(shape, dtype) ? 0 : fwd_layout(shape, plan_of(shape, dtype, false)).total;
}

size_t fa_cross_bwd_workspace_size(const fa_cross_shape* shape, fa_dtype dtype) {
  return check_shape(shape, dtype) ? 0 : bwd_layout(shape, plan_of(shape, dtype, true), dtype).total;
}

int fa_cross_fwd(const fa_cross_shape* shape, const void* q, const void* k, const void* v, void* o, float* lse,
                 fa_strides q_strides, fa_strides k_strides, fa_strides v_strides, fa_strides o_strides, fa_dtype dtype,
                 float scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_shape(shape, dtype);
  if (rc || (rc = check_scale(scale))) return rc;
  if ((rc = check_all({q, k, v, o}, {q_strides, k_strides, v_strides, o_strides}, dtype))) return rc;
  if (!lse) return FA_ERR_INVALID_ARG;
  if (!aligned_to(lse, 16)) return FA_ERR_ALIGNMENT;
  const CrossPlan plan = plan_of(shape, dtype, false);
  const FwdLayout w = fwd_layout(shape, plan);
  if ((rc = check_workspace(workspace, workspace_bytes, w.total))) return rc;
  if ((rc = fa::check_device_ptrs({q, k, v, o, lse, shape->q_lens, shape->k_lens, w.total ? workspace : nullptr})))
    return rc;
  CrossParams p;
  fill(p, shape, plan, scale);
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = o;
  p.lse_out = lse;
  p.q_st = q_strides;
  p.k_st = k_strides;
  p.v_st = v_strides;
  p.out_st = o_strides;
  if (w.total) {
    p.part = static_cast<float*>(workspace);
    p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.lse);
  }
  if ((rc = fa::status_ptr(&p.status))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == FA_F32) {
    e = fa::launch_cross_fwd_f32(p, st);
  } else if (plan.few) {
    e = fa::launch_cross_few(p, dtype == FA_BF16, st);
  } else {
    CUtensorMap maps[3];
    if ((rc = fa::bind_device_context())) return rc;
    if (!q_map(&maps[0], p, q, q_strides, plan.q_tile, dtype) || !k_map(&maps[1], p, k, k_strides, dtype) ||
        !k_map(&maps[2], p, v, v_strides, dtype))
      return FA_ERR_CUDA;
    e = fa::launch_cross_fwd_tc(p, dtype == FA_BF16, maps, st);
  }
  if (e == cudaSuccess && plan.k_splits > 1) e = fa::launch_cross_join_fwd(p, dtype, st);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_cross_bwd(const fa_cross_shape* shape, const void* q, const void* k, const void* v, const void* o,
                 const void* dout, const float* lse, void* dq, void* dk, void* dv, fa_strides q_strides,
                 fa_strides k_strides, fa_strides v_strides, fa_strides o_strides, fa_strides dout_strides,
                 fa_strides dq_strides, fa_strides dk_strides, fa_strides dv_strides, fa_dtype dtype, float scale,
                 void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_shape(shape, dtype);
  if (rc || (rc = check_scale(scale))) return rc;
  if ((rc = check_all({q, k, v, o, dout, dq, dk, dv},
                      {q_strides, k_strides, v_strides, o_strides, dout_strides, dq_strides, dk_strides, dv_strides},
                      dtype)))
    return rc;
  if (!lse) return FA_ERR_INVALID_ARG;
  if (!aligned_to(lse, 16)) return FA_ERR_ALIGNMENT;
  const CrossPlan plan = plan_of(shape, dtype, true);
  const BwdLayout w = bwd_layout(shape, plan, dtype);
  if ((rc = check_workspace(workspace, workspace_bytes, w.total))) return rc;
  if ((rc = fa::check_device_ptrs({q, k, v, o, dout, lse, dq, dk, dv, shape->q_lens, shape->k_lens, workspace})))
    return rc;
  CrossParams p;
  fill(p, shape, plan, scale);
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  p.dout = dout;
  p.lse = lse;
  p.out = dq;
  p.dk = dk;
  p.dv = dv;
  p.q_st = q_strides;
  p.k_st = k_strides;
  p.v_st = v_strides;
  p.o_st = o_strides;
  p.do_st = dout_strides;
  p.out_st = dq_strides;
  p.dk_st = dk_strides;
  p.dv_st = dv_strides;
  char* ws = static_cast<char*>(workspace);
  p.nL2 = reinterpret_cast<float*>(ws);
  p.nD = reinterpret_cast<float*>(ws + w.nD);
  p.dout_norm = reinterpret_cast<float*>(ws + w.dout_norm);
  p.dout_most = reinterpret_cast<unsigned int*>(ws + w.dout_most);
  p.v_norm = reinterpret_cast<float*>(ws + w.v_norm);
  p.v_norms = v_norms(shape);
  p.part = reinterpret_cast<float*>(ws + w.dq);
  p.part_kv = reinterpret_cast<float*>(ws + w.dkdv);
  if ((rc = fa::status_ptr(&p.status))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = dtype == FA_F32, bf16 = dtype == FA_BF16;
  CUtensorMap maps[6];
  if (!f32) {
    if ((rc = fa::bind_device_context())) return rc;
    if (!q_map(&maps[0], p, q, q_strides, plan.step, dtype) ||
        !q_map(&maps[1], p, dout, dout_strides, plan.step, dtype) ||
        !q_map(&maps[2], p, q, q_strides, plan.q_tile, dtype) ||
        !q_map(&maps[3], p, dout, dout_strides, plan.q_tile, dtype) || !k_map(&maps[4], p, k, k_strides, dtype) ||
        !k_map(&maps[5], p, v, v_strides, dtype))
      return FA_ERR_CUDA;
  }
  cudaError_t e = f32 ? fa::launch_cross_preprocess_f32(p, st) : fa::launch_cross_dot(p, bf16, maps + 2, st);
  if (e == cudaSuccess) e = f32 ? fa::launch_cross_bwd_f32(p, st) : fa::launch_cross_bwd_tc(p, bf16, maps, st);
  if (e == cudaSuccess && (plan.q_splits > 1 || plan.k_splits > 1)) e = fa::launch_cross_join_bwd(p, dtype, st);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
