// C entry points of cross attention (fa_cross_*): argument checks, the plan of the
// splits, the workspaces' layouts and the launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "fa_cross.h"

namespace fa {

CrossPlan cross_plan(int B, int Nq, int Nk, int Hq, int Hk, int d, int dtype) {
  CrossPlan c;
  const long long q_units = (long long)B * Hq * ((Nq + 31) / 32), k_units = (long long)B * Hk * ((Nk + 31) / 32);
  cross_splits(Nk, 64, q_units, 304, 2, &c.k_splits, &c.k_chunk);
  cross_splits((Nq + 63) / 64 * (Hq / Hk), 1, k_units, 304, 2, &c.q_splits, &c.q_chunk);
  return c;
}

}  // namespace fa

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
  // batches and heads are grid extents; rows of a head, and query steps of a group, are counted in 31 bits
  if (s->B > 65535 || s->Hq > 65535 || s->Nq > (1 << 24) || s->Nk > (1 << 24)) return FA_ERR_UNSUPPORTED;
  if ((long long)s->B * s->Hq > (1 << 24) || (long long)s->Nq * (s->Hq / s->Hk) > (1 << 30)) return FA_ERR_UNSUPPORTED;
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
  p.nq_pad = (s->Nq + 127) & ~127;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.plan = plan;
}

CrossPlan plan_of(const fa_cross_shape* s, fa_dtype dtype) {
  return fa::cross_plan(s->B, s->Nq, s->Nk, s->Hq, s->Hk, s->d, dtype);
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

// Backward: [-L * log2(e) | -D | dQ of the splits | dK and dV of the splits].
struct BwdLayout {
  size_t nD, dq, dkdv, total;
};
BwdLayout bwd_layout(const fa_cross_shape* s, const CrossPlan& c) {
  const size_t vec = round256((size_t)s->B * s->Hq * (((size_t)s->Nq + 127) & ~size_t(127)) * 4);
  BwdLayout w;
  w.nD = vec;
  w.dq = 2 * vec;
  w.dkdv = w.dq + (c.k_splits > 1 ? round256((size_t)c.k_splits * s->B * s->Nq * s->Hq * s->d * 4) : 0);
  w.total = w.dkdv + (c.q_splits > 1 ? round256((size_t)c.q_splits * 2 * s->B * s->Nk * s->Hk * s->d * 4) : 0);
  return w;
}

}  // namespace

extern "C" {

size_t fa_cross_fwd_workspace_size(const fa_cross_shape* shape, fa_dtype dtype) {
  return check_shape(shape, dtype) ? 0 : fwd_layout(shape, plan_of(shape, dtype)).total;
}

size_t fa_cross_bwd_workspace_size(const fa_cross_shape* shape, fa_dtype dtype) {
  return check_shape(shape, dtype) ? 0 : bwd_layout(shape, plan_of(shape, dtype)).total;
}

int fa_cross_fwd(const fa_cross_shape* shape, const void* q, const void* k, const void* v, void* o, float* lse,
                 fa_strides q_strides, fa_strides k_strides, fa_strides v_strides, fa_strides o_strides, fa_dtype dtype,
                 float scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_shape(shape, dtype);
  if (rc || (rc = check_scale(scale))) return rc;
  if ((rc = check_all({q, k, v, o}, {q_strides, k_strides, v_strides, o_strides}, dtype))) return rc;
  if (!lse) return FA_ERR_INVALID_ARG;
  if (!aligned_to(lse, 16)) return FA_ERR_ALIGNMENT;
  const CrossPlan plan = plan_of(shape, dtype);
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
  cudaError_t e = fa::launch_cross_fwd_simple(p, dtype, st);
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
  const CrossPlan plan = plan_of(shape, dtype);
  const BwdLayout w = bwd_layout(shape, plan);
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
  p.part = reinterpret_cast<float*>(ws + w.dq);
  p.part_kv = reinterpret_cast<float*>(ws + w.dkdv);
  if ((rc = fa::status_ptr(&p.status))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_cross_preprocess(p, dtype, st);
  if (e == cudaSuccess) e = fa::launch_cross_dkdv_simple(p, dtype, st);
  if (e == cudaSuccess && plan.q_splits > 1) e = fa::launch_cross_join_dkdv(p, dtype, st);
  if (e == cudaSuccess) e = fa::launch_cross_dq_simple(p, dtype, st);
  if (e == cudaSuccess && plan.k_splits > 1) e = fa::launch_cross_join_dq(p, dtype, st);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
