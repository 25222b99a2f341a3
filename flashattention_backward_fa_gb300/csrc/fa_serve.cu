// C entry points of the norm-and-rotation operators (fa_qk_norm_rope_*) and of
// the 8-bit key/value cache (fa_kv8_*): argument checks and parameters; the
// kernels are in kernels_rope.cu, kernels_kv8.cu and kernels_kv8_attn.cu.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "fa_serve.h"

namespace {

using fa::aligned_to;

bool positive(fa_strides s) { return s.b >= 1 && s.n >= 1 && s.h >= 1; }
bool multiple_of_8(fa_strides s) { return ((s.b | s.n | s.h) & 7) == 0; }

// Sizes and types of the two tensors of the norm-and-rotation calls.
int check_rope(int B, int N, int Hq, int Hk, int d, int rot_dim, int max_pos, fa_dtype dtype, fa_dtype weight_dtype,
               float eps) {
  if (B < 1 || N < 1 || Hq < 1 || Hk < 1 || d < 1) return FA_ERR_INVALID_ARG;
  if (dtype != FA_F32 && dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (weight_dtype != FA_F32 && weight_dtype != dtype) return FA_ERR_UNSUPPORTED;
  if (dtype == FA_F32 ? d > 128 : (d != 64 && d != 128)) return FA_ERR_UNSUPPORTED;
  if (rot_dim < 0 || rot_dim > d || (rot_dim & 1)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_F32 && (rot_dim & 15)) return FA_ERR_UNSUPPORTED;
  if (rot_dim > 0 && max_pos < 1) return FA_ERR_INVALID_ARG;
  if (!(eps > 0.f) || !std::isfinite(eps)) return FA_ERR_INVALID_ARG;
  if ((long long)B * std::max(Hq, Hk) > (1ll << 24) || N > (1 << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Tables, positions and weights (weights are read element by element).
int check_rope_ptrs(const void* q_weight, const void* k_weight, const float* cos_table, const float* sin_table,
                    const int* positions, int rot_dim, fa_dtype weight_dtype) {
  if (rot_dim > 0 && (!cos_table || !sin_table)) return FA_ERR_INVALID_ARG;
  if (!aligned_to(cos_table, 16) || !aligned_to(sin_table, 16) || !aligned_to(positions, 4)) return FA_ERR_ALIGNMENT;
  const int w = weight_dtype == FA_F32 ? 4 : 2;
  if (!aligned_to(q_weight, w) || !aligned_to(k_weight, w)) return FA_ERR_ALIGNMENT;
  return FA_OK;
}

int check_tensor(const void* ptr, fa_strides st, fa_dtype dtype) {
  if (!ptr || !positive(st)) return FA_ERR_INVALID_ARG;
  if (!aligned_to(ptr, 16)) return FA_ERR_ALIGNMENT;
  if (dtype != FA_F32 && !multiple_of_8(st)) return FA_ERR_ALIGNMENT;
  return FA_OK;
}

// The axes of a call's positions into *to.
int check_axes(const fa_rope_axes* a, int rot_dim, fa::RopeAxes* to) {
  if (!a || a->axes < 1 || a->axes > 4 || rot_dim < 2 || !a->positions) return FA_ERR_INVALID_ARG;
  if (a->stride_b < 0 || a->stride_n < 0 || a->stride_axis < 0) return FA_ERR_INVALID_ARG;
  if (!aligned_to(a->positions, 4)) return FA_ERR_ALIGNMENT;
  std::memset(to, 0, sizeof(*to));
  for (int i = 0; a->pair_axis && i < rot_dim / 2; ++i) {
    if (a->pair_axis[i] >= a->axes) return FA_ERR_INVALID_ARG;
    to->pair_axis[i >> 4] |= (uint32_t)a->pair_axis[i] << (2 * (i & 15));
  }
  to->axes = a->axes;
  to->positions = a->positions;
  to->sb = a->stride_b;
  to->sn = a->stride_n;
  to->sa = a->stride_axis;
  return FA_OK;
}

int first_error(std::initializer_list<int> codes) {
  for (int c : codes)
    if (c) return c;
  return FA_OK;
}

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

void fill_rope(fa::RopeParams& p, const void* q, const void* k, const void* q_weight, const void* k_weight,
               const float* cos_table, const float* sin_table, const int* positions, int64_t pos_stride, int B, int N,
               int Hq, int Hk, int d, int rot_dim, int interleaved, int max_pos, fa_dtype weight_dtype, float eps) {
  std::memset(&p, 0, sizeof(p));
  p.q.x = q;
  p.k.x = k;
  p.q.w = q_weight;
  p.k.w = k_weight;
  p.q.H = Hq;
  p.k.H = Hk;
  p.cos = cos_table;
  p.sin = sin_table;
  p.positions = positions;
  p.pos_stride = pos_stride;
  p.B = B;
  p.N = N;
  p.d = d;
  p.rot = rot_dim;
  p.max_pos = max_pos;
  p.neighbours = interleaved ? 1 : 0;
  p.w_f32 = weight_dtype == FA_F32 ? 1 : 0;
  p.eps = eps;
}

// The cache and its sequences. *shift: log2 of the page size.
int check_cache(const fa_kv8_cache* c, const fa_kv8_seqs* s, int* shift) {
  if (!c || !s) return FA_ERR_INVALID_ARG;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !s->block_table || !s->seq_lens) return FA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->H < 1 || s->B < 1 || s->max_pages < 1) return FA_ERR_INVALID_ARG;
  if (s->table_stride < 0 || !positive(c->strides)) return FA_ERR_INVALID_ARG;
  *shift = -1;
  for (int e = 4; e <= 7; ++e)
    if (c->page_size == 1 << e) *shift = e;
  if (*shift < 0) return FA_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  if (c->H > 1024 || s->B > 65535) return FA_ERR_UNSUPPORTED;
  // positions and page offsets within a sequence stay in 31 bits
  if (s->max_pages > (1 << 30) >> *shift) return FA_ERR_UNSUPPORTED;
  // and so do the offsets of a page's tokens
  if (c->strides.n > (1ll << 30) >> *shift) return FA_ERR_UNSUPPORTED;
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || ((c->strides.b | c->strides.n | c->strides.h) & 15))
    return FA_ERR_ALIGNMENT;
  if (!aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4) || !aligned_to(s->block_table, 4) ||
      !aligned_to(s->seq_lens, 4) || !aligned_to(s->new_lens, 4))
    return FA_ERR_ALIGNMENT;
  return FA_OK;
}

void fill_cache(fa::Kv8Cache& to, const fa_kv8_cache* c, const fa_kv8_seqs* s, int shift) {
  to.k = static_cast<uint8_t*>(c->k);
  to.v = static_cast<uint8_t*>(c->v);
  to.k_scale = c->k_scale;
  to.v_scale = c->v_scale;
  to.num_pages = c->num_pages;
  to.page_shift = shift;
  to.H = c->H;
  to.sp = c->strides.b;
  to.sn = c->strides.n;
  to.sh = c->strides.h;
  to.table = s->block_table;
  to.table_stride = s->table_stride;
  to.max_pages = s->max_pages;
  to.seq_lens = s->seq_lens;
  to.new_lens = s->new_lens;
}

int check_16bit(fa_dtype dtype) { return dtype == FA_F16 || dtype == FA_BF16 ? FA_OK : FA_ERR_UNSUPPORTED; }

// Shared by the two append calls; q == null: no norm, no rotation.
int append_run(const fa_kv8_cache* cache, const fa_kv8_seqs* seqs, const void* q, const void* k, const void* v,
               void* q_out, const void* q_weight, const void* k_weight, const float* cos_table,
               const float* sin_table, int T, int Hq, int rot_dim, int interleaved, int max_pos, fa_strides q_strides,
               fa_strides k_strides, fa_strides v_strides, fa_strides q_out_strides, fa_dtype dtype,
               fa_dtype weight_dtype, float eps, bool norm, bool has_axes, const fa_rope_axes* axes, void* stream) {
  int shift = 0;
  int rc = check_cache(cache, seqs, &shift);
  if (rc) return rc;
  if (T < 1) return FA_ERR_INVALID_ARG;
  if ((rc = check_16bit(dtype))) return rc;
  if (T > (1 << 19)) return FA_ERR_UNSUPPORTED;  // the pages that T tokens reach are a grid's y extent
  if (norm && (rc = check_rope(seqs->B, T, Hq, cache->H, cache->d, rot_dim, max_pos, dtype, weight_dtype, eps)))
    return rc;
  if ((rc = first_error({check_tensor(k, k_strides, dtype), check_tensor(v, v_strides, dtype)}))) return rc;
  if (norm && (rc = first_error({check_tensor(q, q_strides, dtype), check_tensor(q_out, q_out_strides, dtype),
                                 check_rope_ptrs(q_weight, k_weight, cos_table, sin_table, nullptr, rot_dim,
                                                 weight_dtype)})))
    return rc;
  fa::Kv8AppendParams p;
  std::memset(&p, 0, sizeof(p));
  if (has_axes && (rc = check_axes(axes, rot_dim, &p.ax))) return rc;
  fill_cache(p.c, cache, seqs, shift);
  p.k = k;
  p.v = v;
  p.k_st = k_strides;
  p.v_st = v_strides;
  p.B = seqs->B;
  p.T = T;
  p.d = cache->d;
  p.pages = (T - 1 + cache->page_size - 1) / cache->page_size + 1;
  if (!norm) p.pages = std::min(p.pages, seqs->max_pages);  // (q's rows need no page)
  if (norm) {
    p.q = q;
    p.q_out = q_out;
    p.q_st = q_strides;
    p.q_out_st = q_out_strides;
    p.Hq = Hq;
    p.q_w = q_weight;
    p.k_w = k_weight;
    p.cos = cos_table;
    p.sin = sin_table;
    p.rot = rot_dim;
    p.max_pos = max_pos;
    p.neighbours = interleaved ? 1 : 0;
    p.w_f32 = weight_dtype == FA_F32 ? 1 : 0;
    p.eps = eps;
  }
  if ((rc = fa::check_device_ptrs({cache->k, cache->v, cache->k_scale, cache->v_scale, seqs->block_table,
                                   seqs->seq_lens, seqs->new_lens, k, v, p.q, p.q_out, p.q_w, p.k_w, p.cos, p.sin,
                                   p.ax.positions})))
    return rc;
  if ((rc = fa::status_ptr(&p.c.status))) return rc;
  return cuda_rc(fa::launch_kv8_append(p, dtype == FA_BF16, static_cast<cudaStream_t>(stream)));
}

// The two norm-and-rotation calls, with one position a token or (has_axes) positions on several axes.
int norm_rope_fwd_run(const void* q, const void* k, void* q_out, void* k_out, const void* q_weight,
                      const void* k_weight, const float* cos_table, const float* sin_table, const int* positions,
                      int64_t pos_stride, int B, int N, int Hq, int Hk, int d, int rot_dim, int interleaved,
                      int max_pos, fa_strides q_strides, fa_strides k_strides, fa_strides q_out_strides,
                      fa_strides k_out_strides, fa_dtype dtype, fa_dtype weight_dtype, float eps, bool has_axes,
                      const fa_rope_axes* axes, void* stream) {
  int rc = check_rope(B, N, Hq, Hk, d, rot_dim, max_pos, dtype, weight_dtype, eps);
  if (rc) return rc;
  if (pos_stride < 0) return FA_ERR_INVALID_ARG;
  if ((rc = first_error({check_tensor(q, q_strides, dtype), check_tensor(k, k_strides, dtype),
                         check_tensor(q_out, q_out_strides, dtype), check_tensor(k_out, k_out_strides, dtype),
                         check_rope_ptrs(q_weight, k_weight, cos_table, sin_table, positions, rot_dim,
                                         weight_dtype)})))
    return rc;
  fa::RopeParams p;
  fill_rope(p, q, k, q_weight, k_weight, cos_table, sin_table, positions, pos_stride, B, N, Hq, Hk, d, rot_dim,
            interleaved, max_pos, weight_dtype, eps);
  if (has_axes && (rc = check_axes(axes, rot_dim, &p.ax))) return rc;
  p.q.out = q_out;
  p.k.out = k_out;
  p.q.x_st = q_strides;
  p.k.x_st = k_strides;
  p.q.out_st = q_out_strides;
  p.k.out_st = k_out_strides;
  if ((rc = fa::check_device_ptrs({q, k, q_out, k_out, q_weight, k_weight, cos_table, sin_table, positions,
                                   p.ax.positions})))
    return rc;
  return cuda_rc(fa::launch_norm_rope_fwd(p, dtype, static_cast<cudaStream_t>(stream)));
}

int norm_rope_bwd_run(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq, void* dk,
                      const void* q_weight, const void* k_weight, void* dq_weight, void* dk_weight,
                      const float* cos_table, const float* sin_table, const int* positions, int64_t pos_stride,
                      int B, int N, int Hq, int Hk, int d, int rot_dim, int interleaved, int max_pos,
                      fa_strides q_strides, fa_strides k_strides, fa_strides dq_out_strides,
                      fa_strides dk_out_strides, fa_strides dq_strides, fa_strides dk_strides, fa_dtype dtype,
                      fa_dtype weight_dtype, float eps, bool has_axes, const fa_rope_axes* axes, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int rc = check_rope(B, N, Hq, Hk, d, rot_dim, max_pos, dtype, weight_dtype, eps);
  if (rc) return rc;
  if (pos_stride < 0) return FA_ERR_INVALID_ARG;
  if (!q_weight != !dq_weight || !k_weight != !dk_weight) return FA_ERR_INVALID_ARG;
  const int w = weight_dtype == FA_F32 ? 4 : 2;
  if (!aligned_to(dq_weight, w) || !aligned_to(dk_weight, w)) return FA_ERR_ALIGNMENT;
  if ((rc = first_error({check_tensor(q, q_strides, dtype), check_tensor(k, k_strides, dtype),
                         check_tensor(dq_out, dq_out_strides, dtype), check_tensor(dk_out, dk_out_strides, dtype),
                         check_tensor(dq, dq_strides, dtype), check_tensor(dk, dk_strides, dtype),
                         check_rope_ptrs(q_weight, k_weight, cos_table, sin_table, positions, rot_dim,
                                         weight_dtype)})))
    return rc;
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < fa_qk_norm_rope_bwd_workspace_size(d))
    return FA_ERR_WORKSPACE;
  fa::RopeParams p;
  fill_rope(p, q, k, q_weight, k_weight, cos_table, sin_table, positions, pos_stride, B, N, Hq, Hk, d, rot_dim,
            interleaved, max_pos, weight_dtype, eps);
  if (has_axes && (rc = check_axes(axes, rot_dim, &p.ax))) return rc;
  p.q.dout = dq_out;
  p.k.dout = dk_out;
  p.q.dx = dq;
  p.k.dx = dk;
  p.q.dw = dq_weight;
  p.k.dw = dk_weight;
  p.q.x_st = q_strides;
  p.k.x_st = k_strides;
  p.q.out_st = dq_out_strides;
  p.k.out_st = dk_out_strides;
  p.q.dx_st = dq_strides;
  p.k.dx_st = dk_strides;
  p.part = static_cast<float*>(workspace);
  if ((rc = fa::check_device_ptrs({q, k, dq_out, dk_out, dq, dk, q_weight, k_weight, dq_weight, dk_weight, cos_table,
                                   sin_table, positions, p.ax.positions, workspace})))
    return rc;
  return cuda_rc(fa::launch_norm_rope_bwd(p, dtype, static_cast<cudaStream_t>(stream)));
}

// Checks that do not depend on pointers, shared with the workspace size.
int check_attn(int B, int T, int Hq, int H, int d, int page_size, int max_pages, int max_seqlen, int window) {
  if (B < 1 || T < 1 || Hq < 1 || H < 1 || max_pages < 1 || max_seqlen < 1) return FA_ERR_INVALID_ARG;
  if (window < 0 || Hq % H != 0) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || page_size < 16 || page_size > 128 || (page_size & (page_size - 1)))
    return FA_ERR_UNSUPPORTED;
  if (B > 65535 || H > 1024 || Hq > (1 << 16) || T > (1 << 19)) return FA_ERR_UNSUPPORTED;
  // rows, and the blocks of a sequence (the grid's x extent), are counted in 31 bits
  if ((long long)T * Hq > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if ((long long)max_pages * page_size > (1 << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa::Kv8AttnPlan attn_plan(int B, int T, int Hq, int H, int d, int page_size, int max_pages, int max_seqlen,
                          int causal, int window) {
  return fa::kv8_attn_plan(B, T, Hq, H, d, (int)std::min<long long>(max_seqlen, (long long)max_pages * page_size),
                           causal, window);
}

}  // namespace

extern "C" {

int fa_qk_norm_rope_fwd(const void* q, const void* k, void* q_out, void* k_out, const void* q_weight,
                        const void* k_weight, const float* cos_table, const float* sin_table, const int* positions,
                        int64_t pos_stride, int B, int N, int Hq, int Hk, int d, int rot_dim, int interleaved,
                        int max_pos, fa_strides q_strides, fa_strides k_strides, fa_strides q_out_strides,
                        fa_strides k_out_strides, fa_dtype dtype, fa_dtype weight_dtype, float eps, void* stream) {
  return norm_rope_fwd_run(q, k, q_out, k_out, q_weight, k_weight, cos_table, sin_table, positions, pos_stride, B, N, Hq, Hk, d, rot_dim,
                           interleaved, max_pos, q_strides, k_strides, q_out_strides, k_out_strides, dtype, weight_dtype,
                           eps, false, nullptr, stream);
}

int fa_qk_norm_rope_axes_fwd(const void* q, const void* k, void* q_out, void* k_out, const void* q_weight,
                             const void* k_weight, const float* cos_table, const float* sin_table,
                             const fa_rope_axes* axes, int B, int N, int Hq, int Hk, int d, int rot_dim,
                             int interleaved, int max_pos, fa_strides q_strides, fa_strides k_strides,
                             fa_strides q_out_strides, fa_strides k_out_strides, fa_dtype dtype, fa_dtype weight_dtype,
                             float eps, void* stream) {
  return norm_rope_fwd_run(q, k, q_out, k_out, q_weight, k_weight, cos_table, sin_table, nullptr, 0, B, N, Hq, Hk, d, rot_dim,
                           interleaved, max_pos, q_strides, k_strides, q_out_strides, k_out_strides, dtype, weight_dtype,
                           eps, true, axes, stream);
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
  return d < 1 || d > 128 ? 0 : ((size_t)fa::rope_bwd_max_blocks() * d * 4 + 255) / 256 * 256;
}

int fa_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq, void* dk,
                        const void* q_weight, const void* k_weight, void* dq_weight, void* dk_weight,
                        const float* cos_table, const float* sin_table, const int* positions, int64_t pos_stride,
                        int B, int N, int Hq, int Hk, int d, int rot_dim, int interleaved, int max_pos,
                        fa_strides q_strides, fa_strides k_strides, fa_strides dq_out_strides,
                        fa_strides dk_out_strides, fa_strides dq_strides, fa_strides dk_strides, fa_dtype dtype,
                        fa_dtype weight_dtype, float eps, void* workspace, size_t workspace_bytes, void* stream) {
  return norm_rope_bwd_run(q, k, dq_out, dk_out, dq, dk, q_weight, k_weight, dq_weight, dk_weight, cos_table, sin_table,
                           positions, pos_stride, B, N, Hq, Hk, d, rot_dim, interleaved, max_pos, q_strides, k_strides,
                           dq_out_strides, dk_out_strides, dq_strides, dk_strides, dtype, weight_dtype, eps, false, nullptr,
                           workspace, workspace_bytes, stream);
}

int fa_qk_norm_rope_axes_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq, void* dk,
                             const void* q_weight, const void* k_weight, void* dq_weight, void* dk_weight,
                             const float* cos_table, const float* sin_table, const fa_rope_axes* axes, int B, int N,
                             int Hq, int Hk, int d, int rot_dim, int interleaved, int max_pos, fa_strides q_strides,
                             fa_strides k_strides, fa_strides dq_out_strides, fa_strides dk_out_strides,
                             fa_strides dq_strides, fa_strides dk_strides, fa_dtype dtype, fa_dtype weight_dtype,
                             float eps, void* workspace, size_t workspace_bytes, void* stream) {
  return norm_rope_bwd_run(q, k, dq_out, dk_out, dq, dk, q_weight, k_weight, dq_weight, dk_weight, cos_table, sin_table,
                           nullptr, 0, B, N, Hq, Hk, d, rot_dim, interleaved, max_pos, q_strides, k_strides,
                           dq_out_strides, dk_out_strides, dq_strides, dk_strides, dtype, weight_dtype, eps, true, axes,
                           workspace, workspace_bytes, stream);
}

int fa_kv8_append(const fa_kv8_cache* cache, const fa_kv8_seqs* seqs, const void* k, const void* v, int T,
                  fa_strides k_strides, fa_strides v_strides, fa_dtype dtype, void* stream) {
  return append_run(cache, seqs, nullptr, k, v, nullptr, nullptr, nullptr, nullptr, nullptr, T, 0, 0, 0, 0, {},
                    k_strides, v_strides, {}, dtype, dtype, 0.f, false, false, nullptr, stream);
}

int fa_kv8_norm_rope_append(const fa_kv8_cache* cache, const fa_kv8_seqs* seqs, const void* q, const void* k,
                            const void* v, void* q_out, const void* q_weight, const void* k_weight,
                            const float* cos_table, const float* sin_table, int T, int Hq, int rot_dim,
                            int interleaved, int max_pos, fa_strides q_strides, fa_strides k_strides,
                            fa_strides v_strides, fa_strides q_out_strides, fa_dtype dtype, fa_dtype weight_dtype,
                            float eps, void* stream) {
  return append_run(cache, seqs, q, k, v, q_out, q_weight, k_weight, cos_table, sin_table, T, Hq, rot_dim,
                    interleaved, max_pos, q_strides, k_strides, v_strides, q_out_strides, dtype, weight_dtype, eps,
                    true, false, nullptr, stream);
}

int fa_kv8_norm_rope_axes_append(const fa_kv8_cache* cache, const fa_kv8_seqs* seqs, const void* q, const void* k,
                                 const void* v, void* q_out, const void* q_weight, const void* k_weight,
                                 const float* cos_table, const float* sin_table, const fa_rope_axes* axes, int T, int Hq,
                                 int rot_dim, int interleaved, int max_pos, fa_strides q_strides, fa_strides k_strides,
                                 fa_strides v_strides, fa_strides q_out_strides, fa_dtype dtype, fa_dtype weight_dtype,
                                 float eps, void* stream) {
  return append_run(cache, seqs, q, k, v, q_out, q_weight, k_weight, cos_table, sin_table, T, Hq, rot_dim,
                    interleaved, max_pos, q_strides, k_strides, v_strides, q_out_strides, dtype, weight_dtype, eps,
                    true, true, axes, stream);
}

size_t fa_kv8_attn_workspace_size(int B, int T, int Hq, int H, int d, int page_size, int max_pages, int max_seqlen,
                                  int causal, int window) {
  if (check_attn(B, T, Hq, H, d, page_size, max_pages, max_seqlen, window)) return 0;
  return attn_plan(B, T, Hq, H, d, page_size, max_pages, max_seqlen, causal, window).workspace;
}

int fa_kv8_attn(const fa_kv8_cache* cache, const fa_kv8_seqs* seqs, const void* q, void* o, float* lse, int T, int Hq,
                int max_seqlen, fa_strides q_strides, fa_strides o_strides, fa_dtype dtype, float scale, int causal,
                int window, const float* alibi_slopes, int64_t alibi_stride_b, void* workspace,
                size_t workspace_bytes, void* stream) {
  int shift = 0;
  int rc = check_cache(cache, seqs, &shift);
  if (rc) return rc;
  if ((rc = check_16bit(dtype))) return rc;
  if ((rc = check_attn(seqs->B, T, Hq, cache->H, cache->d, cache->page_size, seqs->max_pages, max_seqlen, window)))
    return rc;
  if (!std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if ((rc = first_error({check_tensor(q, q_strides, dtype), check_tensor(o, o_strides, dtype)}))) return rc;
  if (!lse) return FA_ERR_INVALID_ARG;
  if (!aligned_to(lse, 4) || !aligned_to(alibi_slopes, 4)) return FA_ERR_ALIGNMENT;
  if (alibi_stride_b < 0) return FA_ERR_INVALID_ARG;
  const fa::Kv8AttnPlan plan = attn_plan(seqs->B, T, Hq, cache->H, cache->d, cache->page_size, seqs->max_pages,
                                         max_seqlen, causal, window);
  if (plan.workspace > 0 && (!workspace || !aligned_to(workspace, 256) || workspace_bytes < plan.workspace))
    return FA_ERR_WORKSPACE;
  if (plan.workspace == 0) workspace = nullptr;  // not used
  fa::Kv8AttnParams p;
  std::memset(&p, 0, sizeof(p));
  fill_cache(p.c, cache, seqs, shift);
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.q_st = q_strides;
  p.o_st = o_strides;
  p.B = seqs->B;
  p.T = T;
  p.Hq = Hq;
  p.G = Hq / cache->H;
  p.d = cache->d;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.causal = causal ? 1 : 0;
  p.window = window;
  p.alibi = alibi_slopes;
  p.alibi_sb = alibi_stride_b;
  p.key_limit = (int)std::min<long long>(max_seqlen, (long long)seqs->max_pages << shift);
  p.chunk = plan.chunk;
  p.splits = plan.splits;
  p.cluster = plan.cluster;
  p.longest_first = plan.longest_first;
  p.row_tiles = plan.row_tiles;
  if (plan.splits > 1 && !plan.cluster) {
    const size_t rows = (size_t)seqs->B * Hq * T * plan.splits;
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = p.part_o + rows * cache->d;
  }
  if ((rc = fa::check_device_ptrs({cache->k, cache->v, cache->k_scale, cache->v_scale, seqs->block_table,
                                   seqs->seq_lens, seqs->new_lens, q, o, lse, alibi_slopes, workspace})))
    return rc;
  if ((rc = fa::status_ptr(&p.c.status))) return rc;
  return cuda_rc(fa::launch_kv8_attn(p, plan, dtype == FA_BF16, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
