// C ABI of the attention layers' operators and layer norm: argument checks,
// kernel selection, launch.  The operations, layouts and error rules are
// stated in include/gdn.h.

#include <limits.h>
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "gdn.h"
#include "gdn_internal.cuh"

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int done(cudaError_t e) { return e == cudaSuccess ? GDN_OK : gdn::record_cuda_error(e); }

bool any_null(std::initializer_list<const void*> ptrs) {
  for (const void* x : ptrs)
    if (!x) return true;
  return false;
}

bool all_aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* x : ptrs)
    if (!aligned(x, 16)) return false;
  return true;
}

// Heads, head dimension and dtype of an attention call.
int check_heads(int H, int Hkv, int D, int dtype) {
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (H < 0 || Hkv < 0 || H > 65535 || D < 1 || D > 128) return GDN_ERR_SHAPE;
  if (H > 0 && (Hkv == 0 || H % Hkv)) return GDN_ERR_SHAPE;
  return GDN_OK;
}

bool copy_strides(long long (&dst)[3], const long long (&src)[3]) {
  for (int i = 0; i < 3; ++i) {
    if (src[i] < 0) return false;
    dst[i] = src[i];
  }
  return true;
}

int attn_problem(const gdn_attn_shape* s, float scale, const int* cu_q, const int* cu_k, int nseq,
                 gdn::AttnProblem* p) {
  if (!s) return GDN_ERR_ARG;
  int rc = check_heads(s->H, s->Hkv, s->D, s->dtype);
  if (rc != GDN_OK) return rc;
  if (s->B < 0 || s->Tq < 0 || s->Tk < 0) return GDN_ERR_SHAPE;
  if ((long long)s->B * s->Tq > (1LL << 30) || (long long)s->B * s->Tk > (1LL << 30)) return GDN_ERR_SHAPE;
  if (!(scale > 0.f) || !isfinite(scale)) return GDN_ERR_ARG;
  *p = gdn::AttnProblem{};
  if (!copy_strides(p->qs, s->q_stride) || !copy_strides(p->ks, s->k_stride) ||
      !copy_strides(p->vs, s->v_stride))
    return GDN_ERR_SHAPE;
  if (!cu_q != !cu_k) return GDN_ERR_ARG;
  if (cu_q) {
    if (s->B != 1 || nseq < 0 || nseq > (1 << 30)) return GDN_ERR_SHAPE;
    if (nseq == 0 && (s->Tq > 0 || s->Tk > 0)) return GDN_ERR_SHAPE;
    if (!aligned(cu_q, 4) || !aligned(cu_k, 4)) return GDN_ERR_ALIGN;
    p->cu_q = cu_q, p->cu_k = cu_k, p->nseq = nseq;
  }
  p->B = s->B, p->Tq = s->Tq, p->Tk = s->Tk, p->H = s->H, p->Hkv = s->Hkv, p->D = s->D;
  p->bf16 = s->dtype == GDN_BF16;
  p->scale = scale;
  // A grid has at most 2^31 - 1 CTAs: one per tile of 64 rows (or more) and head,
  // empty packed sequences among them, and one per eight (row, head) pairs.
  const long long T = s->Tq > s->Tk ? s->Tq : s->Tk, tiles = cu_q ? T / 64 + nseq : s->B * ((T + 63) / 64);
  if (tiles * s->H > INT_MAX || (long long)s->B * s->Tq * s->H > 8LL * INT_MAX) return GDN_ERR_SHAPE;
  return GDN_OK;
}

// q, k, v: present where they hold data, aligned to their element
int attn_inputs(gdn::AttnProblem* p, const void* q, const void* k, const void* v) {
  const size_t e = p->bf16 ? 2 : 4;
  if ((p->Tq > 0 && !q) || (p->Tk > 0 && any_null({k, v}))) return GDN_ERR_ARG;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e)) return GDN_ERR_ALIGN;
  p->q = q, p->k = k, p->v = v;
  return GDN_OK;
}

// What the tensor-core kernels would need: whether they run depends on the
// pointers' alignment too, which a shape does not say.
size_t fwd_workspace(const gdn::AttnProblem& p) {
  if (!p.bf16 || p.D % 8 || p.B == 0 || p.Tq == 0 || p.Tk == 0 || p.H == 0) return 0;
  return gdn::attn_tc_fwd_workspace(p);
}

int decode_problem(const gdn_attn_decode_shape* s, gdn::AttnDecodeProblem* p) {
  if (!s) return GDN_ERR_ARG;
  int rc = check_heads(s->H, s->Hkv, s->D, s->dtype);
  if (rc != GDN_OK) return rc;
  if (s->B < 0 || s->T < 0 || s->S < 0) return GDN_ERR_SHAPE;
  if (s->S > (1 << 30) || (s->T > s->S && s->B > 0)) return GDN_ERR_SHAPE;
  if (s->H == 0 && s->Hkv > 0) return GDN_ERR_SHAPE;  // the cache's rows go out with the queries' work
  // every CTA sums the rows' lengths; 8 query rows per CTA in grid.y
  if ((long long)s->B * s->Hkv > 65535 || (s->Hkv > 0 && (long long)s->H / s->Hkv * s->T > 65535LL * 8))
    return GDN_ERR_SHAPE;
  *p = gdn::AttnDecodeProblem{};
  if (!copy_strides(p->kcs, s->kc_stride) || !copy_strides(p->vcs, s->vc_stride)) return GDN_ERR_SHAPE;
  p->B = s->B, p->T = s->T, p->S = s->S, p->H = s->H, p->Hkv = s->Hkv, p->D = s->D;
  p->bf16 = s->dtype == GDN_BF16;
  return GDN_OK;
}

bool decode_empty(const gdn::AttnDecodeProblem& p) { return p.B == 0 || p.T == 0 || p.H == 0; }

int ln_problem(const gdn_norm_shape* s, float eps, gdn::LayerNormProblem* p) {
  if (!s) return GDN_ERR_ARG;
  if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (s->rows < 0 || s->D < 1 || s->D > 65536) return GDN_ERR_SHAPE;
  if (!(eps >= 0.f)) return GDN_ERR_ARG;
  *p = gdn::LayerNormProblem{};
  p->rows = (long)s->rows, p->D = s->D, p->bf16 = s->dtype == GDN_BF16, p->eps = eps;
  return GDN_OK;
}

// Rows that are whole 16-byte vectors are read and written in vectors and start on
// one; other rows, and the fp32 vectors and statistics always, go value by value.
bool ln_aligned(const gdn::LayerNormProblem& p, std::initializer_list<const void*> rows,
                std::initializer_list<const void*> values) {
  const size_t e = p.bf16 ? 2 : 4, a = p.D * e % 16 == 0 ? 16 : e;
  for (const void* x : rows)
    if (!aligned(x, a)) return false;
  for (const void* x : values)
    if (!aligned(x, 4)) return false;
  return true;
}

}  // namespace

extern "C" {

size_t gdn_attn_fwd_workspace(const gdn_attn_shape* shape, int nseq) {
  // as a batch and, where nseq and B allow, as packed sequences: the query has no
  // offsets that would tell the two apart
  gdn::AttnProblem p;
  static const int offsets[2] = {0, 0};  // stands for packed sequences; not read
  size_t need = attn_problem(shape, 1.f, nullptr, nullptr, 0, &p) == GDN_OK ? fwd_workspace(p) : 0;
  if (nseq > 0 && attn_problem(shape, 1.f, offsets, offsets, nseq, &p) == GDN_OK) need = std::max(need, fwd_workspace(p));
  return need;
}

int gdn_attn_fwd(const gdn_attn_shape* shape, const void* q, const void* k, const void* v, float scale,
                 const int* cu_q, const int* cu_k, int nseq, void* o, float* lse, void* ws,
                 size_t ws_bytes, void* stream) {
  gdn::AttnProblem p;
  int rc = attn_problem(shape, scale, cu_q, cu_k, nseq, &p);
  if (rc != GDN_OK) return rc;
  if (p.B == 0 || p.Tq == 0 || p.H == 0) return GDN_OK;
  if (any_null({o, lse})) return GDN_ERR_ARG;
  if ((rc = attn_inputs(&p, q, k, v)) != GDN_OK) return rc;
  if (!all_aligned16({o, lse, ws})) return GDN_ERR_ALIGN;
  const size_t need = fwd_workspace(p);
  if (need > 0 && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
  p.o = o, p.lse = lse, p.ws = ws;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return done(gdn::attn_tc_supported(p) ? gdn::attn_tc_fwd(p, st) : gdn::attn_simt_fwd(p, st));
}

size_t gdn_attn_bwd_workspace(const gdn_attn_shape* shape, int nseq) {
  gdn::AttnProblem p;
  (void)nseq;
  if (attn_problem(shape, 1.f, nullptr, nullptr, 0, &p) != GDN_OK) return 0;
  return gdn::attn_bwd_workspace(p);
}

int gdn_attn_bwd(const gdn_attn_shape* shape, const void* q, const void* k, const void* v, float scale,
                 const int* cu_q, const int* cu_k, int nseq, const void* o, const float* lse,
                 const void* do_, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
  gdn::AttnProblem p;
  int rc = attn_problem(shape, scale, cu_q, cu_k, nseq, &p);
  if (rc != GDN_OK) return rc;
  if (p.B == 0 || (p.Tq == 0 && p.Tk == 0)) return GDN_OK;
  if (p.H == 0) {  // key heads without query heads
    const size_t n = (size_t)p.B * p.Tk * p.Hkv * p.D * (p.bf16 ? 2 : 4);
    if (n == 0) return GDN_OK;
    if (any_null({dk, dv})) return GDN_ERR_ARG;
    if (!all_aligned16({dk, dv})) return GDN_ERR_ALIGN;
    cudaError_t e = cudaMemsetAsync(dk, 0, n, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) e = cudaMemsetAsync(dv, 0, n, static_cast<cudaStream_t>(stream));
    return done(e);
  }
  if ((p.Tq > 0 && any_null({o, lse, do_, dq})) || (p.Tk > 0 && any_null({dk, dv}))) return GDN_ERR_ARG;
  if ((rc = attn_inputs(&p, q, k, v)) != GDN_OK) return rc;
  if (!all_aligned16({o, lse, do_, dq, dk, dv, ws})) return GDN_ERR_ALIGN;
  const size_t need = gdn::attn_bwd_workspace(p);
  if (need > 0 && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
  p.o = const_cast<void*>(o), p.lse = const_cast<float*>(lse), p.do_ = do_;
  p.dq = dq, p.dk = dk, p.dv = dv, p.ws = ws;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return done(gdn::attn_tc_supported(p) ? gdn::attn_tc_bwd(p, st) : gdn::attn_simt_bwd(p, st));
}

int gdn_attn_wait_selftest(int clocks, void* stream) {
  if (clocks < 1 || clocks > (1 << 26)) return GDN_ERR_ARG;
  return done(gdn::attn_wait_selftest(clocks, static_cast<cudaStream_t>(stream)));
}

size_t gdn_attn_decode_workspace(const gdn_attn_decode_shape* shape) {
  gdn::AttnDecodeProblem p;
  if (decode_problem(shape, &p) != GDN_OK || decode_empty(p)) return 0;
  return gdn::attn_decode_workspace(p);
}

int gdn_attn_decode(const gdn_attn_decode_shape* shape, const void* q, const void* k, const void* v,
                    void* k_cache, void* v_cache, const int* lens, float scale, void* o, void* ws,
                    size_t ws_bytes, void* stream) {
  gdn::AttnDecodeProblem p;
  int rc = decode_problem(shape, &p);
  if (rc != GDN_OK) return rc;
  if (!(scale > 0.f) || !isfinite(scale)) return GDN_ERR_ARG;
  if (decode_empty(p)) return GDN_OK;
  if (any_null({q, k, v, k_cache, v_cache, lens, o})) return GDN_ERR_ARG;
  const size_t e = p.bf16 ? 2 : 4;
  if (!all_aligned16({q, k, v, o, ws}) || !aligned(k_cache, e) || !aligned(v_cache, e) || !aligned(lens, 4))
    return GDN_ERR_ALIGN;
  const size_t need = gdn::attn_decode_workspace(p);
  if (need > 0 && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
  p.q = q, p.k = k, p.v = v, p.kc = k_cache, p.vc = v_cache, p.lens = lens;
  p.scale = scale, p.o = o, p.ws = ws;
  return done(gdn::attn_decode(p, static_cast<cudaStream_t>(stream)));
}

int gdn_layer_norm_fwd(const gdn_norm_shape* shape, const void* x, const float* weight, const float* bias,
                       void* y, float* mean, float* rstd, float eps, void* stream) {
  gdn::LayerNormProblem p;
  int rc = ln_problem(shape, eps, &p);
  if (rc != GDN_OK || p.rows == 0) return rc;
  if (any_null({x, weight, y})) return GDN_ERR_ARG;
  if (!ln_aligned(p, {x, y}, {weight, bias, mean, rstd})) return GDN_ERR_ALIGN;
  p.x = x, p.weight = weight, p.bias = bias, p.y = y, p.mean = mean, p.rstd = rstd;
  return done(gdn::layer_norm_fwd(p, static_cast<cudaStream_t>(stream)));
}

size_t gdn_layer_norm_bwd_workspace(const gdn_norm_shape* shape) {
  gdn::LayerNormProblem p;
  if (ln_problem(shape, 0.f, &p) != GDN_OK) return 0;
  return gdn::layer_norm_bwd_workspace(p);
}

int gdn_layer_norm_bwd(const gdn_norm_shape* shape, const void* x, const float* weight, const float* mean,
                       const float* rstd, const void* dy, void* dx, float* dweight, float* dbias, void* ws,
                       size_t ws_bytes, void* stream) {
  gdn::LayerNormProblem p;
  int rc = ln_problem(shape, 0.f, &p);
  if (rc != GDN_OK) return rc;
  if (!dweight) return GDN_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.rows == 0) {
    const size_t n = (size_t)p.D * sizeof(float);
    cudaError_t e = cudaMemsetAsync(dweight, 0, n, st);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, n, st);
    return done(e);
  }
  if (any_null({x, weight, mean, rstd, dy, dx})) return GDN_ERR_ARG;
  if (!ln_aligned(p, {x, dy, dx}, {weight, mean, rstd, dweight, dbias}) || !aligned(ws, 16)) return GDN_ERR_ALIGN;
  const size_t need = gdn::layer_norm_bwd_workspace(p);
  if (!ws || ws_bytes < need) return GDN_ERR_WORKSPACE;
  p.x = x, p.weight = weight, p.mean = const_cast<float*>(mean), p.rstd = const_cast<float*>(rstd);
  p.dy = dy, p.dx = dx, p.dweight = dweight, p.dbias = dbias, p.ws = ws;
  return done(gdn::layer_norm_bwd(p, st));
}

}  // extern "C"
