// C ABI of the attention layers' operators, their paged caches and layer norm: argument checks,
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

// Strides of dimensions that have one entry at most do not matter: 0, so that an
// arbitrary one does not decide how rows are read.
void set_strides(long long (&dst)[3], const long long (&src)[3], int n0, int n1, int n2) {
  const int n[3] = {n0, n1, n2};
  for (int i = 0; i < 3; ++i) dst[i] = n[i] > 1 ? src[i] : 0;
}
bool any_negative(std::initializer_list<const long long*> strides) {
  for (const long long* x : strides)
    for (int i = 0; i < 3; ++i)
      if (x[i] < 0) return true;
  return false;
}

// Rotated values, tables and dtype of a call with angles.
int check_rotation(int D, int R, int P, int dtype) {
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (D < 1 || D > 128 || R < 0 || R > D || R % 2 || P < 0) return GDN_ERR_SHAPE;
  return GDN_OK;
}

int rope_problem(const gdn_qk_rope_shape* s, const float* wq, const float* wk, float eps, const float* cos,
                 const float* sin, const int* pos, gdn::QkRopeProblem* p) {
  if (!s) return GDN_ERR_ARG;
  int rc = check_rotation(s->D, s->R, s->P, s->dtype);
  if (rc != GDN_OK) return rc;
  if (s->B < 0 || s->T < 0 || s->H < 0 || s->Hkv < 0 || s->H > 65535 || s->Hkv > 65535) return GDN_ERR_SHAPE;
  const long long tokens = (long long)s->B * s->T;
  if (tokens > (1LL << 30) || tokens * (s->H + s->Hkv) >= (1LL << 40)) return GDN_ERR_SHAPE;
  if (any_negative({s->q_stride, s->k_stride})) return GDN_ERR_SHAPE;
  if (!(eps >= 0.f) || !isfinite(eps) || !wq != !wk || (s->R > 0) != (cos != nullptr) ||
      (s->R > 0) != (sin != nullptr) || (s->R == 0 && (pos || !wq)))
    return GDN_ERR_ARG;
  for (const void* x : {(const void*)wq, (const void*)wk, (const void*)cos, (const void*)sin, (const void*)pos})
    if (!aligned(x, 4)) return GDN_ERR_ALIGN;
  *p = gdn::QkRopeProblem{};
  p->B = s->B, p->T = s->T, p->H = s->H, p->Hkv = s->Hkv, p->D = s->D, p->R = s->R, p->P = s->P;
  p->bf16 = s->dtype == GDN_BF16, p->interleaved = s->interleaved != 0, p->eps = eps;
  set_strides(p->qs, s->q_stride, s->B, s->T, s->H);
  set_strides(p->ks, s->k_stride, s->B, s->T, s->Hkv);
  p->wq = wq, p->wk = wk, p->cos = cos, p->sin = sin, p->pos = pos;
  return GDN_OK;
}

// q and k: present where they hold data, aligned to their element
int rope_inputs(gdn::QkRopeProblem* p, const void* q, const void* k) {
  const size_t e = p->bf16 ? 2 : 4;
  if ((p->H > 0 && !q) || (p->Hkv > 0 && !k)) return GDN_ERR_ARG;
  if (!aligned(q, e) || !aligned(k, e)) return GDN_ERR_ALIGN;
  p->q = q, p->k = k;
  return GDN_OK;
}

bool rope_empty(const gdn::QkRopeProblem& p) { return p.B == 0 || p.T == 0 || p.H + p.Hkv == 0; }

int paged_cache(const gdn_paged_cache* c, gdn::PagedCache* p) {
  if (!c) return GDN_ERR_ARG;
  if (c->format < GDN_CACHE_F32 || c->format > GDN_CACHE_I4) return GDN_ERR_DTYPE;
  const bool i4 = c->format == GDN_CACHE_I4;
  if (c->pages < 0 || c->page < 1 || c->page > (1 << 30) || (c->page & (c->page - 1)) || c->Hkv < 0 ||
      c->Hkv > 65535 || c->D < 1 || c->D > 128 || (i4 && c->D % 32))
    return GDN_ERR_SHAPE;
  if (any_negative({c->k_stride, c->v_stride})) return GDN_ERR_SHAPE;
  if (i4 && any_negative({c->k_scale_stride, c->v_scale_stride})) return GDN_ERR_SHAPE;
  *p = gdn::PagedCache{};
  p->pages = c->pages, p->page = c->page, p->Hkv = c->Hkv, p->D = c->D, p->format = c->format;
  set_strides(p->ks, c->k_stride, c->pages, c->page, c->Hkv);
  set_strides(p->vs, c->v_stride, c->pages, c->page, c->Hkv);
  if (c->pages > 0 && c->Hkv > 0 && (any_null({c->k, c->v}) || (i4 && any_null({c->k_scale, c->v_scale}))))
    return GDN_ERR_ARG;
  p->k = c->k, p->v = c->v;
  const size_t e = i4 ? 16 : c->format == GDN_CACHE_BF16 ? 2 : 4;
  if (!aligned(c->k, e) || !aligned(c->v, e)) return GDN_ERR_ALIGN;
  if (!i4) return GDN_OK;
  set_strides(p->kss, c->k_scale_stride, c->pages, c->page, c->Hkv);
  set_strides(p->vss, c->v_scale_stride, c->pages, c->page, c->Hkv);
  if (!all_aligned16({c->k_scale, c->v_scale})) return GDN_ERR_ALIGN;
  for (int i = 0; i < 3; ++i)
    if (p->ks[i] % 16 || p->vs[i] % 16 || p->kss[i] % (c->D / 32) || p->vss[i] % (c->D / 32)) return GDN_ERR_ALIGN;
  p->k_scale = c->k_scale, p->v_scale = c->v_scale;
  return GDN_OK;
}

// dtype against a cache's format: the same, or 4 bits
int check_format(const gdn::PagedCache& c, int dtype) {
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
  return c.format == GDN_CACHE_I4 || c.format == (dtype == GDN_BF16 ? GDN_CACHE_BF16 : GDN_CACHE_F32) ? GDN_OK
                                                                                                     : GDN_ERR_DTYPE;
}

int page_table(const gdn::PagedCache& c, const int* table, int rows, int max_pages, long long stride,
               gdn::PageTable* t) {
  if (rows < 0 || rows > (1 << 30) || max_pages < 0 || (long long)max_pages * c.page > (1LL << 30) || stride < 0)
    return GDN_ERR_SHAPE;
  if (!aligned(table, 4)) return GDN_ERR_ALIGN;
  if (!table && rows > 0 && max_pages > 0) return GDN_ERR_ARG;
  t->table = table, t->rows = rows, t->max_pages = max_pages, t->stride = stride;
  return GDN_OK;
}

int append_problem(const gdn_kv_append_shape* s, const gdn_paged_cache* cache, const int* table, const int* cu,
                   gdn::KvAppendProblem* p, gdn::PagedCache* c) {
  if (!s) return GDN_ERR_ARG;
  int rc = paged_cache(cache, c);
  if (rc != GDN_OK) return rc;
  if ((rc = check_format(*c, s->dtype)) != GDN_OK) return rc;
  if ((rc = check_rotation(c->D, s->R, s->P, s->dtype)) != GDN_OK) return rc;
  if (s->B < 0 || s->T < 0 || s->H < 0 || s->H > 65535 || (long long)s->B * s->T > (1LL << 30)) return GDN_ERR_SHAPE;
  if (any_negative({s->q_stride, s->k_stride, s->v_stride})) return GDN_ERR_SHAPE;
  if (cu ? s->B != 1 : s->rows != s->B) return GDN_ERR_SHAPE;
  *p = gdn::KvAppendProblem{};
  if ((rc = page_table(*c, table, s->rows, s->max_pages, s->table_stride, &p->pt)) != GDN_OK) return rc;
  p->B = s->B, p->T = s->T, p->H = s->H, p->R = s->R, p->P = s->P;
  p->bf16 = s->dtype == GDN_BF16, p->interleaved = s->interleaved != 0;
  set_strides(p->qs, s->q_stride, s->B, s->T, s->H);
  set_strides(p->ks, s->k_stride, s->B, s->T, c->Hkv);
  set_strides(p->vs, s->v_stride, s->B, s->T, c->Hkv);
  return GDN_OK;
}

int paged_problem(const gdn_attn_paged_shape* s, const gdn_paged_cache* cache, gdn::AttnPagedProblem* p,
                  gdn::PagedCache* c) {
  if (!s) return GDN_ERR_ARG;
  int rc = paged_cache(cache, c);
  if (rc != GDN_OK) return rc;
  if ((rc = check_format(*c, s->dtype)) != GDN_OK) return rc;
  if ((rc = check_heads(s->H, c->Hkv, c->D, s->dtype)) != GDN_OK) return rc;
  if (s->B < 0 || s->T < 0 || (s->H == 0 && c->Hkv > 0)) return GDN_ERR_SHAPE;
  if ((long long)s->B * c->Hkv > 65535 || (c->Hkv > 0 && (long long)s->H / c->Hkv * s->T > 65535LL * 8))
    return GDN_ERR_SHAPE;
  *p = gdn::AttnPagedProblem{};
  if ((rc = page_table(*c, nullptr, 0, s->max_pages, s->table_stride, &p->pt)) != GDN_OK) return rc;
  p->pt.rows = s->B;
  p->B = s->B, p->T = s->T, p->H = s->H, p->bf16 = s->dtype == GDN_BF16;
  return GDN_OK;
}

bool paged_empty(const gdn::AttnPagedProblem& p) { return p.B == 0 || p.T == 0 || p.H == 0; }

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

int gdn_qk_norm_rope_fwd(const gdn_qk_rope_shape* shape, const void* q, const void* k, const float* wq,
                         const float* wk, float eps, const float* cos, const float* sin, const int* positions,
                         void* qo, void* ko, void* stream) {
  gdn::QkRopeProblem p;
  int rc = rope_problem(shape, wq, wk, eps, cos, sin, positions, &p);
  if (rc != GDN_OK || rope_empty(p)) return rc;
  if ((rc = rope_inputs(&p, q, k)) != GDN_OK) return rc;
  if ((p.H > 0 && !qo) || (p.Hkv > 0 && !ko)) return GDN_ERR_ARG;
  if (!all_aligned16({qo, ko})) return GDN_ERR_ALIGN;
  p.qo = qo, p.ko = ko;
  return done(gdn::qk_rope_fwd(p, static_cast<cudaStream_t>(stream)));
}

size_t gdn_qk_norm_rope_bwd_workspace(const gdn_qk_rope_shape* shape) {
  if (!shape || shape->D < 1 || shape->D > 128) return 0;
  gdn::QkRopeProblem p;
  p.D = shape->D;
  return gdn::qk_rope_bwd_workspace(p);
}

int gdn_qk_norm_rope_bwd(const gdn_qk_rope_shape* shape, const void* q, const void* k, const float* wq,
                         const float* wk, float eps, const float* cos, const float* sin, const int* positions,
                         const void* dqo, const void* dko, void* dq, void* dk, float* dwq, float* dwk, void* ws,
                         size_t ws_bytes, void* stream) {
  gdn::QkRopeProblem p;
  int rc = rope_problem(shape, wq, wk, eps, cos, sin, positions, &p);
  if (rc != GDN_OK) return rc;
  if (wq && any_null({dwq, dwk})) return GDN_ERR_ARG;
  if (!aligned(dwq, 4) || !aligned(dwk, 4)) return GDN_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rope_empty(p)) {
    if (!wq) return GDN_OK;
    cudaError_t e = cudaMemsetAsync(dwq, 0, p.D * sizeof(float), st);
    if (e == cudaSuccess) e = cudaMemsetAsync(dwk, 0, p.D * sizeof(float), st);
    return done(e);
  }
  if ((rc = rope_inputs(&p, q, k)) != GDN_OK) return rc;
  if ((p.H > 0 && any_null({dqo, dq})) || (p.Hkv > 0 && any_null({dko, dk}))) return GDN_ERR_ARG;
  if (!all_aligned16({dqo, dko, dq, dk, ws})) return GDN_ERR_ALIGN;
  if (wq && (!ws || ws_bytes < gdn::qk_rope_bwd_workspace(p))) return GDN_ERR_WORKSPACE;
  p.dqo = dqo, p.dko = dko, p.dq = dq, p.dk = dk, p.dwq = dwq, p.dwk = dwk, p.ws = ws;
  return done(gdn::qk_rope_bwd(p, st));
}

int gdn_kv_append(const gdn_kv_append_shape* shape, const gdn_paged_cache* cache, const void* k, const void* v,
                  const void* q, const float* cos, const float* sin, const int* table, const int* lens,
                  const int* cu_seqlens, void* qo, void* stream) {
  gdn::KvAppendProblem p;
  gdn::PagedCache c;
  int rc = append_problem(shape, cache, table, cu_seqlens, &p, &c);
  if (rc != GDN_OK) return rc;
  if ((p.R > 0) != (cos != nullptr) || (p.R > 0) != (sin != nullptr)) return GDN_ERR_ARG;
  if (p.B == 0 || p.T == 0 || p.H + c.Hkv == 0) return GDN_OK;
  if ((c.Hkv > 0 && any_null({k, v})) || (p.H > 0 && any_null({q, qo})) || (p.pt.rows > 0 && !lens)) return GDN_ERR_ARG;
  const size_t e = p.bf16 ? 2 : 4;
  for (const void* x : {k, v, q})
    if (!aligned(x, e)) return GDN_ERR_ALIGN;
  if (!aligned(cos, 4) || !aligned(sin, 4) || !aligned(lens, 4) || !aligned(cu_seqlens, 4) || !aligned(qo, 16))
    return GDN_ERR_ALIGN;
  p.k = k, p.v = v, p.q = q, p.cos = cos, p.sin = sin, p.lens = lens, p.cu = cu_seqlens, p.qo = qo;
  return done(gdn::kv_append(p, c, static_cast<cudaStream_t>(stream)));
}

int gdn_kv_gather(const gdn_paged_cache* cache, const int* table, int rows, int max_pages, long long table_stride,
                  const int* cu_seqlens, int total, int dtype, void* k, void* v, void* stream) {
  gdn::KvGatherProblem p;
  gdn::PagedCache c;
  int rc = paged_cache(cache, &c);
  if (rc != GDN_OK) return rc;
  if ((rc = check_format(c, dtype)) != GDN_OK) return rc;
  if (total < 0 || total > (1 << 30)) return GDN_ERR_SHAPE;
  if ((rc = page_table(c, table, rows, max_pages, table_stride, &p.pt)) != GDN_OK) return rc;
  if (total == 0 || c.Hkv == 0) return GDN_OK;
  if (any_null({cu_seqlens, k, v})) return GDN_ERR_ARG;
  if (!aligned(cu_seqlens, 4) || !all_aligned16({k, v})) return GDN_ERR_ALIGN;
  p.total = total, p.bf16 = dtype == GDN_BF16, p.cu = cu_seqlens, p.k = k, p.v = v;
  return done(gdn::kv_gather(p, c, static_cast<cudaStream_t>(stream)));
}

size_t gdn_attn_paged_workspace(const gdn_attn_paged_shape* shape, const gdn_paged_cache* cache) {
  gdn::AttnPagedProblem p;
  gdn::PagedCache c;
  if (paged_problem(shape, cache, &p, &c) != GDN_OK || paged_empty(p)) return 0;
  return gdn::attn_paged_workspace(p, c);
}

int gdn_attn_paged(const gdn_attn_paged_shape* shape, const gdn_paged_cache* cache, const void* q,
                   const int* table, const int* lens, float scale, void* o, void* ws, size_t ws_bytes,
                   void* stream) {
  gdn::AttnPagedProblem p;
  gdn::PagedCache c;
  int rc = paged_problem(shape, cache, &p, &c);
  if (rc != GDN_OK) return rc;
  if (!(scale > 0.f) || !isfinite(scale)) return GDN_ERR_ARG;
  if (paged_empty(p)) return GDN_OK;
  if (any_null({q, lens, o}) || (!table && p.pt.max_pages > 0)) return GDN_ERR_ARG;
  if (!all_aligned16({q, o, ws}) || !aligned(lens, 4) || !aligned(table, 4)) return GDN_ERR_ALIGN;
  const size_t need = gdn::attn_paged_workspace(p, c);
  if (need > 0 && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
  p.pt.table = table;
  p.q = q, p.lens = lens, p.scale = scale, p.o = o, p.ws = ws;
  return done(gdn::attn_paged(p, c, static_cast<cudaStream_t>(stream)));
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
