// RMS norm of every query and key head and rotation by position, in one pass,
// forward and backward.
//
// A row x of D values (one head of one token), weight w, angles of the token's
// position (rope.cuh):
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w,  y = n rotated
//   g = dy rotated back,  u = g w,  dx = r (u - x r mean(u x r)),  dw = sum_rows g x r
// Without weights n = x, and without angles y = n.
//
// Bound by memory: 2 e bytes per value forward, 3 e backward (x is read again,
// nothing is saved).  The heads of q and those of k are two problems that run side by
// side, each with a share of the CTAs by its heads, so that a lane's weights and its
// columns' sums of dw stay in registers for all of its rows.  A warp takes a token
// (where there are few, a part of its heads) and walks the heads, so that the angles
// are read once per token and lane; a row stays in the registers of its LR lanes,
// the next ones on their way.
//
// dw: the lanes' sums are added per CTA and, by a second kernel, over the CTAs, each
// in a fixed order.
//
// Measured, 16 x 2048 tokens, 8 + 8 heads of 128, bf16: forward 49 us (268 MB, 5.4
// TB/s), backward 82 us (403 MB, 4.9 TB/s) and 4 us for the sums.

#include "rope.cuh"

namespace gdn {

cudaError_t qk_rope_read_and_clear_status(int* status) { return tc::read_and_clear_file_status(status); }

namespace {

using namespace rope;
using tc::sm_count;

constexpr int kThreads = 256, kWarps = kThreads / 32;
// CTAs per SM.  The forward, by measurement at 16 x 2048 tokens, 8 + 8 heads of 128: with
// one pass loaded ahead and 80 registers 48 us; two CTAs and one to three passes ahead
// 55, four CTAs 56.  The backward's 128 registers allow two.
constexpr int kPerSmFwd = 3, kPerSmBwd = 2;

// The heads of q, or those of k.
struct Side {
  const void *x, *dy;
  void *y, *dx;  // contiguous, as dy
  const float* w;
  float* dw;
  long long st[3];
  int H, chunk, parts;  // a warp's job: `chunk` heads of a token, `parts` jobs to a token
};

struct Args {
  Side side[2];
  int T, D, R, P, ctas0;  // the first ctas0 CTAs are q's
  uint32_t tokens;
  float eps, inv_d;
  const float *cos, *sin;
  const int* pos;
  float* partial;  // [ctas][D] sums of dw
};

template <int V, int NP, int LR, bool IL>
struct Lane {
  static constexpr int GW = 32 / LR;  // rows of a warp at once
  Slot<V> slot[NP];
  int grp;
  __device__ __forceinline__ explicit Lane(const Args& a) {
    grp = (threadIdx.x & 31) / LR;
#pragma unroll
    for (int i = 0; i < NP; ++i) slot[i].template set<IL>(first(i), a.D, a.R);
  }
  __device__ __forceinline__ static int first(int i) { return ((threadIdx.x & 31) % LR + i * LR) * V; }

  // The angles of a position, the same for all lanes of the warp; false: it has none.
  __device__ __forceinline__ bool angles(const Args& a, int n, Angles<V> (&g)[NP]) const {
    if (a.R == 0) return true;
    const bool ok = n >= 0 && n < a.P;
    if (n >= a.P && (threadIdx.x & 31) == 0) atomicExch(&tc::g_file_status, GDN_ERR_SEQLENS);
    if (!ok) return false;
#pragma unroll
    for (int i = 0; i < NP; ++i) g[i].set(a.cos, a.sin, (long long)n * (a.R / 2), first(i), slot[i].rot);
    return true;
  }
  // The sum over a row of what its lanes have.
  __device__ __forceinline__ float sum(Num<V> x) const { return row_sum<LR>(V == 1 || slot[0].in ? total(x) : 0.f); }
};

// A warp's way through its jobs: passes of GW heads, loaded ahead across the ends of
// jobs.
struct Pass {
  uint32_t tok, h, h1;  // heads h .. of a token, those below h1; no token: no pass
  int pos;
  bool fresh;           // the first of its job
};
struct Cursor {
  Pass p;
  uint32_t job, end;  // the job's passes end at head `end`
  long long at;       // the token's offset in x
  __device__ __forceinline__ void start(const Args& a, const Side& s, uint32_t j) {
    job = j;
    uint32_t part = 0;
    p.tok = j;
    if (s.parts > 1) p.tok = j / s.parts, part = j % s.parts;
    p.h = part * s.chunk, end = p.h + s.chunk, p.h1 = 0, p.fresh = true, p.pos = 0, at = 0;
    if (p.tok >= a.tokens) return;
    p.h1 = min(end, (uint32_t)s.H);
    const uint32_t b = p.tok / a.T, t = p.tok % a.T;
    p.pos = a.R && a.pos ? a.pos[p.tok] : (int)t;
    at = b * s.st[0] + t * s.st[1];
  }
  template <int GW>
  __device__ __forceinline__ void next(const Args& a, const Side& s, uint32_t stride) {
    p.h += GW, p.fresh = false;
    if (p.h >= end && p.tok < a.tokens) start(a, s, job + stride);
  }
};

// This CTA's side, its index and number among that side's CTAs.
__device__ __forceinline__ Side side_of(const Args& a, uint32_t& cta, uint32_t& ctas) {
  const bool k = blockIdx.x >= a.ctas0;
  cta = k ? blockIdx.x - a.ctas0 : blockIdx.x;
  ctas = k ? gridDim.x - a.ctas0 : a.ctas0;
  return k ? a.side[1] : a.side[0];
}

template <typename T, int V, int NP, int LR, bool IL, bool NORM>
__global__ void __launch_bounds__(kThreads, kPerSmFwd) qk_rope_fwd_kernel(Args a) {
  using L = Lane<V, NP, LR, IL>;
  using N = Num<V>;
  constexpr int GW = L::GW, M = kNums<V>;
  const L lane(a);
  uint32_t cta, ctas;
  const Side s = side_of(a, cta, ctas);
  __shared__ __align__(16) float w[128];
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < a.D; i += kThreads) w[i] = s.w[i];
    __syncthreads();
  }
  const uint32_t stride = ctas * kWarps;
  Cursor f;
  f.start(a, s, cta * kWarps + (threadIdx.x >> 5));
  Raw<T, V> next[NP];
  auto fetch = [&] {
    if (f.p.tok < a.tokens) {  // heads past the last: the last again
      const T* x = static_cast<const T*>(s.x) + f.at + min(f.p.h + lane.grp, f.p.h1 - 1) * s.st[2];
#pragma unroll
      for (int i = 0; i < NP; ++i) next[i] = load(x, lane.slot[i]);
    }
  };
  fetch();
  Angles<V> g[NP];
  bool ok = true;
  while (f.p.tok < a.tokens) {
    const Pass c = f.p;
    if (c.fresh) ok = lane.angles(a, c.pos, g);
    N xa[NP][M], xb[NP][M];
#pragma unroll
    for (int i = 0; i < NP; ++i) widen<IL>(next[i], xa[i], xb[i]);
    f.next<GW>(a, s, stride);
    fetch();
    if constexpr (NORM) {
      N ss = splat<V>(0.f);
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < M; ++e) ss = fma(xa[i][e], xa[i][e], fma(xb[i][e], xb[i][e], ss));
      const N r = splat<V>(rsqrtf(lane.sum(ss) * a.inv_d + a.eps));
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        N wa[M], wb[M];
        widen<IL>(load<float, V>(w, lane.slot[i]), wa, wb);
#pragma unroll
        for (int e = 0; e < M; ++e) xa[i][e] = mul(mul(xa[i][e], r), wa[e]), xb[i][e] = mul(mul(xb[i][e], r), wb[e]);
      }
    }
    const uint32_t h = c.h + lane.grp;
    if (h < c.h1) {
      T* y = static_cast<T*>(s.y) + ((uint64_t)c.tok * s.H + h) * a.D;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (lane.slot[i].rot) NORM ? g[i].turn_fused(xa[i], xb[i]) : g[i].turn(xa[i], xb[i]);
        if (!ok) {
#pragma unroll
          for (int e = 0; e < M; ++e) xa[i][e] = xb[i][e] = splat<V>(0.f);
        }
        store<IL>(y, lane.slot[i], xa[i], xb[i]);
      }
    }
  }
}

template <typename T, int V, int NP, int LR, bool IL, bool NORM>
__global__ void __launch_bounds__(kThreads, kPerSmBwd) qk_rope_bwd_kernel(Args a) {
  using L = Lane<V, NP, LR, IL>;
  using N = Num<V>;
  constexpr int GW = L::GW, U = V == 4 ? 2 : 1, M = kNums<V>;
  extern __shared__ __align__(16) float sums[];  // NORM: [kWarps * GW][D]
  // The weights lie in shared memory: with them in registers, what is loaded ahead
  // was spilled, and so waited for at once.
  __shared__ __align__(16) float w[128];
  tc::grid_dep_launch();
  const L lane(a);
  uint32_t cta, ctas;
  const Side s = side_of(a, cta, ctas);
  N da[NP][M], db[NP][M];
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < a.D; i += kThreads) w[i] = s.w[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int e = 0; e < M; ++e) da[i][e] = db[i][e] = splat<V>(0.f);
  }
  const uint32_t stride = ctas * kWarps;
  Cursor f;
  f.start(a, s, cta * kWarps + (threadIdx.x >> 5));
  Raw<T, V> nx[U][NP], ng[U][NP];
  Pass pass[U];
  auto fetch = [&](int u) {
    if (f.p.tok < a.tokens) {  // heads past the last: the last again
      const uint32_t h = min(f.p.h + lane.grp, f.p.h1 - 1);
      const T* x = static_cast<const T*>(s.x) + f.at + h * s.st[2];
      const T* dy = static_cast<const T*>(s.dy) + ((uint64_t)f.p.tok * s.H + h) * a.D;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if constexpr (NORM) nx[u][i] = load(x, lane.slot[i]);
        ng[u][i] = load(dy, lane.slot[i]);
      }
    }
    pass[u] = f.p;
    f.next<GW>(a, s, stride);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) fetch(u);
  Angles<V> g[NP];
  bool ok = true;
  while (pass[0].tok < a.tokens) {
    const Pass c = pass[0];
    if (c.fresh) ok = lane.angles(a, c.pos, g);
    N xa[NP][M], xb[NP][M], ga[NP][M], gb[NP][M];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if constexpr (NORM) widen<IL>(nx[0][i], xa[i], xb[i]);
      widen<IL>(ng[0][i], ga[i], gb[i]);
    }
#pragma unroll
    for (int u = 0; u + 1 < U; ++u) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if constexpr (NORM) nx[u][i] = nx[u + 1][i];
        ng[u][i] = ng[u + 1][i];
      }
      pass[u] = pass[u + 1];
    }
    fetch(U - 1);
    const uint32_t h = c.h + lane.grp;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (!ok) {  // no gradient (0, not 0 times what may be no number)
#pragma unroll
        for (int e = 0; e < M; ++e) ga[i][e] = gb[i][e] = splat<V>(0.f);
        if constexpr (NORM) {
#pragma unroll
          for (int e = 0; e < M; ++e) xa[i][e] = xb[i][e] = splat<V>(0.f);
        }
      }
      if (lane.slot[i].rot && ok) g[i].turn_back(ga[i], gb[i]);
    }
    if constexpr (NORM) {
      N ss = splat<V>(0.f), sg = ss;
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < M; ++e) ss = fma(xa[i][e], xa[i][e], fma(xb[i][e], xb[i][e], ss));
      // rows past the last (and tokens without angles) add 0, with eps = 0 too
      const float mean = lane.sum(ss) * a.inv_d, rstd = h < c.h1 && ok ? rsqrtf(mean + a.eps) : 0.f;
      const N r = splat<V>(rstd);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        N wa[M], wb[M];
        widen<IL>(load<float, V>(w, lane.slot[i]), wa, wb);
#pragma unroll
        for (int e = 0; e < M; ++e) {
          xa[i][e] = mul(xa[i][e], r), xb[i][e] = mul(xb[i][e], r);
          da[i][e] = fma(ga[i][e], xa[i][e], da[i][e]), db[i][e] = fma(gb[i][e], xb[i][e], db[i][e]);
          ga[i][e] = mul(ga[i][e], wa[e]), gb[i][e] = mul(gb[i][e], wb[e]);
          sg = fma(ga[i][e], xa[i][e], fma(gb[i][e], xb[i][e], sg));
        }
      }
      const N m = splat<V>(-lane.sum(sg) * a.inv_d);
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < M; ++e)
          ga[i][e] = mul(r, fma(xa[i][e], m, ga[i][e])), gb[i][e] = mul(r, fma(xb[i][e], m, gb[i][e]));
    }
    if (h < c.h1) {
      T* dx = static_cast<T*>(s.dx) + ((uint64_t)c.tok * s.H + h) * a.D;
#pragma unroll
      for (int i = 0; i < NP; ++i) store<IL>(dx, lane.slot[i], ga[i], gb[i]);
    }
  }
  if constexpr (NORM) {
    float* mine = sums + (size_t)((threadIdx.x >> 5) * GW + lane.grp) * a.D;
#pragma unroll
    for (int i = 0; i < NP; ++i) store<IL>(mine, lane.slot[i], da[i], db[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      float x = 0.f;
      for (int i = 0; i < kWarps * GW; ++i) x += sums[(size_t)i * a.D + c];
      a.partial[(long)blockIdx.x * a.D + c] = x;
    }
  }
}

// dw: the sums of a side's CTAs.  32 warps take every 32nd CTA for 32 columns, and
// their sums are added in order.
__global__ void __launch_bounds__(1024) qk_rope_sum_kernel(Args a, int ctas) {
  __shared__ float s[32][33];
  tc::grid_dep_wait();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
  const int first = blockIdx.y ? a.ctas0 : 0, end = blockIdx.y ? ctas : a.ctas0;
  float x = 0.f;
  if (c < a.D) {
#pragma unroll 4
    for (int i = first + w; i < end; i += 32) x += a.partial[(long)i * a.D + c];
  }
  s[w][lane] = x;
  __syncthreads();
  if (w > 0 || c >= a.D) return;
  x = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) x += s[i][lane];
  a.side[blockIdx.y].dw[c] = x;
}

// ---------------------------------------------------------------- host

// Whether all rows go in vectors of V pairs' halves.
bool use_vectors(const QkRopeProblem& p, int V) {
  const size_t e = p.bf16 ? 2 : 4;
  if (p.D % (2 * V) || p.R % (2 * V)) return false;
  if (!vectors(p.q, p.qs, e) || !vectors(p.k, p.ks, e)) return false;
  for (const void* x : {(const void*)p.wq, (const void*)p.wk, (const void*)p.cos, (const void*)p.sin})
    if ((uintptr_t)x & 15) return false;
  return true;
}

// Heads per job: all of a token's, or fewer (in passes of gw) until every warp that
// runs at once has a job.
void set_jobs(Side& s, uint32_t tokens, int gw, long warps) {
  const long passes = (s.H + gw - 1) / gw, want = std::max(1L, std::min(passes, (warps + tokens - 1) / tokens));
  s.chunk = (int)((passes + want - 1) / want) * gw;
  s.parts = s.H ? (s.H + s.chunk - 1) / s.chunk : 0;
}

template <typename T, int V, int NP, int LR, bool IL, bool NORM>
cudaError_t launch(Args a, bool bwd, cudaStream_t s) {
  constexpr int GW = 32 / LR;
  const int most = (bwd ? kPerSmBwd : kPerSmFwd) * sm_count(), H = a.side[0].H + a.side[1].H;
  int ctas[2];
  for (int i = 0; i < 2; ++i) {
    Side& x = a.side[i];
    // a token costs what two more heads would
    const long share = std::max(1L, (long)most * (x.H + 2) / (H + 4));
    set_jobs(x, a.tokens, GW, share * kWarps);
    ctas[i] = x.H ? (int)std::min(share, ((long)a.tokens * x.parts + kWarps - 1) / kWarps) : 0;
  }
  a.ctas0 = ctas[0];
  const int all = ctas[0] + ctas[1];
  if (!bwd) {
    prof_before(s);
    qk_rope_fwd_kernel<T, V, NP, LR, IL, NORM><<<all, kThreads, 0, s>>>(a);
    prof_after(s, kQkRopeFwd);
    return cudaGetLastError();
  }
  const size_t smem = NORM ? (size_t)kWarps * GW * a.D * sizeof(float) : 0;
  prof_before(s);
  qk_rope_bwd_kernel<T, V, NP, LR, IL, NORM><<<all, kThreads, smem, s>>>(a);
  prof_after(s, kQkRopeBwd);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !NORM) return e;
  prof_before(s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.D + 31) / 32, 2), cfg.blockDim = dim3(1024), cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, qk_rope_sum_kernel, a, all);
  prof_after(s, kQkRopeSum);
  return e;
}

template <typename T, bool IL, bool NORM>
cudaError_t by_size(const QkRopeProblem& p, const Args& a, bool bwd, cudaStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (use_vectors(p, 8))
      return p.D <= 64 ? launch<T, 8, 1, 4, IL, NORM>(a, bwd, s) : launch<T, 8, 1, 8, IL, NORM>(a, bwd, s);
  }
  if (use_vectors(p, 4))
    return p.D <= 64 ? launch<T, 4, 1, 8, IL, NORM>(a, bwd, s) : launch<T, 4, 1, 16, IL, NORM>(a, bwd, s);
  return launch<T, 1, 2, 32, IL, NORM>(a, bwd, s);
}

template <typename T>
cudaError_t by_kind(const QkRopeProblem& p, const Args& a, bool bwd, cudaStream_t s) {
  if (p.wq) return p.interleaved ? by_size<T, true, true>(p, a, bwd, s) : by_size<T, false, true>(p, a, bwd, s);
  return p.interleaved ? by_size<T, true, false>(p, a, bwd, s) : by_size<T, false, false>(p, a, bwd, s);
}

cudaError_t run(const QkRopeProblem& p, bool bwd, cudaStream_t s) {
  Args a = {};
  a.T = p.T, a.D = p.D, a.R = p.R, a.P = p.P;
  a.tokens = (uint32_t)((long)p.B * p.T);
  a.eps = p.eps, a.inv_d = 1.f / p.D;
  Side &q = a.side[0], &k = a.side[1];
  for (int i = 0; i < 3; ++i) q.st[i] = p.qs[i], k.st[i] = p.ks[i];
  q.x = p.q, q.dy = p.dqo, q.y = p.qo, q.dx = p.dq, q.w = p.wq, q.dw = p.dwq, q.H = p.H;
  k.x = p.k, k.dy = p.dko, k.y = p.ko, k.dx = p.dk, k.w = p.wk, k.dw = p.dwk, k.H = p.Hkv;
  a.cos = p.cos, a.sin = p.sin, a.pos = p.pos;
  a.partial = static_cast<float*>(p.ws);
  return p.bf16 ? by_kind<__nv_bfloat16>(p, a, bwd, s) : by_kind<float>(p, a, bwd, s);
}

}  // namespace

// Sums of every CTA that may run (each side has one at least).
size_t qk_rope_bwd_workspace(const QkRopeProblem& p) {
  return (size_t)(kPerSmBwd * sm_count() + 2) * p.D * sizeof(float);
}

cudaError_t qk_rope_fwd(const QkRopeProblem& p, cudaStream_t s) { return run(p, false, s); }
cudaError_t qk_rope_bwd(const QkRopeProblem& p, cudaStream_t s) { return run(p, true, s); }

}  // namespace gdn
