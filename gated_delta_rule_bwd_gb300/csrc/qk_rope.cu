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
// nothing is saved).  A warp takes a token and walks its heads, so that the
// angles are read once per token and lane; a row stays in the registers of its
// LR lanes, several rows on their way.  Where there are few tokens, several
// warps share one.
//
// dw: a lane keeps its columns' sums over all rows of its warp; they are added
// per CTA and, by a second kernel, over the CTAs, each in a fixed order.

#include "rope.cuh"

namespace gdn {

cudaError_t qk_rope_read_and_clear_status(int* status) { return tc::read_and_clear_file_status(status); }

namespace {

using namespace rope;
using tc::sm_count;

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Args {
  int T, H, rows, D, R, P, split;  // rows: heads of q and of k; split: warps per token
  long tokens;
  float eps, inv_d;
  long long qs[3], ks[3];
  const void *q, *k;
  const float *wq, *wk, *cos, *sin;
  const int* pos;
  void *qo, *ko;           // forward
  const void *dqo, *dko;   // backward
  void *dq, *dk;
  float* partial;          // [ctas][2][D] sums of dw
};

// A token's place and angles, the same for all lanes of the warp.
template <int V, int NP>
struct Token {
  int b, t;
  bool ok;  // its position has angles
  float c[NP][V], s[NP][V];
};

template <int V, int NP, int LR, bool IL>
struct Lane {
  Slot<V> slot[NP];
  int grp;
  __device__ __forceinline__ explicit Lane(const Args& a) {
    grp = (threadIdx.x & 31) / LR;
#pragma unroll
    for (int i = 0; i < NP; ++i) slot[i].template set<IL>(pair(i), a.D, a.R);
  }
  __device__ __forceinline__ static int pair(int i) { return ((threadIdx.x & 31) % LR + i * LR) * V; }

  __device__ __forceinline__ Token<V, NP> token(const Args& a, long tok) const {
    Token<V, NP> k;
    k.b = (int)(tok / a.T), k.t = (int)(tok % a.T);
    int n = 0;
    k.ok = true;
    if (a.R) {
      n = a.pos ? a.pos[tok] : k.t;
      if (n < 0 || n >= a.P) {
        k.ok = false, n = 0;
        if ((threadIdx.x & 31) == 0) atomicExch(&tc::g_file_status, GDN_ERR_SEQLENS);
      }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i)
      angles<V>(a.cos, a.sin, (long long)n * (a.R / 2), pair(i), slot[i].rot && k.ok, k.c[i], k.s[i]);
    return k;
  }
  // the lane's weights
  __device__ __forceinline__ void weights(const float* w, float (&wa)[NP][V], float (&wb)[NP][V]) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) widen<IL>(load(w, slot[i]), wa[i], wb[i]);
  }
};

// x and, in the backward, dy of row r of a token
template <typename T>
__device__ __forceinline__ const T* input(const Args& a, int b, int t, int r) {
  return r < a.H ? static_cast<const T*>(a.q) + b * a.qs[0] + t * a.qs[1] + r * a.qs[2]
                 : static_cast<const T*>(a.k) + b * a.ks[0] + t * a.ks[1] + (r - a.H) * a.ks[2];
}
// a contiguous [B, T, H, D] / [B, T, Hkv, D] pair
template <typename T>
__device__ __forceinline__ T* dense(const Args& a, void* q, void* k, long tok, int r) {
  return r < a.H ? static_cast<T*>(q) + (tok * a.H + r) * a.D
                 : static_cast<T*>(k) + (tok * (a.rows - a.H) + r - a.H) * a.D;
}

template <typename T, int V, int NP, int LR, bool IL, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_rope_fwd_kernel(Args a) {
  constexpr int GW = 32 / LR, U = V == 4 ? 4 : 1;  // rows a warp works on at once, and has on their way
  const Lane<V, NP, LR, IL> L(a);
  const long job = (long)blockIdx.x * kWarps + (threadIdx.x >> 5), tok = job / a.split;
  if (tok >= a.tokens) return;
  const int part = (int)(job % a.split), step = a.split * GW;
  const int b = (int)(tok / a.T), t = (int)(tok % a.T);
  Raw<T, V> x[U][NP];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * step + L.grp;
#pragma unroll
      for (int i = 0; i < NP; ++i)
        x[u][i] = r < a.rows ? load(input<T>(a, b, t, r), L.slot[i]) : Raw<T, V>{};
    }
  };
  int r0 = part * GW;
  fetch(r0);
  const Token<V, NP> k = L.token(a, tok);
  float wq[2][NP][V], wk[2][NP][V];
  if constexpr (NORM) L.weights(a.wq, wq[0], wq[1]), L.weights(a.wk, wk[0], wk[1]);
  for (; r0 < a.rows; r0 += U * step) {
    float xa[U][NP][V], xb[U][NP][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NP; ++i) widen<IL>(x[u][i], xa[u][i], xb[u][i]);
    if (r0 + U * step < a.rows) fetch(r0 + U * step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * step + L.grp;
      if constexpr (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e) ss = fmaf(xa[u][i][e], xa[u][i][e], fmaf(xb[u][i][e], xb[u][i][e], ss));
        const float rstd = rsqrtf(row_sum<LR>(ss) * a.inv_d + a.eps);
        const bool isq = r < a.H;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            xa[u][i][e] = xa[u][i][e] * rstd * (isq ? wq[0][i][e] : wk[0][i][e]);
            xb[u][i][e] = xb[u][i][e] * rstd * (isq ? wq[1][i][e] : wk[1][i][e]);
          }
      }
      if (r >= a.rows) continue;
      T* y = dense<T>(a, a.qo, a.ko, tok, r);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (L.slot[i].rot) rotate<V>(k.c[i], k.s[i], xa[u][i], xb[u][i]);
        if (!k.ok) {
#pragma unroll
          for (int e = 0; e < V; ++e) xa[u][i][e] = xb[u][i][e] = 0.f;
        }
        store<IL>(y, L.slot[i], xa[u][i], xb[u][i]);
      }
    }
  }
}

template <typename T, int V, int NP, int LR, bool IL, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_rope_bwd_kernel(Args a) {
  constexpr int GW = 32 / LR, U = V == 4 ? 2 : 1;
  extern __shared__ float sums[];  // NORM: [kWarps * GW][2][D]
  tc::grid_dep_launch();
  const Lane<V, NP, LR, IL> L(a);
  float dwq[2][NP][V], dwk[2][NP][V], wq[2][NP][V], wk[2][NP][V];
  if constexpr (NORM) {
    L.weights(a.wq, wq[0], wq[1]), L.weights(a.wk, wk[0], wk[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) dwq[h][i][e] = dwk[h][i][e] = 0.f;
  }
  const int step = a.split * GW;
  for (long job = (long)blockIdx.x * kWarps + (threadIdx.x >> 5); job < a.tokens * a.split;
       job += (long)gridDim.x * kWarps) {
    const long tok = job / a.split;
    const Token<V, NP> k = L.token(a, tok);
    for (int r0 = (int)(job % a.split) * GW; r0 < a.rows; r0 += U * step) {
      Raw<T, V> x[U][NP], g[U][NP];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * step + L.grp;
        const bool in = r < a.rows && k.ok;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          x[u][i] = in ? load(input<T>(a, k.b, k.t, r), L.slot[i]) : Raw<T, V>{};
          g[u][i] = in ? load(static_cast<const T*>(dense<T>(a, const_cast<void*>(a.dqo), const_cast<void*>(a.dko), tok, r)),
                              L.slot[i])
                       : Raw<T, V>{};
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * step + L.grp;
        float ga[NP][V], gb[NP][V];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          widen<IL>(g[u][i], ga[i], gb[i]);
          if (L.slot[i].rot) {
            float s[V];
#pragma unroll
            for (int e = 0; e < V; ++e) s[e] = -k.s[i][e];
            rotate<V>(k.c[i], s, ga[i], gb[i]);
          }
        }
        if constexpr (NORM) {
          const bool isq = r < a.H;
          float xa[NP][V], xb[NP][V], ss = 0.f, sg = 0.f;
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            widen<IL>(x[u][i], xa[i], xb[i]);
#pragma unroll
            for (int e = 0; e < V; ++e) ss = fmaf(xa[i][e], xa[i][e], fmaf(xb[i][e], xb[i][e], ss));
          }
          // rows past the last (and tokens without angles) add 0, with eps = 0 too
          const float mean = row_sum<LR>(ss) * a.inv_d, rstd = r < a.rows && k.ok ? rsqrtf(mean + a.eps) : 0.f;
#pragma unroll
          for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              xa[i][e] *= rstd, xb[i][e] *= rstd;
              const float ta = ga[i][e] * xa[i][e], tb = gb[i][e] * xb[i][e];
              const float wa = isq ? wq[0][i][e] : wk[0][i][e], wb = isq ? wq[1][i][e] : wk[1][i][e];
              if (isq) dwq[0][i][e] += ta, dwq[1][i][e] += tb;
              else dwk[0][i][e] += ta, dwk[1][i][e] += tb;
              sg = fmaf(ta, wa, fmaf(tb, wb, sg));
              ga[i][e] *= wa, gb[i][e] *= wb;
            }
          const float m = row_sum<LR>(sg) * a.inv_d;
#pragma unroll
          for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              ga[i][e] = rstd * fmaf(-xa[i][e], m, ga[i][e]);
              gb[i][e] = rstd * fmaf(-xb[i][e], m, gb[i][e]);
            }
        }
        if (r >= a.rows) continue;
        T* d = dense<T>(a, a.dq, a.dk, tok, r);
#pragma unroll
        for (int i = 0; i < NP; ++i) store<IL>(d, L.slot[i], ga[i], gb[i]);
      }
    }
  }
  if constexpr (NORM) {
    float* mine = sums + (size_t)((threadIdx.x >> 5) * GW + L.grp) * 2 * a.D;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      store<IL>(mine, L.slot[i], dwq[0][i], dwq[1][i]);
      store<IL>(mine + a.D, L.slot[i], dwk[0][i], dwk[1][i]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.D; c += kThreads) {
      float s = 0.f;
      for (int i = 0; i < kWarps * GW; ++i) s += sums[(size_t)i * 2 * a.D + c];
      a.partial[(long)blockIdx.x * 2 * a.D + c] = s;
    }
  }
}

// dw of q (columns 0 .. D - 1) and k: the CTAs' sums.  Eight warps take every
// eighth CTA for 32 columns, and their sums are added in order.
__global__ void __launch_bounds__(256) qk_rope_sum_kernel(const float* partial, int ctas, int D, float* dwq, float* dwk) {
  __shared__ float s[8][32];
  tc::grid_dep_wait();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
  float x = 0.f;
  if (c < 2 * D) {
#pragma unroll 8
    for (int i = w; i < ctas; i += 8) x += partial[(long)i * 2 * D + c];
  }
  s[w][lane] = x;
  __syncthreads();
  if (w > 0 || c >= 2 * D) return;
  x = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) x += s[i][lane];
  (c < D ? dwq[c] : dwk[c - D]) = x;
}

// ---------------------------------------------------------------- host

constexpr int kBwdCtasPerSm = 3;

// CTAs of the backward: as many as run at once, and no more than there are tokens' parts.
int bwd_ctas(long tokens, int split) {
  return (int)std::max(1L, std::min((long)kBwdCtasPerSm * sm_count(), (tokens * split + kWarps - 1) / kWarps));
}

bool use_vectors(const QkRopeProblem& p) {
  const size_t e = p.bf16 ? 2 : 4;
  if (p.D % 8 || p.R % 8) return false;
  if (!vectors(p.q, p.qs, e) || !vectors(p.k, p.ks, e)) return false;
  for (const void* x : {(const void*)p.wq, (const void*)p.wk, (const void*)p.cos, (const void*)p.sin})
    if ((uintptr_t)x & 15) return false;
  return true;
}

// Warps per token: enough that the GPU has some 16 warps per SM, if the heads allow.
int split_of(long tokens, int rows, int gw) {
  const long want = (16L * sm_count() + tokens - 1) / tokens;
  return (int)std::max(1L, std::min(want, (long)(rows + gw - 1) / gw));
}

template <typename T, int V, int NP, int LR, bool IL, bool NORM>
cudaError_t launch(const QkRopeProblem& p, Args a, bool bwd, cudaStream_t s) {
  constexpr int GW = 32 / LR;
  a.split = split_of(a.tokens, a.rows, GW);
  if (!bwd) {
    const long ctas = (a.tokens * a.split + kWarps - 1) / kWarps;
    prof_before(s);
    qk_rope_fwd_kernel<T, V, NP, LR, IL, NORM><<<(unsigned)ctas, kThreads, 0, s>>>(a);
    prof_after(s, kQkRopeFwd);
    return cudaGetLastError();
  }
  const int ctas = bwd_ctas(a.tokens, a.split);
  const size_t smem = NORM ? (size_t)kWarps * GW * 2 * a.D * sizeof(float) : 0;
  prof_before(s);
  qk_rope_bwd_kernel<T, V, NP, LR, IL, NORM><<<ctas, kThreads, smem, s>>>(a);
  prof_after(s, kQkRopeBwd);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !NORM) return e;
  prof_before(s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((2 * a.D + 31) / 32), cfg.blockDim = dim3(256), cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, qk_rope_sum_kernel, (const float*)a.partial, ctas, a.D, p.dwq, p.dwk);
  prof_after(s, kQkRopeSum);
  return e;
}

template <typename T, bool IL, bool NORM>
cudaError_t by_size(const QkRopeProblem& p, const Args& a, bool bwd, cudaStream_t s) {
  if (!use_vectors(p)) return launch<T, 1, 2, 32, IL, NORM>(p, a, bwd, s);
  if (p.D <= 64) return launch<T, 4, 1, 8, IL, NORM>(p, a, bwd, s);
  return launch<T, 4, 1, 16, IL, NORM>(p, a, bwd, s);
}

template <typename T>
cudaError_t by_kind(const QkRopeProblem& p, const Args& a, bool bwd, cudaStream_t s) {
  if (p.wq) return p.interleaved ? by_size<T, true, true>(p, a, bwd, s) : by_size<T, false, true>(p, a, bwd, s);
  return p.interleaved ? by_size<T, true, false>(p, a, bwd, s) : by_size<T, false, false>(p, a, bwd, s);
}

cudaError_t run(const QkRopeProblem& p, bool bwd, cudaStream_t s) {
  Args a = {};
  a.T = p.T, a.H = p.H, a.rows = p.H + p.Hkv, a.D = p.D, a.R = p.R, a.P = p.P;
  a.tokens = (long)p.B * p.T;
  a.eps = p.eps, a.inv_d = 1.f / p.D;
  for (int i = 0; i < 3; ++i) a.qs[i] = p.qs[i], a.ks[i] = p.ks[i];
  a.q = p.q, a.k = p.k, a.wq = p.wq, a.wk = p.wk, a.cos = p.cos, a.sin = p.sin, a.pos = p.pos;
  a.qo = p.qo, a.ko = p.ko, a.dqo = p.dqo, a.dko = p.dko, a.dq = p.dq, a.dk = p.dk;
  a.partial = static_cast<float*>(p.ws);
  return p.bf16 ? by_kind<__nv_bfloat16>(p, a, bwd, s) : by_kind<float>(p, a, bwd, s);
}

}  // namespace

// The most CTAs that any choice of kernel has.
size_t qk_rope_bwd_workspace(const QkRopeProblem& p) {
  return (size_t)kBwdCtasPerSm * sm_count() * 2 * p.D * sizeof(float);
}

cudaError_t qk_rope_fwd(const QkRopeProblem& p, cudaStream_t s) { return run(p, false, s); }
cudaError_t qk_rope_bwd(const QkRopeProblem& p, cudaStream_t s) { return run(p, true, s); }

}  // namespace gdn
