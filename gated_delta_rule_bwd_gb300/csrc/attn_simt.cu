// Causal attention on the CUDA cores: fp32 arithmetic, any D <= 128, either
// dtype, any strides.
//
// Per sequence and head, with s_ij = scale q_i . k_j over the keys that query
// i sees (j <= i + lk - lq):
//   forward   m, l the running maximum and sum of exp(s - m) over key tiles;
//             o = sum exp(s - m) v / l,  lse = m + log l
//   backward  p = exp(s - lse), dp = do . v, ds = p (dp - delta) with
//             delta = do . o;  dv = p^T do, dk = scale ds^T q, dq = scale ds k
// A CTA of 256 threads (16 x 16) owns a tile of 64 rows and walks the other
// side in tiles of 64; a thread owns 4 x 4 scores (rows ty + 16 i, columns
// tx + 16 j) and 4 rows of the accumulators.  The tiles lie in shared memory
// as fp32 with rows of DP + 4 floats, so that the float4 reads of eight
// consecutive rows touch all banks once.  dk and dv come from a kernel that
// owns key tiles and sums over the queries (of all heads that share the key
// head, in order), dq from one that owns query tiles: the scores are computed
// twice, and nothing is added atomically, so results do not depend on the
// order in which CTAs run.  Bound by the fp32 FMA rate.

#include <math.h>

#include "attn.cuh"
#include "tc_common.cuh"

namespace gdn {

cudaError_t attn_simt_read_and_clear_status(int* status) {
  return tc::read_and_clear_file_status(status);
}

namespace {

constexpr int kM = 64;       // rows of a tile
constexpr int kThreads = 256;
constexpr int kLdP = kM + 4;
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
  AttnSeqs sq;
  int H, Hkv, D;
  float scale;
  long long qs[3], ks[3], vs[3];
  const void *q, *k, *v, *do_;
  void* o;
  float* lse;
  const float* delta;
  void *dq, *dk, *dv;
};

Args args_of(const AttnProblem& p) {
  Args a;
  a.sq = AttnSeqs::of(p);
  a.H = p.H, a.Hkv = p.Hkv, a.D = p.D, a.scale = p.scale;
  for (int i = 0; i < 3; ++i) a.qs[i] = p.qs[i], a.ks[i] = p.ks[i], a.vs[i] = p.vs[i];
  a.q = p.q, a.k = p.k, a.v = p.v, a.do_ = p.do_, a.o = p.o, a.lse = p.lse;
  a.delta = static_cast<const float*>(p.ws);
  a.dq = p.dq, a.dk = p.dk, a.dv = p.dv;
  return a;
}

// 64 rows of D values (row r at src + r * stride, rows >= n zero) as fp32
template <typename T, int DP>
__device__ __forceinline__ void load_tile(float* dst, const T* src, long long stride, int n, int D) {
  constexpr int LD = DP + 4;
  for (int i = threadIdx.x; i < kM * DP; i += kThreads) {
    const int r = i / DP, c = i % DP;
    dst[r * LD + c] = (r < n && c < D) ? to_f32(src[r * stride + c]) : 0.f;
  }
}

// c[i][j] = A[ty + 16 i] . B[tx + 16 j] over DP columns
template <int DP>
__device__ __forceinline__ void dots(float (&c)[4][4], const float* A, const float* B, int ty, int tx) {
  constexpr int LD = DP + 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
#pragma unroll 2
  for (int d = 0; d < DP; d += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * LD + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * LD + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[i][j] = fmaf(a[i].x, b[j].x, c[i][j]);
        c[i][j] = fmaf(a[i].y, b[j].y, c[i][j]);
        c[i][j] = fmaf(a[i].z, b[j].z, c[i][j]);
        c[i][j] = fmaf(a[i].w, b[j].w, c[i][j]);
      }
  }
}

// acc[i][*] += sum_n P[ty + 16 i][n] X[n][*]: the thread's columns are
// 4 tx + 64 u + {0..3}
template <int DP>
__device__ __forceinline__ void rows_times(float (&acc)[4][DP / 16], const float* P, const float* X,
                                           int ty, int tx) {
  constexpr int LD = DP + 4;
#pragma unroll 2
  for (int n = 0; n < kM; n += 4) {
    float p[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(P + (ty + 16 * i) * kLdP + n);
#pragma unroll
    for (int u = 0; u < DP / 64; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 x = *reinterpret_cast<const float4*>(X + (n + e) * LD + 4 * tx + 64 * u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i][4 * u + 0] = fmaf(p[i][e], x.x, acc[i][4 * u + 0]);
          acc[i][4 * u + 1] = fmaf(p[i][e], x.y, acc[i][4 * u + 1]);
          acc[i][4 * u + 2] = fmaf(p[i][e], x.z, acc[i][4 * u + 2]);
          acc[i][4 * u + 3] = fmaf(p[i][e], x.w, acc[i][4 * u + 3]);
        }
      }
  }
}

// acc[i][*] += sum_r P[r][4 ty + i] X[r][*]
template <int DP>
__device__ __forceinline__ void cols_times(float (&acc)[4][DP / 16], const float* P, const float* X,
                                           int ty, int tx) {
  constexpr int LD = DP + 4;
#pragma unroll 4
  for (int r = 0; r < kM; ++r) {
    float p[4];
    *reinterpret_cast<float4*>(p) = *reinterpret_cast<const float4*>(P + r * kLdP + 4 * ty);
#pragma unroll
    for (int u = 0; u < DP / 64; ++u) {
      const float4 x = *reinterpret_cast<const float4*>(X + r * LD + 4 * tx + 64 * u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][4 * u + 0] = fmaf(p[i], x.x, acc[i][4 * u + 0]);
        acc[i][4 * u + 1] = fmaf(p[i], x.y, acc[i][4 * u + 1]);
        acc[i][4 * u + 2] = fmaf(p[i], x.z, acc[i][4 * u + 2]);
        acc[i][4 * u + 3] = fmaf(p[i], x.w, acc[i][4 * u + 3]);
      }
    }
  }
}

// a thread's columns of one output row
template <typename T, int DP>
__device__ __forceinline__ void store_row(T* dst, const float* acc, float f, int tx, int D) {
#pragma unroll
  for (int u = 0; u < DP / 64; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = 4 * tx + 64 * u + e;
      if (c < D) dst[c] = from_f32<T>(acc[4 * u + e] * f);
    }
}

// over the 16 threads of a row
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int DP>
constexpr int tile_floats() { return kM * (DP + 4); }

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attn_simt_fwd_kernel(Args a) {
  extern __shared__ float sm[];
  float *Q = sm, *K = Q + tile_floats<DP>(), *V = K + tile_floats<DP>(), *P = V + tile_floats<DP>();
  if (blockIdx.x == 0 && blockIdx.y == 0 && !a.sq.valid() && threadIdx.x == 0)
    atomicExch(&tc::g_file_status, GDN_ERR_SEQLENS);
  AttnTile t;
  if (!a.sq.get<false>(blockIdx.x, kM, t)) return;
  const int h = blockIdx.y, hk = h / (a.H / a.Hkv), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int r0 = t.tile * kM, nr = min(kM, t.lq - r0), shift = t.lk - t.lq;
  const T* q = static_cast<const T*>(a.q) + t.b * a.qs[0] + (long long)(t.q0 + r0) * a.qs[1] + h * a.qs[2];
  const T* k = static_cast<const T*>(a.k) + t.b * a.ks[0] + (long long)t.k0 * a.ks[1] + hk * a.ks[2];
  const T* v = static_cast<const T*>(a.v) + t.b * a.vs[0] + (long long)t.k0 * a.vs[1] + hk * a.vs[2];
  load_tile<T, DP>(Q, q, a.qs[1], nr, a.D);
  float acc[4][DP / 16], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) acc[i][c] = 0.f;
  }
  const int nk = min(t.lk, r0 + nr + shift);  // keys that the tile's last row sees
  for (int j0 = 0; j0 < nk; j0 += kM) {
    __syncthreads();
    load_tile<T, DP>(K, k + (long long)j0 * a.ks[1], a.ks[1], t.lk - j0, a.D);
    load_tile<T, DP>(V, v + (long long)j0 * a.vs[1], a.vs[1], t.lk - j0, a.D);
    __syncthreads();
    float s[4][4];
    dots<DP>(s, Q, K, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int last = min(r0 + ty + 16 * i + shift, t.lk - 1);  // the row's last key
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = j0 + tx + 16 * j <= last ? s[i][j] * a.scale : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      mx = row_max(mx);
      const float base = mx == -INFINITY ? 0.f : mx;  // no key yet: every term is 0
      const float f = exp2f((m[i] - base) * kLog2e);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f((s[i][j] - base) * kLog2e);
        sum += p;
        P[(ty + 16 * i) * kLdP + tx + 16 * j] = p;
      }
      l[i] = l[i] * f + row_sum(sum);
      m[i] = mx;
#pragma unroll
      for (int c = 0; c < DP / 16; ++c) acc[i][c] *= f;
    }
    __syncwarp();  // a row of P is written and read by one warp
    rows_times<DP>(acc, P, V, ty, tx);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    if (r >= nr) continue;
    const long long tok = (long long)t.b * a.sq.Tq + t.q0 + r0 + r;
    store_row<T, DP>(static_cast<T*>(a.o) + (tok * a.H + h) * a.D, acc[i], l[i] == 0.f ? 0.f : 1.f / l[i],
                     tx, a.D);
    if (tx == 0)
      a.lse[((long long)t.b * a.H + h) * a.sq.Tq + t.q0 + r0 + r] = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
  }
}

// One warp per (token, head): delta = do . o.
template <typename T>
__global__ void __launch_bounds__(256) attn_delta_kernel(const T* o, const T* do_, float* delta, int Tq,
                                                         int H, int D, long long rows) {
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int lane = threadIdx.x & 31;
  float s = 0.f;
  for (int c = lane; c < D; c += 32) s = fmaf(to_f32(o[r * D + c]), to_f32(do_[r * D + c]), s);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
  const long long tok = r / H;
  if (lane == 0) delta[(tok / Tq * H + r % H) * Tq + tok % Tq] = s;
}

// P = exp(s - lse) and dS = P (dP - delta) of one 64 x 64 tile, in registers
template <int DP>
__device__ __forceinline__ void grads(float (&p)[4][4], float (&ds)[4][4], const float* Q, const float* K,
                                      const float* dO, const float* V, const float* lse,
                                      const float* delta, int r0, int nr, int j0, int shift, int lk,
                                      float scale, int ty, int tx) {
  dots<DP>(p, Q, K, ty, tx);
  dots<DP>(ds, dO, V, ty, tx);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i, last = min(r0 + r + shift, lk - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool see = r < nr && j0 + tx + 16 * j <= last;
      p[i][j] = see ? exp2f((p[i][j] * scale - lse[r]) * kLog2e) : 0.f;
      ds[i][j] = see ? p[i][j] * (ds[i][j] - delta[r]) : 0.f;
    }
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attn_simt_bwd_kv_kernel(Args a) {
  extern __shared__ float sm[];
  constexpr int n = tile_floats<DP>();
  float *K = sm, *V = K + n, *Q = V + n, *dO = Q + n, *P = dO + n, *S = P + kM * kLdP;
  float *lse = S + kM * kLdP, *delta = lse + kM;
  if (blockIdx.x == 0 && blockIdx.y == 0 && !a.sq.valid() && threadIdx.x == 0)
    atomicExch(&tc::g_file_status, GDN_ERR_SEQLENS);
  AttnTile t;
  if (!a.sq.get<true>(blockIdx.x, kM, t)) return;
  const int G = a.H / a.Hkv, hk = blockIdx.y, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int j0 = t.tile * kM, shift = t.lk - t.lq;
  load_tile<T, DP>(K, static_cast<const T*>(a.k) + t.b * a.ks[0] + (long long)(t.k0 + j0) * a.ks[1] + hk * a.ks[2],
                   a.ks[1], t.lk - j0, a.D);
  load_tile<T, DP>(V, static_cast<const T*>(a.v) + t.b * a.vs[0] + (long long)(t.k0 + j0) * a.vs[1] + hk * a.vs[2],
                   a.vs[1], t.lk - j0, a.D);
  float dk[4][DP / 16], dv[4][DP / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) dk[i][c] = dv[i][c] = 0.f;
  const int first = max(0, j0 - shift);  // the first query that sees the tile
  for (int h = hk * G; h < (hk + 1) * G; ++h) {
    const long long st = ((long long)t.b * a.H + h) * a.sq.Tq + t.q0;
    for (int r0 = first / kM * kM; r0 < t.lq; r0 += kM) {
      const int nr = min(kM, t.lq - r0);
      __syncthreads();
      load_tile<T, DP>(Q, static_cast<const T*>(a.q) + t.b * a.qs[0] + (long long)(t.q0 + r0) * a.qs[1] + h * a.qs[2],
                       a.qs[1], nr, a.D);
      load_tile<T, DP>(dO, static_cast<const T*>(a.do_) + (((long long)t.b * a.sq.Tq + t.q0 + r0) * a.H + h) * a.D,
                       (long long)a.H * a.D, nr, a.D);
      if (threadIdx.x < nr) lse[threadIdx.x] = a.lse[st + r0 + threadIdx.x];
      else if (threadIdx.x < kM) lse[threadIdx.x] = 0.f;
      if (threadIdx.x < nr) delta[threadIdx.x] = a.delta[st + r0 + threadIdx.x];
      __syncthreads();
      float p[4][4], ds[4][4];
      grads<DP>(p, ds, Q, K, dO, V, lse, delta, r0, nr, j0, shift, t.lk, a.scale, ty, tx);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          P[(ty + 16 * i) * kLdP + tx + 16 * j] = p[i][j];
          S[(ty + 16 * i) * kLdP + tx + 16 * j] = ds[i][j];
        }
      __syncthreads();
      cols_times<DP>(dv, P, dO, ty, tx);
      cols_times<DP>(dk, S, Q, ty, tx);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + 4 * ty + i;
    if (j >= t.lk) continue;
    const long long at = (((long long)t.b * a.sq.Tk + t.k0 + j) * a.Hkv + hk) * a.D;
    store_row<T, DP>(static_cast<T*>(a.dk) + at, dk[i], a.scale, tx, a.D);
    store_row<T, DP>(static_cast<T*>(a.dv) + at, dv[i], 1.f, tx, a.D);
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attn_simt_bwd_q_kernel(Args a) {
  extern __shared__ float sm[];
  constexpr int n = tile_floats<DP>();
  float *K = sm, *V = K + n, *Q = V + n, *dO = Q + n, *S = dO + n;
  float *lse = S + kM * kLdP, *delta = lse + kM;
  AttnTile t;
  if (!a.sq.get<false>(blockIdx.x, kM, t)) return;
  const int h = blockIdx.y, hk = h / (a.H / a.Hkv), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int r0 = t.tile * kM, nr = min(kM, t.lq - r0), shift = t.lk - t.lq;
  const long long st = ((long long)t.b * a.H + h) * a.sq.Tq + t.q0 + r0;
  const long long tok = (long long)t.b * a.sq.Tq + t.q0 + r0;
  load_tile<T, DP>(Q, static_cast<const T*>(a.q) + t.b * a.qs[0] + (long long)(t.q0 + r0) * a.qs[1] + h * a.qs[2],
                   a.qs[1], nr, a.D);
  load_tile<T, DP>(dO, static_cast<const T*>(a.do_) + (tok * a.H + h) * a.D, (long long)a.H * a.D, nr, a.D);
  if (threadIdx.x < nr) lse[threadIdx.x] = a.lse[st + threadIdx.x], delta[threadIdx.x] = a.delta[st + threadIdx.x];
  else if (threadIdx.x < kM) lse[threadIdx.x] = 0.f, delta[threadIdx.x] = 0.f;
  float dq[4][DP / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) dq[i][c] = 0.f;
  const int nk = min(t.lk, r0 + nr + shift);
  for (int j0 = 0; j0 < nk; j0 += kM) {
    __syncthreads();
    load_tile<T, DP>(K, static_cast<const T*>(a.k) + t.b * a.ks[0] + (long long)(t.k0 + j0) * a.ks[1] + hk * a.ks[2],
                     a.ks[1], t.lk - j0, a.D);
    load_tile<T, DP>(V, static_cast<const T*>(a.v) + t.b * a.vs[0] + (long long)(t.k0 + j0) * a.vs[1] + hk * a.vs[2],
                     a.vs[1], t.lk - j0, a.D);
    __syncthreads();
    float p[4][4], ds[4][4];
    grads<DP>(p, ds, Q, K, dO, V, lse, delta, r0, nr, j0, shift, t.lk, a.scale, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) S[(ty + 16 * i) * kLdP + tx + 16 * j] = ds[i][j];
    __syncwarp();
    rows_times<DP>(dq, S, K, ty, tx);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    if (r < nr) store_row<T, DP>(static_cast<T*>(a.dq) + ((tok + r) * a.H + h) * a.D, dq[i], a.scale, tx, a.D);
  }
}

// delta [B, H, Tq] = rowsum(do * o) into the workspace
cudaError_t attn_delta(const AttnProblem& p, cudaStream_t s) {
  const long long rows = (long long)p.B * p.Tq * p.H;
  if (rows == 0) return cudaSuccess;
  const unsigned grid = (unsigned)((rows + 7) / 8);
  float* delta = static_cast<float*>(p.ws);
  prof_before(s);
  if (p.bf16)
    attn_delta_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(p.o),
                                           static_cast<const __nv_bfloat16*>(p.do_), delta, p.Tq, p.H, p.D, rows);
  else
    attn_delta_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(p.o), static_cast<const float*>(p.do_),
                                           delta, p.Tq, p.H, p.D, rows);
  cudaError_t e = cudaGetLastError();
  prof_after(s, kAttnDelta);
  return e;
}

template <typename K>
cudaError_t launch(K kernel, dim3 grid, int smem, const Args& a, cudaStream_t s, int id) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  prof_before(s);
  kernel<<<grid, kThreads, smem, s>>>(a);
  e = cudaGetLastError();
  prof_after(s, id);
  return e;
}

template <typename T, int DP>
cudaError_t fwd(const AttnProblem& p, cudaStream_t s) {
  const int smem = (3 * tile_floats<DP>() + kM * kLdP) * 4;
  const dim3 grid((unsigned)AttnSeqs::slots(p, kM, false), p.H);
  return launch(attn_simt_fwd_kernel<T, DP>, grid, smem, args_of(p), s, kAttnFwd);
}

template <typename T, int DP>
cudaError_t bwd(const AttnProblem& p, cudaStream_t s) {
  cudaError_t e = attn_delta(p, s);
  const Args a = args_of(p);
  if (e == cudaSuccess && p.Tk > 0) {
    const int smem = (4 * tile_floats<DP>() + 2 * kM * kLdP + 2 * kM) * 4;
    const dim3 grid((unsigned)AttnSeqs::slots(p, kM, true), p.Hkv);
    e = launch(attn_simt_bwd_kv_kernel<T, DP>, grid, smem, a, s, kAttnBwdKv);
  }
  if (e == cudaSuccess && p.Tq > 0) {
    const int smem = (4 * tile_floats<DP>() + kM * kLdP + 2 * kM) * 4;
    const dim3 grid((unsigned)AttnSeqs::slots(p, kM, false), p.H);
    e = launch(attn_simt_bwd_q_kernel<T, DP>, grid, smem, a, s, kAttnBwdQ);
  }
  return e;
}

}  // namespace

size_t attn_bwd_workspace(const AttnProblem& p) { return (size_t)p.B * p.H * p.Tq * sizeof(float); }

cudaError_t attn_simt_fwd(const AttnProblem& p, cudaStream_t s) {
  if (p.bf16) return p.D <= 64 ? fwd<__nv_bfloat16, 64>(p, s) : fwd<__nv_bfloat16, 128>(p, s);
  return p.D <= 64 ? fwd<float, 64>(p, s) : fwd<float, 128>(p, s);
}

cudaError_t attn_simt_bwd(const AttnProblem& p, cudaStream_t s) {
  if (p.bf16) return p.D <= 64 ? bwd<__nv_bfloat16, 64>(p, s) : bwd<__nv_bfloat16, 128>(p, s);
  return p.D <= 64 ? bwd<float, 64>(p, s) : bwd<float, 128>(p, s);
}

}  // namespace gdn
