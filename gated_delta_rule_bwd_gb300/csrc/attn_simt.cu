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
// twice, and nothing is added atomically, so results do not depend on the order
// in which CTAs run.  Both are roles of one launch.
//
// Small problems have fewer jobs than SMs and are bound by the time of one job's
// walk, so a cluster of up to eight CTAs shares a job: each walks a range of the
// other side's tiles, leaves its accumulators in shared memory, and sums a slice
// of the rows over the cluster, in the order of the ranks.  Larger ones are bound
// by the fp32 FMA rate.

#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "attn.cuh"
#include "tc_common.cuh"

namespace gdn {

namespace cg = cooperative_groups;

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
  int ranks;  // CTAs of a cluster, along x
  float scale;
  bool vec;  // rows of q, k, v and do_ are read in fours
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
  long long odd = p.D;
  for (int i = 0; i < 3; ++i) odd |= p.qs[i] | p.ks[i] | p.vs[i];
  const uintptr_t at = (uintptr_t)p.q | (uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)p.do_;
  a.vec = odd % 4 == 0 && at % (p.bf16 ? 8 : 16) == 0;
  return a;
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// 64 rows of D values (row r at src + r * stride, rows >= n zero) as fp32
template <typename T, int DP>
__device__ __forceinline__ void load_tile(float* dst, const T* src, long long stride, int n, int D, bool vec) {
  constexpr int LD = DP + 4;
  if (vec) {
#pragma unroll
    for (int x = 0; x < kM * DP / 4 / kThreads; ++x) {
      const int i = threadIdx.x + x * kThreads, r = i / (DP / 4), c = i % (DP / 4) * 4;
      *reinterpret_cast<float4*>(dst + r * LD + c) =
          r < n && c < D ? load4(src + r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
#pragma unroll 4
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

// a thread's 4 rows of an accumulator, rows first + i * step, to shared memory
template <int DP>
__device__ __forceinline__ void park(float* dst, const float (&acc)[4][DP / 16], int first, int step, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < DP / 64; ++u)
      *reinterpret_cast<float4*>(dst + (first + i * step) * (DP + 4) + 4 * tx + 64 * u) =
          make_float4(acc[i][4 * u], acc[i][4 * u + 1], acc[i][4 * u + 2], acc[i][4 * u + 3]);
}

// this rank's slice of a tile's n rows, summed over the cluster's parked tiles
template <typename T, int DP>
__device__ __forceinline__ void join_rows(T* dst, long long stride, float* tile, float f, int n, int D, int rank,
                                          int ranks) {
  const cg::cluster_group cluster = cg::this_cluster();
  const int rows = kM / ranks;
  for (int i = threadIdx.x; i < rows * DP / 4; i += kThreads) {
    const int r = rank * rows + i / (DP / 4), c = i % (DP / 4) * 4;
    if (r >= n || c >= D) continue;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < ranks; ++x) {
      const float4 y = *reinterpret_cast<const float4*>(cluster.map_shared_rank(tile, x) + r * (DP + 4) + c);
      sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
    }
    const float o[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < D) dst[r * stride + c + e] = from_f32<T>(o[e] * f);
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attn_simt_fwd_kernel(Args a) {
  extern __shared__ float sm[];
  float *Q = sm, *K = Q + tile_floats<DP>(), *V = K + tile_floats<DP>(), *P = V + tile_floats<DP>();
  const int rank = blockIdx.x % a.ranks;
  if (blockIdx.x == 0 && blockIdx.y == 0 && !a.sq.valid() && threadIdx.x == 0)
    atomicExch(&tc::g_file_status, GDN_ERR_SEQLENS);
  AttnTile t;
  if (!a.sq.get<false>(blockIdx.x / a.ranks, kM, t)) return;  // the whole cluster
  const int h = blockIdx.y, hk = h / (a.H / a.Hkv), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int r0 = t.tile * kM, nr = min(kM, t.lq - r0), shift = t.lk - t.lq;
  const T* q = static_cast<const T*>(a.q) + t.b * a.qs[0] + (long long)(t.q0 + r0) * a.qs[1] + h * a.qs[2];
  const T* k = static_cast<const T*>(a.k) + t.b * a.ks[0] + (long long)t.k0 * a.ks[1] + hk * a.ks[2];
  const T* v = static_cast<const T*>(a.v) + t.b * a.vs[0] + (long long)t.k0 * a.vs[1] + hk * a.vs[2];
  load_tile<T, DP>(Q, q, a.qs[1], nr, a.D, a.vec);
  float acc[4][DP / 16], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) acc[i][c] = 0.f;
  }
  const int nk = min(t.lk, r0 + nr + shift);  // keys that the tile's last row sees
  const int steps = (max(0, nk) + kM - 1) / kM, end = steps * (rank + 1) / a.ranks;
  for (int step = steps * rank / a.ranks; step < end; ++step) {
    const int j0 = step * kM;
    __syncthreads();
    load_tile<T, DP>(K, k + (long long)j0 * a.ks[1], a.ks[1], t.lk - j0, a.D, a.vec);
    load_tile<T, DP>(V, v + (long long)j0 * a.vs[1], a.vs[1], t.lk - j0, a.D, a.vec);
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
  if (a.ranks > 1) {
    // o = sum_x e^(m_x - m) acc_x / l,  l = sum_x e^(m_x - m) l_x over the ranks
    const cg::cluster_group cluster = cg::this_cluster();
    __syncthreads();
    park<DP>(K, acc, ty, 16, tx);
    if (tx == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i) V[ty + 16 * i] = m[i], V[kM + ty + 16 * i] = l[i];
    cluster.sync();
    const int rows = kM / a.ranks;
    const long long tok = (long long)t.b * a.sq.Tq + t.q0 + r0;
    for (int i = threadIdx.x; i < rows * DP / 4; i += kThreads) {
      const int r = rank * rows + i / (DP / 4), c = i % (DP / 4) * 4;
      if (r >= nr || c >= a.D) continue;
      float mx = -INFINITY, sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int x = 0; x < a.ranks; ++x) mx = fmaxf(mx, cluster.map_shared_rank(V, x)[r]);
      const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
      for (int x = 0; x < a.ranks; ++x) {
        const float* ml = cluster.map_shared_rank(V, x);
        const float f = exp2f((ml[r] - base) * kLog2e);
        const float4 y = *reinterpret_cast<const float4*>(cluster.map_shared_rank(K, x) + r * (DP + 4) + c);
        sum = fmaf(f, ml[kM + r], sum);
        o[0] = fmaf(f, y.x, o[0]), o[1] = fmaf(f, y.y, o[1]);
        o[2] = fmaf(f, y.z, o[2]), o[3] = fmaf(f, y.w, o[3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.D)
          static_cast<T*>(a.o)[((tok + r) * a.H + h) * a.D + c + e] = from_f32<T>(sum == 0.f ? 0.f : o[e] / sum);
      if (c == 0) a.lse[((long long)t.b * a.H + h) * a.sq.Tq + t.q0 + r0 + r] = sum == 0.f ? -INFINITY : mx + logf(sum);
    }
    cluster.sync();  // the others still read this CTA's shared memory
    return;
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

// dk and dv of a key tile
template <typename T, int DP>
__device__ __forceinline__ void bwd_kv(const Args& a, float* sm, int slot, int hk, int rank) {
  constexpr int n = tile_floats<DP>();
  float *K = sm, *V = K + n, *Q = V + n, *dO = Q + n, *P = dO + n, *S = P + kM * kLdP;
  float *lse = S + kM * kLdP, *delta = lse + kM;
  AttnTile t;
  if (!a.sq.get<true>(slot, kM, t)) return;  // the whole cluster
  const int G = a.H / a.Hkv, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int j0 = t.tile * kM, shift = t.lk - t.lq;
  load_tile<T, DP>(K, static_cast<const T*>(a.k) + t.b * a.ks[0] + (long long)(t.k0 + j0) * a.ks[1] + hk * a.ks[2],
                   a.ks[1], t.lk - j0, a.D, a.vec);
  load_tile<T, DP>(V, static_cast<const T*>(a.v) + t.b * a.vs[0] + (long long)(t.k0 + j0) * a.vs[1] + hk * a.vs[2],
                   a.vs[1], t.lk - j0, a.D, a.vec);
  float dk[4][DP / 16], dv[4][DP / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) dk[i][c] = dv[i][c] = 0.f;
  // the query tiles that see the tile, of each of the G heads
  const int first = max(0, j0 - shift) / kM, per = max(0, (t.lq + kM - 1) / kM - first);
  const int x0 = (int)((long long)G * per * rank / a.ranks), x1 = (int)((long long)G * per * (rank + 1) / a.ranks);
  int h = hk * G + (per ? x0 / per : 0), tile = first + (per ? x0 % per : 0);
  for (int x = x0; x < x1; ++x) {
    const long long st = ((long long)t.b * a.H + h) * a.sq.Tq + t.q0;
    const int r0 = tile * kM, nr = min(kM, t.lq - r0);
    __syncthreads();
    load_tile<T, DP>(Q, static_cast<const T*>(a.q) + t.b * a.qs[0] + (long long)(t.q0 + r0) * a.qs[1] + h * a.qs[2],
                     a.qs[1], nr, a.D, a.vec);
    load_tile<T, DP>(dO, static_cast<const T*>(a.do_) + (((long long)t.b * a.sq.Tq + t.q0 + r0) * a.H + h) * a.D,
                     (long long)a.H * a.D, nr, a.D, a.vec);
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
    if (++tile == first + per) ++h, tile = first;
  }
  if (a.ranks > 1) {
    __syncthreads();
    park<DP>(Q, dk, 4 * ty, 1, tx);
    park<DP>(dO, dv, 4 * ty, 1, tx);
    cg::this_cluster().sync();
    const long long at = (((long long)t.b * a.sq.Tk + t.k0 + j0) * a.Hkv + hk) * a.D;
    join_rows<T, DP>(static_cast<T*>(a.dk) + at, (long long)a.Hkv * a.D, Q, a.scale, t.lk - j0, a.D, rank, a.ranks);
    join_rows<T, DP>(static_cast<T*>(a.dv) + at, (long long)a.Hkv * a.D, dO, 1.f, t.lk - j0, a.D, rank, a.ranks);
    cg::this_cluster().sync();  // the others still read this CTA's shared memory
    return;
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

// dq of a query tile
template <typename T, int DP>
__device__ __forceinline__ void bwd_q(const Args& a, float* sm, int slot, int h, int rank) {
  constexpr int n = tile_floats<DP>();
  float *K = sm, *V = K + n, *Q = V + n, *dO = Q + n, *S = dO + n;
  float *lse = S + kM * kLdP, *delta = lse + kM;
  AttnTile t;
  if (!a.sq.get<false>(slot, kM, t)) return;  // the whole cluster
  const int hk = h / (a.H / a.Hkv), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int r0 = t.tile * kM, nr = min(kM, t.lq - r0), shift = t.lk - t.lq;
  const long long st = ((long long)t.b * a.H + h) * a.sq.Tq + t.q0 + r0;
  const long long tok = (long long)t.b * a.sq.Tq + t.q0 + r0;
  load_tile<T, DP>(Q, static_cast<const T*>(a.q) + t.b * a.qs[0] + (long long)(t.q0 + r0) * a.qs[1] + h * a.qs[2],
                   a.qs[1], nr, a.D, a.vec);
  load_tile<T, DP>(dO, static_cast<const T*>(a.do_) + (tok * a.H + h) * a.D, (long long)a.H * a.D, nr, a.D, a.vec);
  if (threadIdx.x < nr) lse[threadIdx.x] = a.lse[st + threadIdx.x], delta[threadIdx.x] = a.delta[st + threadIdx.x];
  else if (threadIdx.x < kM) lse[threadIdx.x] = 0.f, delta[threadIdx.x] = 0.f;
  float dq[4][DP / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) dq[i][c] = 0.f;
  const int nk = min(t.lk, r0 + nr + shift);
  const int steps = (max(0, nk) + kM - 1) / kM, end = steps * (rank + 1) / a.ranks;
  for (int step = steps * rank / a.ranks; step < end; ++step) {
    const int j0 = step * kM;
    __syncthreads();
    load_tile<T, DP>(K, static_cast<const T*>(a.k) + t.b * a.ks[0] + (long long)(t.k0 + j0) * a.ks[1] + hk * a.ks[2],
                     a.ks[1], t.lk - j0, a.D, a.vec);
    load_tile<T, DP>(V, static_cast<const T*>(a.v) + t.b * a.vs[0] + (long long)(t.k0 + j0) * a.vs[1] + hk * a.vs[2],
                     a.vs[1], t.lk - j0, a.D, a.vec);
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
  if (a.ranks > 1) {
    __syncthreads();
    park<DP>(V, dq, ty, 16, tx);
    cg::this_cluster().sync();
    join_rows<T, DP>(static_cast<T*>(a.dq) + (tok * a.H + h) * a.D, (long long)a.H * a.D, V, a.scale, nr, a.D, rank,
                     a.ranks);
    cg::this_cluster().sync();  // the others still read this CTA's shared memory
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    if (r < nr) store_row<T, DP>(static_cast<T*>(a.dq) + ((tok + r) * a.H + h) * a.D, dq[i], a.scale, tx, a.D);
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attn_simt_bwd_kernel(Args a, int key_slots, int query_slots) {
  extern __shared__ __align__(16) float sm[];
  const int slot = blockIdx.x / a.ranks, rank = blockIdx.x % a.ranks;
  if (blockIdx.x + blockIdx.y + blockIdx.z == 0 && !a.sq.valid() && threadIdx.x == 0)
    atomicExch(&tc::g_file_status, GDN_ERR_SEQLENS);
  if (blockIdx.z == 0) {  // the role with more work first
    if (slot < key_slots && blockIdx.y < a.Hkv) bwd_kv<T, DP>(a, sm, slot, blockIdx.y, rank);
  } else if (slot < query_slots) {
    bwd_q<T, DP>(a, sm, slot, blockIdx.y, rank);
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

template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int smem, cudaStream_t s, int id, const Args& a, A... more) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.ranks, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid, cfg.blockDim = dim3(kThreads), cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  prof_before(s);
  e = cudaLaunchKernelEx(&cfg, kernel, a, more...);
  prof_after(s, id);
  return e;
}

// CTAs that share a job: as many as it takes for the longest walk (in tiles) not
// to outlast an even share of all the walks, `work`, over the CTAs that fit (two
// on an SM for D <= 64, one above); no more than there are tiles, plus one.
// Measured (fp32, us with 1, 2, 4, 8 CTAs, * the choice).  Forward: 2 x 333 tokens,
// 4 heads, D 64: 42, 30, 31*, 36; 1200 tokens, 4 heads: 114, 72, 57*, 61; 4 x 300,
// 16 heads: 52*, 72, 86, 131.  Backward: 2 x 333, 4 heads on 2: 133, 90, 51, 53*;
// 1200, 16 on 4: 874, 491, 371*, 424; 2048, 8 on 2, D 128: 2002, 1016, 967*, 1245.
int ranks_of(const AttnProblem& p, float longest, float work) {
  const float even = work / (float)(tc::sm_count() * (p.D <= 64 ? 2 : 1));
  int ranks = 1;
  while (ranks < 8 && longest / ranks > even && 2 * ranks <= longest + 1) ranks *= 2;
  return ranks;
}

// the mean sequence's tiles
float mean_tiles(const AttnProblem& p, int T) {
  return std::max(1.f, ceilf((float)T / (p.cu_q ? std::max(1, p.nseq) : 1) / kM));
}

template <typename T, int DP>
cudaError_t fwd(const AttnProblem& p, cudaStream_t s) {
  const int smem = (3 * tile_floats<DP>() + kM * kLdP) * 4;
  const long slots = AttnSeqs::slots(p, kM, false);
  Args a = args_of(p);
  // half of the tiles are seen on average; a join costs about as much as a step, so
  // only walks of twice the even share are cut
  const float tiles = mean_tiles(p, p.Tk);
  a.ranks = ranks_of(p, tiles, (float)slots * p.H * tiles);
  return launch(attn_simt_fwd_kernel<T, DP>, dim3((unsigned)(slots * a.ranks), p.H), smem, s, kAttnFwd, a);
}

template <typename T, int DP>
cudaError_t bwd(const AttnProblem& p, cudaStream_t s) {
  const cudaError_t e = attn_delta(p, s);
  const long keys = p.Tk > 0 ? AttnSeqs::slots(p, kM, true) : 0, queries = p.Tq > 0 ? AttnSeqs::slots(p, kM, false) : 0;
  if (e != cudaSuccess || std::max(keys, queries) == 0) return e;
  Args a = args_of(p);
  // a key tile's walk is over the queries of all heads that share the key head
  const float tk = mean_tiles(p, p.Tk), tq = mean_tiles(p, p.Tq) * p.H / p.Hkv;
  a.ranks = ranks_of(p, std::max(tk, tq), ((float)keys * p.Hkv * tq + (float)queries * p.H * tk) / 2);
  const int smem = (4 * tile_floats<DP>() + 2 * kM * kLdP + 2 * kM) * 4;
  return launch(attn_simt_bwd_kernel<T, DP>, dim3((unsigned)(std::max(keys, queries) * a.ranks), p.H, 2), smem, s,
                kAttnBwd, a, (int)keys, (int)queries);
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
