// Layer norm over rows of D values, forward and backward.
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),
//   xh = (x - mean) rstd,  y = xh w + b
//   dx = rstd (w dy - mean(w dy) - xh mean(w dy xh)),
//   dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by memory: 2 e bytes per value forward, 3 e backward.  A row is read
// once, in 16-byte vectors, and stays in the registers of the warps that own
// it (1 to 16, chosen by D so that a lane holds at most NV vectors), with the
// next row's vectors already on their way; w and b, and in the backward the
// lane's columns of the dw and db sums, stay in registers over all rows of a
// warp group.  Sums are fp32, the variance is taken about the mean (the row is
// at hand: no E[x^2] - mean^2).  dw and db are summed per CTA, in row order,
// and a second kernel adds the CTAs' sums in order, so results do not depend
// on the order in which CTAs run.  Rows that are no whole number of vectors,
// or too long for that, take the plain kernels (one CTA per row, the row read
// again from L1 / L2 for each pass).  Measured, 32768 rows of 1024, bf16: forward
// 28 us (4.8 TB/s), backward 33 us (6.1 TB/s) and 3 us for the join.

#include <math.h>

#include <algorithm>

#include "attn_tc.cuh"

namespace gdn {
namespace {

constexpr int kMaxCtas = 608;

struct Args {
  long rows;
  int D, groups;  // groups: row groups of the grid
  float eps, d;  // d: D (divided by, so that the mean of equal values is exact)
  const void* x;
  const float *w, *b;
  void* y;
  float *mean, *rstd;
  const void* dy;
  void* dx;
  float *pw, *pb;  // [ctas][D] sums
};

// 16 bytes of T as floats
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);
__device__ __forceinline__ void widen(const uint4& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void widen(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
}
__device__ __forceinline__ uint4 narrow(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  return make_uint4(tc::pack_bf16(f[0], f[1]), tc::pack_bf16(f[2], f[3]), tc::pack_bf16(f[4], f[5]),
                    tc::pack_bf16(f[6], f[7]));
}
// read once, written once: no place in L1
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float2 warp_sum(float2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

// Sum over the W warps of a row group; red: W slots of the group, used in turn
// (two sets: a set is rewritten only after the barrier of the next call).
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float2 plus(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
template <int W, typename X>
__device__ __forceinline__ X group_sum(X v, X* red, int group, int w, int& turn) {
  v = warp_sum(v);
  if constexpr (W > 1) {
    X* r = red + turn * 16;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) r[w] = v;
    tc::group_sync(1 + group, W * 32);
    v = r[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v = plus(v, r[i]);
  }
  return v;
}

// Threads per SM and rows on their way, by measurement at 32768 x 1024 bf16:
// forward 512 threads and 3 rows (1: 2 us more; 640 threads: 9 us more, the
// registers no longer suffice), backward 512 and 1 (2: 4 us more; 384: 5 us).
constexpr int kFwdThreads = 512, kBwdThreads = 512;
constexpr int kAhead = 3, kAheadBwd = 1;
constexpr int ctas_per_sm(int threads, int cta) { return threads < cta ? 1 : threads / cta; }

template <int W>
constexpr int kGroups = W >= 4 ? 1 : 4 / W;  // row groups per CTA

template <typename T, int W, int NV>
__global__ void __launch_bounds__(32 * W * kGroups<W>, ctas_per_sm(kFwdThreads, 32 * W * kGroups<W>)) ln_fwd_vec_kernel(Args a) {
  constexpr int V = kVec<T>;
  __shared__ float red[kGroups<W>][32];
  const int warp = threadIdx.x >> 5, group = warp / W, w = warp % W, l = w * 32 + (threadIdx.x & 31);
  const int nvec = a.D / V, step = gridDim.x * kGroups<W>;
  float wt[NV][V], bs[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = (l + i * 32 * W) * V + e;
      wt[i][e] = c < a.D ? a.w[c] : 0.f;
      bs[i][e] = c < a.D && a.b ? a.b[c] : 0.f;
    }
  int turn = 0;
  uint4 next[kAhead][NV];
  auto fetch = [&](uint4(&v)[NV], long r) {
    const T* x = static_cast<const T*>(a.x) + r * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      v[i] = r < a.rows && l + i * 32 * W < nvec ? load_once(x + (l + i * 32 * W) * V) : make_uint4(0, 0, 0, 0);
  };
  long r = (long)blockIdx.x * kGroups<W> + group;
#pragma unroll
  for (int d = 0; d < kAhead; ++d) fetch(next[d], r + d * step);
  for (; r < a.rows; r += step) {
    float x[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) widen(next[0][i], x[i]);
#pragma unroll
    for (int d = 0; d + 1 < kAhead; ++d)
#pragma unroll
      for (int i = 0; i < NV; ++i) next[d][i] = next[d + 1][i];
    fetch(next[kAhead - 1], r + kAhead * step);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) s += x[i][e];
    const float mean = group_sum<W>(s, red[group], group, w, turn) / a.d;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = l + i * 32 * W < nvec;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[i][e] -= mean;
        if (in) s = fmaf(x[i][e], x[i][e], s);
      }
    }
    const float rstd = 1.f / sqrtf(group_sum<W>(s, red[group], group, w, turn) / a.d + a.eps);
    T* y = static_cast<T*>(a.y) + r * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(x[i][e] * rstd, wt[i][e], bs[i][e]);
      if (l + i * 32 * W < nvec) *reinterpret_cast<uint4*>(y + (l + i * 32 * W) * V) = narrow(o);
    }
    if (l == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

template <typename T, int W, int NV>
__global__ void __launch_bounds__(32 * W * kGroups<W>, ctas_per_sm(kBwdThreads, 32 * W * kGroups<W>)) ln_bwd_vec_kernel(Args a) {
  constexpr int V = kVec<T>, G = kGroups<W>;
  __shared__ float2 red[G][32];
  extern __shared__ float sums[];  // G > 1: [G][D]
  tc::grid_dep_launch();
  const int warp = threadIdx.x >> 5, group = warp / W, w = warp % W, l = w * 32 + (threadIdx.x & 31);
  const int nvec = a.D / V, step = gridDim.x * G;
  float wt[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = (l + i * 32 * W) * V + e;
      wt[i][e] = c < a.D ? a.w[c] : 0.f;
      dw[i][e] = db[i][e] = 0.f;
    }
  int turn = 0;
  uint4 nx[kAheadBwd][NV], ng[kAheadBwd][NV];
  float nm[kAheadBwd] = {}, nr[kAheadBwd] = {};
  auto fetch = [&](int d, long r) {
    const T *x = static_cast<const T*>(a.x) + r * a.D, *g = static_cast<const T*>(a.dy) + r * a.D;
    if (r < a.rows) nm[d] = a.mean[r], nr[d] = a.rstd[r];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = r < a.rows && l + i * 32 * W < nvec;
      nx[d][i] = in ? load_once(x + (l + i * 32 * W) * V) : make_uint4(0, 0, 0, 0);
      ng[d][i] = in ? load_once(g + (l + i * 32 * W) * V) : make_uint4(0, 0, 0, 0);
    }
  };
  long r = (long)blockIdx.x * G + group;
#pragma unroll
  for (int d = 0; d < kAheadBwd; ++d) fetch(d, r + d * step);
  for (; r < a.rows; r += step) {
    float x[NV][V], g[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) widen(nx[0][i], x[i]), widen(ng[0][i], g[i]);
    const float mean = nm[0], rstd = nr[0];
#pragma unroll
    for (int d = 0; d + 1 < kAheadBwd; ++d) {
      nm[d] = nm[d + 1], nr[d] = nr[d + 1];
#pragma unroll
      for (int i = 0; i < NV; ++i) nx[d][i] = nx[d + 1][i], ng[d][i] = ng[d + 1][i];
    }
    fetch(kAheadBwd - 1, r + kAheadBwd * step);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[i][e] = (x[i][e] - mean) * rstd;
        dw[i][e] = fmaf(g[i][e], x[i][e], dw[i][e]);  // past the row's end g is 0
        db[i][e] += g[i][e];
        g[i][e] *= wt[i][e];
        s.x += g[i][e], s.y = fmaf(g[i][e], x[i][e], s.y);
      }
    s = group_sum<W>(s, red[group], group, w, turn);
    const float m0 = s.x / a.d, m1 = s.y / a.d;
    T* dx = static_cast<T*>(a.dx) + r * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = rstd * (g[i][e] - m0 - x[i][e] * m1);
      if (l + i * 32 * W < nvec) *reinterpret_cast<uint4*>(dx + (l + i * 32 * W) * V) = narrow(o);
    }
  }
  // the CTA's sums: its groups', in order
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float(&d)[NV][V] = q ? db : dw;
    float* out = (q ? a.pb : a.pw) + (long)blockIdx.x * a.D;
    if constexpr (G == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; e += 4)
          if (l + i * 32 * W < nvec)
            *reinterpret_cast<float4*>(out + (l + i * 32 * W) * V + e) =
                make_float4(d[i][e], d[i][e + 1], d[i][e + 2], d[i][e + 3]);
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; e += 4)
          if (l + i * 32 * W < nvec)
            *reinterpret_cast<float4*>(sums + group * a.D + (l + i * 32 * W) * V + e) =
                make_float4(d[i][e], d[i][e + 1], d[i][e + 2], d[i][e + 3]);
      __syncthreads();
      for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
        float t = sums[c];
#pragma unroll
        for (int k = 1; k < G; ++k) t += sums[k * a.D + c];
        out[c] = t;
      }
    }
  }
}

// ---------------------------------------------------------------- any D

constexpr int kThreads = 256;

// sum over the CTA of two values
__device__ __forceinline__ float2 cta_sum(float2 v, float2* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s.x += red[i].x, s.y += red[i].y;
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) ln_fwd_kernel(Args a) {
  __shared__ float2 red[kThreads / 32];
  for (long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.D;
    T* y = static_cast<T*>(a.y) + r * a.D;
    float s = 0.f;
    for (int c = threadIdx.x; c < a.D; c += kThreads) s += to_f32(x[c]);
    const float mean = cta_sum(make_float2(s, 0.f), red).x / a.d;
    s = 0.f;
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      const float d = to_f32(x[c]) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = 1.f / sqrtf(cta_sum(make_float2(s, 0.f), red).x / a.d + a.eps);
    for (int c = threadIdx.x; c < a.D; c += kThreads)
      y[c] = from_f32<T>(fmaf((to_f32(x[c]) - mean) * rstd, a.w[c], a.b ? a.b[c] : 0.f));
    if (threadIdx.x == 0 && a.mean) a.mean[r] = mean;
    if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rstd;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) ln_bwd_kernel(Args a) {
  __shared__ float2 red[kThreads / 32];
  tc::grid_dep_launch();
  float *pw = a.pw + (long)blockIdx.x * a.D, *pb = a.pb + (long)blockIdx.x * a.D;
  for (int c = threadIdx.x; c < a.D; c += kThreads) pw[c] = pb[c] = 0.f;
  for (long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T *x = static_cast<const T*>(a.x) + r * a.D, *dy = static_cast<const T*>(a.dy) + r * a.D;
    T* dx = static_cast<T*>(a.dx) + r * a.D;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float2 s = make_float2(0.f, 0.f);
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      const float g = to_f32(dy[c]), xh = (to_f32(x[c]) - mean) * rstd, wg = g * a.w[c];
      s.x += wg, s.y = fmaf(wg, xh, s.y);
      pw[c] = fmaf(g, xh, pw[c]);  // a thread owns its columns
      pb[c] += g;
    }
    s = cta_sum(s, red);
    const float m0 = s.x / a.d, m1 = s.y / a.d;
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      const float xh = (to_f32(x[c]) - mean) * rstd;
      dx[c] = from_f32<T>(rstd * (to_f32(dy[c]) * a.w[c] - m0 - xh * m1));
    }
  }
}

// out[c] = sum over n CTAs of part[i][c]: 16 threads per column, each over every
// 16th CTA in order, then over the 16 in order; grid.y 0: dw, 1: db.
__global__ void __launch_bounds__(512) ln_sum_kernel(const float* pw, const float* pb, float* dw, float* db,
                                                     int n, int D) {
  __shared__ float s[16][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  const float* part = blockIdx.y ? pb : pw;
  float* out = blockIdx.y ? db : dw;
  tc::grid_dep_wait();
  if (!out) return;
  float t = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int i = y; i < n; i += 16) t += part[(long)i * D + c];
  }
  s[y][x] = t;
  __syncthreads();
  if (y == 0 && c < D) {
#pragma unroll
    for (int i = 1; i < 16; ++i) t += s[i][x];
    out[c] = t;
  }
}

// ---------------------------------------------------------------- host

// Warps per row of the vector kernels for nv vectors a lane; 0: the row is no
// whole number of vectors or takes more than 16 warps.
int warps_per_row(int D, int vec, int nv) {
  if (D % vec) return 0;
  for (int w = 1; w <= 16; w *= 2)
    if (D / vec <= 32 * w * nv) return w;
  return 0;
}

int groups_of(int w) { return w >= 4 ? 1 : 4 / w; }

// CTAs of the backward (each leaves a row of sums): as many as run at once,
// four 128-thread CTAs per SM or the same threads in larger ones.
int bwd_ctas(long rows, int D, bool bf16) {
  const int w = warps_per_row(D, bf16 ? 8 : 4, 2), g = w ? groups_of(w) : 1;
  const long per_sm = w ? ctas_per_sm(kBwdThreads, 32 * w * g) : 4;
  return (int)std::max(1L, std::min({(rows + g - 1) / g, per_sm * tc::sm_count(), (long)kMaxCtas}));
}

Args args_of(const LayerNormProblem& p) {
  Args a = {};
  a.rows = p.rows, a.D = p.D, a.eps = p.eps, a.d = (float)p.D, a.x = p.x, a.w = p.weight, a.b = p.bias, a.y = p.y;
  a.mean = p.mean, a.rstd = p.rstd, a.dy = p.dy, a.dx = p.dx;
  a.pw = static_cast<float*>(p.ws);
  a.pb = a.pw + (size_t)bwd_ctas(p.rows, p.D, p.bf16) * p.D;
  return a;
}

template <typename T, int W>
void fwd(const Args& a, cudaStream_t s) {
  const long n = (a.rows + kGroups<W> - 1) / kGroups<W>;
  const unsigned grid = (unsigned)std::min(n, (long)ctas_per_sm(kFwdThreads, 32 * W * kGroups<W>) * tc::sm_count());
  ln_fwd_vec_kernel<T, W, 2><<<grid, 32 * W * kGroups<W>, 0, s>>>(a);
}

template <typename T>
cudaError_t run_fwd(const LayerNormProblem& p, cudaStream_t s) {
  const Args a = args_of(p);
  prof_before(s);
  switch (warps_per_row(p.D, kVec<T>, 2)) {
    case 1: fwd<T, 1>(a, s); break;
    case 2: fwd<T, 2>(a, s); break;
    case 4: fwd<T, 4>(a, s); break;
    case 8: fwd<T, 8>(a, s); break;
    case 16: fwd<T, 16>(a, s); break;
    default: ln_fwd_kernel<T><<<(unsigned)std::min(p.rows, 65535L), kThreads, 0, s>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  prof_after(s, kLnFwd);
  return e;
}

template <typename T, int W>
void bwd(const Args& a, int ctas, cudaStream_t s) {
  const size_t smem = kGroups<W> > 1 ? (size_t)kGroups<W> * a.D * sizeof(float) : 0;  // at most 16 KB
  ln_bwd_vec_kernel<T, W, 2><<<ctas, 32 * W * kGroups<W>, smem, s>>>(a);
}

template <typename T>
cudaError_t run_bwd(const LayerNormProblem& p, cudaStream_t s) {
  const Args a = args_of(p);
  const int n = bwd_ctas(p.rows, p.D, p.bf16);
  prof_before(s);
  switch (warps_per_row(p.D, kVec<T>, 2)) {
    case 1: bwd<T, 1>(a, n, s); break;
    case 2: bwd<T, 2>(a, n, s); break;
    case 4: bwd<T, 4>(a, n, s); break;
    case 8: bwd<T, 8>(a, n, s); break;
    case 16: bwd<T, 16>(a, n, s); break;
    default: ln_bwd_kernel<T><<<n, kThreads, 0, s>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  prof_after(s, kLnBwd);
  if (e != cudaSuccess) return e;
  prof_before(s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.D + 31) / 32, p.dbias ? 2 : 1);
  cfg.blockDim = dim3(512);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, ln_sum_kernel, (const float*)a.pw, (const float*)a.pb, p.dweight, p.dbias, n, p.D);
  prof_after(s, kLnSum);
  return e;
}

}  // namespace

size_t layer_norm_bwd_workspace(const LayerNormProblem& p) {
  return (size_t)2 * bwd_ctas(p.rows, p.D, p.bf16) * p.D * sizeof(float);
}

cudaError_t layer_norm_fwd(const LayerNormProblem& p, cudaStream_t s) {
  return p.bf16 ? run_fwd<__nv_bfloat16>(p, s) : run_fwd<float>(p, s);
}

cudaError_t layer_norm_bwd(const LayerNormProblem& p, cudaStream_t s) {
  return p.bf16 ? run_bwd<__nv_bfloat16>(p, s) : run_bwd<float>(p, s);
}

}  // namespace gdn
