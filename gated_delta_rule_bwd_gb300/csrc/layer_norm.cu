// Layer norm over rows of D values, forward and backward.
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),
//   xh = (x - mean) rstd,  y = xh w + b
//   dx = rstd (w dy - mean(w dy) - xh mean(w dy xh)),
//   dw = sum_rows dy xh,  db = sum_rows dy
//
// Sums are fp32; the variance is taken about the mean (a second pass over the
// row, not E[x^2] - mean^2).  dw and db are summed per CTA over its rows, in
// row order, and a second kernel adds the CTAs' sums in order.

#include <math.h>

#include "attn.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxCtas = 512;

struct Args {
  long rows;
  int D;
  float eps;
  const void* x;
  const float *w, *b;
  void* y;
  float *mean, *rstd;
  const void* dy;
  void* dx;
  float *pw, *pb;  // [ctas][D] sums
};

// sum over the CTA of two values (red: 2 x 32 floats)
__device__ __forceinline__ float2 cta_sum(float2 v, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
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
    const float mean = cta_sum(make_float2(s, 0.f), red).x / a.D;
    s = 0.f;
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      const float d = to_f32(x[c]) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = 1.f / sqrtf(cta_sum(make_float2(s, 0.f), red).x / a.D + a.eps);
    for (int c = threadIdx.x; c < a.D; c += kThreads)
      y[c] = from_f32<T>(fmaf((to_f32(x[c]) - mean) * rstd, a.w[c], a.b ? a.b[c] : 0.f));
    if (threadIdx.x == 0 && a.mean) a.mean[r] = mean;
    if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rstd;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) ln_bwd_kernel(Args a) {
  __shared__ float2 red[kThreads / 32];
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
    const float m0 = s.x / a.D, m1 = s.y / a.D;
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      const float xh = (to_f32(x[c]) - mean) * rstd;
      dx[c] = from_f32<T>(rstd * (to_f32(dy[c]) * a.w[c] - m0 - xh * m1));
    }
  }
}

// out[c] = sum over n CTAs of part[i][c], in order; grid.y 0: dw, 1: db
__global__ void __launch_bounds__(128) ln_sum_kernel(const float* pw, const float* pb, float* dw, float* db,
                                                     int n, int D) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  const float* part = blockIdx.y ? pb : pw;
  float* out = blockIdx.y ? db : dw;
  if (c >= D || !out) return;
  float s = 0.f;
  for (int i = 0; i < n; ++i) s += part[(long)i * D + c];
  out[c] = s;
}

int bwd_ctas(long rows) { return (int)(rows < kMaxCtas ? rows : kMaxCtas); }

Args args_of(const LayerNormProblem& p) {
  Args a = {};
  a.rows = p.rows, a.D = p.D, a.eps = p.eps, a.x = p.x, a.w = p.weight, a.b = p.bias, a.y = p.y;
  a.mean = p.mean, a.rstd = p.rstd, a.dy = p.dy, a.dx = p.dx;
  a.pw = static_cast<float*>(p.ws);
  a.pb = a.pw + (size_t)bwd_ctas(p.rows) * p.D;
  return a;
}

}  // namespace

size_t layer_norm_bwd_workspace(const LayerNormProblem& p) {
  return (size_t)2 * bwd_ctas(p.rows) * p.D * sizeof(float);
}

cudaError_t layer_norm_fwd(const LayerNormProblem& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(p.rows < 65535 ? p.rows : 65535);
  prof_before(s);
  if (p.bf16) ln_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(args_of(p));
  else ln_fwd_kernel<float><<<grid, kThreads, 0, s>>>(args_of(p));
  cudaError_t e = cudaGetLastError();
  prof_after(s, kLnFwd);
  return e;
}

cudaError_t layer_norm_bwd(const LayerNormProblem& p, cudaStream_t s) {
  const Args a = args_of(p);
  const int n = bwd_ctas(p.rows);
  prof_before(s);
  if (p.bf16) ln_bwd_kernel<__nv_bfloat16><<<n, kThreads, 0, s>>>(a);
  else ln_bwd_kernel<float><<<n, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  prof_after(s, kLnBwd);
  if (e != cudaSuccess) return e;
  prof_before(s);
  ln_sum_kernel<<<dim3((p.D + 127) / 128, 2), 128, 0, s>>>(a.pw, a.pb, p.dweight, p.dbias, n, p.D);
  e = cudaGetLastError();
  prof_after(s, kLnSum);
  return e;
}

}  // namespace gdn
