// Attention of a few new tokens per row against a cache that the call extends
// (single-token generation).
//
// Row b holds n = lens[b] tokens; the T new tokens go to slots n .. n+T-1 and
// new token t attends to the slots j <= n + t:
//   o = sum_j exp(scale q . k_j - m) v_j / sum_j exp(scale q . k_j - m).
// The G = H / Hkv query heads of a key head and the T tokens are the rows of
// one product with the cache, so the used part of the cache is read once per
// row block.  The n + T slots of a row are split into parts of whole key
// tiles; a part keeps the running maximum m, sum l and accumulator over its
// tiles and writes them (fp32) to the workspace, where a second kernel joins
// them: m = max m_p, o = sum exp(m_p - m) acc_p / sum exp(m_p - m) l_p.  With
// one part per row the result is written directly.  Bound by the cache's
// bytes: 2 Hkv D (n + T) elements per row.
//
// The new tokens' k and v are read from the call's inputs, never from the
// cache; the part that owns their slots writes them there.  No CTA reads a
// slot that another one writes.

#include <math.h>

#include <algorithm>

#include "attn.cuh"
#include "tc_common.cuh"

namespace gdn {

cudaError_t attn_decode_read_and_clear_status(int* status) {
  return tc::read_and_clear_file_status(status);
}

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxParts = 256;

struct Args {
  int B, T, S, H, Hkv, D, G, R;  // R = G T rows per key head
  int parts, tile;               // parts per row; keys per tile
  float scale;
  long long kcs[3], vcs[3];
  const void *q, *k, *v;
  void *kc, *vc;
  const int* lens;
  void* o;
  float *acc, *ml;  // workspace: [b, hkv, row][part][D] and [..][part][2] (maximum, sum)
};

// Row b's tokens after the call (0: bad length, nothing is done) and the
// slots [j0, j1) of part p: whole tiles, spread evenly.
__device__ __forceinline__ int row_keys(const Args& a, int b) {
  const int n = a.lens[b];
  return n < 0 || n > a.S - a.T ? 0 : n + a.T;
}
__device__ __forceinline__ void part_range(const Args& a, int keys, int p, int& j0, int& j1) {
  const int tiles = (keys + a.tile - 1) / a.tile, per = (tiles + a.parts - 1) / a.parts;
  j0 = min(keys, p * per * a.tile), j1 = min(keys, (p + 1) * per * a.tile);
}

// ---------------------------------------------------------------- CUDA cores
//
// Any dtype and D: 4 warps, tiles of 32 keys in shared memory as fp32, 8 query
// rows per CTA (two per warp).  A lane owns one key of the scores and DP / 32
// columns of the accumulators.
constexpr int kRows = 8, kKeys = 32;

template <typename T, int DP>
__global__ void __launch_bounds__(128) attn_decode_simt_kernel(Args a) {
  constexpr int LD = DP + 4, NC = DP / 32;
  __shared__ float K[kKeys * LD], V[kKeys * LD], Q[kRows * DP];
  const int p = blockIdx.x, b = blockIdx.y / a.Hkv, hk = blockIdx.y % a.Hkv, row0 = blockIdx.z * kRows;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int keys = row_keys(a, b), old = keys - a.T;
  if (keys == 0 && p == 0 && hk == 0 && row0 == 0 && threadIdx.x == 0)
    atomicExch(&tc::g_file_status, GDN_ERR_SEQLENS);
  int j0, j1;
  part_range(a, keys, p, j0, j1);
  for (int i = threadIdx.x; i < kRows * DP; i += 128) {
    const int r = row0 + i / DP, c = i % DP;  // row r: token r / G, head hk G + r % G
    Q[i] = r < a.R && c < a.D
               ? to_f32(static_cast<const T*>(a.q)[(((long long)b * a.T + r / a.G) * a.H + hk * a.G + r % a.G) * a.D + c])
               : 0.f;
  }
  T* kc = static_cast<T*>(a.kc) + b * a.kcs[0] + hk * a.kcs[2];
  T* vc = static_cast<T*>(a.vc) + b * a.vcs[0] + hk * a.vcs[2];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[2][NC] = {};
  for (int t0 = j0; t0 < j1; t0 += kKeys) {
    __syncthreads();
    for (int i = threadIdx.x; i < kKeys * DP; i += 128) {
      const int r = i / DP, c = i % DP, j = t0 + r;
      float x = 0.f, y = 0.f;
      if (j < j1 && c < a.D) {
        if (j < old) {
          x = to_f32(kc[j * a.kcs[1] + c]), y = to_f32(vc[j * a.vcs[1] + c]);
        } else {
          const long long at = (((long long)b * a.T + j - old) * a.Hkv + hk) * a.D + c;
          const T kx = static_cast<const T*>(a.k)[at], vx = static_cast<const T*>(a.v)[at];
          if (blockIdx.z == 0) kc[j * a.kcs[1] + c] = kx, vc[j * a.vcs[1] + c] = vx;
          x = to_f32(kx), y = to_f32(vx);
        }
      }
      K[r * LD + c] = x, V[r * LD + c] = y;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row0 + w + 4 * i;
      const float* q = Q + (w + 4 * i) * DP;
      float s = 0.f;
#pragma unroll 8
      for (int d = 0; d < DP; d += 4) {
        const float4 x = *reinterpret_cast<const float4*>(K + lane * LD + d);
        const float4 y = *reinterpret_cast<const float4*>(q + d);
        s = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
      }
      const bool see = t0 + lane < j1 && t0 + lane <= old + r / a.G && r < a.R;
      s = see ? s * a.scale : -INFINITY;
      float mx = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = fmaxf(mx, m[i]);
      const float base = mx == -INFINITY ? 0.f : mx;
      const float f = exp2f((m[i] - base) * kLog2e), e = exp2f((s - base) * kLog2e);
      float sum = e;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[i] = l[i] * f + sum;
      m[i] = mx;
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[i][c] *= f;
      const int last = min(kKeys, min(j1 - t0, old + r / a.G - t0 + 1));  // keys the row sees
      for (int j = 0; j < last; ++j) {
        const float pj = __shfl_sync(0xffffffffu, e, j);
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[i][c] = fmaf(pj, V[j * LD + lane + 32 * c], acc[i][c]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row0 + w + 4 * i;
    if (r >= a.R) continue;
    if (a.parts == 1) {
      T* o = static_cast<T*>(a.o) + (((long long)b * a.T + r / a.G) * a.H + hk * a.G + r % a.G) * a.D;
      const float f = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (lane + 32 * c < a.D) o[lane + 32 * c] = from_f32<T>(acc[i][c] * f);
    } else {
      const long long at = ((long long)blockIdx.y * a.R + r) * a.parts + p;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (lane + 32 * c < a.D) a.acc[at * a.D + lane + 32 * c] = acc[i][c];
      if (lane == 0) a.ml[2 * at] = m[i], a.ml[2 * at + 1] = l[i];
    }
  }
}

// One CTA of 128 threads per (b, hkv, row): joins the parts.
template <typename T>
__global__ void __launch_bounds__(128) attn_combine_kernel(Args a) {
  __shared__ float f[kMaxParts];
  __shared__ float red[8];
  const long long row = blockIdx.x;
  const int r = (int)(row % a.R), hk = (int)(row / a.R % a.Hkv), b = (int)(row / a.R / a.Hkv);
  const int c = threadIdx.x;
  const float* ml = a.ml + 2 * row * a.parts;
  float m = -INFINITY;
  for (int p = c; p < a.parts; p += 128) m = fmaxf(m, ml[2 * p]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((c & 31) == 0) red[c >> 5] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float base = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
  for (int p = c; p < a.parts; p += 128) {
    const float e = exp2f((ml[2 * p] - base) * kLog2e);
    f[p] = e;
    sum = fmaf(e, ml[2 * p + 1], sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((c & 31) == 0) red[4 + (c >> 5)] = sum;
  __syncthreads();
  sum = red[4] + red[5] + red[6] + red[7];
  if (c >= a.D) return;
  float x = 0.f;
  for (int p = 0; p < a.parts; ++p)  // an empty part's accumulator is zero
    x = fmaf(f[p], a.acc[(row * a.parts + p) * a.D + c], x);
  static_cast<T*>(a.o)[(((long long)b * a.T + r / a.G) * a.H + hk * a.G + r % a.G) * a.D + c] =
      from_f32<T>(sum == 0.f ? 0.f : x / sum);
}

// Parts per row: enough CTAs for two per SM, no part shorter than 256 slots of
// a full cache.
int num_parts(const AttnDecodeProblem& p, int row_block) {
  const long ctas = (long)p.B * p.Hkv * ((p.H / p.Hkv * p.T + row_block - 1) / row_block);
  const long want = (2L * tc::sm_count() + ctas - 1) / ctas;
  const long most = (p.S + 255) / 256;
  return (int)std::max(1L, std::min({want, most, (long)kMaxParts}));
}

Args args_of(const AttnDecodeProblem& p, int parts, int tile) {
  Args a;
  a.B = p.B, a.T = p.T, a.S = p.S, a.H = p.H, a.Hkv = p.Hkv, a.D = p.D, a.G = p.H / p.Hkv;
  a.R = a.G * p.T, a.parts = parts, a.tile = tile, a.scale = p.scale;
  for (int i = 0; i < 3; ++i) a.kcs[i] = p.kcs[i], a.vcs[i] = p.vcs[i];
  a.q = p.q, a.k = p.k, a.v = p.v, a.kc = p.kc, a.vc = p.vc, a.lens = p.lens, a.o = p.o;
  a.ml = static_cast<float*>(p.ws);
  a.acc = a.ml + align_up((size_t)2 * p.B * p.Hkv * a.R * parts, 4);
  return a;
}

template <typename T>
cudaError_t run(const AttnDecodeProblem& p, cudaStream_t s) {
  const int parts = num_parts(p, kRows);
  const Args a = args_of(p, parts, kKeys);
  const dim3 grid(parts, p.B * p.Hkv, (a.R + kRows - 1) / kRows);
  prof_before(s);
  if (p.D <= 64) attn_decode_simt_kernel<T, 64><<<grid, 128, 0, s>>>(a);
  else attn_decode_simt_kernel<T, 128><<<grid, 128, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  prof_after(s, kAttnDecode);
  if (e != cudaSuccess || parts == 1) return e;
  prof_before(s);
  attn_combine_kernel<T><<<(unsigned)((long)p.B * p.Hkv * a.R), 128, 0, s>>>(a);
  e = cudaGetLastError();
  prof_after(s, kAttnCombine);
  return e;
}

}  // namespace

size_t attn_decode_workspace(const AttnDecodeProblem& p) {
  const size_t parts = num_parts(p, kRows);
  if (parts == 1) return 0;
  const size_t rows = (size_t)p.B * p.H * p.T;
  return (align_up(2 * rows * parts, 4) + rows * parts * p.D) * sizeof(float);
}

cudaError_t attn_decode(const AttnDecodeProblem& p, cudaStream_t s) {
  return p.bf16 ? run<__nv_bfloat16>(p, s) : run<float>(p, s);
}

}  // namespace gdn
