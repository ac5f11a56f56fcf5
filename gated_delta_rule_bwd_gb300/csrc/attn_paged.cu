// Attention of a few new tokens per row against pages of keys and values that
// hold them already (single-token generation from a paged cache).
//
// Row b holds lens[b] tokens and the T new ones; new token t attends to the
// slots j <= lens[b] + t:
//   o = sum_j exp(scale q . k_j - m) v_j / sum_j exp(scale q . k_j - m).
// Slot j lies at place j % page of page table[b][j / page].  The G = H / Hkv
// query heads of a key head and the T tokens are the R = G T rows of one product
// with the cache.  Work split: the batch's units of 64 keys evenly over the CTAs,
// and a second kernel that joins what is split (attn_split.cuh).

#include "attn_split.cuh"
#include "paged.cuh"

namespace gdn {

cudaError_t attn_paged_read_and_clear_status(int* status) { return tc::read_and_clear_file_status(status); }

namespace {

using namespace paged;
using namespace split;
using namespace tc;

struct Args {
  int B, T, S, H, Hkv, D, G, R;  // S = max_pages page; R = G T rows per key head
  int pages, shift;
  bool vec;                      // rows in vectors of four values
  float c;                       // scale log2 e
  long long table_stride;
  long long ks[3], vs[3], kss[3], vss[3];  // page, token, head
  const int *table, *lens;
  const void *q, *k, *v;
  const __nv_bfloat16 *k_scale, *v_scale;
  void* o;
  int4* starts;
  float *ml, *acc;
  // Row b's keys (0: not in use, or a bad length).
  __device__ __forceinline__ int keys(int b) const {
    const int n = lens[b];
    return n < 0 || n > S - T ? 0 : n + T;
  }
  // The page of row b's slot j, or -1 (reported): its keys count as zeros.
  __device__ __forceinline__ int page_of(int b, int j) const {
    const int n = table[b * table_stride + (j >> shift)];
    if ((unsigned)n < (unsigned)pages) return n;
    atomicExch(&g_file_status, GDN_ERR_PAGE);
    return -1;
  }
};

// Rows without keys: o = 0; the status word says so where the length is a bad one.
template <typename T>
__device__ void empty_rows(const Args& a) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (a.keys(b) || blockIdx.y) continue;
    const long long n = (long long)a.T * a.H * a.D;
    for (long long i = threadIdx.x; i < n; i += kThreads) static_cast<T*>(a.o)[b * n + i] = from_f32<T>(0.f);
    if (threadIdx.x == 0 && a.lens[b] >= 0) atomicExch(&g_file_status, GDN_ERR_SEQLENS);
  }
}

// ---------------------------------------------------------------- CUDA cores
//
// Any format and D: 4 warps, tiles of 32 keys in shared memory as fp32, 8 query
// rows per CTA (two per warp).  A lane owns one key of the scores and DP / 32
// columns of the accumulators.
constexpr int kRows = 8, kKeys = 32;

// Four values of a row from its value c on, or those of them that it has.
template <typename T>
__device__ __forceinline__ float4 four(const void* base, long long at, int c, int D, bool vec, const __nv_bfloat16*) {
  const T* p = static_cast<const T*>(base) + at + c;
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      return *reinterpret_cast<const float4*>(p);
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                         __uint_as_float(v.y & 0xffff0000u));
    }
  }
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = c + e < D ? to_f32(p[e]) : 0.f;
  return make_float4(x[0], x[1], x[2], x[3]);
}
struct I4 {};
template <>
__device__ __forceinline__ float4 four<I4>(const void* base, long long at, int c, int, bool, const __nv_bfloat16* step) {
  const uint32_t w = *reinterpret_cast<const uint16_t*>(static_cast<const unsigned char*>(base) + at + c / 2);
  const float s = __bfloat162float(step[c / kStepGroup]);
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = (float)((int)(w >> (4 * e) & 15) - 8) * s;
  return make_float4(x[0], x[1], x[2], x[3]);
}

// T: the queries' and output's type; C: the cache's (T or I4).
template <typename T, typename C, int DP>
__global__ void __launch_bounds__(kThreads) attn_paged_simt_kernel(Args a) {
  constexpr int LD = DP + 4, NC = DP / 32;
  __shared__ __align__(16) float K[kKeys * LD], V[kKeys * LD], Q[kRows * DP];
  __shared__ int page[kKeys];
  const int row0 = blockIdx.y * kRows, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_launch();
  empty_rows<T>(a);
  if (threadIdx.x == 0) a.starts[(long)blockIdx.y * gridDim.x + blockIdx.x].x = -1;
  Walk<Args> wk;
  if (!wk.init(a)) return;
  while (wk.segment(a)) {
    const int b = wk.b, hk = wk.hk, old = wk.keys - a.T;
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * DP; i += kThreads) {
      const int r = row0 + i / DP, c = i % DP;
      Q[i] = r < a.R && c < a.D ? to_f32(static_cast<const T*>(a.q)[row_at(a, b, hk, r) + c]) : 0.f;
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[2][NC] = {};
    for (int t0 = wk.k0; t0 < wk.k1; t0 += kKeys) {
      __syncthreads();
      if (threadIdx.x < kKeys) page[threadIdx.x] = t0 + threadIdx.x < wk.k1 ? a.page_of(b, t0 + threadIdx.x) : -1;
      __syncthreads();
      {
        const int c = threadIdx.x % (DP / 4) * 4;
#pragma unroll 4
        for (int r = threadIdx.x / (DP / 4); r < kKeys; r += kThreads / (DP / 4)) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
          const int p = page[r], at = (t0 + r) & ((1 << a.shift) - 1);
          if (p >= 0 && c < a.D) {
            const __nv_bfloat16 *xs = nullptr, *ys = nullptr;
            if constexpr (sizeof(C) == 1) {
              xs = a.k_scale + p * a.kss[0] + at * a.kss[1] + hk * a.kss[2];
              ys = a.v_scale + p * a.vss[0] + at * a.vss[1] + hk * a.vss[2];
            }
            x = four<C>(a.k, p * a.ks[0] + at * a.ks[1] + hk * a.ks[2], c, a.D, a.vec, xs);
            y = four<C>(a.v, p * a.vs[0] + at * a.vs[1] + hk * a.vs[2], c, a.D, a.vec, ys);
          }
          *reinterpret_cast<float4*>(K + r * LD + c) = x;
          *reinterpret_cast<float4*>(V + r * LD + c) = y;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row0 + w + 4 * i;
        if (r >= a.R) continue;
        const float* q = Q + (w + 4 * i) * DP;
        float s = 0.f;
#pragma unroll 8
        for (int d = 0; d < DP; d += 4) {
          const float4 x = *reinterpret_cast<const float4*>(K + lane * LD + d);
          const float4 y = *reinterpret_cast<const float4*>(q + d);
          s = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
        }
        const int last = min(wk.k1 - t0, old + r / a.G - t0 + 1);  // keys of the tile that the row sees
        s = lane < last ? s * a.c : -INFINITY;
        float mx = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = fmaxf(mx, m[i]);
        const float base = mx == -INFINITY ? 0.f : mx;
        const float f = exp2f(m[i] - base), e = exp2f(s - base);
        float sum = e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * f + sum;
        m[i] = mx;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[i][c] *= f;
        const int seen = max(0, min(last, kKeys));
        for (int j = 0; j < seen; ++j) {
          const float pj = __shfl_sync(0xffffffffu, e, j);
#pragma unroll
          for (int c = 0; c < NC; ++c) acc[i][c] = fmaf(pj, V[j * LD + lane + 32 * c], acc[i][c]);
        }
      }
    }
    const long slot = wk.whole ? 0 : slot_of(a, wk) * kRows;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row0 + w + 4 * i;
      if (r >= a.R) continue;
      if (wk.whole) {
        T* o = static_cast<T*>(a.o) + row_at(a, b, hk, r);
        const float f = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (lane + 32 * c < a.D) o[lane + 32 * c] = from_f32<T>(acc[i][c] * f);
      } else {
        const long at = slot + w + 4 * i;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (lane + 32 * c < a.D) a.acc[at * a.D + lane + 32 * c] = acc[i][c];
        if (lane == 0) a.ml[2 * at] = m[i], a.ml[2 * at + 1] = l[i];
      }
    }
  }
}

// ---------------------------------------------------------------- host

struct Plan {
  int rows, blocks, ctas;  // query rows per CTA, row blocks (grid.y), CTAs that share the units (grid.x)
};

Plan plan_of(const AttnPagedProblem& p, const PagedCache& c) {
  Plan q;
  const int R = p.H / c.Hkv * p.T;
  q.rows = kRows;
  q.blocks = (R + q.rows - 1) / q.rows;
  q.ctas = ctas_for(p.B, c.Hkv, (long)p.pt.max_pages * c.page, q.blocks, 4);
  return q;
}

template <typename T>
cudaError_t run(const AttnPagedProblem& p, const PagedCache& c, cudaStream_t s) {
  const Plan pl = plan_of(p, c);
  Args a = {};
  a.B = p.B, a.T = p.T, a.S = p.pt.max_pages * c.page, a.H = p.H, a.Hkv = c.Hkv, a.D = c.D, a.G = p.H / c.Hkv;
  a.R = a.G * p.T, a.c = p.scale * kLog2e;
  a.pages = c.pages, a.shift = page_shift(c.page);
  a.table = p.pt.table, a.table_stride = p.pt.stride, a.lens = p.lens;
  a.vec = c.D % 4 == 0 && !(((uintptr_t)c.k | (uintptr_t)c.v) & 15);
  for (int i = 0; i < 3; ++i) {
    a.ks[i] = c.ks[i], a.vs[i] = c.vs[i], a.kss[i] = c.kss[i], a.vss[i] = c.vss[i];
    a.vec = a.vec && c.ks[i] % 4 == 0 && c.vs[i] % 4 == 0;
  }
  a.q = p.q, a.k = c.k, a.v = c.v, a.o = p.o;
  a.k_scale = static_cast<const __nv_bfloat16*>(c.k_scale), a.v_scale = static_cast<const __nv_bfloat16*>(c.v_scale);
  unsigned char* ws = static_cast<unsigned char*>(p.ws);
  a.starts = reinterpret_cast<int4*>(ws);
  a.ml = reinterpret_cast<float*>(ws + ws_starts(pl.blocks, pl.ctas));
  a.acc = reinterpret_cast<float*>(ws + ws_starts(pl.blocks, pl.ctas) + ws_ml(pl.blocks, pl.ctas, pl.rows));
  const dim3 grid(pl.ctas, pl.blocks);
  const bool i4 = c.format == GDN_CACHE_I4;
  prof_before(s);
  if (c.D <= 64)
    i4 ? attn_paged_simt_kernel<T, I4, 64><<<grid, kThreads, 0, s>>>(a)
       : attn_paged_simt_kernel<T, T, 64><<<grid, kThreads, 0, s>>>(a);
  else
    i4 ? attn_paged_simt_kernel<T, I4, 128><<<grid, kThreads, 0, s>>>(a)
       : attn_paged_simt_kernel<T, T, 128><<<grid, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  prof_after(s, kAttnPaged);
  if (e != cudaSuccess || pl.ctas == 1) return e;
  prof_before(s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.ctas, std::min(a.R, pl.rows), pl.blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_combine_kernel<T, Args>, a, pl.ctas, pl.rows);
  prof_after(s, kAttnPagedCombine);
  return e;
}

}  // namespace

size_t attn_paged_workspace(const AttnPagedProblem& p, const PagedCache& c) {
  const Plan pl = plan_of(p, c);
  return ws_bytes(pl.blocks, pl.ctas, pl.rows, c.D);
}

cudaError_t attn_paged(const AttnPagedProblem& p, const PagedCache& c, cudaStream_t s) {
  return p.bf16 ? run<__nv_bfloat16>(p, c, s) : run<float>(p, c, s);
}

}  // namespace gdn
