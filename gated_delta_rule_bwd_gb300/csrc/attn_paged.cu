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
//
// Bound by the cache's bytes: 2 Hkv D (old + T) values per row, 2 bytes each or, in 4
// bits, 9 / 16 of one.  Measured, 64 rows of 1638 to 8192 tokens, 16 heads on 4, D 128:
// bf16 pages of 16 tokens 105 us the call, 6.1 TB/s; 4 bits, pages of 64: 60 us, 3.0
// TB/s, one row of 1022361 tokens, 16 heads on 2: 82 us, 3.6 TB/s.  In 4 bits no pipe and
// not the memory is full: a warp is one chain of products, maxima, exponentials and
// products per 32 keys, and three warps per scheduler do not cover its waits.

#include <cuda_fp16.h>

#include <type_traits>

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
  uint32_t k16[3], v16[3], ksr[3], vsr[3];  // tensor path: the same in 16-byte vectors, and in a key's steps
  bool dense;                               // a page's tokens of one head lie together
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
// rows per CTA (two per warp, which share what is read of the tile).  A lane owns one
// key of the scores and DP / 32 columns of the accumulators.
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
  constexpr int LD = DP + 4, NC = DP / 64;
  __shared__ __align__(16) float K[kKeys * LD], V[kKeys * LD], Q[kRows * DP];
  __shared__ long long at[2][4][kKeys];  // offsets of a tile's rows in k, v and their steps (-1: none); the next tile's
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
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    F2 acc[2][NC];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[i][c] = f2(0.f, 0.f);
    // warp w looks up k's, v's, k_scale's, v_scale's rows of the tile at t
    auto lookup = [&](int t, int buf) {
      const int j = t + lane, p = j < wk.k1 ? a.page_of(b, j) : -1, place = j & ((1 << a.shift) - 1);
      const long long* st = w == 0 ? a.ks : w == 1 ? a.vs : w == 2 ? a.kss : a.vss;
      at[buf][w][lane] = p < 0 ? -1 : p * st[0] + place * st[1] + hk * st[2];
    };
    lookup(wk.k0, 0);
    int buf = 0;
    for (int t0 = wk.k0; t0 < wk.k1; t0 += kKeys, buf ^= 1) {
      __syncthreads();
      {
        // All loads on their way together: rows without a page read the first and are zeroed.
        const int c = threadIdx.x % (DP / 4) * 4, c0 = c < a.D ? c : 0, r0 = threadIdx.x / (DP / 4);
        constexpr int N = DP / 16, step = 4 * kThreads / DP;
        float4 x[N], y[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = r0 + i * step;
          const long long ka = max(at[buf][0][r], 0ll), va = max(at[buf][1][r], 0ll);
          x[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (a.pages > 0) {
            x[i] = four<C>(a.k, ka, c0, a.D, a.vec, a.k_scale + (sizeof(C) == 1 ? max(at[buf][2][r], 0ll) : 0));
            y[i] = four<C>(a.v, va, c0, a.D, a.vec, a.v_scale + (sizeof(C) == 1 ? max(at[buf][3][r], 0ll) : 0));
          }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = r0 + i * step;
          const bool in = at[buf][0][r] >= 0 && c < a.D;
          const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
          *reinterpret_cast<float4*>(K + r * LD + c) = in ? x[i] : zero;
          *reinterpret_cast<float4*>(V + r * LD + c) = in ? y[i] : zero;
        }
      }
      if (t0 + kKeys < wk.k1) lookup(t0 + kKeys, buf ^ 1);
      __syncthreads();
      if (row0 + w >= a.R) continue;
      // a lane's key against the warp's two rows
      F2 d2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
      const float* q = Q + w * DP;
      const bool two = row0 + w + 4 < a.R;
      auto dots = [&](auto rows) {
#pragma unroll 8
        for (int d = 0; d < DP; d += 4) {
          const float4 x = *reinterpret_cast<const float4*>(K + lane * LD + d);
#pragma unroll
          for (int i = 0; i < decltype(rows)::value; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(q + 4 * i * DP + d);
            d2[i] = fma2(f2(x.x, x.y), f2(y.x, y.y), fma2(f2(x.z, x.w), f2(y.z, y.w), d2[i]));
          }
        }
      };
      two ? dots(std::integral_constant<int, 2>{}) : dots(std::integral_constant<int, 1>{});
      float e[2];
      int seen = 0;  // keys of the tile that any of the two sees
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row0 + w + 4 * i;
        const int last = r < a.R ? min(wk.k1 - t0, old + r / a.G - t0 + 1) : 0;  // keys that the row sees
        seen = max(seen, min(last, kKeys));
        const float2 dd = unpack(d2[i]);
        const float s = lane < last ? (dd.x + dd.y) * a.c : -INFINITY;
        float mx = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = fmaxf(mx, m[i]);
        const float base = mx == -INFINITY ? 0.f : mx;
        const float f = exp2f(m[i] - base);
        e[i] = exp2f(s - base);
        float sum = e[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * f + sum;
        m[i] = mx;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[i][c] = mul2(acc[i][c], f2(f, f));
      }
      auto add = [&](int j, bool both) {  // key j's values, the lane's columns 2 lane, 2 lane + 1, ..
        const float p0 = __shfl_sync(0xffffffffu, e[0], j), p1 = __shfl_sync(0xffffffffu, e[1], j);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float2 x = *reinterpret_cast<const float2*>(V + j * LD + 2 * lane + 64 * c);
          acc[0][c] = fma2(f2(p0, p0), f2(x.x, x.y), acc[0][c]);
          if (both) acc[1][c] = fma2(f2(p1, p1), f2(x.x, x.y), acc[1][c]);
        }
      };
      // A key that a row does not see is left out, not taken times 0: its values may
      // be no numbers.
      const int last0 = min(kKeys, min(wk.k1 - t0, old + (row0 + w) / a.G - t0 + 1));
      if (last0 == kKeys && seen == kKeys) {
        if (two) {
#pragma unroll
          for (int j = 0; j < kKeys; ++j) add(j, true);
        } else {
#pragma unroll
          for (int j = 0; j < kKeys; ++j) add(j, false);
        }
      } else {
        for (int j = 0; j < seen; ++j) {
          const float p0 = __shfl_sync(0xffffffffu, e[0], j), p1 = __shfl_sync(0xffffffffu, e[1], j);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float2 x = *reinterpret_cast<const float2*>(V + j * LD + 2 * lane + 64 * c);
            if (j < last0) acc[0][c] = fma2(f2(p0, p0), f2(x.x, x.y), acc[0][c]);
            if (two) acc[1][c] = fma2(f2(p1, p1), f2(x.x, x.y), acc[1][c]);
          }
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
        for (int c = 0; c < NC; ++c) {
          const int d = 2 * lane + 64 * c;
          const float2 x = unpack(acc[i][c]);
          if (d < a.D) o[d] = from_f32<T>(x.x * f);
          if (d + 1 < a.D) o[d + 1] = from_f32<T>(x.y * f);
        }
      } else {
        const long at = slot + w + 4 * i;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int d = 2 * lane + 64 * c;
          const float2 x = unpack(acc[i][c]);
          if (d < a.D) a.acc[at * a.D + d] = x.x;
          if (d + 1 < a.D) a.acc[at * a.D + d + 1] = x.y;
        }
        if (lane == 0) a.ml[2 * at] = m[i], a.ml[2 * at + 1] = l[i];
      }
    }
  }
}

// ---------------------------------------------------------------- warp-level tensor path
//
// bf16 queries, D a multiple of 8 (bf16 pages, padded with zeros to DP) or D = DP
// (4 bits), 16-byte aligned pages.  Few rows and a bandwidth bound leave nothing
// for tcgen05's 128-row tiles to do: mma.m16n8k16 takes them.  A lane is (g, t) =
// (lane / 4, lane % 4) in the fragments below.
//
//   S^T = K Q^T: M = 16 keys, N = 8 query rows (NR tiles of them), K = 16 of the D
//   values.  Lane (g, t) gets keys g and g + 8 of rows 2 t and 2 t + 1.
//   O^T = V^T P^T: M = 16 of the D values, N = 8 rows, K = 16 keys; P comes from S^T by
//   movmatrix (8 x 8 transpositions between registers), and the accumulators' rows
//   are 2 t and 2 t + 1 again, so that a lane scales its own.
//   Few rows fill N = 8 better than M = 16, and what is made anew for each product,
//   K's and V's fragments, are whole A operands: with q there, half of it zeros for
//   8 rows, the registers were moved together again for each product.
//
// P goes in in two bf16 terms, so that its rounding does not show beside the output's:
// what is left is 2^-16 of it, whatever the probabilities and values are.
// bf16: fragments by ldmatrix (V transposed on the way).  64 rows of up to 8192 keys: 105 us
// so, 104 with one term; memory bounds both.
// 4 bits: the order of the D values within a product is free, and a lane takes whole
// words of 8 codes, held c = code + 8.  Integers become floats by being put into the
// mantissa of a constant, the published way for 4-bit weights:
//   K: a byte below the exponent of an fp16 1024 is X = 1024 + c0 + 16 c1 (two bytes of a
//   word by one byte permutation), and without its upper four bits L = 1024 + c0 (one
//   logic operation), so that
//     q0 c0 + q1 c1 = (q1 / 16) X + (q0 - q1 / 16) L - 1024 (both weights):
//   half an operation a code.  The weights are fp16 (q scaled by a power of two per row,
//   so that its largest value is in [1, 2)): the first is exact, the second off by up to
//   2^-11 of itself, which moves scores of normal queries and keys by 1.5e-4 of their spread.
//   The constants, with the 8 in c, go back once per key, with the steps, which are
//   applied to the scores:
//     s = sum_j step_j (sum_d of the group's products) + sum_j step_j base_j,
//   the second sum (j a key's groups) as one product of the steps with base in three
//   bf16 terms.  1024 against c of about 3 costs the fp32 sums over a group some 9 of
//   their 24 bits.
//   V: w & 0x000f000f (a word of two keys' halves; then w >> 4, ..) in the mantissas of two
//   bf16 128s is 128 + c; less 136 (exactly: sums over thousands of keys of one sign would
//   drown what is left of codes that cancel) and times the keys' steps it is the values
//   as kv_gather gives them, exact for steps of 5 bits.  Every key then has its own
//   exponent, as in 16-bit pages: a large value takes no bits from others, weighted or
//   not.  (One fp16 weight per key, row and 32 values, p step in units of the largest step met,
//   took 56 and 76 us for 60 and 82, but left keys out beside a hardly weighted value some 2^16
//   above theirs.)
//
// Each warp streams its own blocks of KS keys (w, w + 4, ...) through a ring of
// kStages stages (cp.async) and keeps its own m, l and accumulators, so the warps
// meet only at a segment's end.
constexpr int kStages = 3;
// CTAs per SM.  4 bits: at three, 165 registers; four (128) kept the same share of the
// issue slots busy, with more of them to set up (57 us for 55, with fp16 weights).
constexpr int kPerSm16 = 2, kPerSm4 = 3;

template <int n>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {
  if constexpr (n == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16u : 0u) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(n), "r"(valid ? (uint32_t)n : 0u)
                 : "memory");
}
template <int n>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}
// Whether the bf16 in the low half is infinite or NaN.
__device__ __forceinline__ bool no_number(uint32_t v) { return (v & 0x7f80) == 0x7f80; }
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {  // d += a b
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {  // d = a b
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// the same of fp16
__device__ __forceinline__ void mma0_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// The codes of a word of two keys' halves, by twos, as bf16, and the values that they
// stand for.  The constants come as registers: with both as immediates it takes two
// logic operations.
struct Magic {
  uint32_t low, one;
  __device__ __forceinline__ Magic() {
    asm volatile("mov.b32 %0, 0x000f000f;" : "=r"(low));
    asm volatile("mov.b32 %0, 0x43004300;" : "=r"(one));
  }
  __device__ __forceinline__ static __nv_bfloat162 twos(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }
  // the codes at bits 0-3 of w's halves, times the steps
  __device__ __forceinline__ uint32_t values(uint32_t w, uint32_t steps) const {
    uint32_t x;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(w), "r"(low), "r"(one));
    const __nv_bfloat162 v = __hmul2_rn(__hadd2_rn(twos(x), twos(0xc308c308u)), twos(steps));  // - 136
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

template <int DP, bool I4>
struct Stage {
  static constexpr int KS = I4 ? 32 : 16;           // keys
  static constexpr int row = I4 ? DP / 2 : DP * 2;  // bytes of a key's row
  static constexpr int NC = row / 16;               // 16-byte chunks of it
  using Steps = std::conditional_t<DP == 128, uint2, uint32_t>;  // a key's steps (4 bits)
  static constexpr int step = I4 ? (int)sizeof(Steps) : 0;
  static constexpr int v = KS * row, ks = 2 * v, vs = ks + KS * step, bytes = vs + KS * step;
  // Chunk c of key r lies at c ^ f(r), so that the lanes of a load (bf16: eight keys'
  // chunks; 4 bits: eight keys' words of a chunk, two words each of four keys two
  // apart) meet no bank twice.
  // The same for r + 8; 4 bits: for r + 1 of an even r.
  __device__ __forceinline__ static uint32_t f(int r) {
    return (!I4 ? r & 7 : DP == 128 ? (r >> 1) & 3 : (r >> 2) & 1) << 4;
  }
  __device__ __forceinline__ static uint32_t at(int r, int c) { return r * row + ((c << 4) ^ f(r)); }
};

// LATER: several new tokens per row, of which the first do not see the last.  As a kernel
// of its own, because the code alone, never run, costs single tokens 1.5 % (64 rows in
// 4 bits 60.4 for 59.5 us).
template <int DP, int NR, bool I4, bool LATER>
__global__ void __launch_bounds__(kThreads, I4 ? kPerSm4 : kPerSm16) attn_paged_mma_kernel(Args a) {
  using St = Stage<DP, I4>;
  constexpr int KS = St::KS, NG = DP / 32, NT = KS / 16, kQ = 8 * NR;  // kQ: query rows per CTA
  extern __shared__ __align__(128) unsigned char sm[];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane / 4, t = lane % 4, row0 = blockIdx.y * kQ;
  const uint32_t ring = smem_u32(sm) + w * kStages * St::bytes;
  grid_dep_launch();
  empty_rows<__nv_bfloat16>(a);
  if (threadIdx.x == 0) a.starts[(long)blockIdx.y * gridDim.x + blockIdx.x].x = -1;
  __shared__ Walk<Args> kept;  // not in registers while a segment runs
  __shared__ uint4 q_frag[I4 ? NG : 1][NR][32];  // 4 bits: q's fragments, group sums and powers of two
  __shared__ float q_sum[kQ][NG], q_up[kQ];
  Walk<Args> wk;
  if (!wk.init(a)) return;
  while (wk.segment(a)) {
    const int b = wk.b, hk = wk.hk, old = wk.keys - a.T, k0 = wk.k0, k1 = wk.k1;
    if (threadIdx.x == 0) kept = wk;
    using Steps = typename St::Steps;
    const uint4* kb = static_cast<const uint4*>(a.k) + (size_t)hk * a.k16[2];
    const uint4* vb = static_cast<const uint4*>(a.v) + (size_t)hk * a.v16[2];
    const Steps* ksb = reinterpret_cast<const Steps*>(a.k_scale) + (size_t)hk * a.ksr[2];
    const Steps* vsb = reinterpret_cast<const Steps*>(a.v_scale) + (size_t)hk * a.vsr[2];
    const int blocks = (k1 - k0 + KS - 1) / KS;  // this warp's are w, w + 4, ...
    const int mine = blocks > w ? (blocks - w + 3) / 4 : 0;

    // the page of this lane's key of block i
    auto lookup = [&](int i) {
      const int j = k0 + (w + 4 * i) * KS + lane % KS;
      return i < mine && j < k1 ? a.page_of(b, j) : -1;
    };
    // block i into its stage; pg: lookup(i)
    auto fetch = [&](int i, int pg) {
      const int j0 = k0 + (w + 4 * i) * KS, mask = (1 << a.shift) - 1;
      const uint32_t dst = ring + i % kStages * St::bytes;
      constexpr int RS = 32 / St::NC;  // rows of the warp's copies at once
      const int c = lane % St::NC, r0 = lane / St::NC;
      const int p0 = __shfl_sync(0xffffffffu, pg, 0);
      if (mask >= KS - 1 && j0 + KS <= k1 && p0 >= 0 && a.D == DP) {  // a whole block in one page
        const uint32_t at = j0 & mask, r4 = lane % KS;
        const uint4 *ks = kb + (uint64_t)p0 * a.k16[0], *vs = vb + (uint64_t)p0 * a.v16[0];
        auto to = [&](int r) { return dst + (RS % 8 == 0 ? r * St::row + St::at(r0, c) : St::at(r0 + r, c)); };
        const Steps *kt = ksb, *vt = vsb;
        if constexpr (I4) kt += (uint64_t)p0 * a.ksr[0], vt += (uint64_t)p0 * a.vsr[0];
        if (a.dense) {  // the keys of a head one after another: the warp copies what follows
          ks += (uint64_t)at * St::NC + lane, vs += (uint64_t)at * St::NC + lane;
#pragma unroll
          for (int r = 0; r < KS; r += RS) {
            cp_async<16>(to(r), ks + r * St::NC, true);
            cp_async<16>(to(r) + St::v, vs + r * St::NC, true);
          }
          kt += at + r4, vt += at + r4;
        } else {
          ks += (uint64_t)(at + r0) * a.k16[1] + c, vs += (uint64_t)(at + r0) * a.v16[1] + c;
#pragma unroll
          for (int r = 0; r < KS; r += RS) {
            cp_async<16>(to(r), ks, true);
            cp_async<16>(to(r) + St::v, vs, true);
            ks += (size_t)RS * a.k16[1], vs += (size_t)RS * a.v16[1];
          }
          kt += (uint64_t)(at + r4) * a.ksr[1], vt += (uint64_t)(at + r4) * a.vsr[1];
        }
        if constexpr (I4) {
          if (lane < KS) cp_async<St::step>(dst + St::ks + r4 * St::step, kt, true);
          if (lane >= 32 - KS) cp_async<St::step>(dst + St::vs + r4 * St::step, vt, true);
        }
        return;
      }
#pragma unroll 1
      for (int r = r0; r < KS; r += RS) {
        const int p = __shfl_sync(0xffffffffu, pg, r);
        const uint32_t at = (j0 + r) & mask;
        const bool in = p >= 0 && c * (I4 ? 32 : 8) < a.D;
        cp_async<16>(dst + St::at(r, c), in ? kb + (uint64_t)p * a.k16[0] + (uint64_t)at * a.k16[1] + c : kb, in);
        cp_async<16>(dst + St::v + St::at(r, c), in ? vb + (uint64_t)p * a.v16[0] + (uint64_t)at * a.v16[1] + c : vb, in);
      }
      if constexpr (I4) {
        const uint32_t r = lane % KS, at = (j0 + r) & mask;
        const bool in = pg >= 0;
        if (lane < KS)
          cp_async<St::step>(dst + St::ks + r * St::step, in ? ksb + (uint64_t)pg * a.ksr[0] + (uint64_t)at * a.ksr[1] : ksb, in);
        if (lane >= 32 - KS)
          cp_async<St::step>(dst + St::vs + r * St::step, in ? vsb + (uint64_t)pg * a.vsr[0] + (uint64_t)at * a.vsr[1] : vsb, in);
      }
    };
    int pg = lookup(0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      const int next = lookup(i + 1);
      if (i < mine) fetch(i, pg);
      cp_async_commit();
      pg = next;
    }

    // q as B fragments, row g of tile x: the values that face a lane's words of K
    uint32_t qf[DP / 16][NR][2], base[NR][2];  // base: 4 bits, see below
    float c[NR][2];                            // log2 e times the scale, and 4 bits: what was taken out of the row of q
    if constexpr (I4) {
      // Warp j makes group j's for all: values 32 j + 8 t .. of the rows.
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        const int r = row0 + g + 8 * x;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (r < a.R ? row_at(a, b, hk, r) : 0);
        uint4 mine_q = make_uint4(0, 0, 0, 0);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const uint4 v = r < a.R ? *reinterpret_cast<const uint4*>(q + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);
          for (uint32_t u : {v.x, v.y, v.z, v.w}) top = max(top, max(u << 16 & 0x7fff0000u, u & 0x7fff0000u));
          if (j == w) mine_q = v;
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e and 2^e for the largest magnitude's exponent e (0, subnormal, infinite or NaN: 1)
        const uint32_t e = top >> 23 == 0 || top >> 23 == 255 ? 127 : min(top >> 23, 253u);
        const float down = __uint_as_float((254 - e) << 23);
        if (w < NG) {
          const uint32_t u[4] = {mine_q.x, mine_q.y, mine_q.z, mine_q.w};  // byte b of the word: values 2 b, 2 b + 1
          uint32_t f[4];
          float y = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // bytes 2 h, 2 h + 1: product 2 j + h
            const float q0 = lo16(u[2 * h]) * down, q1 = hi16(u[2 * h]) * down, q2 = lo16(u[2 * h + 1]) * down,
                        q3 = hi16(u[2 * h + 1]) * down;
            const __half2 wx = __floats2half2_rn(q1 * 0.0625f, q3 * 0.0625f);
            const __half2 wl = __floats2half2_rn(q0 - q1 * 0.0625f, q2 - q3 * 0.0625f);
            f[2 * h] = *reinterpret_cast<const uint32_t*>(&wx), f[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&wl);
            const float2 fx = __half22float2(wx), fl = __half22float2(wl);
            // 1024 + 16 * 8 + 8 in X, 1024 + 8 in L
            y = fmaf(-1160.f, fx.x + fx.y, fmaf(-1032.f, fl.x + fl.y, y));
          }
          y += __shfl_xor_sync(0xffffffffu, y, 1);
          y += __shfl_xor_sync(0xffffffffu, y, 2);
          q_frag[w][x][lane] = make_uint4(f[0], f[1], f[2], f[3]);
          if (t == 0) {
            q_sum[8 * x + g][w] = y;
            if (w == 0) q_up[8 * x + g] = __uint_as_float(e << 23);
          }
        }
      }
      __syncthreads();
      // A row's sums as three terms of 8 bits, against the groups' steps: k = NG i + j
      // is term i of group j; a lane has k = 2 t, 2 t + 1 and 2 t + 8, 2 t + 9.
      auto term = [&](int r, int k) {
        const int i = k / NG;
        const float y = q_sum[r][k % NG], hi = __bfloat162float(__float2bfloat16_rn(y)), rest = y - hi;
        const float mid = __bfloat162float(__float2bfloat16_rn(rest));
        return i == 0 ? hi : i == 1 ? mid : i == 2 ? rest - mid : 0.f;
      };
#pragma unroll
      for (int x = 0; x < NR; ++x) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const uint4 v = q_frag[j][x][lane];
          qf[2 * j][x][0] = v.x, qf[2 * j][x][1] = v.y, qf[2 * j + 1][x][0] = v.z, qf[2 * j + 1][x][1] = v.w;
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) base[x][y] = pack_bf16(term(8 * x + g, 2 * t + 8 * y), term(8 * x + g, 2 * t + 8 * y + 1));
#pragma unroll
        for (int e = 0; e < 2; ++e) c[x][e] = a.c * q_up[8 * x + 2 * t + e];
      }
    } else {
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        const int r = row0 + g + 8 * x;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (r < a.R ? row_at(a, b, hk, r) : 0);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int d = 16 * k + 8 * y + 2 * t;
            qf[k][x][y] = r < a.R && d < a.D ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
          }
        c[x][0] = c[x][1] = a.c;
      }
    }
    float acc[DP / 16][NR][4], m[NR][2], l[NR][2];
    int last[NR][2];  // last key that the row sees
#pragma unroll
    for (int x = 0; x < NR; ++x) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[x][e] = -INFINITY, l[x][e] = 0.f;
        last[x][e] = min(k1 - 1, old + (row0 + 8 * x + 2 * t + e) / a.G);
      }
#pragma unroll
      for (int n = 0; n < DP / 16; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][x][e] = 0.f;
    }
    // 4 bits: this lane's words of keys g, .. and of keys 2 t, ..
    const uint32_t k_at = g * St::row + 4 * t, k_f = St::f(g), v_at = 2 * t * St::row + 4 * (g / 2), v_f = St::f(2 * t);
    const Magic magic;
    for (int i = 0; i < mine; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      {
        const int next = lookup(i + kStages);
        if (i + kStages - 1 < mine) fetch(i + kStages - 1, pg);  // over the stage read in the pass before
        cp_async_commit();
        pg = next;
      }
      const uint32_t st = ring + i % kStages * St::bytes;
      const int j0 = k0 + (w + 4 * i) * KS;
      float s[NT][NR][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (I4) {
          uint32_t sc[2][NG / 2];  // steps of keys g and g + 8, two groups to a word
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t at = st + St::ks + (16 * n + 8 * y + g) * St::step;
            if constexpr (NG == 4) {
              const uint2 v = lds64(at);
              sc[y][0] = v.x, sc[y][1] = v.y;
            } else {
              sc[y][0] = lds32(at);
            }
          }
          {
            const uint32_t c0 = NG == 4 && t & 1 ? sc[0][NG / 2 - 1] : sc[0][0], c1 = NG == 4 && t & 1 ? sc[1][NG / 2 - 1] : sc[1][0];
            const uint32_t steps[4] = {c0, c1, c0, c1};
#pragma unroll
            for (int x = 0; x < NR; ++x) mma0(s[n][x], steps, base[x][0], base[x][1]);
          }
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            const uint32_t at = st + 16 * n * St::row + k_at + ((j << 4) ^ k_f);
            const uint32_t u0 = lds32(at), u1 = lds32(at + 8 * St::row);
            // bytes 0 and 1, 2 and 3 of keys g and g + 8
            const uint32_t x0 = __byte_perm(u0, 0x64u, 0x4140), x1 = __byte_perm(u1, 0x64u, 0x4140);
            const uint32_t x2 = __byte_perm(u0, 0x64u, 0x4342), x3 = __byte_perm(u1, 0x64u, 0x4342);
            constexpr uint32_t low = 0x640f640fu;
            const float e0 = j & 1 ? hi16(sc[0][j / 2]) : lo16(sc[0][j / 2]), e1 = j & 1 ? hi16(sc[1][j / 2]) : lo16(sc[1][j / 2]);
#pragma unroll
            for (int x = 0; x < NR; ++x) {
              float d[4];
              mma0_f16(d, x0, x1, x0 & low, x1 & low, qf[2 * j][x][0], qf[2 * j][x][1]);
              mma_f16(d, x2, x3, x2 & low, x3 & low, qf[2 * j + 1][x][0], qf[2 * j + 1][x][1]);
              s[n][x][0] = fmaf(d[0], e0, s[n][x][0]), s[n][x][1] = fmaf(d[1], e0, s[n][x][1]);
              s[n][x][2] = fmaf(d[2], e1, s[n][x][2]), s[n][x][3] = fmaf(d[3], e1, s[n][x][3]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            uint32_t f[4];
            ldsm4(f, st + St::at(16 * n + lane % 16, 2 * k + lane / 16));
#pragma unroll
            for (int x = 0; x < NR; ++x)
              k == 0 ? mma0(s[n][x], f, qf[k][x][0], qf[k][x][1]) : mma(s[n][x], f, qf[k][x][0], qf[k][x][1]);
          }
        }
      }
      const bool edge = j0 + KS - 1 > old || j0 + KS > k1;  // new tokens' causal order, the segment's end
      bool raise = false;
      float f[NR][2];
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (edge) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int y = 0; y < 2; ++y)
                if (j0 + 16 * n + 8 * y + g > last[x][e]) s[n][x][2 * y + e] = -INFINITY;
          }
          float top = fmaxf(s[0][x][e], s[0][x][2 + e]);
#pragma unroll
          for (int n = 1; n < NT; ++n) top = fmaxf(top, fmaxf(s[n][x][e], s[n][x][2 + e]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          top *= c[x][e];
          f[x][e] = 1.f;
          if (top - m[x][e] > 8.f) {  // see the prompt kernel: P at most 2^8
            f[x][e] = ex2(m[x][e] - top);
            m[x][e] = top;
            raise = true;
          }
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < NR; ++x) {
          l[x][0] *= f[x][0], l[x][1] *= f[x][1];
#pragma unroll
          for (int n = 0; n < DP / 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][x][e] *= f[x][e & 1];
        }
      }
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float low = m[x][e] == -INFINITY ? 0.f : m[x][e];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            s[n][x][e] = ex2(fmaf(s[n][x][e], c[x][e], -low)), s[n][x][2 + e] = ex2(fmaf(s[n][x][2 + e], c[x][e], -low));
            l[x][e] += s[n][x][e] + s[n][x][2 + e];
          }
        }
      // A later new token's values that are no numbers: rows that see the token take them
      // here, and the products find zeros (the others' weight of 0 times them is none).
      if (LATER && j0 + KS - 1 > old) {
        bool bad = false;
        if constexpr (I4) {
          for (int i = lane; i < KS * NG / 2; i += 32) {
            const uint32_t u = lds32(st + St::vs + 4 * i);
            bad |= no_number(u) || no_number(u >> 16);
          }
        } else {
          for (int i = lane; i < KS * St::NC; i += 32) {
            const uint4 v = lds128(st + St::v + 16 * i);
            for (uint32_t u : {v.x, v.y, v.z, v.w}) bad |= no_number(u) || no_number(u >> 16);
          }
        }
        if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
          for (int r = max(0, old + 1 - j0); r < KS; ++r) {
            auto take = [&](int n, int y, uint32_t u) {  // acc[n][.][2 y + e] of the rows that see key r
              if (!no_number(u)) return;
#pragma unroll
              for (int x = 0; x < NR; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (j0 + r <= last[x][e]) acc[n][x][2 * y + e] += I4 ? NAN : lo16(u);
            };
#pragma unroll
            for (int n = 0; n < DP / 16; ++n)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                if constexpr (I4) take(n, y, lds16(st + St::vs + r * St::step + 2 * (n / 2)));
                else take(n, y, lds16(st + St::v + St::at(r, 2 * n + y) + 2 * g));
              }
            __syncwarp();
            if constexpr (I4) {
              const uint32_t at = st + St::vs + r * St::step + 2 * (lane % NG);
              if (lane < NG && no_number(lds16(at))) sts16(at, 0);
            } else {
              for (int c = lane; c < DP; c += 32) {
                const uint32_t at = st + St::v + r * St::row + 2 * c;
                if (no_number(lds16(at))) sts16(at, 0);
              }
            }
          }
          __syncwarp();
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t pf[NR][2], pl[NR][2];  // P and what its rounding to bf16 leaves
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float p0 = s[n][x][2 * y], p1 = s[n][x][2 * y + 1];
            const uint32_t p = pack_bf16(p0, p1);
            pf[x][y] = transposed(p), pl[x][y] = transposed(pack_bf16(p0 - lo16(p), p1 - hi16(p)));
          }
        if constexpr (I4) {
          // steps of keys 2 t and 2 t + 1, 2 t + 8 and 2 t + 9
          uint32_t sa[2][NG / 2], sb[2][NG / 2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t at = st + St::vs + (16 * n + 8 * y + 2 * t) * St::step;
            if constexpr (NG == 4) {
              const uint4 v = lds128(at);
              sa[y][0] = v.x, sa[y][1] = v.y, sb[y][0] = v.z, sb[y][1] = v.w;
            } else {
              const uint2 v = lds64(at);
              sa[y][0] = v.x, sb[y][0] = v.y;
            }
          }
          const uint32_t half = g & 1 ? 0x7632 : 0x5410;
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            // values 32 j + 4 g .. + 3 of those keys
            const uint32_t at = st + St::v + 16 * n * St::row + v_at + ((j << 4) ^ v_f);
            const uint32_t v0 = __byte_perm(lds32(at), lds32(at + St::row), half);
            const uint32_t v1 = __byte_perm(lds32(at + 8 * St::row), lds32(at + 9 * St::row), half);
            const uint32_t e0 = __byte_perm(sa[0][j / 2], sb[0][j / 2], j & 1 ? 0x7632 : 0x5410);
            const uint32_t e1 = __byte_perm(sa[1][j / 2], sb[1][j / 2], j & 1 ? 0x7632 : 0x5410);
            uint32_t f[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              f[y][0] = magic.values(v0 >> (8 * y), e0), f[y][1] = magic.values(v0 >> (8 * y + 4), e0);
              f[y][2] = magic.values(v1 >> (8 * y), e1), f[y][3] = magic.values(v1 >> (8 * y + 4), e1);
#pragma unroll
              for (int x = 0; x < NR; ++x) mma(acc[2 * j + y][x], f[y], pl[x][0], pl[x][1]);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int x = 0; x < NR; ++x) mma(acc[2 * j + y][x], f[y], pf[x][0], pf[x][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            uint32_t v[4];
            ldsm4_trans(v, st + St::v + St::at(16 * n + (lane & 7) + (lane >> 4) * 8, 2 * k + ((lane >> 3) & 1)));
#pragma unroll
            for (int x = 0; x < NR; ++x) {
              mma(acc[k][x], v, pl[x][0], pl[x][1]);
              mma(acc[k][x], v, pf[x][0], pf[x][1]);
            }
          }
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();
    // the four warps' pieces: maxima and sums, then the scaled accumulators
    float* ml = reinterpret_cast<float*>(sm);  // [4][kQ][2]
    float* part = ml + 4 * kQ * 2;             // [4][kQ][DP]
    __syncthreads();
    wk = kept;
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], o);
        if (g == 0) {
          float* p = ml + (w * kQ + 8 * x + 2 * t + e) * 2;
          p[0] = m[x][e], p[1] = l[x][e];
        }
      }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * x + 2 * t + e;
        float top = -INFINITY;
#pragma unroll
        for (int p = 0; p < 4; ++p) top = fmaxf(top, ml[(p * kQ + r) * 2]);
        const float f = m[x][e] == -INFINITY ? 0.f : ex2(m[x][e] - top);
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
          float* p = part + (w * kQ + r) * DP;
          if constexpr (I4) {  // rows g and g + 8 of a product are neighbours
            *reinterpret_cast<float2*>(p + 32 * (n / 2) + 4 * g + 2 * (n % 2)) = make_float2(acc[n][x][e] * f, acc[n][x][2 + e] * f);
          } else {
            p[16 * n + g] = acc[n][x][e] * f, p[16 * n + g + 8] = acc[n][x][2 + e] * f;
          }
        }
      }
    __syncthreads();
    const long slot = wk.whole ? 0 : slot_of(a, wk) * kQ;
    for (int i = threadIdx.x; i < kQ * (DP / 4); i += kThreads) {
      const int rl = i / (DP / 4), c = i % (DP / 4) * 4, r = row0 + rl;
      if (r >= a.R || c >= a.D) continue;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int p = 0; p < 4; ++p) top = fmaxf(top, ml[(p * kQ + rl) * 2]);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        // a piece without keys adds 0; one whose scores are all NaN has m = -inf too, and adds its l
        const float mp = ml[(p * kQ + rl) * 2], base = top == -INFINITY ? 0.f : top;
        sum = fmaf(ex2(mp - base), ml[(p * kQ + rl) * 2 + 1], sum);
        const float4 y = *reinterpret_cast<const float4*>(part + (p * kQ + rl) * DP + c);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      if (wk.whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row_at(a, b, hk, r) + c) =
            make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
      } else {
        *reinterpret_cast<float4*>(a.acc + (slot + rl) * a.D + c) = x;
        if (c == 0) a.ml[2 * (slot + rl)] = top, a.ml[2 * (slot + rl) + 1] = sum;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- host

bool use_mma(const AttnPagedProblem& p, const PagedCache& c) {
  if (!p.bf16) return false;
  const bool i4 = c.format == GDN_CACHE_I4;
  if (i4 ? c.D != 64 && c.D != 128 : c.D % 8 || (uintptr_t)c.k & 15 || (uintptr_t)c.v & 15) return false;
  const long long vec = i4 ? 16 : 8, most = vec << 32;  // strides in vectors (and steps) fit 32 bits
  for (int i = 0; i < 3; ++i) {
    if (c.ks[i] % vec || c.vs[i] % vec || c.ks[i] >= most || c.vs[i] >= most) return false;
    if (i4 && (c.kss[i] / (c.D / kStepGroup) > UINT32_MAX || c.vss[i] / (c.D / kStepGroup) > UINT32_MAX)) return false;
  }
  return true;
}

struct Plan {
  bool mma;
  int rows, blocks, ctas;  // query rows per CTA, row blocks (grid.y), CTAs that share the units (grid.x)
};

Plan plan_of(const AttnPagedProblem& p, const PagedCache& c) {
  Plan q;
  const int R = p.H / c.Hkv * p.T;
  q.mma = use_mma(p, c);
  q.rows = !q.mma ? kRows : R <= 8 ? 8 : 16;
  q.blocks = (R + q.rows - 1) / q.rows;
  const int per_sm = !q.mma ? 4 : c.format == GDN_CACHE_I4 ? kPerSm4 : kPerSm16;
  q.ctas = ctas_for(p.B, c.Hkv, (long)p.pt.max_pages * c.page, q.blocks, per_sm);
  return q;
}

template <bool I4>
cudaError_t launch_mma(const Args& a, const Plan& pl, cudaStream_t s) {
  const dim3 grid(pl.ctas, pl.blocks);
  auto go = [&](auto kernel, int smem) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) kernel<<<grid, kThreads, smem, s>>>(a);
    return e == cudaSuccess ? cudaGetLastError() : e;
  };
  // the ring, or the four warps' pieces
  auto smem = [&](int stage, int DP) {
    return std::max(4 * kStages * stage, 4 * pl.rows * (DP + 2) * (int)sizeof(float));
  };
  auto by_size = [&](auto size) {
    constexpr int DP = decltype(size)::value;
    const int n = smem(Stage<DP, I4>::bytes, DP);
    if (a.T > 1)
      return pl.rows == 8 ? go(attn_paged_mma_kernel<DP, 1, I4, true>, n) : go(attn_paged_mma_kernel<DP, 2, I4, true>, n);
    return pl.rows == 8 ? go(attn_paged_mma_kernel<DP, 1, I4, false>, n) : go(attn_paged_mma_kernel<DP, 2, I4, false>, n);
  };
  return a.D <= 64 ? by_size(std::integral_constant<int, 64>{}) : by_size(std::integral_constant<int, 128>{});
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
    if (pl.mma) {
      const int vec = c.format == GDN_CACHE_I4 ? 16 : 8, steps = std::max(1, c.D / kStepGroup);
      a.k16[i] = (uint32_t)(c.ks[i] / vec), a.v16[i] = (uint32_t)(c.vs[i] / vec);
      a.ksr[i] = (uint32_t)(c.kss[i] / steps), a.vsr[i] = (uint32_t)(c.vss[i] / steps);
    }
  }
  const uint32_t row16 = c.format == GDN_CACHE_I4 ? c.D / 32 : c.D / 8;
  a.dense = a.k16[1] == row16 && a.v16[1] == row16 && (c.format != GDN_CACHE_I4 || (a.ksr[1] == 1 && a.vsr[1] == 1));
  a.q = p.q, a.k = c.k, a.v = c.v, a.o = p.o;
  a.k_scale = static_cast<const __nv_bfloat16*>(c.k_scale), a.v_scale = static_cast<const __nv_bfloat16*>(c.v_scale);
  unsigned char* ws = static_cast<unsigned char*>(p.ws);
  a.starts = reinterpret_cast<int4*>(ws);
  a.ml = reinterpret_cast<float*>(ws + ws_starts(pl.blocks, pl.ctas));
  a.acc = reinterpret_cast<float*>(ws + ws_starts(pl.blocks, pl.ctas) + ws_ml(pl.blocks, pl.ctas, pl.rows));
  const dim3 grid(pl.ctas, pl.blocks);
  const bool i4 = c.format == GDN_CACHE_I4;
  cudaError_t e = cudaSuccess;
  prof_before(s);
  if (pl.mma)
    e = i4 ? launch_mma<true>(a, pl, s) : launch_mma<false>(a, pl, s);
  else if (c.D <= 64)
    i4 ? attn_paged_simt_kernel<T, I4, 64><<<grid, kThreads, 0, s>>>(a)
       : attn_paged_simt_kernel<T, T, 64><<<grid, kThreads, 0, s>>>(a);
  else
    i4 ? attn_paged_simt_kernel<T, I4, 128><<<grid, kThreads, 0, s>>>(a)
       : attn_paged_simt_kernel<T, T, 128><<<grid, kThreads, 0, s>>>(a);
  if (e == cudaSuccess) e = cudaGetLastError();
  prof_after(s, kAttnPaged);
  if (e != cudaSuccess || pl.ctas == 1) return e;
  prof_before(s);
  cudaLaunchConfig_t cfg = {};
  const bool wide = pl.ctas >= 16 * p.B * c.Hkv;  // few rows in many pieces
  cfg.gridDim = dim3(wide ? p.B * c.Hkv : pl.ctas, std::min(a.R, pl.rows), pl.blocks);
  cfg.blockDim = dim3(wide ? 8 * kThreads : kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  e = wide ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<T, 8, Args>, a, pl.ctas, pl.rows)
           : cudaLaunchKernelEx(&cfg, attn_combine_kernel<T, 1, Args>, a, pl.ctas, pl.rows);
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
