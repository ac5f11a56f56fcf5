// Attention of a few new tokens per row against a cache that the call extends
// (single-token generation).
//
// Row b holds old = lens[b] tokens; the T new tokens go to slots old ..
// old+T-1 and new token t attends to the slots j <= old + t:
//   o = sum_j exp(scale q . k_j - m) v_j / sum_j exp(scale q . k_j - m).
// The G = H / Hkv query heads of a key head and the T tokens are the R = G T
// rows of one product with the cache.  Bound by the cache's bytes: 2 Hkv D
// (old + T) elements per row, read once per block of 16 or 32 rows.
//
// Work split: the batch's units of 64 keys evenly over the CTAs, and a second
// kernel that joins what is split (attn_split.cuh).
//
// Measured: 64 rows of 1638 to 8191 tokens, 16 heads on 4, D 128, bf16: 110 us the
// call, 5.9 TB/s (104 us and 6.2 TB/s the first kernel); one row of 1M slots, 95 %
// full, 16 heads on 2: 171 us, 6.1 TB/s.
//
// The new tokens' k and v are read from the call's inputs, never from the
// cache; the CTA that has their keys writes them there.  No CTA reads a slot
// that another one writes, and slots past a row's end are not read.

#include <math.h>

#include <algorithm>

#include "attn_split.cuh"

namespace gdn {

cudaError_t attn_decode_read_and_clear_status(int* status) {
  return tc::read_and_clear_file_status(status);
}

namespace {

using namespace tc;
using namespace split;

struct Args {
  int B, T, S, H, Hkv, D, G, R;  // R = G T rows per key head
  bool vec;                      // 16-byte loads of the caches
  float c;                       // scale log2 e
  long long kcs[3], vcs[3];
  const void *q, *k, *v;
  void *kc, *vc;
  const int* lens;
  void* o;
  int4* starts;
  float *ml, *acc;
  // Row b's tokens after the call (0: bad length, nothing is done).
  __device__ __forceinline__ int keys(int b) const {
    const int n = lens[b];
    return n < 0 || n > S - T ? 0 : n + T;
  }
};

// Rows with a bad length: o = 0, and the status word says so.
template <typename T>
__device__ void bad_rows(const Args& a) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (a.keys(b) || blockIdx.y) continue;
    const long long n = (long long)a.T * a.H * a.D;
    for (long long i = threadIdx.x; i < n; i += kThreads) static_cast<T*>(a.o)[b * n + i] = from_f32<T>(0.f);
    if (threadIdx.x == 0) atomicExch(&g_file_status, GDN_ERR_SEQLENS);
  }
}

// ---------------------------------------------------------------- CUDA cores
//
// Any dtype and D: 4 warps, tiles of 32 keys in shared memory as fp32, 8 query
// rows per CTA (two per warp).  A lane owns one key of the scores and DP / 32
// columns of the accumulators.
constexpr int kRows = 8, kKeys = 32;

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attn_decode_simt_kernel(Args a) {
  constexpr int LD = DP + 4, NC = DP / 32;
  __shared__ __align__(16) float K[kKeys * LD], V[kKeys * LD], Q[kRows * DP];
  const int row0 = blockIdx.y * kRows, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_launch();
  bad_rows<T>(a);
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
    T* kc = static_cast<T*>(a.kc) + b * a.kcs[0] + hk * a.kcs[2];
    T* vc = static_cast<T*>(a.vc) + b * a.vcs[0] + hk * a.vcs[2];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[2][NC] = {};
    for (int t0 = wk.k0; t0 < wk.k1; t0 += kKeys) {
      __syncthreads();
      if (sizeof(T) == 4 && a.vec && t0 + kKeys <= min(old, wk.k1)) {
        const int c = threadIdx.x % (DP / 4) * 4;
#pragma unroll
        for (int r = threadIdx.x / (DP / 4); r < kKeys; r += kThreads / (DP / 4)) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
          if (c < a.D) {
            x = *reinterpret_cast<const float4*>(kc + (t0 + r) * a.kcs[1] + c);
            y = *reinterpret_cast<const float4*>(vc + (t0 + r) * a.vcs[1] + c);
          }
          *reinterpret_cast<float4*>(K + r * LD + c) = x;
          *reinterpret_cast<float4*>(V + r * LD + c) = y;
        }
      } else {
        for (int i = threadIdx.x; i < kKeys * DP; i += kThreads) {
          const int r = i / DP, c = i % DP, j = t0 + r;
          float x = 0.f, y = 0.f;
          if (j < wk.k1 && c < a.D) {
            if (j < old) {
              x = to_f32(kc[j * a.kcs[1] + c]), y = to_f32(vc[j * a.vcs[1] + c]);
            } else {
              const long long at = (((long long)b * a.T + j - old) * a.Hkv + hk) * a.D + c;
              const T kx = static_cast<const T*>(a.k)[at], vx = static_cast<const T*>(a.v)[at];
              if (blockIdx.y == 0) kc[j * a.kcs[1] + c] = kx, vc[j * a.vcs[1] + c] = vx;
              x = to_f32(kx), y = to_f32(vx);
            }
          }
          K[r * LD + c] = x, V[r * LD + c] = y;
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
        if (last >= kKeys) {
#pragma unroll
          for (int j = 0; j < kKeys; ++j) {
            const float pj = __shfl_sync(0xffffffffu, e, j);
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[i][c] = fmaf(pj, V[j * LD + lane + 32 * c], acc[i][c]);
          }
        } else {
          for (int j = 0; j < last; ++j) {
            const float pj = __shfl_sync(0xffffffffu, e, j);
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[i][c] = fmaf(pj, V[j * LD + lane + 32 * c], acc[i][c]);
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

// ---------------------------------------------------------------- warp-level tensor path
//
// bf16, D a multiple of 8 (padded with zeros to DP = 64 or 128), 16-byte
// aligned caches.  The rows are the M = 16 (MB = 2: 32) of mma.m16n8k16 (few
// rows and a bandwidth bound leave nothing for tcgen05's 128-row tiles to do).
// A unit's 64 keys are 16 per warp; each warp streams its own keys through a
// ring of three 16-key stages (cp.async, chunk c of row r at c ^ (r & 7)) and
// keeps its own m, l and accumulators, so the warps meet only at a segment's
// end.  Two CTAs per SM, 192 KB of copies in flight.
constexpr int kStages = 3;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16u : 0u)
               : "memory");
}
template <int n>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
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
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DP, int MB>
__global__ void __launch_bounds__(kThreads, 2) attn_decode_mma_kernel(Args a) {
  constexpr int kRowB = DP * 2, kHalf = 16 * kRowB, kStage = 2 * kHalf;  // 16 keys: K, then V
  constexpr int NC = DP / 8;                                             // 16-byte chunks of a row
  extern __shared__ __align__(128) unsigned char sm[];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, row0 = blockIdx.y * 16 * MB;
  const uint32_t ring = smem_u32(sm) + w * kStages * kStage;
  grid_dep_launch();
  bad_rows<__nv_bfloat16>(a);
  if (threadIdx.x == 0) a.starts[(long)blockIdx.y * gridDim.x + blockIdx.x].x = -1;
  Walk<Args> wk;
  if (!wk.init(a)) return;
  while (wk.segment(a)) {
    const int b = wk.b, hk = wk.hk, old = wk.keys - a.T, k1 = wk.k1;
    __nv_bfloat16* kc = static_cast<__nv_bfloat16*>(a.kc) + b * a.kcs[0] + hk * a.kcs[2];
    __nv_bfloat16* vc = static_cast<__nv_bfloat16*>(a.vc) + b * a.vcs[0] + hk * a.vcs[2];
    const int blocks = (k1 - wk.k0 + 15) / 16;  // of 16 keys; this warp's are w, w + 4, ...
    const int mine = blocks > w ? (blocks - w + 3) / 4 : 0;

    // 16 keys into stage st: lane l copies chunk l % NC of the rows l / NC, ...
    auto fetch = [&](int i) {
      const int j0 = wk.k0 + (w + 4 * i) * 16, c = lane % NC;
      const uint32_t dst = ring + i % kStages * kStage;
#pragma unroll
      for (int r = lane / NC; r < 16; r += 32 / NC) {
        const int j = j0 + r;
        const bool in = j < k1 && c * 8 < a.D;
        const __nv_bfloat16 *ks = kc + j * a.kcs[1] + c * 8, *vs = vc + j * a.vcs[1] + c * 8;
        if (in && j >= old) {  // a new token
          const long long at = (((long long)b * a.T + j - old) * a.Hkv + hk) * a.D + c * 8;
          const __nv_bfloat16 *kn = static_cast<const __nv_bfloat16*>(a.k) + at,
                              *vn = static_cast<const __nv_bfloat16*>(a.v) + at;
          if (blockIdx.y == 0) {
            *reinterpret_cast<uint4*>(kc + j * a.kcs[1] + c * 8) = *reinterpret_cast<const uint4*>(kn);
            *reinterpret_cast<uint4*>(vc + j * a.vcs[1] + c * 8) = *reinterpret_cast<const uint4*>(vn);
          }
          ks = kn, vs = vn;
        }
        const uint32_t at = dst + r * kRowB + ((c ^ (r & 7)) << 4);
        cp_async16(at, in ? ks : kc, in);
        cp_async16(at + kHalf, in ? vs : vc, in);
      }
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < mine) fetch(i);
      cp_async_commit();
    }
    // q as A fragments: rows lane / 4 + {0, 8}, columns 2 (lane % 4) + {0, 1} + {0, 8}
    uint32_t qf[MB][DP / 16][4];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = row0 + 16 * mb + lane / 4 + 8 * x;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (r < a.R ? row_at(a, b, hk, r) : 0);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int c = 16 * k + 8 * y + 2 * (lane % 4);
            qf[mb][k][x + 2 * y] = r < a.R && c < a.D ? *reinterpret_cast<const uint32_t*>(q + c) : 0u;
          }
      }
    float acc[MB][NC][4], m[MB][2], l[MB][2];
    int last[MB][2];  // last key that the row sees
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m[mb][x] = -INFINITY, l[mb][x] = 0.f;
        last[mb][x] = min(k1 - 1, old + (row0 + 16 * mb + lane / 4 + 8 * x) / a.G);
      }
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[mb][n][x] = 0.f;
    }
    for (int i = 0; i < mine; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      if (i + kStages - 1 < mine) fetch(i + kStages - 1);  // over the stage read in the pass before
      cp_async_commit();
      const uint32_t st = ring + i % kStages * kStage;
      const int j0 = wk.k0 + (w + 4 * i) * 16;
      float s[MB][2][4] = {};
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        uint32_t kf[4];
        const int key = (lane >> 4) * 8 + (lane & 7), c = 2 * k + ((lane >> 3) & 1);
        ldsm4(kf, st + key * kRowB + ((c ^ (key & 7)) << 4));
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          mma16816(s[mb][0], qf[mb][k], kf[0], kf[1]);
          mma16816(s[mb][1], qf[mb][k], kf[2], kf[3]);
        }
      }
      uint32_t pf[MB][4];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        if (j0 + 15 > old || j0 + 15 >= k1) {  // new tokens' causal order, the segment's end
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (j0 + 8 * n + 2 * (lane % 4) + (x & 1) > last[mb][x >> 1]) s[mb][n][x] = -INFINITY;
        }
        bool raise = false;
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float top = fmaxf(fmaxf(s[mb][0][2 * x], s[mb][0][2 * x + 1]), fmaxf(s[mb][1][2 * x], s[mb][1][2 * x + 1]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * a.c;
          f[x] = 1.f;
          if (top - m[mb][x] > 8.f) {  // see the prompt kernel: P at most 2^8
            f[x] = ex2(m[mb][x] - top);
            m[mb][x] = top;
            raise = true;
          }
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) l[mb][x] *= f[x];
#pragma unroll
          for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[mb][n][x] *= f[x >> 1];
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float base = m[mb][x] == -INFINITY ? 0.f : m[mb][x];
            const float e0 = ex2(fmaf(s[mb][n][2 * x], a.c, -base)), e1 = ex2(fmaf(s[mb][n][2 * x + 1], a.c, -base));
            l[mb][x] += e0 + e1;
            pf[mb][2 * n + x] = pack_bf16(e0, e1);
          }
      }
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        uint32_t vf[4];
        const int key = ((lane >> 3) & 1) * 8 + (lane & 7), c = 2 * n + (lane >> 4);
        ldsm4_trans(vf, st + kHalf + key * kRowB + ((c ^ (key & 7)) << 4));
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          mma16816(acc[mb][2 * n], pf[mb], vf[0], vf[1]);
          mma16816(acc[mb][2 * n + 1], pf[mb], vf[2], vf[3]);
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();
    // the four warps' pieces: maxima and sums, then the scaled accumulators
    float* ml = reinterpret_cast<float*>(sm);            // [4][16 MB][2]
    float* part = ml + 4 * 16 * MB * 2;                  // [4][16 MB][DP]
    __syncthreads();
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[mb][x] += __shfl_xor_sync(0xffffffffu, l[mb][x], 1);
        l[mb][x] += __shfl_xor_sync(0xffffffffu, l[mb][x], 2);
        if (lane % 4 == 0) {
          float* p = ml + (w * 16 * MB + 16 * mb + lane / 4 + 8 * x) * 2;
          p[0] = m[mb][x], p[1] = l[mb][x];
        }
      }
    __syncthreads();
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 16 * mb + lane / 4 + 8 * x;
        float top = -INFINITY;
#pragma unroll
        for (int p = 0; p < 4; ++p) top = fmaxf(top, ml[(p * 16 * MB + r) * 2]);
        const float f = m[mb][x] == -INFINITY ? 0.f : ex2(m[mb][x] - top);
#pragma unroll
        for (int n = 0; n < NC; ++n)
          *reinterpret_cast<float2*>(part + (w * 16 * MB + r) * DP + 8 * n + 2 * (lane % 4)) =
              make_float2(acc[mb][n][2 * x] * f, acc[mb][n][2 * x + 1] * f);
      }
    __syncthreads();
    const long slot = wk.whole ? 0 : slot_of(a, wk) * 16 * MB;
    for (int i = threadIdx.x; i < 16 * MB * (DP / 4); i += kThreads) {
      const int rl = i / (DP / 4), c = i % (DP / 4) * 4, r = row0 + rl;
      if (r >= a.R || c >= a.D) continue;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int p = 0; p < 4; ++p) top = fmaxf(top, ml[(p * 16 * MB + rl) * 2]);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        // a piece without keys adds 0; one whose scores are all NaN has m = -inf too, and adds its l
        const float mp = ml[(p * 16 * MB + rl) * 2], base = top == -INFINITY ? 0.f : top;
        sum = fmaf(ex2(mp - base), ml[(p * 16 * MB + rl) * 2 + 1], sum);
        const float4 y = *reinterpret_cast<const float4*>(part + (p * 16 * MB + rl) * DP + c);
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

bool use_mma(const AttnDecodeProblem& p) {
  if (!p.bf16 || p.D % 8) return false;
  for (const void* x : {p.kc, p.vc})
    if ((uintptr_t)x & 15) return false;
  for (int i = 0; i < 3; ++i)
    if (p.kcs[i] % 8 || p.vcs[i] % 8) return false;
  return true;
}

struct Plan {
  bool mma;
  int rows, blocks, ctas;  // query rows per CTA, row blocks (grid.y), CTAs that share the units (grid.x)
};

// Two CTAs per SM (mma), four (CUDA cores).
Plan plan_of(const AttnDecodeProblem& p, bool mma) {
  Plan q;
  const int R = p.H / p.Hkv * p.T;
  q.mma = mma;
  q.rows = !mma ? kRows : R <= 16 ? 16 : 32;
  q.blocks = (R + q.rows - 1) / q.rows;
  q.ctas = ctas_for(p.B, p.Hkv, p.S, q.blocks, mma ? 2 : 4);
  return q;
}

size_t need(const Plan& q, int D) { return ws_bytes(q.blocks, q.ctas, q.rows, D); }

template <typename T>
cudaError_t run(const AttnDecodeProblem& p, cudaStream_t s) {
  const Plan pl = plan_of(p, use_mma(p));
  Args a;
  a.B = p.B, a.T = p.T, a.S = p.S, a.H = p.H, a.Hkv = p.Hkv, a.D = p.D, a.G = p.H / p.Hkv;
  a.R = a.G * p.T, a.c = p.scale * kLog2e;
  a.vec = p.D % 4 == 0 && !(((uintptr_t)p.kc | (uintptr_t)p.vc) & 15);
  for (int i = 0; i < 3; ++i) {
    a.kcs[i] = p.kcs[i], a.vcs[i] = p.vcs[i];
    a.vec = a.vec && p.kcs[i] % 4 == 0 && p.vcs[i] % 4 == 0;
  }
  a.q = p.q, a.k = p.k, a.v = p.v, a.kc = p.kc, a.vc = p.vc, a.lens = p.lens, a.o = p.o;
  unsigned char* ws = static_cast<unsigned char*>(p.ws);
  a.starts = reinterpret_cast<int4*>(ws);
  a.ml = reinterpret_cast<float*>(ws + ws_starts(pl.blocks, pl.ctas));
  a.acc = reinterpret_cast<float*>(ws + ws_starts(pl.blocks, pl.ctas) + ws_ml(pl.blocks, pl.ctas, pl.rows));
  const dim3 grid(pl.ctas, pl.blocks);
  cudaError_t e = cudaSuccess;
  auto mma = [&](auto kernel, int smem) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) kernel<<<grid, kThreads, smem, s>>>(a);
  };
  prof_before(s);
  if (pl.mma) {
    const int smem = 4 * kStages * 64 * (p.D <= 64 ? 64 : 128);
    if (p.D <= 64) pl.rows == 16 ? mma(attn_decode_mma_kernel<64, 1>, smem) : mma(attn_decode_mma_kernel<64, 2>, smem);
    else pl.rows == 16 ? mma(attn_decode_mma_kernel<128, 1>, smem) : mma(attn_decode_mma_kernel<128, 2>, smem);
  } else if (p.D <= 64) {
    attn_decode_simt_kernel<T, 64><<<grid, kThreads, 0, s>>>(a);
  } else {
    attn_decode_simt_kernel<T, 128><<<grid, kThreads, 0, s>>>(a);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  prof_after(s, kAttnDecode);
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
  e = cudaLaunchKernelEx(&cfg, attn_combine_kernel<T, 1, Args>, a, pl.ctas, pl.rows);
  prof_after(s, kAttnCombine);
  return e;
}

}  // namespace

// The larger of the two kernels' needs: which one runs depends on the caches'
// alignment, which a shape does not say.
size_t attn_decode_workspace(const AttnDecodeProblem& p) {
  return std::max(need(plan_of(p, true), p.D), need(plan_of(p, false), p.D));
}

cudaError_t attn_decode(const AttnDecodeProblem& p, cudaStream_t s) {
  return p.bf16 ? run<__nv_bfloat16>(p, s) : run<float>(p, s);
}

}  // namespace gdn
