// Dealing out the keys of a single-token attention call evenly over the CTAs,
// and joining what is split: shared by the kernels on contiguous caches and on
// pages.
//
// The (row b, key head, unit of 64 keys) triples of the whole batch, in that
// order, are dealt out evenly: CTA c takes the units [c U / N, (c + 1) U / N),
// whatever the rows' lengths are.  A CTA thus walks segments: runs of units of
// one (b, key head).  A segment that covers all of a row's keys writes the
// output; of the others each CTA has at most one that goes on from the CTA
// before it (slot 2 c of the workspace) and one that starts a row that the next
// CTA goes on with (slot 2 c + 1).  A second kernel joins the slots of each such
// row: m = max m_p, o = sum exp(m_p - m) acc_p / sum exp(m_p - m) l_p.  No
// atomics: the order of every sum is fixed.
//
// `A` is a kernel's arguments: B, T, H, Hkv, D, G, R = G T (rows per key head),
// keys(b) (row b's keys in this call, 0 for none), o, and the workspace's starts
// [grid.y][grid.x] (the row that CTA c starts and does not end: x = b or -1,
// y = key head, z = last CTA), ml [grid.y][2 grid.x][rows][2] (maximum in
// exponents, sum) and acc [..][D].
#pragma once

#include <algorithm>

#include "attn_tc.cuh"

namespace gdn {
namespace split {

constexpr int kUnit = 64;      // keys per unit
constexpr int kMinUnits = 2;   // per CTA: fewer CTAs rather than shorter pieces
constexpr int kThreads = 128;
constexpr int kMaxCtas = 2048;

template <class A>
__device__ __forceinline__ int row_units(const A& a, int b) { return (a.keys(b) + kUnit - 1) / kUnit; }

// One CTA's walk through its units.
template <class A>
struct Walk {
  long u, end, U, base;  // next unit, end, all units, first unit of row b
  int N, b, units;       // CTAs that share the work; row and its units
  int hk, keys, k0, k1;  // the segment: key head, the row's keys, keys [k0, k1)
  bool starts, whole;    // it begins its row; it is all of it
  long row0;             // first unit of (b, hk)

  // All 128 threads; false if the CTA has no units.
  __device__ bool init(const A& a) {
    __shared__ long sums[kThreads + 1];
    __shared__ long at[2];
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    long mine = 0;
    for (int i = b0; i < b1; ++i) mine += (long)row_units(a, i) * a.Hkv;
    sums[threadIdx.x + 1] = mine;
    __syncthreads();
    if (threadIdx.x < 32) {  // prefix sums, four per lane
      const int l = threadIdx.x;
      long s[4], x = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = x += sums[4 * l + i + 1];
      long y = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long z = __shfl_up_sync(0xffffffffu, y, o);
        if (l >= o) y += z;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[4 * l + i + 1] = y - x + s[i];
      if (l == 0) sums[0] = 0;
    }
    __syncthreads();
    U = sums[kThreads];
    N = (int)min((long)gridDim.x, max(1L, U / kMinUnits));
    u = (long)blockIdx.x * U / N, end = ((long)blockIdx.x + 1) * U / N;
    if ((int)blockIdx.x >= N || u == end) return false;
    if (u >= sums[threadIdx.x] && u < sums[threadIdx.x + 1]) {
      long s = sums[threadIdx.x];
      int i = b0;
      for (;; ++i) {
        const long n = (long)row_units(a, i) * a.Hkv;
        if (u < s + n) break;
        s += n;
      }
      at[0] = i, at[1] = s;
    }
    __syncthreads();
    b = (int)at[0], base = at[1];
    units = row_units(a, b);
    return true;
  }
  __device__ bool segment(const A& a) {
    if (u == end) return false;
    while (u >= base + (long)units * a.Hkv) {
      base += (long)units * a.Hkv;
      units = row_units(a, ++b);
    }
    hk = (int)((u - base) / units);
    const int unit = (int)((u - base) % units), n = (int)min(end - u, (long)(units - unit));
    row0 = u - unit;
    keys = a.keys(b);
    k0 = unit * kUnit, k1 = min(keys, (unit + n) * kUnit);
    starts = unit == 0, whole = starts && n == units;
    u += n;
    return true;
  }
  // the CTA that has unit x
  __device__ int owner(long x) const { return (int)(((x + 1) * N - 1) / U); }
};

// Workspace slot of this CTA's piece, and the note for the joining kernel.
template <class A>
__device__ __forceinline__ long slot_of(const A& a, const Walk<A>& w) {
  if (w.starts && threadIdx.x == 0)
    a.starts[(long)blockIdx.y * gridDim.x + blockIdx.x] = make_int4(w.b, w.hk, w.owner(w.row0 + w.units - 1), 0);
  return (long)blockIdx.y * 2 * gridDim.x + 2 * blockIdx.x + (w.starts ? 1 : 0);
}

// Element offset of row r (token r / G, head hk G + r % G) in q and o.
template <class A>
__device__ __forceinline__ long long row_at(const A& a, int b, int hk, int r) {
  return (((long long)b * a.T + r / a.G) * a.H + hk * a.G + r % a.G) * a.D;
}

// One CTA per (row of a block, CTA that starts a row it does not end): slots 2 c + 1,
// 2 (c + 1), 2 (c + 2), ... of the row.  P > 1, for few rows in many pieces: one CTA of
// P times 128 threads per (row of a block, b, key head), which finds the CTA that
// starts it; the P groups of threads take every P-th slot, and their sums are added
// in order.
template <typename T, int P, class A>
__global__ void __launch_bounds__(P * kThreads) attn_combine_kernel(A a, int ctas, int rows) {
  __shared__ float f[kMaxCtas];
  __shared__ float red[8 * P];
  __shared__ __align__(16) float sums[P > 1 ? 4 * P * kThreads : 1];
  tc::grid_dep_wait();
  const int r = blockIdx.z * rows + blockIdx.y, th = threadIdx.x, d = th % kThreads, part = th / kThreads;
  const int4* starts = a.starts + (long)blockIdx.z * ctas;
  int c0 = blockIdx.x;
  if constexpr (P > 1) {
    __shared__ int found;
    if (th == 0) found = -1;
    __syncthreads();
    for (int i = th; i < ctas; i += P * kThreads)
      if (starts[i].x >= 0 && starts[i].x * a.Hkv + starts[i].y == (int)blockIdx.x) found = i;  // one at most
    __syncthreads();
    c0 = found;
    if (c0 < 0) return;
  }
  const int4 st = starts[c0];
  if (st.x < 0 || r >= a.R) return;
  const int n = st.z - c0 + 1;
  auto at = [&](int i) {
    return ((long)blockIdx.z * 2 * ctas + (i ? 2 * (c0 + i) : 2 * c0 + 1)) * rows + blockIdx.y;
  };
  float m = -INFINITY;
  for (int i = th; i < n; i += P * kThreads) m = fmaxf(m, a.ml[2 * at(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((th & 31) == 0) red[th >> 5] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int i = 1; i < 4 * P; ++i) m = fmaxf(m, red[i]);
  float sum = 0.f;
  for (int i = th; i < n; i += P * kThreads) {
    const float mi = a.ml[2 * at(i)], e = mi == -INFINITY ? 0.f : exp2f(mi - m);
    f[i] = e;
    sum = fmaf(e, a.ml[2 * at(i) + 1], sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((th & 31) == 0) red[4 * P + (th >> 5)] = sum;
  __syncthreads();
  sum = red[4 * P];
#pragma unroll
  for (int i = 1; i < 4 * P; ++i) sum += red[4 * P + i];
  float x = 0.f;
  if (P > 1 && a.D % 4 == 0) {  // 32 groups of a vector each, and their sums in order
    constexpr int N = P * kThreads / 32;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    const int c = th % 32 * 4;
    if (c < a.D) {
#pragma unroll 8
      for (int i = th / 32; i < n; i += N) {
        const float4 y = *reinterpret_cast<const float4*>(a.acc + at(i) * a.D + c);
        v.x = fmaf(f[i], y.x, v.x), v.y = fmaf(f[i], y.y, v.y), v.z = fmaf(f[i], y.z, v.z), v.w = fmaf(f[i], y.w, v.w);
      }
    }
    *reinterpret_cast<float4*>(sums + th * 4) = v;
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int i = 0; i < N; ++i) x += sums[i * kThreads + d];
  } else {
    if (d < a.D) {
#pragma unroll 8
      for (int i = part; i < n; i += P) x = fmaf(f[i], a.acc[at(i) * a.D + d], x);
    }
    if constexpr (P > 1) {
      sums[th] = x;
      __syncthreads();
      if (part > 0) return;
#pragma unroll
      for (int i = 1; i < P; ++i) x += sums[i * kThreads + d];
    }
  }
  if (d >= a.D) return;
  static_cast<T*>(a.o)[row_at(a, st.x, st.y, r) + d] = from_f32<T>(sum == 0.f ? 0.f : x / sum);
}

// At most as many CTAs as run at once (per_sm on each SM), and no more than there
// are pieces of kMinUnits units in full caches of S slots.
inline int ctas_for(long B, int Hkv, long S, int blocks, long per_sm) {
  const long units = B * Hkv * ((S + kUnit - 1) / kUnit);
  const long most = std::max(1L, std::min(units / kMinUnits, (long)kMaxCtas));
  return (int)std::min(most, std::max(1L, per_sm * tc::sm_count() / blocks));
}

// The workspace: starts, ml, acc.
inline size_t ws_starts(int blocks, int ctas) { return align_up((size_t)blocks * ctas * sizeof(int4), 256); }
inline size_t ws_ml(int blocks, int ctas, int rows) {
  return align_up((size_t)blocks * 2 * ctas * rows * 2 * sizeof(float), 256);
}
inline size_t ws_bytes(int blocks, int ctas, int rows, int D) {
  return ws_starts(blocks, ctas) + ws_ml(blocks, ctas, rows) + (size_t)blocks * 2 * ctas * rows * D * sizeof(float);
}

}  // namespace split
}  // namespace gdn
