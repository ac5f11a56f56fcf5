// Rotation of heads by position, shared by the kernels that norm, rotate and
// store rows of queries and keys.
//
// A row is the D values of one head of one token.  Its first R values are R / 2
// pairs, (i, i + R / 2) or, interleaved, (2 i, 2 i + 1); pair i of a token at
// position n is turned by the angle whose cosine and sine stand in row n of two
// tables:
//   y_a = x_a c - x_b s,   y_b = x_b c + x_a s.
// Each product and each sum is rounded once (no fused multiply-add), so that a
// rotated row has the same bits whichever kernel makes it, with or without a
// cache behind it.
//
// Lanes.  LR lanes share a row and hold whole pairs, V of them in a row, so that a
// pair never needs another lane: V = 8 (bf16) or 4 takes rows as 16-byte vectors
// (V = 4 of bf16: 8-byte ones), two per lane; V = 1 takes any D, R, stride and
// alignment, value by value.  Arithmetic goes by twos (f32x2) where V allows.
#pragma once

#include <type_traits>

#include "attn_tc.cuh"

namespace gdn {
namespace rope {

// V pairs as they lie in memory.
template <typename T, int V>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 a, b;
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 a, b;
};
template <>
struct Raw<float, 8> {
  float4 a, a2, b, b2;
};
template <>
struct Raw<float, 4> {
  float4 a, b;
};
template <typename T>
struct Raw<T, 1> {
  T a, b;
};

// Values that are worked on together: two, or one.
using tc::F2;
template <int V>
using Num = std::conditional_t<V == 1, float, F2>;
template <int V>
constexpr int kNums = V == 1 ? 1 : V / 2;

__device__ __forceinline__ float mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float add(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float total(float a) { return a; }
__device__ __forceinline__ void both(float& r, float x) { r = x; }
__device__ __forceinline__ F2 mul(F2 a, F2 b) { return tc::mul2(a, b); }
__device__ __forceinline__ F2 add(F2 a, F2 b) { return tc::add2(a, b); }
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) { return tc::fma2(a, b, c); }
__device__ __forceinline__ float2 parts(F2 a) { return tc::unpack(a); }
__device__ __forceinline__ F2 pair(float a, float b) { return tc::f2(a, b); }
__device__ __forceinline__ float total(F2 a) {
  const float2 p = parts(a);
  return p.x + p.y;
}
__device__ __forceinline__ void both(F2& r, float x) { r = pair(x, x); }
template <int V>
__device__ __forceinline__ Num<V> splat(float x) {
  Num<V> r;
  both(r, x);
  return r;
}

__device__ __forceinline__ F2 wide(uint32_t v) { return pair(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
__device__ __forceinline__ uint32_t thin(F2 v) {
  const float2 p = parts(v);
  return tc::pack_bf16(p.x, p.y);
}

// Where slot p (pairs p .. p + V - 1) of a row lies: offsets of its two halves,
// and whether it is rotated.  Past the rotated pairs a slot is 2 V values in a row;
// a lane without a slot reads the row's first.
template <int V>
struct Slot {
  int oa, ob;
  bool in, in_b, rot;
  template <bool IL>
  __device__ __forceinline__ void set(int p, int D, int R) {
    in = 2 * p < D;
    rot = in && 2 * p < R;
    if (IL) oa = 2 * p, ob = oa + V;
    else if (rot) oa = p, ob = p + R / 2;
    else oa = R + 2 * (p - R / 2), ob = oa + V;
    in_b = in && ob < D;  // an odd D leaves the last value without a partner
    if (!in) oa = ob = 0;
  }
};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load(const T* row, const Slot<V>& s) {
  Raw<T, V> r;
  if constexpr (V == 1) {
    r.a = s.in ? row[s.oa] : from_f32<T>(0.f);
    r.b = s.in_b ? row[s.ob] : from_f32<T>(0.f);
  } else {
    using X = decltype(r.a);
    r.a = *reinterpret_cast<const X*>(row + s.oa), r.b = *reinterpret_cast<const X*>(row + s.ob);
    if constexpr (sizeof(T) == 4 && V == 8) {
      r.a2 = *reinterpret_cast<const X*>(row + s.oa + 4), r.b2 = *reinterpret_cast<const X*>(row + s.ob + 4);
    }
  }
  return r;
}

// The slot's two halves as twos, in the order of memory.
template <typename T, int V>
__device__ __forceinline__ void halves(const Raw<T, V>& r, F2 (&x)[V / 2], F2 (&y)[V / 2]) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t *a = reinterpret_cast<const uint32_t*>(&r.a), *b = reinterpret_cast<const uint32_t*>(&r.b);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) x[i] = wide(a[i]), y[i] = wide(b[i]);
  } else {
    x[0] = pair(r.a.x, r.a.y), x[1] = pair(r.a.z, r.a.w), y[0] = pair(r.b.x, r.b.y), y[1] = pair(r.b.z, r.b.w);
    if constexpr (V == 8) {
      x[2] = pair(r.a2.x, r.a2.y), x[3] = pair(r.a2.z, r.a2.w), y[2] = pair(r.b2.x, r.b2.y), y[3] = pair(r.b2.z, r.b2.w);
    }
  }
}
// Neighbours (IL) into first and second values of pairs, and back: pairs 0 .. V / 2 - 1
// lie in x, the others in y.
template <int N>
__device__ __forceinline__ void apart(F2 (&x)[N], F2 (&y)[N]) {
  F2 a[N], b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 p = parts(2 * i < N ? x[2 * i % N] : y[2 * i % N]), q = parts(2 * i + 1 < N ? x[(2 * i + 1) % N] : y[(2 * i + 1) % N]);
    a[i] = pair(p.x, q.x), b[i] = pair(p.y, q.y);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = a[i], y[i] = b[i];
}
template <int N>
__device__ __forceinline__ void together(F2 (&x)[N], F2 (&y)[N]) {
  F2 a[N], b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 p = parts(x[i]), q = parts(y[i]);
    (2 * i < N ? a : b)[2 * i % N] = pair(p.x, q.x);
    (2 * i + 1 < N ? a : b)[(2 * i + 1) % N] = pair(p.y, q.y);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = a[i], y[i] = b[i];
}

// As pairs (a[i], b[i]) in fp32.
template <bool IL, typename T, int V>
__device__ __forceinline__ void widen(const Raw<T, V>& r, Num<V> (&a)[kNums<V>], Num<V> (&b)[kNums<V>]) {
  if constexpr (V == 1) {
    a[0] = to_f32(r.a), b[0] = to_f32(r.b);
  } else {
    halves(r, a, b);
    if (IL) apart(a, b);
  }
}
template <bool IL, typename T, int V>
__device__ __forceinline__ void store(T* row, const Slot<V>& s, const Num<V> (&a)[kNums<V>], const Num<V> (&b)[kNums<V>]) {
  if constexpr (V == 1) {
    if (s.in) row[s.oa] = from_f32<T>(a[0]);
    if (s.in_b) row[s.ob] = from_f32<T>(b[0]);
  } else {
    if (!s.in) return;
    constexpr int N = V / 2;
    F2 x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = a[i], y[i] = b[i];
    if (IL) together(x, y);
    if constexpr (sizeof(T) == 2) {
      Raw<T, V> r;
      uint32_t *u = reinterpret_cast<uint32_t*>(&r.a), *v = reinterpret_cast<uint32_t*>(&r.b);
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = thin(x[i]), v[i] = thin(y[i]);
      *reinterpret_cast<decltype(r.a)*>(row + s.oa) = r.a;
      *reinterpret_cast<decltype(r.b)*>(row + s.ob) = r.b;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 p = parts(x[i]), q = parts(x[i + 1]), u = parts(y[i]), v = parts(y[i + 1]);
        *reinterpret_cast<float4*>(row + s.oa + 2 * i) = make_float4(p.x, p.y, q.x, q.y);
        *reinterpret_cast<float4*>(row + s.ob + 2 * i) = make_float4(u.x, u.y, v.x, v.y);
      }
    }
  }
}

// The cosines and sines of a slot's pairs at a position (row: its tables' row, p: the
// slot's first pair).
template <int V>
struct Angles {
  Num<V> c[kNums<V>], s[kNums<V>];
  // rot: whether the slot is rotated at all (what else is loaded is not used)
  __device__ __forceinline__ void set(const float* cos, const float* sin, long long row, int p, bool rot) {
    row += rot ? p : 0;
    if constexpr (V == 1) {
      c[0] = cos[row], s[0] = sin[row];
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(cos + row + i), y = *reinterpret_cast<const float4*>(sin + row + i);
        c[i / 2] = pair(x.x, x.y), c[i / 2 + 1] = pair(x.z, x.w);
        s[i / 2] = pair(y.x, y.y), s[i / 2 + 1] = pair(y.z, y.w);
      }
    }
  }
  // Value by value: products and sums of twos came out fused, with one rounding.
  __device__ __forceinline__ static void turn1(float& a, float& b, float c, float s) {
    const float x = a, y = b;
    a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  }
  __device__ __forceinline__ void turn(Num<V> (&a)[kNums<V>], Num<V> (&b)[kNums<V>]) const {
#pragma unroll
    for (int i = 0; i < kNums<V>; ++i) {
      if constexpr (V == 1) {
        turn1(a[i], b[i], c[i], s[i]);
      } else {
        float2 x = parts(a[i]), y = parts(b[i]);
        const float2 p = parts(c[i]), q = parts(s[i]);
        turn1(x.x, y.x, p.x, q.x), turn1(x.y, y.y, p.y, q.y);
        a[i] = pair(x.x, x.y), b[i] = pair(y.x, y.y);
      }
    }
  }
  // The same with fused multiply-adds, for rows that a norm has scaled before.
  __device__ __forceinline__ void turn_fused(Num<V> (&a)[kNums<V>], Num<V> (&b)[kNums<V>]) const {
    const Num<V> minus = splat<V>(-1.f);
#pragma unroll
    for (int i = 0; i < kNums<V>; ++i) {
      const Num<V> x = a[i], y = b[i];
      a[i] = fma(mul(y, s[i]), minus, mul(x, c[i]));
      b[i] = fma(y, c[i], mul(x, s[i]));
    }
  }
  // By the opposite angle (of a gradient).
  __device__ __forceinline__ void turn_back(Num<V> (&a)[kNums<V>], Num<V> (&b)[kNums<V>]) const {
    const Num<V> minus = splat<V>(-1.f);
#pragma unroll
    for (int i = 0; i < kNums<V>; ++i) {
      const Num<V> x = a[i], y = b[i];
      a[i] = fma(x, c[i], mul(y, s[i]));
      b[i] = fma(mul(x, s[i]), minus, mul(y, c[i]));
    }
  }
};

// Sum over the LR lanes of a row.
template <int LR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Whether rows at p with these strides (elements of e bytes) can go in vectors.
inline bool vectors(const void* p, const long long (&st)[3], size_t e) {
  const long long n = 16 / (long long)e;
  return !((uintptr_t)p & 15) && st[0] % n == 0 && st[1] % n == 0 && st[2] % n == 0;
}

}  // namespace rope
}  // namespace gdn
