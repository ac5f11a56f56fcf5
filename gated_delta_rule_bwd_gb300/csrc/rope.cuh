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
// Lanes.  LR lanes share a row and hold whole pairs, V of them in a row: with
// V = 4 a lane has two vectors of four values (rows of whole 16-byte vectors on
// 16-byte boundaries), and a pair never needs another lane.  V = 1 takes any D,
// R, stride and alignment, value by value.
#pragma once

#include "attn_tc.cuh"

namespace gdn {
namespace rope {

// V pairs as they lie in memory.
template <typename T, int V>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 a, b;
};
template <>
struct Raw<float, 4> {
  float4 a, b;
};
template <typename T>
struct Raw<T, 1> {
  T a, b;
};

__device__ __forceinline__ float4 wide(uint2 v) {
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ float4 wide(float4 v) { return v; }
__device__ __forceinline__ void thin(const float4& v, uint2& o) {
  o = make_uint2(tc::pack_bf16(v.x, v.y), tc::pack_bf16(v.z, v.w));
}
__device__ __forceinline__ void thin(const float4& v, float4& o) { o = v; }

// Where slot p (pairs p .. p + V - 1) of a row lies: offsets of its two halves,
// and whether it is rotated.  Past the rotated pairs a slot is 2 V values in a row.
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
  }
};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load(const T* row, const Slot<V>& s) {
  Raw<T, V> r;
  if constexpr (V == 4) {
    using X = decltype(r.a);
    r.a = r.b = X{};
    if (s.in) r.a = *reinterpret_cast<const X*>(row + s.oa), r.b = *reinterpret_cast<const X*>(row + s.ob);
  } else {
    r.a = s.in ? row[s.oa] : from_f32<T>(0.f);
    r.b = s.in_b ? row[s.ob] : from_f32<T>(0.f);
  }
  return r;
}

// As pairs (a[i], b[i]) in fp32.  A slot of neighbours in memory (IL) is taken apart.
template <bool IL, typename T, int V>
__device__ __forceinline__ void widen(const Raw<T, V>& r, float (&a)[V], float (&b)[V]) {
  if constexpr (V == 4) {
    const float4 x = wide(r.a), y = wide(r.b);
    if (IL) {
      a[0] = x.x, b[0] = x.y, a[1] = x.z, b[1] = x.w, a[2] = y.x, b[2] = y.y, a[3] = y.z, b[3] = y.w;
    } else {
      a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w, b[0] = y.x, b[1] = y.y, b[2] = y.z, b[3] = y.w;
    }
  } else {
    a[0] = to_f32(r.a), b[0] = to_f32(r.b);
  }
}
// Back to the order of memory: the slot's two halves.
template <bool IL>
__device__ __forceinline__ void halves(const float (&a)[4], const float (&b)[4], float4& x, float4& y) {
  if (IL) {
    x = make_float4(a[0], b[0], a[1], b[1]), y = make_float4(a[2], b[2], a[3], b[3]);
  } else {
    x = make_float4(a[0], a[1], a[2], a[3]), y = make_float4(b[0], b[1], b[2], b[3]);
  }
}
template <bool IL, typename T, int V>
__device__ __forceinline__ void store(T* row, const Slot<V>& s, const float (&a)[V], const float (&b)[V]) {
  if constexpr (V == 4) {
    if (!s.in) return;
    Raw<T, 4> r;
    float4 x, y;
    halves<IL>(a, b, x, y);
    thin(x, r.a), thin(y, r.b);
    *reinterpret_cast<decltype(r.a)*>(row + s.oa) = r.a;
    *reinterpret_cast<decltype(r.b)*>(row + s.ob) = r.b;
  } else {
    if (s.in) row[s.oa] = from_f32<T>(a[0]);
    if (s.in_b) row[s.ob] = from_f32<T>(b[0]);
  }
}

// The cosines and sines of a slot's pairs at a position; p: its first pair.
template <int V>
__device__ __forceinline__ void angles(const float* cos, const float* sin, long long row, int p, bool rot, float (&c)[V],
                                       float (&s)[V]) {
  if constexpr (V == 4) {
    float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (rot) x = *reinterpret_cast<const float4*>(cos + row + p), y = *reinterpret_cast<const float4*>(sin + row + p);
    c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w, s[0] = y.x, s[1] = y.y, s[2] = y.z, s[3] = y.w;
  } else {
    c[0] = rot ? cos[row + p] : 1.f;
    s[0] = rot ? sin[row + p] : 0.f;
  }
}

template <int V>
__device__ __forceinline__ void rotate(const float (&c)[V], const float (&s)[V], float (&a)[V], float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float x = a[i], y = b[i];
    a[i] = __fsub_rn(__fmul_rn(x, c[i]), __fmul_rn(y, s[i]));
    b[i] = __fadd_rn(__fmul_rn(y, c[i]), __fmul_rn(x, s[i]));
  }
}

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
