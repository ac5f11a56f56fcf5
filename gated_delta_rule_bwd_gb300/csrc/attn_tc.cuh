// Building blocks of the attention kernels on the tensor cores (bf16): tensor
// maps of strided token tensors, MMAs with A in TMEM, packed fp32 arithmetic,
// and bounded waits that give up together.
#pragma once

#include <math.h>

#include "attn.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace tc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- waits

// Bounded wait that also gives up once another warp of the CTA has
// (*dead != 0); running out sets *dead.
__device__ __forceinline__ bool wait_live(uint64_t* bar, uint32_t parity, volatile int* dead) {
  for (uint32_t i = 0; i < 100000; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*dead) return false;
  }
  *dead = 1;
  return false;
}

// One lane of a converged warp.  A role that one lane plays is put behind it
// as a whole: the compiler then knows that a single lane is active and feeds
// an MMA's descriptors straight to its uniform registers (9-17 cycles per MMA
// to issue; behind lane == 0 it is 60, as long as the MMA itself runs).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// wait_live for a whole warp: one lane polls.
__device__ __forceinline__ bool warp_wait_live(uint64_t* bar, uint32_t parity, volatile int* dead) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_live(bar, parity, dead);
  return __shfl_sync(0xffffffffu, ok, 0);
}

// ---------------------------------------------------------------- MMA with A in TMEM

// D[tmem] (+)= A[tmem] * B[smem]^T: A is K-major, two bf16 of a row per 32-bit
// column, so 16 values of K are 8 columns.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ---------------------------------------------------------------- TMEM in flight

// 32 columns without the wait; the values may be used after tmem_landed().
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Ties 32 loaded values to the wait before it: no use of them moves above.
__device__ __forceinline__ void tmem_landed(float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                      "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// 32 columns of packed values, without the wait
__device__ __forceinline__ void tmem_st32_start(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st16_start(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ---------------------------------------------------------------- arithmetic

struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// 2^x, the hardware approximation (2 ulp; 0 for -inf)
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- tensor maps

// [B, T, H, D] bf16 with any aligned strides (in elements: batch, token, head);
// box = 64 values x 1 head x 128 tokens, 128-byte swizzle.  Rows past T and
// values past D read as zero.
inline cudaError_t make_attn_map(CUtensorMap* m, const void* ptr, int B, int T, int H, int D,
                                 const long long (&st)[3]) {
  auto enc = get_encoder();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
  // a dimension of length 1 is never stepped over: any legal stride will do
  cuuint64_t strides[3] = {H > 1 ? (cuuint64_t)st[2] * 2 : 16, T > 1 ? (cuuint64_t)st[1] * 2 : 16,
                           B > 1 ? (cuuint64_t)st[0] * 2 : 16};
  cuuint32_t box[4] = {64, 1, 128, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Whether such a map can be made: 16-byte base and strides, below 2^40 bytes.
inline bool attn_map_ok(const void* ptr, int B, int T, int H, int D, const long long (&st)[3]) {
  if (((uintptr_t)ptr & 15) || D % 8) return false;
  const int n[3] = {B, T, H};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (st[i] <= 0 || st[i] % 8 || st[i] >= (1LL << 38))) return false;
  return true;
}

// Loads a tile of 128 tokens x 64 NH values: NH boxes of 16 KB, one after another.
template <int NH>
__device__ __forceinline__ void load_tile(void* dst, const CUtensorMap* tm, uint64_t* bar, int h, int t, int b) {
#pragma unroll
  for (int i = 0; i < NH; ++i) tma_load_4d(static_cast<unsigned char*>(dst) + i * 16384, tm, bar, 64 * i, h, t, b);
}

// Zeroes rows [r0, 128) of a tile (one warp) and makes that visible to the
// tensor core.  Packed sequences: the rows belong to the next sequence, and a
// product with a zero probability would still carry over its infinities.
template <int NH>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int r0, int lane) {
#pragma unroll
  for (int i = 0; i < NH; ++i)
    for (int c = r0 * 8 + lane; c < 128 * 8; c += 32)
      *reinterpret_cast<uint4*>(tile + i * 16384 + c * 16) = make_uint4(0, 0, 0, 0);
  fence_async_shared();
  __syncwarp();
}

}  // namespace tc
}  // namespace gdn
