// Building blocks of the attention kernels on the tensor cores (bf16): tensor
// maps of strided token tensors, MMAs with A in TMEM, packed fp32 arithmetic,
// and bounded waits that give up together.
#pragma once

#include <math.h>

#include <algorithm>
#include <cmath>

#include "attn.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace tc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The tiles' swizzle wants shared memory that starts at a multiple of 1024
// bytes, which is where the dynamic part of a kernel without static arrays starts.
__device__ __forceinline__ bool aligned_smem(const void* sm) {
  if ((smem_u32(sm) & 1023) == 0) return true;
  if (threadIdx.x == 0) atomicExch(&g_file_status, GDN_ERR_ALIGN);
  return false;
}

// ---------------------------------------------------------------- waits

// One poll with the hardware's own suspend limit.
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// What the roles of a CTA tell each other about a wait that runs out.
struct Liveness {
  int dead;         // a wait ran out: everyone gives up
  int progress[2];  // counted up by the issuing thread per iteration and by the scheduler per CTA it asks for
};

// Bounded wait for a hand-over within an iteration or two, which take microseconds;
// it also gives up once another warp of the CTA has (live->dead != 0), and running
// out of polls sets that: after about a second, as a poll that nothing answers was
// measured to last 7800 clocks (and after 2 ms even if one lasted 20).  Kept small: it
// stands at every hand-over, and what does not fit the instruction cache is fetched
// again at every turn of a job.
__device__ __forceinline__ bool wait_live(uint64_t* bar, uint32_t parity, volatile Liveness* live) {
  if (try_wait(bar, parity)) return true;
#pragma unroll 1
  for (uint32_t i = 0; i < (1u << 18); ++i) {
    if (try_wait(bar, parity)) return true;
    if (live->dead) return false;
  }
  live->dead = 1;
  return false;
}

// The same for a wait that may rightly last a whole job (the scheduler's; a warp's
// without rows in a job).  A job has no longest time, so what runs out is `patience`
// clocks of the SM (2^31: about a second) in which nothing has moved: all roles hang
// on the issuing thread and, between jobs, on the scheduler.
constexpr uint32_t kPatience = 1u << 31;
__device__ __forceinline__ bool wait_job(uint64_t* bar, uint32_t parity, volatile Liveness* live,
                                         uint32_t patience = kPatience) {
  uint32_t since = clock();
  int seen = live->progress[0] + live->progress[1];
#pragma unroll 1
  while (!try_wait(bar, parity)) {
    if (live->dead) return false;
    if ((uint32_t)clock() - since <= patience) continue;
    const int now = live->progress[0] + live->progress[1];
    if (now == seen) live->dead = 1;
    seen = now;
    since = clock();
  }
  return true;
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

// The waits for a whole warp.  Where one lane polls, that orders its accesses alone
// behind the barrier; the others', of shared memory next, need the __syncwarp of
// warp_wait_data.  What follows warp_wait_live is a tcgen05.ld of the whole warp, or
// nothing (the __syncwarp costs the forward 5 % at its hand-over of S).  Once per job
// every lane polls for itself (1 % less than one lane and the __syncwarp at 74 us).
__device__ __forceinline__ bool warp_wait_live(uint64_t* bar, uint32_t parity, volatile Liveness* live) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_live(bar, parity, live);
  return __shfl_sync(0xffffffffu, ok, 0);
}
__device__ __forceinline__ bool warp_wait_data(uint64_t* bar, uint32_t parity, volatile Liveness* live) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_live(bar, parity, live);
  __syncwarp();
  return __shfl_sync(0xffffffffu, ok, 0);
}
__device__ __forceinline__ bool warp_wait_job(uint64_t* bar, uint32_t parity, volatile Liveness* live,
                                              uint32_t patience = kPatience) {
  return __all_sync(0xffffffffu, wait_job(bar, parity, live, patience));
}

// A position in a ring of n barriers: its index and the parity of its use.  A
// consumer waits for full[i] with ph; a producer for empty[i] with ph ^ 1,
// which a fresh barrier passes.
template <int n>
struct Ring {
  int i = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++i == n) i = 0, ph ^= 1;
  }
};

// After giving up: waits (bounded) for the loads last issued to each stage of
// a ring whose next stage is r, so that nothing is written at exit.
template <int n>
__device__ __forceinline__ void drain_loads(uint64_t* full, const Ring<n>& r) {
  for (int i = 0; i < n; ++i) mbar_wait(full + i, i < r.i ? r.ph : r.ph ^ 1, 10000);
}

// ---------------------------------------------------------------- tiles of a persistent CTA
//
// A CTA works on its own tile and then takes over tiles of CTAs that have not
// started (cluster launch control), so that setting up barriers and TMEM
// happens once per SM and the next tile's loads overlap the last one's
// epilogue, while tiles still go out in the order of the grid, heaviest first.
// One warp runs the scheduler: when the thread that issues the MMAs is some
// iterations from the end of a tile it gets and decodes the next one and puts it
// into one of two slots, from which every other warp takes it.  (Asking earlier
// would deal the tiles out before it is known which SMs are free first: 1.6 times
// the time for a few long sequences.)
struct __align__(16) TileSlots {
  int job[2][12];  // what the roles need to know of a tile; [11] = 0: no more tiles
  uint4 response;
  uint64_t full[2], empty[2], response_full;
  uint64_t soon;  // the issuing thread is near the end of a job

  __device__ void init(int takers) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, takers);
    }
    mbar_init(&response_full, 1);
    mbar_init(&soon, 1);
  }
};

// The next tile's job, for one lane (whole = false) or a whole warp; NULL: none.
// It stays in place until the taker says done.
__device__ __forceinline__ const int* next_job(TileSlots* ts, const Ring<2>& r, bool whole, volatile Liveness* live) {
  const bool ok = whole ? warp_wait_job(ts->full + r.i, r.ph, live) : wait_job(ts->full + r.i, r.ph, live);
  const int* j = ts->job[r.i];
  return ok && j[11] ? j : nullptr;
}
__device__ __forceinline__ void job_done(TileSlots* ts, Ring<2>& r, bool whole) {
  if (whole) __syncwarp();
  if (!whole || (threadIdx.x & 31) == 0) mbar_arrive(ts->empty + r.i);
  r.next();
}

// The u-th job's slot in a batch: the batch rows go out in groups (see
// batch_group), a group's tiles in order or, with `back`, in reverse: the tiles
// with the most work first.
__device__ __forceinline__ int batch_slot(int u, int B, int tiles, int group, bool back) {
  const int g = u / (group * tiles), x = u - g * group * tiles, rows = min(group, B - g * group);
  return (g * group + x % rows) * tiles + (back ? tiles - 1 - x / rows : x / rows);
}

// Batch rows of a group.  With the heaviest tiles of the whole batch first, every
// row's streamed side (`bytes` a row) is in use at once and does not stay in L2; with
// groups of 24 MB it does.  A group still has one and a half jobs per SM, for an even
// end, and the groups are about equal.  Measured, 16 rows of 2048 tokens, 8 heads,
// D 128 (8.4 MB a row), one group -> eight: q 239 -> 202 us, kv 246 -> 223; four:
// 206, 221; forward one -> four: 140 -> 137.
inline int batch_group(int B, double bytes, long jobs) {
  const double fit = std::max(24e6 / std::max(1.0, bytes), 1.5 * sm_count() / (double)std::max(1L, jobs));
  const int groups = std::max(1, (int)(B / std::max(1.0, std::min((double)B, std::floor(fit)))));
  return (B + groups - 1) / groups;
}

// Scheduler warp: puts a job into the next slot.
__device__ __forceinline__ bool put_job(TileSlots* ts, Ring<2>& r, const int (&j)[12], volatile Liveness* live) {
  if (!warp_wait_live(ts->empty + r.i, r.ph ^ 1, live)) return false;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < 12; i += 4)
      *reinterpret_cast<int4*>(ts->job[r.i] + i) = make_int4(j[i], j[i + 1], j[i + 2], j[i + 3]);
    mbar_arrive(ts->full + r.i);
  }
  __syncwarp();
  r.next();
  return true;
}

// Scheduler warp: takes over a CTA that has not started; its index in x, or
// false if there is none left (after which this must not be called again).
__device__ __forceinline__ bool next_cta(TileSlots* ts, uint32_t& ph, int& x, volatile Liveness* live) {
  if ((threadIdx.x & 31) == 0) {
    mbar_arrive_expect_tx(&ts->response_full, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_u32(&ts->response)),
        "r"(smem_u32(&ts->response_full))
        : "memory");
  }
  __syncwarp();
  if (!warp_wait_data(&ts->response_full, ph, live)) {
    mbar_wait(&ts->response_full, ph, 10000);  // nothing may still be written at exit (bounded)
    return false;
  }
  ph ^= 1;
  uint32_t got, at = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "+r"(at)
      : "r"(smem_u32(&ts->response))
      : "memory");
  fence_async_shared();  // the response is overwritten by the next request
  __syncwarp();
  x = (int)at;
  return got != 0;
}

// The scheduler warp.  decode(cta, job) fills a job or says that the CTA's tile is
// empty; early(job) and late(job) do what else a running job needs from this
// warp, before and after the next job is put out (they read it from its slot,
// which is rewritten only by the job after the next).
template <class Decode, class Early, class Late>
__device__ __forceinline__ void schedule(TileSlots* slots, volatile Liveness* live, Decode decode, Early early, Late late) {
  Ring<2> put;
  int cta = blockIdx.x, j[12];
  uint32_t ph = 0, soon_ph = 0;
  bool left = true, fresh = true;
  int asked = 0;
  const volatile int* now = nullptr;
  for (;;) {
    if (now) {
      if (!early(now) || !warp_wait_job(&slots->soon, soon_ph, live)) break;
      soon_ph ^= 1;
    }
    bool more = false;
    while (left && !more) {  // the next CTA whose tile is not empty
      if (!fresh) left = next_cta(slots, ph, cta, live);
      fresh = false;
      live->progress[1] = ++asked;  // thousands of empty packed sequences may lie in a row
      if (left) more = decode(cta, j);
    }
    j[11] = more;
    const volatile int* next = slots->job[put.i];
    if (!put_job(slots, put, j, live)) break;
    if (now && !late(now)) break;
    if (!more) break;
    now = next;
  }
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

// The products of the attention kernels.  The descriptors step from MMA to MMA
// and are hidden from the optimiser in between: as constants off a loop
// invariant base it would keep all of them in registers and spill.
__device__ __forceinline__ void step_desc(uint64_t& d, uint32_t bytes) {
  d += bytes >> 4;
  asm volatile("" : "+l"(d));
}

// D = A B^T over DP columns: both tiles of 128 rows, K-major in shared memory
template <int DP>
__device__ __forceinline__ void mma_rows(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t id = idesc_bf16(128, 128, false, false);
#pragma unroll
  for (int k = 0; k < DP / 16; ++k) {
    if (k) {
      step_desc(a, k % 4 ? 32 : 16384 - 96);
      step_desc(b, k % 4 ? 32 : 16384 - 96);
    }
    mma_bf16(d, a, b, id, k > 0);
  }
}

// D (+)= A B over 16 n: A in TMEM, its K-step k at column a + (k / per) * skip +
// (k % per) * 8; B rows of a tile, DP columns, in shared memory (MN-major)
template <int DP, int n, int per = n, int skip = 0>
__device__ __forceinline__ void mma_sum(uint32_t d, uint32_t a, uint64_t b, bool acc) {
  constexpr uint32_t id = idesc_bf16(128, DP, false, true);
#pragma unroll
  for (int k = 0; k < n; ++k) {
    if (k) step_desc(b, 2048);
    mma_bf16_ts(d, a + (k / per) * skip + (k % per) * 8, b, id, acc || k > 0);
  }
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

// 16 columns of packed values, without the wait
__device__ __forceinline__ void tmem_st16_start(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A warp's 16 lanes x 64 columns (shape 16x256b, from the lane of taddr on):
// v[4 g + 2 a + e] is lane t / 4 + 8 a, column 8 g + 2 (t % 4) + e.  A row is
// spread over four neighbouring threads, so two warps can share a
// sub-partition's 32 lanes and a row still needs no exchange between warps.
__device__ __forceinline__ void tmem_ld16x64_start(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// 16 lanes x 32 packed columns (shape 16x128b): r[2 g + a] is lane t / 4 + 8 a,
// column 4 g + t % 4.
__device__ __forceinline__ void tmem_st16x32_start(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
        "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 16 lanes x 32 columns and back, with the waits (shape 16x256b).
__device__ __forceinline__ void tmem_ld16x32(uint32_t taddr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                      "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tmem_st16x32(uint32_t taddr, const float (&v)[16]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
        "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
  tmem_st_wait();
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 1 / x and log2 x, the hardware approximations (1 ulp; 2^-22)
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// ---------------------------------------------------------------- epilogue

// Writes 16 rows x 32 columns [c0, c0 + 32) held as by tmem_ld16x32, times f[a]
// per row half a, as bf16: row r goes to base + r * stride (elements), rows below
// `rows` and columns below D are written.  The four threads of a row trade their
// 4-byte pieces so that each has 16 bytes, and a row 64, to store.
__device__ __forceinline__ void store_rows16x32(const float (&v)[16], const float (&f)[2], __nv_bfloat16* base,
                                                long long stride, int rows, int c0, int D) {
  const int t = threadIdx.x & 31, q = t & 3, c = c0 + 8 * q;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    uint32_t w[4];  // piece q of the 8-column groups 0 .. 3
#pragma unroll
    for (int g = 0; g < 4; ++g) w[g] = pack_bf16(v[4 * g + 2 * a] * f[a], v[4 * g + 2 * a + 1] * f[a]);
    auto swap = [&](uint32_t& x, uint32_t& y, bool up, int off) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x : y, off);
      if (up) x = got;
      else y = got;
    };
    swap(w[0], w[1], q & 1, 1);
    swap(w[2], w[3], q & 1, 1);
    swap(w[0], w[2], q & 2, 2);
    swap(w[1], w[3], q & 2, 2);  // now pieces 0 .. 3 of group q
    const int r = t / 4 + 8 * a;
    if (r < rows && c < D) *reinterpret_cast<uint4*>(base + r * stride + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
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
#pragma unroll 1
  for (int c = r0 * 8 + lane; c < 128 * 8; c += 32)
#pragma unroll
    for (int i = 0; i < NH; ++i) *reinterpret_cast<uint4*>(tile + i * 16384 + c * 16) = make_uint4(0, 0, 0, 0);
  fence_async_shared();
  __syncwarp();
}

}  // namespace tc
}  // namespace gdn
