// Causal attention on the tensor cores, backward: bf16, D a multiple of 8 up
// to 128 (padded with zeros to 64 or 128).
//
// With P = exp2(c S - lse log2 e), S = Q K^T, dP = dO V^T, dS = P (dP - delta):
//   dV = P^T dO,   dK = scale dS^T Q,   dQ = scale dS K.
// Two kernels, each with its sums in TMEM for all of its work and no atomics,
// so that results do not depend on the order of CTAs:
//   kv: a CTA owns 128 keys of one key head and walks the queries that see
//       them, for every head of the group; it works on the transposes
//       S^T = K Q^T and dP^T = V dO^T, whose rows (TMEM lanes) are its keys,
//       so that P^T and dS^T are the A operands (in TMEM) of the products.
//   q:  a CTA owns 128 queries of one head and walks their keys; dS is the A
//       operand of dS K.
// That is seven products per tile pair instead of the five of a single pass
// that adds dQ up in memory; in exchange dQ is written once, in bf16.
//
// Four groups of four warps each own 32 of the 128 columns of a tile (a thread
// owns a row's 32 values), warp 16 issues the TMA loads, warp 17 the MMAs, warp
// 18 zeroes the rows of a packed sequence's last tile that belong to the next
// sequence, warp 19 loads lse and delta (kv kernel).  A bf16 operand is written
// over the columns its own warps have read: group g's 32 values of a row into
// columns 32 g .. 32 g + 15 of the tile.
//
// delta is made by the q kernel, which runs first: it has dO in shared memory
// and reads o once.  delta = sum_j P_ij dP_ij as well, and where the rows' keys
// are a single tile the kernel takes that sum, in fp32, instead of do . o with
// o's bf16 rounding: with few keys dP and delta nearly cancel.

#include <math.h>

#include "attn_tc.cuh"

namespace gdn {

cudaError_t attn_tc_bwd_read_and_clear_status(int* status) {
  return tc::read_and_clear_file_status(status);
}

namespace {

using namespace tc;

constexpr int kCompute = 512, kThreads = kCompute + 128;
// 96 registers a thread at launch: 512 * 104 + 128 * 64 = 640 * 96
constexpr int kRegCompute = 104, kRegOther = 64;

template <int DP>
struct Cfg {
  static constexpr int NH = DP / 64;
  static constexpr int kTile = 128 * DP * 2;
  // kv: K, V, then three stages of Q and two of dO.  q: Q, dO, three of K, two
  // of V.  (The scores of iteration i + 1 read Q or K before the last product
  // of iteration i does: with two stages the load of i + 1 would start late.)
  static constexpr int kStats = 7 * kTile;  // kv: [2][2][128] floats (lse, delta); q: [4][128]
  static constexpr int kBar = kStats + 2 * 1024;
  static constexpr int kSmem = kBar + 384;  // at most 227 KB: no slack for an alignment
};

struct Args {
  AttnSeqs sq;
  int H, Hkv, D, tiles;  // tiles: 128-row tiles per batch row (0: packed)
  float c, scale;
  const float* lse;
  float* delta;
  const __nv_bfloat16* o;
  __nv_bfloat16 *dq, *dk, *dv;
};

// The TMEM column of K-step k of an operand written by the four column groups.
__device__ __forceinline__ uint32_t a_col(int k) { return (k >> 1) * 32 + (k & 1) * 8; }

// K-major product over DP: D = A B^T (both tiles of 128 rows in shared memory)
template <int DP>
__device__ __forceinline__ void mma_rows(uint32_t d, uint64_t da, uint64_t db) {
  constexpr uint32_t id = idesc_bf16(128, 128, false, false);
#pragma unroll
  for (int k = 0; k < DP / 16; ++k) {
    const uint32_t off = (k / 4) * 16384 + (k % 4) * 32;
    mma_bf16(d, desc_at(da, off), desc_at(db, off), id, k > 0);
  }
}

// D (+)= A B over 128: A in TMEM (see a_col), B a tile of 128 rows, DP columns
template <int DP>
__device__ __forceinline__ void mma_sum(uint32_t d, uint32_t a, uint64_t db, bool acc) {
  constexpr uint32_t id = idesc_bf16(128, DP, false, true);
#pragma unroll
  for (int k = 0; k < 8; ++k) mma_bf16_ts(d, a + a_col(k), desc_at(db, k * 2048), id, acc || k > 0);
}

// n fp32 columns of an accumulator row, times f, as bf16 to dst[c0 .. c0 + n)
// (what is below D); dst NULL: not stored
template <int n>
__device__ __forceinline__ void store_acc(uint32_t taddr, float f, __nv_bfloat16* dst, int c0, int D) {
#pragma unroll
  for (int q = 0; q < n / 32; ++q) {
    float x[32];
    tmem_ld32(taddr + 32 * q, x);
#pragma unroll
    for (int y = 0; y < 32; y += 8) {
      uint4 w;
      w.x = pack_bf16(x[y] * f, x[y + 1] * f), w.y = pack_bf16(x[y + 2] * f, x[y + 3] * f);
      w.z = pack_bf16(x[y + 4] * f, x[y + 5] * f), w.w = pack_bf16(x[y + 6] * f, x[y + 7] * f);
      const int c = c0 + 32 * q + y;
      if (dst && c < D) *reinterpret_cast<uint4*>(dst + c) = w;
    }
  }
}

// ---------------------------------------------------------------- dK, dV

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_bwd_kv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                      Args a) {
  using C = Cfg<DP>;
  extern __shared__ __align__(1024) unsigned char sm[];
  float* stats = reinterpret_cast<float*>(sm + C::kStats);      // [2][lse | delta][128]
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(sm + C::kBar);
  uint64_t* q_full = kv_full + 1;     // [3]
  uint64_t* q_empty = q_full + 3;     // [3]
  uint64_t* do_full = q_empty + 3;    // [2]
  uint64_t* do_empty = do_full + 2;   // [2]
  uint64_t* st_full = do_empty + 2;   // [2]
  uint64_t* st_empty = st_full + 2;   // [2]
  uint64_t* s_full = st_empty + 2;
  uint64_t* p_full = s_full + 1;
  uint64_t* dp_full = p_full + 1;
  uint64_t* ds_full = dp_full + 1;
  uint64_t* acc_full = ds_full + 1;
  uint64_t* landed = acc_full + 1;    // a head's last tiles are there; foreign rows are zero
  uint64_t* fixed = landed + 1;
  uint64_t* drain = fixed + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t kS = 0, kDP = 128, kDV = 256, kDK = 256 + DP;  // TMEM columns
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (!aligned_smem(sm)) return;
  // the tiles that the most queries see first
  const int hk = blockIdx.x % a.Hkv, u = blockIdx.x / a.Hkv;
  const int slot = a.tiles ? u % a.sq.B * a.tiles + u / a.sq.B : u;
  AttnTile t;
  if (!a.sq.get<true>(slot, 128, t)) return;
  const int G = a.H / a.Hkv, j0 = t.tile * 128, shift = t.lk - t.lq;
  const int i0 = max(0, j0 - shift) / 128;                      // first query tile that sees a key here
  const int ni = max(0, (t.lq + 127) / 128 - i0), N = ni * G;   // per head; all iterations
  const bool fix = a.sq.cu_q && t.lq % 128;                     // a head's last tile has foreign rows

  if (threadIdx.x == kCompute) {
    *dead = 0;
    mbar_init(kv_full, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(do_full + i, 1);
      mbar_init(do_empty + i, 1);
      mbar_init(st_full + i, 1);
      mbar_init(st_empty + i, 16);
    }
    mbar_init(s_full, 1);
    mbar_init(p_full, 16);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 16);
    mbar_init(acc_full, 1);
    mbar_init(landed, 1);
    mbar_init(fixed, 1);
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 17) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  cta_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
    if (warp == 16 && N && elect_one()) {
      // ------------------------------------------------------------ loads
      mbar_arrive_expect_tx(kv_full, 2 * C::kTile);
      load_tile<C::NH>(sm, &tm_k, kv_full, hk, t.k0 + j0, t.b);
      load_tile<C::NH>(sm + C::kTile, &tm_v, kv_full, hk, t.k0 + j0, t.b);
      int it = 0;
      for (; it < N; ++it) {
        const int sq = it % 3, sd = it & 1, h = hk * G + it / ni, row = t.q0 + (i0 + it % ni) * 128;
        if (it >= 3 && !wait_live(q_empty + sq, (it / 3 - 1) & 1, dead)) break;
        mbar_arrive_expect_tx(q_full + sq, C::kTile);
        load_tile<C::NH>(sm + (2 + sq) * C::kTile, &tm_q, q_full + sq, h, row, t.b);
        if (it >= 2 && !wait_live(do_empty + sd, (it / 2 - 1) & 1, dead)) {
          mbar_wait(q_full + sq, (it / 3) & 1, 10000);
          break;
        }
        mbar_arrive_expect_tx(do_full + sd, C::kTile);
        load_tile<C::NH>(sm + (5 + sd) * C::kTile, &tm_do, do_full + sd, h, row, t.b);
      }
      if (*dead) {  // nothing may still be written at exit (bounded)
        mbar_wait(kv_full, 0, 10000);
        for (int x = max(0, it - 3); x < it; ++x) mbar_wait(q_full + x % 3, (x / 3) & 1, 10000);
        for (int x = max(0, it - 2); x < it; ++x) mbar_wait(do_full + (x & 1), (x >> 1) & 1, 10000);
      }
    } else if (warp == 17 && N && elect_one()) {
      // ------------------------------------------------------------ MMAs
      const uint64_t rows = sw128_desc(smem_u32(sm), 16, 1024);      // K-major
      const uint64_t cols = sw128_desc(smem_u32(sm), 16384, 1024);   // MN-major, 64-column blocks 16 KB apart
      auto q_tile = [&](int it) { return (uint32_t)(2 + it % 3) * C::kTile; };
      auto do_tile = [&](int it) { return (uint32_t)(5 + (it & 1)) * C::kTile; };
      // S^T of iteration it; a head's last tiles are cleaned first
      auto scores = [&](int it) {
        if (!wait_live(q_full + it % 3, (it / 3) & 1, dead)) return false;
        if (fix && it % ni == ni - 1) {
          if (!wait_live(do_full + (it & 1), (it >> 1) & 1, dead)) return false;
          mbar_arrive(landed);
          if (!wait_live(fixed, (it / ni) & 1, dead)) return false;
        }
        mma_rows<DP>(tmem + kS, rows, desc_at(rows, q_tile(it)));
        mma_commit(s_full);
        return true;
      };
      auto dprobs = [&](int it) {
        if (!wait_live(do_full + (it & 1), (it >> 1) & 1, dead)) return false;
        mma_rows<DP>(tmem + kDP, desc_at(rows, C::kTile), desc_at(rows, do_tile(it)));
        mma_commit(dp_full);
        return true;
      };
      bool ok = wait_live(kv_full, 0, dead) && scores(0) && dprobs(0);
      for (int it = 0; it < N && ok; ++it) {
        ok = wait_live(p_full, it & 1, dead);
        if (!ok) break;
        tc_fence_after();
        mma_sum<DP>(tmem + kDV, tmem + kS, desc_at(cols, do_tile(it)), it > 0);
        mma_commit(do_empty + (it & 1));
        if (it + 1 < N && !(ok = scores(it + 1))) break;  // over P^T, behind the product that reads it
        ok = wait_live(ds_full, it & 1, dead);
        if (!ok) break;
        tc_fence_after();
        mma_sum<DP>(tmem + kDK, tmem + kDP, desc_at(cols, q_tile(it)), it > 0);
        mma_commit(q_empty + it % 3);
        if (it + 1 < N) ok = dprobs(it + 1);
      }
      mma_commit(acc_full);
      if (*dead) {
        mma_commit(drain);
        mbar_wait(drain, 0, 10000);
      }
    } else if (warp == 18 && fix && N) {
      for (int g = 0; g < G; ++g) {
        const int it = g * ni + ni - 1;
        bool ok = true;
        if (lane == 0) ok = wait_live(landed, g & 1, dead);
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        zero_rows<C::NH>(sm + (2 + it % 3) * C::kTile, t.lq % 128, lane);
        zero_rows<C::NH>(sm + (5 + (it & 1)) * C::kTile, t.lq % 128, lane);
        if (lane == 0) mbar_arrive(fixed);
      }
    } else if (warp == 19) {
      float ls[4], dl[4];  // an iteration ahead of the one that is stored
      auto fetch = [&](int it) {
        const int r = (i0 + it % ni) * 128 + lane;
        const long long at = ((long long)t.b * a.H + hk * G + it / ni) * a.sq.Tq + t.q0 + r;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const bool in = r + 32 * x < t.lq;
          ls[x] = in ? a.lse[at + 32 * x] * kLog2e : 0.f;
          dl[x] = in ? a.delta[at + 32 * x] : 0.f;
        }
      };
      if (N) fetch(0);
      for (int it = 0; it < N; ++it) {
        const int st = it & 1;
        if (it >= 2 && !warp_wait_live(st_empty + st, (it / 2 - 1) & 1, dead)) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          stats[st * 256 + lane + 32 * x] = ls[x];
          stats[st * 256 + 128 + lane + 32 * x] = dl[x];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(st_full + st);
        if (it + 1 < N) fetch(it + 1);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- P^T, dS^T
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegCompute));
    const int g = warp >> 2, key = j0 + (threadIdx.x & 127);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + kS + 32 * g, td = tmem + lanes + kDP + 32 * g;
    const F2 cc = f2(a.c, a.c);
    bool ok = true;
    for (int it = 0; it < N; ++it) {
      const int r = (i0 + it % ni) * 128;
      const float *lse = stats + (it & 1) * 256 + 32 * g, *delta = lse + 128;
      if (!(ok = warp_wait_live(st_full + (it & 1), (it >> 1) & 1, dead))) break;
      float p[32], n[32];
#pragma unroll
      for (int x = 0; x < 32; x += 4) *reinterpret_cast<float4*>(n + x) = *reinterpret_cast<const float4*>(lse + x);
      if (!(ok = warp_wait_live(s_full, it & 1, dead))) break;
      tc_fence_after();
      tmem_ld32_start(ts, p);
      tmem_ld_wait();
      tmem_landed(p);
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        const float2 e = unpack(fma2(f2(p[x], p[x + 1]), cc, f2(-n[x], -n[x + 1])));
        p[x] = ex2(e.x), p[x + 1] = ex2(e.y);
      }
      // queries [lo, hi) of this thread's columns see the key
      const int lo = key - shift - r - 32 * g, hi = t.lq - r - 32 * g;
      if (j0 + 127 > r + shift || r + 128 > t.lq) {
#pragma unroll
        for (int x = 0; x < 32; ++x) p[x] = x >= lo && x < hi ? p[x] : 0.f;
      }
      uint32_t w[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) w[x] = pack_bf16(p[2 * x], p[2 * x + 1]);
      tmem_st16_start(ts, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);

#pragma unroll
      for (int x = 0; x < 32; x += 4) *reinterpret_cast<float4*>(n + x) = *reinterpret_cast<const float4*>(delta + x);
      if (!(ok = warp_wait_live(dp_full, it & 1, dead))) break;
      tc_fence_after();
      float d[32];
      tmem_ld32_start(td, d);
      tmem_ld_wait();
      tmem_landed(d);
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        const float2 e = unpack(mul2(f2(p[x], p[x + 1]), add2(f2(d[x], d[x + 1]), f2(-n[x], -n[x + 1]))));
        d[x] = e.x, d[x + 1] = e.y;
      }
      if (r + 128 > t.lq) {  // dO rows past the sequence may hold anything
#pragma unroll
        for (int x = 0; x < 32; ++x) d[x] = x < hi ? d[x] : 0.f;
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) w[x] = pack_bf16(d[2 * x], d[2 * x + 1]);
      tmem_st16_start(td, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ds_full);
        mbar_arrive(st_empty + (it & 1));
      }
    }
    // groups 0 and 1 write dV, 2 and 3 dK, half of the columns each
    __nv_bfloat16* dst = g & 2 ? a.dk : a.dv;
    const int half = (g & 1) * (DP / 2);
    dst = key < t.lk ? dst + (((long long)t.b * a.sq.Tk + t.k0 + key) * a.Hkv + hk) * a.D : nullptr;
    if (N) {
      ok = ok && warp_wait_live(acc_full, 0, dead);
      tc_fence_after();
      if (ok) store_acc<DP / 2>(tmem + lanes + (g & 2 ? kDK : kDV) + half, g & 2 ? a.scale : 1.f, dst, half, a.D);
    } else if (dst && !(g & 1)) {
      for (int x = 0; x < a.D; x += 8) *reinterpret_cast<uint4*>(dst + x) = make_uint4(0, 0, 0, 0);
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *dead) report_timeout();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- dQ

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_bwd_q_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     Args a) {
  using C = Cfg<DP>;
  extern __shared__ __align__(1024) unsigned char sm[];
  float* part = reinterpret_cast<float*>(sm + C::kStats);        // [4][128]
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + C::kBar);  // Q and dO
  uint64_t* k_full = q_full + 1;      // [3]
  uint64_t* k_empty = k_full + 3;     // [3]
  uint64_t* v_full = k_empty + 3;     // [2]
  uint64_t* v_empty = v_full + 2;     // [2]
  uint64_t* s_full = v_empty + 2;     // [2]
  uint64_t* dp_full = s_full + 2;
  uint64_t* dp_read = dp_full + 1;
  uint64_t* ds_full = dp_read + 1;
  uint64_t* acc_full = ds_full + 1;
  uint64_t* landed = acc_full + 1;
  uint64_t* fixed = landed + 1;
  uint64_t* drain = fixed + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t kS = 0, kDP = 256, kDQ = 384;  // TMEM columns; S has two buffers
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (!aligned_smem(sm)) return;
  if (blockIdx.x == 0 && !a.sq.valid() && threadIdx.x == 0) atomicExch(&g_file_status, GDN_ERR_SEQLENS);
  const int h = blockIdx.x % a.H, u = blockIdx.x / a.H;
  const int slot = a.tiles ? u % a.sq.B * a.tiles + a.tiles - 1 - u / a.sq.B : gridDim.x / a.H - 1 - u;
  AttnTile t;
  if (!a.sq.get<false>(slot, 128, t)) return;
  const int r0 = t.tile * 128, shift = t.lk - t.lq, hk = h / (a.H / a.Hkv);
  const int nr = min(128, t.lq - r0);
  const int N = (max(0, min(t.lk, r0 + nr + shift)) + 127) / 128;  // key tiles that the rows see
  const bool fix = a.sq.cu_q && N * 128 > t.lk;                    // the last has foreign rows

  if (threadIdx.x == kCompute) {
    *dead = 0;
    mbar_init(q_full, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, 1);
      mbar_init(s_full + i, 1);
    }
    mbar_init(dp_full, 1);
    mbar_init(dp_read, 16);
    mbar_init(ds_full, 16);
    mbar_init(acc_full, 1);
    mbar_init(landed, 1);
    mbar_init(fixed, 1);
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 17) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  cta_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
    if (warp == 16 && N && elect_one()) {
      // ------------------------------------------------------------ loads
      mbar_arrive_expect_tx(q_full, 2 * C::kTile);
      load_tile<C::NH>(sm, &tm_q, q_full, h, t.q0 + r0, t.b);
      load_tile<C::NH>(sm + C::kTile, &tm_do, q_full, h, t.q0 + r0, t.b);
      int j = 0;
      for (; j < N; ++j) {
        const int sk = j % 3, sv = j & 1, row = t.k0 + j * 128;
        if (j >= 3 && !wait_live(k_empty + sk, (j / 3 - 1) & 1, dead)) break;
        mbar_arrive_expect_tx(k_full + sk, C::kTile);
        load_tile<C::NH>(sm + (2 + sk) * C::kTile, &tm_k, k_full + sk, hk, row, t.b);
        if (j >= 2 && !wait_live(v_empty + sv, (j / 2 - 1) & 1, dead)) {
          mbar_wait(k_full + sk, (j / 3) & 1, 10000);
          break;
        }
        mbar_arrive_expect_tx(v_full + sv, C::kTile);
        load_tile<C::NH>(sm + (5 + sv) * C::kTile, &tm_v, v_full + sv, hk, row, t.b);
      }
      if (*dead) {  // nothing may still be written at exit (bounded)
        mbar_wait(q_full, 0, 10000);
        for (int x = max(0, j - 3); x < j; ++x) mbar_wait(k_full + x % 3, (x / 3) & 1, 10000);
        for (int x = max(0, j - 2); x < j; ++x) mbar_wait(v_full + (x & 1), (x >> 1) & 1, 10000);
      }
    } else if (warp == 17 && N && elect_one()) {
      // ------------------------------------------------------------ MMAs
      const uint64_t rows = sw128_desc(smem_u32(sm), 16, 1024);
      const uint64_t cols = sw128_desc(smem_u32(sm), 16384, 1024);
      auto k_tile = [&](int j) { return (uint32_t)(2 + j % 3) * C::kTile; };
      auto v_tile = [&](int j) { return (uint32_t)(5 + (j & 1)) * C::kTile; };
      auto scores = [&](int j) {
        if (!wait_live(k_full + j % 3, (j / 3) & 1, dead)) return false;
        if (fix && j == N - 1) {
          mbar_arrive(landed);
          if (!wait_live(fixed, 0, dead)) return false;
        }
        mma_rows<DP>(tmem + kS + 128 * (j & 1), rows, desc_at(rows, k_tile(j)));
        mma_commit(s_full + (j & 1));
        return true;
      };
      auto dprobs = [&](int j) {
        if (!wait_live(v_full + (j & 1), (j >> 1) & 1, dead)) return false;
        mma_rows<DP>(tmem + kDP, desc_at(rows, C::kTile), desc_at(rows, v_tile(j)));
        mma_commit(dp_full);
        mma_commit(v_empty + (j & 1));
        return true;
      };
      bool ok = wait_live(q_full, 0, dead) && scores(0) && dprobs(0);
      for (int j = 0; j < N && ok; ++j) {
        if (j + 1 < N) {  // its buffer was read by dS K (j - 1), issued before
          ok = scores(j + 1) && wait_live(dp_read, j & 1, dead);
          if (!ok) break;
          tc_fence_after();
          if (!(ok = dprobs(j + 1))) break;
        }
        ok = wait_live(ds_full, j & 1, dead);
        if (!ok) break;
        tc_fence_after();
        mma_sum<DP>(tmem + kDQ, tmem + kS + 128 * (j & 1), desc_at(cols, k_tile(j)), j > 0);
        mma_commit(k_empty + j % 3);
      }
      mma_commit(acc_full);
      if (*dead) {
        mma_commit(drain);
        mbar_wait(drain, 0, 10000);
      }
    } else if (warp == 18 && fix) {
      bool ok = true;
      if (lane == 0) ok = wait_live(landed, 0, dead);
      if (__shfl_sync(0xffffffffu, ok, 0)) {
        zero_rows<C::NH>(sm + (2 + (N - 1) % 3) * C::kTile, t.lk - (N - 1) * 128, lane);
        if (lane == 0) mbar_arrive(fixed);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- dS
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegCompute));
    const int g = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t td = tmem + lanes + kDP + 32 * g;
    const long long at = ((long long)t.b * a.H + h) * a.sq.Tq + t.q0 + r0 + row;
    const long long at_o = (((long long)t.b * a.sq.Tq + t.q0 + r0 + row) * a.H + h) * a.D;
    const float lse = row < nr ? a.lse[at] * kLog2e : 0.f;
    // the sum over the four threads of a row
    auto row_sum = [&](float x) {
      part[g * 128 + row] = x;
      group_sync(1, kCompute);
      return part[row] + part[128 + row] + part[256 + row] + part[384 + row];
    };
    bool ok = true;
    float delta = 0.f;
    if (N > 1) {  // delta = do . o: a thread takes DP / 4 values of its row
      uint4 ov[DP / 32];
#pragma unroll
      for (int x = 0; x < DP / 32; ++x) {
        const int c = g * (DP / 4) + 8 * x;
        ov[x] = row < nr && c < a.D ? *reinterpret_cast<const uint4*>(a.o + at_o + c) : make_uint4(0, 0, 0, 0);
      }
      ok = warp_wait_live(q_full, 0, dead);
#pragma unroll
      for (int x = 0; x < DP / 32; ++x) {
        const int c = g * (DP / 4) + 8 * x;
        const uint4 dv = *reinterpret_cast<const uint4*>(sm + C::kTile + (c >> 6) * 16384 + sw_row_off(row, (c & 63) >> 3));
        const uint32_t o4[4] = {ov[x].x, ov[x].y, ov[x].z, ov[x].w}, d4[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          delta = fmaf(__uint_as_float(o4[y] << 16), __uint_as_float(d4[y] << 16), delta);
          delta = fmaf(__uint_as_float(o4[y] & 0xffff0000u), __uint_as_float(d4[y] & 0xffff0000u), delta);
        }
      }
      delta = row_sum(delta);
    }
    const F2 cc = f2(a.c, a.c), ls = f2(-lse, -lse);
    const int first = min(r0 + shift, t.lk - 1), last = min(r0 + row + shift, t.lk - 1);
    for (int j = 0; ok && j < N; ++j) {
      const uint32_t ts = tmem + lanes + kS + 128 * (j & 1) + 32 * g;
      if (!(ok = warp_wait_live(s_full + (j & 1), (j >> 1) & 1, dead))) {
        if (N == 1) row_sum(0.f);  // the other warps may be at its barrier
        break;
      }
      tc_fence_after();
      float p[32], d[32];
      tmem_ld32_start(ts, p);
      tmem_ld_wait();
      tmem_landed(p);
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        const float2 e = unpack(fma2(f2(p[x], p[x + 1]), cc, ls));
        p[x] = ex2(e.x), p[x + 1] = ex2(e.y);
      }
      if (!(ok = warp_wait_live(dp_full, j & 1, dead))) {
        if (N == 1) row_sum(0.f);
        break;
      }
      tc_fence_after();
      tmem_ld32_start(td, d);
      tmem_ld_wait();
      tmem_landed(d);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dp_read);
      if (j * 128 + 127 > first) {
        const int see = last - j * 128 - 32 * g;
#pragma unroll
        for (int x = 0; x < 32; ++x) p[x] = x <= see ? p[x] : 0.f, d[x] = x <= see ? d[x] : 0.f;
      }
      if (N == 1) {
        F2 sum = f2(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 32; x += 2) sum = fma2(f2(p[x], p[x + 1]), f2(d[x], d[x + 1]), sum);
        const float2 two = unpack(sum);
        delta = row_sum(two.x + two.y);
      }
      const F2 dl = f2(-delta, -delta);
      uint32_t w[16];
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        const float2 e = unpack(mul2(f2(p[x], p[x + 1]), add2(f2(d[x], d[x + 1]), dl)));
        w[x / 2] = pack_bf16(e.x, e.y);
      }
      tmem_st16_start(ts, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    if (g == 0 && row < nr) a.delta[at] = delta;
    __nv_bfloat16* dst = row < nr ? a.dq + at_o : nullptr;
    constexpr int kPart = DP / 4 < 32 ? 32 : DP / 4;  // columns a group writes
    if (N) {
      ok = ok && warp_wait_live(acc_full, 0, dead);
      tc_fence_after();
      if (ok && g * kPart < DP) store_acc<kPart>(tmem + lanes + kDQ + g * kPart, a.scale, dst, g * kPart, a.D);
    } else if (dst && g == 0) {
      for (int x = 0; x < a.D; x += 8) *reinterpret_cast<uint4*>(dst + x) = make_uint4(0, 0, 0, 0);
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *dead) report_timeout();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

template <int DP>
cudaError_t run(const AttnProblem& p, cudaStream_t s) {
  using C = Cfg<DP>;
  CUtensorMap mq, mk, mv, md;
  const long long ds[3] = {(long long)p.Tq * p.H * p.D, (long long)p.H * p.D, p.D};
  cudaError_t e = make_attn_map(&mq, p.q, p.B, p.Tq, p.H, p.D, p.qs);
  if (e == cudaSuccess) e = make_attn_map(&mk, p.k, p.B, p.Tk, p.Hkv, p.D, p.ks);
  if (e == cudaSuccess) e = make_attn_map(&mv, p.v, p.B, p.Tk, p.Hkv, p.D, p.vs);
  if (e == cudaSuccess) e = make_attn_map(&md, p.do_, p.B, p.Tq, p.H, p.D, ds);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_tc_bwd_kv_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_tc_bwd_q_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  Args a;
  a.sq = AttnSeqs::of(p);
  a.H = p.H, a.Hkv = p.Hkv, a.D = p.D;
  a.scale = p.scale, a.c = p.scale * kLog2e;
  a.lse = p.lse, a.delta = static_cast<float*>(p.ws), a.o = static_cast<const __nv_bfloat16*>(p.o);
  a.dq = static_cast<__nv_bfloat16*>(p.dq);
  a.dk = static_cast<__nv_bfloat16*>(p.dk), a.dv = static_cast<__nv_bfloat16*>(p.dv);
  a.tiles = p.cu_q ? 0 : (p.Tq + 127) / 128;
  prof_before(s);
  attn_tc_bwd_q_kernel<DP>
      <<<(unsigned)(AttnSeqs::slots(p, 128, false) * p.H), kThreads, C::kSmem, s>>>(mq, mk, mv, md, a);
  e = cudaGetLastError();
  prof_after(s, kAttnBwdQ);
  if (e != cudaSuccess) return e;
  a.tiles = p.cu_q ? 0 : (p.Tk + 127) / 128;
  prof_before(s);
  attn_tc_bwd_kv_kernel<DP>
      <<<(unsigned)(AttnSeqs::slots(p, 128, true) * p.Hkv), kThreads, C::kSmem, s>>>(mq, mk, mv, md, a);
  e = cudaGetLastError();
  prof_after(s, kAttnBwdKv);
  return e;
}

}  // namespace

cudaError_t attn_tc_bwd(const AttnProblem& p, cudaStream_t s) {
  return p.D <= 64 ? run<64>(p, s) : run<128>(p, s);
}

}  // namespace gdn
