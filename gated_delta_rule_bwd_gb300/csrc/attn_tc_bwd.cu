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
// owns a row's 32 values), warp 16 issues the TMA loads, warp 17 the MMAs, warp 18
// gets the next tiles and zeroes the rows of a packed sequence's last tile that
// belong to the next sequence, warp 19 loads lse and delta (kv kernel).  CTAs are
// persistent (see TileSlots).  One thread issues all MMAs, in the order in which
// their results are wanted (one per chain of products was no faster here and 21 %
// slower in the forward, where their MMAs interleave and both chains wait).
// It waits for a tile's loads while the products before it run.  A bf16 operand is
// written over the columns its own warps have read: group g's 32 values of a row
// into columns 32 g .. 32 g + 15 of the tile.
//
// delta is made by the q kernel, which runs first: it has dO in shared memory
// and reads o once.  delta = sum_j P_ij dP_ij as well, and where the rows' keys
// are a single tile the kernel takes that sum, in fp32, instead of do . o with
// o's bf16 rounding: with few keys dP and delta nearly cancel.
//
// Measured, 16 rows of 2048 tokens, 8 heads, D 128: q 192 us, kv 221 us, which is
// 1074 and 1244 TFLOP/s of their three and four products over the pairs seen; the
// tensor pipe is active about half of the time.  What bounds both is the chain
// of an iteration (scores, exponentials, P and dS into TMEM, products) and the
// turn of a job, some 11000 cycles for 8.5 iterations on average here.

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
  static constexpr int kSmem = kBar + 512;  // at most 227 KB: no slack for an alignment
};

struct Args {
  AttnSeqs sq;
  int H, Hkv, D, tiles;  // tiles: 128-row tiles per batch row (0: packed)
  int group;             // see batch_group
  float c, scale;
  const float* lse;
  float* delta;
  const __nv_bfloat16* o;
  __nv_bfloat16 *dq, *dk, *dv;
};

// A warp's 32 rows x n fp32 columns of an accumulator, times f, as bf16: row r to
// base + r * stride, columns from c0 on; rows below `rows`, columns below D.
template <int n>
__device__ __forceinline__ void store_acc(uint32_t taddr, float f, __nv_bfloat16* base, long long stride, int rows,
                                          int c0, int D) {
  const float ff[2] = {f, f};
#pragma unroll 1
  for (int q = 0; q < n / 16; ++q) {
    float x[16];
    const int r = 16 * (q & 1), c = 32 * (q >> 1);
    tmem_ld16x32(taddr + ((uint32_t)r << 16) + c, x);
    store_rows16x32(x, ff, base + r * stride, stride, rows - r, c0 + c, D);
  }
}

// A warp's 32 rows of D zeros.
__device__ __forceinline__ void store_zeros(__nv_bfloat16* base, long long stride, int rows, int D) {
  const int lane = threadIdx.x & 31;
  if (lane < rows)
    for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(base + lane * stride + c) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------- dK, dV

// A job: 128 keys of one key head.
enum { kHead, kB, kQ0, kLq, kK0, kNk, kI0, kNi, kJs };
// kQ0: the sequence's first query token; kK0: first key token; kNk: keys; kI0, kNi:
// first query tile that sees one, and number (per head); kJs: first query that
// sees the first key (may be negative).

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_bwd_kv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                      Args a) {
  using C = Cfg<DP>;
  extern __shared__ __align__(1024) unsigned char sm[];
  float* stats = reinterpret_cast<float*>(sm + C::kStats);  // [2][lse | delta][128]
  TileSlots* slots = reinterpret_cast<TileSlots*>(sm + C::kBar);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(slots + 1);
  uint64_t* v_full = k_full + 1;
  uint64_t* k_empty = v_full + 1;
  uint64_t* v_empty = k_empty + 1;
  uint64_t* q_full = v_empty + 1;     // [3]
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
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* landed = acc_empty + 1;   // a head's last tiles are there; foreign rows are zero
  uint64_t* fixed = landed + 1;
  uint64_t* drain = fixed + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile Liveness* live = reinterpret_cast<volatile Liveness*>(tmem_slot + 1);
  constexpr uint32_t kS = 0, kDP = 128, kAcc = 256;  // TMEM columns; dV, then dK
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.H / a.Hkv;

  if (!aligned_smem(sm)) return;
  if (threadIdx.x == kCompute) {
    live->dead = live->progress[0] = live->progress[1] = 0;
    slots->init(19);
    for (uint64_t* x : {k_full, v_full, k_empty, v_empty, s_full, dp_full, acc_full, landed, fixed, drain}) mbar_init(x, 1);
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
    for (uint64_t* x : {p_full, ds_full, acc_empty}) mbar_init(x, 16);
    fence_barrier_init();
    for (const CUtensorMap* x : {&tm_q, &tm_k, &tm_v, &tm_do}) tma_prefetch_desc(x);
  }
  if (warp == 17) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  cta_sync();
  const uint32_t tmem = *tmem_slot;
  const bool packed = a.sq.cu_q != nullptr;

  Ring<2> take;
  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
    if (warp == 16 && elect_one()) {
      // ------------------------------------------------------------ loads
      Ring<3> rq;
      Ring<2> rd;
      uint32_t kph = 0;
      bool ok = true;
      while (const int* j = ok ? next_job(slots, take, false, live) : nullptr) {
        const int hk = j[kHead], b = j[kB], k0 = j[kK0], i0 = j[kI0], ni = j[kNi], q0 = j[kQ0] + i0 * 128;
        job_done(slots, take, false);
        for (int h = hk * G, first = 1; h < (hk + 1) * G && ok; ++h)
          for (int i = 0; i < ni; ++i, first = 0) {
            if (first) {
              if (!(ok = wait_live(k_empty, kph ^ 1, live))) break;
              mbar_arrive_expect_tx(k_full, C::kTile);
              load_tile<C::NH>(sm, &tm_k, k_full, hk, k0, b);
            }
            if (!(ok = wait_live(q_empty + rq.i, rq.ph ^ 1, live))) break;
            mbar_arrive_expect_tx(q_full + rq.i, C::kTile);
            load_tile<C::NH>(sm + (2 + rq.i) * C::kTile, &tm_q, q_full + rq.i, h, q0 + i * 128, b);
            rq.next();
            if (first) {
              if (!(ok = wait_live(v_empty, kph ^ 1, live))) break;
              kph ^= 1;
              mbar_arrive_expect_tx(v_full, C::kTile);
              load_tile<C::NH>(sm + C::kTile, &tm_v, v_full, hk, k0, b);
            }
            if (!(ok = wait_live(do_empty + rd.i, rd.ph ^ 1, live))) break;
            mbar_arrive_expect_tx(do_full + rd.i, C::kTile);
            load_tile<C::NH>(sm + (5 + rd.i) * C::kTile, &tm_do, do_full + rd.i, h, q0 + i * 128, b);
            rd.next();
          }
      }
      if (live->dead) {  // nothing may still be written at exit (bounded)
        mbar_wait(k_full, kph, 10000);  // of a load that has only just begun, if any
        mbar_wait(k_full, kph ^ 1, 10000);
        mbar_wait(v_full, kph ^ 1, 10000);
        drain_loads(q_full, rq);
        drain_loads(do_full, rd);
      }
    } else if (warp == 17 && elect_one()) {
      // ------------------------------------------------------------ MMAs
      const uint64_t rows = sw128_desc(smem_u32(sm), 16, 1024);      // K-major
      const uint64_t cols = sw128_desc(smem_u32(sm), 16384, 1024);   // MN-major, 64-column blocks 16 KB apart
      Ring<3> rq, rk;   // Q for S^T (an iteration ahead) and for dK
      Ring<2> rd, rv;   // dO for dP^T (an iteration ahead) and for dV
      uint32_t kph = 0, ph = 0, fph = 0, aph = 0;
      int turns = 0;
      bool ok = true;
      auto have_q = [&] { return wait_live(q_full + rq.i, rq.ph, live); };
      auto have_do = [&] { return wait_live(do_full + rd.i, rd.ph, live); };
      // K and V are free behind a job's last scores and dP^T: the next job's are
      // loaded while this one ends
      auto scores = [&](bool last) {
        mma_rows<DP>(tmem + kS, rows, desc_at(rows, (2 + rq.i) * C::kTile));
        mma_commit(s_full);
        if (last) mma_commit(k_empty);
        rq.next();
      };
      auto dprobs = [&](bool last) {
        mma_rows<DP>(tmem + kDP, desc_at(rows, C::kTile), desc_at(rows, (5 + rd.i) * C::kTile));
        mma_commit(dp_full);
        if (last) mma_commit(v_empty);
        rd.next();
      };
      while (const int* j = ok ? next_job(slots, take, false, live) : nullptr) {
        const int ni = j[kNi], N = ni * G;
        const bool fix = packed && j[kLq] % 128;
        job_done(slots, take, false);
        if (!N) {
          mbar_arrive(&slots->soon);
          continue;
        }
        if (!(ok = wait_live(k_full, kph, live) && have_q())) break;
        scores(N == 1);
        if (!(ok = wait_live(v_full, kph, live) && have_do())) break;
        dprobs(N == 1);
        kph ^= 1;
        if (!(ok = wait_live(acc_empty, aph ^ 1, live))) break;  // the job before has read its sums
        aph ^= 1;
        int left = ni;  // iterations of the head
        ok = N == 1 || have_q();
#pragma unroll 1
        for (int it = 0; it < N && ok; ++it) {
          live->progress[0] = ++turns;
          if (it == max(0, N - 3)) mbar_arrive(&slots->soon);
          if (--left == 0) {
            left = ni;
            if (fix) {
              mbar_arrive(landed);
              if (!(ok = wait_live(fixed, fph, live))) break;
              fph ^= 1;
            }
          }
          if (!(ok = wait_live(p_full, ph, live))) break;
          tc_fence_after();
          mma_sum<DP, 8, 2, 32>(tmem + kAcc, tmem + kS, desc_at(cols, (5 + rv.i) * C::kTile), it > 0);
          mma_commit(do_empty + rv.i);
          rv.next();
          if (it + 1 < N) {
            scores(it + 2 == N);  // over P^T, behind the product that reads it
            if (!(ok = have_do())) break;
          }
          if (!(ok = wait_live(ds_full, ph, live))) break;
          ph ^= 1;
          tc_fence_after();
          mma_sum<DP, 8, 2, 32>(tmem + kAcc + DP, tmem + kDP, desc_at(cols, (2 + rk.i) * C::kTile), it > 0);
          mma_commit(q_empty + rk.i);
          rk.next();
          if (it + 1 < N) {
            dprobs(it + 2 == N);
            if (it + 2 < N) ok = have_q();
          }
        }
        mma_commit(acc_full);
      }
      if (live->dead) {
        mma_commit(drain);
        mbar_wait(drain, 0, 10000);
      }
    } else if (warp == 19) {
      // ------------------------------------------------------------ lse, delta
      Ring<2> rs;
      bool ok = true;
      while (const int* j = ok ? next_job(slots, take, true, live) : nullptr) {
        const int lq = j[kLq], i0 = j[kI0], ni = j[kNi];
        long long at = ((long long)j[kB] * a.H + j[kHead] * G) * a.sq.Tq + j[kQ0];
        job_done(slots, take, true);
        float ls[4], dl[4];  // an iteration ahead of the one that is stored
        auto fetch = [&](int i) {
          const int r = i * 128 + lane;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const bool in = r + 32 * x < lq;
            ls[x] = in ? a.lse[at + r + 32 * x] * kLog2e : 0.f;
            dl[x] = in ? a.delta[at + r + 32 * x] : 0.f;
          }
        };
        if (ni) fetch(i0);
        for (int g = 0; g < G && ok; ++g)
          for (int i = i0; i < i0 + ni; ++i) {
            if (!(ok = warp_wait_data(st_empty + rs.i, rs.ph ^ 1, live))) break;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              stats[rs.i * 256 + lane + 32 * x] = ls[x];
              stats[rs.i * 256 + 128 + lane + 32 * x] = dl[x];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(st_full + rs.i);
            rs.next();
            if (i + 1 == i0 + ni) at += a.sq.Tq;
            if (i + 1 < i0 + ni) fetch(i + 1);
            else if (g + 1 < G) fetch(i0);
          }
      }
    } else if (warp == 18) {
      // ------------------------------------------------------------ the next tiles; foreign rows
      int it = 0, head = 0;  // iterations of the jobs before; heads of this one
      uint32_t ph = 0;
      auto clean = [&](const volatile int* j) {
        if (!packed || j[kLq] % 128 == 0 || !j[kNi]) return true;
        if (!warp_wait_job(landed, ph, live)) return false;
        ph ^= 1;
        const int x = it + ++head * j[kNi] - 1;
        zero_rows<C::NH>(sm + (2 + x % 3) * C::kTile, j[kLq] % 128, lane);
        zero_rows<C::NH>(sm + (5 + (x & 1)) * C::kTile, j[kLq] % 128, lane);
        if (lane == 0) mbar_arrive(fixed);
        __syncwarp();
        return true;
      };
      schedule(
          slots, live,
          [&](int cta, int(&j)[12]) {
            // the tiles that the most queries see first (packed: of a sequence)
            const int u = cta / a.Hkv;
            AttnTile t;
            if (!a.sq.get<true>(a.tiles ? batch_slot(u, a.sq.B, a.tiles, a.group, false) : u, 128, t)) return false;
            const int j0 = t.tile * 128;
            j[kHead] = cta % a.Hkv, j[kB] = t.b, j[kQ0] = t.q0, j[kLq] = t.lq, j[kK0] = t.k0 + j0;
            j[kNk] = min(128, t.lk - j0), j[kJs] = j0 - (t.lk - t.lq);
            j[kI0] = max(0, j[kJs]) / 128, j[kNi] = max(0, (t.lq + 127) / 128 - j[kI0]);
            return true;
          },
          [&](const volatile int* j) {  // every head's last tiles but the last head's
            head = 0;
            for (int g = 1; g < G; ++g)
              if (!clean(j)) return false;
            return true;
          },
          [&](const volatile int* j) {
            const bool ok = clean(j);
            it += j[kNi] * G;
            return ok;
          });
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- P^T, dS^T
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegCompute));
    const int g = warp >> 2, key = threadIdx.x & 127, w0 = 32 * (warp & 3);
    const uint32_t lanes = (uint32_t)w0 << 16;
    const uint32_t ts = tmem + lanes + kS + 32 * g, td = tmem + lanes + kDP + 32 * g;
    const F2 cc = f2(a.c, a.c);
    Ring<2> rs;
    uint32_t ph = 0, aph = 0;
    bool ok = true;
    while (const int* j = ok ? next_job(slots, take, true, live) : nullptr) {
      const int ni = j[kNi], N = ni * G, lq = j[kLq], js = j[kJs];
      int r = j[kI0] * 128, left = ni;
#pragma unroll 1
      for (int it = 0; it < N; ++it) {
        const float *lse = stats + rs.i * 256 + 32 * g, *delta = lse + 128;
        if (!(ok = warp_wait_data(st_full + rs.i, rs.ph, live))) break;
        float p[32], n[32];
#pragma unroll
        for (int x = 0; x < 32; x += 4) *reinterpret_cast<float4*>(n + x) = *reinterpret_cast<const float4*>(lse + x);
        if (!(ok = warp_wait_live(s_full, ph, live))) break;
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
        const int lo = js + key - r - 32 * g, hi = lq - r - 32 * g;
        if (js + 127 > r || r + 128 > lq) {
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
        if (!(ok = warp_wait_live(dp_full, ph, live))) break;
        ph ^= 1;
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
        if (r + 128 > lq) {  // dO rows past the sequence may hold anything
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
          mbar_arrive(st_empty + rs.i);
        }
        rs.next();
        r += 128;
        if (--left == 0) left = ni, r = j[kI0] * 128;
      }
      if (!ok) break;
      // groups 0 and 1 write dV, 2 and 3 dK, half of the columns each
      const int half = (g & 1) * (DP / 2), which = g >> 1, rows = j[kNk] - w0;
      const long long stride = (long long)a.Hkv * a.D;
      __nv_bfloat16* dst = (which ? a.dk : a.dv) + (((long long)j[kB] * a.sq.Tk + j[kK0] + w0) * a.Hkv + j[kHead]) * a.D;
      job_done(slots, take, true);
      if (N) {
        if (!(ok = warp_wait_live(acc_full, aph, live))) break;
        aph ^= 1;
        tc_fence_after();
        store_acc<DP / 2>(tmem + lanes + kAcc + DP * which + half, which ? a.scale : 1.f, dst, stride, rows, half, a.D);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty);
      } else if (half == 0) {
        store_zeros(dst, stride, rows, a.D);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && live->dead) report_timeout();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- dQ

// A job: 128 queries of one head (kHead, kB as above).
enum { qQ0 = 2, qNr, qK0, qLk, qFirst, qN };
// qQ0: first query token; qNr: queries; qK0: the sequence's first key token; qLk:
// its keys; qFirst: last key that the first query sees; qN: key tiles seen.

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_bwd_q_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     Args a) {
  using C = Cfg<DP>;
  extern __shared__ __align__(1024) unsigned char sm[];
  float* part = reinterpret_cast<float*>(sm + C::kStats);  // [4][128]
  TileSlots* slots = reinterpret_cast<TileSlots*>(sm + C::kBar);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(slots + 1);
  uint64_t* do_full = q_full + 1;
  uint64_t* q_empty = do_full + 1;
  uint64_t* do_empty = q_empty + 1;
  uint64_t* k_full = do_empty + 1;    // [3]
  uint64_t* k_empty = k_full + 3;     // [3]
  uint64_t* v_full = k_empty + 3;     // [2]
  uint64_t* v_empty = v_full + 2;     // [2]
  uint64_t* s_full = v_empty + 2;     // [2]
  uint64_t* dp_full = s_full + 2;
  uint64_t* dp_read = dp_full + 1;
  uint64_t* ds_full = dp_read + 1;    // [2]: one per S buffer, as two dS may be ready at once
  uint64_t* part_full = ds_full + 2;
  uint64_t* acc_full = part_full + 1;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* landed = acc_empty + 1;
  uint64_t* fixed = landed + 1;
  uint64_t* drain = fixed + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile Liveness* live = reinterpret_cast<volatile Liveness*>(tmem_slot + 1);
  constexpr uint32_t kS = 0, kDP = 256, kDQ = 384;  // TMEM columns; S has two buffers
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.H / a.Hkv;

  if (!aligned_smem(sm)) return;
  if (blockIdx.x == 0 && !a.sq.valid() && threadIdx.x == 0) atomicExch(&g_file_status, GDN_ERR_SEQLENS);
  if (threadIdx.x == kCompute) {
    live->dead = live->progress[0] = live->progress[1] = 0;
    slots->init(18);
    for (uint64_t* x : {q_full, do_full, q_empty, do_empty, s_full, s_full + 1, dp_full, acc_full, landed, fixed, drain})
      mbar_init(x, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, 1);
    }
    for (uint64_t* x : {dp_read, ds_full, ds_full + 1, part_full, acc_empty}) mbar_init(x, 16);
    fence_barrier_init();
    for (const CUtensorMap* x : {&tm_q, &tm_k, &tm_v, &tm_do}) tma_prefetch_desc(x);
  }
  if (warp == 17) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  cta_sync();
  const uint32_t tmem = *tmem_slot;
  const bool packed = a.sq.cu_q != nullptr;

  Ring<2> take;
  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
    if (warp == 16 && elect_one()) {
      // ------------------------------------------------------------ loads
      Ring<3> rk;
      Ring<2> rv;
      uint32_t qph = 0;
      bool ok = true;
      while (const int* j = ok ? next_job(slots, take, false, live) : nullptr) {
        const int h = j[kHead], hk = h / G, b = j[kB], q0 = j[qQ0], k0 = j[qK0], N = j[qN];
        job_done(slots, take, false);
        if (!N) continue;
        if (!(ok = wait_live(q_empty, qph ^ 1, live))) break;
        mbar_arrive_expect_tx(q_full, C::kTile);
        load_tile<C::NH>(sm, &tm_q, q_full, h, q0, b);
        for (int x = 0; x < N; ++x) {
          if (!(ok = wait_live(k_empty + rk.i, rk.ph ^ 1, live))) break;
          mbar_arrive_expect_tx(k_full + rk.i, C::kTile);
          load_tile<C::NH>(sm + (2 + rk.i) * C::kTile, &tm_k, k_full + rk.i, hk, k0 + x * 128, b);
          rk.next();
          if (x == 0) {
            if (!(ok = wait_live(do_empty, qph ^ 1, live))) break;
            qph ^= 1;
            mbar_arrive_expect_tx(do_full, C::kTile);
            load_tile<C::NH>(sm + C::kTile, &tm_do, do_full, h, q0, b);
          }
          if (!(ok = wait_live(v_empty + rv.i, rv.ph ^ 1, live))) break;
          mbar_arrive_expect_tx(v_full + rv.i, C::kTile);
          load_tile<C::NH>(sm + (5 + rv.i) * C::kTile, &tm_v, v_full + rv.i, hk, k0 + x * 128, b);
          rv.next();
        }
      }
      if (live->dead) {  // nothing may still be written at exit (bounded)
        mbar_wait(q_full, qph, 10000);  // of a load that has only just begun, if any
        mbar_wait(q_full, qph ^ 1, 10000);
        mbar_wait(do_full, qph ^ 1, 10000);
        drain_loads(k_full, rk);
        drain_loads(v_full, rv);
      }
    } else if (warp == 17 && elect_one()) {
      // ------------------------------------------------------------ MMAs
      const uint64_t rows = sw128_desc(smem_u32(sm), 16, 1024);
      const uint64_t cols = sw128_desc(smem_u32(sm), 16384, 1024);
      Ring<3> rk, rd;   // K for S (a tile ahead) and for dQ
      Ring<2> rv, ss, sd;  // V; S buffer written, dS buffer read
      uint32_t qph = 0, fph = 0, aph = 0, rph = 0;
      int turns = 0;
      bool ok = true;
      auto have_k = [&](bool last) {
        if (!wait_live(k_full + rk.i, rk.ph, live)) return false;
        if (!last) return true;
        mbar_arrive(landed);
        const bool got = wait_live(fixed, fph, live);
        fph ^= 1;
        return got;
      };
      // Q and dO are free behind a job's last scores and dP (the warps that make
      // delta from dO have read the dP before, or N is 1 and none does): the next
      // job's are loaded while this one ends
      auto scores = [&](bool last) {
        mma_rows<DP>(tmem + kS + 128 * ss.i, rows, desc_at(rows, (2 + rk.i) * C::kTile));
        mma_commit(s_full + ss.i);
        if (last) mma_commit(q_empty);
        rk.next();
        ss.next();
      };
      auto dprobs = [&](bool last) {
        mma_rows<DP>(tmem + kDP, desc_at(rows, C::kTile), desc_at(rows, (5 + rv.i) * C::kTile));
        mma_commit(dp_full);
        if (last) mma_commit(do_empty);
        mma_commit(v_empty + rv.i);
        rv.next();
      };
      while (const int* j = ok ? next_job(slots, take, false, live) : nullptr) {
        const int N = j[qN];
        const bool fix = packed && N * 128 > j[qLk];
        job_done(slots, take, false);
        if (N <= 3) mbar_arrive(&slots->soon);  // before the scheduler is asked to clean the last tile
        if (!N) continue;
        if (!(ok = wait_live(q_full, qph, live) && have_k(fix && N == 1))) break;
        scores(N == 1);
        // the dP before (of the last job, too) has been read
        if (!(ok = wait_live(do_full, qph, live) && wait_live(v_full + rv.i, rv.ph, live) &&
                   wait_live(dp_read, rph ^ 1, live)))
          break;
        rph ^= 1;
        qph ^= 1;
        tc_fence_after();
        dprobs(N == 1);
        if (!(ok = wait_live(acc_empty, aph ^ 1, live))) break;
        aph ^= 1;
        ok = N == 1 || have_k(fix && N == 2);
#pragma unroll 1
        for (int x = 0; x < N && ok; ++x) {
          live->progress[0] = ++turns;
          if (x > 0 && x == N - 3) mbar_arrive(&slots->soon);
          if (x + 1 < N) {
            scores(x + 2 == N);  // over the dS of tile x - 1, behind the product that reads it
            if (!(ok = wait_live(v_full + rv.i, rv.ph, live) && wait_live(dp_read, rph ^ 1, live))) break;
            rph ^= 1;
            tc_fence_after();
            dprobs(x + 2 == N);
            if (x + 2 < N && !(ok = have_k(fix && x + 3 == N))) break;
          }
          if (!(ok = wait_live(ds_full + sd.i, sd.ph, live))) break;
          tc_fence_after();
          mma_sum<DP, 8, 2, 32>(tmem + kDQ, tmem + kS + 128 * sd.i, desc_at(cols, (2 + rd.i) * C::kTile), x > 0);
          mma_commit(k_empty + rd.i);
          rd.next();
          sd.next();
        }
        mma_commit(acc_full);
      }
      if (live->dead) {
        mma_commit(drain);
        mbar_wait(drain, 0, 10000);
      }
    } else if (warp == 18) {
      // ------------------------------------------------------------ the next tiles; foreign rows
      int it = 0;  // key tiles so far
      uint32_t ph = 0;
      const int ctas = gridDim.x;
      schedule(
          slots, live,
          [&](int cta, int(&j)[12]) {
            // the tiles with the most keys first (packed: of a sequence, the last sequence first)
            const int u = cta / a.H;
            const int slot = a.tiles ? batch_slot(u, a.sq.B, a.tiles, a.group, true) : ctas / a.H - 1 - u;
            AttnTile t;
            if (!a.sq.get<false>(slot, 128, t)) return false;
            const int r0 = t.tile * 128, nr = min(128, t.lq - r0);
            j[kHead] = cta % a.H, j[kB] = t.b, j[qQ0] = t.q0 + r0, j[qNr] = nr, j[qK0] = t.k0, j[qLk] = t.lk;
            j[qFirst] = r0 + t.lk - t.lq, j[qN] = (max(0, min(t.lk, j[qFirst] + nr)) + 127) / 128;
            return true;
          },
          [](const volatile int*) { return true; },
          [&](const volatile int* j) {
            it += j[qN];
            if (!packed || j[qN] * 128 <= j[qLk]) return true;
            if (!warp_wait_data(landed, ph, live)) return false;
            ph ^= 1;
            zero_rows<C::NH>(sm + (2 + (it - 1) % 3) * C::kTile, j[qLk] - (j[qN] - 1) * 128, lane);
            if (lane == 0) mbar_arrive(fixed);
            __syncwarp();
            return true;
          });
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- dS
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegCompute));
    const int g = warp >> 2, row = threadIdx.x & 127, w0 = 32 * (warp & 3);
    const uint32_t lanes = (uint32_t)w0 << 16;
    const uint32_t td = tmem + lanes + kDP + 32 * g;
    const F2 cc = f2(a.c, a.c);
    Ring<2> rs;
    uint32_t oph = 0, dph = 0, aph = 0, pph = 0;
    bool ok = true;
    // the sum over the four threads of a row (once per job)
    auto row_sum = [&](float x) {
      part[g * 128 + row] = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(part_full);
      ok = warp_wait_data(part_full, pph, live);
      pph ^= 1;
      return part[row] + part[128 + row] + part[256 + row] + part[384 + row];
    };
    float lse;
    uint4 ov[DP / 32];
    // a job's lse and its part of o: asked for before the last job's sums are written
    auto fetch = [&](const int* j) {
      const bool in = j && row < j[qNr];
      lse = in ? a.lse[((long long)j[kB] * a.H + j[kHead]) * a.sq.Tq + j[qQ0] + row] : 0.f;
#pragma unroll
      for (int x = 0; x < DP / 32; ++x) {
        const int c = g * (DP / 4) + 8 * x;
        ov[x] = make_uint4(0, 0, 0, 0);
        if (in && j[qN] > 1 && c < a.D) {
          const long long tok = (long long)j[kB] * a.sq.Tq + j[qQ0] + row;
          ov[x] = *reinterpret_cast<const uint4*>(a.o + (tok * a.H + j[kHead]) * a.D + c);
        }
      }
    };
    const int* j = next_job(slots, take, true, live);
    fetch(j);
    while (j) {
      const int N = j[qN], nr = j[qNr];
      const long long tok = (long long)j[kB] * a.sq.Tq + j[qQ0] + row;
      float delta = 0.f;
      lse *= kLog2e;
      if (N) {
        // (for N = 1, dO may be the next job's by now, and do_full a phase further)
        if (N > 1 && !(ok = warp_wait_data(do_full, oph, live))) break;
        oph ^= 1;
        if (N > 1) {  // delta = do . o: a thread takes DP / 4 values of its row
#pragma unroll
          for (int x = 0; x < DP / 32; ++x) {
            const int c = g * (DP / 4) + 8 * x;
            const uint4 dv =
                *reinterpret_cast<const uint4*>(sm + C::kTile + (c >> 6) * 16384 + sw_row_off(row, (c & 63) >> 3));
            const uint32_t o4[4] = {ov[x].x, ov[x].y, ov[x].z, ov[x].w}, d4[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              delta = fmaf(__uint_as_float(o4[y] << 16), __uint_as_float(d4[y] << 16), delta);
              delta = fmaf(__uint_as_float(o4[y] & 0xffff0000u), __uint_as_float(d4[y] & 0xffff0000u), delta);
            }
          }
          delta = row_sum(delta);
          if (!ok) break;
        }
      }
      const F2 ls = f2(-lse, -lse);
      const int first = min(j[qFirst], j[qLk] - 1), last = min(j[qFirst] + row, j[qLk] - 1);
#pragma unroll 1
      for (int x = 0; x < N; ++x) {
        const int buf = rs.i;
        const uint32_t ts = tmem + lanes + kS + 128 * buf + 32 * g;
        if (!(ok = warp_wait_live(s_full + buf, rs.ph, live))) break;
        rs.next();
        tc_fence_after();
        float p[32], d[32];
        tmem_ld32_start(ts, p);
        tmem_ld_wait();
        tmem_landed(p);
#pragma unroll
        for (int y = 0; y < 32; y += 2) {
          const float2 e = unpack(fma2(f2(p[y], p[y + 1]), cc, ls));
          p[y] = ex2(e.x), p[y + 1] = ex2(e.y);
        }
        if (!(ok = warp_wait_live(dp_full, dph, live))) break;
        dph ^= 1;
        tc_fence_after();
        tmem_ld32_start(td, d);
        tmem_ld_wait();
        tmem_landed(d);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dp_read);
        if (x * 128 + 127 > first) {
          const int see = last - x * 128 - 32 * g;
#pragma unroll
          for (int y = 0; y < 32; ++y) p[y] = y <= see ? p[y] : 0.f, d[y] = y <= see ? d[y] : 0.f;
        }
        if (N == 1) {
          F2 sum = f2(0.f, 0.f);
#pragma unroll
          for (int y = 0; y < 32; y += 2) sum = fma2(f2(p[y], p[y + 1]), f2(d[y], d[y + 1]), sum);
          const float2 two = unpack(sum);
          delta = row_sum(two.x + two.y);
          if (!ok) break;
        }
        const F2 dl = f2(-delta, -delta);
        uint32_t w[16];
#pragma unroll
        for (int y = 0; y < 32; y += 2) {
          const float2 e = unpack(mul2(f2(p[y], p[y + 1]), add2(f2(d[y], d[y + 1]), dl)));
          w[y / 2] = pack_bf16(e.x, e.y);
        }
        tmem_st16_start(ts, w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full + buf);
      }
      if (!ok) break;
      if (g == 0 && row < nr) a.delta[((long long)j[kB] * a.H + j[kHead]) * a.sq.Tq + j[qQ0] + row] = delta;
      constexpr int kPart = DP / 4 < 32 ? 32 : DP / 4;  // columns a group writes
      const long long stride = (long long)a.H * a.D;
      __nv_bfloat16* dst = a.dq + ((tok - row + w0) * a.H + j[kHead]) * a.D;
      job_done(slots, take, true);
      j = next_job(slots, take, true, live);
      fetch(j);
      if (N) {
        if (!(ok = warp_wait_live(acc_full, aph, live))) break;
        aph ^= 1;
        tc_fence_after();
        if (g * kPart < DP)
          store_acc<kPart>(tmem + lanes + kDQ + g * kPart, a.scale, dst, stride, nr - w0, g * kPart, a.D);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty);
      } else if (g == 0) {
        store_zeros(dst, stride, nr - w0, a.D);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && live->dead) report_timeout();
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
  a.group = batch_group(p.B, 4.0 * p.Tk * p.Hkv * p.D, (long)a.tiles * p.H);  // K and V
  prof_before(s);
  attn_tc_bwd_q_kernel<DP>
      <<<(unsigned)(AttnSeqs::slots(p, 128, false) * p.H), kThreads, C::kSmem, s>>>(mq, mk, mv, md, a);
  e = cudaGetLastError();
  prof_after(s, kAttnBwdQ);
  if (e != cudaSuccess) return e;
  a.tiles = p.cu_q ? 0 : (p.Tk + 127) / 128;
  a.group = batch_group(p.B, 4.0 * p.Tq * p.H * p.D, (long)a.tiles * p.Hkv);  // Q and dO
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
