// Causal attention on the tensor cores, forward: bf16, D a multiple of 8 up to
// 128 (padded with zeros to 64 or 128).
//
// One CTA takes 256 query rows of one head as two tiles of 128 and walks the
// keys they see in tiles of 128.  Per tile t and key tile j:
//   S = Q K^T                      (128 x 128, fp32 in TMEM)
//   P = exp2(c S - c m), c = scale log2 e: bf16, written over S in TMEM
//   O += P V                       (P is the MMA's A operand in TMEM)
// with a running row maximum m and row sum l in the registers of the four
// threads that share a row.  A warp has 16 rows (TMEM shape 16x256b), so that
// eight warps work on a tile and none needs another for a row.  The maximum that scales P may lag behind: it is only
// raised, and O and l rescaled, when the row's maximum has grown by more than
// 8 in the exponent; P is then at most 2^8, which costs no bits, and the
// rescaling passes over O in TMEM nearly vanish.
//
// Where there are fewer such jobs than SMs, each is split along its keys into
// parts that write o (fp32) and lse to the workspace; a second kernel joins them:
// o = sum_p exp(lse_p - lse) o_p, lse = log sum_p exp(lse_p).
//
// Warps 0-7 and 8-15 are the two tiles' softmax, warp 16 issues the TMA loads (a
// ring of K and V tiles), warp 17 the MMAs, warp 18 gets the next tiles and zeroes
// the rows of a packed sequence's last V tile that belong to the next one.  CTAs
// are persistent (see TileSlots).  The two tiles take turns: while one is in its softmax the tensor cores run the other's
// products, in the order P V (j), Q K^T (j + 1) per tile.  That Q K^T
// overwrites P, which is safe behind the P V issued before it; its completion
// also says that O is up to date.  What bounds the kernel is that turn: a
// softmax (load, maximum, 64 exponentials a thread, store) has to fit into the
// other tile's products.  Code that runs once per job is kept rolled: its
// instructions come from beyond the instruction cache, at some 2 cycles a byte.
// Measured, D 128: one row of 16384 tokens, 16 heads on 2: 750 us, 1466 TFLOP/s of
// the pairs seen; 16 rows of 2048 tokens, 8 heads: 138 us, 996 TFLOP/s, the tensor
// pipe active 47 % of the time (tiles on the diagonal and the turn of the jobs).

#include <math.h>

#include <algorithm>

#include "attn_tc.cuh"

namespace gdn {

cudaError_t attn_tc_fwd_read_and_clear_status(int* status) {
  return tc::read_and_clear_file_status(status);
}

namespace {

using namespace tc;

constexpr int kSoftmax = 512, kThreads = kSoftmax + 128;
// 96 registers a thread at launch: 512 * 104 + 128 * 64 = 640 * 96
constexpr int kRegSoftmax = 104, kRegOther = 64;
constexpr int kMaxParts = 32;  // of a job's keys: a lane each when they are joined
constexpr float kLag = 8.f;  // exponent by which the row maximum may lag

template <int DP>
struct Cfg {
  static constexpr int NH = DP / 64;
  static constexpr int kTile = 128 * DP * 2;
  static constexpr int kStages = DP == 128 ? 5 : 8;
  static constexpr int kBar = (2 + kStages) * kTile;
  static constexpr int kSmem = kBar + 640;  // at most 227 KB: no slack for an alignment
  static constexpr uint32_t kS = 0, kO = 256;  // TMEM columns: S of tile t at 128 t, O at 256 + DP t
};

struct Args {
  AttnSeqs sq;
  int H, G, D, tiles;  // tiles: 256-row tiles per batch row (0: packed)
  int group;           // see batch_group
  int parts;           // of a job's keys
  float c, scale;
  __nv_bfloat16* o;
  float* lse;          // parts > 1: [parts][B, H, Tq] in the workspace
  float* po;           // parts > 1: [parts][B, Tq, H, D]
};

// A job (256 query rows of one head) as the scheduler hands it out.
enum { kHead, kPart, kQ0, kK0, kLk, kFirst, kNr, kB, kN0, kN1, kFix, kValid };
// kQ0, kK0: first query and key token; kLk: keys; kFirst: the last key that the
// first row sees (both counted from kK0); kNr: rows; kN: key tiles that each
// 128-row tile sees; kFix: the last one holds rows of the next packed sequence.

__device__ __forceinline__ bool decode(const Args& a, int cta, int ctas, int (&j)[12]) {
  // the tiles with the most keys first (packed: of a sequence, the last sequence first)
  const int part = cta % a.parts, u = cta / a.parts / a.H;
  const int slot = a.tiles ? batch_slot(u, a.sq.B, a.tiles, a.group, true) : ctas / a.parts / a.H - 1 - u;
  AttnTile t;
  j[kValid] = a.sq.get<false>(slot, 256, t);
  if (!j[kValid]) return false;
  const int r0 = t.tile * 256, shift = t.lk - t.lq;
  j[kHead] = cta / a.parts % a.H, j[kPart] = part, j[kB] = t.b, j[kQ0] = t.q0 + r0, j[kNr] = min(256, t.lq - r0);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int nr = min(128, j[kNr] - 128 * i);
    j[kN0 + i] = nr > 0 ? (max(0, min(t.lk, r0 + 128 * i + nr + shift)) + 127) / 128 : 0;
  }
  // this part's key tiles: [x0, x1) of those that the job sees
  const int n = max(j[kN0], j[kN1]), x0 = n * part / a.parts, x1 = n * (part + 1) / a.parts;
#pragma unroll
  for (int i = 0; i < 2; ++i) j[kN0 + i] = max(0, min(j[kN0 + i], x1) - x0);
  j[kK0] = t.k0 + x0 * 128, j[kLk] = t.lk - x0 * 128, j[kFirst] = r0 + shift - x0 * 128;
  j[kFix] = a.sq.cu_q && max(j[kN0], j[kN1]) * 128 > j[kLk];
  return true;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, Args a) {
  using C = Cfg<DP>;
  extern __shared__ __align__(1024) unsigned char sm[];
  TileSlots* slots = reinterpret_cast<TileSlots*>(sm + C::kBar);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(slots + 1);  // [2]
  uint64_t* q_empty = q_full + 2;                             // [2]
  uint64_t* s_full = q_empty + 2;                             // [2]
  uint64_t* p_full = s_full + 2;                              // [2][2]: per half of the keys
  uint64_t* o_full = p_full + 4;                              // [2]
  uint64_t* o_empty = o_full + 2;                             // [2]
  uint64_t* v_landed = o_empty + 2;  // a job's last V tile is there; its foreign rows are zero
  uint64_t* v_fixed = v_landed + 1;
  uint64_t* drain = v_fixed + 1;
  uint64_t* kv_full = drain + 1;              // [kStages]
  uint64_t* kv_empty = kv_full + C::kStages;  // [kStages]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_empty + C::kStages);
  volatile Liveness* live = reinterpret_cast<volatile Liveness*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (!aligned_smem(sm)) return;
  if (blockIdx.x == 0 && !a.sq.valid() && threadIdx.x == 0) atomicExch(&g_file_status, GDN_ERR_SEQLENS);
  if (threadIdx.x == kSoftmax) {
    live->dead = live->progress[0] = live->progress[1] = 0;
    slots->init(18);
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + 2 * i, 8);
      mbar_init(p_full + 2 * i + 1, 8);
      mbar_init(o_full + i, 1);
      mbar_init(o_empty + i, 8);
    }
    mbar_init(v_landed, 1);
    mbar_init(v_fixed, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(kv_full + i, 1);
      mbar_init(kv_empty + i, 1);
    }
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 17) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  cta_sync();
  const uint32_t tmem = *tmem_slot;

  Ring<2> take;
  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
    if (warp == 16 && elect_one()) {
      // ------------------------------------------------------------ loads
      Ring<C::kStages> kv;
      uint32_t qph[2] = {0, 0};
      bool ok = true;
      while (const int* j = ok ? next_job(slots, take, false, live) : nullptr) {
        const int h = j[kHead], hk = h / a.G, b = j[kB], q0 = j[kQ0], k0 = j[kK0], n[2] = {j[kN0], j[kN1]};
        const int nmax = max(n[0], n[1]);
        job_done(slots, take, false);
        auto load_q = [&](int i) {
          if (!n[i]) return;
          ok = ok && wait_live(q_empty + i, qph[i] ^ 1, live);
          if (!ok) return;
          qph[i] ^= 1;
          mbar_arrive_expect_tx(q_full + i, C::kTile);
          load_tile<C::NH>(sm + i * C::kTile, &tm_q, q_full + i, h, q0 + 128 * i, b);
        };
        auto load_kv = [&](const CUtensorMap* tm, int x) {
          ok = ok && wait_live(kv_empty + kv.i, kv.ph ^ 1, live);
          if (!ok) return;
          mbar_arrive_expect_tx(kv_full + kv.i, C::kTile);
          load_tile<C::NH>(sm + (2 + kv.i) * C::kTile, tm, kv_full + kv.i, hk, k0 + x * 128, b);
          kv.next();
        };
        load_q(0);
        if (nmax) load_kv(&tm_k, 0);
        load_q(1);
        for (int x = 0; x < nmax && ok; ++x) {  // K 0, V 0, K 1, V 1, ...
          if (x) load_kv(&tm_k, x);
          load_kv(&tm_v, x);
        }
      }
      if (live->dead) {
        for (int i = 0; i < 2; ++i) mbar_wait(q_full + i, qph[i] ^ 1, 10000);
        drain_loads(kv_full, kv);
      }
    } else if (warp == 17 && elect_one()) {
      // ------------------------------------------------------------ MMAs
      const uint64_t dq = sw128_desc(smem_u32(sm), 16, 1024);     // K-major
      const uint64_t dv = sw128_desc(smem_u32(sm), 16384, 1024);  // MN-major, 64-column blocks 16 KB apart
      Ring<C::kStages> kv;  // the next tile to wait for
      uint32_t qph0 = 0, qph1 = 0, pph0 = 0, pph1 = 0, oph0 = 0, oph1 = 0, fph = 0;
      int turns = 0;
      bool ok = true;
      auto qk = [&](int i, int stage) {
        mma_rows<DP>(tmem + C::kS + 128 * i, desc_at(dq, i * C::kTile), desc_at(dq, (2 + stage) * C::kTile));
        mma_commit(s_full + i);
      };
      // P V of key tile x from stage vs, then Q K^T of tile x + 1 from stage ks
      auto turn = [&](int i, int x, int n, int vs, int ks, uint32_t& pph, uint32_t& oph) {
        if (x >= n) return true;
        if (x == 0) {  // the job before has read O
          if (!wait_live(o_empty + i, oph ^ 1, live)) return false;
          oph ^= 1;
        }
        // the first 64 keys' products run while the others' exponentials are made
        const uint32_t o = tmem + C::kO + DP * i, p = tmem + C::kS + 128 * i;
        const uint64_t v = desc_at(dv, (2 + vs) * C::kTile);
        if (!wait_live(p_full + 2 * i, pph, live)) return false;
        tc_fence_after();
        mma_sum<DP, 4>(o, p, v, x > 0);
        if (!wait_live(p_full + 2 * i + 1, pph, live)) return false;
        pph ^= 1;
        tc_fence_after();
        mma_sum<DP, 4>(o, p + 32, desc_at(v, 8192), true);
        if (x + 1 < n) {
          qk(i, ks);
          if (x + 2 == n) mma_commit(q_empty + i);
        } else {
          mma_commit(o_full + i);
        }
        return true;
      };
      while (const int* j = ok ? next_job(slots, take, false, live) : nullptr) {
        const int n0 = j[kN0], n1 = j[kN1], nmax = max(n0, n1);
        const bool fix = j[kFix];
        job_done(slots, take, false);
        if (!nmax) {
          mbar_arrive(&slots->soon);
          continue;
        }
        if (!(ok = wait_live(kv_full + kv.i, kv.ph, live))) break;
        if (n0) {
          if (!(ok = wait_live(q_full, qph0, live))) break;
          qph0 ^= 1;
          qk(0, kv.i);
          if (n0 == 1) mma_commit(q_empty);
        }
        if (n1) {
          if (!(ok = wait_live(q_full + 1, qph1, live))) break;
          qph1 ^= 1;
          qk(1, kv.i);
          if (n1 == 1) mma_commit(q_empty + 1);
        }
        mma_commit(kv_empty + kv.i);
        kv.next();
        int vs = kv.i, ks = 0;  // V of key tile x, K of x + 1
        if (!(ok = wait_live(kv_full + vs, kv.ph, live))) break;
        kv.next();
        if (nmax > 1) {
          ks = kv.i;
          if (!(ok = wait_live(kv_full + ks, kv.ph, live))) break;
          kv.next();
        }
#pragma unroll 1
        for (int x = 0; x < nmax; ++x) {
          live->progress[0] = ++turns;
          if (x == max(0, nmax - 2)) mbar_arrive(&slots->soon);
          if (fix && x + 1 == nmax) {
            mbar_arrive(v_landed);
            if (!(ok = wait_live(v_fixed, fph, live))) break;
            fph ^= 1;
          }
          if (!(ok = turn(0, x, n0, vs, ks, pph0, oph0))) break;
          // the other tile is still in its softmax: time to wait for the next loads
          int vn = 0, kn = 0;
          if (x + 1 < nmax) {
            vn = kv.i;
            if (!(ok = wait_live(kv_full + vn, kv.ph, live))) break;
            kv.next();
          }
          if (x + 2 < nmax) {
            kn = kv.i;
            if (!(ok = wait_live(kv_full + kn, kv.ph, live))) break;
            kv.next();
          }
          if (!(ok = turn(1, x, n1, vs, ks, pph1, oph1))) break;
          mma_commit(kv_empty + vs);
          if (x + 1 < nmax) mma_commit(kv_empty + ks);
          vs = vn, ks = kn;
        }
      }
      if (live->dead) {
        mma_commit(drain);
        mbar_wait(drain, 0, 10000);
      }
    } else if (warp == 18) {
      // ------------------------------------------------------------ the next tiles; foreign rows
      int it = 0;  // K and V tiles so far
      uint32_t ph = 0;
      const int ctas = gridDim.x;
      schedule(
          slots, live, [&](int cta, int(&j)[12]) { return decode(a, cta, ctas, j); },
          [](const volatile int*) { return true; },
          [&](const volatile int* j) {
            const int n = max(j[kN0], j[kN1]);
            it += 2 * n;
            if (!j[kFix]) return true;
            if (!warp_wait_data(v_landed, ph, live)) return false;
            ph ^= 1;
            zero_rows<C::NH>(sm + (2 + (it - 1) % C::kStages) * C::kTile, j[kLk] - (n - 1) * 128, lane);
            if (lane == 0) mbar_arrive(v_fixed);
            __syncwarp();
            return true;
          });
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoftmax));
    // this thread: rows w0 + lane / 4 + {0, 8} of tile i, columns 8 g + 2 (lane % 4) + {0, 1}
    const int i = warp >> 3, w0 = 32 * (warp & 3) + 4 * (warp & 4), col = 2 * (lane & 3);
    const uint32_t lanes = (uint32_t)w0 << 16, ts = tmem + lanes + C::kS + 128 * i, to = tmem + lanes + C::kO + DP * i;
    const float c = a.c;
    const F2 cc = f2(c, c);
    uint32_t sph = 0, oph = 0;
    bool ok = true;
    while (const int* j = ok ? next_job(slots, take, true, live) : nullptr) {
      const int n = j[kN0 + i], lk = j[kLk];
      const int first = min(j[kFirst] + 128 * i + w0, lk - 1);  // last key that the warp's first row sees
      float m[2] = {-INFINITY, -INFINITY};
      F2 l[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll 1
      for (int x = 0; x < n; ++x) {
        if (!(ok = warp_wait_live(s_full + i, sph, live))) break;
        sph ^= 1;
        tc_fence_after();
        float s[64];
        tmem_ld16x64_start(ts, s);
        tmem_ld16x64_start(ts + 64, s + 32);
        tmem_ld_wait();
        tmem_landed(s);
        tmem_landed(s + 32);
        if (x * 128 + 127 > first) {
          const int see = j[kFirst] + 128 * i + w0 + lane / 4 - x * 128 - col, end = lk - 1 - x * 128 - col;
#pragma unroll
          for (int y = 0; y < 64; ++y)
            s[y] = 8 * (y >> 2) + (y & 1) <= min(see + 4 * (y & 2), end) ? s[y] : -INFINITY;
        }
        float f[2], base[2];
        bool raise = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float u = fmaxf(s[2 * r], s[2 * r + 1]), v = fmaxf(s[2 * r + 4], s[2 * r + 5]);
#pragma unroll
          for (int y = 8; y < 64; y += 8) {
            u = max3(u, s[y + 2 * r], s[y + 2 * r + 1]);
            v = max3(v, s[y + 2 * r + 4], s[y + 2 * r + 5]);
          }
          u = fmaxf(u, v);
          u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 1));
          u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 2));
          f[r] = 1.f;
          if ((u - m[r]) * c > kLag) {  // also the row's first keys (m = -inf)
            f[r] = ex2((m[r] - u) * c);
            m[r] = u;
            raise = true;
          }
          base[r] = m[r] == -INFINITY ? 0.f : -m[r] * c;  // no key so far: every term is 0
        }
        if (x > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) l[r] = mul2(l[r], f2(f[r], f[r]));
#pragma unroll 1
          for (int q = 0; q < DP / 32; ++q) {
            float o[16];
            tmem_ld16x32(to + 32 * q, o);
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] *= f[(y >> 1) & 1];
            tmem_st16x32(to + 32 * q, o);
          }
        }
        const F2 mm[2] = {f2(base[0], base[0]), f2(base[1], base[1])};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t p[16];
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const float2 e = unpack(fma2(f2(s[32 * q + 2 * y], s[32 * q + 2 * y + 1]), cc, mm[y & 1]));
            const float e0 = ex2(e.x), e1 = ex2(e.y);
            l[y & 1] = add2(l[y & 1], f2(e0, e1));
            p[y] = pack_bf16(e0, e1);
          }
          tmem_st16x32_start(ts + 32 * q, p);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 2 * i + q);
        }
      }
      if (ok && n) {
        ok = warp_wait_live(o_full + i, oph, live);
        oph ^= 1;
        tc_fence_after();
      }
      if (!ok) break;
      const int h = j[kHead], nr = min(128, j[kNr] - 128 * i) - w0, q0 = j[kQ0] + 128 * i + w0, b = j[kB], part = j[kPart];
      job_done(slots, take, true);
      float inv[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 two = unpack(l[r]);
        float sum = two.x + two.y;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        inv[r] = sum == 0.f ? 0.f : rcp(sum);
        if (col == 0 && lane / 4 + 8 * r < nr)
          a.lse[((long long)(part * a.sq.B + b) * a.H + h) * a.sq.Tq + q0 + lane / 4 + 8 * r] =
              sum == 0.f ? -INFINITY : m[r] * a.scale + kLn2 * lg2(sum);
      }
      const long long at = (((long long)(part * a.sq.B + b) * a.sq.Tq + q0) * a.H + h) * a.D;
#pragma unroll 1
      for (int q = 0; q < DP / 32; ++q) {
        float v[16];
        if (n) {
          tmem_ld16x32(to + 32 * q, v);
        } else {
#pragma unroll
          for (int y = 0; y < 16; ++y) v[y] = 0.f;
        }
        if (q + 1 == DP / 32 && n) {  // O has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_empty + i);
        }
        if (a.parts == 1) {
          store_rows16x32(v, inv, a.o + at, (long long)a.H * a.D, nr, 32 * q, a.D);
        } else {
#pragma unroll
          for (int y = 0; y < 16; y += 2) {
            const int r = lane / 4 + 4 * (y & 2), x = 32 * q + 2 * y - (y & 2) * 2 + col;
            if (r < nr && x < a.D)
              *reinterpret_cast<float2*>(a.po + at + (long long)r * a.H * a.D + x) =
                  make_float2(v[y] * inv[(y >> 1) & 1], v[y + 1] * inv[(y >> 1) & 1]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && live->dead) report_timeout();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// One warp per (token, head): joins the parts.
__global__ void __launch_bounds__(256) attn_join_kernel(Args a, __nv_bfloat16* o, float* lse, long long rows) {
  grid_dep_wait();
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int lane = threadIdx.x & 31, h = (int)(r % a.H), Tq = a.sq.Tq;
  const long long tok = r / a.H, b = tok / Tq, at = (b * a.H + h) * Tq + tok % Tq, all = (long long)a.sq.B * a.H * Tq;
  // lane p < parts holds part p's lse
  const float l = lane < a.parts ? a.lse[lane * all + at] : -INFINITY;
  float m = l;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  // 0 for a part without keys only: a NaN (which fmaxf passes over) stays in the sum
  const float w = l == -INFINITY ? 0.f : ex2((l - (m == -INFINITY ? 0.f : m)) * kLog2e);
  float sum = w;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  if (lane == 0) lse[at] = sum == 0.f ? -INFINITY : m + kLn2 * lg2(sum);
  const float f = sum == 0.f ? 0.f : w * rcp(sum);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < a.parts; ++p) {
    const float g = __shfl_sync(0xffffffffu, f, p);
    if (g == 0.f) continue;  // a part without keys
    const float* x = a.po + (p * all + r) * a.D + 4 * lane;
    if (4 * lane < a.D) {
      const float4 y = *reinterpret_cast<const float4*>(x);
      acc[0] = fmaf(g, y.x, acc[0]), acc[1] = fmaf(g, y.y, acc[1]);
      acc[2] = fmaf(g, y.z, acc[2]), acc[3] = fmaf(g, y.w, acc[3]);
    }
  }
  if (4 * lane < a.D)
    *reinterpret_cast<uint2*>(o + r * a.D + 4 * lane) = make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
}

// One warp waits for an arrival that comes after eight times its patience, with
// signs of progress all the while, then for one that never comes; the other warp
// gives the signs.  Nothing else is in flight.
__global__ void __launch_bounds__(64) attn_wait_selftest_kernel(uint32_t patience) {
  __shared__ uint64_t late, never;
  __shared__ Liveness state;
  volatile Liveness* live = &state;
  if (threadIdx.x == 0) {
    mbar_init(&late, 1);
    mbar_init(&never, 1);
    live->dead = live->progress[0] = live->progress[1] = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const bool came = warp_wait_job(&late, 0, live, patience) && !live->dead;
    const bool ran_out = !warp_wait_job(&never, 0, live, patience) && live->dead;
    if (threadIdx.x == 0) atomicExch(&g_file_status, came && ran_out ? GDN_ERR_DEVICE_TIMEOUT : GDN_ERR_ARG);
  } else if (threadIdx.x == 32) {
    for (int i = 1; i <= 32; ++i) {
      const uint32_t since = clock();  // a turn takes a clock at least
      for (uint32_t k = 0; k < patience && (uint32_t)clock() - since < patience / 4; ++k) {
      }
      live->progress[0] = i;
    }
    mbar_arrive(&late);
  }
}

// Parts of a job's keys, from the sizes alone (a packed sequence's own length is
// on the device: the mean stands for it, and a quarter more for the longest).  The estimate in microseconds: 1.9 per
// key tile of the longest job, or of the average one times the rounds of jobs
// over the SMs; 5 for the join's launch, and the parts' o written and read.
// Measured (one row, D 128; one part -> best number of parts): 2048 tokens and 16
// heads, 128 jobs, 43 us -> 48 with two, not split; 4096 and 8 heads 69 -> 59;
// 4096 and 4 heads 68 -> 44; 512 queries, 65536 keys, 8 heads 852 -> 121.
int parts_of(const AttnProblem& p) {
  const int nseq = p.cu_q ? std::max(1, p.nseq) : p.B, sms = sm_count();
  const float tq = (float)p.Tq * p.B / nseq, tk = (float)p.Tk * p.B / nseq;  // mean lengths
  // a packed sequence's last job is half empty on average
  const float jobs = (p.cu_q ? tq / 256.f + .5f : (float)((p.Tq + 255) / 256)) * nseq * p.H;
  if (jobs >= sms) return 1;
  const float longest = tk / (p.cu_q ? 102.f : 128.f), mean = std::max(tk - std::min(tk, tq) / 2, 0.f) / 128.f;
  int best = 1;
  float least = INFINITY;
  for (int n = 1; n <= kMaxParts; ++n) {
    const float rounds = ceilf(n * jobs / sms);
    const float t = 1.9f * std::max(longest, mean * rounds) / n + (n > 1 ? 5.f + 4e-4f * p.D * n * jobs : 0.f);
    if (t < least) best = n, least = t;
  }
  return best;
}

size_t part_lse_bytes(const AttnProblem& p, int parts) {
  return align_up((size_t)parts * p.B * p.H * p.Tq * sizeof(float), 256);
}

template <int DP>
cudaError_t run(const AttnProblem& p, cudaStream_t s) {
  using C = Cfg<DP>;
  CUtensorMap mq, mk, mv;
  cudaError_t e = make_attn_map(&mq, p.q, p.B, p.Tq, p.H, p.D, p.qs);
  if (e == cudaSuccess) e = make_attn_map(&mk, p.k, p.B, p.Tk, p.Hkv, p.D, p.ks);
  if (e == cudaSuccess) e = make_attn_map(&mv, p.v, p.B, p.Tk, p.Hkv, p.D, p.vs);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_tc_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  Args a;
  a.sq = AttnSeqs::of(p);
  a.H = p.H, a.G = p.H / p.Hkv, a.D = p.D;
  a.tiles = p.cu_q ? 0 : (p.Tq + 255) / 256;
  a.scale = p.scale, a.c = p.scale * kLog2e;
  a.o = static_cast<__nv_bfloat16*>(p.o), a.lse = p.lse;
  a.group = batch_group(p.B, 4.0 * p.Tk * p.Hkv * p.D, (long)a.tiles * p.H);  // K and V
  a.parts = parts_of(p);
  a.po = nullptr;
  if (a.parts > 1) {
    a.lse = static_cast<float*>(p.ws);
    a.po = reinterpret_cast<float*>(static_cast<unsigned char*>(p.ws) + part_lse_bytes(p, a.parts));
  }
  prof_before(s);
  attn_tc_fwd_kernel<DP>
      <<<(unsigned)(AttnSeqs::slots(p, 256, false) * p.H * a.parts), kThreads, C::kSmem, s>>>(mq, mk, mv, a);
  e = cudaGetLastError();
  prof_after(s, kAttnFwd);
  if (e != cudaSuccess || a.parts == 1) return e;
  const long long rows = (long long)p.B * p.Tq * p.H;
  prof_before(s);
  e = launch_overlapped(attn_join_kernel, (unsigned)((rows + 7) / 8), 256, 0, s, a, static_cast<__nv_bfloat16*>(p.o),
                        p.lse, rows);
  prof_after(s, kAttnCombine);
  return e;
}

}  // namespace

cudaError_t attn_wait_selftest(int clocks, cudaStream_t s) {
  attn_wait_selftest_kernel<<<1, 64, 0, s>>>((uint32_t)clocks);
  return cudaGetLastError();
}

bool attn_tc_supported(const AttnProblem& p) {
  return p.bf16 && p.Tq > 0 && p.Tk > 0 && attn_map_ok(p.q, p.B, p.Tq, p.H, p.D, p.qs) &&
         attn_map_ok(p.k, p.B, p.Tk, p.Hkv, p.D, p.ks) && attn_map_ok(p.v, p.B, p.Tk, p.Hkv, p.D, p.vs);
}

size_t attn_tc_fwd_workspace(const AttnProblem& p) {
  const int parts = parts_of(p);
  return parts == 1 ? 0 : part_lse_bytes(p, parts) + (size_t)parts * p.B * p.Tq * p.H * p.D * sizeof(float);
}

cudaError_t attn_tc_fwd(const AttnProblem& p, cudaStream_t s) {
  return p.D <= 64 ? run<64>(p, s) : run<128>(p, s);
}

}  // namespace gdn
