// Causal attention on the tensor cores, forward: bf16, D a multiple of 8 up to
// 128 (padded with zeros to 64 or 128).
//
// One CTA takes 256 query rows of one head as two tiles of 128 and walks the
// keys they see in tiles of 128.  Per tile t and key tile j:
//   S = Q K^T                      (128 x 128, fp32 in TMEM)
//   P = exp2(c S - c m), c = scale log2 e: bf16, written over S in TMEM
//   O += P V                       (P is the MMA's A operand in TMEM)
// with a running row maximum m and row sum l in the registers of the thread
// that owns the row (128 threads per tile, one row each, so neither needs
// another thread).  The maximum that scales P may lag behind: it is only
// raised, and O and l rescaled, when the row's maximum has grown by more than
// 8 in the exponent; P is then at most 2^8, which costs no bits, and the
// rescaling passes over O in TMEM nearly vanish.
//
// Warps 0-3 and 4-7 are the two tiles' softmax, warp 8 issues the TMA loads (a
// ring of K and V tiles), warp 9 the MMAs, warp 10 zeroes the rows of a packed
// sequence's last V tile that belong to the next one.  The two tiles take
// turns: while one is in its softmax the tensor cores run the other's
// products, in the order P V (j), Q K^T (j + 1) per tile.  That Q K^T
// overwrites P, which is safe behind the P V issued before it; its completion
// also says that O is up to date.

#include <math.h>

#include "attn_tc.cuh"

namespace gdn {

cudaError_t attn_tc_fwd_read_and_clear_status(int* status) {
  return tc::read_and_clear_file_status(status);
}

namespace {

using namespace tc;

constexpr int kThreads = 384;
// 168 registers a thread at launch; the softmax warps take 208, the others 88:
// 256 * 208 + 128 * 88 = 384 * 168.
constexpr int kRegSoftmax = 208, kRegOther = 88;
constexpr float kLag = 8.f;  // exponent by which the row maximum may lag

template <int DP>
struct Cfg {
  static constexpr int NH = DP / 64;
  static constexpr int kTile = 128 * DP * 2;
  static constexpr int kStages = DP == 128 ? 5 : 8;
  static constexpr int kBar = (2 + kStages) * kTile;
  static constexpr int kSmem = kBar + 512 + 1024;
  static constexpr uint32_t kS = 0, kO = 256;  // TMEM columns: S of tile t at 128 t, O at 256 + DP t
};

struct Args {
  AttnSeqs sq;
  int H, Hkv, D, tiles;  // tiles: 256-row tiles per batch row (0: packed)
  float c, scale;
  __nv_bfloat16* o;
  float* lse;
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, Args a) {
  using C = Cfg<DP>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + C::kBar);  // [2]
  uint64_t* s_full = q_full + 2;                                 // [2]
  uint64_t* p_full = s_full + 2;                                 // [2]
  uint64_t* o_full = p_full + 2;                                 // [2]
  uint64_t* v_landed = o_full + 2;  // the last V tile is there; its foreign rows are zero
  uint64_t* v_fixed = v_landed + 1;
  uint64_t* drain = v_fixed + 1;
  uint64_t* kv_full = drain + 1;                                 // [kStages]
  uint64_t* kv_empty = kv_full + C::kStages;                     // [kStages]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_empty + C::kStages);
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (blockIdx.x == 0 && !a.sq.valid() && threadIdx.x == 0) atomicExch(&g_file_status, GDN_ERR_SEQLENS);
  // the tiles with the most keys first
  const int h = blockIdx.x % a.H, u = blockIdx.x / a.H;
  const int slot = a.tiles ? u % a.sq.B * a.tiles + a.tiles - 1 - u / a.sq.B : gridDim.x / a.H - 1 - u;
  AttnTile t;
  if (!a.sq.get<false>(slot, 256, t)) return;
  const int r0 = t.tile * 256, shift = t.lk - t.lq, hk = h / (a.H / a.Hkv);
  int nr[2], n[2];  // rows of each tile, key tiles they see
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    nr[i] = max(0, min(128, t.lq - r0 - 128 * i));
    n[i] = nr[i] ? (max(0, min(t.lk, r0 + 128 * i + nr[i] + shift)) + 127) / 128 : 0;
  }
  const int nmax = max(n[0], n[1]);
  // the last V tile holds rows of the next packed sequence
  const bool fix = a.sq.cu_q && nmax * 128 > t.lk;

  if (threadIdx.x == 256) {
    *dead = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_full + i, 1);
    }
    mbar_init(v_landed, 1);
    mbar_init(v_fixed, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(kv_full + i, 1);
      mbar_init(kv_empty + i, 1);
    }
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  cta_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
    if (warp == 8 && elect_one()) {
      // ------------------------------------------------------------ loads
      for (int i = 0; i < 2; ++i)
        if (n[i]) {
          mbar_arrive_expect_tx(q_full + i, C::kTile);
          load_tile<C::NH>(sm + i * C::kTile, &tm_q, q_full + i, h, t.q0 + r0 + 128 * i, t.b);
        }
      int it = 0;  // ring use: K 0, V 0, K 1, V 1, ...
      for (; it < 2 * nmax; ++it) {
        const int st = it % C::kStages, use = it / C::kStages;
        if (use && !wait_live(kv_empty + st, (use - 1) & 1, dead)) break;
        mbar_arrive_expect_tx(kv_full + st, C::kTile);
        load_tile<C::NH>(sm + (2 + st) * C::kTile, it & 1 ? &tm_v : &tm_k, kv_full + st, hk,
                         t.k0 + it / 2 * 128, t.b);
      }
      if (*dead) {  // nothing may still be written at exit (bounded)
        for (int i = 0; i < 2; ++i)
          if (n[i]) mbar_wait(q_full + i, 0, 10000);
        for (int x = max(0, it - C::kStages); x < it; ++x)
          mbar_wait(kv_full + x % C::kStages, (x / C::kStages) & 1, 10000);
      }
    } else if (warp == 9 && elect_one()) {
      // ------------------------------------------------------------ MMAs
      const uint64_t dq = sw128_desc(smem_u32(sm), 16, 1024);     // K-major
      const uint64_t dv = sw128_desc(smem_u32(sm), 16384, 1024);  // MN-major, 64-column blocks 16 KB apart
      constexpr uint32_t id_s = idesc_bf16(128, 128, false, false), id_o = idesc_bf16(128, DP, false, true);
      auto full = [&](int it) { return wait_live(kv_full + it % C::kStages, (it / C::kStages) & 1, dead); };
      auto tile = [&](int it) { return (uint32_t)(2 + it % C::kStages) * C::kTile; };
      auto qk = [&](int i, int j) {
        const uint32_t kt = tile(2 * j);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t off = (k / 4) * 16384 + (k % 4) * 32;
          mma_bf16(tmem + C::kS + 128 * i, desc_at(dq, i * C::kTile + off), desc_at(dq, kt + off), id_s, k > 0);
        }
        mma_commit(s_full + i);
      };
      bool ok = true;
      if (nmax) {
        ok = full(0);
        for (int i = 0; i < 2 && ok; ++i)
          if (n[i]) {
            ok = wait_live(q_full + i, 0, dead);
            if (ok) qk(i, 0);
          }
        mma_commit(kv_empty + 0);
      }
      for (int j = 0; j < nmax && ok; ++j) {
        ok = full(2 * j + 1) && (j + 1 == nmax || full(2 * j + 2));
        if (ok && fix && j + 1 == nmax) {
          mbar_arrive(v_landed);
          ok = wait_live(v_fixed, 0, dead);
        }
        const uint32_t vt = tile(2 * j + 1);
        for (int i = 0; i < 2 && ok; ++i) {
          if (j >= n[i]) continue;
          ok = wait_live(p_full + i, j & 1, dead);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ts(tmem + C::kO + DP * i, tmem + C::kS + 128 * i + 8 * k, desc_at(dv, vt + k * 2048), id_o,
                        j > 0 || k > 0);
          if (j + 1 < n[i]) qk(i, j + 1);
          else mma_commit(o_full + i);
        }
        mma_commit(kv_empty + (2 * j + 1) % C::kStages);
        if (j + 1 < nmax) mma_commit(kv_empty + (2 * j + 2) % C::kStages);
      }
      if (*dead) {
        mma_commit(drain);
        mbar_wait(drain, 0, 10000);
      }
    } else if (warp == 10 && fix) {
      const int it = 2 * nmax - 1;
      bool ok = true;
      if (lane == 0) ok = wait_live(v_landed, 0, dead);
      if (__shfl_sync(0xffffffffu, ok, 0)) {
        zero_rows<C::NH>(sm + (2 + it % C::kStages) * C::kTile, t.lk - (nmax - 1) * 128, lane);
        if (lane == 0) mbar_arrive(v_fixed);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoftmax));
    const int i = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + C::kS + 128 * i, to = tmem + lanes + C::kO + DP * i;
    const int first = r0 + 128 * i + shift;         // last key of the tile's first row
    const int last = min(first + row, t.lk - 1);    // and of this row
    const float c = a.c;
    float m = -INFINITY;
    F2 l0 = f2(0.f, 0.f), l1 = l0;
    bool ok = true;
    for (int j = 0; j < n[i]; ++j) {
      ok = warp_wait_live(s_full + i, j & 1, dead);
      if (!ok) break;
      tc_fence_after();
      float s[128];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32_start(ts + 32 * q, s + 32 * q);
      tmem_ld_wait();
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_landed(s + 32 * q);
      if (j * 128 + 127 > min(first, t.lk - 1)) {
        const int see = last - j * 128;
#pragma unroll
        for (int x = 0; x < 128; ++x) s[x] = x <= see ? s[x] : -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int x = 4; x < 128; ++x) mx[x & 3] = fmaxf(mx[x & 3], s[x]);
      const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
      float f = 1.f;
      if ((top - m) * c > kLag) {  // also the row's first keys (m = -inf)
        f = ex2((m - top) * c);
        m = top;
      }
      if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
        const F2 ff = f2(f, f);
        l0 = mul2(l0, ff), l1 = mul2(l1, ff);
#pragma unroll
        for (int q = 0; q < DP / 32; ++q) {
          float x[32];
          tmem_ld32(to + 32 * q, x);
#pragma unroll
          for (int y = 0; y < 32; ++y) x[y] *= f;
          tmem_st32(to + 32 * q, x);
        }
      }
      const float base = m == -INFINITY ? 0.f : m * c;  // no key so far: every term is 0
      const F2 cc = f2(c, c), mm = f2(-base, -base);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t p[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float2 e = unpack(fma2(f2(s[64 * q + 2 * x], s[64 * q + 2 * x + 1]), cc, mm));
          const float e0 = ex2(e.x), e1 = ex2(e.y);
          if (x & 1) l1 = add2(l1, f2(e0, e1));
          else l0 = add2(l0, f2(e0, e1));
          p[x] = pack_bf16(e0, e1);
        }
        tmem_st32_start(ts + 32 * q, p);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + i);
    }
    if (ok && n[i]) {
      ok = warp_wait_live(o_full + i, 0, dead);
      tc_fence_after();
    }
    if (ok && nr[i]) {
      const float2 la = unpack(add2(l0, l1));
      const float l = la.x + la.y, inv = l == 0.f ? 0.f : 1.f / l;
      const int r = r0 + 128 * i + row;
      __nv_bfloat16* o = a.o + (((long long)t.b * a.sq.Tq + t.q0 + r) * a.H + h) * a.D;
#pragma unroll
      for (int q = 0; q < DP / 32; ++q) {
        float x[32];
        if (n[i]) {
          tmem_ld32(to + 32 * q, x);
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) x[y] = 0.f;
        }
#pragma unroll
        for (int y = 0; y < 32; y += 8) {
          uint4 w;
          w.x = pack_bf16(x[y] * inv, x[y + 1] * inv), w.y = pack_bf16(x[y + 2] * inv, x[y + 3] * inv);
          w.z = pack_bf16(x[y + 4] * inv, x[y + 5] * inv), w.w = pack_bf16(x[y + 6] * inv, x[y + 7] * inv);
          if (row < nr[i] && 32 * q + y < a.D) *reinterpret_cast<uint4*>(o + 32 * q + y) = w;
        }
      }
      if (row < nr[i])
        a.lse[((long long)t.b * a.H + h) * a.sq.Tq + t.q0 + r] = l == 0.f ? -INFINITY : m * a.scale + kLn2 * log2f(l);
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *dead) report_timeout();
  if (warp == 9) tmem_dealloc(tmem, 512);
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
  a.H = p.H, a.Hkv = p.Hkv, a.D = p.D;
  a.tiles = p.cu_q ? 0 : (p.Tq + 255) / 256;
  a.scale = p.scale, a.c = p.scale * kLog2e;
  a.o = static_cast<__nv_bfloat16*>(p.o), a.lse = p.lse;
  prof_before(s);
  attn_tc_fwd_kernel<DP><<<(unsigned)(AttnSeqs::slots(p, 256, false) * p.H), kThreads, C::kSmem, s>>>(mq, mk, mv, a);
  e = cudaGetLastError();
  prof_after(s, kAttnFwd);
  return e;
}

}  // namespace

bool attn_tc_supported(const AttnProblem& p) {
  return p.bf16 && p.Tq > 0 && p.Tk > 0 && attn_map_ok(p.q, p.B, p.Tq, p.H, p.D, p.qs) &&
         attn_map_ok(p.k, p.B, p.Tk, p.Hkv, p.D, p.ks) && attn_map_ok(p.v, p.B, p.Tk, p.Hkv, p.D, p.vs);
}

cudaError_t attn_tc_fwd(const AttnProblem& p, cudaStream_t s) {
  return p.D <= 64 ? run<64>(p, s) : run<128>(p, s);
}

}  // namespace gdn
