// Pages of keys and values: new tokens in (kv_append, rotating keys and queries
// by position on the way) and rows out again (kv_gather).
//
// Append: token t of row b goes to slot n = lens[b] + t, that is place n % page of
// page table[b][n / page].  A CTA takes a run of tokens and looks up their places
// together (the offsets, the length and the table stand behind one another); its
// warps then take a token each (where there are few, a part of its heads) and walk
// the heads of q (if given), k and v as the norm-and-rotation kernel does
// (rope.cuh).  4-bit rows pass through shared memory to bring 8 neighbouring values
// into a lane (a pair's halves lie R / 2 apart).
// Gather: a CTA takes a run of packed tokens, looks up their pages once, and
// copies (or widens) 16-byte vectors.  Both are bound by memory: each byte is
// read and written once.  Measured, heads of 128: 10541 packed tokens of 4 heads into
// bf16 pages 13 us (the tokens' lookups, then three tokens per warp one after another);
// 60898 tokens of 4 heads out of them 42 us (5.9 TB/s); 23128 out of 4 bits 17 us.

#include "paged.cuh"
#include "rope.cuh"

namespace gdn {

cudaError_t kv_cache_read_and_clear_status(int* status) { return tc::read_and_clear_file_status(status); }

namespace {

using namespace paged;
using namespace rope;
using tc::sm_count;

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Pages {
  int pages, shift, max_pages, nseq;
  long long table_stride;
  const int* table;
  void *k, *v, *k_scale, *v_scale;
  long long ks[3], vs[3], kss[3], vss[3];  // page, token, head
};

Pages pages_of(const PagedCache& c, const PageTable& t) {
  Pages p = {};
  p.pages = c.pages, p.shift = page_shift(c.page), p.max_pages = t.max_pages, p.nseq = t.rows;
  p.table_stride = t.stride, p.table = t.table;
  p.k = c.k, p.v = c.v, p.k_scale = c.k_scale, p.v_scale = c.v_scale;
  for (int i = 0; i < 3; ++i) p.ks[i] = c.ks[i], p.vs[i] = c.vs[i], p.kss[i] = c.kss[i], p.vss[i] = c.vss[i];
  return p;
}

__device__ __forceinline__ void report(int status) { atomicExch(&tc::g_file_status, status); }

// Whether the packed offsets rise from 0 to at most (or, `all`, exactly) total.
// All threads of the CTA call.
__device__ bool rises(const int* cu, int nseq, int total, bool all) {
  int bad = 0;
  if (threadIdx.x == 0) bad = cu[0] != 0 || cu[nseq] > total || (all && cu[nseq] != total);
  for (int s = threadIdx.x; s < nseq; s += blockDim.x) bad |= cu[s + 1] < cu[s];
  return !__syncthreads_or(bad);
}

// The page that holds a row's slot, or -1 (reported).
__device__ __forceinline__ int page_of(const Pages& p, int row, long long slot) {
  const int n = p.table[row * p.table_stride + (slot >> p.shift)];
  if ((unsigned)n < (unsigned)p.pages) return n;
  report(GDN_ERR_PAGE);
  return -1;
}

// ---------------------------------------------------------------- append

constexpr int kTokens = 64;  // most tokens of a CTA
constexpr int kPerSm = 3;    // CTAs that run at once on an SM

struct AppendArgs {
  Pages c;
  int T, H, Hkv, rows, D, R, P, per, parts;  // rows = H + 2 Hkv; per: tokens of a CTA, parts: warps that share one
  uint32_t tokens;
  long long qs[3], ks[3], vs[3];
  const void *q, *k, *v;
  const float *cos, *sin;
  const int *lens, *cu;
  void* qo;
};

// What becomes of a token: its slot's page and place, its position.
struct Place {
  int page, at, n;
  bool turn, keep;  // its queries and keys are rotated (q is zeros otherwise); k and v are stored
};

__device__ __forceinline__ Place place_of(const AppendArgs& a, uint32_t tok) {
  Place p = {0, 0, 0, false, false};
  int row = (int)(tok / a.T), t = (int)(tok % a.T), fresh = a.T;
  if (a.cu) {
    if (a.c.nseq == 0) return p;
    row = sequence_of(a.cu, a.c.nseq, (int)tok);
    t = (int)tok - a.cu[row], fresh = a.cu[row + 1] - a.cu[row];
    if (t < 0 || t >= fresh) return p;  // behind the last sequence
  }
  const int used = a.lens[row];
  if (used < 0) return p;  // a row that is not in use
  const long long n = (long long)used + t;
  if ((long long)used + fresh > ((long long)a.c.max_pages << a.c.shift) || (a.R && n >= a.P)) {
    report(GDN_ERR_SEQLENS);
    return p;
  }
  p.n = (int)n, p.at = (int)n & ((1 << a.c.shift) - 1);
  p.turn = true;
  p.page = page_of(a.c, row, n);
  p.keep = p.page >= 0;
  return p;
}

template <typename T, int V, int NP, int LR, bool IL, bool I4>
__global__ void __launch_bounds__(kThreads, kPerSm) kv_append_kernel(AppendArgs a) {
  using N = Num<V>;
  constexpr int GW = 32 / LR, M = kNums<V>, RB = V == 1 ? 128 : LR * 2 * V;  // RB: a row's place in shared memory
  __shared__ Place place[kTokens];
  __shared__ __align__(16) float rows[I4 ? kWarps * GW * RB : 1];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, grp = lane / LR, l = lane % LR;
  const uint32_t t0 = blockIdx.x * a.per, n = min((uint32_t)a.per, a.tokens - t0);
  Slot<V> slot[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) slot[i].template set<IL>((l + i * LR) * V, a.D, a.R);
  // row r of the token at its place in q, k and v
  auto fetch = [&](Raw<T, V> (&x)[NP], uint32_t tok, int r) {
    const uint32_t b = tok / a.T, t = tok % a.T;
    r = min(r, a.rows - 1);  // rows past the last: the last again
    const int h = r - a.H;
    const T* p = r < a.H      ? static_cast<const T*>(a.q) + b * a.qs[0] + t * a.qs[1] + r * a.qs[2]
                 : h < a.Hkv  ? static_cast<const T*>(a.k) + b * a.ks[0] + t * a.ks[1] + h * a.ks[2]
                              : static_cast<const T*>(a.v) + b * a.vs[0] + t * a.vs[1] + (h - a.Hkv) * a.vs[2];
#pragma unroll
    for (int i = 0; i < NP; ++i) x[i] = load(p, slot[i]);
  };
  const int step = a.parts * GW;
  const uint32_t jobs = n * a.parts;
  Raw<T, V> next[NP];
  if ((uint32_t)w < jobs) fetch(next, t0 + w / a.parts, w % a.parts * GW + grp);  // on its way while the places are looked up
  if (threadIdx.x < n) place[threadIdx.x] = place_of(a, t0 + threadIdx.x);
  if (a.cu && blockIdx.x == 0 && !rises(a.cu, a.c.nseq, (int)a.tokens, false) && threadIdx.x == 0) report(GDN_ERR_SEQLENS);
  __syncthreads();
  for (uint32_t job = w; job < jobs; job += kWarps) {
    const uint32_t i0 = job / a.parts, tok = t0 + i0;
    const int part = job % a.parts;
    const Place at = place[i0];
    Angles<V> g[NP];
    if (a.R && at.turn) {
#pragma unroll
      for (int i = 0; i < NP; ++i) g[i].set(a.cos, a.sin, (long long)at.n * (a.R / 2), (l + i * LR) * V, slot[i].rot);
    }
    for (int r0 = part * GW; r0 < a.rows; r0 += step) {
      const int r = r0 + grp, h = r - a.H;
      N xa[NP][M], xb[NP][M];
#pragma unroll
      for (int i = 0; i < NP; ++i) widen<IL>(next[i], xa[i], xb[i]);
      if (r0 + step < a.rows) {
        fetch(next, tok, r + step);
      } else if (job + kWarps < jobs) {
        fetch(next, t0 + (job + kWarps) / a.parts, (job + kWarps) % a.parts * GW + grp);
      }
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (slot[i].rot && h < a.Hkv && at.turn) g[i].turn(xa[i], xb[i]);
      if (r < a.H) {
        T* y = static_cast<T*>(a.qo) + ((uint64_t)tok * a.H + r) * a.D;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (!at.turn) {
#pragma unroll
            for (int e = 0; e < M; ++e) xa[i][e] = xb[i][e] = splat<V>(0.f);
          }
          store<IL>(y, slot[i], xa[i], xb[i]);
        }
      }
      const bool isk = h < a.Hkv, keep = h >= 0 && r < a.rows && at.keep;
      const int hk = isk ? h : h - a.Hkv;
      const long long* st = isk ? a.c.ks : a.c.vs;
      const long long to = at.page * st[0] + at.at * st[1] + hk * st[2];
      if constexpr (!I4) {
        if (!keep) continue;
        T* y = static_cast<T*>(isk ? a.c.k : a.c.v) + to;
#pragma unroll
        for (int i = 0; i < NP; ++i) store<IL>(y, slot[i], xa[i], xb[i]);
      } else {
        if (r0 + GW <= a.H) continue;  // only queries: the same for the whole warp
        float* row = rows + (w * GW + grp) * RB;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NP; ++i) store<IL>(row, slot[i], xa[i], xb[i]);
        __syncwarp();
        // 8 values in a row of each lane (V = 8: two passes of half a row's lanes)
        constexpr int Q = V == 8 ? 2 : 1;
#pragma unroll
        for (int p = 0; p < Q; ++p) {
          const int c = l + p * LR;
          const bool in = c < a.D / 8;
          float y[8], step8;
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const float4 x = in ? *reinterpret_cast<const float4*>(row + 8 * c + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            y[e] = x.x, y[e + 1] = x.y, y[e + 2] = x.z, y[e + 3] = x.w;
          }
          const uint32_t codes = quantise8(y, step8);
          if (!keep || !in) continue;
          const long long* ss = isk ? a.c.kss : a.c.vss;
          *reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(isk ? a.c.k : a.c.v) + to + 4 * c) = codes;
          if (c % 4 == 0)
            static_cast<__nv_bfloat16*>(isk ? a.c.k_scale : a.c.v_scale)[at.page * ss[0] + at.at * ss[1] + hk * ss[2] + c / 4] =
                __float2bfloat16_rn(step8);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- gather

constexpr int kRun = 256;  // most tokens of a CTA

struct GatherArgs {
  Pages c;
  int total, Hkv, D, tokens;  // tokens per CTA
  uint32_t magic;             // ceil(2^32 / vectors of a row)
  const int* cu;
  void *k, *v;
};

template <typename O, int N>
struct alignas(16) Vec {
  O x[N];
};

// What eight codes stand for.  Put into the mantissas of bf16 128s, two at a time,
// they are 128 + (code + 8); less 136 and times the step each is rounded once at most.
__device__ __forceinline__ void codes_of(uint32_t w, __nv_bfloat162 (&c)[4]) {  // values (n, n + 4)
  const uint32_t off = 0xc308c308u;  // -136
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const uint32_t x = (w >> (4 * n) & 0x000f000fu) | 0x43004300u;
    c[n] = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&off));
  }
}
__device__ __forceinline__ void values8(uint32_t w, __nv_bfloat16 step, __nv_bfloat16 (&y)[8]) {
  __nv_bfloat162 c[4];
  codes_of(w, c);
  uint32_t v[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const __nv_bfloat162 p = __hmul2_rn(c[n], __halves2bfloat162(step, step));
    v[n] = *reinterpret_cast<const uint32_t*>(&p);
  }
  uint32_t* o = reinterpret_cast<uint32_t*>(y);
  o[0] = __byte_perm(v[0], v[1], 0x5410), o[1] = __byte_perm(v[2], v[3], 0x5410);
  o[2] = __byte_perm(v[0], v[1], 0x7632), o[3] = __byte_perm(v[2], v[3], 0x7632);
}
__device__ __forceinline__ void values8(uint32_t w, __nv_bfloat16 step, float (&y)[8]) {
  __nv_bfloat162 c[4];
  codes_of(w, c);
  const float s = __bfloat162float(step);
#pragma unroll
  for (int n = 0; n < 4; ++n) y[n] = __low2float(c[n]) * s, y[n + 4] = __high2float(c[n]) * s;
}

template <typename O, bool I4, int V>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(GatherArgs a) {
  __shared__ long long from[kRun], step_from[I4 ? kRun : 1];
  const bool isv = blockIdx.y;
  const int t0 = blockIdx.x * a.tokens, n = min(a.tokens, a.total - t0);
  if (blockIdx.x == 0 && !isv && !rises(a.cu, a.c.nseq, a.total, true) && threadIdx.x == 0) report(GDN_ERR_SEQLENS);
  const long long* st = isv ? a.c.vs : a.c.ks;
  const long long* ss = isv ? a.c.vss : a.c.kss;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    long long at = -1;  // not of any row: left as it is
    if (a.c.nseq > 0) {
      const int tok = t0 + i, row = sequence_of(a.cu, a.c.nseq, tok);
      const long long slot = (long long)tok - a.cu[row];
      if (slot >= 0 && tok < a.cu[row + 1]) {
        at = -2;  // without a page: zeros
        if (slot < ((long long)a.c.max_pages << a.c.shift)) {
          const int page = page_of(a.c, row, slot);
          const int place = (int)slot & ((1 << a.c.shift) - 1);
          if (page >= 0) {
            at = page * st[0] + place * st[1];
            if constexpr (I4) step_from[i] = page * ss[0] + place * ss[1];
          }
        } else {
          report(GDN_ERR_SEQLENS);
        }
      }
    }
    from[i] = at;
  }
  __syncthreads();
  // Vector i of the run is number i % per of token i / per, kept up by steps of a CTA's
  // threads; head and vector of the row by a multiplication (rem < 2^20 or so, a
  // reciprocal rounded up: exact).
  const uint32_t nv = a.D / V, per = a.Hkv * nv, all = n * per, dt = kThreads / per, dr = kThreads % per;
  O* out = static_cast<O*>(isv ? a.v : a.k) + (long long)t0 * a.Hkv * a.D;
  const unsigned char* src = static_cast<const unsigned char*>(isv ? a.c.v : a.c.k);
  const __nv_bfloat16* scale = static_cast<const __nv_bfloat16*>(isv ? a.c.v_scale : a.c.k_scale);
  constexpr int U = 2;  // (4 and 8 on their way: 45 and 62 us for 42)
  uint32_t t = threadIdx.x / per, rem = threadIdx.x % per;
  for (uint32_t i0 = threadIdx.x; i0 < all; i0 += U * kThreads) {
    Vec<O, V> y[U];
    bool put[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i0 + u * kThreads, h = nv == 1 ? rem : __umulhi(rem, a.magic), d = (rem - h * nv) * V;
      put[u] = false;
      if (i < all) {
        const long long at = from[t];
        put[u] = at != -1;
        if (at < 0) {
#pragma unroll
          for (int e = 0; e < V; ++e) y[u].x[e] = from_f32<O>(0.f);
        } else if constexpr (I4) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(src + at + h * st[2] + d / 2);
          values8(w, scale[step_from[t] + h * ss[2] + d / kStepGroup], y[u].x);
        } else {
          const O* p = reinterpret_cast<const O*>(src) + at + h * st[2] + d;
          if constexpr (V > 1) y[u] = *reinterpret_cast<const Vec<O, V>*>(p);
          else y[u].x[0] = p[0];
        }
      }
      t += dt, rem += dr;
      if (rem >= per) rem -= per, ++t;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      O* to = out + (uint64_t)(i0 + u * kThreads) * V;
      if (!put[u]) continue;
      if constexpr (V > 1) *reinterpret_cast<Vec<O, V>*>(to) = y[u];
      else to[0] = y[u].x[0];
    }
  }
}

// ---------------------------------------------------------------- host

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, int V, int NP, int LR>
cudaError_t append(AppendArgs a, bool interleaved, bool i4, cudaStream_t s) {
  constexpr int GW = 32 / LR;
  // All CTAs at once, where their runs are long enough (10541 tokens of 4 heads: 13 us;
  // two, three and four times as many CTAs 16, 15 and 17); a short run's tokens are
  // shared by warps.
  const long fit = kPerSm * sm_count();
  a.per = (int)std::min((long)kTokens, (a.tokens + fit - 1) / fit);
  a.parts = std::max(1, std::min((a.rows + GW - 1) / GW, kWarps / a.per));
  const unsigned ctas = (a.tokens + a.per - 1) / a.per;
  prof_before(s);
  if (interleaved)
    i4 ? kv_append_kernel<T, V, NP, LR, true, true><<<ctas, kThreads, 0, s>>>(a)
       : kv_append_kernel<T, V, NP, LR, true, false><<<ctas, kThreads, 0, s>>>(a);
  else
    i4 ? kv_append_kernel<T, V, NP, LR, false, true><<<ctas, kThreads, 0, s>>>(a)
       : kv_append_kernel<T, V, NP, LR, false, false><<<ctas, kThreads, 0, s>>>(a);
  prof_after(s, kKvAppend);
  return cudaGetLastError();
}

template <typename T>
cudaError_t append(const KvAppendProblem& p, const PagedCache& c, cudaStream_t s) {
  AppendArgs a = {};
  a.c = pages_of(c, p.pt);
  a.T = p.T, a.H = p.H, a.Hkv = c.Hkv, a.rows = p.H + 2 * c.Hkv, a.D = c.D, a.R = p.R, a.P = p.P;
  a.tokens = (uint32_t)((long)p.B * p.T);
  for (int i = 0; i < 3; ++i) a.qs[i] = p.qs[i], a.ks[i] = p.ks[i], a.vs[i] = p.vs[i];
  a.q = p.q, a.k = p.k, a.v = p.v, a.cos = p.cos, a.sin = p.sin, a.lens = p.lens, a.cu = p.cu, a.qo = p.qo;
  const bool i4 = c.format == GDN_CACHE_I4;
  bool vec = vectors(p.k, p.ks, sizeof(T)) && vectors(p.v, p.vs, sizeof(T)) &&
             (p.H == 0 || (vectors(p.q, p.qs, sizeof(T)))) && aligned16(p.cos) && aligned16(p.sin);
  if (!i4) vec = vec && vectors(c.k, c.ks, sizeof(T)) && vectors(c.v, c.vs, sizeof(T));
  if constexpr (sizeof(T) == 2) {
    if (vec && a.D % 16 == 0 && a.R % 16 == 0)
      return a.D <= 64 ? append<T, 8, 1, 4>(a, p.interleaved, i4, s) : append<T, 8, 1, 8>(a, p.interleaved, i4, s);
  }
  if (vec && a.D % 8 == 0 && a.R % 8 == 0)
    return a.D <= 64 ? append<T, 4, 1, 8>(a, p.interleaved, i4, s) : append<T, 4, 1, 16>(a, p.interleaved, i4, s);
  return append<T, 1, 2, 32>(a, p.interleaved, i4, s);
}

template <typename O, bool I4, int V>
cudaError_t gather(GatherArgs a, cudaStream_t s) {
  // About four vectors per thread; more where there is work for 32 CTAs per SM (16 for
  // k, 16 for v) all the same: short runs end together.  60898 tokens of 4 heads of
  // 128, bf16: 42 us, with runs eight times as long 51.
  const int nv = a.D / V, few = 4 * kThreads / (a.Hkv * nv);
  a.tokens = std::max(1, std::min(kRun, std::max(few, a.total / (16 * sm_count()))));
  a.magic = nv == 1 ? 0 : (uint32_t)(((1ull << 32) + nv - 1) / nv);
  prof_before(s);
  kv_gather_kernel<O, I4, V><<<dim3((a.total + a.tokens - 1) / a.tokens, 2), kThreads, 0, s>>>(a);
  prof_after(s, kKvGather);
  return cudaGetLastError();
}

template <typename O>
cudaError_t gather(const KvGatherProblem& p, const PagedCache& c, cudaStream_t s) {
  GatherArgs a = {};
  a.c = pages_of(c, p.pt);
  a.total = p.total, a.Hkv = c.Hkv, a.D = c.D, a.cu = p.cu, a.k = p.k, a.v = p.v;
  constexpr int V = 16 / (int)sizeof(O);
  if (c.format == GDN_CACHE_I4) return gather<O, true, 8>(a, s);
  if (a.D % V == 0 && vectors(c.k, c.ks, sizeof(O)) && vectors(c.v, c.vs, sizeof(O))) return gather<O, false, V>(a, s);
  return gather<O, false, 1>(a, s);
}

}  // namespace

cudaError_t kv_append(const KvAppendProblem& p, const PagedCache& c, cudaStream_t s) {
  return p.bf16 ? append<__nv_bfloat16>(p, c, s) : append<float>(p, c, s);
}

cudaError_t kv_gather(const KvGatherProblem& p, const PagedCache& c, cudaStream_t s) {
  return p.bf16 ? gather<__nv_bfloat16>(p, c, s) : gather<float>(p, c, s);
}

}  // namespace gdn
