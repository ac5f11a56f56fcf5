// The sequences of an attention call, shared by the attention kernel files.
#pragma once

#include <cuda_bf16.h>

#include "gdn.h"
#include "gdn_internal.cuh"

namespace gdn {

// One tile of rows of one sequence: its batch row, first query / key token
// (within the row), lengths, and the tile's index.
struct AttnTile {
  int seq, b, q0, lq, k0, lk, tile;
};

// Tiles are numbered without a set-up pass.  A batch: tile t of row b is slot
// b * ceil(T / M) + t.  Packed: tile t of sequence s is slot cu[s] / M + s + t.
// The numbers of different sequences do not meet, since
// floor(b / M) - floor(a / M) + 1 >= ceil((b - a) / M); at most nseq + T / M
// slots are needed and those past a sequence's end are empty.
struct AttnSeqs {
  const int *cu_q, *cu_k;
  int nseq, B, Tq, Tk;

  static AttnSeqs of(const AttnProblem& p) {
    return AttnSeqs{p.cu_q, p.cu_k, p.cu_q ? p.nseq : p.B, p.B, p.Tq, p.Tk};
  }
  // slots of tiles of M rows of the queries (or of the keys)
  static long slots(const AttnProblem& p, int M, bool keys) {
    const int T = keys ? p.Tk : p.Tq;
    return p.cu_q ? (long)(T / M) + p.nseq : (long)p.B * ((T + M - 1) / M);
  }

  // Offsets are clamped into [0, T]: bad ones give wrong rows, never an
  // access outside the tensors.
  __device__ __forceinline__ void lengths(int s, AttnTile& t) const {
    t.seq = s;
    if (!cu_q) {
      t.b = s, t.q0 = 0, t.lq = Tq, t.k0 = 0, t.lk = Tk;
      return;
    }
    t.b = 0;
    t.q0 = min(max(cu_q[s], 0), Tq);
    t.lq = min(max(cu_q[s + 1], t.q0), Tq) - t.q0;
    t.k0 = min(max(cu_k[s], 0), Tk);
    t.lk = min(max(cu_k[s + 1], t.k0), Tk) - t.k0;
  }

  // The tile of a slot of tiles of M rows; false for an empty slot.
  template <bool kKeys>
  __device__ __forceinline__ bool get(int slot, int M, AttnTile& t) const {
    const int T = kKeys ? Tk : Tq;
    if (!cu_q) {
      const int n = (T + M - 1) / M;
      lengths(slot / n, t);
      t.tile = slot % n;
      return true;
    }
    const int* cu = kKeys ? cu_k : cu_q;
    int lo = 0, hi = nseq - 1;  // the last s whose first slot is <= slot
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (cu[mid] / M + mid <= slot) lo = mid;
      else hi = mid - 1;
    }
    lengths(lo, t);
    t.tile = slot - (cu[lo] / M + lo);
    return t.tile >= 0 && t.tile < ((kKeys ? t.lk : t.lq) + M - 1) / M;
  }

  // Whether the packed offsets rise from 0 to T (all threads of the CTA call).
  __device__ bool valid() const {
    if (!cu_q) return true;
    int bad = 0;
    if (threadIdx.x == 0)
      bad = cu_q[0] != 0 || cu_q[nseq] != Tq || cu_k[0] != 0 || cu_k[nseq] != Tk;
    for (int s = threadIdx.x; s < nseq; s += blockDim.x)
      bad |= (cu_q[s + 1] < cu_q[s]) | (cu_k[s + 1] < cu_k[s]);
    return !__syncthreads_or(bad);
  }
};

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

}  // namespace gdn
