// packed.cuh -- what the packed-attention kernels share: the sequences of a
// packed token axis, and the tile of a sequence that a CTA works on.
//
// The lengths stand in device memory (cumulative, values out of range or
// order clamped to the tensors), and no call knows them on the host: a grid
// covers the most tiles the lengths could give (tokens / tile + sequences)
// and every CTA finds its tile by itself.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace hsnf4 {

constexpr float kLog2e = 1.4426950408889634f;

struct PackedSeqs {
  const int32_t *cu_q, *cu_k;
  int Tq, Tk, n_seq, causal;
};

struct PackedTile {
  int q0, lq, k0, lk;  // the sequence's first query and key token and its lengths
  int t;               // tile of the sequence (of its queries or of its keys)
};

__device__ __forceinline__ void seq_range(const int32_t* cu, int s, int T, int& a, int& len) {
  const int b = min(max(__ldg(cu + s), 0), T), e = min(__ldg(cu + s + 1), T);
  a = b;
  len = max(e - b, 0);
}

// Tile number `slot` over all sequences in order, tiles of `rows` tokens of
// the queries (or keys).  Within a sequence the longest work comes first
// under a causal mask: query tiles from the last, key tiles from the first.
// Whole warp; false if there is no such tile.
__device__ __forceinline__ bool find_tile(const PackedSeqs& S, bool keys, int slot, int rows,
                                          PackedTile& x) {
  const int lane = threadIdx.x & 31;
  const int32_t* cu = keys ? S.cu_k : S.cu_q;
  const int T = keys ? S.Tk : S.Tq;
  int before = 0;
  for (int s0 = 0; s0 < S.n_seq; s0 += 32) {
    int a = 0, len = 0;
    if (s0 + lane < S.n_seq) seq_range(cu, s0 + lane, T, a, len);
    const int n = (len + rows - 1) / rows;
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const int lo = before + inc - n;
    const unsigned hit = __ballot_sync(0xffffffffu, slot >= lo && slot < lo + n);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int s = s0 + src;
      x.t = __shfl_sync(0xffffffffu, keys ? slot - lo : n - 1 - (slot - lo), src);
      seq_range(S.cu_q, s, S.Tq, x.q0, x.lq);
      seq_range(S.cu_k, s, S.Tk, x.k0, x.lk);
      return true;
    }
    before = __shfl_sync(0xffffffffu, before + inc, 31);
  }
  return false;
}

// keys that query row i of the tile's sequence sees: [0, limit)
__device__ __forceinline__ int key_limit(const PackedSeqs& S, const PackedTile& x, int i) {
  return S.causal ? min(max(i + x.lk - x.lq + 1, 0), x.lk) : x.lk;
}

}  // namespace hsnf4
