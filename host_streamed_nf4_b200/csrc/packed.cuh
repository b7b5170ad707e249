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
  int sorted;  // key tiles in the order of their work, over all sequences (n_seq <= 128)
};

struct PackedTile {
  int q0, lq, k0, lk;  // the sequence's first query and key token and its lengths
  int t;               // tile of the sequence (of its queries or of its keys)
};

// The tokens of [start, end) that a tensor of T has, from any two values.  Both
// are clamped before they are subtracted: from one that is not the difference
// of two int32 may wrap around to a length far beyond the tensor.
struct Span {
  int at, len;
};
__host__ __device__ __forceinline__ Span span_of(int start, int end, int T) {
  const int a = start < 0 ? 0 : start > T ? T : start, b = end < 0 ? 0 : end > T ? T : end;
  return {a, b > a ? b - a : 0};
}

// Tile number `slot` over all sequences in order, tiles of `rows` tokens of
// the queries (or keys).  Within a sequence the longest work comes first
// under a causal mask: query tiles from the last, key tiles from the first.
// Whole warp, four sequences a lane at a time: up to 128 sequences cost one
// round trip to memory.  False if there is no such tile.
//
// SORT, where S.sorted: the longest work of all sequences first.  Under a
// causal mask a sequence of n tiles has tiles of the levels n, n - 1 ... 1
// (query tiles that see them, for queries as many as keys); without one its
// tiles all have the level of its query tiles.
template <bool SORT = false>
__device__ __forceinline__ bool find_tile(const PackedSeqs& S, bool keys, int slot, int rows,
                                          PackedTile& x) {
  const int lane = threadIdx.x & 31;
  const bool same = S.cu_q == S.cu_k;
  int before = 0;
  for (int s0 = 0; s0 < S.n_seq; s0 += 128) {
    int cq[5], ck[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      const int i = min(s0 + 4 * lane + j, S.n_seq);  // behind the last: empty
      cq[j] = __ldg(S.cu_q + i);
      ck[j] = same ? cq[j] : __ldg(S.cu_k + i);
    }
    int n[4], sum = 0;  // tiles to number
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int len =
          keys ? span_of(ck[j], ck[j + 1], S.Tk).len : span_of(cq[j], cq[j + 1], S.Tq).len;
      n[j] = (len + rows - 1) / rows;
      sum += n[j];
    }
    int level = 0, first[4] = {};  // sorted: of the tile; of the first tile of that level
    if (SORT && S.sorted) {
      int top[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int lq = span_of(cq[j], cq[j + 1], S.Tq).len;
        top[j] = n[j] == 0 ? 0 : S.causal ? n[j] : 1 + (lq + rows - 1) / rows;
      }
      // tiles of level v and above
      auto count = [&](int v) {
        int k = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) k += S.causal ? max(n[j] - v + 1, 0) : top[j] >= v ? n[j] : 0;
        return __reduce_add_sync(0xffffffffu, k);
      };
      if (slot >= count(1)) return false;
      int low = 1, high = __reduce_max_sync(0xffffffffu,
                                            max(max(top[0], top[1]), max(top[2], top[3])));
      while (low < high) {  // the highest level that has, with those above, more than `slot`
        const int mid = (low + high + 1) / 2;
        if (count(mid) > slot)
          low = mid;
        else
          high = mid - 1;
      }
      level = low;
      before = count(level + 1);
      sum = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        first[j] = S.causal ? n[j] - level : 0;
        n[j] = S.causal ? n[j] >= level : top[j] == level ? n[j] : 0;
        sum += n[j];
      }
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const int lo = before + inc - sum;
    const unsigned hit = __ballot_sync(0xffffffffu, slot >= lo && slot < lo + sum);
    if (hit) {
      const int src = __ffs(hit) - 1;
      int at = slot - lo, t = 0, aq = 0, eq = 0, ak = 0, ek = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (at >= 0 && at < n[j]) {
          t = keys ? first[j] + at : n[j] - 1 - at;
          aq = cq[j], eq = cq[j + 1], ak = ck[j], ek = ck[j + 1];
        }
        at -= n[j];
      }
      x.t = __shfl_sync(0xffffffffu, t, src);
      const Span q = span_of(__shfl_sync(0xffffffffu, aq, src), __shfl_sync(0xffffffffu, eq, src),
                             S.Tq);
      const Span k = span_of(__shfl_sync(0xffffffffu, ak, src), __shfl_sync(0xffffffffu, ek, src),
                             S.Tk);
      x = {q.at, q.len, k.at, k.len, __shfl_sync(0xffffffffu, t, src)};
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
