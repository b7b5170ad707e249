// attention_packed.cu -- attention over several sequences packed into one
// token axis, forward and backward, head_dim 64 or 128, causal or not, on the
// tcgen05 tensor cores.
//
// Per sequence (lq queries, lk keys) and query head h with KV head
// h / (H / KV):
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j <= i + lk - lq
//   (causal) or all keys;  lse_i = log sum_j e^{scale q_i . k_j}
//   D_i = dout_i . o_i,  P_ij = e^{scale q_i . k_j - lse_i},
//   dS_ij = P_ij (dout_i . v_j - D_i)
//   dq = scale dS k,  dk = scale dS^T q,  dv = P^T dout
// Scores, statistics and sums are fp32; P and dS are rounded to bf16 as
// operands of the second products (2^-8 relative at most, the size of the
// outputs' own rounding).
//
// No atomics: dQ and dK/dV come from two kernels that each recompute P (seven
// products where five would do with unordered additions), and heads that
// share a KV head are added in order.
#include <cuda_bf16.h>

#include <string.h>

#include <algorithm>
#include <atomic>

#include "attention_tc.cuh"
#include "internal.h"
#include "packed.cuh"

namespace hsnf4 {

__device__ unsigned int g_attn_flags;

namespace {

enum : unsigned int {
  kAtFlagLoad = 1u << 19,
  kAtFlagMma = 1u << 20,
  kAtFlagCompute = 1u << 21,
  kAtFlagDrain = 1u << 22,
};

// Of every kPolyOf pairs of exponentials, kPolyPart go to the fp32 pipe.
constexpr int kPolyOf = 8, kPolyPart = 2;
constexpr int kReduceThreads = 512;
// The least reference of a row's exponentials, of a row whose first keys'
// scores are all -inf: with any more, later scores far below it would be lost.
constexpr float kLowRef = -3.402823466e38f;

// mbar_wait with the abort word and the timer looked at every 32 polls only:
// reading the timer takes hundreds of cycles, by which each wait ended late.
__device__ __forceinline__ bool spin_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          unsigned int site) {
  const uint32_t a = smem_u32(bar);
  unsigned long long t0 = 0;
  for (uint32_t k = 1;; ++k) {
    if (mbar_try_wait(a, parity)) return true;
    if (k % 32) continue;
    if (*abort) return false;
    const unsigned long long t = global_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitLimitNs) {
      *abort = 1;
      atomicOr(&g_attn_flags, site);
      return false;
    }
  }
}

// A wait of a whole warp, which leaves whole when it gives up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, int phase, volatile int* abort,
                                          unsigned int site) {
  return __all_sync(0xffffffffu, spin_wait(bar, phase & 1, abort, site));
}

// Whether the phase has completed, without waiting (whole warp).
__device__ __forceinline__ bool warp_test(uint64_t* bar, int phase) {
  return __all_sync(0xffffffffu, mbar_test(bar, phase & 1));
}

// Wait of the whole loading warp for a tile that it will patch.  Giving up,
// it first lets the copy land (or the limit pass) before the shared memory
// goes away.
__device__ __forceinline__ bool tail_landed(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (warp_wait(bar, parity, abort, kAtFlagLoad)) return true;
  volatile int never = 0;
  spin_wait(bar, parity, &never, kAtFlagDrain);
  return false;
}

// Two warps (64 threads) that share the rows of a tile: a barrier, and votes
// over both.
__device__ __forceinline__ void pair_sync(int id) {
  __syncwarp();
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool pair_any(int id, bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool pair_all(int id, bool v) { return !pair_any(id, !v); }

template <int THREADS>
__device__ __forceinline__ void bar_compute() {  // the computing threads
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

constexpr int kStep = 64;  // keys of a step where a step is not a tile

// 32 columns of this warp's lanes
__device__ __forceinline__ void load_quarter(uint32_t taddr, uint32_t* r) {
  tmem_ld32_at(taddr, r);
  tmem_wait_ld();
  tie32(r);
}

// ---------------------------------------------------------------- forward

struct FwdTc {
  CUtensorMap mq, mk, mv;
  uint16_t* out;
  float* lse;
  int64_t os;
  PackedSeqs S;
  int H, KV;
  float c;  // scale * log2(e)
};

__device__ __forceinline__ void prefetch_maps(const FwdTc& P) {
  tma_prefetch_desc(&P.mq);
  tma_prefetch_desc(&P.mk);
  tma_prefetch_desc(&P.mv);
}

// NQ query tiles of 128 rows per CTA: two share the keys' loads and keep the
// tensor cores busy in turn; with one, two CTAs fit an SM, so that one's start
// and end hide behind the other's work (short sequences).
template <int D, int NQ>
struct FwdGeo {
  static constexpr int kTile = tile_bytes<D>();
  static constexpr int kStages = NQ == 1 ? (D == 128 ? 2 : 4) : (D == 128 ? 4 : 8);
  static constexpr int kSmem = (NQ + kStages) * kTile;
  static constexpr int kWarps = 8 * NQ;  // computing warps; then the MMA issuer and the loader
  static constexpr int kThreads = 32 * (kWarps + 2);
  static constexpr uint32_t kO = 128 * NQ, kCols = 256 * NQ;  // TMEM: S per tile, then O per tile
};

// A CTA takes NQ tiles of 128 query rows of one head and walks the keys 128 at
// a time.  Each tile has eight warps: a row belongs to two threads, in two
// warps, 64 of the 128 keys each.  TMEM: an S per tile (P overwrites it as
// bf16), an O per tile.  The tensor cores work on one tile's products while
// the warps of the other (of the other CTA) compute its probabilities.
//
// One causal sequence, head_dim 128: 16384 tokens of 32/8 heads 2115 us, 1040
// TFLOP/s, in a loop, where the power limit lowers the clock to about 1.64 GHz
// with the tensor pipe 53 % busy (a call from rest: 1890); 4096 of 28/4 heads
// 119 us.  Short calls are bound by the latency of a CTA's start, chain and
// end, 5 us and 2 us a step (nine sequences of 512 tokens: 8.6 us).
template <int D, int NQ>
__global__ void __launch_bounds__(FwdGeo<D, NQ>::kThreads, 3 - NQ)
    packed_fwd_tc(const __grid_constant__ FwdTc P) {
  using G = FwdGeo<D, NQ>;
  constexpr int NS = G::kStages, kMmaWarp = G::kWarps, kLoadWarp = G::kWarps + 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t q_full, kv_full[NS], kv_empty[NS], aux, s_full[NQ], p_full[NQ][2], o_full[NQ],
      drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ float row_x[2][NQ][kRows];  // [half][tile][row]: exchanged between two warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0 && lane == 0) prefetch_maps(P);
  pdl_wait();
  // (before anything is set up: the grid covers the most tiles there could be)
  PackedTile x;
  if (!find_tile(P.S, false, blockIdx.x / P.H, NQ * kRows, x)) return;
  if (threadIdx.x == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&aux, 1);
    mbar_init(&drain, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int t = 0; t < NQ; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t][0], 8);
      mbar_init(&p_full[t][1], 8);
      mbar_init(&o_full[t], 1);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_slot, G::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_release();  // (after the allocation)
  // with two tiles all 512 columns are this CTA's: a base known at compile time
  const uint32_t tmem = NQ == 2 ? 0u : tmem_slot;
  volatile int* abort_p = &abort_flag;
  // the swizzled tiles need the alignment asked for
  if ((smem_u32(smem) & 1023u) || tmem_slot != tmem) {
    if (threadIdx.x == 0) atomicOr(&g_attn_flags, kAtFlagLoad);
    if (warp == kMmaWarp) tmem_dealloc(tmem_slot, G::kCols);
    return;
  }

  const int h = blockIdx.x % P.H, kh = h / (P.H / P.KV);
  int last_load = -1, n = 0, nt[NQ] = {};
  bool q_loaded = false, mma_issued = false;
  const int r0 = x.t * NQ * kRows;
  for (int t = 0; t < NQ; ++t) {
    const int first = r0 + t * kRows, end = min(first + kRows, x.lq);
    if (first < end) nt[t] = (key_limit(P.S, x, end - 1) + kRows - 1) / kRows;
    n = max(n, nt[t]);
  }
  uint8_t* ring = smem + NQ * G::kTile;

  if (warp == kLoadWarp && n) {
    // ---------------------------------------------- TMA: Q, then K0 V0 K1 V1 ...
    // (of a tile that sees no key only the output's zeros are staged there,
    // without a wait: no copy may be on its way)
    if (lane == 0) {
      int tiles = 0;
      for (int t = 0; t < NQ; ++t) tiles += nt[t] > 0;
      mbar_arrive_expect_tx(&q_full, tiles * G::kTile);
      for (int t = 0; t < NQ; ++t)
        if (nt[t])
          tma_tile<D>(smem + t * G::kTile, &P.mq, &q_full, h * D, x.q0 + r0 + t * kRows);
    }
    q_loaded = true;
    for (int i = 0; i < 2 * n; ++i) {
      const int s = i % NS, row = (i >> 1) * kRows;
      if (i >= NS && !warp_wait(&kv_empty[s], (i / NS) - 1, abort_p, kAtFlagLoad))
        break;
      uint8_t* st = ring + s * G::kTile;
      const CUtensorMap* map = (i & 1) ? &P.mv : &P.mk;
      if ((i & 1) && row + kRows > x.lk) {
        // the keys behind the sequence have probability 0; their values must
        // be finite for the product: zeros
        if (lane == 0) {
          mbar_arrive_expect_tx(&aux, G::kTile);
          tma_tile<D>(st, map, &aux, kh * D, x.k0 + row);
        }
        __syncwarp();
        if (!tail_landed(&aux, 0, abort_p)) break;
        zero_rows<D>(st, x.lk - row);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[s]);
      } else if (lane == 0) {
        mbar_arrive_expect_tx(&kv_full[s], G::kTile);
        tma_tile<D>(st, map, &kv_full[s], kh * D, x.k0 + row);
      }
      last_load = i;
    }
  } else if (warp == kMmaWarp && n) {
    // ---------------------------------------------- MMA issuer
    auto wait = [&](uint64_t* bar, int phase) {
      const bool ok = warp_wait(bar, phase, abort_p, kAtFlagMma);
      tc_fence_after();
      return ok;
    };
    auto full = [&](int i) { return wait(&kv_full[i % NS], i / NS); };
    auto stage = [&](int i) { return ring + (i % NS) * G::kTile; };
    auto scores = [&](int t, int j) {  // S_t = Q_t K_j^T
      if (elect_one()) {
        mma_xyt<D>(tmem + t * 128, smem + t * G::kTile, stage(2 * j));
        umma_commit(&s_full[t]);
      }
      __syncwarp();
    };
    auto values = [&](int t, int j) {  // O_t += P_t V_j
      // P becomes ready in two parts, 32 of each half's 64 keys
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (!wait(&p_full[t][part], j)) return false;
        if (elect_one()) {
          mma_ay_steps<D, 64>(tmem + G::kO + t * 128, tmem + t * 128, 64, stage(2 * j + 1),
                              2 * part, 2, j > 0 || part > 0);
          if (part == 1) umma_commit(&o_full[t]);
        }
        __syncwarp();
      }
      return true;
    };
    auto release = [&](int i) {
      if (elect_one()) umma_commit(&kv_empty[i % NS]);
      __syncwarp();
    };
    bool ok = wait(&q_full, 0) && full(0);
    if (ok) {
      mma_issued = true;
      for (int t = 0; t < NQ; ++t)
        if (nt[t]) scores(t, 0);
      release(0);
    }
    for (int j = 0; j < n && ok; ++j) {
      const bool more = j + 1 < n;
      ok = full(2 * j + 1);
      if (ok && j < nt[0]) ok = values(0, j);
      if (ok && more) ok = full(2 * j + 2);
      if (ok && j + 1 < nt[0]) scores(0, j + 1);
      if (ok && NQ == 2 && j < nt[NQ - 1]) ok = values(NQ - 1, j);
      if (!ok) break;
      release(2 * j + 1);
      if (NQ == 2 && j + 1 < nt[NQ - 1]) scores(NQ - 1, j + 1);
      if (more) release(2 * j + 2);
    }
  } else if (warp < G::kWarps) {
    // ---------------------------------------------- softmax: half a row per thread
    // tile t, half of the 128 keys, and the TMEM lane quarter of the warp
    const int t = warp >> 3, half = (warp >> 2) & 1, q4 = warp & 3, tid = q4 * 32 + lane;
    const int row = r0 + t * kRows + tid;
    const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t S_h = tmem + t * 128 + half * 64 + lanes;
    const uint32_t O_h = tmem + G::kO + t * 128 + half * (D / 2) + lanes;
    const int pair = 1 + t * 4 + q4;  // barrier of the two warps that share the rows
    const int limit = key_limit(P.S, x, row);
    const uint64_t c2 = f32x2_pack(P.c, P.c);
    float ref = 0.0f, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < nt[t]; ++j) {
      // both warps of a row leave together: their barriers must match
      ok = pair_all(pair, warp_wait(&s_full[t], j, abort_p, kAtFlagCompute));
      if (!ok) break;
      tc_fence_after();
      const int lim = limit - j * kRows - half * 64;
      const bool mask = __any_sync(0xffffffffu, lim < 64);
      // 32 columns at a time, read once for the maximum and once more for the
      // probabilities: holding all 64 spilled registers
      auto scores = [&](int b, uint32_t* s) {
        load_quarter(S_h + 32 * b, s);
        if (!mask) return;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (32 * b + e >= lim) s[e] = 0xff800000u;  // -inf
      };
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t s[32];
        scores(b, s);
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          m4[(e >> 1) & 3] = max_nan(max_nan(m4[(e >> 1) & 3], __uint_as_float(s[e])),
                                     __uint_as_float(s[e + 1]));
      }
      // (a row behind the sequence holds another's values and has no say)
      const float mt = row < x.lq ? max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3])) * P.c
                                  : -INFINITY;
      // The reference of a row's exponentials moves only when a score passes
      // it by 2^8 (fp32 sums and bf16 probabilities lose nothing at that
      // size); then O and the sum are scaled to the new one.
      if (pair_any(pair, j == 0 || mt > ref + 8.0f)) {
        row_x[half][t][tid] = mt;
        pair_sync(pair);
        const float m = fmaxf(mt, row_x[half ^ 1][t][tid]);
        if (j == 0) {
          ref = fmaxf(m, kLowRef);
        } else {
          ok = pair_all(pair, warp_wait(&o_full[t], (j - 1), abort_p, kAtFlagCompute));
          if (!ok) break;
          tc_fence_after();
          const float next = fmaxf(ref, m), f = ex2(ref - next);
          ref = next;
          l *= f;
          const uint64_t f2 = f32x2_pack(f, f);
#pragma unroll
          for (int b = 0; b < D / 64; ++b) {
            uint32_t o[32];
            tmem_ld32_at(O_h + 32 * b, o);
            tmem_wait_ld();
            tie32(o);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float lo, hi;
              f32x2_unpack(f32x2_mul_rn(f32x2_pack_bits(o[e], o[e + 1]), f2), lo, hi);
              o[e] = __float_as_uint(lo);
              o[e + 1] = __float_as_uint(hi);
            }
            tmem_st32(O_h + 32 * b, o);
          }
        }
      }
      const uint64_t r2 = f32x2_pack(-ref, -ref);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t s[32], p[16];
        scores(b, s);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t y = f32x2_fma_rn(f32x2_pack_bits(s[2 * e], s[2 * e + 1]), c2, r2);
          const uint64_t pr = e % kPolyOf < kPolyPart ? ex2_poly<false>(y) : ex2_pair(y);
          sum[e & 1] = f32x2_add_rn(sum[e & 1], pr);
          p[e] = f32x2_to_bf16x2(pr);
        }
        tmem_st16(S_h + 16 * b, p);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t][b]);
      }
      float a0, a1;
      f32x2_unpack(f32x2_add_rn(sum[0], sum[1]), a0, a1);
      l += a0 + a1;
      // a NaN or an infinite score makes the row NaN (the polynomial gives 0 for it)
      if (!(mt < INFINITY)) l = NAN;
    }
    if (ok && nt[t])
      ok = pair_all(pair, warp_wait(&o_full[t], (nt[t] - 1), abort_p, kAtFlagCompute));
    if (ok) {
      tc_fence_after();
      row_x[half][t][tid] = l;
      pair_sync(pair);
      l = row_x[0][t][tid] + row_x[1][t][tid];
      const bool some = limit > 0;
      const float inv = some ? 1.0f / l : 0.0f;
      // the tile's Q is read: its shared memory stages the rows
      const int first = r0 + t * kRows + q4 * 32;
      uint4 v[D / 16];
#pragma unroll
      for (int b = 0; b < D / 64; ++b) {
        uint32_t o[32];
        if (nt[t]) load_quarter(O_h + 32 * b, o);
        if (!nt[t] || !some) {  // (also where 0 times a value that is not finite was added)
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) v[4 * b + c] = pack8_scaled(o + 8 * c, inv);
      }
      put_rows<D / 16>(smem + t * G::kTile + (warp & 7) * (32 * D), v,
                       P.out + static_cast<int64_t>(x.q0 + first) * P.os + h * D + half * (D / 2),
                       P.os * 2, x.lq - first);
      if (row < x.lq && half == 0)
        P.lse[static_cast<int64_t>(h) * P.S.Tq + x.q0 + row] =
            some ? (ref + log2f(l)) / kLog2e : -INFINITY;
    }
  }

  __syncthreads();  // every thread sees the final abort word
  if (*abort_p && warp == kLoadWarp && lane == 0) {
    // drain what this CTA started before its shared memory and TMEM go away
    volatile int never = 0;
    if (q_loaded) spin_wait(&q_full, 0, &never, kAtFlagDrain);
    for (int i = max(0, last_load - NS + 1); i <= last_load; ++i)
      if (!spin_wait(&kv_full[i % NS], (i / NS) & 1, &never, kAtFlagDrain)) break;
  }
  if (*abort_p && warp == kMmaWarp && mma_issued && elect_one()) {
    volatile int never = 0;
    umma_commit(&drain);
    spin_wait(&drain, 0, &never, kAtFlagDrain);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kCols);
  }
}

// head_dim 64: 128 query rows of one head, the keys 64 at a time, so that S
// and O need 128 TMEM columns and four CTAs fit an SM: with 64 columns a
// tile's products are half as long as with 128 and the chain from scores to
// probabilities to the next scores weighs twice as much; four chains at once
// hide it.  A thread owns a row (no exchange between warps).  One sequence of
// 8192, 16/16 heads, no mask: 377 us, 730 TFLOP/s, in a short burst with issue
// slots 58 % and the special-function unit 50 % busy; 465 us in a loop at the
// power limit.
struct Fwd64Geo {
  static constexpr int kD = 64;
  static constexpr int kQ = tile_bytes<kD>(), kHalf = kStep * kD * 2;  // bytes of Q; of K or V
  static constexpr int kStages = 4;
  static constexpr int kSmem = kQ + kStages * kHalf;
  static constexpr int kThreads = 32 * (4 + 2);
  static constexpr uint32_t kO = kStep, kCols = kStep + kD;
};

__global__ void __launch_bounds__(Fwd64Geo::kThreads, 4)
    packed_fwd64_tc(const __grid_constant__ FwdTc P) {
  using G = Fwd64Geo;
  constexpr int D = G::kD, NS = G::kStages, kMmaWarp = 4, kLoadWarp = 5;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t q_full, kv_full[NS], kv_empty[NS], aux, s_full, p_full, o_full, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0 && lane == 0) prefetch_maps(P);
  pdl_wait();
  // (before anything is set up: the grid covers the most tiles there could be)
  PackedTile x;
  if (!find_tile(P.S, false, blockIdx.x / P.H, kRows, x)) return;
  if (threadIdx.x == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&aux, 1);
    mbar_init(&drain, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&p_full, 4);
    mbar_init(&o_full, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_slot, G::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_release();  // (after the allocation)
  const uint32_t tmem = tmem_slot;
  volatile int* abort_p = &abort_flag;
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need the alignment asked for
    if (threadIdx.x == 0) atomicOr(&g_attn_flags, kAtFlagLoad);
    if (warp == kMmaWarp) tmem_dealloc(tmem, G::kCols);
    return;
  }
  const int h = blockIdx.x % P.H, kh = h / (P.H / P.KV), r0 = x.t * kRows;
  const int n = (key_limit(P.S, x, min(r0 + kRows, x.lq) - 1) + kStep - 1) / kStep;
  int last_load = -1;
  bool q_loaded = false, mma_issued = false;
  uint8_t* ring = smem + G::kQ;

  if (warp == kLoadWarp && n) {
    // Q, then K0 V0 K1 V1 ...
    if (lane == 0) {
      mbar_arrive_expect_tx(&q_full, G::kQ);
      tma_tile<D>(smem, &P.mq, &q_full, h * D, x.q0 + r0);
    }
    q_loaded = true;
    for (int i = 0; i < 2 * n; ++i) {
      const int s = i % NS, row = (i >> 1) * kStep;
      if (i >= NS && !warp_wait(&kv_empty[s], (i / NS) - 1, abort_p, kAtFlagLoad)) break;
      uint8_t* st = ring + s * G::kHalf;
      const CUtensorMap* map = (i & 1) ? &P.mv : &P.mk;
      // the keys behind the sequence have probability 0, their values must be
      // finite
      const bool tail = (i & 1) && row + kStep > x.lk;
      uint64_t* bar = tail ? &aux : &kv_full[s];
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, G::kHalf);
        tma_tile<D, kStep>(st, map, bar, kh * D, x.k0 + row);
      }
      if (tail) {
        __syncwarp();
        if (!tail_landed(&aux, 0, abort_p)) break;
        zero_rows<D, kStep>(st, x.lk - row);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_full[s]);
      }
      last_load = i;
    }
  } else if (warp == kMmaWarp && n) {
    auto wait = [&](uint64_t* bar, int phase) {
      return warp_wait(bar, phase, abort_p, kAtFlagMma);
    };
    auto stage = [&](int i) { return ring + (i % NS) * G::kHalf; };
    bool ok = wait(&q_full, 0);
    for (int j = 0; j <= n && ok; ++j) {
      // O += P V of the step before, then this step's S = Q K^T, which goes
      // over that P
      const int i = 2 * j;
      ok = (j == n || wait(&kv_full[i % NS], i / NS)) &&
           (j == 0 || (wait(&kv_full[(i - 1) % NS], (i - 1) / NS) && wait(&p_full, j - 1)));
      if (!ok) break;
      mma_issued = true;
      tc_fence_after();
      if (elect_one()) {
        if (j > 0) {
          mma_ay<D, kStep, kStep>(tmem + G::kO, tmem, 0, stage(i - 1), j > 1);
          umma_commit(&o_full);
          umma_commit(&kv_empty[(i - 1) % NS]);
        }
        if (j < n) {
          mma_xyt<D, kStep>(tmem, smem, stage(i));
          umma_commit(&s_full);
          umma_commit(&kv_empty[i % NS]);
        }
      }
      __syncwarp();
    }
  } else if (warp < kMmaWarp) {
    const int row = r0 + threadIdx.x;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t S_r = tmem + lanes, O_r = S_r + G::kO;
    const int limit = key_limit(P.S, x, row);
    const uint64_t c2 = f32x2_pack(P.c, P.c);
    float ref = 0.0f, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      ok = warp_wait(&s_full, j, abort_p, kAtFlagCompute);
      if (!ok) break;
      tc_fence_after();
      const int lim = limit - j * kStep;
      const bool mask = __any_sync(0xffffffffu, lim < kStep);
      auto scores = [&](int b, uint32_t* s) {  // 32 columns, read once for the maximum and again
        load_quarter(S_r + 32 * b, s);
        if (!mask) return;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (32 * b + e >= lim) s[e] = 0xff800000u;  // -inf
      };
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t s[32];
        scores(b, s);
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          m4[(e >> 1) & 3] = max_nan(max_nan(m4[(e >> 1) & 3], __uint_as_float(s[e])),
                                     __uint_as_float(s[e + 1]));
      }
      // (as in the kernel above: rows behind the sequence, the reference that
      // moves by 2^8, and NaN)
      const float mt = row < x.lq ? max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3])) * P.c
                                  : -INFINITY;
      if (j == 0) {
        ref = fmaxf(mt, kLowRef);
      } else if (__any_sync(0xffffffffu, mt > ref + 8.0f)) {
        ok = warp_wait(&o_full, j - 1, abort_p, kAtFlagCompute);
        if (!ok) break;
        tc_fence_after();
        const float next = fmaxf(ref, mt), f = ex2(ref - next);
        ref = next;
        l *= f;
        const uint64_t f2 = f32x2_pack(f, f);
#pragma unroll 1
        for (int b = 0; b < D / 16; ++b) {
          uint32_t o[16];
          tmem_ld16(O_r + 16 * b, o);
          tmem_wait_ld();
          tie16(o);
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float lo, hi;
            f32x2_unpack(f32x2_mul_rn(f32x2_pack_bits(o[e], o[e + 1]), f2), lo, hi);
            o[e] = __float_as_uint(lo);
            o[e + 1] = __float_as_uint(hi);
          }
          tmem_st16(O_r + 16 * b, o);
        }
      }
      const uint64_t r2 = f32x2_pack(-ref, -ref);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t s[32], p[16];
        scores(b, s);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t y = f32x2_fma_rn(f32x2_pack_bits(s[2 * e], s[2 * e + 1]), c2, r2);
          const uint64_t pr = e % kPolyOf < kPolyPart ? ex2_poly<false>(y) : ex2_pair(y);
          sum[e & 1] = f32x2_add_rn(sum[e & 1], pr);
          p[e] = f32x2_to_bf16x2(pr);
        }
        tmem_st16(S_r + 16 * b, p);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full);
      float a0, a1;
      f32x2_unpack(f32x2_add_rn(sum[0], sum[1]), a0, a1);
      l += a0 + a1;
      if (!(mt < INFINITY)) l = NAN;
    }
    if (ok && n) ok = warp_wait(&o_full, n - 1, abort_p, kAtFlagCompute);
    if (ok) {
      tc_fence_after();
      const bool some = limit > 0;
      const float inv = some ? 1.0f / l : 0.0f;
      // the tile's Q is read: its shared memory stages the rows
      const int first = r0 + warp * 32;
      uint4 v[D / 8];
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        uint32_t o[32];
        if (n) load_quarter(O_r + 32 * b, o);
        if (!n || !some) {  // (as above)
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) v[4 * b + c] = pack8_scaled(o + 8 * c, inv);
      }
      put_rows<D / 8>(smem + warp * (64 * D), v,
                      P.out + static_cast<int64_t>(x.q0 + first) * P.os + h * D, P.os * 2,
                      x.lq - first);
      if (row < x.lq)
        P.lse[static_cast<int64_t>(h) * P.S.Tq + x.q0 + row] =
            some ? (ref + log2f(l)) / kLog2e : -INFINITY;
    }
  }

  __syncthreads();  // every thread sees the final abort word
  if (*abort_p && warp == kLoadWarp && lane == 0) {
    // drain what this CTA started before its shared memory and TMEM go away
    volatile int never = 0;
    if (q_loaded) spin_wait(&q_full, 0, &never, kAtFlagDrain);
    for (int i = max(0, last_load - NS + 1); i <= last_load; ++i)
      if (!spin_wait(&kv_full[i % NS], (i / NS) & 1, &never, kAtFlagDrain)) break;
  }
  if (*abort_p && warp == kMmaWarp && mma_issued && elect_one()) {
    volatile int never = 0;
    umma_commit(&drain);
    spin_wait(&drain, 0, &never, kAtFlagDrain);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kCols);
  }
}

// ---------------------------------------------------------------- backward

struct BwdTc {
  CUtensorMap mq, mk, mv, mdo, mo;  // boxes of 128 rows (mk, mv in the dQ kernel: of kStep)
  const float* lse;
  float* D;     // [H, Tq]: written by the dQ kernel, read by the dK/dV kernel
  float4* part;  // shares' dK, dV sums: [key tile][KV][splits], part_size each
  uint16_t *dq, *dk, *dv;
  int64_t dqs, dks, dvs;
  PackedSeqs S;
  int H, KV;
  int splits, limit;  // the most shares of a KV group's heads; see tile_shares
  float scale, c;  // c = scale * log2(e)
};

__device__ __forceinline__ void prefetch_maps(const BwdTc& P) {
  tma_prefetch_desc(&P.mq);
  tma_prefetch_desc(&P.mk);
  tma_prefetch_desc(&P.mv);
  tma_prefetch_desc(&P.mdo);
}

// Geometry of the dK/dV kernel: the queries of a step are 128 with one CTA per
// SM, or 64 with two (head_dim 64 only: a CTA has half of TMEM).  Two rings: a
// step's last product reads Q, which is held longest and gets one stage more
// than dO.
template <int D, int CTAS>
struct KvGeo {
  static constexpr int kStep = 128 / CTAS, kParts = kStep / 32;  // queries; 32 to a thread
  static constexpr int kWarps = 4 * kParts;                      // computing warps
  static constexpr int kMmaWarp = kWarps, kLoadWarp = kWarps + 1, kPatchWarp = kWarps + 2;
  static constexpr int kThreads = 32 * (kWarps + 3);
  static constexpr int kTile = tile_bytes<D>(), kRow = kStep * D * 2;  // bytes of K, V; of Q, dO
  static constexpr int kA = D == 128 ? 3 : 6 - CTAS, kB = kA - 1;
  static constexpr int kSmem = 2 * kTile + (kA + kB) * kRow;
  static constexpr uint32_t kDp = kStep, kDv = 2 * kStep, kDk = kDv + D,  // TMEM
      kCols = 512 / CTAS;
  static constexpr int kOut = 2 * D / kParts;  // of dV's and dK's columns: a thread's
  static_assert(kDk + D <= kCols && kWarps * 64 * kOut <= (kA + kB) * kRow, "");
};

// dQ of 128 query rows of one head, the keys 64 at a time: S = Q K^T,
// dP = dO V^T, dS = P (dP - D) as bf16 over its dP, dQ += dS K.  The kernel
// also writes D = dO . O for the dK/dV kernel.
//
// Two CTAs per SM (256 TMEM columns each: dQ, S, dP), so that one's start,
// end and waits hide behind the other's products: a tile's start and end are
// about 10000 cycles of latency, as much as eight steps.  S of the next step
// is computed as soon as the threads have read this one's; its dP follows
// dQ's product, which reads dS.  16384 tokens of 32/8 heads of 128: 3080 us,
// 1070 TFLOP/s of its three products, in a loop at the power limit (products
// of 64 columns run at two thirds of the rate of 128), 2740 from rest; 8150
// tokens in 17, 28/4 heads: 145 us.
template <int D>
struct DqGeo {
  static constexpr int kTile = tile_bytes<D>();  // Q, dO, O: 128 rows
  static constexpr int kHalf = kStep * D * 2;    // K or V of a step
  static constexpr int kK = D == 128 ? 2 : 4, kV = D == 128 ? 1 : 3;  // stages
  static constexpr int kSmem = 2 * kTile + (kK + kV) * kHalf;
  static constexpr int kWarps = 8, kThreads = 32 * (kWarps + 2);
  static constexpr uint32_t kS = D, kDp = D + kStep, kCols = 256;  // TMEM: dQ, S, dP
};

template <int D>
__global__ void __launch_bounds__(DqGeo<D>::kThreads, 2)
    packed_dq_tc(const __grid_constant__ BwdTc P) {
  using G = DqGeo<D>;
  constexpr int NK = G::kK, NV = G::kV, kMmaWarp = G::kWarps, kLoadWarp = G::kWarps + 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t q_full, o_full, o_used, k_full[NK], k_empty[NK], v_full[NV], v_empty[NV], aux,
      s_full, s_free, dp_full, ds_full, done, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ float row_x[kRows];  // dO . O, exchanged between the two threads of a row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0 && lane == 0) prefetch_maps(P);
  pdl_wait();
  // (before anything is set up: the grid covers the most tiles there could be)
  PackedTile x;
  if (!find_tile(P.S, false, blockIdx.x / P.H, kRows, x)) return;
  if (threadIdx.x == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&o_full, 1);
    mbar_init(&o_used, G::kWarps);
    mbar_init(&aux, 1);
    mbar_init(&drain, 1);
    for (int i = 0; i < NK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&s_free, G::kWarps);
    mbar_init(&dp_full, 1);
    mbar_init(&ds_full, G::kWarps);
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_slot, G::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_release();  // (after the allocation)
  const uint32_t tmem = tmem_slot;
  volatile int* abort_p = &abort_flag;
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need the alignment asked for
    if (threadIdx.x == 0) atomicOr(&g_attn_flags, kAtFlagLoad);
    if (warp == kMmaWarp) tmem_dealloc(tmem, G::kCols);
    return;
  }
  const int h = blockIdx.x % P.H, kh = h / (P.H / P.KV), r0 = x.t * kRows;
  const int n = (key_limit(P.S, x, min(r0 + kRows, x.lq) - 1) + kStep - 1) / kStep;
  int last_k = -1, last_v = -1;
  bool q_loaded = false, mma_issued = false;
  uint8_t* const Q = smem;
  uint8_t* const dO = smem + G::kTile;
  uint8_t* const Ks = smem + 2 * G::kTile;
  uint8_t* const Vs = Ks + NK * G::kHalf;
  uint8_t* const O = Vs - G::kHalf;  // the last K stage and the first V stage, before their use

  if (warp == kLoadWarp && n) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&q_full, 2 * G::kTile);
      tma_tile<D>(Q, &P.mq, &q_full, h * D, x.q0 + r0);
      tma_tile<D>(dO, &P.mdo, &q_full, h * D, x.q0 + r0);
      mbar_arrive_expect_tx(&o_full, G::kTile);
      tma_tile<D>(O, &P.mo, &o_full, h * D, x.q0 + r0);
    }
    q_loaded = true;
    for (int i = 0; i < n; ++i) {
      const int s = i % NK, v = i % NV, row = i * kStep;
      if (i >= NK && !warp_wait(&k_empty[s], (i / NK) - 1, abort_p, kAtFlagLoad)) break;
      const bool tail = row + kStep > x.lk;  // dS is 0 there; K must be finite
      uint64_t* bar = tail ? &aux : &k_full[s];
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, G::kHalf);
        tma_tile<D, kStep>(Ks + s * G::kHalf, &P.mk, bar, kh * D, x.k0 + row);
      }
      if (tail) {
        __syncwarp();
        if (!tail_landed(&aux, 0, abort_p)) break;
        zero_rows<D, kStep>(Ks + s * G::kHalf, x.lk - row);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[s]);
      }
      last_k = i;
      // O lies in the last K stage (used from i = NK - 1 on) and the first V stage
      if (i == 0 && !warp_wait(&o_used, 0, abort_p, kAtFlagLoad)) break;
      if (i >= NV && !warp_wait(&v_empty[v], (i / NV) - 1, abort_p, kAtFlagLoad)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&v_full[v], G::kHalf);
        tma_tile<D, kStep>(Vs + v * G::kHalf, &P.mv, &v_full[v], kh * D, x.k0 + row);
      }
      last_v = i;
    }
  } else if (warp == kMmaWarp && n) {
    auto wait = [&](uint64_t* bar, int phase) {
      return warp_wait(bar, phase, abort_p, kAtFlagMma);
    };
    auto scores = [&](int i) {  // S = Q K^T
      if (!wait(&k_full[i % NK], i / NK)) return false;
      mma_issued = true;
      tc_fence_after();
      if (elect_one()) {
        mma_xyt<D, kStep>(tmem + G::kS, Q, Ks + (i % NK) * G::kHalf);
        umma_commit(&s_full);
      }
      __syncwarp();
      return true;
    };
    bool ok = wait(&q_full, 0) && scores(0);
    for (int i = 0; i < n && ok; ++i) {
      // dQ += dS K of the step before, then this step's dP = dO V^T
      ok = wait(&v_full[i % NV], i / NV) && (i == 0 || wait(&ds_full, i - 1));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        if (i > 0) {
          mma_ay<D, 32, kStep>(tmem, tmem + G::kDp, 32, Ks + ((i - 1) % NK) * G::kHalf, i > 1);
          umma_commit(&k_empty[(i - 1) % NK]);
        }
        mma_xyt<D, kStep>(tmem + G::kDp, dO, Vs + (i % NV) * G::kHalf);
        umma_commit(&dp_full);
        umma_commit(&v_empty[i % NV]);
      }
      __syncwarp();
      if (i + 1 < n) ok = wait(&s_free, i) && scores(i + 1);
    }
    ok = ok && wait(&ds_full, n - 1);
    tc_fence_after();
    if (ok && elect_one()) {
      mma_ay<D, 32, kStep>(tmem, tmem + G::kDp, 32, Ks + ((n - 1) % NK) * G::kHalf, n > 1);
      umma_commit(&done);
    }
    __syncwarp();
  } else if (warp < G::kWarps) {
    // a row per two threads: half of its columns at the start and the end, 32
    // of each step's keys in between
    const int part = warp >> 2, q4 = warp & 3, tid = q4 * 32 + lane, row = r0 + tid;
    const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
    const bool in = row < x.lq;
    const int64_t at = static_cast<int64_t>(h) * P.S.Tq + x.q0 + row;
    const float lse = in ? P.lse[at] : 0.0f;
    bool ok = true;
    float Dr = 0.0f;
    if (n) {
      ok = warp_wait(&q_full, 0, abort_p, kAtFlagCompute) &&
           warp_wait(&o_full, 0, abort_p, kAtFlagCompute);
#pragma unroll 2
      for (int i = 0; i < D / 16; ++i) {  // 16-byte pieces of the row in its swizzled boxes
        const int piece = part * (D / 16) + i;
        const int off = (piece >> 3) * kBoxBytes + tid * 128 + (((piece & 7) ^ (tid & 7)) * 16);
        const uint4 a = *reinterpret_cast<const uint4*>(dO + off);
        const uint4 b = *reinterpret_cast<const uint4*>(O + off);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          Dr = __fmaf_rn(__uint_as_float(u[e] << 16), __uint_as_float(v[e] << 16), Dr);
          Dr = __fmaf_rn(__uint_as_float(u[e] & 0xFFFF0000u), __uint_as_float(v[e] & 0xFFFF0000u),
                         Dr);
        }
      }
    }
    // the halves, added in one order (every computing warp comes here)
    if (part == 1) row_x[tid] = Dr;
    bar_compute<32 * G::kWarps>();
    if (part == 0) row_x[tid] = Dr + row_x[tid];
    bar_compute<32 * G::kWarps>();
    Dr = row_x[tid];
    if (n && lane == 0) mbar_arrive(&o_used);  // (after the barriers: O is read)
    if (in && part == 0) P.D[at] = Dr;
    const int limit = in ? key_limit(P.S, x, row) : 0;
    const float lse2 = lse * kLog2e;
    const uint64_t c2 = f32x2_pack(P.c, P.c), l2 = f32x2_pack(-lse2, -lse2),
                   d2 = f32x2_pack(-Dr, -Dr);
    const uint32_t S_p = tmem + G::kS + part * 32 + lanes, dP_p = S_p + kStep;
    for (int i = 0; i < n && ok; ++i) {
      const int lim = limit - i * kStep - part * 32;
      ok = warp_wait(&s_full, i, abort_p, kAtFlagCompute);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[32];
      load_quarter(S_p, s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free);
      uint64_t p[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        p[e] = ex2_pair(f32x2_fma_rn(f32x2_pack_bits(s[2 * e], s[2 * e + 1]), c2, l2));
      ok = warp_wait(&dp_full, i, abort_p, kAtFlagCompute);
      if (!ok) break;
      tc_fence_after();
      load_quarter(dP_p, s);
      uint32_t ds[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        ds[e] = f32x2_to_bf16x2(f32x2_mul_rn(
            p[e], f32x2_add_rn(f32x2_pack_bits(s[2 * e], s[2 * e + 1]), d2)));
      if (__any_sync(0xffffffffu, lim < 32)) {  // select: what is masked may be infinite or NaN
#pragma unroll
        for (int e = 0; e < 16; ++e)
          ds[e] &= (2 * e < lim ? 0x0000FFFFu : 0u) | (2 * e + 1 < lim ? 0xFFFF0000u : 0u);
      }
      tmem_st16(dP_p, ds);  // over the first half of this thread's columns
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_full);
    }
    if (ok && n) ok = warp_wait(&done, 0, abort_p, kAtFlagCompute);
    if (ok) {
      tc_fence_after();
      // all products are done: Q's shared memory stages the rows
      const int first = r0 + q4 * 32;
      uint4 v[D / 16];
#pragma unroll
      for (int b = 0; b < D / 64; ++b) {
        uint32_t o[32];
        if (n) load_quarter(tmem + part * (D / 2) + 32 * b + lanes, o);
        if (limit <= 0) {  // no key (also where 0 times a key that is not finite was added)
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) v[4 * b + c] = pack8_scaled(o + 8 * c, P.scale);
      }
      put_rows<D / 16>(Q + warp * (32 * D), v,
                       P.dq + static_cast<int64_t>(x.q0 + first) * P.dqs + h * D + part * (D / 2),
                       P.dqs * 2, x.lq - first);
    }
  }

  __syncthreads();  // every thread sees the final abort word
  if (*abort_p && warp == kLoadWarp && lane == 0) {
    // drain what this CTA started before its shared memory and TMEM go away
    volatile int never = 0;
    if (q_loaded) {
      spin_wait(&q_full, 0, &never, kAtFlagDrain);
      spin_wait(&o_full, 0, &never, kAtFlagDrain);
    }
    for (int i = max(0, last_k - NK + 1); i <= last_k; ++i)
      if (!spin_wait(&k_full[i % NK], (i / NK) & 1, &never, kAtFlagDrain)) break;
    for (int i = max(0, last_v - NV + 1); i <= last_v; ++i)
      if (!spin_wait(&v_full[i % NV], (i / NV) & 1, &never, kAtFlagDrain)) break;
  }
  if (*abort_p && warp == kMmaWarp && mma_issued && elect_one()) {
    volatile int never = 0;
    umma_commit(&drain);
    spin_wait(&drain, 0, &never, kAtFlagDrain);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kCols);
  }
}

// the first query that sees keys of tile x
__device__ __forceinline__ int first_query(const PackedSeqs& S, const PackedTile& x) {
  return S.causal ? max(x.t * kRows - (x.lk - x.lq), 0) : 0;
}

// Shares that a key tile's query heads are cut into: so many that none has
// more than `limit` query tiles to go through, within the grid's `splits`.  A
// long sequence among short ones would otherwise keep one CTA busy long after
// the others (8150 tokens in 17 sequences, the longest 1855: 168 us of 350).
__device__ __forceinline__ int tile_shares(const BwdTc& P, const PackedTile& x) {
  const int all = max((x.lq + kRows - 1) / kRows - first_query(P.S, x) / kRows, 0) * (P.H / P.KV);
  return min(max((all + P.limit - 1) / P.limit, 1), P.splits);
}

// A share's fp32 sums of a tile and KV head, as float4: dV and dK of 128 keys.
template <int D>
__host__ __device__ constexpr int64_t part_size() {
  return 2 * kRows * D / 4;
}
template <int D>
__device__ __forceinline__ int64_t part_at(const BwdTc& P, int slot, int kh, int split) {
  return ((static_cast<int64_t>(slot) * P.KV + kh) * P.splits + split) * part_size<D>();
}

// dK, dV of 128 keys of one KV head, over one share of the group's query
// heads and, in each, the query tiles that see the keys, in order.  The
// scores are computed transposed (a thread owns a key row, 32 of the step's
// queries), so that P^T and dS^T, written as bf16 over the scores they came
// from, are the tensor-memory operands of dV += P^T dO and dK += dS^T Q.
// TMEM: S^T, dP^T, dV, dK.  16384 tokens of 32/8 heads of 128: 3520 us, 1250
// TFLOP/s of its four products, in a loop at the power limit, 0.90 of a library
// product's rate under it (3340 us from rest); 8150 tokens in 17, 28/4 heads:
// 149 us, 1.7 us a step and 9 us of a CTA's start and end.  While the threads
// compute P^T the tensor cores run the tile before's dK product and this
// tile's dP^T; while they compute dS^T, dV and the next S^T.
template <int D, int CTAS>
__global__ void __launch_bounds__(KvGeo<D, CTAS>::kThreads, CTAS)
    packed_dkdv_tc(const __grid_constant__ BwdTc P) {
  using G = KvGeo<D, CTAS>;
  constexpr int NA = G::kA, NB = G::kB, kStep = G::kStep;  // stages of Q, of dO; queries of a step
  constexpr int kMmaWarp = G::kMmaWarp, kLoadWarp = G::kLoadWarp, kPatchWarp = G::kPatchWarp;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t kv_full, q_full[NA], q_raw[NA], q_empty[NA], ld_full[2], do_full[NB],
      do_raw[NB], do_empty[NB], s_full, dp_full, p_full, ds_full, done, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ __align__(16) float nlse[2][kStep], nD[2][kStep];  // -lse log2(e), -D
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = P.KV * P.splits, kh = blockIdx.x % per / P.splits,
            split = blockIdx.x % per % P.splits;
  if (warp == 0 && lane == 0) prefetch_maps(P);
  // The CTA starts while the dQ kernel ends.  That kernel let this one in after
  // its own wait, so the call's inputs stand; only D is waited for (every CTA
  // waits, so that this kernel never ends before that one).  It holds TMEM
  // meanwhile, which no dQ CTA waits for: they have theirs before they let it in.
  // (before anything is set up: the grid covers the most tiles and shares)
  PackedTile x;
  const bool found = find_tile<true>(P.S, true, blockIdx.x / per, kRows, x);
  const int shares = found ? tile_shares(P, x) : 0;
  if (split >= shares) {
    pdl_wait();
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(&kv_full, 1);
    mbar_init(&drain, 1);
    for (int i = 0; i < NA; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_raw[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&ld_full[i], 32);
    for (int i = 0; i < NB; ++i) {
      mbar_init(&do_full[i], 1);
      mbar_init(&do_raw[i], 1);
      mbar_init(&do_empty[i], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&dp_full, 1);
    mbar_init(&done, 1);
    mbar_init(&p_full, G::kWarps);
    mbar_init(&ds_full, G::kWarps);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_slot, G::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_release();  // (after the allocation)
  // with all 512 columns this CTA's: a base known at compile time
  const uint32_t tmem = G::kCols == 512 ? 0u : tmem_slot;
  volatile int* abort_p = &abort_flag;
  // the swizzled tiles need the alignment asked for
  if ((smem_u32(smem) & 1023u) || tmem_slot != tmem) {
    if (threadIdx.x == 0) atomicOr(&g_attn_flags, kAtFlagLoad);
    if (warp == kMmaWarp) tmem_dealloc(tmem_slot, G::kCols);
    pdl_wait();
    return;
  }

  const int grp = P.H / P.KV;
  const int h0 = kh * grp + grp * split / shares, h1 = kh * grp + grp * (split + 1) / shares;
  const int c0 = x.t * kRows;
  const int qt0 = first_query(P.S, x) / kStep;  // (in steps)
  const int per_head = max((x.lq + kStep - 1) / kStep - qt0, 0);
  const int n = per_head * (h1 - h0);
  int last_a = -1, last_b = -1;
  bool kv_loaded = false, mma_issued = false;
  uint8_t* ring = smem + 2 * G::kTile;

  if (warp == kLoadWarp && n) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&kv_full, 2 * G::kTile);
      tma_tile<D>(smem, &P.mk, &kv_full, kh * D, x.k0 + c0);
      tma_tile<D>(smem + G::kTile, &P.mv, &kv_full, kh * D, x.k0 + c0);
    }
    kv_loaded = true;
    int h = h0, qt = qt0;
    for (int i = 0; i < n; ++i) {
      const int s = i % NA, v = i % NB, row = qt * kStep;
      const bool tail = row + kStep > x.lq;  // goes through the patching warp
      auto load = [&](uint8_t* st, const CUtensorMap* map, uint64_t* bar) {
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, G::kRow);
          tma_tile<D, kStep>(st, map, bar, h * D, x.q0 + row);
        }
      };
      if (i >= NA && !warp_wait(&q_empty[s], (i / NA) - 1, abort_p, kAtFlagLoad)) break;
      load(ring + s * G::kRow, &P.mq, tail ? &q_raw[s] : &q_full[s]);
      last_a = i;
      if (i < NB) {
        load(ring + (NA + v) * G::kRow, &P.mdo, tail ? &do_raw[v] : &do_full[v]);
        last_b = i;
      }
      if (i == 0) pdl_wait();  // D
      float a[kStep / 32], b[kStep / 32];
#pragma unroll
      for (int e = 0; e < kStep / 32; ++e) {
        const int j = lane + 32 * e;
        const int64_t at = static_cast<int64_t>(h) * P.S.Tq + x.q0 + row + j;
        a[e] = row + j < x.lq ? P.lse[at] * -kLog2e : 0.0f;
        b[e] = row + j < x.lq ? -P.D[at] : 0.0f;
      }
      // their slot was last read for tile i - 2, before its dK product
      if (i >= 2 && !warp_wait(&q_empty[(i - 2) % NA], (i - 2) / NA, abort_p, kAtFlagLoad)) break;
#pragma unroll
      for (int e = 0; e < kStep / 32; ++e) {
        nlse[i & 1][lane + 32 * e] = a[e];
        nD[i & 1][lane + 32 * e] = b[e];
      }
      mbar_arrive(&ld_full[i & 1]);
      if (i >= NB) {
        if (!warp_wait(&do_empty[v], (i / NB) - 1, abort_p, kAtFlagLoad)) break;
        load(ring + (NA + v) * G::kRow, &P.mdo, tail ? &do_raw[v] : &do_full[v]);
        last_b = i;
      }
      if (++qt == qt0 + per_head) {
        qt = qt0;
        ++h;
      }
    }
  } else if (warp == kPatchWarp && n) {
    // The rows behind the sequence in each head's last query tile: P and dS
    // are 0 there, Q and dO must be finite.  (A warp of its own: the loader
    // would wait for every such tile instead of running ahead, 3.7 us a tile
    // where each is one.)
    const int row = (qt0 + per_head - 1) * kStep;
    uint32_t q_phase = 0, do_phase = 0;  // a bit per stage
    if (row + kStep > x.lq) {
      for (int i = per_head - 1; i < n; i += per_head) {
        const int s = i % NA, v = i % NB;
        if (!tail_landed(&q_raw[s], (q_phase >> s) & 1, abort_p)) break;
        q_phase ^= 1u << s;
        zero_rows<D, kStep>(ring + s * G::kRow, x.lq - row);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[s]);
        if (!tail_landed(&do_raw[v], (do_phase >> v) & 1, abort_p)) break;
        do_phase ^= 1u << v;
        zero_rows<D, kStep>(ring + (NA + v) * G::kRow, x.lq - row);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&do_full[v]);
      }
    }
  } else if (warp == kMmaWarp && n) {
    // As in the forward, conditions are tested before the products that
    // precede their use.
    auto wait = [&](uint64_t* bar, int phase) {
      return warp_wait(bar, phase, abort_p, kAtFlagMma);
    };
    auto Q = [&](int i) { return ring + (i % NA) * G::kRow; };
    auto dO = [&](int i) { return ring + (NA + i % NB) * G::kRow; };
    auto scores = [&](int i) {  // S^T = K Q^T (one thread)
      mma_xyt<D, kStep>(tmem, smem, Q(i));
      umma_commit(&s_full);
    };
    auto dprobs = [&](int i) {  // dP^T = V dO^T
      mma_xyt<D, kStep>(tmem + G::kDp, smem + G::kTile, dO(i));
      umma_commit(&dp_full);
    };
    bool ok = wait(&kv_full, 0) && wait(&q_full[0], 0) && wait(&do_full[0], 0);
    if (ok) {
      mma_issued = true;
      if (elect_one()) {
        scores(0);
        dprobs(0);
      }
      __syncwarp();
    }
    bool q_in = false;
    for (int i = 0; i < n && ok; ++i) {
      const bool more = i + 1 < n;
      ok = (!more || q_in || wait(&q_full[(i + 1) % NA], (i + 1) / NA)) && wait(&p_full, i);
      if (!ok) break;
      const bool do_in = more && warp_test(&do_full[(i + 1) % NB], (i + 1) / NB);
      tc_fence_after();
      if (elect_one()) {
        mma_ay<D, 32, kStep>(tmem + G::kDv, tmem, 32, dO(i), i > 0);  // dV += P^T dO
        umma_commit(&do_empty[i % NB]);
        if (more) scores(i + 1);
      }
      __syncwarp();
      ok = (!more || do_in || wait(&do_full[(i + 1) % NB], (i + 1) / NB)) && wait(&ds_full, i);
      if (!ok) break;
      q_in = i + 2 < n && warp_test(&q_full[(i + 2) % NA], (i + 2) / NA);
      tc_fence_after();
      if (elect_one()) {
        mma_ay<D, 32, kStep>(tmem + G::kDk, tmem + G::kDp, 32, Q(i), i > 0);  // dK += dS^T Q
        umma_commit(&q_empty[i % NA]);
        if (more) dprobs(i + 1);
      }
      __syncwarp();
    }
    if (ok && elect_one()) umma_commit(&done);
    __syncwarp();
  } else if (warp < G::kWarps) {
    const int part = warp >> 2, q4 = warp & 3, key = c0 + q4 * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t S_p = tmem + part * 32 + lanes, dP_p = S_p + G::kDp;
    const bool in = key < x.lk;
    // query rows of the sequence that see this key: [first, lq)
    const int first = in ? (P.S.causal ? max(key - (x.lk - x.lq), 0) : 0) : x.lq;
    const uint64_t c2 = f32x2_pack(P.c, P.c);
    bool ok = true;
    int qt = qt0;
    for (int i = 0; i < n; ++i) {
      const int s = i & 1;
      // bit b of keep: query b of this thread's 32 sees the key
      const int lo = first - qt * kStep - part * 32, hi = x.lq - qt * kStep - part * 32;
      const uint32_t keep = (hi >= 32 ? ~0u : hi > 0 ? (1u << hi) - 1 : 0u) &
                            (lo <= 0 ? ~0u : lo < 32 ? ~0u << lo : 0u);
      const bool mask = __any_sync(0xffffffffu, keep != ~0u);
      if (++qt == qt0 + per_head) qt = qt0;
      ok = warp_wait(&ld_full[s], i >> 1, abort_p, kAtFlagCompute) &&
           warp_wait(&s_full, i, abort_p, kAtFlagCompute);
      if (!ok) break;
      tc_fence_after();
      uint32_t v[32];
      load_quarter(S_p, v);
      uint64_t p[16];
      uint32_t w[16];
      const ulonglong2* ls = reinterpret_cast<const ulonglong2*>(nlse[s] + part * 32);
      auto drop = [&] {  // select: what is masked may be infinite or NaN
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] &= ((keep >> (2 * e)) & 1 ? 0x0000FFFFu : 0u) |
                  ((keep >> (2 * e)) & 2 ? 0xFFFF0000u : 0u);
      };
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const ulonglong2 l4 = ls[e / 2];
        const uint64_t y0 = f32x2_fma_rn(f32x2_pack_bits(v[2 * e], v[2 * e + 1]), c2, l4.x);
        const uint64_t y1 = f32x2_fma_rn(f32x2_pack_bits(v[2 * e + 2], v[2 * e + 3]), c2, l4.y);
        p[e] = e % kPolyOf < kPolyPart ? ex2_poly<true>(y0) : ex2_pair(y0);
        p[e + 1] = (e + 1) % kPolyOf < kPolyPart ? ex2_poly<true>(y1) : ex2_pair(y1);
        w[e] = f32x2_to_bf16x2(p[e]);
        w[e + 1] = f32x2_to_bf16x2(p[e + 1]);
      }
      if (mask) drop();
      tmem_st16(S_p, w);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full);
      ok = warp_wait(&dp_full, i, abort_p, kAtFlagCompute);
      if (!ok) break;
      tc_fence_after();
      load_quarter(dP_p, v);
      const ulonglong2* ds = reinterpret_cast<const ulonglong2*>(nD[s] + part * 32);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const ulonglong2 d4 = ds[e];
        w[2 * e] = f32x2_to_bf16x2(f32x2_mul_rn(
            p[2 * e], f32x2_add_rn(f32x2_pack_bits(v[4 * e], v[4 * e + 1]), d4.x)));
        w[2 * e + 1] = f32x2_to_bf16x2(f32x2_mul_rn(
            p[2 * e + 1], f32x2_add_rn(f32x2_pack_bits(v[4 * e + 2], v[4 * e + 3]), d4.y)));
      }
      if (mask) drop();
      tmem_st16(dP_p, w);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_full);
    }
    if (ok && n) ok = warp_wait(&done, 0, abort_p, kAtFlagCompute);
    if (ok) {
      tc_fence_after();
      // half of the warps write dV, half dK
      const int which = part / (G::kParts / 2), col = part % (G::kParts / 2) * G::kOut;  // 1: dK
      const uint32_t src = tmem + G::kDv + which * D + col + lanes;
      const int first = c0 + q4 * 32;
      float4* share =
          P.part + part_at<D>(P, blockIdx.x / per, kh, split) + warp * (8 * G::kOut) + lane;
      uint4 v[G::kOut / 8];
#pragma unroll
      for (int b = 0; b < G::kOut / 32; ++b) {
        uint32_t o[32];
        if (n) {
          load_quarter(src + 32 * b, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (shares > 1) {  // in the threads' order, which packed_kv_reduce shares
#pragma unroll
          for (int c = 0; c < 8; ++c)
            share[(8 * b + c) * 32] =
                make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                            __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            v[4 * b + c] = pack8_scaled(o + 8 * c, which ? P.scale : 1.0f);
        }
      }
      if (shares == 1) {  // all products are done: the ring stages the rows
        const int64_t pitch = which ? P.dks : P.dvs;
        put_rows<G::kOut / 8>(ring + warp * (64 * G::kOut), v,
                         (which ? P.dk : P.dv) + (x.k0 + first) * pitch + kh * D + col, pitch * 2,
                         x.lk - first);
      }
    }
  }

  if (warp == kLoadWarp) pdl_wait();  // (a tile that no query sees has not waited)
  __syncthreads();
  if (*abort_p && warp == kLoadWarp && lane == 0) {
    volatile int never = 0;
    if (kv_loaded) spin_wait(&kv_full, 0, &never, kAtFlagDrain);
    for (int i = max(0, last_a - NA + 1); i <= last_a; ++i)
      if (!spin_wait(&q_full[i % NA], (i / NA) & 1, &never, kAtFlagDrain)) break;
    for (int i = max(0, last_b - NB + 1); i <= last_b; ++i)
      if (!spin_wait(&do_full[i % NB], (i / NB) & 1, &never, kAtFlagDrain)) break;
  }
  if (*abort_p && warp == kMmaWarp && mma_issued && elect_one()) {
    volatile int never = 0;
    umma_commit(&drain);
    spin_wait(&drain, 0, &never, kAtFlagDrain);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kCols);
  }
}

// dK, dV of the key tiles with several shares, which are added in order.  A
// step takes 128 rows of 32 columns, what four warps of the kernel above wrote
// in one step; a thread takes eight columns of a row and up to four shares at
// once, so that many loads are in flight (it is bound by their latency).
// gridDim.y CTAs share a tile's steps: one each if the tiles are few, but no
// more than the device holds at once, since many tiles may have one share and
// no work here.  With a whole tile and KV head per CTA the backward of 512
// tokens (28/4 heads) took 40.0 us for 33.4, of 1024 tokens 65.0 for 57.9, of
// 8150 in 17 sequences 306 for 309.
template <int D, int CTAS>
__global__ void __launch_bounds__(kReduceThreads)
    packed_kv_reduce(const __grid_constant__ BwdTc P) {
  __shared__ __align__(16) uint4 stage[4][32][4];
  constexpr int kParts = KvGeo<D, CTAS>::kParts, kOut = KvGeo<D, CTAS>::kOut;
  constexpr int kSteps = kParts * (kOut / 32);  // steps of a KV head
  PackedTile x;
  const int slot = blockIdx.x;
  // (the lengths are an input, as in the kernel above)
  const bool found = find_tile<true>(P.S, true, slot, kRows, x);
  const int shares = found ? tile_shares(P, x) : 1;
  pdl_wait_then_release();
  if (shares == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q4 = warp >> 2, piece = warp & 3;
  const int r = piece * 8 + (lane >> 2), c = lane & 3, row = x.t * kRows + q4 * 32 + r;
  for (int u = blockIdx.y; u < P.KV * kSteps; u += gridDim.y) {
    const int kh = u / kSteps, part = u % kSteps / (kOut / 32), b = u % (kOut / 32),
              which = part / (kParts / 2);
    const float4* p = P.part + part_at<D>(P, slot, kh, 0) + (part * 4 + q4) * (8 * kOut) +
                      (8 * b + 2 * piece) * 32 + lane;
    float4 sum[2] = {};
    for (int s = 0; s < shares; s += 4) {  // four shares' loads at once
      float4 y[4][2];
#pragma unroll
      for (int e = 0; e < 4; ++e, p += part_size<D>())
        if (s + e < shares) y[e][0] = p[0], y[e][1] = p[32];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (s + e >= shares) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sum[i].x += y[e][i].x, sum[i].y += y[e][i].y;
          sum[i].z += y[e][i].z, sum[i].w += y[e][i].w;
        }
      }
    }
    // through shared memory: whole row segments per store
    stage[q4][lane][piece ^ ((lane >> 1) & 3)] =
        pack8_scaled(reinterpret_cast<const uint32_t*>(sum), which ? P.scale : 1.0f);
    __syncthreads();
    const int64_t pitch = which ? P.dks : P.dvs;
    if (row < x.lk)
      *reinterpret_cast<uint4*>((which ? P.dk : P.dv) + (x.k0 + row) * pitch + kh * D +
                                part % (kParts / 2) * kOut + 32 * b + 8 * c) =
          stage[q4][r][c ^ ((r >> 1) & 3)];
    __syncthreads();
  }
}

// Raise a kernel's dynamic shared memory limit, once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

bool map_rows(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t stride,
              int box = kRows) {
  return encode_tma_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, cols, rows, stride * 2, 64, box,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

// The host knows the sequences' number and tokens, not their lengths: this and
// the rules below go by the mean.  One of 8000 tokens among 40 of 50 takes the
// kernels for short ones: 446 us forward and 1469 backward (28/4 heads of 128,
// causal), the two parts alone 410 + 33 and 1340 + 96.
int64_t most_tiles(int64_t T, int n_seq, int rows) {
  return T / rows + std::min<int64_t>(n_seq, T);
}

template <int D, int NQ>
cudaError_t fwd_tc(const FwdTc& P, cudaStream_t st) {
  using G = FwdGeo<D, NQ>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(packed_fwd_tc<D, NQ>, G::kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = most_tiles(P.S.Tq, P.S.n_seq, NQ * kRows) * P.H;
  return launch_pdl(packed_fwd_tc<D, NQ>, dim3(static_cast<unsigned>(grid)), dim3(G::kThreads),
                    G::kSmem, st, P);
}

cudaError_t fwd64_tc(const FwdTc& P, cudaStream_t st) {
  using G = Fwd64Geo;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(packed_fwd64_tc, G::kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = most_tiles(P.S.Tq, P.S.n_seq, kRows) * P.H;
  return launch_pdl(packed_fwd64_tc, dim3(static_cast<unsigned>(grid)), dim3(G::kThreads),
                    G::kSmem, st, P);
}

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// The most shares of a KV group's query heads: with four CTAs per SM and more
// the order of the tiles (longest first) evens them out, below that up to
// twice as many as would fill them.
int head_splits(int64_t Tk, int n_seq, int H, int KV) {
  const int64_t tiles = most_tiles(Tk, n_seq, kRows) * KV, full = 4 * sm_count();
  if (tiles >= full) return 1;
  return static_cast<int>(std::min<int64_t>(H / KV, 2 * ((full + tiles - 1) / tiles)));
}

// Query tiles per share: an SM's part of them all, were the sequences equal,
// and three more, which cost about as much as a share's start and end.
int share_limit(const hsnf4_packed_attention& a) {
  const int64_t mean = (a.Tq / a.n_seq + kRows - 1) / kRows, tiles = (a.Tk + kRows - 1) / kRows;
  const int64_t all = a.H * tiles * (a.causal ? mean + 1 : 2 * mean) / 2;
  return static_cast<int>(std::min<int64_t>(all / sm_count() + 3, 1 << 30));
}

// Whether the key tiles of all sequences come in the order of their work: where
// there are few per SM (so few that heads are shared out), the sequences have
// three tiles and more on average, and one lane of the search holds four of
// them at most.  28/4 heads, causal, in turn against sorted: 16 sequences of
// 512 tokens 203 / 183 us, 16 of 384 147 / 135, 8150 tokens in 17 311 / 299,
// 16 of 256 93 / 95; 25167 tokens in 20, 32/8 heads, 1414 / 1486 (their
// queries no longer stay in the L2 from tile to tile of a sequence).
bool sort_tiles(int64_t Tk, int n_seq, int splits) {
  return splits > 1 && n_seq > 1 && n_seq <= 128 && Tk >= 3 * kRows * static_cast<int64_t>(n_seq);
}

// The dK/dV kernel and the sum of its shares, after the dQ kernel with the
// same parameters.
template <int D, int CTAS>
cudaError_t kv_tc(const hsnf4_packed_attention& a, const PackedBwd& b, BwdTc& P, cudaStream_t st) {
  using G = KvGeo<D, CTAS>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(packed_dkdv_tc<D, CTAS>, G::kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t wq = static_cast<int64_t>(a.H) * D, wk = static_cast<int64_t>(a.KV) * D;
  if (!map_rows(&P.mk, a.k, wk, a.Tk, a.k_stride) ||
      !map_rows(&P.mv, a.v, wk, a.Tk, a.v_stride) ||
      !map_rows(&P.mq, a.q, wq, a.Tq, a.q_stride, G::kStep) ||
      !map_rows(&P.mdo, b.dout, wq, a.Tq, b.do_stride, G::kStep))
    return cudaErrorInvalidValue;
  const int64_t tiles = most_tiles(a.Tk, a.n_seq, kRows);
  e = launch_pdl(packed_dkdv_tc<D, CTAS>, dim3(static_cast<unsigned>(tiles * a.KV * P.splits)),
                 dim3(G::kThreads), G::kSmem, st, P);
  if (e != cudaSuccess || P.splits == 1) return e;
  const int64_t steps = a.KV * G::kParts * (G::kOut / 32);
  const int64_t ctas = sm_count() * (2048 / kReduceThreads);
  const int64_t ways = std::min(std::max<int64_t>(ctas / tiles, 1), steps);
  return launch_pdl(packed_kv_reduce<D, CTAS>,
                    dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(ways)),
                    dim3(kReduceThreads), 0, st, P);
}

// Whether two dK/dV CTAs share an SM (head_dim 64): where four and more come
// per SM, or two of sequences of about a tile, and the sequences are not long.
// One hides the other's start, end and waits, but each step takes half as many
// queries.  One CTA per SM against two, the whole backward, 16/16 heads, no
// mask: 64 sequences of 64 tokens 78 / 51 us, 23 ragged ones (4100 tokens) 71
// / 62, 16 of 512 129 / 114; 28/4 heads, causal: 64 of 64 93 / 77, 16 of 512
// 144 / 161, one of 1024 45 / 57, 25167 tokens in 20 823 / 877.
bool two_ctas(const hsnf4_packed_attention& a) {
  const int64_t ctas = most_tiles(a.Tk, a.n_seq, kRows) * a.KV, mean = a.Tk / a.n_seq;
  return mean < 1024 && ctas >= (mean <= kRows ? 2 : 4) * sm_count();
}

template <int D>
cudaError_t bwd_tc(const hsnf4_packed_attention& a, const PackedBwd& b, void* ws,
                   cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  BwdTc P;
  memset(&P, 0, sizeof P);
  const int64_t wq = static_cast<int64_t>(a.H) * D, wk = static_cast<int64_t>(a.KV) * D;
  if (!map_rows(&P.mk, a.k, wk, a.Tk, a.k_stride, kStep) ||
      !map_rows(&P.mv, a.v, wk, a.Tk, a.v_stride, kStep) ||
      !map_rows(&P.mq, a.q, wq, a.Tq, a.q_stride) ||
      !map_rows(&P.mdo, b.dout, wq, a.Tq, b.do_stride) ||
      !map_rows(&P.mo, b.o, wq, a.Tq, b.o_stride))
    return cudaErrorInvalidValue;
  P.lse = b.lse;
  P.D = static_cast<float*>(ws);
  P.part = reinterpret_cast<float4*>(static_cast<uint8_t*>(ws) +
                                    round_up(static_cast<size_t>(a.H) * a.Tq * 4, 256));
  P.dq = static_cast<uint16_t*>(b.dq);
  P.dk = static_cast<uint16_t*>(b.dk);
  P.dv = static_cast<uint16_t*>(b.dv);
  P.dqs = b.dq_stride;
  P.dks = b.dk_stride;
  P.dvs = b.dv_stride;
  P.S = {a.cu_q, a.cu_k, static_cast<int>(a.Tq), static_cast<int>(a.Tk), a.n_seq, a.causal, 0};
  P.H = a.H;
  P.KV = a.KV;
  P.splits = head_splits(a.Tk, a.n_seq, a.H, a.KV);
  P.S.sorted = sort_tiles(a.Tk, a.n_seq, P.splits);
  P.limit = share_limit(a);
  P.scale = a.scale;
  P.c = a.scale * kLog2e;
  cudaError_t e = allow_smem(packed_dq_tc<D>, DqGeo<D>::kSmem, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(packed_dq_tc<D>,
                 dim3(static_cast<unsigned>(most_tiles(a.Tq, a.n_seq, kRows) * a.H)),
                 dim3(DqGeo<D>::kThreads), DqGeo<D>::kSmem, st, P);
  if (e != cudaSuccess) return e;
  if constexpr (D == 64) {
    if (two_ctas(a)) return kv_tc<64, 2>(a, b, P, st);
  }
  return kv_tc<D, 1>(a, b, P, st);
}

}  // namespace

// D [H, Tq] fp32, then the shares' fp32 dK, dV
size_t packed_workspace_bytes(int64_t Tq, int64_t Tk, int n_seq, int H, int KV, int d) {
  const int splits = head_splits(Tk, n_seq, H, KV);
  size_t n = round_up(static_cast<size_t>(H) * Tq * 4, 256);
  if (splits > 1)
    n += static_cast<size_t>(most_tiles(Tk, n_seq, kRows)) * KV * splits * 2 * kRows * d * 4;
  return n;
}

cudaError_t launch_packed_bwd(const hsnf4_packed_attention& a, const PackedBwd& b, void* ws,
                                 cudaStream_t st) {
  return a.head_dim == 128 ? bwd_tc<128>(a, b, ws, st) : bwd_tc<64>(a, b, ws, st);
}

cudaError_t launch_packed_fwd(const hsnf4_packed_attention& a, void* o, int64_t o_stride,
                                 float* lse, cudaStream_t st) {
  FwdTc P;
  memset(&P, 0, sizeof P);
  const int64_t wq = static_cast<int64_t>(a.H) * a.head_dim,
                wk = static_cast<int64_t>(a.KV) * a.head_dim;
  // head_dim 64: 64 keys a step and four CTAs per SM where that many come.
  // 16/16 heads, 128 keys a step against 64: 64 sequences of 64 tokens 24.5 /
  // 15.1 us, 23 ragged ones of 4100 25.5 / 21.7, 16 of 512 41.1 / 34.8, one of
  // 8192 426 / 377 (no mask); with fewer CTAs the shorter chain of 128 wins,
  // one of 512 9.9 / 12.1, one of 2048 27.4 / 35.2.
  const bool many = a.head_dim == 64 && most_tiles(a.Tq, a.n_seq, kRows) * a.H >= 4 * sm_count();
  const int box = many ? kStep : kRows;
  if (!map_rows(&P.mq, a.q, wq, a.Tq, a.q_stride) ||
      !map_rows(&P.mk, a.k, wk, a.Tk, a.k_stride, box) ||
      !map_rows(&P.mv, a.v, wk, a.Tk, a.v_stride, box))
    return cudaErrorInvalidValue;
  P.out = static_cast<uint16_t*>(o);
  P.os = o_stride;
  P.lse = lse;
  P.S = {a.cu_q, a.cu_k, static_cast<int>(a.Tq), static_cast<int>(a.Tk), a.n_seq, a.causal, 0};
  P.H = a.H;
  P.KV = a.KV;
  P.c = a.scale * kLog2e;
  // One query tile per CTA unless the sequences are long on average.  28/4
  // heads, head_dim 128, causal, one tile against two, short bursts from rest:
  // 64 sequences of 64 tokens 48 / 88 us, 16 of 512 70 / 83, one of 4096 119 /
  // 122, one of 8192 438 / 417, one of 16384 (32/8 heads) 1935 / 1820 to 1875.
  const bool two = a.Tq >= 6144 * static_cast<int64_t>(a.n_seq);
  if (a.head_dim == 128) return two ? fwd_tc<128, 2>(P, st) : fwd_tc<128, 1>(P, st);
  if (many) return fwd64_tc(P, st);
  return two ? fwd_tc<64, 2>(P, st) : fwd_tc<64, 1>(P, st);
}

cudaError_t read_attn_flags(uint32_t* flags) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_flags, sizeof v);
  if (e != cudaSuccess) return e;
  *flags = v;
  if (v) {
    const unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_attn_flags, &z, sizeof z);
  }
  return e;
}

}  // namespace hsnf4
