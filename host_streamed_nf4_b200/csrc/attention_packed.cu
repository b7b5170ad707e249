// attention_packed.cu -- attention over several sequences packed into one
// token axis, forward and backward, head_dim 64 or 128, causal or not.
//
// Per sequence (lq queries, lk keys) and query head h with KV head
// h / (H / KV):
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j <= i + lk - lq
//   (causal) or all keys;  lse_i = log sum_j e^{scale q_i . k_j}
//   D_i = dout_i . o_i,  P_ij = e^{scale q_i . k_j - lse_i},
//   dS_ij = P_ij (dout_i . v_j - D_i)
//   dq = scale dS k,  dk = scale dS^T q,  dv = P^T dout
//
// Every kernel finds its tile (sequence, tile of the sequence) by itself from
// the device's cumulative lengths: the grid covers the most tiles the lengths
// could give (tokens / tile + sequences), so no length is needed on the host.
#include <cuda_bf16.h>

#include <stdlib.h>
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "packed.cuh"

namespace hsnf4 {

namespace {

constexpr int kTile = 64;

struct PackedArgs {
  const uint16_t *q, *k, *v, *o, *dout;
  uint16_t *out, *dq, *dk, *dv;
  float* lse;         // [H, Tq]
  float* D;           // [H, Tq]
  float* part;        // backward: [splits][2][Tk][KV][d] partial dK, dV (splits > 1)
  int64_t qs, ks, vs, os, dos, dqs, dks, dvs;  // token strides
  PackedSeqs S;
  int H, KV, splits;
  float scale;
};

__device__ __forceinline__ uint32_t su32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(src_bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 64 rows x D columns of a sequence's rows (len of them from `src`, one head)
// from row r0 on into a padded tile; rows past the sequence become zeros, so
// that what stands behind it in memory (other sequences, unset rows, even
// NaN) meets no product.
template <int D>
__device__ __forceinline__ void load_rows(uint16_t* dst, const uint16_t* src, int r0, int len,
                                          int64_t stride) {
  for (int v = threadIdx.x; v < kTile * (D / 8); v += blockDim.x) {
    const int row = v / (D / 8), col = (v % (D / 8)) * 8;
    const bool in = r0 + row < len;
    const uint16_t* s = in ? src + static_cast<int64_t>(r0 + row) * stride + col : src;
    cp_async16(su32(dst + row * (D + 8) + col), s, in ? 16 : 0);
  }
}

template <int D>
__device__ __forceinline__ void frag_a(uint32_t (&a)[4], const uint16_t* tile, int m0, int k0) {
  const int lane = threadIdx.x & 31;
  ldm_x4(a, su32(tile + (m0 + (lane & 15)) * (D + 8) + k0 + (lane >> 4) * 8));
}
template <int D>
__device__ __forceinline__ void frag_bt(uint32_t (&b)[4], const uint16_t* tile, int n0, int k0) {
  const int lane = threadIdx.x & 31;
  ldm_x4(b, su32(tile + (n0 + (lane & 7)) * (D + 8) + k0 + (lane >> 3) * 8));
}
template <int D>
__device__ __forceinline__ void frag_b(uint32_t (&b)[4], const uint16_t* tile, int k0, int n0) {
  const int lane = threadIdx.x & 31;
  ldm_x4_t(b, su32(tile + (k0 + (lane & 7) + ((lane >> 3) & 1) * 8) * (D + 8) + n0 +
                   (lane >> 4) * 8));
}

// S[16 x 64] = 16 rows (m0) of tile X . Y^T
template <int D>
__device__ __forceinline__ void gemm_xyt(float (&s)[8][4], const uint16_t* X, int m0,
                                         const uint16_t* Y) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[j][e] = 0.0f;
#pragma unroll
  for (int k0 = 0; k0 < D; k0 += 32) {
    uint32_t a0[4], a1[4];
    frag_a<D>(a0, X, m0, k0);
    frag_a<D>(a1, X, m0, k0 + 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t b[4];
      frag_bt<D>(b, Y, j * 8, k0);
      mma16816(s[j], a0, b[0], b[1]);
      mma16816(s[j], a1, b[2], b[3]);
    }
  }
}

// acc[16 x D] += P (16 x 64, rounded to bf16) . Y (64 x D tile)
template <int D>
__device__ __forceinline__ void gemm_py(float (&acc)[D / 8][4], const float (&p)[8][4],
                                        const uint16_t* Y) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    uint32_t a[4];
    a[0] = pack_bf16(p[2 * kk][0], p[2 * kk][1]);
    a[1] = pack_bf16(p[2 * kk][2], p[2 * kk][3]);
    a[2] = pack_bf16(p[2 * kk + 1][0], p[2 * kk + 1][1]);
    a[3] = pack_bf16(p[2 * kk + 1][2], p[2 * kk + 1][3]);
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t b[4];
      frag_b<D>(b, Y, kk * 16, n * 16);
      mma16816(acc[2 * n], a, b[0], b[1]);
      mma16816(acc[2 * n + 1], a, b[2], b[3]);
    }
  }
}

template <int D>
__device__ __forceinline__ void zero(float (&acc)[D / 8][4]) {
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
}

// ---------------------------------------------------------------- forward
template <int D>
__global__ void __launch_bounds__(128) packed_fwd_kernel(const __grid_constant__ PackedArgs P) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kEl = kTile * (D + 8);
  uint16_t* Qs = reinterpret_cast<uint16_t*>(smem);
  uint16_t* KVs = Qs + kEl;  // K0 V0 K1 V1
  PackedTile x;
  const int h = blockIdx.x % P.H;
  if (!find_tile(P.S, false, blockIdx.x / P.H, kTile, x)) return;
  const int kh = h / (P.H / P.KV);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, qd = lane & 3;
  const int m0 = warp * 16, r0 = x.t * kTile;
  const uint16_t* q = P.q + x.q0 * P.qs + h * D;
  const uint16_t* k = P.k + x.k0 * P.ks + kh * D;
  const uint16_t* v = P.v + x.k0 * P.vs + kh * D;
  const int tiles = (key_limit(P.S, x, min(r0 + kTile, x.lq) - 1) + kTile - 1) / kTile;
  load_rows<D>(Qs, q, r0, x.lq, P.qs);
  if (tiles) {
    load_rows<D>(KVs, k, 0, x.lk, P.ks);
    load_rows<D>(KVs + kEl, v, 0, x.lk, P.vs);
  }
  cp_async_commit();
  const float c = P.scale * kLog2e;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  float acc[D / 8][4];
  zero<D>(acc);
  const int rows[2] = {r0 + m0 + g, r0 + m0 + g + 8};
  const int lim[2] = {key_limit(P.S, x, rows[0]), key_limit(P.S, x, rows[1])};
  for (int kt = 0; kt < tiles; ++kt) {
    const uint16_t* Ks = KVs + ((kt & 1) * 2) * kEl;
    if (kt + 1 < tiles) {
      uint16_t* Kn = KVs + (((kt + 1) & 1) * 2) * kEl;
      load_rows<D>(Kn, k, (kt + 1) * kTile, x.lk, P.ks);
      load_rows<D>(Kn + kEl, v, (kt + 1) * kTile, x.lk, P.vs);
    }
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    float s[8][4];
    gemm_xyt<D>(s, Qs, m0, Ks);
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      float mx = m[hr];
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = kt * kTile + j * 8 + 2 * qd + e;
          float& y = s[j][2 * hr + e];
          y = key < lim[hr] ? y * c : -INFINITY;
          mx = fmaxf(mx, y);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float ref = mx == -INFINITY ? 0.0f : mx;  // nothing seen yet: e^-inf = 0
      const float corr = exp2f(m[hr] - ref);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& y = s[j][2 * hr + e];
          y = exp2f(y - ref);
          sum += y;
        }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      l[hr] = l[hr] * corr + sum;
      m[hr] = mx;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        acc[n][2 * hr] *= corr;
        acc[n][2 * hr + 1] *= corr;
      }
    }
    gemm_py<D>(acc, s, Ks + kEl);
    __syncthreads();
  }
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    if (rows[hr] >= x.lq) continue;
    const float inv = lim[hr] ? 1.0f / l[hr] : 0.0f;
    uint16_t* dst = P.out + (x.q0 + rows[hr]) * P.os + h * D;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<uint32_t*>(dst + n * 8 + 2 * qd) =
          pack_bf16(acc[n][2 * hr] * inv, acc[n][2 * hr + 1] * inv);
    if (qd == 0)
      P.lse[static_cast<int64_t>(h) * P.S.Tq + x.q0 + rows[hr]] =
          lim[hr] ? (m[hr] + log2f(l[hr])) / kLog2e : -INFINITY;
  }
}

// ---------------------------------------------------------------- dQ
template <int D>
__global__ void __launch_bounds__(128) packed_dq_kernel(const __grid_constant__ PackedArgs P) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kEl = kTile * (D + 8);
  uint16_t* Qs = reinterpret_cast<uint16_t*>(smem);
  uint16_t* dOs = Qs + kEl;
  uint16_t* Os = dOs + kEl;
  uint16_t* KVs = Os + kEl;  // K0 V0 K1 V1
  __shared__ float Ds[kTile];
  PackedTile x;
  const int h = blockIdx.x % P.H;
  if (!find_tile(P.S, false, blockIdx.x / P.H, kTile, x)) return;
  const int kh = h / (P.H / P.KV);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, qd = lane & 3;
  const int m0 = warp * 16, r0 = x.t * kTile;
  const uint16_t* k = P.k + x.k0 * P.ks + kh * D;
  const uint16_t* v = P.v + x.k0 * P.vs + kh * D;
  const int tiles = (key_limit(P.S, x, min(r0 + kTile, x.lq) - 1) + kTile - 1) / kTile;
  load_rows<D>(Qs, P.q + x.q0 * P.qs + h * D, r0, x.lq, P.qs);
  load_rows<D>(dOs, P.dout + x.q0 * P.dos + h * D, r0, x.lq, P.dos);
  load_rows<D>(Os, P.o + x.q0 * P.os + h * D, r0, x.lq, P.os);
  cp_async_commit();
  if (tiles) {
    load_rows<D>(KVs, k, 0, x.lk, P.ks);
    load_rows<D>(KVs + kEl, v, 0, x.lk, P.vs);
  }
  cp_async_commit();
  cp_async_wait<1>();
  __syncthreads();
  {  // D = dout . o, two threads a row
    const int row = threadIdx.x >> 1, half = threadIdx.x & 1;
    const uint32_t* a = reinterpret_cast<const uint32_t*>(dOs + row * (D + 8) + half * (D / 2));
    const uint32_t* b = reinterpret_cast<const uint32_t*>(Os + row * (D + 8) + half * (D / 2));
    float sum = 0.0f;
#pragma unroll 8
    for (int i = 0; i < D / 4; ++i) {
      sum += __uint_as_float(a[i] << 16) * __uint_as_float(b[i] << 16);
      sum += __uint_as_float(a[i] & 0xFFFF0000u) * __uint_as_float(b[i] & 0xFFFF0000u);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    if (!half) {
      Ds[row] = sum;
      if (r0 + row < x.lq) P.D[static_cast<int64_t>(h) * P.S.Tq + x.q0 + r0 + row] = sum;
    }
  }
  __syncthreads();
  const float c = P.scale * kLog2e;
  const int rows[2] = {r0 + m0 + g, r0 + m0 + g + 8};
  float lse2[2], Dr[2];
  int lim[2];
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    const bool in = rows[hr] < x.lq;
    lse2[hr] = in ? P.lse[static_cast<int64_t>(h) * P.S.Tq + x.q0 + rows[hr]] * kLog2e : 0.0f;
    Dr[hr] = Ds[m0 + g + 8 * hr];
    lim[hr] = in ? key_limit(P.S, x, rows[hr]) : 0;
  }
  float acc[D / 8][4];
  zero<D>(acc);
  for (int kt = 0; kt < tiles; ++kt) {
    const uint16_t* Ks = KVs + ((kt & 1) * 2) * kEl;
    if (kt + 1 < tiles) {
      uint16_t* Kn = KVs + (((kt + 1) & 1) * 2) * kEl;
      load_rows<D>(Kn, k, (kt + 1) * kTile, x.lk, P.ks);
      load_rows<D>(Kn + kEl, v, (kt + 1) * kTile, x.lk, P.vs);
    }
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    float s[8][4], dp[8][4];
    gemm_xyt<D>(s, Qs, m0, Ks);
    gemm_xyt<D>(dp, dOs, m0, Ks + kEl);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int hr = e >> 1, key = kt * kTile + j * 8 + 2 * qd + (e & 1);
        const float p = key < lim[hr] ? exp2f(s[j][e] * c - lse2[hr]) : 0.0f;
        s[j][e] = key < lim[hr] ? p * (dp[j][e] - Dr[hr]) : 0.0f;
      }
    gemm_py<D>(acc, s, Ks);
    __syncthreads();
  }
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    if (rows[hr] >= x.lq) continue;
    uint16_t* dst = P.dq + (x.q0 + rows[hr]) * P.dqs + h * D;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<uint32_t*>(dst + n * 8 + 2 * qd) =
          pack_bf16(acc[n][2 * hr] * P.scale, acc[n][2 * hr + 1] * P.scale);
  }
}

// ---------------------------------------------------------------- dK, dV
// A CTA takes one key tile, one KV head and one share of the group's query
// heads, which it adds in order; with several shares the fp32 sums go to
// `part` and packed_kv_reduce adds the shares in order.
template <int D>
__global__ void __launch_bounds__(128) packed_dkdv_kernel(const __grid_constant__ PackedArgs P) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kEl = kTile * (D + 8);
  uint16_t* Ks = reinterpret_cast<uint16_t*>(smem);
  uint16_t* Vs = Ks + kEl;
  uint16_t* QD = Vs + kEl;  // Q0 dO0 Q1 dO1
  float* LD = reinterpret_cast<float*>(QD + 4 * kEl);  // per buffer: lse [64], D [64]
  const int per = P.KV * P.splits;
  const int kh = blockIdx.x % per / P.splits, split = blockIdx.x % per % P.splits;
  PackedTile x;
  if (!find_tile(P.S, true, blockIdx.x / per, kTile, x)) return;
  const int G = P.H / P.KV;
  const int h0 = kh * G + G * split / P.splits, h1 = kh * G + G * (split + 1) / P.splits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, qd = lane & 3;
  const int m0 = warp * 16, c0 = x.t * kTile;
  // the first query that sees the tile's first key, and so the first query tile
  const int first = P.S.causal ? max(c0 - (x.lk - x.lq), 0) : 0;
  const int qt0 = first / kTile, qt1 = (x.lq + kTile - 1) / kTile;
  const int per_head = max(qt1 - qt0, 0), n = per_head * (h1 - h0);
  auto stage = [&](int i, int b) {
    const int h = h0 + i / per_head, qt = qt0 + i % per_head;
    uint16_t* q = QD + (b * 2) * kEl;
    load_rows<D>(q, P.q + x.q0 * P.qs + h * D, qt * kTile, x.lq, P.qs);
    load_rows<D>(q + kEl, P.dout + x.q0 * P.dos + h * D, qt * kTile, x.lq, P.dos);
    for (int j = threadIdx.x; j < kTile; j += blockDim.x) {
      const int row = qt * kTile + j;
      const int64_t at = static_cast<int64_t>(h) * P.S.Tq + x.q0 + row;
      LD[b * 128 + j] = row < x.lq ? P.lse[at] * kLog2e : 0.0f;
      LD[b * 128 + 64 + j] = row < x.lq ? P.D[at] : 0.0f;
    }
  };
  load_rows<D>(Ks, P.k + x.k0 * P.ks + kh * D, c0, x.lk, P.ks);
  load_rows<D>(Vs, P.v + x.k0 * P.vs + kh * D, c0, x.lk, P.vs);
  if (n) stage(0, 0);
  cp_async_commit();
  const float c = P.scale * kLog2e;
  const int keys[2] = {c0 + m0 + g, c0 + m0 + g + 8};
  float dk[D / 8][4], dv[D / 8][4];
  zero<D>(dk);
  zero<D>(dv);
  for (int i = 0; i < n; ++i) {
    const int b = i & 1, qt = qt0 + i % per_head;
    const uint16_t* Qs = QD + (b * 2) * kEl;
    const uint16_t* dOs = Qs + kEl;
    const float* lse_s = LD + b * 128;
    const float* D_s = lse_s + 64;
    if (i + 1 < n) stage(i + 1, b ^ 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    float s[8][4];
    gemm_xyt<D>(s, Ks, m0, Qs);  // S^T = K Q^T
    // an entry is on if the key exists and the query, which exists, sees it
    auto on = [&](int j, int e) {
      const int key = keys[e >> 1], row = qt * kTile + j * 8 + 2 * qd + (e & 1);
      return key < x.lk && row < x.lq && (!P.S.causal || key <= row + x.lk - x.lq);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[j][e] = on(j, e) ? exp2f(s[j][e] * c - lse_s[j * 8 + 2 * qd + (e & 1)]) : 0.0f;
    gemm_py<D>(dv, s, dOs);  // dV += P^T dO
    float dp[8][4];
    gemm_xyt<D>(dp, Vs, m0, dOs);  // dP^T = V dO^T
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[j][e] = on(j, e) ? s[j][e] * (dp[j][e] - D_s[j * 8 + 2 * qd + (e & 1)]) : 0.0f;
    gemm_py<D>(dk, s, Qs);  // dK += dS^T Q
    __syncthreads();
  }
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    if (keys[hr] >= x.lk) continue;
    const int64_t tok = x.k0 + keys[hr];
    if (P.splits > 1) {
      const int64_t one = static_cast<int64_t>(P.S.Tk) * P.KV * D;
      float* pk = P.part + 2 * split * one + (tok * P.KV + kh) * D;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        *reinterpret_cast<float2*>(pk + n * 8 + 2 * qd) =
            make_float2(dk[n][2 * hr], dk[n][2 * hr + 1]);
        *reinterpret_cast<float2*>(pk + one + n * 8 + 2 * qd) =
            make_float2(dv[n][2 * hr], dv[n][2 * hr + 1]);
      }
    } else {
      uint16_t* pk = P.dk + tok * P.dks + kh * D;
      uint16_t* pv = P.dv + tok * P.dvs + kh * D;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        *reinterpret_cast<uint32_t*>(pk + n * 8 + 2 * qd) =
            pack_bf16(dk[n][2 * hr] * P.scale, dk[n][2 * hr + 1] * P.scale);
        *reinterpret_cast<uint32_t*>(pv + n * 8 + 2 * qd) =
            pack_bf16(dv[n][2 * hr], dv[n][2 * hr + 1]);
      }
    }
  }
}

// dK, dV of every token that belongs to a sequence, the shares added in order
template <int D>
__global__ void __launch_bounds__(256) packed_kv_reduce_kernel(const __grid_constant__ PackedArgs P) {
  PackedTile x;
  if (!find_tile(P.S, true, blockIdx.x, kTile, x)) return;
  const int rows = min(kTile, x.lk - x.t * kTile);
  const int64_t one = static_cast<int64_t>(P.S.Tk) * P.KV * D;
  const int per_row = P.KV * (D / 4);
  for (int i = threadIdx.x; i < rows * per_row; i += 256) {
    const int64_t tok = x.k0 + x.t * kTile + i / per_row;
    const int e = (i % per_row) * 4;  // element of the token's KV * D
    const float* p = P.part + tok * P.KV * D + e;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    for (int s = 0; s < P.splits; ++s) {
      const float4 y = *reinterpret_cast<const float4*>(p + 2 * s * one);
      const float4 z = *reinterpret_cast<const float4*>(p + (2 * s + 1) * one);
      a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
      b.x += z.x, b.y += z.y, b.z += z.z, b.w += z.w;
    }
    *reinterpret_cast<uint2*>(P.dk + tok * P.dks + e) = make_uint2(
        pack_bf16(a.x * P.scale, a.y * P.scale), pack_bf16(a.z * P.scale, a.w * P.scale));
    *reinterpret_cast<uint2*>(P.dv + tok * P.dvs + e) =
        make_uint2(pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
  }
}

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// the most tiles of `rows` tokens that n_seq sequences of T tokens can have
int64_t most_tiles(int64_t T, int n_seq, int rows) { return T / rows + std::min<int64_t>(n_seq, T); }

// shares of a KV group's query heads: enough CTAs for two per SM
int head_splits(int64_t Tk, int H, int KV) {
  const int64_t tiles = (Tk + kTile - 1) / kTile * KV;
  const int64_t want = (2 * sm_count() + tiles - 1) / tiles;
  return static_cast<int>(std::min<int64_t>(H / KV, std::max<int64_t>(want, 1)));
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

PackedArgs args_of(const hsnf4_packed_attention& a) {
  PackedArgs P{};
  P.q = static_cast<const uint16_t*>(a.q);
  P.k = static_cast<const uint16_t*>(a.k);
  P.v = static_cast<const uint16_t*>(a.v);
  P.qs = a.q_stride;
  P.ks = a.k_stride;
  P.vs = a.v_stride;
  P.S.cu_q = a.cu_q;
  P.S.cu_k = a.cu_k;
  P.S.Tq = static_cast<int>(a.Tq);
  P.S.Tk = static_cast<int>(a.Tk);
  P.S.n_seq = a.n_seq;
  P.H = a.H;
  P.KV = a.KV;
  P.S.causal = a.causal;
  P.scale = a.scale;
  P.splits = 1;
  return P;
}

template <int D>
cudaError_t fwd(const PackedArgs& P, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const int smem = 5 * kTile * (D + 8) * 2;
  cudaError_t e = allow_smem(packed_fwd_kernel<D>, smem, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = most_tiles(P.S.Tq, P.S.n_seq, kTile) * P.H;
  count_launch();
  packed_fwd_kernel<D><<<static_cast<unsigned>(grid), 128, smem, st>>>(P);
  return cudaGetLastError();
}

template <int D>
cudaError_t bwd(const PackedArgs& P, cudaStream_t st) {
  static std::atomic<uint64_t> done_q{0}, done_kv{0};
  const int el = kTile * (D + 8) * 2;
  const int smem_q = 7 * el, smem_kv = 6 * el + 2 * 2 * 64 * 4;
  cudaError_t e = allow_smem(packed_dq_kernel<D>, smem_q, done_q);
  if (e == cudaSuccess) e = allow_smem(packed_dkdv_kernel<D>, smem_kv, done_kv);
  if (e != cudaSuccess) return e;
  const int64_t kt = most_tiles(P.S.Tk, P.S.n_seq, kTile);
  count_launch();
  packed_dq_kernel<D><<<static_cast<unsigned>(most_tiles(P.S.Tq, P.S.n_seq, kTile) * P.H), 128, smem_q,
                        st>>>(P);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch();
  packed_dkdv_kernel<D><<<static_cast<unsigned>(kt * P.KV * P.splits), 128, smem_kv, st>>>(P);
  e = cudaGetLastError();
  if (e != cudaSuccess || P.splits == 1) return e;
  count_launch();
  packed_kv_reduce_kernel<D><<<static_cast<unsigned>(kt), 256, 0, st>>>(P);
  return cudaGetLastError();
}

}  // namespace

// D [H, Tq] fp32, then the shares' fp32 dK, dV
size_t packed_workspace_bytes(int64_t Tq, int64_t Tk, int n_seq, int H, int KV, int d) {
  if (!getenv("HX")) return packed_tc_workspace_bytes(Tq, Tk, n_seq, H, KV, d);
  const int splits = head_splits(Tk, H, KV);
  size_t n = round_up(static_cast<size_t>(H) * Tq * 4, 256);
  if (splits > 1) n += static_cast<size_t>(splits) * 2 * Tk * KV * d * 4;
  return n;
}

cudaError_t launch_packed_fwd(const hsnf4_packed_attention& a, void* o, int64_t o_stride,
                              float* lse, cudaStream_t st) {
  if (!getenv("HX")) return launch_packed_fwd_tc(a, o, o_stride, lse, st);
  PackedArgs P = args_of(a);
  P.out = static_cast<uint16_t*>(o);
  P.os = o_stride;
  P.lse = lse;
  return a.head_dim == 128 ? fwd<128>(P, st) : fwd<64>(P, st);
}

cudaError_t launch_packed_bwd(const hsnf4_packed_attention& a, const PackedBwd& b, void* ws,
                              cudaStream_t st) {
  if (!getenv("HX")) return launch_packed_bwd_tc(a, b, ws, st);
  PackedArgs P = args_of(a);
  P.o = static_cast<const uint16_t*>(b.o);
  P.os = b.o_stride;
  P.lse = const_cast<float*>(b.lse);
  P.dout = static_cast<const uint16_t*>(b.dout);
  P.dos = b.do_stride;
  P.dq = static_cast<uint16_t*>(b.dq);
  P.dk = static_cast<uint16_t*>(b.dk);
  P.dv = static_cast<uint16_t*>(b.dv);
  P.dqs = b.dq_stride;
  P.dks = b.dk_stride;
  P.dvs = b.dv_stride;
  P.splits = head_splits(a.Tk, a.H, a.KV);
  P.D = static_cast<float*>(ws);
  P.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                    round_up(static_cast<size_t>(a.H) * a.Tq * 4, 256));
  return a.head_dim == 128 ? bwd<128>(P, st) : bwd<64>(P, st);
}

}  // namespace hsnf4
