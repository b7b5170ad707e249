// attention_tc.cuh -- pieces of the tcgen05 attention kernels: 128-row
// operand tiles in 128B-swizzled shared memory, the products between them,
// and the barrier waits.
//
// A tile holds 128 tokens x D bf16 of one head as D / 64 boxes of 64 columns
// ([128 rows][128 bytes] each, 16 KiB).  One tile serves as a K-major
// operand (contraction over the head's columns: 16 columns are 32 bytes on)
// and as an MN-major one (contraction over the tokens: 16 tokens are 2 KiB
// on, 64-column atoms a box apart).
#pragma once

#include "ptx.cuh"

namespace hsnf4 {

constexpr int kRows = 128;         // tokens of a tile
constexpr int kBoxBytes = 16384;   // 128 rows x 64 columns of bf16

template <int D>
constexpr int tile_bytes() {
  return D / 64 * kBoxBytes;
}

// N: the tile's tokens, and the rows of a box of `map` (64 rows: boxes of 8 KiB)
template <int D, int N = kRows>
__device__ __forceinline__ void tma_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                         int col, int row) {
#pragma unroll
  for (int b = 0; b < D / 64; ++b) tma_load_2d(dst + b * (N * 128), map, bar, col + 64 * b, row);
}

// Rows from `from` on of a tile become zeros (one warp; swizzling permutes
// the 16-byte pieces inside a row only).
template <int D, int N = kRows>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from) {
  for (int i = threadIdx.x & 31; i < (N - from) * (D / 8); i += 32) {
    const int row = from + i / (D / 8), c = i % (D / 8);
    *reinterpret_cast<uint4*>(tile + (c / 8) * (N * 128) + row * 128 + (c % 8) * 16) =
        make_uint4(0, 0, 0, 0);
  }
}

// d[128 x N] = X Y^T over the D columns of two tiles, Y of N tokens (one
// thread issues)
template <int D, int N = kRows>
__device__ __forceinline__ void mma_xyt(uint32_t d, const uint8_t* X, const uint8_t* Y) {
  const uint64_t x0 = make_sdesc(smem_u32(X), 16, 1024, kLayoutSw128);
  const uint64_t y0 = make_sdesc(smem_u32(Y), 16, 1024, kLayoutSw128);
  constexpr uint32_t idesc = make_idesc_bf16(kRows, N, 0, 0);
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
    umma_bf16(d, x0 + (((k / 4) * kBoxBytes + (k % 4) * 32) >> 4),
              y0 + (((k / 4) * (N * 128) + (k % 4) * 32) >> 4), idesc, k > 0 ? 1u : 0u);
}

// d[128 x D] (+)= A Y over the N tokens of tile Y; A is bf16 in tensor memory,
// 16 tokens to 8 columns, in groups of GROUP tokens `stride` columns apart.
template <int D, int GROUP, int N = kRows>
__device__ __forceinline__ void mma_ay(uint32_t d, uint32_t a, uint32_t stride, const uint8_t* Y,
                                       bool accumulate) {
  const uint64_t y0 = make_sdesc(smem_u32(Y), N * 128, 1024, kLayoutSw128);
  constexpr uint32_t idesc = make_idesc_bf16(kRows, D, 0, 1);
#pragma unroll
  for (int k = 0; k < N / 16; ++k)
    umma_bf16_ta(d, a + (k * 16 / GROUP) * stride + (k * 16 % GROUP) / 2,
                 y0 + ((k * 2048) >> 4), idesc, accumulate || k > 0 ? 1u : 0u);
}

// Part of mma_ay: the 16-token steps `first`, `first` + 1 ... of every group
// (count of them), for an A that becomes ready in parts.
template <int D, int GROUP>
__device__ __forceinline__ void mma_ay_steps(uint32_t d, uint32_t a, uint32_t stride,
                                             const uint8_t* Y, int first, int count,
                                             bool accumulate) {
  const uint64_t y0 = make_sdesc(smem_u32(Y), kBoxBytes, 1024, kLayoutSw128);
  constexpr uint32_t idesc = make_idesc_bf16(kRows, D, 0, 1);
  bool acc = accumulate;
#pragma unroll
  for (int g = 0; g < kRows / GROUP; ++g)
#pragma unroll
    for (int c = 0; c < count; ++c) {
      const int k = g * (GROUP / 16) + first + c;
      umma_bf16_ta(d, a + g * stride + (first + c) * 8, y0 + ((k * 2048) >> 4), idesc,
                   acc ? 1u : 0u);
      acc = true;
    }
}

// 2^x of two values at once on the fp32 pipe: x = n + f with n the nearest
// integer (Cody and Waite's reduction), 2^f by a polynomial of degree 4 that
// is 1 at f = 0 and minimises the relative error on [-1/2, 1/2] (2.9e-6 in
// fp32; found by linear programming), times 2^n.  x below -127 gives 0; x must
// be below 128.  KEEP_NAN: NaN stays NaN (it goes through every step but 2^n),
// for one product more; else it gives 0.
// The special-function unit gives 16 results per clock and SM, half of what
// the tensor cores need beside it, so a share of the exponentials goes this way.
template <bool KEEP_NAN>
__device__ __forceinline__ uint64_t ex2_poly(uint64_t x) {
  float a, b;
  f32x2_unpack(x, a, b);
  const uint64_t y = KEEP_NAN ? f32x2_pack(max_nan(a, -127.0f), max_nan(b, -127.0f))
                              : f32x2_pack(fmaxf(a, -127.0f), fmaxf(b, -127.0f));
  const float magic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer
  const uint64_t t = f32x2_add_rn(y, f32x2_pack(magic, magic));
  const uint64_t n = f32x2_add_rn(t, f32x2_pack(-magic, -magic));
  const uint64_t f = f32x2_fma_rn(n, f32x2_pack(-1.0f, -1.0f), y);
  uint64_t p = f32x2_fma_rn(f32x2_pack(0.009582576341927052f, 0.009582576341927052f), f,
                            f32x2_pack(0.05590682849287987f, 0.05590682849287987f));
  p = f32x2_fma_rn(p, f, f32x2_pack(0.24024106562137604f, 0.24024106562137604f));
  p = f32x2_fma_rn(p, f, f32x2_pack(0.6931241154670715f, 0.6931241154670715f));
  p = f32x2_fma_rn(p, f, f32x2_pack(1.0f, 1.0f));
  float t0, t1, p0, p1;
  f32x2_unpack(t, t0, t1);
  f32x2_unpack(p, p0, p1);
  if (!KEEP_NAN)  // n added to the exponent
    return f32x2_pack_bits(__float_as_uint(p0) + (__float_as_uint(t0) << 23),
                           __float_as_uint(p1) + (__float_as_uint(t1) << 23));
  return f32x2_mul_rn(p, f32x2_pack_bits((__float_as_uint(t0) << 23) + 0x3F800000u,
                                         (__float_as_uint(t1) << 23) + 0x3F800000u));
}

// 2^x of two values on the special-function unit
__device__ __forceinline__ uint64_t ex2_pair(uint64_t x) {
  float a, b;
  f32x2_unpack(x, a, b);
  return f32x2_pack(ex2(a), ex2(b));
}

// 32 columns of this warp's lanes, without the wait
__device__ __forceinline__ void tmem_ld32_at(uint32_t taddr, uint32_t* r) {
  tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(r));
}

// 8 fp32, times `by`, rounded to bf16
__device__ __forceinline__ uint4 pack8_scaled(const uint32_t* r, float by) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = f32x2_to_bf16x2(
        f32x2_mul_rn(f32x2_pack_bits(r[2 * e], r[2 * e + 1]), f32x2_pack(by, by)));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Write 32 rows, one per lane, of PIECES (4 or 8) 16-byte pieces to global
// memory `pitch` bytes apart, the first `rows` of them.  They go through
// shared memory (512 PIECES bytes of this warp's own) so that a store
// instruction covers whole row segments: one row per lane touches 32 lines an
// instruction, which took up to 13000 cycles of a dK/dV tile's epilogue.
template <int PIECES>
__device__ __forceinline__ void put_rows(uint8_t* stage, const uint4* v, void* dst, int64_t pitch,
                                         int rows) {
  const int lane = threadIdx.x & 31;
  auto slot = [&](int r, int c) {  // pieces rotated so that a warp's accesses spread over banks
    return reinterpret_cast<uint4*>(stage) + r * PIECES +
           (c ^ (PIECES == 8 ? r & 7 : (r >> 1) & 3));
  };
#pragma unroll
  for (int c = 0; c < PIECES; ++c) *slot(lane, c) = v[c];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int r = (i * 32 + lane) / PIECES, c = (i * 32 + lane) % PIECES;
    if (r < rows)
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(dst) + r * pitch + c * 16) = *slot(r, c);
  }
  __syncwarp();
}

}  // namespace hsnf4
