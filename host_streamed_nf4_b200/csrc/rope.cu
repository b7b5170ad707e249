// rope.cu -- rotary positions with several axes (time, height, width) for
// the decoder layer's q and k, and the gradient's way back.
//
// Each head's first R = rot_dim values are R / 2 pairs, (i, i + R/2) or
// (2i, 2i + 1); pair i of token t turns by the angle
//   a = pos[axis[i]][t] * inv_freq[i]:
//   forward   y1 = s (x1 cos a - x2 sin a),   y2 = s (x2 cos a + x1 sin a)
//   backward  the transpose: the same with -a.
// The values from R on pass unchanged (times 1, bitwise).
//
// The angle is a double product reduced in double to [-1, 1] half turns
// (positions of a long context times the leading frequency 1 would lose the
// angle in fp32: at position 2^17 the product's rounding alone is 2^-7), then
// sincospif in fp32; the rotation is fp32 and is rounded once to bf16.
//
// Bound by memory: 4 bytes per element of q and k.  A CTA takes one token or
// more (few heads: as many as fill its threads), puts the tokens' cos and sin
// into shared memory once, and every head reads them from there; a thread's
// q/k values are in flight while the angles are computed.
#include <cuda_bf16.h>

#include "internal.h"

namespace hsnf4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;   // tokens per CTA at most
constexpr int kMaxHalf = 128;    // rot_dim / 2 at most

struct RopeParams {
  const uint16_t* in[2];  // q, k
  uint16_t* out[2];
  int64_t in_stride[2], out_stride[2];  // elements between tokens
  const int32_t* pos;                   // [n_axes, T]
  int64_t T;
  int H, KV, d, half;
  int tokens;        // per CTA
  int per_head;      // 16-byte items of a head: rotation items, then pass-through ones
  int rot_items;
  float scale, sign;
  float inv_freq[kMaxHalf];
  uint8_t axis[kMaxHalf];
};

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    f[2 * h] = __uint_as_float(w[h] << 16);
    f[2 * h + 1] = __uint_as_float(w[h] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * h], f[2 * h + 1]);
    w[h] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// in and out may be the same memory (each item's thread reads it whole
// before it writes), so no read-only loads here
template <bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams P) {
  extern __shared__ float2 cs[];  // [tokens][half]: {s cos, s sin}
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.tokens;
  const int nt = static_cast<int>(P.T - t0 < P.tokens ? P.T - t0 : P.tokens);
  const int per_token = (P.H + P.KV) * P.per_head;
  const int items = nt * per_token;

  struct Item {
    uint16_t* dst;
    uint4 a, b;
    int tok, i;  // i: first pair of a rotation item, or -1: pass-through
  };
  auto load = [&](int it) {
    Item x;
    x.tok = it / per_token;
    const int r = it - x.tok * per_token;
    const int head = r / P.per_head, v = r - head * P.per_head;
    const int w = head < P.H ? 0 : 1;
    const int64_t h = w ? head - P.H : head, t = t0 + x.tok;
    int e;  // first element inside the head
    if (v < P.rot_items) {
      x.i = HALF ? v * 8 : v * 4;
      e = v * 8;
    } else {
      x.i = -1;
      e = 2 * P.half + (v - P.rot_items) * 8;
    }
    const uint16_t* src = P.in[w] + t * P.in_stride[w] + h * P.d + e;
    x.dst = P.out[w] + t * P.out_stride[w] + h * P.d + e;
    x.a = *reinterpret_cast<const uint4*>(src);
    if (HALF && x.i >= 0) x.b = *reinterpret_cast<const uint4*>(src + P.half);
    return x;
  };
  auto store = [&](const Item& x) {
    if (x.i < 0) {
      *reinterpret_cast<uint4*>(x.dst) = x.a;
      return;
    }
    const float2* c = cs + x.tok * P.half + x.i;
    float a[8], b[8];
    unpack8(x.a, a);
    if (HALF) {
      unpack8(x.b, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 k = c[e];
        const float y1 = a[e] * k.x - b[e] * k.y, y2 = b[e] * k.x + a[e] * k.y;
        a[e] = y1;
        b[e] = y2;
      }
      *reinterpret_cast<uint4*>(x.dst + P.half) = pack8(b);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 k = c[e];
        const float y1 = a[2 * e] * k.x - a[2 * e + 1] * k.y;
        a[2 * e + 1] = a[2 * e + 1] * k.x + a[2 * e] * k.y;
        a[2 * e] = y1;
      }
    }
    *reinterpret_cast<uint4*>(x.dst) = pack8(a);
  };

  Item first;
  const bool any = static_cast<int>(threadIdx.x) < items;
  if (any) first = load(threadIdx.x);
  for (int j = threadIdx.x; j < nt * P.half; j += kThreads) {
    const int tok = j / P.half, i = j - tok * P.half;
    const double p = P.pos[static_cast<int64_t>(P.axis[i]) * P.T + t0 + tok];
    double turn = p * static_cast<double>(P.inv_freq[i]) * 0.31830988618379067154;  // / pi
    turn -= 2.0 * rint(0.5 * turn);
    float s, c;
    sincospif(static_cast<float>(turn), &s, &c);
    cs[j] = make_float2(P.scale * c, P.sign * P.scale * s);
  }
  __syncthreads();
  if (any) store(first);
  for (int it = threadIdx.x + kThreads; it < items; it += kThreads) store(load(it));
}

}  // namespace

cudaError_t launch_rope(const hsnf4_rope& R, const RopeTensors& t, int64_t T, int H, int KV,
                        bool backward, cudaStream_t st) {
  RopeParams P{};
  bool copy_tail = false;
  for (int w = 0; w < 2; ++w) {
    P.in[w] = static_cast<const uint16_t*>(t.in[w]);
    P.out[w] = static_cast<uint16_t*>(t.out[w]);
    P.in_stride[w] = t.in_stride[w];
    P.out_stride[w] = t.out_stride[w];
    if (t.in[w] != t.out[w]) copy_tail = true;
  }
  P.pos = t.pos;
  P.T = T;
  P.H = H;
  P.KV = KV;
  P.d = R.head_dim;
  P.half = R.rot_dim / 2;
  const bool half = R.pairing == HSNF4_ROPE_HALF;
  P.rot_items = half ? R.rot_dim / 16 : R.rot_dim / 8;
  P.per_head = P.rot_items + (copy_tail ? (R.head_dim - R.rot_dim) / 8 : 0);
  P.scale = R.scale;
  P.sign = backward ? -1.0f : 1.0f;
  for (int i = 0; i < P.half; ++i) {
    P.inv_freq[i] = R.inv_freq[i];
    P.axis[i] = R.axis[i];
  }
  const int per_token = (H + KV) * P.per_head;
  P.tokens = kThreads / per_token;
  if (P.tokens < 1) P.tokens = 1;
  if (P.tokens > kMaxTokens) P.tokens = kMaxTokens;
  const int64_t grid = (T + P.tokens - 1) / P.tokens;
  const size_t smem = static_cast<size_t>(P.tokens) * P.half * sizeof(float2);
  count_launch();
  if (half)
    rope_kernel<true><<<static_cast<unsigned>(grid), kThreads, smem, st>>>(P);
  else
    rope_kernel<false><<<static_cast<unsigned>(grid), kThreads, smem, st>>>(P);
  return cudaGetLastError();
}

}  // namespace hsnf4
