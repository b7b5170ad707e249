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
// more (as many as 32 KiB hold the cos and sin of) and computes those once.
// A thread keeps its place in the head and walks the heads and tokens, its
// first loads in flight while the angles are computed.  8191 tokens of 64/8
// heads of 128: 51.4 us, 5.9 TB/s; 16000 of 16/16 heads of 64: 25.5 us, 29.0
// with at most 16 tokens a CTA; with few heads a token the angles are the time
// (32768 tokens of 2/1 heads of 128: 17.8 us, 2.8 TB/s).
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"

namespace hsnf4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxAngles = 4096;  // of a CTA: tokens x rot_dim / 2
constexpr int kMaxHalf = 128;     // rot_dim / 2 at most

struct RopeParams {
  const uint16_t* in[2];  // q, k
  uint16_t* out[2];
  int64_t in_stride[2], out_stride[2];  // elements between tokens
  const int32_t* pos;                   // [n_axes, T]
  int64_t T;
  int H, KV, d, half;
  int tokens;        // per CTA
  int par;           // of them at once
  int step;          // heads a token's threads take at once
  int half_pow2;     // half, rounded up to a power of two
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
// before it writes), so no read-only loads of them here
template <bool HALF, int kBatch>
__global__ void __launch_bounds__(kThreads, kBatch == 1 ? 5 : 4)
    rope_kernel(const __grid_constant__ RopeParams P) {
  extern __shared__ __align__(16) float2 cs[];  // [tokens][half]: {s cos, s sin}
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.tokens;
  const int nt = static_cast<int>(P.T - t0 < P.tokens ? P.T - t0 : P.tokens);
  const int heads = P.H + P.KV;
  // this thread: tokens tok, tok + par, ..., item v of heads h0, h0 + step, ...
  const int tok = threadIdx.x / (P.step * P.per_head);
  const int rest = threadIdx.x - tok * P.step * P.per_head;
  const int h0 = rest / P.per_head, v = rest - h0 * P.per_head;
  const bool turn = v < P.rot_items;
  const int e0 = turn ? v * 8 : 2 * P.half + (v - P.rot_items) * 8;  // element inside the head

  uint4 a[kBatch], b[kBatch];
  auto load = [&](int tl, int h1) {
    const uint16_t* q = P.in[0] + (t0 + tl) * P.in_stride[0] + e0;
    const uint16_t* k = P.in[1] + (t0 + tl) * P.in_stride[1] + e0;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = h1 + j * P.step;
      if (h >= heads) continue;
      const uint16_t* src = h < P.H ? q + h * P.d : k + (h - P.H) * P.d;
      a[j] = *reinterpret_cast<const uint4*>(src);
      if (HALF && turn) b[j] = *reinterpret_cast<const uint4*>(src + P.half);
    }
  };
  const bool any = tok < P.par && tok < nt;
  if (any) load(tok, h0);
  {  // this thread's pair i, of tokens tk, tk + stride, ...
    const int i = threadIdx.x & (P.half_pow2 - 1), stride = blockDim.x / P.half_pow2;
    if (i < P.half) {
      const double f = static_cast<double>(P.inv_freq[i]) * 0.31830988618379067154;  // / pi
      const int32_t* pos = P.pos + static_cast<int64_t>(P.axis[i]) * P.T + t0;
      for (int tk0 = threadIdx.x / P.half_pow2; tk0 < nt; tk0 += 4 * stride) {
        int32_t p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (tk0 + j * stride < nt) p[j] = __ldg(pos + tk0 + j * stride);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (tk0 + j * stride >= nt) break;
          double turns = p[j] * f;
          turns -= 2.0 * rint(0.5 * turns);
          float s, c;
          sincospif(static_cast<float>(turns), &s, &c);
          cs[(tk0 + j * stride) * P.half + i] = make_float2(P.scale * c, P.sign * P.scale * s);
        }
      }
    }
  }
  __syncthreads();
  if (!any) return;
  for (int tl = tok; tl < nt; tl += P.par) {
    const float2* c = cs + tl * P.half + (HALF ? v * 8 : v * 4);
    for (int h1 = h0; h1 < heads; h1 += kBatch * P.step) {
      if (tl != tok || h1 != h0) load(tl, h1);
      uint16_t* q = P.out[0] + (t0 + tl) * P.out_stride[0] + e0;
      uint16_t* k = P.out[1] + (t0 + tl) * P.out_stride[1] + e0;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int h = h1 + j * P.step;
        if (h >= heads) break;
        uint16_t* dst = h < P.H ? q + h * P.d : k + (h - P.H) * P.d;
        if (!turn) {
          *reinterpret_cast<uint4*>(dst) = a[j];
          continue;
        }
        float x[8];
        unpack8(a[j], x);
        if (HALF) {
          float y[8];
          unpack8(b[j], y);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float4 w = *reinterpret_cast<const float4*>(c + e);
            const float y0 = x[e] * w.x - y[e] * w.y, y1 = x[e + 1] * w.z - y[e + 1] * w.w;
            y[e] = y[e] * w.x + x[e] * w.y;
            y[e + 1] = y[e + 1] * w.z + x[e + 1] * w.w;
            x[e] = y0;
            x[e + 1] = y1;
          }
          *reinterpret_cast<uint4*>(dst + P.half) = pack8(y);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 w = c[e];
            const float y1 = x[2 * e] * w.x - x[2 * e + 1] * w.y;
            x[2 * e + 1] = x[2 * e + 1] * w.x + x[2 * e] * w.y;
            x[2 * e] = y1;
          }
        }
        *reinterpret_cast<uint4*>(dst) = pack8(x);
      }
    }
  }
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
  // several tokens at once if all their heads fit the threads, else the heads
  // of one in equal passes, two or three of them at once; and, in a long
  // sequence, more tokens in turn, so that each SM gets its CTAs once
  const int heads = H + KV, per_token = heads * P.per_head;
  const int max_tokens = kMaxAngles / P.half;
  P.par = std::min(std::max(kThreads / per_token, 1), max_tokens);
  const int most = kThreads / P.per_head, passes = (heads + most - 1) / most;
  P.step = (heads + passes - 1) / passes;
  int threads = (P.par * P.step * P.per_head + 31) / 32 * 32;
  for (P.half_pow2 = 8; P.half_pow2 < P.half;) P.half_pow2 *= 2;
  threads = std::max(threads, P.half_pow2);
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // As many CTAs per SM as fit, unless fewer share the turns out more evenly
  // (8191 tokens of 72 heads of 128: four with 14 turns 51.4 us, five with 12
  // 55.2; 9000 of 40 heads: four with 16 38.2, six with 11 35.8).
  const int fit = 65536 / ((passes == 1 ? 48 : 64) * threads);
  int64_t turns = 1, least = 0;
  for (int c = std::min(fit, 8); c >= 4; --c) {
    const int64_t n = (T + int64_t(sms) * c * P.par - 1) / (int64_t(sms) * c * P.par);
    const int64_t ctas = (T + n * P.par - 1) / (n * P.par), per_sm = (ctas + sms - 1) / sms * n;
    if (least == 0 || per_sm * 20 < least * 19) turns = n, least = per_sm;
  }
  P.tokens = P.par * static_cast<int>(std::min<int64_t>(turns, std::max(1, max_tokens / P.par)));
  const int64_t grid = (T + P.tokens - 1) / P.tokens;
  const size_t smem = static_cast<size_t>(P.tokens) * P.half * sizeof(float2);
  const int batch = passes == 1 ? 1 : passes == 2 || passes == 4 ? 2 : 3;
  const auto kernel = half ? (batch == 1   ? rope_kernel<true, 1>
                              : batch == 2 ? rope_kernel<true, 2>
                                           : rope_kernel<true, 3>)
                           : (batch == 1   ? rope_kernel<false, 1>
                              : batch == 2 ? rope_kernel<false, 2>
                                           : rope_kernel<false, 3>);
  count_launch();
  kernel<<<static_cast<unsigned>(grid), threads, smem, st>>>(P);
  return cudaGetLastError();
}

}  // namespace hsnf4
