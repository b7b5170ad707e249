// grad_norm.cu -- the global 2-norm of many gradient tensors, and clipping:
//
//   norm = sqrt(sum over all tensors g^2),
//   out  = round(g * min(1, max_norm / (norm + 1e-6)))
//
// Bound by memory: one read for the norm, one read and one write for the
// scaling.  The tensors are cut into 16 KiB chunks numbered through all of
// them (a table in device memory gives each tensor's first chunk, so one
// launch serves any number of tensors); each CTA takes an equal contiguous
// range of chunks, and the scaling pass walks its range from the end, where
// the norm pass has just been, so that what the L2 still holds is not read
// again from HBM: of 84 MB out of place 47 MB (their outputs take the rest of
// the cache), of 84 MB in place 81, of 161 MB in place 75 to 80.  The second
// launch is a programmatic dependent one.  The next
// chunk's loads (16 KiB) are in flight while one is worked on, and three
// CTAs per SM: 1120 fp32 tensors of 842 MB 406 us, 6.2 TB/s over the three
// passes (418 with four CTAs and one chunk each); 448 bf16 ones of odd sizes,
// 84 MB: 47 us (42 if they are aligned: the pieces at a tensor's ends go element
// by element, with loads that nothing is ahead of); 14 of 5.8 MB: 8.5 us, of which the two
// launches are 6.
//
// Squares are added in fp32 over one 16-byte load, then in double; a load
// whose fp32 sum leaves the safe range (overflow, underflow, NaN) is squared
// in double instead, so no finite gradient overflows the norm.  Every CTA
// adds the CTAs' partial sums in the same order: results do not depend on
// timing, and no counter or atomic is needed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <memory>
#include <new>

#include "internal.h"
#include "ptx.cuh"

namespace hsnf4 {

namespace {

constexpr int kThreads = 256;
constexpr int kChunkBytes = 16384;
constexpr int kCtasPerSm = 3;
constexpr double kEps = 1e-6;

struct Entry {  // one tensor, in the device table
  const uint8_t* g;
  uint8_t* out;
  int64_t bytes;
  int64_t chunk0;  // its first chunk
  int32_t dtype;
  int16_t shift;   // bytes of g past a 16-byte boundary: its chunks start that much before g
  int16_t same;    // out is as far past one: 16-byte stores
};

struct NormParams {
  const Entry* table;
  int n;
  int64_t chunks;
  double* partial;  // [parts]: a sum per CTA of the first pass
  int parts;
  float* norm;
  float max_norm;
  int scale;  // second pass: write out (0: the norm only)
};

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  return s;
}

template <int DT>
struct Type;
template <>
struct Type<HSNF4_F32> {
  using S = float;
  static constexpr int kVec = 4;
  static __device__ float up(S x) { return x; }
  static __device__ S down(float x) { return x; }
};
template <>
struct Type<HSNF4_BF16> {
  using S = __nv_bfloat16;
  static constexpr int kVec = 8;
  static __device__ float up(S x) { return __bfloat162float(x); }
  static __device__ S down(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Type<HSNF4_F16> {
  using S = __half;
  static constexpr int kVec = 8;
  static __device__ float up(S x) { return __half2float(x); }
  static __device__ S down(float x) { return __float2half_rn(x); }
};

// The tensor that holds a chunk (all threads; empty tensors have no chunks
// and share the next one's first).
struct Cursor {
  int e;
  Entry x;
};

__device__ __forceinline__ Cursor locate(const NormParams& P, int64_t c) {
  __shared__ int found;
  int count = 0;
  for (int i = threadIdx.x; i < P.n; i += kThreads) count += P.table[i].chunk0 <= c;
  if (threadIdx.x == 0) found = 0;
  __syncthreads();
  if (count) atomicAdd(&found, count);
  __syncthreads();
  Cursor k;
  k.e = found - 1;
  k.x = P.table[k.e];
  return k;
}

__device__ __forceinline__ void move_to(const NormParams& P, Cursor& k, int64_t c) {
  while (c < k.x.chunk0) k.x = P.table[--k.e];
  while (k.e + 1 < P.n && P.table[k.e + 1].chunk0 <= c) k.x = P.table[++k.e];
}

constexpr int kLoads = kChunkBytes / 16 / kThreads;

// A chunk's 16-byte pieces of this thread: piece j at byte at(j) of the
// tensor; those that lie in it wholly are loaded.
struct Piece {
  int64_t first;  // byte of piece 0
  bool whole;     // the chunk lies in the tensor wholly
  __device__ Piece(const Entry& x, int64_t c) {
    const int64_t b = (c - x.chunk0) * kChunkBytes - x.shift;
    first = b + threadIdx.x * 16;
    whole = b >= 0 && b + kChunkBytes <= x.bytes;
  }
  __device__ int64_t at(int j) const { return first + j * (kThreads * 16); }
  __device__ bool in(const Entry& x, int j) const {
    return whole || (at(j) >= 0 && at(j) + 16 <= x.bytes);
  }
};

__device__ __forceinline__ void load_chunk(const Entry& x, const Piece& p, uint4 (&v)[kLoads]) {
#pragma unroll
  for (int j = 0; j < kLoads; ++j)
    if (p.in(x, j)) v[j] = *reinterpret_cast<const uint4*>(x.g + p.at(j));
}

// sum of squares of a chunk, this thread's share
template <int DT>
__device__ __forceinline__ double squares(const Entry& x, const Piece& p,
                                          const uint4 (&v)[kLoads]) {
  using Ty = Type<DT>;
  using S = typename Ty::S;
  constexpr int V = Ty::kVec;
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    if (p.in(x, j)) {
      const S* e = reinterpret_cast<const S*>(&v[j]);
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const float f = Ty::up(e[q]);
        s = __fmaf_rn(f, f, s);
      }
      if (s > 1e-30f && s < 1e38f) {
        sum += s;
      } else {
#pragma unroll
        for (int q = 0; q < V; ++q) {
          const double f = Ty::up(e[q]);
          sum += f * f;
        }
      }
    } else {  // the tensor's ends
      for (int64_t b = p.at(j); b < p.at(j) + 16; b += sizeof(S))
        if (b >= 0 && b < x.bytes) {
          const double f = Ty::up(*reinterpret_cast<const S*>(x.g + b));
          sum += f * f;
        }
    }
  }
  return sum;
}

template <int DT>
__device__ __forceinline__ void scale_chunk(const Entry& x, const Piece& p, uint4 (&v)[kLoads],
                                            float coef) {
  using Ty = Type<DT>;
  using S = typename Ty::S;
  constexpr int V = Ty::kVec;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    if (p.in(x, j)) {
      S* e = reinterpret_cast<S*>(&v[j]);
#pragma unroll
      for (int q = 0; q < V; ++q) e[q] = Ty::down(__fmul_rn(Ty::up(e[q]), coef));
      uint8_t* out = x.out + p.at(j);
      if (x.same) {
        *reinterpret_cast<uint4*>(out) = v[j];
      } else {
#pragma unroll
        for (int q = 0; q < V; ++q) reinterpret_cast<S*>(out)[q] = e[q];
      }
    } else {
      for (int64_t b = p.at(j); b < p.at(j) + 16; b += sizeof(S))
        if (b >= 0 && b < x.bytes)
          *reinterpret_cast<S*>(x.out + b) =
              Ty::down(__fmul_rn(Ty::up(*reinterpret_cast<const S*>(x.g + b)), coef));
    }
  }
}

// the CTA's part [c0, c1) of all chunks
__device__ __forceinline__ void my_range(const NormParams& P, int64_t& c0, int64_t& c1) {
  const int64_t q = P.chunks / gridDim.x, r = P.chunks % gridDim.x, b = blockIdx.x;
  c0 = b * q + (b < r ? b : r);
  c1 = c0 + q + (b < r ? 1 : 0);
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_norm_kernel(const NormParams P) {
  __shared__ double red[kThreads / 32];
  pdl_wait_then_release();
  int64_t c0, c1;
  my_range(P, c0, c1);
  double sum = 0.0;
  if (c0 < c1) {
    Cursor k = locate(P, c0);
    uint4 next[kLoads];
    load_chunk(k.x, Piece(k.x, c0), next);
    for (int64_t c = c0; c < c1; ++c) {
      const Cursor k0 = k;  // of this chunk; the next one's loads are in flight meanwhile
      const Piece p(k0.x, c);
      uint4 v[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) v[j] = next[j];
      if (c + 1 < c1) {
        move_to(P, k, c + 1);
        load_chunk(k.x, Piece(k.x, c + 1), next);
      }
      if (k0.x.dtype == HSNF4_F32)
        sum += squares<HSNF4_F32>(k0.x, p, v);
      else if (k0.x.dtype == HSNF4_BF16)
        sum += squares<HSNF4_BF16>(k0.x, p, v);
      else
        sum += squares<HSNF4_F16>(k0.x, p, v);
    }
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) P.partial[blockIdx.x] = sum;
}

// the norm from the partial sums (each CTA adds them all, in one order), and
// the scaling, from the end of the CTA's part; the first chunk is in flight
// while the sums are added
__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_scale_kernel(const NormParams P) {
  __shared__ double red[kThreads / 32];
  pdl_wait_then_release();
  double sum = 0.0;
  for (int i = threadIdx.x; i < P.parts; i += kThreads) sum += P.partial[i];
  int64_t c0 = 0, c1 = 0;
  if (P.scale) my_range(P, c0, c1);
  Cursor k;
  uint4 v[kLoads];
  if (c0 < c1) {
    k = locate(P, c1 - 1);
    load_chunk(k.x, Piece(k.x, c1 - 1), v);
  }
  const float norm = static_cast<float>(sqrt(block_sum(sum, red)));
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.norm = norm;
  // a NaN norm stays a NaN factor, an infinite one makes it 0
  double f = isinf(P.max_norm) ? 1.0 : P.max_norm / (static_cast<double>(norm) + kEps);
  if (f > 1.0) f = 1.0;
  const float coef = static_cast<float>(f);
  for (int64_t c = c1 - 1; c >= c0; --c) {
    const Cursor k0 = k;
    const Piece p(k0.x, c);
    uint4 now[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) now[j] = v[j];
    if (c > c0) {
      move_to(P, k, c - 1);
      // (nothing to clip, in place: not read)
      if (coef != 1.0f || k.x.g != k.x.out) load_chunk(k.x, Piece(k.x, c - 1), v);
    }
    if (coef == 1.0f && k0.x.g == k0.x.out) continue;
    if (k0.x.dtype == HSNF4_F32)
      scale_chunk<HSNF4_F32>(k0.x, p, now, coef);
    else if (k0.x.dtype == HSNF4_BF16)
      scale_chunk<HSNF4_BF16>(k0.x, p, now, coef);
    else
      scale_chunk<HSNF4_F16>(k0.x, p, now, coef);
  }
}

int grid_of(int64_t chunks) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t g = std::min<int64_t>(chunks, static_cast<int64_t>(sms) * kCtasPerSm);
  return static_cast<int>(g < 1 ? 1 : g);
}

}  // namespace

size_t grad_table_bytes(int n) { return static_cast<size_t>(n) * sizeof(Entry); }

size_t grad_workspace_bytes(int64_t chunks) {
  return round_up(static_cast<size_t>(grid_of(chunks)) * sizeof(double), 256);
}

cudaError_t fill_grad_table(const hsnf4_grad* grads, int n, void* table, int64_t* chunks,
                            cudaStream_t st) {
  std::unique_ptr<Entry[]> e(new (std::nothrow) Entry[n]);
  if (!e) return cudaErrorMemoryAllocation;
  int64_t c = 0;
  for (int i = 0; i < n; ++i) {
    const hsnf4_grad& g = grads[i];
    const int64_t bytes = g.n * (g.dtype == HSNF4_F32 ? 4 : 2);
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(g.g) & 15u);
    const bool same = shift == static_cast<int>(reinterpret_cast<uintptr_t>(g.out) & 15u);
    e[i] = {static_cast<const uint8_t*>(g.g), static_cast<uint8_t*>(g.out), bytes, c, g.dtype,
            static_cast<int16_t>(shift), static_cast<int16_t>(same)};
    if (g.n) c += (bytes + shift + kChunkBytes - 1) / kChunkBytes;
  }
  *chunks = c;
  const cudaError_t rc =
      cudaMemcpyAsync(table, e.get(), grad_table_bytes(n), cudaMemcpyHostToDevice, st);
  // the plan may be used on any stream from here on
  return rc != cudaSuccess ? rc : cudaStreamSynchronize(st);
}

cudaError_t launch_grad_norm(const void* table, int n, int64_t chunks, float max_norm, bool scale,
                             float* norm, void* ws, cudaStream_t st) {
  NormParams P{};
  P.table = static_cast<const Entry*>(table);
  P.n = n;
  P.chunks = chunks;
  P.partial = static_cast<double*>(ws);
  P.norm = norm;
  P.max_norm = max_norm;
  P.scale = scale ? 1 : 0;
  const int grid = grid_of(chunks);
  P.parts = grid;
  cudaError_t e = launch_pdl(grad_norm_kernel, dim3(grid), dim3(kThreads), 0, st, P);
  if (e != cudaSuccess) return e;
  // norm only: one CTA adds the partial sums
  return launch_pdl(grad_scale_kernel, dim3(scale ? grid : 1), dim3(kThreads), 0, st, P);
}

}  // namespace hsnf4
