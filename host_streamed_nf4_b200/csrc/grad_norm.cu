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
// again from HBM.  The second launch is a programmatic dependent one.
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
constexpr int kCtasPerSm = 4;
constexpr double kEps = 1e-6;

struct Entry {  // one tensor, in the device table
  const void* g;
  void* out;
  int64_t n;
  int64_t chunk0;  // its first chunk
  int32_t dtype;
  int16_t shift;     // elements of g past a 16-byte boundary: chunks start that much before g
  int16_t same;      // out is as far past one: 16-byte stores
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

__host__ __device__ inline int chunk_elems(int dtype) {
  return dtype == HSNF4_F32 ? kChunkBytes / 4 : kChunkBytes / 2;
}

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

// The CTA's part [c0, c1) of all chunks, tensor by tensor, in order or from
// the end: f(entry, first element), the first element at a 16-byte boundary
// (before the tensor's start in its first chunk).
template <typename F>
__device__ __forceinline__ void walk(const NormParams& P, int64_t c0, int64_t c1, bool back, F f) {
  __shared__ int found;
  // tensors whose first chunk is <= c: the last of them (empty tensors have
  // no chunks and share the next one's first) holds c
  const int64_t start = back ? c1 - 1 : c0;
  int count = 0;
  for (int i = threadIdx.x; i < P.n; i += kThreads) count += P.table[i].chunk0 <= start;
  if (threadIdx.x == 0) found = 0;
  __syncthreads();
  if (count) atomicAdd(&found, count);
  __syncthreads();
  int e = found - 1;
  Entry x = P.table[e];
  for (int64_t i = 0; i < c1 - c0; ++i) {
    const int64_t c = back ? c1 - 1 - i : c0 + i;
    if (back) {
      while (c < x.chunk0) x = P.table[--e];
    } else {
      while (e + 1 < P.n && P.table[e + 1].chunk0 <= c) x = P.table[++e];
    }
    f(x, (c - x.chunk0) * chunk_elems(x.dtype) - x.shift);
  }
}

// sum of squares of a chunk, this thread's share
template <int DT>
__device__ __forceinline__ double squares(const Entry& x, int64_t at) {
  using Ty = Type<DT>;
  using S = typename Ty::S;
  constexpr int V = Ty::kVec, kLoads = kChunkBytes / 16 / kThreads;
  const S* g = static_cast<const S*>(x.g);
  double sum = 0.0;
  uint4 v[kLoads];
  const bool whole = at >= 0 && at + kLoads * kThreads * V <= x.n;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int64_t e0 = at + (threadIdx.x + j * kThreads) * V;
    if (whole || (e0 >= 0 && e0 + V <= x.n)) v[j] = __ldg(reinterpret_cast<const uint4*>(g + e0));
  }
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int64_t e0 = at + (threadIdx.x + j * kThreads) * V;
    if (whole || (e0 >= 0 && e0 + V <= x.n)) {
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
      for (int q = 0; q < V; ++q)
        if (e0 + q >= 0 && e0 + q < x.n) {
          const double f = Ty::up(g[e0 + q]);
          sum += f * f;
        }
    }
  }
  return sum;
}

template <int DT>
__device__ __forceinline__ void scale_chunk(const Entry& x, int64_t at, float coef) {
  using Ty = Type<DT>;
  using S = typename Ty::S;
  constexpr int V = Ty::kVec, kLoads = kChunkBytes / 16 / kThreads;
  const S* g = static_cast<const S*>(x.g);
  S* out = static_cast<S*>(x.out);
  uint4 v[kLoads];
  const bool whole = at >= 0 && at + kLoads * kThreads * V <= x.n;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int64_t e0 = at + (threadIdx.x + j * kThreads) * V;
    if (whole || (e0 >= 0 && e0 + V <= x.n)) v[j] = *reinterpret_cast<const uint4*>(g + e0);
  }
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int64_t e0 = at + (threadIdx.x + j * kThreads) * V;
    if (whole || (e0 >= 0 && e0 + V <= x.n)) {
      S* e = reinterpret_cast<S*>(&v[j]);
#pragma unroll
      for (int q = 0; q < V; ++q) e[q] = Ty::down(__fmul_rn(Ty::up(e[q]), coef));
      if (x.same) {
        *reinterpret_cast<uint4*>(out + e0) = v[j];
      } else {
#pragma unroll
        for (int q = 0; q < V; ++q) out[e0 + q] = e[q];
      }
    } else {
      for (int q = 0; q < V; ++q)
        if (e0 + q >= 0 && e0 + q < x.n) out[e0 + q] = Ty::down(__fmul_rn(Ty::up(g[e0 + q]), coef));
    }
  }
}

__device__ __forceinline__ void my_range(const NormParams& P, int64_t& c0, int64_t& c1) {
  const int64_t q = P.chunks / gridDim.x, r = P.chunks % gridDim.x, b = blockIdx.x;
  c0 = b * q + (b < r ? b : r);
  c1 = c0 + q + (b < r ? 1 : 0);
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const NormParams P) {
  __shared__ double red[kThreads / 32];
  pdl_wait_then_release();
  int64_t c0, c1;
  my_range(P, c0, c1);
  double sum = 0.0;
  if (c0 < c1)
    walk(P, c0, c1, false, [&](const Entry& x, int64_t at) {
      if (x.dtype == HSNF4_F32)
        sum += squares<HSNF4_F32>(x, at);
      else if (x.dtype == HSNF4_BF16)
        sum += squares<HSNF4_BF16>(x, at);
      else
        sum += squares<HSNF4_F16>(x, at);
    });
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) P.partial[blockIdx.x] = sum;
}

// the norm from the partial sums (each CTA adds them all, in one order), and
// the scaling
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const NormParams P) {
  __shared__ double red[kThreads / 32];
  pdl_wait_then_release();
  double sum = 0.0;
  for (int i = threadIdx.x; i < P.parts; i += kThreads) sum += P.partial[i];
  const float norm = static_cast<float>(sqrt(block_sum(sum, red)));
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.norm = norm;
  if (!P.scale) return;
  // a NaN norm stays a NaN factor, an infinite one makes it 0
  double c = isinf(P.max_norm) ? 1.0 : P.max_norm / (static_cast<double>(norm) + kEps);
  if (c > 1.0) c = 1.0;
  const float coef = static_cast<float>(c);
  int64_t c0, c1;
  my_range(P, c0, c1);
  if (c0 < c1)
    walk(P, c0, c1, true, [&](const Entry& x, int64_t at) {
      if (coef == 1.0f && x.g == x.out) return;  // nothing to clip, in place
      if (x.dtype == HSNF4_F32)
        scale_chunk<HSNF4_F32>(x, at, coef);
      else if (x.dtype == HSNF4_BF16)
        scale_chunk<HSNF4_BF16>(x, at, coef);
      else
        scale_chunk<HSNF4_F16>(x, at, coef);
    });
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
    const int ce = chunk_elems(g.dtype), size = kChunkBytes / ce;
    const uintptr_t off = reinterpret_cast<uintptr_t>(g.g) & 15u;
    const int shift = static_cast<int>(off) / size;
    const bool same = off == (reinterpret_cast<uintptr_t>(g.out) & 15u);
    e[i] = {g.g, g.out, g.n, c, g.dtype, static_cast<int16_t>(shift),
            static_cast<int16_t>(same)};
    if (g.n) c += (g.n + shift + ce - 1) / ce;
  }
  *chunks = c;
  // pageable source: the copy has left it when the call returns
  return cudaMemcpyAsync(table, e.get(), grad_table_bytes(n), cudaMemcpyHostToDevice, st);
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
