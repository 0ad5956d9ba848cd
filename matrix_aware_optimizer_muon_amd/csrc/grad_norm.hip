// Global gradient norm and clipping factor of one step:
//
//   norm = sqrt(sum over every registered gradient of g^2),
//   factor = min(1, max_norm / norm)
//
// The gradients are read only; the kernels that read them next multiply by
// the factor as they do.  Squares and sums are float64: no overflow for any
// finite float32 gradient, and no dependence on the order to speak of; the
// order is fixed all the same (each block a contiguous range of chunks, the
// blocks' sums added in block order), so a step repeats bit for bit.
#include "device_common.h"
#include "muon_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kSegs = kNormChunk / (kThreads * 8);   // 8-element groups per thread and chunk

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Sum over a block of 256 threads, in a fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum64(double v, double* red) {
  v = wave_sum64(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

template <bool F32>
__device__ __forceinline__ double chunk_sum(const NormDev& d, int64_t c0) {
  float g[kSegs][8];
#pragma unroll
  for (int q = 0; q < kSegs; ++q) {
    const int64_t i = c0 + (threadIdx.x + kThreads * q) * 8;
    if (d.vec && i + 8 <= d.n) {
      const int64_t r = d.flat ? 0 : i / d.cols;
      ld8<F32>(d.grad, d.flat ? i : r * d.ld + (i - r * d.cols), g[q]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g[q][e] = 0.f;
        if (i + e < d.n) {
          const int64_t r = d.flat ? 0 : (i + e) / d.cols;
          const int64_t at = d.flat ? i + e : r * d.ld + (i + e - r * d.cols);
          if constexpr (F32) g[q][e] = gld<float>(static_cast<const float*>(d.grad) + at);
          else g[q][e] = bf16_to_f32(gld<uint16_t>(static_cast<const uint16_t*>(d.grad) + at));
        }
      }
    }
  }
  double s = 0.0;
#pragma unroll
  for (int q = 0; q < kSegs; ++q)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double x = g[q][e];
      s = fma(x, x, s);
    }
  return s;
}

__global__ __launch_bounds__(kThreads) void square_sum_kernel(const NormDev* __restrict__ tensors, int n_tensors,
                                                              int64_t n_chunks, double* partials) {
  __shared__ double red[4];
  int64_t c = n_chunks * blockIdx.x / gridDim.x;
  const int64_t end = n_chunks * (blockIdx.x + 1) / gridDim.x;
  int lo = 0, hi = n_tensors - 1;              // the last tensor whose first chunk is not after c
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tensors[mid].chunk0 <= c) lo = mid;
    else hi = mid - 1;
  }
  double s = 0.0;
  for (; c < end; ++c) {
    while (lo + 1 < n_tensors && tensors[lo + 1].chunk0 <= c) ++lo;
    const NormDev& d = tensors[lo];
    const int64_t c0 = (c - d.chunk0) * kNormChunk;
    s += d.f32 ? chunk_sum<true>(d, c0) : chunk_sum<false>(d, c0);
  }
  s = block_sum64(s, red);
  if (threadIdx.x == 0) gst(partials + blockIdx.x, s);
}

__global__ __launch_bounds__(kThreads) void finish_norm_kernel(const double* partials, int n, NormState* st,
                                                               float max_norm, float* norm_out) {
  __shared__ double red[4];
  double s = 0.0;
  for (int k = threadIdx.x; k < n; k += kThreads) s += gld<double>(partials + k);
  s = block_sum64(s, red);
  if (threadIdx.x != 0) return;
  const double norm = sqrt(s);
  // a NaN among the gradients makes the norm, and so every gradient, NaN
  const float factor = norm <= max_norm ? 1.f : static_cast<float>(max_norm / norm);
  st->norm = static_cast<float>(norm);
  st->factor = factor;
  if (norm_out) {
    gst(norm_out, static_cast<float>(norm));
    gst(norm_out + 1, factor);
  }
}

}  // namespace

hipError_t launch_grad_norm(const NormDev* tensors, int n_tensors, int64_t n_chunks, double* partials,
                            NormState* state, float max_norm, float* norm_out, hipStream_t s) {
  const int blocks = static_cast<int>(n_chunks < kNormBlocks ? n_chunks : kNormBlocks);
  if (blocks > 0) square_sum_kernel<<<blocks, kThreads, 0, s>>>(tensors, n_tensors, n_chunks, partials);
  finish_norm_kernel<<<1, kThreads, 0, s>>>(partials, blocks, state, max_norm, norm_out);
  return hipGetLastError();
}

}  // namespace muon
