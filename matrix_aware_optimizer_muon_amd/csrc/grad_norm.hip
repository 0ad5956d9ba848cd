// Global gradient norm and clipping factor of one step:
//
//   norm = sqrt(sum over every registered gradient of g^2),
//   factor = min(1, max_norm / norm), always 1 with an infinite max_norm
//
// The gradients are read only; the kernels that read them next multiply by
// the factor as they do.  Squares and sums are float64: no overflow for any
// finite float32 gradient, and no dependence on the order to speak of; the
// order is fixed all the same (block b of n adds chunks b, b + n, ..., and the
// blocks' sums are added in block order), so a step repeats bit for bit.
//
// HBM-bound: 2 bytes per bf16 element, 4 per float32 one (38.5 M of them 30
// us, 5.2 TB/s).  The blocks stride through the chunks together: with a
// contiguous range each, 39 M bf16 elements took 24 us, so 19, of which about 4
// are the launch and the last block's sums.  Rows with gaps: 38.5 M elements in
// rows of 767 take 48 to 57 us in bf16 and 48 to 66 in float32, as a thread has
// one load in flight there, behind a 64-bit division, and goes element by
// element where a row ends in its 16 bytes.
#include "device_common.h"
#include "muon_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;

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

// 16 bytes at any multiple of the element.
typedef unsigned int u32x4h_t __attribute__((ext_vector_type(4), aligned(2)));
template <bool F32> constexpr int kGroup = F32 ? 4 : 8;       // elements of 16 bytes

// The squares of 16 bytes, into four sums.
template <bool F32>
__device__ __forceinline__ void add_squares(const u32x4_t& q, double* s) {
  float x[kGroup<F32>];
  if constexpr (F32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(q[e]);
  } else {
    unpack8_bf16(q, x);
  }
#pragma unroll
  for (int e = 0; e < kGroup<F32>; ++e) {
    const double d = x[e];
    s[e & 3] = fma(d, d, s[e & 3]);
  }
}

// A chunk that lies inside its tensor, contiguous in memory: every load before
// the first use of one.  The loads stream past the caches although the step
// reads the gradients once more: of 157 M bf16 elements the norm takes 55 us
// so and 94 us otherwise, of 629 M 184 and 258 us (6.8 and 4.9 TB/s), and where
// they would fit in the cache (39 M) the step takes 62.4 us in place of 61.7.
template <bool F32>
__device__ __forceinline__ void add_whole_chunk(const NormDev& d, int64_t c0, double* s) {
  constexpr int G = kNormChunk / (kThreads * kGroup<F32>);
  const char* base = static_cast<const char*>(d.grad) + c0 * (F32 ? 4 : 2);
  u32x4_t q[G];
#pragma unroll
  for (int k = 0; k < G; ++k)
    q[k] = __builtin_nontemporal_load((const MUON_GLOBAL u32x4h_t*)(base + (threadIdx.x + kThreads * k) * 16));
#pragma unroll
  for (int k = 0; k < G; ++k) add_squares<F32>(q[k], s);
}

// Any other chunk: a tensor's last one, or one of rows with gaps.
template <bool F32>
__device__ __forceinline__ void add_any_chunk(const NormDev& d, int64_t c0, double* s) {
  const int64_t end = c0 + kNormChunk < d.n ? c0 + kNormChunk : d.n;
  const char* base = static_cast<const char*>(d.grad);
  constexpr int es = F32 ? 4 : 2, W = kGroup<F32>;
#pragma unroll 1
  for (int64_t i = c0 + threadIdx.x * W; i < end; i += kThreads * W) {
    int64_t r = 0, col = i;
    if (!d.flat) {
      r = i / d.cols;
      col = i - r * d.cols;
    }
    if ((d.flat || col + W <= d.cols) && i + W <= end) {
      add_squares<F32>(gld<u32x4h_t>(base + (r * d.ld + col) * es), s);
      continue;
    }
#pragma unroll 1
    for (int64_t k = i; k < end && k < i + W; ++k) {
      const char* at = base + (r * d.ld + col) * es;
      const double x = F32 ? gld<float>(at) : bf16_to_f32(gld<uint16_t>(at));
      s[0] = fma(x, x, s[0]);
      if (!d.flat && col + 1 == d.cols) {
        col = 0;
        ++r;
      } else {
        ++col;
      }
    }
  }
}

template <bool F32>
__device__ __forceinline__ void add_chunk(const NormDev& d, int64_t c0, double* s) {
  if (d.flat && c0 + kNormChunk <= d.n) add_whole_chunk<F32>(d, c0, s);
  else add_any_chunk<F32>(d, c0, s);
}

// Adds the blocks' sums in their order (256 threads), writes norm and factor,
// and advances the AdamW count.
__device__ __forceinline__ void finish(const NormParams& p, int blocks, double* red) {
  double s = 0.0;
  // past the dies' caches, which hold no sum of another die's block
  for (int b = threadIdx.x; b < blocks; b += kThreads)
    s += __hip_atomic_load(p.partials + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();                             // red may still be read
  s = block_sum64(s, red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(s);
    // a NaN among the gradients makes the norm, and so every gradient, NaN,
    // but for a norm that is only measured
    const bool keep = norm <= p.max_norm || p.max_norm == INFINITY;
    const float factor = keep ? 1.f : static_cast<float>(p.max_norm / norm);
    p.state->norm = static_cast<float>(norm);
    p.state->factor = factor;
    if (p.norm_out) {
      gst(p.norm_out, static_cast<float>(norm));
      gst(p.norm_out + 1, factor);
    }
  } else if (threadIdx.x == 64 && p.adam) {    // in a wave of its own, beside the sums
    adam_advance(p.adam, p.beta1, p.beta2);
  }
}

// Debug builds: a chunk is one of the tensor that the list gives it to; flag
// bit 2 otherwise.
__device__ __forceinline__ bool chunk_in_bounds(const NormParams& p, int64_t c, int32_t tensor) {
  bool ok = tensor >= 0 && tensor < p.n_tensors;
  if (ok) {
    const NormDev& d = p.tensors[tensor];
    ok = c >= d.chunk0 && (c - d.chunk0) * kNormChunk < d.n && d.cols > 0 && d.n % d.cols == 0 &&
         (d.flat || d.ld >= d.cols);
  }
  if (!ok && threadIdx.x == 0) atomicOr(p.flags, kFlagBounds);
  return ok;
}

// The block that is done last finishes: a launch of its own for that takes 6 us
// and another one's gap.
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(NormParams p) {
  __shared__ double red[4];
  __shared__ bool last;
  double sum[4] = {};
  for (int64_t c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    const int32_t tensor = p.chunk_tensor[c];
    if constexpr (MUON_DEBUG_BOUNDS)
      if (!chunk_in_bounds(p, c, tensor)) continue;
    const NormDev& d = p.tensors[tensor];
    const int64_t c0 = (c - d.chunk0) * kNormChunk;
    if (d.f32) add_chunk<true>(d, c0, sum);
    else add_chunk<false>(d, c0, sum);
  }
  const double s = block_sum64((sum[0] + sum[1]) + (sum[2] + sum[3]), red);
  if (threadIdx.x == 0) {
    __hip_atomic_store(p.partials + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = arrive_last(p.arrivals);
  }
  __syncthreads();
  if (last) finish(p, gridDim.x, red);
}

}  // namespace

hipError_t launch_grad_norm(const NormParams& p, hipStream_t s) {
  grad_norm_kernel<<<norm_blocks(p.chunks), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace muon
