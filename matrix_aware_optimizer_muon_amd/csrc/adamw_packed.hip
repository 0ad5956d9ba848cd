// AdamW with its moments in 8 bits, and the conversion of such moments from
// and to float32 or bf16 values.
//
//   m' = b1 m + (1-b1) g,   v' = b2 v + ((1-b2) g) g,
//   w' = w - lr wd w - lr (m' / (1-b1^t)) / (sqrt(v' / (1-b2^t)) + eps)
//
// with g the gradient times the clipping factor.  m and v are the values of
// the bytes; the update uses m' and v' as computed, and the bytes get them
// rounded.  The moments are computed in float32 without fused multiply-adds:
// every operation is rounded by itself, so that another program that follows
// the formulas gets the same bytes.
//
// Bytes.  A block is 256 consecutive elements of the row-major tensor.
//   first moment   an OCP e4m3 number times 2^(e-127), one e for each block,
//                  the smallest (from 9 on) that brings the block's largest
//                  magnitude to 448 or below.  Above 2^-14 of the largest,
//                  neighbouring values are 6 to 12 % apart; below it they
//                  run linearly to zero.
//   second moment  never negative, so all 8 bits are magnitude: the float32
//                  whose bits are (code + base) << 20, code 1..255, i.e. 8
//                  values a binade over 31 binades below the block's
//                  largest.  Code 0 is zero and only zero gets it: a second
//                  moment lost to rounding would turn m / sqrt(v) into
//                  m / eps.
// A moment changes by a few per cent of itself a step (by 1-b1, 1-b2), less
// than half the distance of two codes, so rounding to nearest would hold many
// where they are: a v whose gradient has vanished would never decay.  The
// step therefore rounds up or down at random, with the probabilities that
// make the mean the value itself.  The random word of an element is a
// function of (seed, t, tensor, element) alone, so a replayed graph, a
// resumed run and any launch shape give the same bytes: a hash of the group
// of 16 elements plus the element's multiple of 2^32 / golden ratio; its upper
// 20 bits round the first moment, its lower 20 the second.
// The conversion from values rounds to nearest, ties to even.
//
// A first moment that is not finite becomes e4m3's NaN and takes no part in
// its block's scales; its second moment's byte is then without meaning.
#include <type_traits>

#include "device_common.h"
#include "muon_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                      // elements per thread: 16 lanes hold a block
static_assert(kThreads * kPer == kPackChunk && kPackBlock == 16 * kPer, "a row of 16 lanes holds one block");

constexpr uint32_t kGolden = 0x9E3779B9u;     // 2^32 over the golden ratio, odd
constexpr uint32_t kRoot3 = 0xBB67AE85u;      // 2^32 (sqrt(3) - 1), odd
constexpr uint32_t kInf = 0x7F800000u;
constexpr uint32_t kSecondMost = 0x7F700000u; // 1.875 * 2^127, the largest second moment a byte stands for
constexpr uint32_t kScaleLeast = 9;           // keeps e4m3's smallest value times the scale exact in bf16

// Two rounds of xor-shift and multiplication: a bijection of 32 bits.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * kGolden;
  x = (x ^ (x >> 15)) * kRoot3;
  return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t tensor_key(uint32_t seed_lo, uint32_t seed_hi, uint32_t t, uint32_t tensor) {
  return mix(mix(mix(mix(seed_lo) + seed_hi) + t) + tensor);
}

// Maximum over the 16 lanes that hold a block (rotations within a DPP row).
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x128, 0xF, 0xF, false)));
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x124, 0xF, 0xF, false)));
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x122, 0xF, 0xF, false)));
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x121, 0xF, 0xF, false)));
  return x;
}

struct Scales { uint32_t e, base; };

// The scales of the block that holds element i.
__device__ __forceinline__ const uint16_t* scale_at(const uint8_t* codes, int64_t blocks, int64_t i) {
  return reinterpret_cast<const uint16_t*>(codes + blocks * kPackBlock) + i / kPackBlock;
}
__device__ __forceinline__ Scales load_scales(const PackedDev& d, int64_t i) {
  Scales s;
  s.e = max(static_cast<uint32_t>(gld<uint16_t>(scale_at(d.m, d.blocks, i))), kScaleLeast);
  s.base = gld<uint16_t>(scale_at(d.v, d.blocks, i));
  return s;
}

// 16 bytes of each moment to values.
__device__ __forceinline__ void decode(const u32x4_t& mc, const u32x4_t& vc, const Scales& s, float* m, float* v) {
  const float scale = __uint_as_float(s.e << 23);
  const uint32_t vb = s.base << 20;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(mc[q], scale, false);
    const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(mc[q], scale, true);
    m[4 * q] = lo[0]; m[4 * q + 1] = lo[1]; m[4 * q + 2] = hi[0]; m[4 * q + 3] = hi[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t c = (vc[q] >> (8 * k)) & 0xFFu;
      v[4 * q + k] = c ? __uint_as_float((c << 20) + vb) : 0.f;
    }
  }
}

// Values of 16 elements to bytes; all lanes of a block call it together.
// `word` is the random word of the first element; NEAREST rounds to nearest
// instead.  Returns whether a first moment was not finite.
template <bool NEAREST>
__device__ __forceinline__ bool encode(const float* m, const float* v, uint32_t word, u32x4_t& mc, u32x4_t& vc,
                                       Scales& s) {
  uint32_t vb[kPer];
  uint32_t mx = 0, vx = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    vb[e] = __float_as_uint(v[e]) & 0x7FFFFFFFu;
    mx = max(mx, __float_as_uint(m[e]) & 0x7FFFFFFFu);
    vx = max(vx, vb[e]);
  }
  const bool bad = mx >= kInf;
  uint32_t m_top = row_max(mx), v_top = row_max(vx);
  const bool odd = m_top >= kInf || v_top > kSecondMost;   // the same in the 16 lanes of a block
  if (odd) {                       // leave non-finite elements out, bound the second moments
    mx = vx = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const uint32_t a = __float_as_uint(m[e]) & 0x7FFFFFFFu;
      vb[e] = a < kInf ? min(vb[e], kSecondMost) : 0u;
      mx = max(mx, a < kInf ? a : 0u);
      vx = max(vx, vb[e]);
    }
    m_top = row_max(mx);
    v_top = row_max(vx);
  }
  s.e = max(static_cast<int>((m_top + 0x1FFFFFu) >> 23) - 8, static_cast<int>(kScaleLeast));
  s.base = max(static_cast<int>((v_top + 0xFFFFFu) >> 20) - 255, 0);
  const float scale = __uint_as_float(s.e << 23);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t cm = 0, cv = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = 4 * q + k;
      uint32_t idx;
      if constexpr (NEAREST) {
        idx = (vb[e] + 0x7FFFFu + ((vb[e] >> 20) & 1u)) >> 20;
      } else {
        const uint32_t w = word + static_cast<uint32_t>(e) * kGolden;
        idx = (vb[e] + (w & 0xFFFFFu)) >> 20;
        switch (k) {
          case 0: cm = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(static_cast<int>(cm), m[e], w, scale, 0); break;
          case 1: cm = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(static_cast<int>(cm), m[e], w, scale, 1); break;
          case 2: cm = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(static_cast<int>(cm), m[e], w, scale, 2); break;
          default: cm = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(static_cast<int>(cm), m[e], w, scale, 3);
        }
      }
      // at most 255, as base + 255 is not below the largest; at least 1 but for zero
      const int c = max(static_cast<int>(idx - s.base), static_cast<int>(min(vb[e], 1u)));
      cv |= static_cast<uint32_t>(c) << (8 * k);
    }
    if constexpr (NEAREST) {
      typedef short s16x2_t __attribute__((ext_vector_type(2)));
      s16x2_t h = {0, 0};
      h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(h, m[4 * q], m[4 * q + 1], scale, false);
      h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(h, m[4 * q + 2], m[4 * q + 3], scale, true);
      cm = __builtin_bit_cast(uint32_t, h);
    }
    mc[q] = cm;
    vc[q] = cv;
  }
  return bad;
}

// Where an element of param or grad lies: at its index, or in the row that
// holds it.
struct Place {
  int64_t i, r, c;
  __device__ __forceinline__ Place(const PackedDev& d, int64_t i0) : i(i0), r(d.flat ? 0 : i0 / d.cols), c(i0 - r * d.cols) {}
  __device__ __forceinline__ int64_t at(const PackedDev& d, int64_t ld) const { return d.flat ? i : r * ld + c; }
  __device__ __forceinline__ void next(const PackedDev& d) {
    ++i;
    if (!d.flat && ++c == d.cols) { c = 0; ++r; }
  }
};

// 16 consecutive elements at element offset `at` of `base`, aligned to their
// element only: the hardware takes 16-byte accesses at any such address.
typedef float f32x4e_t __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x4h_t __attribute__((ext_vector_type(4), aligned(2)));
template <bool F32>
__device__ __forceinline__ void ld16(const void* base, int64_t at, float* x) {
  if constexpr (F32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4e_t a = gld<f32x4e_t>(static_cast<const float*>(base) + at + 4 * q);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * q + k] = a[k];
    }
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      unpack8_bf16(gld<u32x4h_t>(static_cast<const uint16_t*>(base) + at + 8 * q), x + 8 * q);
  }
}
template <bool F32>
__device__ __forceinline__ void st16(void* base, int64_t at, const float* x) {
  if constexpr (F32) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      gst<f32x4e_t>(static_cast<float*>(base) + at + 4 * q,
                    f32x4e_t{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]});
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) gst<u32x4h_t>(static_cast<uint16_t*>(base) + at + 8 * q, pack8_bf16(x + 8 * q));
  }
}
template <bool F32>
__device__ __forceinline__ float ld1(const void* base, int64_t at) {
  if constexpr (F32) return gld<float>(static_cast<const float*>(base) + at);
  else return bf16_to_f32(gld<uint16_t>(static_cast<const uint16_t*>(base) + at));
}
template <bool F32>
__device__ __forceinline__ void st1(void* base, int64_t at, float x) {
  if constexpr (F32) gst(static_cast<float*>(base) + at, x);
  else gst(static_cast<uint16_t*>(base) + at, f32_to_bf16(x));
}

// 16 elements from i on of param or grad; elements from n on are zero.
template <bool F32>
__device__ __forceinline__ void load_group(const PackedDev& d, const void* base, int64_t ld, int64_t i, float* x) {
  Place pl(d, i);
  if (d.vec && i + kPer <= d.n) {
    ld16<F32>(base, pl.at(d, ld), x);
    return;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    x[e] = pl.i < d.n ? ld1<F32>(base, pl.at(d, ld)) : 0.f;
    pl.next(d);
  }
}

template <bool F32>
__device__ __forceinline__ void store_group(const PackedDev& d, void* base, int64_t ld, int64_t i, const float* x) {
  Place pl(d, i);
  if (d.vec && i + kPer <= d.n) {
    st16<F32>(base, pl.at(d, ld), x);
    return;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    if (pl.i < d.n) st1<F32>(base, pl.at(d, ld), x[e]);
    pl.next(d);
  }
}

__device__ __forceinline__ void store_packed(const PackedDev& d, int64_t i, const u32x4_t& mc, const u32x4_t& vc,
                                             const Scales& s) {
  gst(d.m + i, mc);
  gst(d.v + i, vc);
  if ((threadIdx.x & 15) == 0) {
    gst(const_cast<uint16_t*>(scale_at(d.m, d.blocks, i)), static_cast<uint16_t>(s.e));
    gst(const_cast<uint16_t*>(scale_at(d.v, d.blocks, i)), static_cast<uint16_t>(s.base));
  }
}

template <bool F32>
__device__ __forceinline__ void step_group(const PackedDev& d, const PackedParams& p, int64_t i) {
  const AdamParams& a = p.adam;
  const u32x4_t mc0 = gld<u32x4_t>(d.m + i), vc0 = gld<u32x4_t>(d.v + i);
  Scales s = load_scales(d, i);
  float w[kPer], g[kPer], m[kPer], v[kPer];
  load_group<F32>(d, d.param, d.ld_param, i, w);
  load_group<F32>(d, d.grad, d.ld_grad, i, g);
  decode(mc0, vc0, s, m, v);
  const float factor = a.factor ? gld<float>(a.factor) : 1.f;
  const float lr = a.lr * d.lr_mult, inv_bc1 = a.state->inv_bc1, inv_sqrt_bc2 = a.state->inv_sqrt_bc2;
  const float c1 = 1.f - a.beta1, c2 = 1.f - a.beta2;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
#pragma clang fp contract(off)
    const float ge = g[e] * factor;
    m[e] = a.beta1 * m[e] + c1 * ge;
    v[e] = a.beta2 * v[e] + (c2 * ge) * ge;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const float den = sqrtf(v[e]) * inv_sqrt_bc2 + a.eps;
    w[e] = w[e] - lr * a.weight_decay * w[e] - lr * (m[e] * inv_bc1 / den);
  }
  store_group<F32>(d, d.param, d.ld_param, i, w);
  const uint32_t key = tensor_key(p.seed_lo, p.seed_hi, a.state->t, d.tensor);
  u32x4_t mc, vc;
  const bool bad = encode<false>(m, v, mix(key + static_cast<uint32_t>(i / kPer)), mc, vc, s);
  store_packed(d, i, mc, vc, s);
  if (__any(bad) && (threadIdx.x & 63) == 0) atomicOr(a.flags, 1u);
}

__global__ __launch_bounds__(kThreads) void adamw_packed_kernel(const PackedDev* __restrict__ tensors,
                                                                const PackedTask* __restrict__ tasks,
                                                                PackedParams p) {
  const PackedTask tk = tasks[blockIdx.x];
  const PackedDev& d = tensors[tk.tensor];
  const int64_t i = tk.c0 + static_cast<int64_t>(threadIdx.x) * kPer;
  if (i >= d.blocks * kPackBlock) return;      // whole blocks: the 16 lanes of one stay or leave together
  if (d.f32) step_group<true>(d, p, i);
  else step_group<false>(d, p, i);
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void pack_kernel(const PackedDev* __restrict__ tensors,
                                                        const PackedTask* __restrict__ tasks, const void* values,
                                                        int64_t n_values, uint32_t* flags) {
  const PackedTask tk = tasks[blockIdx.x];
  const PackedDev& d = tensors[tk.tensor];
  const int64_t i = tk.c0 + static_cast<int64_t>(threadIdx.x) * kPer;
  if (i >= d.blocks * kPackBlock) return;
  float m[kPer], v[kPer];
  const int64_t at = d.value0 + i;
  if (i + kPer <= d.n) {
    ld16<F32>(values, at, m);
    ld16<F32>(values, n_values + at, v);
  } else {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      m[e] = i + e < d.n ? ld1<F32>(values, at + e) : 0.f;
      v[e] = i + e < d.n ? ld1<F32>(values, n_values + at + e) : 0.f;
    }
  }
  // a second moment below zero has no root: as in the update, NaN
#pragma unroll
  for (int e = 0; e < kPer; ++e) m[e] = v[e] >= 0.f ? m[e] : __uint_as_float(0x7FC00000u);
  u32x4_t mc, vc;
  Scales s;
  const bool bad = encode<true>(m, v, 0, mc, vc, s);
  store_packed(d, i, mc, vc, s);
  if (__any(bad) && (threadIdx.x & 63) == 0) atomicOr(flags, 1u);
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const PackedDev* __restrict__ tensors,
                                                          const PackedTask* __restrict__ tasks, void* values,
                                                          int64_t n_values) {
  const PackedTask tk = tasks[blockIdx.x];
  const PackedDev& d = tensors[tk.tensor];
  const int64_t i = tk.c0 + static_cast<int64_t>(threadIdx.x) * kPer;
  if (i >= d.n) return;
  float m[kPer], v[kPer];
  decode(gld<u32x4_t>(d.m + i), gld<u32x4_t>(d.v + i), load_scales(d, i), m, v);
  const int64_t at = d.value0 + i;
  if (i + kPer <= d.n) {
    st16<F32>(values, at, m);
    st16<F32>(values, n_values + at, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if (i + e < d.n) {
      st1<F32>(values, at + e, m[e]);
      st1<F32>(values, n_values + at + e, v[e]);
    }
}

}  // namespace

hipError_t launch_adamw_packed(const PackedDev* tensors, const PackedTask* tasks, int n_tasks, const PackedParams& p,
                               hipStream_t s) {
  if (n_tasks <= 0) return hipSuccess;
  adamw_packed_kernel<<<n_tasks, kThreads, 0, s>>>(tensors, tasks, p);
  return hipGetLastError();
}

hipError_t launch_pack_moments(const PackedDev* tensors, const PackedTask* tasks, int n_tasks, const void* values,
                               int64_t n_values, bool f32, uint32_t* flags, hipStream_t s) {
  if (n_tasks <= 0) return hipSuccess;
  if (f32) pack_kernel<true><<<n_tasks, kThreads, 0, s>>>(tensors, tasks, values, n_values, flags);
  else pack_kernel<false><<<n_tasks, kThreads, 0, s>>>(tensors, tasks, values, n_values, flags);
  return hipGetLastError();
}

hipError_t launch_unpack_moments(const PackedDev* tensors, const PackedTask* tasks, int n_tasks, void* values,
                                 int64_t n_values, bool f32, hipStream_t s) {
  if (n_tasks <= 0) return hipSuccess;
  if (f32) unpack_kernel<true><<<n_tasks, kThreads, 0, s>>>(tensors, tasks, values, n_values);
  else unpack_kernel<false><<<n_tasks, kThreads, 0, s>>>(tensors, tasks, values, n_values);
  return hipGetLastError();
}

}  // namespace muon
