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
//                  magnitude to 448 or below.  Above 2^-13 of the largest,
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
// its block's scales; its second moment's byte is then without meaning.  What
// is above 1.875 * 2^127 is held as that, in either moment: the next values
// up, 2^128, are infinite as float32.
#include <cmath>

#include "device_common.h"
#include "muon_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
// A thread takes 8 elements in groups of 16 bytes of the tensor (8 of bf16, 4
// of float32), so that a wave's access is one run of 1 KB: at half that, 32
// bytes apart, float32 values were written back in parts (unpacking 38.6 M
// elements 113 us with streaming stores, 67 us without, 64 to 70 us as it is now).
constexpr int kPer = 8;
constexpr int kWave = 64 * kPer;              // elements per wave
static_assert(kThreads * kPer == kPackChunk && kWave == 2 * kPackBlock, "a wave holds two blocks");
template <bool F32> constexpr int kWidth = F32 ? 4 : 8;           // elements of a group
template <bool F32> constexpr int kGroups = kPer / kWidth<F32>;   // groups of a thread
constexpr int kWordGroup = 16;                // elements that share a hash
template <int W> using codes_t = unsigned int __attribute__((ext_vector_type(W / 4)));

constexpr uint32_t kInf = 0x7F800000u;
constexpr uint32_t kMost = 0x7F700000u;       // 1.875 * 2^127, the largest magnitude a byte stands for
constexpr uint32_t kScaleMost = 247;          // of a block with a first moment above 1.75 * 2^127
constexpr uint32_t kScaleLeast = 9;           // keeps e4m3's smallest value times the scale exact in bf16

// Maximum over the lanes that hold a block (W elements each): rotations within
// the DPP rows of 16 lanes, the neighbouring row, and the other half.
template <int W>
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x128, 0xF, 0xF, false)));
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x124, 0xF, 0xF, false)));
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x122, 0xF, 0xF, false)));
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x121, 0xF, 0xF, false)));
  const auto y = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max(y[0], y[1]);
  if constexpr (W == 4) {
    const auto z = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = max(z[0], z[1]);
  }
  return x;
}

// Streaming accesses for weights, gradients, values and every store: of 82 M
// bf16 elements a step takes 129 us with them and 150 without, unpacking 72 and
// 84.  The moments' bytes are read the ordinary way: read streaming they take
// the step to 136 us, unpacking to 80.
template <typename T>
__device__ __forceinline__ T gld_nt(const void* p) {
  return __builtin_nontemporal_load((const MUON_GLOBAL T*)p);
}
template <typename T>
__device__ __forceinline__ void gst_nt(void* p, T v) {
  __builtin_nontemporal_store(v, (MUON_GLOBAL T*)p);
}

// A descriptor held in scalar registers, read at once: left to itself the
// compiler reads each field where it is used, one wait after another.
__device__ __forceinline__ PackedDev load_desc(const PackedDev* p) {
  PackedDev d = *p;
  d.param = sreg_ptr(d.param);
  d.grad = sreg_ptr(d.grad);
  d.m = sreg_ptr(d.m);
  d.v = sreg_ptr(d.v);
  d.m_scales = sreg_ptr(d.m_scales);
  d.v_scales = sreg_ptr(d.v_scales);
  d.n = sreg_i64(d.n);
  d.blocks = sreg_i64(d.blocks);
  d.value0 = sreg_i64(d.value0);
  return d;
}

struct Scales { uint32_t e, base; };

// One group's bytes and scales as they lie in memory.
template <int W>
struct Packed {
  codes_t<W> m, v;
  Scales s;
  template <typename I>
  __device__ __forceinline__ void load(const PackedDev& d, I i) {
    m = gld<codes_t<W>>(d.m + i);
    v = gld<codes_t<W>>(d.v + i);
    s.e = gld<uint16_t>(d.m_scales + i / kPackBlock);
    s.base = gld<uint16_t>(d.v_scales + i / kPackBlock);
  }
  template <typename I>
  __device__ __forceinline__ void store(const PackedDev& d, I i) const {
    gst_nt(d.m + i, m);
    gst_nt(d.v + i, v);
    if ((threadIdx.x & (kPackBlock / W - 1)) == 0) {
      gst(d.m_scales + i / kPackBlock, static_cast<uint16_t>(s.e));
      gst(d.v_scales + i / kPackBlock, static_cast<uint16_t>(s.base));
    }
    // 256 units (code 0x78) of the largest scale are 2^128: 240 (0x77) in their
    // place.  Stored once more, as a correction before the first store kept the
    // weights in registers past it: up to 9 spilled of 64.
    if (s.e == kScaleMost) {
      codes_t<W> x = m;
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const uint32_t apart = (x[q] & 0x7F7F7F7Fu) ^ 0x78787878u;   // byte by byte, zero where the code is 0x78
        x[q] -= ((0x80808080u - apart) & 0x80808080u) >> 7;
      }
      gst_nt(d.m + i, x);
    }
  }
  __device__ __forceinline__ void decode(float* mo, float* vo) const {
    const float scale = __uint_as_float(max(s.e, kScaleLeast) << 23);   // a zero-filled buffer has no scales
    const uint32_t vb = s.base << 20;
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(m[q], scale, false);
      const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(m[q], scale, true);
      mo[4 * q] = lo[0]; mo[4 * q + 1] = lo[1]; mo[4 * q + 2] = hi[0]; mo[4 * q + 3] = hi[1];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t c = (v[q] >> (8 * k)) & 0xFFu;
        vo[4 * q + k] = c ? __uint_as_float((c << 20) + vb) : 0.f;
      }
    }
  }
  // Values to bytes and scales; all lanes of a block call it together.  `word`
  // is the random word of the first element; NEAREST rounds to nearest instead.
  // Returns whether a first moment was not finite.
  template <bool NEAREST>
  __device__ __forceinline__ bool encode(const float* mi, float* vi, uint32_t word);
};

template <int W>
template <bool NEAREST>
__device__ __forceinline__ bool Packed<W>::encode(const float* mi, float* vi, uint32_t word) {
  uint32_t mx = 0, vx = 0;
#pragma unroll
  for (int e = 0; e < W; ++e) {
    // the step's second moments carry no sign bit but a NaN's, which `odd` sees
    if constexpr (NEAREST) vi[e] = fabsf(vi[e]);
    mx = max(mx, __float_as_uint(mi[e]) & 0x7FFFFFFFu);
    vx = max(vx, __float_as_uint(vi[e]));
  }
  const bool bad = mx >= kInf;
  uint32_t m_top = block_max<W>(mx), v_top = block_max<W>(vx);
  const bool odd = m_top >= kInf || v_top > kMost;   // the same in all lanes of a block
  if (odd) {                       // leave non-finite elements out, bound the second moments
    mx = vx = 0;
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const uint32_t a = __float_as_uint(mi[e]) & 0x7FFFFFFFu;
      const uint32_t b = a < kInf ? min(__float_as_uint(vi[e]), kMost) : 0u;
      mx = max(mx, a < kInf ? a : 0u);
      vx = max(vx, b);
      vi[e] = __uint_as_float(b);
    }
    m_top = block_max<W>(mx);
    v_top = block_max<W>(vx);
  }
  s.e = max(static_cast<int>((m_top + 0x1FFFFFu) >> 23) - 8, static_cast<int>(kScaleLeast));
  s.base = max(static_cast<int>((v_top + 0xFFFFFu) >> 20) - 255, 0);
  const float scale = __uint_as_float(s.e << 23);
  const uint32_t below = s.base << 20;
#pragma unroll
  for (int q = 0; q < W / 4; ++q) {
    uint32_t cm = 0, cv = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = 4 * q + k;
      const uint32_t vb = __float_as_uint(vi[e]);
      uint32_t add;            // what carries a share of the lower 20 bits into the index
      if constexpr (NEAREST) {
        add = 0x7FFFFu + ((vb >> 20) & 1u);
      } else {
        const uint32_t w = word + static_cast<uint32_t>(e) * kGolden;
        add = w & 0xFFFFFu;
        switch (k) {
          case 0: cm = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(static_cast<int>(cm), mi[e], w, scale, 0); break;
          case 1: cm = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(static_cast<int>(cm), mi[e], w, scale, 1); break;
          case 2: cm = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(static_cast<int>(cm), mi[e], w, scale, 2); break;
          default: cm = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(static_cast<int>(cm), mi[e], w, scale, 3);
        }
      }
      // at most 255, as base + 255 is not below the largest; at least 1 but for zero
      const int c = max(static_cast<int>(vb + add - below) >> 20, static_cast<int>(min(vb, 1u)));
      cv |= static_cast<uint32_t>(c) << (8 * k);
    }
    if constexpr (NEAREST) {
      typedef short s16x2_t __attribute__((ext_vector_type(2)));
      s16x2_t h = {0, 0};
      h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(h, mi[4 * q], mi[4 * q + 1], scale, false);
      h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(h, mi[4 * q + 2], mi[4 * q + 3], scale, true);
      cm = __builtin_bit_cast(uint32_t, h);
    }
    m[q] = cm;
    v[q] = cv;
  }
  return bad;
}

// One group of param, grad or plain values, at element offset `at` of `base`:
// 16 bytes, aligned to their element only (the hardware takes such accesses
// at any address).
typedef float f32x4e_t __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x4h_t __attribute__((ext_vector_type(4), aligned(2)));
template <bool F32> struct Raw;
template <> struct Raw<true> {
  f32x4_t q;
  template <typename I>
  __device__ __forceinline__ void load(const void* base, I at) {
    q = gld_nt<f32x4e_t>(static_cast<const float*>(base) + at);
  }
  __device__ __forceinline__ void values(float* x) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = q[e];
  }
};
template <> struct Raw<false> {
  u32x4_t q;
  template <typename I>
  __device__ __forceinline__ void load(const void* base, I at) {
    q = gld_nt<u32x4h_t>(static_cast<const uint16_t*>(base) + at);
  }
  __device__ __forceinline__ void values(float* x) const { unpack8_bf16(q, x); }
};
template <bool F32, typename I>
__device__ __forceinline__ void store_group(void* base, I at, const float* x) {
  if constexpr (F32) gst_nt<f32x4e_t>(static_cast<float*>(base) + at, f32x4e_t{x[0], x[1], x[2], x[3]});
  else gst_nt<u32x4h_t>(static_cast<uint16_t*>(base) + at, pack8_bf16(x));
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

// First element, from the chunk's start, of this thread's group q: a wave's
// groups of one q lie side by side.
template <bool F32>
__device__ __forceinline__ uint32_t group_start(int q) {
  return (threadIdx.x >> 6) * kWave + q * (64 * kWidth<F32>) + (threadIdx.x & 63) * kWidth<F32>;
}

// The descriptor with its buffers moved on to element c0, a chunk's first.
template <bool F32>
__device__ __forceinline__ PackedDev chunk_desc(PackedDev d, int64_t c0) {
  constexpr int es = F32 ? 4 : 2;
  d.param = static_cast<char*>(d.param) + c0 * es;
  d.grad = static_cast<const char*>(d.grad) + c0 * es;
  d.m += c0;
  d.v += c0;
  d.m_scales += c0 / kPackBlock;
  d.v_scales += c0 / kPackBlock;
  return d;
}

// Debug builds: a chunk starts inside its tensor, at a multiple of its size,
// and the tensor's blocks are those of its elements; flag bit 2 otherwise.
__device__ __forceinline__ bool task_in_bounds(const PackedDev& d, int64_t c0, uint32_t* flags) {
  const bool ok = c0 >= 0 && c0 < d.n && c0 % kPackChunk == 0 && d.blocks == (d.n + kPackBlock - 1) / kPackBlock &&
                  d.cols > 0 && d.n % d.cols == 0 && d.ld_param >= d.cols && d.ld_grad >= d.cols;
  if (!ok && threadIdx.x == 0) atomicOr(flags, kFlagBounds);
  return ok;
}

// ... and its values lie inside the caller's.
__device__ __forceinline__ bool values_in_bounds(const PackedDev& d, int64_t n_values, uint32_t* flags) {
  const bool ok = d.value0 >= 0 && d.value0 + d.n <= n_values;
  if (!ok && threadIdx.x == 0) atomicOr(flags, kFlagBounds);
  return ok;
}

// What one step holds for all elements of a tensor.
struct StepScalars {
  float factor, beta1, beta2, c1, c2, inv_sqrt_bc2, eps, decay, step;
  uint32_t key;
  __device__ __forceinline__ StepScalars(const PackedDev& d, const PackedParams& p, const AdamBias& bias,
                                         uint32_t tensor_key) {
    const AdamParams& a = p.adam;
    factor = a.factor ? gld<float>(a.factor) : 1.f;
    const float lr = a.lr * d.lr_mult;
    beta1 = a.beta1;
    beta2 = a.beta2;
    c1 = 1.f - a.beta1;
    c2 = 1.f - a.beta2;
    inv_sqrt_bc2 = bias.inv_sqrt_bc2;
    eps = a.eps;
    decay = lr * a.weight_decay;
    step = lr * bias.inv_bc1;
    key = tensor_key;
  }
};

// One group's update: w to the new weight, the moments to their new bytes.
// Returns whether a first moment is not finite.
// PRECISE: sqrtf and division as the language has them.  Otherwise the
// hardware's own square root and reciprocal, each within one unit in the
// last place; that square root takes denormal numbers as zero, so it is used
// where 2^-63, the largest root lost, leaves eps as it is (launch_adamw_packed).
template <bool PRECISE, int W>
__device__ __forceinline__ bool update_group(const StepScalars& k, Packed<W>& pk, float* w, const float* g,
                                             uint32_t word) {
  float m[W], v[W];
  pk.decode(m, v);
#pragma unroll
  for (int e = 0; e < W; ++e) {
#pragma clang fp contract(off)
    const float ge = g[e] * k.factor;
    m[e] = k.beta1 * m[e] + k.c1 * ge;
    v[e] = k.beta2 * v[e] + (k.c2 * ge) * ge;
  }
#pragma unroll
  for (int e = 0; e < W; ++e) {
    const float root = PRECISE ? sqrtf(v[e]) : __builtin_amdgcn_sqrtf(v[e]);
    const float den = fmaf(root, k.inv_sqrt_bc2, k.eps);
    const float term = PRECISE ? m[e] / den : m[e] * __builtin_amdgcn_rcpf(den);
    w[e] = fmaf(-k.step, term, fmaf(-k.decay, w[e], w[e]));
  }
  return pk.template encode<false>(m, v, word);
}

// The random word of element i of a tensor.
__device__ __forceinline__ uint32_t random_word(uint32_t key, int64_t i) {
  return mix(key + static_cast<uint32_t>(i / kWordGroup)) + static_cast<uint32_t>(i % kWordGroup) * kGolden;
}

// A chunk that lies inside its tensor, contiguous in memory: one base for the
// block and 32-bit offsets for the lanes, every load before the first use of
// one.
template <bool F32, bool PRECISE, typename Begin>
__device__ __forceinline__ bool step_whole_chunk(const PackedDev& d, const PackedParams& p, const Begin& begin,
                                                 int64_t c0) {
  constexpr int W = kWidth<F32>, G = kGroups<F32>;
  const PackedDev c = chunk_desc<F32>(d, c0);
  Packed<W> pk[G];
  Raw<F32> wr[G], gr[G];
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const uint32_t i = group_start<F32>(q);
    pk[q].load(c, i);
    wr[q].load(c.param, i);
    gr[q].load(c.grad, i);
  }
  const StepScalars k = begin(d, p);
  const uint32_t key = k.key + static_cast<uint32_t>(c0 / kWordGroup);
  bool bad = false;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const uint32_t i = group_start<F32>(q);
    float w[W], g[W];
    wr[q].values(w);
    gr[q].values(g);
    bad |= update_group<PRECISE, W>(k, pk[q], w, g, random_word(key, i));
    store_group<F32>(c.param, i, w);
    pk[q].store(c, i);
  }
  return bad;
}

// A contiguous tensor's last chunk, of which `left` elements are its own.
template <bool F32, bool PRECISE, typename Begin>
__device__ __forceinline__ bool step_last_chunk(const PackedDev& d, const PackedParams& p, const Begin& begin,
                                                int64_t c0, uint32_t left) {
  constexpr int W = kWidth<F32>, G = kGroups<F32>;
  const PackedDev c = chunk_desc<F32>(d, c0);
  const uint32_t blocks_left = (left + kPackBlock - 1) / kPackBlock * kPackBlock;
  const StepScalars k = begin(d, p);
  const uint32_t key = k.key + static_cast<uint32_t>(c0 / kWordGroup);
  bool bad = false;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const uint32_t i = group_start<F32>(q);
    if (i >= blocks_left) break;               // whole blocks: the lanes of one stay or leave together
    Packed<W> pk;
    pk.load(c, i);
    float w[W], g[W];
    if (i + W <= left) {
      Raw<F32> wr, gr;
      wr.load(c.param, i);
      gr.load(c.grad, i);
      wr.values(w);
      gr.values(g);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        w[e] = i + e < left ? ld1<F32>(c.param, i + e) : 0.f;
        g[e] = i + e < left ? ld1<F32>(c.grad, i + e) : 0.f;
      }
    }
    bad |= update_group<PRECISE, W>(k, pk, w, g, random_word(key, i));
    if (i + W <= left) {
      store_group<F32>(c.param, i, w);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e)
        if (i + e < left) st1<F32>(c.param, i + e, w[e]);
    }
    pk.store(c, i);
  }
  return bad;
}

// Where an element of a tensor with gaps between its rows lies.
struct Place {
  int64_t i, r, c, cols;
  __device__ __forceinline__ Place(const PackedDev& d, int64_t i0) : i(i0), r(i0 / d.cols), c(i0 - r * d.cols), cols(d.cols) {}
  __device__ __forceinline__ int64_t at(int64_t ld) const { return r * ld + c; }
  __device__ __forceinline__ void next() {
    ++i;
    if (++c == cols) { c = 0; ++r; }
  }
};

// A chunk of a tensor with gaps between its rows: whole groups inside a row,
// one element after another where a row ends in a group.
template <bool F32, bool PRECISE, typename Begin>
__device__ __forceinline__ bool step_rows_chunk(const PackedDev& d, const PackedParams& p, const Begin& begin,
                                                 int64_t c0) {
  constexpr int W = kWidth<F32>, G = kGroups<F32>;
  const StepScalars k = begin(d, p);
  bool bad = false;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const int64_t i = c0 + group_start<F32>(q);
    if (i >= d.blocks * kPackBlock) break;     // whole blocks: the lanes of one stay or leave together
    Packed<W> pk;
    pk.load(d, i);
    float w[W], g[W];
    const Place pl(d, i);
    const bool whole = pl.c + W <= d.cols && i + W <= d.n;
    if (whole) {
      Raw<F32> wr, gr;
      wr.load(d.param, pl.at(d.ld_param));
      gr.load(d.grad, pl.at(d.ld_grad));
      wr.values(w);
      gr.values(g);
    } else {
      Place x = pl;
#pragma unroll
      for (int e = 0; e < W; ++e, x.next()) {
        w[e] = x.i < d.n ? ld1<F32>(d.param, x.at(d.ld_param)) : 0.f;
        g[e] = x.i < d.n ? ld1<F32>(d.grad, x.at(d.ld_grad)) : 0.f;
      }
    }
    bad |= update_group<PRECISE, W>(k, pk, w, g, random_word(k.key, i));
    if (whole) {
      store_group<F32>(d.param, pl.at(d.ld_param), w);
    } else {
      Place x = pl;
#pragma unroll
      for (int e = 0; e < W; ++e, x.next())
        if (x.i < d.n) st1<F32>(d.param, x.at(d.ld_param), w[e]);
    }
    pk.store(d, i);
  }
  return bad;
}

// Tensors with gaps between their rows (ROWS) have a kernel of their own, as
// their addressing took the other one from 64 to 78 registers, from 8 waves a
// SIMD to 6 (82 M bf16 elements 128 and 137 us).
//
// HBM-bound: 10 bytes per bf16 element, 16 per float32 one: 82 M bf16 elements
// in 128 us (6.4 TB/s), 38.6 M float32 ones in 93 us (6.6 TB/s).  The vector
// units are busy for about 100 of the 128 us (42 instructions an element), so
// the root and the reciprocal are the hardware's: with the language's, 65
// instructions an element, the same takes 156 us, float32 99 in place of 95.
// Rows with gaps: 38.5 M bf16 elements in rows of 767 take 110 us (62 without
// gaps), float32 ones 104 (94): a 64-bit division a group, the loads only after
// it, and one element after another where a row ends in a group (71
// instructions an element).
// BEGINS: no launch has advanced the step count before this one.  Its waves
// take the next step's count and corrections; the last block that is done
// advances the count, and a block before the others takes the corrections of
// the step after (launch_adamw_packed).
template <bool F32, bool PRECISE, bool ROWS, bool BEGINS>
__global__ __launch_bounds__(kThreads, 8) void adamw_packed_kernel(const PackedDev* __restrict__ tensors,
                                                                   const PackedTask* __restrict__ tasks,
                                                                   PackedParams p) {
  const uint32_t t = sreg_i32(gld<uint32_t>(&p.adam.state->t)) + BEGINS;
  const uint32_t before = BEGINS && p.advance != nullptr;    // blocks before the tasks'
  if (blockIdx.x >= before) {
    const PackedTask tk = tasks[blockIdx.x - before];
    const PackedDev d = load_desc(tensors + tk.tensor);
    const auto begin = [&](const PackedDev& d, const PackedParams& p) {
      const AdamState& st = *p.adam.state;
      return StepScalars(d, p, BEGINS ? st.next[t & 1] : st.now, tensor_key(p.seed, t, d.tensor));
    };
    const auto step = [&]() -> bool {
      if constexpr (ROWS) {
        return step_rows_chunk<F32, PRECISE>(d, p, begin, tk.c0);
      } else {
        const int64_t left = d.n - tk.c0;
        if (left >= kPackChunk) return step_whole_chunk<F32, PRECISE>(d, p, begin, tk.c0);
        return step_last_chunk<F32, PRECISE>(d, p, begin, tk.c0, static_cast<uint32_t>(left));
      }
    };
    const bool bad = (!MUON_DEBUG_BOUNDS || task_in_bounds(d, tk.c0, p.adam.flags)) && step();
    if (__any(bad) && (threadIdx.x & 63) == 0) atomicOr(p.adam.flags, 1u);
  } else if (threadIdx.x == 0) {
    adam_prepare(p.advance, t + 1, p.adam.beta1, p.adam.beta2);    // in the place that no wave of step t reads
  }
  if constexpr (BEGINS) {
    if (p.advance == nullptr) return;          // a launch after this one advances it
    __syncthreads();                           // every wave has read the count and its corrections
    if (threadIdx.x == 0 && arrive_last(p.arrivals)) p.advance->t = t;
  }
}

// A chunk's plain values: first moments at `first`, second ones at `second`.
template <bool F32>
struct ValueRuns {
  char *first, *second;
  __device__ __forceinline__ ValueRuns(const void* values, int64_t n_values, const PackedDev& d, int64_t c0) {
    constexpr int es = F32 ? 4 : 2;
    first = static_cast<char*>(const_cast<void*>(values)) + (d.value0 + c0) * es;
    second = first + n_values * es;
  }
};

template <bool F32>
__global__ __launch_bounds__(kThreads) void pack_kernel(const PackedDev* __restrict__ tensors,
                                                        const PackedTask* __restrict__ tasks, const void* values,
                                                        int64_t n_values, uint32_t* flags) {
  constexpr int W = kWidth<F32>, G = kGroups<F32>;
  const PackedTask tk = tasks[blockIdx.x];
  const PackedDev d = load_desc(tensors + tk.tensor);
  if constexpr (MUON_DEBUG_BOUNDS)
    if (!task_in_bounds(d, tk.c0, flags) || !values_in_bounds(d, n_values, flags)) return;
  const ValueRuns<F32> runs(values, n_values, d, tk.c0);
  const int64_t left = d.n - tk.c0, blocks_left = d.blocks * kPackBlock - tk.c0;
  float m[G][W], v[G][W];
  if (left >= kPackChunk) {
    Raw<F32> mr[G], vr[G];
#pragma unroll
    for (int q = 0; q < G; ++q) {
      mr[q].load(runs.first, group_start<F32>(q));
      vr[q].load(runs.second, group_start<F32>(q));
    }
#pragma unroll
    for (int q = 0; q < G; ++q) {
      mr[q].values(m[q]);
      vr[q].values(v[q]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < G; ++q)
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const uint32_t i = group_start<F32>(q) + e;
        m[q][e] = i < left ? ld1<F32>(runs.first, i) : 0.f;
        v[q][e] = i < left ? ld1<F32>(runs.second, i) : 0.f;
      }
  }
  const PackedDev c = chunk_desc<F32>(d, tk.c0);
  bool bad = false;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const uint32_t i = group_start<F32>(q);
    if (i >= blocks_left) break;               // whole blocks: the lanes of one stay or leave together
    // a second moment below zero has no root: as in the update, NaN
#pragma unroll
    for (int e = 0; e < W; ++e) m[q][e] = v[q][e] >= 0.f ? m[q][e] : __uint_as_float(0x7FC00000u);
    Packed<W> pk;
    bad |= pk.template encode<true>(m[q], v[q], 0);
    pk.store(c, i);
  }
  if (__any(bad) && (threadIdx.x & 63) == 0) atomicOr(flags, 1u);
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const PackedDev* __restrict__ tensors,
                                                          const PackedTask* __restrict__ tasks, void* values,
                                                          int64_t n_values, uint32_t* flags) {
  constexpr int W = kWidth<F32>, G = kGroups<F32>;
  const PackedTask tk = tasks[blockIdx.x];
  const PackedDev d = load_desc(tensors + tk.tensor);
  if constexpr (MUON_DEBUG_BOUNDS)
    if (!task_in_bounds(d, tk.c0, flags) || !values_in_bounds(d, n_values, flags)) return;
  const ValueRuns<F32> runs(values, n_values, d, tk.c0);
  const PackedDev c = chunk_desc<F32>(d, tk.c0);
  const int64_t left = d.n - tk.c0;
  Packed<W> pk[G];
  if (left >= kPackChunk) {
#pragma unroll
    for (int q = 0; q < G; ++q) pk[q].load(c, group_start<F32>(q));
#pragma unroll
    for (int q = 0; q < G; ++q) {
      float m[W], v[W];
      pk[q].decode(m, v);
      store_group<F32>(runs.first, group_start<F32>(q), m);
      store_group<F32>(runs.second, group_start<F32>(q), v);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const uint32_t i = group_start<F32>(q);
    if (i >= left) break;
    pk[q].load(c, i);
    float m[W], v[W];
    pk[q].decode(m, v);
    if (i + W <= left) {
      store_group<F32>(runs.first, i, m);
      store_group<F32>(runs.second, i, v);
      continue;
    }
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (i + e < left) {
        st1<F32>(runs.first, i + e, m[e]);
        st1<F32>(runs.second, i + e, v[e]);
      }
  }
}

template <bool F32, bool ROWS>
const PackedTask* launch_step(bool precise, bool begins, const PackedDev* tensors, const PackedTask* tasks, int n,
                              const PackedParams& p, hipStream_t s) {
  if (n > 0) {
    const auto kernel = precise ? (begins ? adamw_packed_kernel<F32, true, ROWS, true>
                                          : adamw_packed_kernel<F32, true, ROWS, false>)
                                : (begins ? adamw_packed_kernel<F32, false, ROWS, true>
                                          : adamw_packed_kernel<F32, false, ROWS, false>);
    kernel<<<n + (p.advance != nullptr), kThreads, 0, s>>>(tensors, tasks, p);
  }
  return tasks + n;
}

}  // namespace

hipError_t launch_adamw_packed(const PackedDev* tensors, const PackedTask* tasks, const int* n, bool begins,
                               PackedParams p, hipStream_t s) {
  // a root below 2^-63 times at most 1 / sqrt(1 - b2) stays under half a unit (2^-24) of eps
  const bool precise = !(p.adam.eps * std::sqrt(1.f - p.adam.beta2) >= 0x1p-39f);
  int last = 0;
  for (int k = 0; k < kPackKinds; ++k)
    if (n[k] > 0) last = k;
  AdamState* const state = const_cast<AdamState*>(p.adam.state);
  const auto params = [&](int k) -> const PackedParams& {
    p.advance = begins && k == last ? state : nullptr;
    return p;
  };
  tasks = launch_step<false, false>(precise, begins, tensors, tasks, n[0], params(0), s);
  tasks = launch_step<false, true>(precise, begins, tensors, tasks, n[1], params(1), s);
  tasks = launch_step<true, false>(precise, begins, tensors, tasks, n[2], params(2), s);
  (void)launch_step<true, true>(precise, begins, tensors, tasks, n[3], params(3), s);
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
                                 int64_t n_values, bool f32, uint32_t* flags, hipStream_t s) {
  if (n_tasks <= 0) return hipSuccess;
  if (f32) unpack_kernel<true><<<n_tasks, kThreads, 0, s>>>(tensors, tasks, values, n_values, flags);
  else unpack_kernel<false><<<n_tasks, kThreads, 0, s>>>(tensors, tasks, values, n_values, flags);
  return hipGetLastError();
}

}  // namespace muon
