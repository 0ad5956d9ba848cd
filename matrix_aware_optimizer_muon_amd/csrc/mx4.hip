// Microscaled 4-bit floats: rounding matrices to them and reading them back.
//
// A block of 32 consecutive elements of a row (or of a column) shares a scale
// 2^(e-127), e one byte: the smallest with which no element is beyond the
// largest magnitude, 6.  With amax = (1 + f) 2^k that is k - 2 for f <= 1/2
// (6 = 1.5 * 4) and k - 1 above, so e = ((bits(amax) + 0x3fffff) >> 23) - 2:
// the addition carries into the exponent just where f > 1/2.  e ends at 252:
// with 253 the next code up from the largest float32 would stand for 2^128.
//
// gfx950 converts two float32 or bf16 to e2m1 with their scale in one
// instruction (nearest, ties to even, saturating), and one at random:
// floor(a / step + seed / 2^32) in the code's binade, of which the seed's upper
// 22 bits count.  Its scale operand is a float32 of which the exponent field
// alone is read, so e << 23 serves for every e, 0 (2^-127) and 255 (NaN)
// included.
//
// Bound by memory: 2 or 4 bytes read and 17/32 written an element and form.
#include <type_traits>

#include "device_common.h"
#include "muon_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = kMx4Tile;
constexpr int kChunks = kTile / 8;             // groups of 8 elements across a tile
constexpr int kPasses = kTile * kChunks / kThreads;
constexpr uint32_t kInf = 0x7F800000u;

typedef float f32x2 __attribute__((ext_vector_type(2)));

// The matrix of this block's tile, and the tile's first row and column.
struct Tile { Mx4Dev m; int r0, c0; };
__device__ __forceinline__ Tile find_tile(const Mx4List& l) {
  const int b = static_cast<int>(blockIdx.x);
  int k = 0;
  while (k + 1 < l.n && b >= l.m[k + 1].tile0) ++k;
  Tile t;
  t.m = l.m[k];
  const int local = b - t.m.tile0, tr = local / t.m.tiles_c;
  t.r0 = tr * kTile;
  t.c0 = (local - tr * t.m.tiles_c) * kTile;
  return t;
}

// Scale byte of a block with the largest magnitude's bits, 255 where one is not finite.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t e = max(static_cast<int>((amax + 0x3FFFFFu) >> 23) - 2, 0);
  return amax >= kInf ? 255u : min(e, 252u);
}

// Eight values to their codes, the first in the lowest four bits.
template <bool RANDOM>
__device__ __forceinline__ uint32_t codes8(const float* v, uint32_t e, const uint32_t* words) {
  const float scale = __uint_as_float(e << 23);
  uint32_t w = 0;
  if constexpr (!RANDOM) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
  } else {
    // A seed serves both elements of a conversion, so each element takes one of its own, whose lowest byte
    // is then its code (the other element is zero); the bytes above it are not taken over from the operand
    // that should hold them (seen in the code that hipcc 7.2 makes), so they are left out here.
    uint32_t k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{v[i], 0.f}, words[i], scale, 0);
    const auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {   // their lowest bytes
      return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
    };
    w = four(k[0], k[2], k[4], k[6]) | (four(k[1], k[3], k[5], k[7]) << 4);
  }
  return e == 255u ? 0u : w;
}

// Eight codes to their values.
__device__ __forceinline__ void values8(uint32_t w, uint32_t e, float* v) {
  const float scale = __uint_as_float(e << 23);
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
}

// Random words: 16 consecutive elements of a row share a hash.
__device__ __forceinline__ uint32_t matrix_key(const RoundingSeed& seed, uint32_t index) {
  return mix(mix(mix(seed.lo) + seed.hi) + index);
}
__device__ __forceinline__ uint32_t group_hash(uint32_t key, uint32_t row, uint32_t col) {
  return mix(mix(key + row) + (col >> 4));
}

// Element (r, c) of a tile staged in LDS: the 32-row bands are turned by 32
// columns each, so that four threads that read one column in the four bands
// do not meet in a bank.
__device__ __forceinline__ int turned(int r, int c) { return r * kTile + ((c + (r & ~31)) & (kTile - 1)); }

// One thread of four has the codes of eight elements of a block each.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xF, 0xF, true)));   // lanes 1 0 3 2
  return max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xF, 0xF, true)));  // 2 3 0 1
}

template <bool F32, bool ROW, bool COL, bool RANDOM>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const Mx4List l, const RoundingSeed seed) {
  using E = typename std::conditional<F32, uint32_t, uint16_t>::type;
  __shared__ __attribute__((aligned(16))) E smem[COL ? kTile * kTile : 8];
  __shared__ uint32_t hashes[COL && RANDOM ? kTile * kTile / 16 : 1];
  const Tile t = find_tile(l);
  const Mx4Dev& m = t.m;
  const int q = threadIdx.x % kChunks, rq = threadIdx.x / kChunks;
  const int c = t.c0 + q * 8;
  const uint32_t key = RANDOM ? matrix_key(seed, m.index) : 0u;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int lr = rq + p * (kThreads / kChunks), r = t.r0 + lr;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
    if (r < m.rows) load_row8(m.values, F32, m.ld, r, c, m.cols, m.vec, v);
    uint32_t hash = 0;
    if constexpr (RANDOM) hash = group_hash(key, r, c);
    if constexpr (ROW) {
      uint32_t amax = 0, words[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        amax = max(amax, __float_as_uint(v[k]) & 0x7FFFFFFFu);
        words[k] = RANDOM ? hash + ((c + k) & 15) * kGolden : 0u;
      }
      const uint32_t e = scale_byte(quad_max(amax));
      const uint32_t w = codes8<RANDOM>(v, e, words);
      if (r < m.rows && (c & ~31) < m.cols) {
        gst(m.row.codes + static_cast<size_t>(r) * m.row_ld16 * 16 + (c >> 1), w);
        if ((threadIdx.x & 3) == 0) gst(m.row.scales + static_cast<size_t>(r) * m.row_ld4 * 4 + (c >> 5), static_cast<uint8_t>(e));
      }
    }
    if constexpr (COL) {
      E* dst = smem + turned(lr, q * 8);
      if constexpr (F32) {
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k] = __float_as_uint(v[k]);
      } else {
        *reinterpret_cast<u32x4_t*>(dst) = pack8_bf16(v);
      }
      if constexpr (RANDOM)
        if ((q & 1) == 0) hashes[lr * (kTile / 16) + (q >> 1)] = hash;
    }
  }
  if constexpr (COL) {
    __syncthreads();
    // four neighbouring threads take the four blocks of one column, 64 bytes of its line
    const int band = threadIdx.x & 3;
    const int r = t.r0 + band * 32;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int lc = (threadIdx.x >> 2) + p * 64, cc = t.c0 + lc;
      if (cc >= m.cols || r >= m.rows) continue;
      float v[32];
      uint32_t amax = 0;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const E x = smem[turned(band * 32 + k, lc)];
        v[k] = F32 ? __uint_as_float(x) : bf16_to_f32(static_cast<uint16_t>(x));
        amax = max(amax, __float_as_uint(v[k]) & 0x7FFFFFFFu);
      }
      const uint32_t e = scale_byte(amax);
      u32x4_t w;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t words[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          words[k] = RANDOM ? hashes[(band * 32 + g * 8 + k) * (kTile / 16) + (lc >> 4)] + (lc & 15) * kGolden : 0u;
        w[g] = codes8<RANDOM>(v + g * 8, e, words);
      }
      gst(m.col.codes + (static_cast<size_t>(cc) * m.col_ld16 + (r >> 5)) * 16, w);
      gst(m.col.scales + static_cast<size_t>(cc) * m.col_ld4 * 4 + (r >> 5), static_cast<uint8_t>(e));
    }
  }
}

template <bool F32, int AXIS>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const Mx4List l) {
  using E = typename std::conditional<F32, uint32_t, uint16_t>::type;
  __shared__ __attribute__((aligned(16))) E smem[AXIS == 0 ? kTile * kTile : 8];
  const Tile t = find_tile(l);
  const Mx4Dev& m = t.m;
  if constexpr (AXIS == 0) {
    const int band = threadIdx.x & 3, r = t.r0 + band * 32;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int lc = (threadIdx.x >> 2) + p * 64, cc = t.c0 + lc;
      if (cc >= m.cols || r >= m.rows) continue;
      const u32x4_t w = gld<u32x4_t>(m.col.codes + (static_cast<size_t>(cc) * m.col_ld16 + (r >> 5)) * 16);
      const uint32_t e = gld<uint8_t>(m.col.scales + static_cast<size_t>(cc) * m.col_ld4 * 4 + (r >> 5));
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[8];
        values8(w[g], e, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          smem[turned(band * 32 + g * 8 + k, lc)] = F32 ? __float_as_uint(v[k]) : f32_to_bf16(v[k]);
      }
    }
    __syncthreads();
  }
  const int q = threadIdx.x % kChunks, rq = threadIdx.x / kChunks;
  const int c = t.c0 + q * 8;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int lr = rq + p * (kThreads / kChunks), r = t.r0 + lr;
    if (r >= m.rows || c >= m.cols) continue;
    float v[8];
    if constexpr (AXIS == 1) {
      const uint32_t w = gld<uint32_t>(m.row.codes + static_cast<size_t>(r) * m.row_ld16 * 16 + (c >> 1));
      values8(w, gld<uint8_t>(m.row.scales + static_cast<size_t>(r) * m.row_ld4 * 4 + (c >> 5)), v);
    } else {
      const E* src = smem + turned(lr, q * 8);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = F32 ? __uint_as_float(src[k]) : bf16_to_f32(static_cast<uint16_t>(src[k]));
    }
    store_row8(m.values, F32, m.ld, r, c, m.cols, m.vec, v);
  }
}

template <bool F32, bool RANDOM>
hipError_t launch_forms(const Mx4List& l, const RoundingSeed& seed, hipStream_t s) {
  const bool row = l.m[0].row.codes != nullptr, col = l.m[0].col.codes != nullptr;
  const auto kernel = row && col ? quantize_kernel<F32, true, true, RANDOM>
                      : row      ? quantize_kernel<F32, true, false, RANDOM>
                                 : quantize_kernel<F32, false, true, RANDOM>;
  kernel<<<l.tiles, kThreads, 0, s>>>(l, seed);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_quantize(const Mx4List& l, bool f32, bool random, RoundingSeed seed, hipStream_t s) {
  if (f32) return random ? launch_forms<true, true>(l, seed, s) : launch_forms<true, false>(l, seed, s);
  return random ? launch_forms<false, true>(l, seed, s) : launch_forms<false, false>(l, seed, s);
}

hipError_t launch_mx4_dequantize(const Mx4List& l, bool f32, int axis, hipStream_t s) {
  const auto kernel = f32 ? (axis ? dequantize_kernel<true, 1> : dequantize_kernel<true, 0>)
                          : (axis ? dequantize_kernel<false, 1> : dequantize_kernel<false, 0>);
  kernel<<<l.tiles, kThreads, 0, s>>>(l);
  return hipGetLastError();
}

}  // namespace muon
