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
// 22 bits count for float32 (fewer for bf16, which is widened first therefore).
// Its scale operand is a float32 of which the exponent field alone is read, so
// e << 23 serves for every e, 0 (2^-127) and 255 (NaN) included.
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
constexpr int kRows = kThreads / kChunks;      // rows that the block's threads take at a time
constexpr int kPasses = kTile / kRows;
constexpr uint32_t kInf = 0x7F800000u;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
// 16 bytes at any element's address
typedef unsigned int u32x4e_t __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x4h_t __attribute__((ext_vector_type(4), aligned(2)));
template <bool F32> using raw_t = typename std::conditional<F32, u32x4e_t, u32x4h_t>::type;

// The matrix of this block's tile, and the tile's first row and column.  Dies
// (blockIdx % 8) take runs of tiles, whose neighbours share the cache lines
// that they write.
struct Tile { Mx4Dev m; int r0, c0; };
__device__ __forceinline__ Tile find_tile(const Mx4List& l) {
  const int die = static_cast<int>(blockIdx.x) % 8;
  const int b = die * (l.tiles / 8) + min(die, l.tiles % 8) + static_cast<int>(blockIdx.x) / 8;
  // each lane asks of one matrix whether it starts behind the tile
  const uint64_t before = __ballot(l.tile0[threadIdx.x & 63] <= b);
  const int k = sreg_i32(__popcll(before) - 1);
  Tile t;
  t.m = l.m[k];
  const int local = b - l.tile0[k], tr = local / t.m.tiles_c;
  t.r0 = tr * kTile;
  t.c0 = (local - tr * t.m.tiles_c) * kTile;
  return t;
}

// Scale byte of a block with the largest magnitude's bits, 255 where one is not finite.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t e = max(static_cast<int>((amax + 0x3FFFFFu) >> 23) - 2, 0);
  return amax >= kInf ? 255u : min(e, 252u);
}

// Two elements as they lie in memory, the first in the lower bits: one word of
// bf16, two of float32.
template <bool F32> struct Pair;
template <> struct Pair<true> {
  float a, b;
  __device__ __forceinline__ uint32_t amax() const {
    return max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu);
  }
  template <int SEL>
  __device__ __forceinline__ uint32_t nearest(uint32_t w, float scale) const {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a, b, scale, SEL);
  }
  __device__ __forceinline__ uint32_t random_a(uint32_t word, float scale) const {
    return __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{a, 0.f}, word, scale, 0);
  }
  __device__ __forceinline__ uint32_t random_b(uint32_t word, float scale) const {
    return __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{b, 0.f}, word, scale, 0);
  }
};
template <> struct Pair<false> {
  uint32_t ab;
  __device__ __forceinline__ uint32_t magnitudes() const { return ab & 0x7FFF7FFFu; }
  template <int SEL>
  __device__ __forceinline__ uint32_t nearest(uint32_t w, float scale) const {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, ab), scale, SEL);
  }
  __device__ __forceinline__ uint32_t random_a(uint32_t word, float scale) const {
    return __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{__uint_as_float(ab << 16), 0.f}, word, scale, 0);
  }
  __device__ __forceinline__ uint32_t random_b(uint32_t word, float scale) const {
    return __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{__uint_as_float(ab & 0xFFFF0000u), 0.f}, word, scale, 0);
  }
};

// The largest magnitude of N pairs, as float32 bits.
template <int N>
__device__ __forceinline__ uint32_t amax_of(const Pair<true>* x) {
  uint32_t m = x[0].amax();
#pragma unroll
  for (int k = 1; k < N; ++k) m = max(m, x[k].amax());
  return m;
}
__device__ __forceinline__ u16x2_t max_u16(uint32_t a, u16x2_t b) {
  return __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), b);
}
template <int N>
__device__ __forceinline__ uint32_t amax_of(const Pair<false>* x) {
  u16x2_t m = {0, 0};
#pragma unroll
  for (int k = 0; k < N; ++k) m = max_u16(x[k].magnitudes(), m);
  return static_cast<uint32_t>(max(m.x, m.y)) << 16;
}

// Four pairs to their codes, the first in the lowest four bits.  At random a
// seed serves both elements of a conversion, so each element takes one of its
// own, whose lowest byte is then its code (the other element is zero).  The
// bytes above it are not taken over from the operand that should hold them
// (seen in the code that hipcc 7.2 makes), so they are left out here.
template <bool RANDOM, bool F32>
__device__ __forceinline__ uint32_t codes8(const Pair<F32>* x, uint32_t e, const uint32_t* words) {
  const float scale = __uint_as_float(e << 23);
  uint32_t w = 0;
  if constexpr (!RANDOM) {
    w = x[0].template nearest<0>(w, scale);
    w = x[1].template nearest<1>(w, scale);
    w = x[2].template nearest<2>(w, scale);
    w = x[3].template nearest<3>(w, scale);
  } else {
    const auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {   // their lowest bytes
      return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
    };
    uint32_t a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = x[k].random_a(words[2 * k], scale);
      b[k] = x[k].random_b(words[2 * k + 1], scale);
    }
    w = four(a[0], a[1], a[2], a[3]) | (four(b[0], b[1], b[2], b[3]) << 4);
  }
  return e == 255u ? 0u : w;
}

// Random words: 16 consecutive elements of a row share a hash.
__device__ __forceinline__ uint32_t matrix_key(const RoundingSeed& seed, uint32_t index) {
  return mix(mix(mix(seed.lo) + seed.hi) + index);
}
__device__ __forceinline__ uint32_t group_hash(uint32_t key, uint32_t row, uint32_t col) {
  return mix(mix(key + row) + (col >> 4));
}

// Element (r, c) of a tile staged in LDS: the 32-row bands are turned by 32
// columns each, so that four threads that read a column in the four bands do
// not meet in a bank.
__device__ __forceinline__ int turned(int r, int c) { return r * kTile + ((c + (r & ~31)) & (kTile - 1)); }

// The hash of row r's 16 columns g of a tile: a column's rows follow each other,
// and the four bands, and the eight groups, begin in different banks: a quarter
// of the LDS reads that they take row by row, and none of the conflicts (4099 x
// 1025 bf16 at random along the columns 7.1 -> 6.9 us).
constexpr int kHashPitch = kTile + 12;
__device__ __forceinline__ int hash_at(int r, int g) { return g * kHashPitch + r + (r >> 5) * 4; }

// Four threads have the elements of a block.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xF, 0xF, true)));   // lanes 1 0 3 2
  return max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xF, 0xF, true)));  // 2 3 0 1
}

// Four blocks' scale bytes as one word, in the first of the lanes that hold
// them: a row's sixteen, of which each four hold a block's, and a quad.
__device__ __forceinline__ uint32_t e4_of_row(uint32_t e) {
  e |= static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(e), 0x104, 0xF, 0xF, true)) << 8;    // lane + 4
  return e | static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(e), 0x108, 0xF, 0xF, true)) << 16;   // lane + 8
}
__device__ __forceinline__ uint32_t e4_of_quad(uint32_t e) {
  e |= static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(e), 0xB1, 0xF, 0xF, true)) << 8;     // lanes 1 0 3 2
  return e | static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(e), 0x4E, 0xF, 0xF, true)) << 16;    // 2 3 0 1
}

// Eight elements of a row.
template <bool F32>
struct Chunk {
  static constexpr int N = F32 ? 2 : 1;
  raw_t<F32> w[N];
  template <bool STREAM>
  __device__ __forceinline__ void load(const Mx4Dev& m, int r, int c) {
    const auto* p = static_cast<const typename std::conditional<F32, float, uint16_t>::type*>(m.values) + r * m.ld + c;
#pragma unroll
    for (int k = 0; k < N; ++k)
      w[k] = STREAM ? __builtin_nontemporal_load((const MUON_GLOBAL raw_t<F32>*)(p + 4 * k)) : gld<raw_t<F32>>(p + 4 * k);
  }
  // Where the row may end in them.  No branch, so that the loads of all passes
  // are on their way together: the row's last eight elements, whose first
  // `skip` ones belong before these, and then the shift; rows shorter than
  // eight element by element.
  __device__ __forceinline__ void load_last(const Mx4Dev& m, int r, int c) { load<false>(m, r, min(c, m.cols - 8)); }
  __device__ __forceinline__ void shift(int skip) {
    constexpr int per = F32 ? 1 : 2;             // elements of a word
    uint32_t v[4 * N];
#pragma unroll
    for (int k = 0; k < 4 * N; ++k) v[k] = w[k >> 2][k & 3];
#pragma unroll
    for (int by = 4; by >= per; by >>= 1)
#pragma unroll
      for (int k = 0; k < 4 * N; ++k) {
        const uint32_t from = k + by / per < 4 * N ? v[k + by / per] : 0u;
        v[k] = skip & by ? from : v[k];
      }
    if constexpr (!F32)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = skip & 1 ? __builtin_amdgcn_alignbit(k < 3 ? v[k + 1] : 0u, v[k], 16) : v[k];
#pragma unroll
    for (int k = 0; k < 4 * N; ++k) w[k >> 2][k & 3] = skip < 8 ? v[k] : 0u;
  }
  __device__ __forceinline__ void load_short(const Mx4Dev& m, int r, int c) {
    using E = typename std::conditional<F32, uint32_t, uint16_t>::type;
    const E* const p = static_cast<const E*>(m.values) + r * m.ld;
    uint32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = gld<E>(p + min(c + k, m.cols - 1));
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (c + k >= m.cols) v[k] = 0u;
      if (F32) w[k >> 2][k & 3] = v[k];
      else if (k & 1) w[0][k >> 1] = v[k - 1] | (v[k] << 16);
    }
  }
  __device__ __forceinline__ void pairs(Pair<F32>* x) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (F32) x[k] = {__uint_as_float(w[k >> 1][2 * (k & 1)]), __uint_as_float(w[k >> 1][2 * (k & 1) + 1])};
      else x[k].ab = w[0][k];
    }
  }
};

// STREAM: the values are loaded without keeping them in the caches.
template <bool F32, bool ROW, bool COL, bool RANDOM, bool STREAM>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const Mx4List l, const RoundingSeed seed) {
  using E = typename std::conditional<F32, uint32_t, uint16_t>::type;
  __shared__ __attribute__((aligned(16))) E smem[COL ? kTile * kTile : 8];
  __shared__ __attribute__((aligned(16))) uint32_t hashes[COL && RANDOM ? kTile / 16 * kHashPitch : 1];
  const Tile t = find_tile(l);
  const Mx4Dev& m = t.m;
  const int q = threadIdx.x % kChunks, rq = threadIdx.x / kChunks;
  const int c = t.c0 + q * 8;
  const uint32_t key = RANDOM ? matrix_key(seed, m.index) : 0u;
  // all loads first; rows behind the last one take its elements, and are left out below
  Chunk<F32> x[kPasses];
  if (t.c0 + kTile <= m.cols) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) x[p].template load<STREAM>(m, min(t.r0 + rq + p * kRows, m.rows - 1), c);
  } else if (m.cols >= 8) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) x[p].load_last(m, min(t.r0 + rq + p * kRows, m.rows - 1), c);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) x[p].shift(max(c - (m.cols - 8), 0));
  } else {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) x[p].load_short(m, min(t.r0 + rq + p * kRows, m.rows - 1), c);
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int lr = rq + p * kRows, r = t.r0 + lr;
    uint32_t hash = 0;
    if constexpr (RANDOM) hash = group_hash(key, r, c);
    if constexpr (ROW) {
      Pair<F32> v[4];
      x[p].pairs(v);
      uint32_t words[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) words[k] = RANDOM ? hash + ((c & 8) + k) * kGolden : 0u;
      const uint32_t e = scale_byte(quad_max(amax_of<4>(v)));
      const uint32_t w = codes8<RANDOM, F32>(v, e, words);
      if (r < m.rows && (c & ~31) < m.cols) {
        gst(m.row.codes + static_cast<size_t>(r) * m.row_ld16 * 16 + (c >> 1), w);
        uint8_t* const to = m.row.scales + static_cast<size_t>(r) * m.row_ld4 * 4 + (c >> 5);
        if (t.c0 + kTile - kMx4Block < m.cols) {
          const uint32_t four = e4_of_row(e);
          if (q == 0) gst(to, four);
        } else if ((q & 3) == 0) {
          gst(to, static_cast<uint8_t>(e));
        }
      }
    }
    if constexpr (COL) {
      const bool real = r < m.rows;              // zeros behind the last row
#pragma unroll
      for (int k = 0; k < Chunk<F32>::N; ++k)
        *reinterpret_cast<u32x4_t*>(smem + turned(lr, q * 8) + 4 * k) = real ? u32x4_t(x[p].w[k]) : u32x4_t{0u, 0u, 0u, 0u};
      if constexpr (RANDOM)
        if ((q & 1) == 0) hashes[hash_at(lr, q >> 1)] = hash;
    }
  }
  if constexpr (COL) {
    __syncthreads();
    // four neighbouring threads take the four blocks of two columns, 64 bytes of each line
    const int band = threadIdx.x & 3, lc = (threadIdx.x >> 2) * 2;
    const int r = t.r0 + band * 32, cc = t.c0 + lc;
    if (cc >= m.cols || r >= m.rows) return;
    Pair<F32> v[2][16];                          // of each column, two rows
    uint32_t amax[2];
    if constexpr (F32) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(smem + turned(band * 32 + k, lc));
#pragma unroll
        for (int s = 0; s < 2; ++s) (k & 1 ? v[s][k >> 1].b : v[s][k >> 1].a) = __uint_as_float(w[s]);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) amax[s] = amax_of<16>(v[s]);
    } else {
      u16x2_t big = {0, 0};
#pragma unroll
      for (int k = 0; k < 32; k += 2) {
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(smem + turned(band * 32 + k, lc));
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(smem + turned(band * 32 + k + 1, lc));
        big = max_u16(w1 & 0x7FFF7FFFu, max_u16(w0 & 0x7FFF7FFFu, big));
        v[0][k >> 1].ab = __builtin_amdgcn_perm(w1, w0, 0x05040100u);
        v[1][k >> 1].ab = __builtin_amdgcn_perm(w1, w0, 0x07060302u);
      }
      amax[0] = static_cast<uint32_t>(big.x) << 16;
      amax[1] = static_cast<uint32_t>(big.y) << 16;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (cc + s >= m.cols) return;
      const uint32_t e = scale_byte(amax[s]);
      u32x4_t w;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t words[8];
        u32x4_t hash[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          hash[k] = RANDOM ? *reinterpret_cast<const u32x4_t*>(hashes + (RANDOM ? hash_at(band * 32 + g * 8 + k * 4, lc >> 4) : 0))
                           : u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; ++k) words[k] = RANDOM ? hash[k >> 2][k & 3] + ((lc & 15) + s) * kGolden : 0u;
        w[g] = codes8<RANDOM, F32>(v[s] + g * 4, e, words);
      }
      gst(m.col.codes + (static_cast<size_t>(cc + s) * m.col_ld16 + (r >> 5)) * 16, w);
      uint8_t* const to = m.col.scales + static_cast<size_t>(cc + s) * m.col_ld4 * 4 + (r >> 5);
      if (t.r0 + kTile - kMx4Block < m.rows) {
        const uint32_t four = e4_of_quad(e);
        if (band == 0) gst(to, four);
      } else {
        gst(to, static_cast<uint8_t>(e));
      }
    }
  }
}

// Elements of a row that a thread writes: 16 bytes, so that a wave's store is
// whole cache lines.
template <bool F32> constexpr int kWidth = F32 ? 4 : 8;

// Codes of kWidth elements (the lowest bits of w) to their 16 bytes.
template <bool F32>
__device__ __forceinline__ u32x4_t decode(uint32_t w, uint32_t e) {
  const float scale = __uint_as_float(e << 23);
  if constexpr (F32) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
    return u32x4_t{__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y)};
  } else {
    return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
  }
}

// STREAM: past the caches, as the values are not read again here (246 M bf16
// elements 87 us, 148 not, over and over into the same buffer; into one after
// another 115); mx4_back_streams has the rule by size.  Not for rows that do not
// begin at multiples of 16 bytes (65536 x 1601 bf16: 81 us streamed, 40 not).
template <bool F32, bool STREAM>
__device__ __forceinline__ void store_values(const Mx4Dev& m, int r, int c, const u32x4_t& w) {
  using E = typename std::conditional<F32, uint32_t, uint16_t>::type;
  E* const p = static_cast<E*>(m.values) + r * m.ld + c;
  if (c + kWidth<F32> <= m.cols) {
    if constexpr (STREAM) __builtin_nontemporal_store(raw_t<F32>(w), (MUON_GLOBAL raw_t<F32>*)p);
    else gst(p, raw_t<F32>(w));
    return;
  }
#pragma unroll
  for (int k = 0; k < kWidth<F32>; ++k)
    if (c + k < m.cols) gst(p + k, static_cast<E>(F32 ? w[k & 3] : w[k >> 1] >> (16 * (k & 1))));
}

template <bool F32, int AXIS, bool STREAM>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const Mx4List l) {
  using E = typename std::conditional<F32, uint32_t, uint16_t>::type;
  constexpr int W = kWidth<F32>, across = kTile / W, rows = kThreads / across, passes = kTile / rows;
  __shared__ __attribute__((aligned(16))) E smem[AXIS == 0 ? kTile * kTile : 8];
  const Tile t = find_tile(l);
  const Mx4Dev& m = t.m;
  const int q = threadIdx.x % across, rq = threadIdx.x / across;
  const int c = t.c0 + q * W;
  if constexpr (AXIS == 1) {
    if (c >= m.cols) return;
    uint32_t w[passes], e[passes];
#pragma unroll
    for (int p = 0; p < passes; ++p) {
      const size_t r = min(t.r0 + rq + p * rows, m.rows - 1);
      const uint8_t* const at = m.row.codes + r * m.row_ld16 * 16 + (c >> 1);
      w[p] = F32 ? gld<uint16_t>(at) : gld<uint32_t>(at);
      e[p] = gld<uint8_t>(m.row.scales + r * m.row_ld4 * 4 + (c >> 5));
    }
#pragma unroll
    for (int p = 0; p < passes; ++p) {
      const int r = t.r0 + rq + p * rows;
      if (r < m.rows) store_values<F32, STREAM>(m, r, c, decode<F32>(w[p], e[p]));
    }
    return;
  }
  // two columns' blocks of a band each
  const int band = threadIdx.x & 3, lc = (threadIdx.x >> 2) * 2, r0 = t.r0 + band * 32, cc = t.c0 + lc;
  if (cc < m.cols && r0 < m.rows) {
    u32x4_t w[2];
    float scale[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const size_t line = min(cc + s, m.cols - 1);
      w[s] = gld<u32x4_t>(m.col.codes + (line * m.col_ld16 + (r0 >> 5)) * 16);
      scale[s] = __uint_as_float(static_cast<uint32_t>(gld<uint8_t>(m.col.scales + line * m.col_ld4 * 4 + (r0 >> 5))) << 23);
    }
    const auto two = [&](auto gc, auto kc) {     // rows 8g + 2k and the next
      constexpr int g = decltype(gc)::value, k = decltype(kc)::value, lr = 8 * g + 2 * k;
      E* const at = smem + turned(band * 32 + lr, lc);
      if constexpr (F32) {
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0][g], scale[0], k);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[1][g], scale[1], k);
        *reinterpret_cast<u32x2_t*>(at) = u32x2_t{__float_as_uint(a.x), __float_as_uint(b.x)};
        *reinterpret_cast<u32x2_t*>(at + kTile) = u32x2_t{__float_as_uint(a.y), __float_as_uint(b.y)};
      } else {
        const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0][g], scale[0], k));
        const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[1][g], scale[1], k));
        *reinterpret_cast<uint32_t*>(at) = __builtin_amdgcn_perm(b, a, 0x05040100u);
        *reinterpret_cast<uint32_t*>(at + kTile) = __builtin_amdgcn_perm(b, a, 0x07060302u);
      }
    };
    const auto word = [&](auto gc) {
      two(gc, std::integral_constant<int, 0>{});
      two(gc, std::integral_constant<int, 1>{});
      two(gc, std::integral_constant<int, 2>{});
      two(gc, std::integral_constant<int, 3>{});
    };
    word(std::integral_constant<int, 0>{});
    word(std::integral_constant<int, 1>{});
    word(std::integral_constant<int, 2>{});
    word(std::integral_constant<int, 3>{});
  }
  __syncthreads();
  if (c >= m.cols) return;
#pragma unroll
  for (int p = 0; p < passes; ++p) {
    const int lr = rq + p * rows, r = t.r0 + lr;
    if (r < m.rows) store_values<F32, STREAM>(m, r, c, *reinterpret_cast<const u32x4_t*>(smem + turned(lr, q * W)));
  }
}

template <bool F32, bool RANDOM, bool STREAM>
hipError_t launch_forms(const Mx4List& l, const RoundingSeed& seed, hipStream_t s) {
  const bool row = l.m[0].row.codes != nullptr, col = l.m[0].col.codes != nullptr;
  const auto kernel = row && col ? quantize_kernel<F32, true, true, RANDOM, STREAM>
                      : row      ? quantize_kernel<F32, true, false, RANDOM, STREAM>
                                 : quantize_kernel<F32, false, true, RANDOM, STREAM>;
  kernel<<<l.tiles, kThreads, 0, s>>>(l, seed);
  return hipGetLastError();
}
template <bool F32>
hipError_t launch_rounding(const Mx4List& l, bool random, const RoundingSeed& seed, hipStream_t s) {
  const bool stream = mx4_round_streams(l, F32);
  if (random) return stream ? launch_forms<F32, true, true>(l, seed, s) : launch_forms<F32, true, false>(l, seed, s);
  return stream ? launch_forms<F32, false, true>(l, seed, s) : launch_forms<F32, false, false>(l, seed, s);
}

}  // namespace

hipError_t launch_mx4_quantize(const Mx4List& l, bool f32, bool random, RoundingSeed seed, hipStream_t s) {
  return f32 ? launch_rounding<true>(l, random, seed, s) : launch_rounding<false>(l, random, seed, s);
}

hipError_t launch_mx4_dequantize(const Mx4List& l, bool f32, int axis, bool aligned, hipStream_t s) {
  const bool stream = aligned && mx4_back_streams(l, f32);
  const auto of = [&](auto k) {
    constexpr bool F32 = decltype(k)::value;
    return axis ? (stream ? dequantize_kernel<F32, 1, true> : dequantize_kernel<F32, 1, false>)
                : (stream ? dequantize_kernel<F32, 0, true> : dequantize_kernel<F32, 0, false>);
  };
  const auto kernel = f32 ? of(std::true_type{}) : of(std::false_type{});
  kernel<<<l.tiles, kThreads, 0, s>>>(l);
  return hipGetLastError();
}

}  // namespace muon
