// Second moment of activations held in microscaled 4-bit floats, X^T X for n
// samples of d features, in blocks of 32 samples of one feature (the form that
// a weight gradient's product takes): line i of the codes is feature i, its
// blocks follow each other, so both operands of
//     (X^T X)[i][j] = sum over samples of x_i x_j
// are K-contiguous, and the matrix cores take codes and scales as they are
// (v_mfma_scale_f32_32x32x64_f8f6f4: a lane holds the 32 samples of one block of
// one feature, 16 bytes, and its scale).  Products of two codes and their scales
// are exact in float32; the sums are float32.
//
// Upper tiles only, stored both ways.  The order of a block's samples in the
// sum is of no matter as long as both operands keep to it, so the lanes of
// group g (lane / 32) take the blocks 4g .. 4g+3 of a 256-sample stage one after
// another: their four scales are then one aligned word, of which each matrix
// instruction names a byte.
#include <type_traits>

#include "device_common.h"
#include "muon_internal.h"

namespace muon {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kTile = 128;                     // output tile
constexpr int kStageBlocks = 8;                // blocks of a stage: 256 samples
constexpr int kBand = 32;                      // matrix instruction: 32 x 32 of the output
constexpr int kBands = kTile / 2 / kBand;      // each of 2 x 2 waves: 64 x 64
constexpr int kSlab = kTile * kTile;           // partial sums of a tile

__device__ __forceinline__ int swizzled(int row, int c) { return c ^ ((row >> 1) & 7); }

// Upper tile number t of nt x nt tiles.
__device__ __forceinline__ void upper_tile(int t, int nt, int& ti, int& tj) {
  ti = 0;
  while (t >= nt - ti) { t -= nt - ti; ++ti; }
  tj = ti + t;
}

// Four rows gr.. of column gc of the product: S = sum / n + damping (the padded
// diagonal 1), or, accumulating, S = beta S + sum; stored both ways, but for
// the tiles on the diagonal, which hold both halves.
__device__ __forceinline__ void finish4(const Mx4MomentParams& p, int gr, int gc, bool mirror, const f32x4_t& sum) {
  f32x4_t v;
  float* const at = p.out + static_cast<size_t>(gr) * p.dp + gc;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool inside = gr + e < p.d && gc < p.d;
    if (p.accumulate) {
      const float s = inside ? sum[e] : 0.f;
      v[e] = p.beta != 0.0 ? static_cast<float>(fma(p.beta, static_cast<double>(gld<float>(at + static_cast<size_t>(e) * p.dp)),
                                                    static_cast<double>(s)))
                           : s;
    } else {
      v[e] = inside ? sum[e] * p.inv_n : 0.f;
      if (gr + e == gc) v[e] = gc < p.d ? v[e] + p.damping : 1.0f;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) gst(at + static_cast<size_t>(e) * p.dp, v[e]);
  if (mirror) gst(p.out + static_cast<size_t>(gc) * p.dp + gr, v);
}

__device__ __forceinline__ void count_samples(const Mx4MomentParams& p) {
  if (p.cnt && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    *p.cnt = p.beta * *p.cnt + static_cast<double>(p.n_rows);
}

// One tile over one range of stages (blockIdx.y).
__global__ __launch_bounds__(kThreads) void moment_kernel(const Mx4MomentParams p) {
  __shared__ __attribute__((aligned(16))) u32x4_t codes[2][kTile * kStageBlocks];
  __shared__ uint32_t scales[2][kTile * 2];
  int ti, tj;
  upper_tile(blockIdx.x, p.dp / kTile, ti, tj);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1, group = lane >> 5, lr = lane & 31;
  const int64_t blocks = (p.n_rows + kMx4Block - 1) / kMx4Block;
  const int tail = static_cast<int>(p.n_rows % kMx4Block);       // samples of the last block, 0: all
  const int64_t s0 = blockIdx.y * p.stages, s_all = (blocks + kStageBlocks - 1) / kStageBlocks;
  const int64_t s1 = s0 + p.stages < s_all ? s0 + p.stages : s_all;
  f32x16_t acc[kBands][kBands];
#pragma unroll
  for (int i = 0; i < kBands; ++i)
#pragma unroll
    for (int j = 0; j < kBands; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  for (int64_t s = s0; s < s1; ++s) {
    __syncthreads();
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const int f0 = (o ? tj : ti) * kTile;
      for (int k = tid; k < kTile * kStageBlocks; k += kThreads) {
        const int row = k / kStageBlocks, c = k % kStageBlocks;
        const int64_t b = s * kStageBlocks + c;
        const int f = min(f0 + row, p.d - 1);
        u32x4_t w = {0u, 0u, 0u, 0u};
        if (b < blocks) w = gld<u32x4_t>(p.codes + f * p.ld_codes + b * 16);
        if (b == blocks - 1 && tail)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int keep = tail - 8 * g;       // elements of this word that are samples
            w[g] &= keep >= 8 ? ~0u : keep <= 0 ? 0u : (1u << (4 * keep)) - 1u;
          }
        codes[o][row * kStageBlocks + swizzled(row, c)] = w;
      }
      for (int k = tid; k < kTile * 2; k += kThreads) {
        const int row = k / 2;
        const int64_t b = s * kStageBlocks + (k % 2) * 4;
        const int f = min(f0 + row, p.d - 1);
        uint32_t e = 0;
        if (b < blocks) e = gld<uint32_t>(p.scales + f * p.ld_scales + b);
        if (b + 4 > blocks && b < blocks) e &= (1u << (8 * static_cast<int>(blocks - b))) - 1u;
        scales[o][k] = e;
      }
    }
    __syncthreads();
    uint32_t ea[kBands], eb[kBands];
#pragma unroll
    for (int i = 0; i < kBands; ++i) {
      ea[i] = scales[0][(wm * 64 + i * kBand + lr) * 2 + group];
      eb[i] = scales[1][(wn * 64 + i * kBand + lr) * 2 + group];
    }
    const auto step = [&](auto ic) {
      constexpr int k = decltype(ic)::value;
      i32x8_t a[kBands], b[kBands];
#pragma unroll
      for (int i = 0; i < kBands; ++i) {
        const int ra = wm * 64 + i * kBand + lr, rb = wn * 64 + i * kBand + lr;
        const u32x4_t x = codes[0][ra * kStageBlocks + swizzled(ra, group * 4 + k)];
        const u32x4_t y = codes[1][rb * kStageBlocks + swizzled(rb, group * 4 + k)];
        a[i] = i32x8_t{int(x[0]), int(x[1]), int(x[2]), int(x[3]), 0, 0, 0, 0};
        b[i] = i32x8_t{int(y[0]), int(y[1]), int(y[2]), int(y[3]), 0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < kBands; ++i)
#pragma unroll
        for (int j = 0; j < kBands; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[i], b[j], acc[i][j], 4, 4, k, ea[i], k, eb[j]);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }
  // lane l, register 4q + e of a band: row 8q + 4(l/32) + e, column l % 32
  float* const part = p.part ? p.part + (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kSlab : nullptr;
#pragma unroll
  for (int i = 0; i < kBands; ++i)
#pragma unroll
    for (int j = 0; j < kBands; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if (part)
          gst(part + (((wave * kBands + i) * kBands + j) * 4 + q) * 256 + lane * 4, v);
        else
          finish4(p, ti * kTile + wm * 64 + i * kBand + 8 * q + 4 * group, tj * kTile + wn * 64 + j * kBand + lr, ti != tj, v);
      }
  if (!part) count_samples(p);
}

// The ranges' partial sums, added in their order; a thread takes four rows of
// one column, in the order in which the waves stored them.
__global__ __launch_bounds__(kThreads) void reduce_kernel(const Mx4MomentParams p, int tiles, int splits) {
  const int per = kSlab / 4 / kThreads;          // thread blocks of a tile
  const int tile = blockIdx.x / per, at = (blockIdx.x % per) * kThreads + threadIdx.x;
  int ti, tj;
  upper_tile(tile, p.dp / kTile, ti, tj);
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s)
    sum += gld<f32x4_t>(p.part + (static_cast<size_t>(s) * tiles + tile) * kSlab + at * 4);
  const int lane = at & 63, q = (at >> 6) & 3, j = (at >> 8) & 1, i = (at >> 9) & 1, wn = (at >> 10) & 1, wm = at >> 11;
  finish4(p, ti * kTile + wm * 64 + i * kBand + 8 * q + 4 * (lane >> 5), tj * kTile + wn * 64 + j * kBand + (lane & 31),
          ti != tj, sum);
  count_samples(p);
}

}  // namespace

hipError_t launch_mx4_moment(Mx4MomentParams p, size_t part_floats, hipStream_t s) {
  const int nt = p.dp / kTile, tiles = nt * (nt + 1) / 2;
  const int64_t blocks = (p.n_rows + kMx4Block - 1) / kMx4Block, all = (blocks + kStageBlocks - 1) / kStageBlocks;
  int64_t splits = p.part ? static_cast<int64_t>(part_floats / (static_cast<size_t>(tiles) * kSlab)) : 1;
  splits = splits < 512 / tiles ? splits : 512 / tiles;
  splits = splits < all ? splits : all;
  if (splits < 1) splits = 1;
  p.stages = (all + splits - 1) / splits;
  splits = (all + p.stages - 1) / p.stages;      // those that hold stages
  if (splits == 1) p.part = nullptr;
  moment_kernel<<<dim3(tiles, static_cast<unsigned>(splits)), kThreads, 0, s>>>(p);
  if (p.part) reduce_kernel<<<tiles * (kSlab / 4 / kThreads), kThreads, 0, s>>>(p, tiles, static_cast<int>(splits));
  return hipGetLastError();
}

}  // namespace muon
