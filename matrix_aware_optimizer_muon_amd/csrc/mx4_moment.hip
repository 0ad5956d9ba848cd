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
// group g (lane / 32) take neighbouring blocks one after another: their scales
// are then bytes of one word, of which each matrix instruction names one.
//
// Four ways, by size (launch_mx4_moment):
//   bands   few samples: a wave takes 32 x 32 of the output and loads its
//           operands from memory; as many waves as there are bands.  Bound by
//           its launch and two trips to memory: 64 samples of 768 features 4.9
//           us, where the sums' 4.7 MB take 1
//   64      tiles of 64 x 64, 4 waves of 32 x 32, four blocks a CU: many CUs at
//           work on little.  Bound by a trip to memory a stage: 4096 samples of
//           1025 features 10 us (14 from no cache); 5003 of them 15, 10 without
//           the loop's loads
//   128     tiles of 128 x 128, 4 waves of 64 x 64, two blocks a CU.  Bound by
//           its loads: 65536 samples of 4096 features 315 us, 280 without the
//           products (4.7 GB of operands, 66 GB/s a CU), 206 without the loads
//   256     tiles of 256 x 256, 8 waves of 128 x 64, one block a CU: half the
//           operand bytes a product.  Bound by loads and products alike: 65536
//           samples of 6400 features 638 us, 4.4 PFLOP/s of the whole tiles'
//           products; 526 without the loads, at 1.6 GHz, the clock under this
//           load, and 613 without the products
// Tiles that would leave CUs idle are cut into ranges of samples, whose partial
// sums a second launch adds in order.
// For the last of these, when it took 684 us: stages of 128 samples (half a cache
// line a load, four stages in LDS) 750, scales loaded 4 bytes a line and stage
// 920, 8 bytes 757.
#include <algorithm>
#include <cmath>

#include "device_common.h"
#include "lds_ring.h"
#include "muon_internal.h"

namespace muon {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kStageBlocks = 8;                // blocks of a stage: 256 samples, a line's 128 bytes (one cache line)
constexpr int kStages = 2;                     // in LDS: one is read, one on its way
constexpr int kGroup = 4;                      // stages whose scales are loaded together, 32 bytes a line
constexpr int kBand = 32;                      // a matrix instruction's part of the output, 32 x 32
constexpr int kCUs = 256;

// Tiles of BT x BT: WM x WN waves, each of NA x NB bands.
template <int BT_, int WM_, int WN_>
struct Cfg {
  static constexpr int BT = BT_, WM = WM_, WN = WN_, WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int NA = BT / WM / kBand, NB = BT / WN / kBand;
  static constexpr int SLAB = BT * BT;                     // partial sums of a tile
  static constexpr int CODES = 2 * BT * kStageBlocks * 16; // bytes of a stage's codes, both operands
  static constexpr int SCALES = 2 * BT * kGroup * kStageBlocks;   // of a group's scales
  static constexpr int LDS = kStages * CODES + 2 * SCALES;
  static constexpr int BLOCKS = (160 << 10) / LDS;         // of a CU: 4, 2, 1
  static constexpr int LOADS = CODES / 2 / 16 / THREADS;   // 16 bytes a lane, one operand
  static constexpr int SCALE_WAVES = SCALES / 2 / 1024;    // whose one load fills a group's scales of one operand
  static_assert(WAVES == SCALE_WAVES || WAVES == 2 * SCALE_WAVES, "all waves load scales, of one operand or of both");
};
using Cfg64 = Cfg<64, 2, 2>;
using Cfg128 = Cfg<128, 2, 2>;
using Cfg256 = Cfg<256, 2, 4>;

// Upper tile number t of nt x nt tiles, in strips of four tile rows, down the
// strip's columns: neighbours in this order share rows and columns.
__device__ __forceinline__ void upper_tile(int t, int nt, int& ti, int& tj) {
  int r0 = 0, h;
  for (;; r0 += 4) {
    h = min(4, nt - r0);
    const int in_strip = h * (nt - r0) - h * (h - 1) / 2;
    if (t < in_strip) break;
    t -= in_strip;
  }
  const int corner = h * (h + 1) / 2;            // columns r0 .. r0+h-1 have 1 .. h tiles
  if (t < corner) {
    int c = 0;
    while (t > c) { t -= c + 1; ++c; }
    ti = r0 + t;
    tj = r0 + c;
  } else {
    ti = r0 + (t - corner) % h;
    tj = r0 + h + (t - corner) / h;
  }
}

// Four rows gr.. of column gc of the product: S = sum / n + damping (the padded
// diagonal 1), or, accumulating, S = beta S + sum; stored both ways, but for
// the tiles on the diagonal, which hold both halves.
__device__ __forceinline__ bool reads_old(const Mx4MomentParams& p) { return p.accumulate && p.beta != 0.0; }
__device__ __forceinline__ f32x4_t load_old4(const Mx4MomentParams& p, int gr, int gc) {
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (reads_old(p))
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = gld<float>(p.out + static_cast<size_t>(gr + e) * p.dp + gc);
  return v;
}
__device__ __forceinline__ void finish4(const Mx4MomentParams& p, int gr, int gc, bool mirror, const f32x4_t& sum,
                                        const f32x4_t& old) {
  f32x4_t v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool inside = gr + e < p.d && gc < p.d;
    if (p.accumulate) {
      const float s = inside ? sum[e] : 0.f;
      v[e] = p.beta != 0.0 ? static_cast<float>(fma(p.beta, static_cast<double>(old[e]), static_cast<double>(s))) : s;
    } else {
      v[e] = inside ? sum[e] * p.inv_n : 0.f;
      if (gr + e == gc) v[e] = gc < p.d ? v[e] + p.damping : 1.0f;
    }
  }
  float* const at = p.out + static_cast<size_t>(gr) * p.dp + gc;
#pragma unroll
  for (int e = 0; e < 4; ++e) gst(at + static_cast<size_t>(e) * p.dp, v[e]);
  if (mirror) gst(p.out + static_cast<size_t>(gc) * p.dp + gr, v);
}
// A lane's registers 4q .. 4q+3 of a band are rows 8q + 4 (lane / 32) .. of column lane % 32.
__device__ __forceinline__ f32x4_t quad(const f32x16_t& v, int q) {
  return f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
}

__device__ __forceinline__ void count_samples(const Mx4MomentParams& p) {
  if (p.cnt && blockIdx.x == 0 && threadIdx.x == 0)
    *p.cnt = (p.beta != 0.0 ? p.beta * *p.cnt : 0.0) + static_cast<double>(p.n_rows);
}

// k, a constant where it is called: the byte of each scale word.
__device__ __forceinline__ f32x16_t mma(const u32x4_t& a, const u32x4_t& b, const f32x16_t& c, uint32_t ea, uint32_t eb,
                                        int k) {
  const i32x8_t x = {int(a[0]), int(a[1]), int(a[2]), int(a[3]), 0, 0, 0, 0};
  const i32x8_t y = {int(b[0]), int(b[1]), int(b[2]), int(b[3]), 0, 0, 0, 0};
  // format 4 is e2m1
  switch (k) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 0, int(ea), 0, int(eb));
    case 1: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 1, int(ea), 1, int(eb));
    case 2: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 2, int(ea), 2, int(eb));
    default: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 3, int(ea), 3, int(eb));
  }
}

// One feature's line, with what lies behind the samples taken as zeros.
struct Line {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t blocks;
  int tail;                                      // samples of the last block, 0: all
  __device__ __forceinline__ Line(const Mx4MomentParams& p, int f)
      : codes(p.codes + min(f, p.d - 1) * p.ld_codes), scales(p.scales + min(f, p.d - 1) * p.ld_scales),
        blocks((p.n_rows + kMx4Block - 1) / kMx4Block), tail(static_cast<int>(p.n_rows % kMx4Block)) {}
  __device__ __forceinline__ u32x4_t block(int64_t b) const {
    u32x4_t w = {0u, 0u, 0u, 0u};
    if (b < blocks) w = gld<u32x4_t>(codes + b * 16);
    if (b == blocks - 1 && tail)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int keep = tail - 8 * g;           // elements of this word that are samples
        w[g] &= keep >= 8 ? ~0u : keep <= 0 ? 0u : (1u << (4 * keep)) - 1u;
      }
    return w;
  }
  __device__ __forceinline__ uint32_t scales4(int64_t b) const {   // b a multiple of 4
    if (b >= blocks) return 0u;
    const uint32_t e = gld<uint32_t>(scales + b);
    return b + 4 > blocks ? e & ((1u << (8 * static_cast<int>(blocks - b))) - 1u) : e;
  }
};

// ------------------------------------------------------------------ tiles

// One tile over one range of stages.  Blocks below p.whole take a tile each
// over all samples and finish it; the others take a range of a later tile,
// p.splits ranges a tile, and store its partial sums.
template <typename C>
__global__ __launch_bounds__(C::THREADS, C::BLOCKS) void tile_kernel(const Mx4MomentParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS];
  const int nt = (p.dp + C::BT - 1) / C::BT;
  const int b = blockIdx.x;
  // The blocks of one die (b % 8) take a run of neighbouring tiles, and of the
  // cut ones of the same range: what they read is shared in the die's cache.
  const auto die_run = [](int k, int n) {
    const int die = k % 8;
    return die * (n / 8) + min(die, n % 8) + k / 8;
  };
  const int cut = (gridDim.x - p.whole) / max(p.splits, 1);
  int t, split = 0, slab = 0;
  if (b < p.whole) {
    t = die_run(b, p.whole);
  } else {
    slab = die_run(b - p.whole, cut * p.splits);
    split = slab / cut;
    t = p.whole + slab % cut;
  }
  int ti, tj;
  upper_tile(t, nt, ti, tj);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN, group = lane >> 5, lr = lane & 31;
  const int64_t blocks = (p.n_rows + kMx4Block - 1) / kMx4Block;
  const int stages = static_cast<int>((blocks + kStageBlocks - 1) / kStageBlocks);
  const int s0 = b < p.whole ? 0 : split * p.stages, s1 = b < p.whole ? stages : min(s0 + p.stages, stages);
  if constexpr (MUON_DEBUG_BOUNDS) {
    const size_t floats = b < p.whole ? 0 : static_cast<size_t>(slab + 1) * C::SLAB;
    if (ti < 0 || ti > tj || tj >= nt || s0 < 0 || s0 >= s1 || s1 > stages || floats > p.part_floats) {
      if (tid == 0) atomicOr(p.flags, kFlagBounds);
      return;
    }
  }
  const int fa0 = ti * C::BT, fb0 = tj * C::BT;
  const int row_a = wm * (C::BT / C::WM) + lr, row_b = wn * (C::BT / C::WN) + lr;

  const int full = static_cast<int>(p.n_rows / (kStageBlocks * kMx4Block));   // stages that are whole, at least 2
  f32x16_t acc[C::NA][C::NB];
#pragma unroll
  for (int i = 0; i < C::NA; ++i)
#pragma unroll
    for (int j = 0; j < C::NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // LDS: two stages of codes (A's lines, then B's, 128 bytes each) and two
  // groups of four stages' scales (32 bytes a line; a load's cost is its cache
  // lines, so that 8 bytes a line and stage would take as long as the codes
  // do).  Chunk (block) c of line r lies at place c ^ (r / 2) % 8 of its 128
  // bytes: sixteen lines read at one chunk then cover the banks evenly.  The
  // two halves of a line's scales are exchanged in every other eight lines.
  struct Frags { u32x4_t a[C::NA], b[C::NB]; };
  struct Scales { uint32_t a[C::NA], b[C::NB]; };
  const uint32_t line_a = row_a * 128, line_b = C::CODES / 2 + row_b * 128;
  const auto read_frags = [&](int buf, int k) {   // step k: blocks k and 4 + k, by group
    const uint32_t at = buf * C::CODES + ((group * 4 + k) ^ ((lr >> 1) & 7)) * 16;
    const uint8_t *const a = smem + (line_a + at), *const b = smem + (line_b + at);
    Frags f;
#pragma unroll
    for (int i = 0; i < C::NA; ++i) f.a[i] = *reinterpret_cast<const u32x4_t*>(a + i * kBand * 128);
#pragma unroll
    for (int j = 0; j < C::NB; ++j) f.b[j] = *reinterpret_cast<const u32x4_t*>(b + j * kBand * 128);
    return f;
  };
  // First stage of the half group that stage s (s0 + k) belongs to: the last one of a line ends with its last whole stage.
  const auto half_start = [&](int k) { return min(s0 + (k & ~1), full - 2); };
  const auto read_scales = [&](int k) {           // of stage s0 + k, the four of the lane group's blocks
    const int in_half = (s0 + k - half_start(k)) & 1;
    const uint8_t* const at = smem + kStages * C::CODES + (k / kGroup & 1) * C::SCALES +
                              (((k >> 1 & 1) ^ ((lr >> 3) & 1)) * 16 + in_half * 8 + group * 4);
    Scales e;
#pragma unroll
    for (int i = 0; i < C::NA; ++i) e.a[i] = *reinterpret_cast<const uint32_t*>(at + (row_a + i * kBand) * 32);
#pragma unroll
    for (int j = 0; j < C::NB; ++j) e.b[j] = *reinterpret_cast<const uint32_t*>(at + C::SCALES / 2 + (row_b + j * kBand) * 32);
    return e;
  };
  const auto multiply = [&](const Frags& f, const Scales& e, int k) {
#pragma unroll
    for (int i = 0; i < C::NA; ++i)
#pragma unroll
      for (int j = 0; j < C::NB; ++j) acc[i][j] = mma(f.a[i], f.b[j], acc[i][j], e.a[i], e.b[j], k);
  };

  // The range as pairs of whole stages and what is left: at the most a whole stage and the last one, which may end
  // inside (its blocks behind the samples are loaded from the last block there is, and masked).
  const int pairs = (min(s1, full) - s0) / 2, left = s1 - s0 - 2 * pairs;
  const int last_blocks = static_cast<int>(blocks - static_cast<int64_t>(full) * kStageBlocks);
  const int last_samples = static_cast<int>(p.n_rows - static_cast<int64_t>(full) * (kStageBlocks * kMx4Block));
  Scales e_last;
  if (s1 > full) {
    const int64_t b0 = static_cast<int64_t>(full) * kStageBlocks + group * 4;
#pragma unroll
    for (int i = 0; i < C::NA; ++i) e_last.a[i] = Line(p, fa0 + row_a + i * kBand).scales4(b0);
#pragma unroll
    for (int j = 0; j < C::NB; ++j) e_last.b[j] = Line(p, fb0 + row_b + j * kBand).scales4(b0);
  }

  // Direct-to-LDS loads: 16 bytes a lane into consecutive places, so lane L of
  // load i of wave w fills place (i WAVES + w) 64 + L, line place / 8.  A stage's
  // loads are issued when every wave has read the stage before the last from
  // its buffer, ahead of the last step of that one's products, and waited for
  // a stage later.  Behind the last stage it is loaded again, for nobody: a
  // branch in the loop would let the compiler move the products below it.
  {
    // Eight lines a load: their first is the wave's own (a scalar base), a lane's
    // line and chunk the same in every load, but where the features end among them.
    const uint32_t chunk = ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) * 16;
    const uint32_t off = (lane >> 3) * static_cast<uint32_t>(p.ld_codes);
    const uint32_t off_end = min(lane >> 3, (p.d - 1) & 7) * static_cast<uint32_t>(p.ld_codes);
    const uint32_t lds0 = lds_addr(smem);
    constexpr int kLoads = 2 * C::LOADS;         // of a stage's codes, A's and B's
    const auto load_codes = [&](int k, int buf, int n) {
      const int s = min(s0 + k, s1 - 1);
      const uint32_t chunks = s == full ? (last_blocks - 1) * 16 : (kStageBlocks - 1) * 16;
      const int o = n / C::LOADS, i = n % C::LOADS, line = (o ? fb0 : fa0) + (i * C::WAVES + wave) * 8;
      dma16(p.codes + static_cast<size_t>(s) * (kStageBlocks * 16) + min(line, (p.d - 1) & ~7) * p.ld_codes,
            (line + 8 <= p.d ? off : off_end) + min(chunk, chunks),
            lds0 + buf * C::CODES + o * (C::CODES / 2) + (i * C::WAVES + wave) * 1024);
    };
    // A group's scales of one operand (64-tiles: of both, twice), 32 lines a load, two lanes a line.
    const bool second = ((lane ^ (lane >> 4)) & 1) != 0;
    const uint32_t off_e = (lane >> 1) * static_cast<uint32_t>(p.ld_scales);
    const uint32_t off_e_end = min(lane >> 1, (p.d - 1) & 31) * static_cast<uint32_t>(p.ld_scales);
    const auto load_scales = [&](int v, int of) {
      const int o = C::WAVES == C::SCALE_WAVES ? of : wave / C::SCALE_WAVES, part = wave % C::SCALE_WAVES;
      const int line = (o ? fb0 : fa0) + part * 32;
      const uint32_t half0 = half_start(kGroup * v) * kStageBlocks, half1 = half_start(kGroup * v + 2) * kStageBlocks;
      dma16(p.scales + min(line, (p.d - 1) & ~31) * p.ld_scales, (line + 32 <= p.d ? off_e : off_e_end) + (second ? half1 : half0),
            lds0 + kStages * C::CODES + (v & 1) * C::SCALES + o * (C::SCALES / 2) + part * 1024);
    };
    load_scales(0, 0);
    load_scales(0, 1);
#pragma unroll
    for (int k = 0; k < kStages; ++k)
#pragma unroll
      for (int n = 0; n < kLoads; ++n) load_codes(k, k, n);
    wait_vmcnt<0>();
    ring_barrier();
    Frags f[2];
    f[0] = read_frags(0, 0);
    Scales e_now = read_scales(0);
#pragma unroll 1
    for (int u = 0; u < pairs; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          f[(k + 1) & 1] = read_frags(h, k + 1);
          multiply(f[k & 1], e_now, k);
          __builtin_amdgcn_sched_barrier(0);
        }
        // the next stage has landed; this one has been read by every wave, so its buffer takes the one after it
        wait_vmcnt<0>();
        ring_barrier();
        const Scales e_then = e_now;
        const int next = 2 * u + h + 1;
        f[0] = read_frags(h ^ 1, 0);
        e_now = read_scales(next);               // (behind the last whole stage of no matter)
        if (h == 0) load_scales(u / 2 + 1, u & 1);   // the next group's, of A and then of B, into the buffer of the one before
        __builtin_amdgcn_sched_barrier(0);
        // the loads' issue between the products, which it would hold up
#pragma unroll
        for (int t = 0; t < C::NA * C::NB; ++t) {
          const int i = t / C::NB, j = t % C::NB;
          acc[i][j] = mma(f[1].a[i], f[1].b[j], acc[i][j], e_then.a[i], e_then.b[j], 3);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int n = t * kLoads / (C::NA * C::NB); n < (t + 1) * kLoads / (C::NA * C::NB); ++n)
            load_codes(next + 1, h, n);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    const auto rest = [&](int buf, int s) {
      const Scales e = s == full ? e_last : read_scales(s - s0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        Frags x = read_frags(buf, k);
        if (s == full) {
          u32x4_t keep;                          // of each word, the elements that are samples
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int n = last_samples - (group * 4 + k) * kMx4Block - 8 * g;
            keep[g] = n >= 8 ? ~0u : n <= 0 ? 0u : (1u << (4 * n)) - 1u;
          }
#pragma unroll
          for (int i = 0; i < C::NA; ++i) x.a[i] &= keep;
#pragma unroll
          for (int j = 0; j < C::NB; ++j) x.b[j] &= keep;
        }
        multiply(x, e, k);
      }
    };
    wait_vmcnt<0>();                             // (also: nothing is on its way to LDS when the block ends)
    ring_barrier();
    if (left > 0) rest(0, s0 + 2 * pairs);
    if (left > 1) rest(1, s0 + 2 * pairs + 1);
  }

  if (b >= p.whole) {
    float* const part = p.part + static_cast<size_t>(slab) * C::SLAB;
#pragma unroll
    for (int i = 0; i < C::NA; ++i)
#pragma unroll
      for (int j = 0; j < C::NB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          gst(part + (((wave * C::NA + i) * C::NB + j) * 4 + q) * 256 + lane * 4, quad(acc[i][j], q));
    return;
  }
#pragma unroll
  for (int i = 0; i < C::NA; ++i)
#pragma unroll
    for (int j = 0; j < C::NB; ++j) {
      const int gr = fa0 + wm * (C::BT / C::WM) + i * kBand + 4 * group, gc = fb0 + row_b + j * kBand;
      if (gr - 4 * group >= p.dp || gc - lr >= p.dp) continue;   // behind the last whole tile: dp is a multiple of 128
      f32x4_t old[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) old[q] = load_old4(p, gr + 8 * q, gc);
#pragma unroll
      for (int q = 0; q < 4; ++q) finish4(p, gr + 8 * q, gc, ti != tj, quad(acc[i][j], q), old[q]);
    }
  if (p.splits == 0) count_samples(p);
}

// The ranges' partial sums, added in their order; a thread takes four rows of
// one column, in the order in which the waves stored them.
template <typename C>
__global__ __launch_bounds__(256) void reduce_kernel(const Mx4MomentParams p) {
  constexpr int per = C::SLAB / 4 / 256;         // thread blocks of a tile
  const int tile = blockIdx.x / per, at = (blockIdx.x % per) * 256 + threadIdx.x;
  int ti, tj;
  upper_tile(p.whole + tile, (p.dp + C::BT - 1) / C::BT, ti, tj);
  const int lane = at & 63, q = (at >> 6) & 3, band = at >> 8;
  const int j = band % C::NB, i = band / C::NB % C::NA, wave = band / (C::NA * C::NB);
  const int gr = ti * C::BT + (wave / C::WN * C::NA + i) * kBand + 8 * q + 4 * (lane >> 5);
  const int gc = tj * C::BT + (wave % C::WN * C::NB + j) * kBand + (lane & 31);
  if (gr < p.dp && gc < p.dp) {
    const size_t next = static_cast<size_t>(gridDim.x / per) * C::SLAB;     // from a range to the next
    const float* const part = p.part + static_cast<size_t>(tile) * C::SLAB + at * 4;
    const f32x4_t old = load_old4(p, gr, gc);
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < p.splits; s += 8) {      // eight loads on their way, added in order
      f32x4_t x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = gld<f32x4_t>(part + min(s + k, p.splits - 1) * next);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (s + k < p.splits) sum += x[k];
    }
    finish4(p, gr, gc, ti != tj, sum, old);
  }
  count_samples(p);
}

// ------------------------------------------------------------------ bands

// A wave for 32 x 32 of the output: its operands from memory, no LDS.
__global__ __launch_bounds__(64) void band_kernel(const Mx4MomentParams p) {
  int bi = 0, bj = blockIdx.x;
  const int nb = p.dp / kBand;
  while (bj >= nb - bi) { bj -= nb - bi; ++bi; }
  bj += bi;
  const int lane = threadIdx.x, group = lane >> 5, lr = lane & 31;
  const Line a(p, bi * kBand + lr), b(p, bj * kBand + lr);
  const int gr = bi * kBand + 4 * group, gc = bj * kBand + lr;
  f32x4_t old[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) old[q] = load_old4(p, gr + 8 * q, gc);
  f32x16_t acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  for (int64_t at = 4 * group; at - 4 * group < a.blocks; at += 8) {   // four blocks of each group
    u32x4_t x[4], y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = a.block(at + k);
      y[k] = b.block(at + k);
    }
    const uint32_t ex = a.scales4(at), ey = b.scales4(at);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc = mma(x[k], y[k], acc, ex, ey, k);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) finish4(p, gr + 8 * q, gc, bi != bj, quad(acc, q), old[q]);
  count_samples(p);
}

// How the tiles of a launch are cut: whole rounds of the chip take whole tiles,
// and each of the `left` others is taken in as many ranges as make the time
// least, within one more round and the room for partial sums.
struct Cut { int whole, splits, stages; double us; };

// The time in us, fitted to measurements on activations that are in no die's
// cache: a stage of a tile, by how crowded the CUs are (alone it waits for
// memory, of 64-tiles a second block is nearly free); a launch that ends in whole
// tiles, and each of them; with ranges, two launches and each range's partial
// sums, written and read; a round before the last.  Fitted to half of 115 sizes
// of 512 to 65536 samples of 64 to 6400 features, each with tiles of 64 and 128
// whole and in up to 24 ranges: on all of them the way taken is within 5.2 % of the
// best one measured, 0.9 % on average.  From a die's cache fewer ranges of smaller
// tiles would often be faster (8192 samples of 1025 features 18.7 us for 15.0).
template <int BT> struct Cost;
template <> struct Cost<64> { static constexpr double stage = 0.55, one = 3.5, tile = 0.0035, two = 6.0, sum = 0.0101, round = 0; };
template <> struct Cost<128> { static constexpr double stage = 0.81, one = 6.9, tile = 0.0168, two = 6.6, sum = 0.0288, round = 10.7; };
template <> struct Cost<256> { static constexpr double stage = 2.0, one = 3.5, tile = 0, two = 4.0, sum = 0.12, round = 0; };
template <int BT>
double crowded(int blocks) {
  if (blocks <= kCUs) return 1.0;
  const double each = static_cast<double>(blocks) / kCUs;
  return BT == 64 ? std::max(1.0, 0.62 * (each + std::ceil(each)) / 2) : 1.21 + 0.26 * (each - 1.0);
}
template <typename C>
Cut cut_tiles(const Mx4MomentParams& p, int stages) {
  using T = Cost<C::BT>;
  constexpr int slots = kCUs * C::BLOCKS;
  const int nt = (p.dp + C::BT - 1) / C::BT, tiles = nt * (nt + 1) / 2, left = tiles % slots, rounds = tiles / slots;
  const double before = rounds * (stages * T::stage * crowded<C::BT>(slots) + T::round);
  Cut best = {tiles, 0, 0, before + T::one + T::tile * tiles + (left ? stages * T::stage * crowded<C::BT>(left) : 0.0)};
  if (!left || !p.part) return best;
  const int64_t fit = static_cast<int64_t>(p.part_floats / (static_cast<size_t>(left) * C::SLAB));
  const int most = static_cast<int>(std::min<int64_t>(std::min(slots / left, (stages + 1) / 2), fit));
  for (int k = 2; k <= most; ++k) {
    const int per = ((stages + k - 1) / k + 1) / 2 * 2;          // pairs, but for the last range
    const int used = (stages + per - 1) / per;                   // those that hold stages
    const double us = before + T::two + T::tile * (tiles - left) + T::sum * left * used +
                      per * T::stage * crowded<C::BT>(left * used);
    if (used > 1 && us < best.us) best = {tiles - left, used, per, us};
  }
  return best;
}

template <typename C>
hipError_t launch_tiles(Mx4MomentParams p, const Cut& cut, hipStream_t s) {
  const int nt = (p.dp + C::BT - 1) / C::BT, others = nt * (nt + 1) / 2 - cut.whole;
  p.whole = cut.whole;
  p.splits = cut.splits;
  p.stages = cut.stages;
  tile_kernel<C><<<p.whole + others * p.splits, C::THREADS, 0, s>>>(p);
  if (others) reduce_kernel<C><<<others * (C::SLAB / 4 / 256), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_moment(Mx4MomentParams p, hipStream_t s) {
  const int64_t blocks = (p.n_rows + kMx4Block - 1) / kMx4Block;
  const int stages = static_cast<int>((blocks + kStageBlocks - 1) / kStageBlocks);
  // Tiles need two whole stages.  With as many, 64-tiles are faster than bands: 512 samples of 768 features 5.1 and
  // 5.5 us, 1024 5.6 and 7.2.
  if (p.n_rows < 2 * kStageBlocks * kMx4Block) {
    const int nb = p.dp / kBand;
    band_kernel<<<nb * (nb + 1) / 2, 64, 0, s>>>(p);
    return hipGetLastError();
  }
  // 256-tiles where there is enough to do for their longer start and end, and they fill their last round.
  // Against 128-tiles, from no cache: 65536 samples of 6400 features 657 and 762 us, 16384 of them 227 and 240, 65536
  // of 2560 137 and 147; 4096 features (136 tiles on 256 CUs) 405 and 312; 16384 of 2560 62 and 50.
  const int nt = (p.dp + 255) / 256, tiles = nt * (nt + 1) / 2, left = tiles % kCUs;
  const bool fills = left == 0 || left * (kCUs / left) >= kCUs * 7 / 10;
  if (p.dp >= 2048 && fills && static_cast<int64_t>(stages) * tiles >= 6000)
    return launch_tiles<Cfg256>(p, cut_tiles<Cfg256>(p, stages), s);
  // 64-tiles have more CUs at work, and less to do at a tile's end; 128-tiles read half as much a product.  64 against
  // 128 at its best, from no cache: 1024 samples of 1025 features 7.7 and 11.8 us, 4096 14.3 and 15.3, 4096 of 1600
  // 17.0 and 20.1; 16384 of 1600 36 and 31, 4096 of 2560 26.4 and 23.9.
  const Cut small = cut_tiles<Cfg64>(p, stages), large = cut_tiles<Cfg128>(p, stages);
  return small.us < large.us ? launch_tiles<Cfg64>(p, small, s) : launch_tiles<Cfg128>(p, large, s);
}

}  // namespace muon
