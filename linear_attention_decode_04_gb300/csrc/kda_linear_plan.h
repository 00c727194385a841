// kda_linear_plan.h -- the variants of the matrix product kernel and the choice
// between them.  Plain C++, so that a host without CUDA can ask which one a call
// takes.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace {

constexpr int kTileN = 128;                // channels of a CTA's tile
constexpr int kBlock = 128;                // bytes of k per stage
constexpr int kMaxSplit = 4;
constexpr int kMaxStages = 12;
// A gate's two halves: in two accumulators, or 16 and 16 channels in turn in one.
constexpr int kNoGate = 0, kTwoSums = 1, kInterleaved = 2;

// ROWS of x per tile; FEW warpgroups that write results, see kFewPlain.
template <int ROWS, int GATE, bool PAIR, bool FEW = false>
struct Cfg {
  static constexpr int kAcc = GATE == kTwoSums ? 2 : 1;
  static constexpr int kChannels = GATE == kInterleaved ? kTileN / 2 : kTileN;  // of out, of a CTA
  static constexpr int kUnroll = PAIR || ROWS > 64 ? 4 : 2;  // blocks of eight rows that a warp writes at a time
  static constexpr int kRowBytes = 8 * kUnroll * kChannels / 4 * 2;  // of these rows
  static constexpr int kWeightBytes = kAcc * kTileN * kBlock, kStageBytes = kWeightBytes + ROWS / (PAIR ? 2 : 1) * kBlock;
  static constexpr int kCols = kAcc * ROWS;      // accumulator columns of a tile, of which there are two sets
  static constexpr int kTmemCols = 2 * kCols;    // a power of two from 32 on
  // One CTA takes an SM's shared memory; where a short range of k leaves room, the next call's CTAs start beside it.
  static constexpr int kCtasPerSm = PAIR || ROWS > 32 ? 1 : 2;
  // warpgroups that write results; then a warp that copies weights, one that copies rows, and the issuer
  static constexpr int kGroups = FEW ? 2 : GATE == kTwoSums ? (ROWS > 32 ? 2 : 1) : ROWS < 64 ? ROWS / 16 : 4, kThreads = 128 * kGroups + 96;
  // sums of a tile that several CTAs share: in the stages, when its products have ended, lie a CTA's own and those sent to it
  static constexpr int kPartBytes = kCols / 2 * (kTileN * 8 + 64 * kMaxSplit);
  static_assert(kTmemCols * kCtasPerSm <= 512, "tensor memory");
};

// Shared memory: the stages, then this.
template <class C>
struct Head {
  alignas(16) uint8_t rows[4 * C::kGroups][C::kRowBytes];  // of the warps that write results
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], joined, done;
  uint32_t tmem;
  int failed;
};

// What a call needs to know of a variant.
struct Variant {
  int rows, unit, channels;    // rows of a tile, at most, and what they are a multiple of; channels of out per tile
  bool pair, interleaved;
  int threads;
  int stage_bytes, part_bytes, head_bytes;
  float start, block, join, results;  // us, see plan_of
};
// ROWS, GATE, PAIR, FEW; start, block, join, results: first those without a gate, then those with one, then those of FEW.
#define KDA_LINEAR_VARIANTS(X)                             \
  X(16, kNoGate, false, false, 4.5f, .146f, .55f, .8f)     \
  X(32, kNoGate, false, false, 4.7f, .17f, 1.f, 1.2f)      \
  X(64, kNoGate, false, false, 5.3f, .22f, 1.6f, 2.4f)     \
  X(128, kNoGate, false, false, 6.f, .246f, 4.f, 2.1f)     \
  X(128, kNoGate, true, false, 6.3f, .195f, 3.f, 1.7f)     \
  X(256, kNoGate, true, false, 7.2f, .26f, 0.f, 3.2f)      \
  X(16, kTwoSums, false, false, 4.8f, .26f, 1.f, 1.f)      \
  X(32, kTwoSums, false, false, 5.f, .28f, 1.5f, 1.6f)     \
  X(64, kTwoSums, false, false, 5.8f, .33f, 2.5f, 3.f)     \
  X(128, kTwoSums, false, false, 7.f, .4f, 0.f, 4.f)       \
  X(256, kInterleaved, true, false, 8.f, .3f, 0.f, 3.2f)   \
  X(256, kNoGate, true, true, 7.2f, .26f, 0.f, 3.2f)       \
  X(256, kInterleaved, true, true, 8.f, .3f, 0.f, 3.2f)
constexpr int kPlain = 6, kGatedVariants = 5;  // (of the first two kinds)
template <int ROWS, int GATE, bool PAIR, bool FEW>
constexpr Variant variant(float start, float block, float join, float results) {
  using C = Cfg<ROWS, GATE, PAIR, FEW>;
  return {ROWS, 8 * C::kUnroll, C::kChannels * (PAIR ? 2 : 1), PAIR, GATE == kInterleaved, C::kThreads,
          C::kStageBytes, C::kPartBytes, static_cast<int>(sizeof(Head<C>)), start, block, join, results};
}
#define KDA_LINEAR_VARIANT(ROWS, GATE, PAIR, FEW, ...) variant<ROWS, GATE, PAIR, FEW>(__VA_ARGS__),
const Variant kVariants[] = {KDA_LINEAR_VARIANTS(KDA_LINEAR_VARIANT)};
#undef KDA_LINEAR_VARIANT
// The variants of 256 rows (plain, gated) with two warpgroups that write results instead of four: fewer waiting warps (16,384 x
// 18,432 x 6,144 1,098 us, with four 1,119, both at the power limit), more registers (8,192 x 8,192 x 512 with residual 86 and
// 91) and fewer rows written at a time (fp32 59 and 64, on no boundary 75 and 101).  Four are for bf16 rows off 16-byte
// boundaries, which a group writes together (8,192 x 8,191 x 512 83, with two 100), and gates of short k (4,096 x 16,384 x
// 512 45 and 52, x 2,048 81 and 79).
constexpr int kFewPlain = kPlain + kGatedVariants, kFewGated = kFewPlain + 1;
constexpr int kFewGatedBlocks = 12;
constexpr int kSmemLimit = 227 * 1024;  // of a CTA

// What a call runs with: the variant, CTAs (or pairs) that share a tile, ring depth.
struct Plan {
  int variant, split, stages, tile_rows;
};
inline int64_t tiles_of(int64_t n, int64_t size) { return (n + size - 1) / size; }
// The variant and split with the least expected time, in us: what a launch takes from its start to its first product and
// from its last to its results (start); waves of tiles, at a time per block of k each (block, where row tiles are cut
// short half of it in proportion) or what their results take if that is longer (results); the weights from HBM
// meanwhile; and what joining takes each time a tile is shared by twice as many (join).  Measured on these shapes, with
// e4m3 (other choices in brackets): 4 x 4,608 x 2,048 6.2 us in two parts (5.9 in four, 6.5 whole), 64 x 4,096 x 4,096
// 9.6 with tiles of 32 rows in two (10.7 whole; with 64 9.5 in two, 10.1 in four, 11.6 whole), 64 x 18,432 x 6,144 21.9
// with 64 rows (26.9 with 32, 21.7 with 128), 256 x 2,048 x 2,048 7.5 with 32 (7.6 with 64, 7.7 with pairs and 128, 8.3
// with 128 and one CTA, 10.2 with 256), 256 x 65,536 x 128 16.7 with 256 (18.2 with 128 and one CTA, 19.6 with pairs,
// 23.7 with 64); with bf16 64 x 6,144 x 6,144 20.0 with 64 in two (28.2 whole, 26.2 with 32), 300 x 8,192 x 4,096 21.1
// with 256 (31.1 with pairs and 128), 512 x 4,096 x 4,096 19.1 with pairs and 128 (23.0 with 256, 22.2 with one CTA).
// (whole: results go out in whole 16-byte pieces, or are fp32.)
inline Plan plan_of(int M, int width, int blocks, bool gated, double bytes, int sms, bool whole) {
  Plan best{-1, 1, 0, 0};
  double least = 0;
  for (int i = gated ? kPlain : 0; i < (gated ? kPlain + kGatedVariants : kPlain); ++i) {
    const Variant& v = kVariants[i];
    const int most = std::min((kSmemLimit - v.head_bytes) / v.stage_bytes, kMaxStages);
    // row tiles of much the same height (300 rows as 160 and 140 instead of 256 and 44)
    const int64_t m_tiles = tiles_of(M, v.rows);
    const int tile_rows = static_cast<int>(std::min<int64_t>(v.rows, tiles_of(tiles_of(M, m_tiles), v.unit) * v.unit));
    const double height = m_tiles > 1 ? static_cast<double>(tile_rows) / v.rows : 1;
    const int64_t tiles = tiles_of(width, v.channels) * m_tiles, at_once = v.pair ? sms / 2 : sms;
    for (int split = 1, log2 = 0; split <= kMaxSplit; split *= 2, ++log2) {
      if (split > 1 && (v.interleaved || tiles * split > at_once || split > blocks || 2 * v.part_bytes > most * v.stage_bytes)) break;
      const int64_t waves = (tiles * split + at_once - 1) / at_once;
      // (of the waves' time and the weights' the shorter hides behind the longer but for some three tenths)
      const double products = tiles_of(blocks, split) * v.block * (.5 + .5 * height), results = v.results * height;
      const double compute = products + (waves - 1) * std::max(products, results), memory = bytes / 6.5e6;
      const double us = v.start + std::max(compute, memory) + .3 * std::min(compute, memory) + log2 * v.join;
      if (best.variant >= 0 && us >= least) continue;
      // no more stages than there is to copy, but room for the sums of a tile in parts
      const int64_t copies = waves * tiles_of(blocks, split), sums = split > 1 ? tiles_of(2 * v.part_bytes, v.stage_bytes) : 1;
      best = {i, split, static_cast<int>(std::min<int64_t>(most, std::max(copies, sums))), tile_rows};
      least = us;
    }
  }
  if (kVariants[best.variant].rows == 256 && whole && (!gated || blocks >= kFewGatedBlocks)) best.variant = gated ? kFewGated : kFewPlain;
  return best;
}

}  // namespace
