// How the normalisations' rows are laid over lanes, workgroups and launches.  Host code
// only, apart from the constants.
#pragma once

#include <algorithm>

#include "launch_train.hpp"

namespace cgtp {

constexpr int kCapSmall = 8;      // terms of the plans that most launches are made for
constexpr int kWideSlices = 32;   // partial sums of a wide stretch
constexpr int kSumThreads = 1024; // most threads of a workgroup that joins partial sums
constexpr int kInFlight = 16;     // of which a thread reads this many at once
constexpr int64_t kGridThreads = (int64_t(1) << 32) - 1;   // most threads of a launch

// How many lanes G hold a stretch, and in how many vectors C each: the first that has room
// for its nv = ceil(len / V) vectors.  B is the workgroup's size.
enum Variant : int {
  kElem8,   // V = 1, G = 8: shorter than a vector
  kG4C1,    // nv <= 4
  kG8C1,    // nv <= 8
  kG16C1,   // nv <= 16
  kG32C1,   // nv <= 32
  kG64C1,   // nv <= 64
  kG64C2,   // nv <= 128, if a lane holds that many elements
  kG64C4,   // nv <= 256, likewise
  kGBC1,    // nv <= B
  kGBC2,    // nv <= 2 B, likewise
  kGBC4,    // nv <= 4 B, likewise
  kWide     // any: the row is read again for each sum
};

// Elements per lane for a plan whose longest stretch is `longest`, as long as a workgroup's
// lanes reach.  The more, the fewer waves fit a SIMD's registers; the fewer, the more waves
// share a stretch and wait for one another.  With 8 and with 16, us for 400 MB: forward of
// 4096 columns 75 and 78 (fp32), 94 and 108 (bf16), of 4097 93 and 81 (fp32), of 6000 84 and
// 81 (fp32), of 8192 76 and 79 (fp32), 97 and 112 (bf16); backward of 1024 columns 99 and 86
// (fp32), 107 and 115 (bf16), of 4096 88 and 95 (fp32), 94 and 132 (bf16), of 8192 98 and 108
// (fp32), 135 and 133 (bf16).
inline int elems_of(int longest, int elem_bytes, bool backward) {
  if (longest > 4096) return (elem_bytes == 4) != backward ? 16 : 8;
  return longest > 512 && longest <= 1024 && backward && elem_bytes == 4 ? 16 : 8;
}
constexpr int kMaxE = 16;

// The workgroup that the longest stretch of a plan needs, with e elements per lane.
inline int block_of(int longest, int e) {
  return longest <= 64 * e ? 256 : longest <= 128 * e ? 128 : longest <= 256 * e ? 256 : longest <= 512 * e ? 512 : 1024;
}

inline int variant_of(int len, int elem_bytes, int block, int e) {
  const int v = 16 / elem_bytes;
  if (len > block * kMaxE) return kWide;
  if (len < v) return kElem8;
  const int nv = (len + v - 1) / v;
  if (nv <= 4) return kG4C1;
  if (nv <= 8) return kG8C1;
  if (nv <= 16) return kG16C1;
  if (nv <= 32) return kG32C1;
  if (nv <= 64) return kG64C1;
  if (nv <= 128 && e >= 2 * v) return kG64C2;
  if (nv <= 256 && e >= 4 * v) return kG64C4;
  if (nv <= block) return kGBC1;
  return nv <= 2 * block ? kGBC2 : kGBC4;
}
// Lanes per stretch and vectors per lane.
inline int lanes_of(int variant, int block) {
  constexpr int g[] = {8, 4, 8, 16, 32, 64, 64, 64};
  return variant <= kG64C4 ? g[variant] : block;
}
inline int vectors_of(int variant) {
  return variant == kG64C2 || variant == kGBC2 ? 2 : variant == kG64C4 || variant == kGBC4 ? 4 : 1;
}

// Workgroups of a launch, shared among the terms by their cost: enough to keep the
// memory busy, which takes more of them where every access goes to HBM, and in the
// backward no more, since each leaves a row of partial sums.  Measured: forward of 114688 x
// 1312 fp32 231, 230 and 224 us with 1024, 2048 and 4096, of 4096 x 5472 (cached) 47, 37 and
// 40, of 300000 x 64 (cached) 31, 32 and 31; backward and sums of 768 x 9088 (cached) 23.3,
// 23.3, 25.0 and 27.8 us with 512, 768, 1024 and 1536, of 32768 x 704 82, 67, 60 and 56.  Past
// the cache the forward takes more, as long as each has 28 / element bytes turns for the
// weights that it loads: without, with 28 and with 14, 114688 x 1312 fp32 224, 212 and 212 us,
// 100000 x 704 113, 107 and 107; 24414 x 4096 bf16 94, 94 and 105.
constexpr int kTurnBytes = 28;
constexpr int kForwardBlocks = 2048, kForwardBlocksStream = 4096;
constexpr int kBackwardBlocks = 768, kBackwardBlocksStream = 1536;

inline int longest(const NormShape& p) {
  int n = 0;
  for (int k = 0; k < p.n_terms; ++k) n = std::max(n, p.terms[k].len);
  return n;
}

// How the rows are laid over workgroups.
struct Layout {
  int block;                      // threads of a workgroup
  bool stream;                    // rows pass by the last-level cache
  bool direct;                    // backward: one workgroup per term
  int max_e;                      // most elements per lane
  int64_t part;                   // backward: floats of partial sums
  int variant[kMaxNormTerms], n_blocks[kMaxNormTerms], n_parts[kMaxNormTerms];
};

inline Layout lay_out(int64_t rows, const NormShape& p, int elem_bytes, bool backward) {
  Layout y;
  const int e = elems_of(longest(p), elem_bytes, backward);
  y.block = block_of(longest(p), e);
  // rows that outgrow the last-level cache, in plans of up to kCapSmall terms
  y.stream = p.n_terms <= kCapSmall && double(rows) * p.features * elem_bytes * (backward ? 3 : 2) > kCacheBytes;
  // rows so few that one workgroup per term takes them all, in at most four turns: it then
  // writes the weight's and bias's gradients itself
  y.direct = backward;
  y.max_e = 1;
  int64_t cost = 0, part = 0, each[kMaxNormTerms];
  for (int k = 0; k < p.n_terms; ++k) {
    const int v = variant_of(p.terms[k].len, elem_bytes, y.block, e), g = lanes_of(v, y.block), c = vectors_of(v);
    y.variant[k] = v;
    if (v == kWide || rows > 4 * (y.block / g)) y.direct = false;
    y.max_e = std::max(y.max_e, v == kElem8 || v == kWide ? 1 : c * 16 / elem_bytes);
    // what a stretch costs: its lanes, for its vectors and a part that every stretch has
    each[k] = v == kWide ? 0 : int64_t(g) * (c + 1);
    cost += each[k];
  }
  const int64_t total = (backward ? (y.stream ? kBackwardBlocksStream : kBackwardBlocks)
                                  : (y.stream ? kForwardBlocksStream : kForwardBlocks)) * 256 / y.block;
  for (int k = 0; k < p.n_terms; ++k) {
    if (y.variant[k] == kWide) {
      y.n_blocks[k] = 0;   // launched by itself
    } else {
      const int64_t groups = y.block / lanes_of(y.variant[k], y.block);
      const int64_t want = std::max<int64_t>((rows + groups - 1) / groups, 1);
      int64_t most = std::max<int64_t>(total * each[k] / cost, 1);
      if (y.stream && !backward) most = std::max(most, want * elem_bytes / kTurnBytes);
      most = std::min(most, kGridThreads / y.block / p.n_terms);
      y.n_blocks[k] = y.direct ? 1 : int(std::min(want, most));
    }
    y.n_parts[k] = y.variant[k] == kWide ? kWideSlices : y.n_blocks[k];
    part += int64_t(y.n_parts[k]) * p.terms[k].len * (p.terms[k].b_off >= 0 ? 2 : 1);
  }
  y.part = y.direct ? 0 : part;
  return y;
}

// How the second launch of the backward joins the partial sums.
struct SumGrid {
  int tile;      // elements of a workgroup
  int threads;
  int blocks;
};
// Workgroups of one term.
inline int sum_blocks(const NormTerm& t, int tile) {
  const int whole = tile / t.d * t.d;   // they take whole channels
  return (t.len + whole - 1) / whole;
}
// Wide tiles read whole lines (a tile that ends inside one has it fetched again by
// another die's L2), narrow ones spread short stretches over more workgroups: 9088
// columns took 10.1 us in tiles of 16 and 5.4 in tiles of 64, 481 columns 6.6 and 10.2.
inline SumGrid lay_out_sums(const NormShape& p, const Layout& y) {
  SumGrid g{};
  int tiles = 0, most = 0;
  for (int k = 0; k < p.n_terms; ++k) {
    tiles += p.terms[k].len / 64;
    most = std::max(most, y.n_parts[k]);
  }
  g.tile = tiles >= 16 ? 64 : 16;
  for (int k = 0; k < p.n_terms; ++k) g.blocks += sum_blocks(p.terms[k], g.tile);
  // as many slices as keep every load in flight, two at least
  const int want = (most + kInFlight - 1) / kInFlight * g.tile;
  g.threads = want <= 128 ? 128 : want <= 256 ? 256 : want <= 512 ? 512 : kSumThreads;
  while (int64_t(g.blocks) * g.threads > kGridThreads) g.threads /= 2;   // 2^24 tiles at most: 128 fit
  return g;
}

}  // namespace cgtp
