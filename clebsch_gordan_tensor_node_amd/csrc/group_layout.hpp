// How group normalisation lays rows and columns over workgroups.  Host code only, apart from
// the constants.
#pragma once

#include <algorithm>

#include "launch_branch.hpp"

namespace cgtp {

constexpr int kTileBlock = 256;        // threads of a tile's workgroup
constexpr int64_t kGroupGrid = (int64_t(1) << 32) - 1;   // most threads of a launch

// A chunk is the columns that a workgroup takes: whole groups, or where a group is wider than
// a workgroup's lanes reach, a part of one.  A thread has a place of `vec` columns among its
// chunk's `lanes` and every slices-th row.
struct GroupLayout {
  int whole;             // 1: a workgroup has all rows of one sample, and holds them in registers;
                         // 0: tiles of rows, whose sums a second launch joins
  int vec;               // columns of a place: kGroupVec, or 1 where the row has fewer
  int block;             // threads of a workgroup
  int held;              // whole: rows that a thread holds
  int per_group;         // columns of a group
  int per_chunk;         // groups of a chunk
  int split;             // parts of a group (1 unless a group is wider than a workgroup reaches)
  int part;              // columns of a part; the last of a group may have fewer
  int chunks;
  int lanes, slices;
  int tile_rows, tiles;  // tiles only
  int equal;             // rows of each sample, where there are no offsets
  int stream;            // the output passes by the caches: the call moves more than they hold
};

// Columns of a thread's place.  Everything that a thread has per column (weights, statistics,
// sums) is in 32 bits: of eight columns it would take the registers that 16-bit rows leave
// (forward of 114688 x 128 bf16 27 us with four, 31 with eight, 30 with two).
constexpr int kGroupVec = 4;

// Rows that a thread holds of a whole sample: 64 registers of x, or 48 of x and grad_out.
constexpr int kHeldFew = 4;
// Most rows that a thread reads of a whole sample.  With 64, that 16-bit rows allow, the forward of
// 96000 x 128 bf16 in 24 samples took 44 us as whole samples, 26 as tiles; of 48000 x 128 (31 rows
// a thread) it takes 22.
constexpr int kWholeTurns = 32;
constexpr int held_most(int elem_bytes, bool backward) { return (backward ? 24 : 64) / elem_bytes; }

// Workgroups with a tile each: one for every place that the device has for them (some 1000), or,
// past the caches, as many as keep the addresses that are read at one time together.  Measured
// with 512, 1024 and 2048: forward of 114688 x 128 bf16 28, 25 and 28 us, backward of 20060 x 481
// fp32 in 48 samples 48, 49 and 54; with 1024, 2048, 4096 and 6144: forward of 114688 x 1312 fp32
// 391, 373, 350 and 351 us, backward of 400000 x 128 in 20 samples 207, 196, 190 and 189.
constexpr int64_t kTiles = 1024, kTilesStream = 4096;
constexpr int kTileTurn = 8;   // rows that a thread reads at once

inline void set_lanes(GroupLayout& y, int64_t columns) {
  y.lanes = int((columns + y.vec - 1) / y.vec);
  y.slices = y.block / y.lanes;
}

inline GroupLayout lay_out_group(const GroupCall& c, int elem_bytes, bool backward) {
  GroupLayout y{};
  const int64_t cg = c.width / c.groups;
  y.per_group = int(cg);
  y.equal = c.offsets || c.samples == 0 ? 0 : int(c.rows / c.samples);
  y.vec = c.width >= kGroupVec ? kGroupVec : 1;
  y.split = 1;
  y.stream = double(c.rows) * double(c.width) * elem_bytes * (backward ? 3 : 2) > double(kCacheBytes);
  y.part = int(cg);
  // the longest sample: as told, as equal samples have it, or eight times the mean
  const int64_t mean = c.samples ? (c.rows + c.samples - 1) / c.samples : 0;
  const int64_t longest = c.longest > 0 ? std::min(c.longest, c.rows) : std::min(c.rows, c.offsets ? 8 * mean : mean);
  const int most = held_most(elem_bytes, backward);
  // A workgroup for a whole sample: 64 threads with the widest chunk that leaves kWant
  // workgroups, else 256 with chunks down to 32 bytes of a row; both hold half of the longest
  // sample at least, and read the rest again.  Else tiles.  Measured, us of whole samples and of
  // tiles: forward of 40000 x 64 fp32 in 100 samples 14 and 21 (in workgroups that hold all 17),
  // of 600000 x 64 in 1500 75 and 114 (86; 124 where a quarter is held).  Workgroups of 1024
  // threads, for samples that less do not hold: 18 and 21 for the backward of 4000 x 128 fp32 in
  // 4, but 41 and 31 for the forward of 144000 x 128 bf16 in 24, 40 and 24 for 96808 x 60 in 38.
  constexpr int64_t kWant = 512;
  for (const int block : {64, 256}) {
    y.block = block;
    int64_t take = 0, items = 0;
    for (int64_t m = std::min(c.groups, block * int64_t(y.vec) / cg); m >= 1; m = m == 1 ? 0 : (m + 1) / 2) {
      set_lanes(y, m * cg);
      if (int64_t(y.slices) * std::min(2 * most, kWholeTurns) < longest) continue;
      if (take && m * cg * elem_bytes < 32) break;
      take = m;
      items = c.samples * ((c.groups + m - 1) / m);
      if (items >= kWant) break;
    }
    if (!take || (block == 64 && items < kWant)) continue;
    y.whole = 1;
    y.per_chunk = int(take);
    y.chunks = int((c.groups + take - 1) / take);
    set_lanes(y, take * cg);
    y.held = int64_t(y.slices) * kHeldFew >= longest ? kHeldFew : most;
    return y;
  }
  y.whole = 0;
  y.block = kTileBlock;
  const int64_t reach = int64_t(kTileBlock) * y.vec;
  if (cg > reach) {
    const int64_t parts = (cg + reach - 1) / reach;
    y.part = int(((cg + parts - 1) / parts + y.vec - 1) / y.vec * y.vec);
    y.split = int((cg + y.part - 1) / y.part);
    y.per_chunk = 1;
    y.chunks = int(c.groups * y.split);
    set_lanes(y, y.part);
  } else {
    // the number of chunks that leaves the fewest threads idle, the smallest unless another
    // gains 3 %
    const int64_t least = (c.groups + reach / cg - 1) / (reach / cg);
    double best = 0;
    for (int64_t n = least; n < least + 8 && n <= c.groups; ++n) {
      const int64_t m = (c.groups + n - 1) / n;
      set_lanes(y, m * cg);
      const double busy = double(y.slices) * double(c.width) / double((c.groups + m - 1) / m) / y.vec / kTileBlock;
      if (busy > best * 1.03) {
        best = busy;
        y.per_chunk = int(m);
      }
    }
    y.chunks = int((c.groups + y.per_chunk - 1) / y.per_chunk);
    set_lanes(y, y.per_chunk * cg);
  }
  // whole turns of kTileTurn rows a thread, four rows at least
  const int64_t most_tiles = y.stream ? kTilesStream : kTiles, turn = int64_t(kTileTurn) * y.slices;
  int64_t rows = std::max<int64_t>((c.rows * y.chunks + most_tiles - 1) / most_tiles, 4 * y.slices);
  if (rows > turn / 2) rows = (rows + turn - 1) / turn * turn;
  rows = std::max<int64_t>(std::min(rows, c.rows), 1);
  y.tile_rows = int(rows);
  y.tiles = int((c.rows + rows - 1) / rows);
  return y;
}

// The workspace: sums of the pieces (a tile's part of a sample: tile t of sample s is piece
// t + s, which no other pair is, since a walk through the pieces moves on in one of them at a
// time), then per sample what they join to.
struct GroupWork {
  int64_t pieces, join, coef, total;   // floats before each, and of all
};
// sums: the backward's weights' gradients are wanted.
inline GroupWork group_work(const GroupCall& c, const GroupLayout& y, bool backward, bool sums = true) {
  GroupWork w{};
  const int64_t pieces = y.whole ? 0 : y.tiles + c.samples;
  const int64_t per_piece = backward ? 2 * c.width : 2 * c.groups * y.split;
  w.pieces = 0;
  w.join = pieces * per_piece;
  // backward: [samples][2][width] sums per channel (one sample's are the gradients), then
  // [samples][groups][2] means; forward: the statistics, if the caller wants none
  w.coef = w.join + (backward && sums && c.samples > 1 ? c.samples * 2 * c.width : 0);
  w.total = w.coef + (y.whole ? 0 : c.samples * c.groups * 2);
  return w;
}

}  // namespace cgtp
