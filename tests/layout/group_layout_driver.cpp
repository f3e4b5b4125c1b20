// Prints the layout that group normalisation chooses, one line per call read from stdin:
// rows width groups samples ragged longest element_bytes backward.
#include <cstdio>

#include "../../clebsch_gordan_tensor_node_amd/csrc/group_layout.hpp"

int main() {
  long long rows, width, groups, samples, longest;
  int ragged, bytes, backward;
  static const int32_t some = 0;
  while (std::scanf("%lld %lld %lld %lld %d %lld %d %d", &rows, &width, &groups, &samples, &ragged, &longest, &bytes,
                    &backward) == 8) {
    cgtp::GroupCall c{};
    c.rows = rows;
    c.width = width;
    c.groups = groups;
    c.samples = samples;
    c.longest = longest;
    c.offsets = ragged ? &some : nullptr;
    const cgtp::GroupLayout y = cgtp::lay_out_group(c, bytes, backward != 0);
    const cgtp::GroupWork w = cgtp::group_work(c, y, backward != 0);
    std::printf("%d %d %d %d %lld %lld %lld %lld %d %d %lld %lld %lld\n", y.whole, y.vec, y.block, y.held,
                (long long)y.per_chunk, (long long)y.split, (long long)y.part, (long long)y.chunks, y.lanes, y.slices,
                (long long)y.tile_rows, (long long)y.tiles, (long long)w.total);
  }
  return 0;
}
