// Prints the launches that the normalisations' layout asks for, one line per call read
// from standard input:  rows elem_bytes backward n_terms (len d centred)...
//   -> threads of a workgroup, workgroups, threads and workgroups of the partial sums, most
//      elements of a lane
#include <cstdio>
#include <vector>

#include "../../clebsch_gordan_tensor_node_amd/csrc/norm_layout.hpp"

int main() {
  using namespace cgtp;
  long long rows;
  int bytes, back, n;
  while (std::scanf("%lld %d %d %d", &rows, &bytes, &back, &n) == 4) {
    std::vector<NormTerm> terms;
    NormShape p{0, 0, 0, nullptr, n};
    for (int k = 0; k < n; ++k) {
      int len, d, centred;
      if (std::scanf("%d %d %d", &len, &d, &centred) != 3) return 1;
      terms.push_back(NormTerm{int32_t(p.features), len, d, int32_t(p.weights), centred ? int32_t(p.biases) : -1});
      p.features += len;
      p.weights += len / d;
      if (centred) p.biases += len / d;
    }
    p.terms = terms.data();
    const Layout y = lay_out(rows, p, bytes, back != 0);
    long long blocks = 0;
    for (int k = 0; k < n; ++k) blocks += y.n_blocks[k];
    const SumGrid g = lay_out_sums(p, y);
    std::printf("%d %lld %d %d %d\n", y.block, blocks, g.threads, g.blocks, y.max_e);
  }
  return 0;
}
