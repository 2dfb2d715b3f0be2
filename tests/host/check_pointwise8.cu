// CPU check of the 8-bit 1x1 product's choice of kernel: for every "rows cin
// cout" of the command line, "row", "tile" or "pair", then the rounds of pairs
// that the GPU takes and the blocks of channels.
#include <cstdio>
#include <cstdlib>

#include "pointwise8_tc.cu"

int main(int argc, char** argv) {
  using namespace dwconv::pw8;
  for (int i = 1; i + 2 < argc; i += 3) {
    Pw g{};
    g.rows = atoll(argv[i]);
    g.cin = atoi(argv[i + 1]);
    g.cout = atoi(argv[i + 2]);
    g.pitch = pitch_of(g.cin);
    g.nkb = (int)(g.pitch / kBlock);
    printf("%s %lld %d\n", plan(g) == Plan::Row ? "row" : by_pairs(g) ? "pair" : "tile",
           (long long)((tiles_of(g, 2 * kM, Pair::kN) + 75) / 76), g.nkb);
  }
  return 0;
}
