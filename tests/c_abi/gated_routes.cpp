// Prints, for each line "m d f" of its input, whether the gated product's backward
// pass takes dx and dw in one launch (1 or 0), dx's splits there, its blocks and dw's
// tiles, and the tile (0 large, 1 middle, 2 small) and splits of forward, dx and dw
// alone. `room` floats of scratch is the argument.
#include <stdio.h>
#include <stdlib.h>

#include "../../zero_dp_partitioned_amd/csrc/gated_route.h"

int main(int, char** argv) {
  const int64_t room = atoll(argv[1]);
  long long m, d, f;
  while (scanf("%lld %lld %lld", &m, &d, &f) == 3) {
    const zdp::PairRoute p = zdp::pair_route(m, d, f, room);
    const zdp::Route a = zdp::route_of(zdp::kForward, m, f, d, room), x = zdp::route_of(zdp::kDx, m, d, f, room),
                     w = zdp::route_of(zdp::kDw, f, d, m, room);
    printf("%d %lld %lld %lld %d %lld %d %lld %d %lld\n", p.together, (long long)p.splits, (long long)p.dx_blocks,
           (long long)p.tiles, a.tile, (long long)a.splits, x.tile, (long long)x.splits, w.tile, (long long)w.splits);
  }
  return 0;
}
