// mx_plan_print.cpp -- test infrastructure only (tests/test_mx_paths.py): prints, for
// each argument m,n,k,experts, the kernel that the rules of rz_mx_plan.h choose on a
// device of 256 compute units and how it is cut.
#include <stdio.h>

#include "rz_mx_plan.h"

namespace rz {
int device_cu_count() { return 256; }
}  // namespace rz

int main(int argc, char** argv) {
  for (int i = 1; i < argc; i++) {
    long long m, n, k, experts;
    if (sscanf(argv[i], "%lld,%lld,%lld,%lld", &m, &n, &k, &experts) != 4) return 1;
    rz::StreamPlan s;
    if (rz::streams(m, n, k, experts, s)) {
      printf("stream %d %d %d %d\n", s.rt, s.ck, s.mt, s.rows);
    } else {
      double us;
      const rz::TilePlan t = rz::tile_plan(m, n, k, experts, us);
      printf("tile %d %d %d %d\n", t.high, t.full, t.rest, t.split);
    }
  }
}
