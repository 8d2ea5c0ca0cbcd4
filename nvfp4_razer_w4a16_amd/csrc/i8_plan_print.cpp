// i8_plan_print.cpp -- test infrastructure only (tests/test_i8_paths.py): prints, for
// each argument m,n,k,experts, the kernel that the rules of rz_i8_plan.h choose on a
// device of 256 compute units and how it is cut.
#include <stdio.h>

#include "rz_i8_plan.h"

int main(int argc, char** argv) {
  for (int i = 1; i < argc; i++) {
    long long m, n, k, experts;
    if (sscanf(argv[i], "%lld,%lld,%lld,%lld", &m, &n, &k, &experts) != 4) return 1;
    rz::i8::StreamPlan s;
    if (rz::i8::streams(m, n, k, experts, 256, s)) {
      printf("stream %d %d %d %d\n", s.rt, s.ck, s.mt, s.rows);
    } else {
      double us;
      const rz::i8::TilePlan t = rz::i8::tile_plan(m, n, k, experts, 256, us);
      printf("tile %d %d %d %d %d %d\n", t.wide, t.high, t.full, t.rest, t.split, t.halves);
    }
  }
}
