// Prints the launch shapes that csrc/expert_shapes.hpp chooses for the sizes
// given on standard input, one line each: a rule's name and its arguments.
#include <stdio.h>
#include <string.h>

#include "expert_shapes.hpp"

int main() {
  char what[32];
  while (scanf("%31s", what) == 1) {
    if (!strcmp(what, "dispatch_backward")) {
      long long T;
      int nv, k, cus;
      if (scanf("%lld %d %d %d", &T, &nv, &k, &cus) != 4) return 1;
      const ep::GatherShape s = ep::dispatch_backward_shape(T, nv, k, cus);
      printf("%d %d %d\n", s.vs, s.nseg, s.steps);
    } else if (!strcmp(what, "wide_rows")) {
      long long rows;
      int cus, E, N;
      if (scanf("%d %lld %d %d", &cus, &rows, &E, &N) != 4) return 1;
      printf("%d\n", ep::wide_rows(cus, rows, E, N));
    } else if (!strcmp(what, "swiglu")) {
      long long rows;
      int E, blocks;
      if (scanf("%lld %d %d", &rows, &E, &blocks) != 3) return 1;
      const ep::SwigluShape s = ep::swiglu_shape(rows, E, blocks);
      printf("%d %d\n", s.tokens, s.depth);
    } else {
      return 1;
    }
  }
  return 0;
}
