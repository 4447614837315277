// Prints the launch shapes that csrc/linear_shapes.hpp and csrc/route_shapes.hpp
// choose for the sizes given on standard input, one line each: a rule's name
// and its arguments.
#include <stdio.h>
#include <string.h>

#include "linear_shapes.hpp"
#include "route_shapes.hpp"

int main() {
  char what[32];
  while (scanf("%31s", what) == 1) {
    long long rows;
    int a, b, c;
    if (scanf("%lld %d %d %d", &rows, &a, &b, &c) != 4) return 1;
    if (!strcmp(what, "linear")) {  // rows, experts, columns, depth
      const ep::LinearShape s = ep::linear_shape(rows, a, b, c, rows * b);
      printf("%d %d %lld\n", s.rows, s.splits, (long long)s.items);
    } else if (!strcmp(what, "wgrad")) {  // rows, experts, N, K
      const ep::LinearShape s = ep::wgrad_shape(rows, a, b, c);
      printf("%d %d %lld\n", s.rows, s.splits, (long long)s.items);
    } else if (!strcmp(what, "route")) {  // tokens, experts, k, compute units
      const ep::RouteLanes r = ep::route_lanes(rows, a, b, c);
      printf("%d %d\n", r.lanes, r.each);
    } else {
      return 1;
    }
  }
  return 0;
}
