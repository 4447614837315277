// How ep_route spreads a token over lanes, from sizes alone: plain C++ without
// HIP, so that the rules can be checked on any host.
#pragma once

#include <stdint.h>

namespace ep {

struct RouteLanes {
  int lanes, each;  // lanes of a token, experts of a lane
};

// A token's lanes hold its k choices and the best that is left.
inline RouteLanes route_lanes(int64_t T, int E, int k, int cus) {
  const bool few = T <= 8LL * cus;
  RouteLanes r;
  r.lanes = k > 15 || E > 512 || few ? 64 : 16;
  r.each = 4;
  while (r.lanes * r.each < E) r.each *= 2;
  return r;
}

}  // namespace ep
