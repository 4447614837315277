// How ep_route spreads a token over lanes, from sizes alone: plain C++ without
// HIP, so that the rules can be checked on any host.
#pragma once

#include <stdint.h>

namespace ep {

struct RouteLanes {
  int lanes, each;  // lanes of a token, experts of a lane
};

// A token's lanes hold its k choices and the best that is left.  Few tokens take
// 64 lanes: a lane's share is shorter, and there are CUs enough.  us, 16 / 64
// lanes, E 256, k 8: 1 token 4.9 / 4.0, 2048 7.4 / 6.4, 4096 7.5 / 7.7, 16384
// 10.6 / 17.1; E 512: 128 8.1 / 5.2, 4096 10.7 / 8.7, 16384 19.6 / 20.7.  64
// experts or fewer are four a lane on 16 lanes as well: 128 tokens 4.0 / 4.4.
inline RouteLanes route_lanes(int64_t T, int E, int k, int cus) {
  const bool few = T <= 8LL * cus && E > 64;
  RouteLanes r;
  r.lanes = k > 15 || E > 512 || few ? 64 : 16;
  r.each = 4;
  while (r.lanes * r.each < E) r.each *= 2;
  return r;
}

}  // namespace ep
