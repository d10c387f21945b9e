// Which cache slots a tree node sees, with a sliding window and sinks.
//
// A key has a position: a prefix slot p < L its index, tree node a its token
// position L + depth(a).  A query node at depth D (position L + D) sees a key
// iff the key is a prefix slot or one of the node's ancestors (itself
// included) and, with a window W > 0, its position is below `sinks` or above
// L + D - W.  W = 0 is no window.  A node always sees itself (W >= 1).
#pragma once

#include "common.cuh"

namespace medusa {

// Slots any node can see, as two runs [0, head) and [tail, L + N): the sinks
// and, from the root's window start (the root sees furthest back), the rest.
struct VisibleRuns {
  int head, tail, total;  // total = head + (L + N - tail)
};
__device__ __forceinline__ VisibleRuns visible_runs(int L, int N, int window, int sinks) {
  VisibleRuns r{0, 0, L + N};
  if (window > 0) {
    const int lo = max(0, (int)min((long long)L, (long long)L - window + 1));
    r.head = min(min(sinks, L), lo);
    r.tail = lo;
    r.total = r.head + (L + N - lo);
  }
  return r;
}

// Window rule alone (the tree's ancestor rule is the caller's).
__device__ __forceinline__ bool in_window(int pos, int q_pos, int window, int sinks) {
  return window <= 0 || pos < sinks || (long long)pos > (long long)q_pos - window;
}

}  // namespace medusa
