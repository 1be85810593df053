// kv_tree.cuh — which keys the nodes of a tree of drafted tokens see.
#pragma once

#include "kv.h"

namespace moe {

namespace {

// The lowest n bits, of all n below 0 or above 64 too.
__device__ __forceinline__ unsigned long long low_bits(int n) {
  return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull;
}

// Which of the keys k0 .. k0 + 63 the node of a row tile's token `tok` sees, by bits.
__device__ __noinline__ unsigned long long tree_seen(const KvAttn& a, const KvRowTile& t, int tok, int k0) {
  if (tok >= t.nt) return 0ull;
  const int first = t.p0 + 1, node = t.node0 + tok;  // key of node 0
  const uint4* m = reinterpret_cast<const uint4*>(a.tree) + 2LL * (t.row0 + tok);
  const uint4 lo4 = m[0], hi4 = m[1];
  const unsigned long long words[4] = {lo4.x | static_cast<unsigned long long>(lo4.y) << 32,
                                       lo4.z | static_cast<unsigned long long>(lo4.w) << 32,
                                       hi4.x | static_cast<unsigned long long>(hi4.y) << 32,
                                       hi4.z | static_cast<unsigned long long>(hi4.w) << 32};
  // Ancestors in the order of their numbers stand at depths 0, 1, ...: those whose rank is within the window of the
  // node's, or whose position is a sink's, are seen.
  const int own = first - k0;  // bit of node 0
  int depth = -1;
#pragma unroll
  for (int i = 0; i < 4; ++i) depth += __popcll(words[i] & low_bits(node + 1 - 64 * i));
  const int least = a.window > 0 ? depth - a.window + 1 : 0;  // rank
  unsigned long long seen = 0ull;
  int rank = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned long long w = words[i] & low_bits(node + 1 - 64 * i);
    const int here = __popcll(w);
    if (rank < least) {
      // Its lowest bits, of ranks below `least` that are no sinks', go.
      int r = rank;
      for (unsigned long long rest = w; rest != 0ull && r < least; rest &= rest - 1ull, ++r)
        if (first + r >= a.sinks) w &= ~(rest & (0ull - rest));
    }
    rank += here;
    const int shift = own + 64 * i;
    if (shift > -64 && shift < 64) seen |= shift >= 0 ? w << shift : w >> -shift;
  }
  const int lo = a.window > 0 ? first + depth - a.window + 1 : 0;
  return seen | (low_bits(first - k0) & ~(low_bits(lo - k0) & ~low_bits(a.sinks - k0)));
}

}  // namespace

}  // namespace moe
