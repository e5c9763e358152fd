// mk_ops_parts.h -- where the parts of an item of the attention of shared
// prefixes lie in the workspace, between the kernel that writes them and the
// one that joins them.  No CUDA in it: the host's tests compile it too.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MK_BOTH __host__ __device__ __forceinline__
#else
#define MK_BOTH inline
#endif

namespace mk {
namespace ops {

// The first and the last CTA that an item's tiles were dealt to (each writes its own number).
struct Placed {
  int32_t first, last;
};

// An item's parts, one of each CTA; 0 where the numbers are none of `grid`
// CTAs': the CTA that would have written them gave up a wait before it planned
// the item, and they are what the workspace held.
MK_BOTH int parts_of(Placed p, int grid) {
  return p.first < 0 || p.last < p.first || p.last >= grid ? 0 : p.last - p.first + 1;
}

// Part k's slot, of two for each CTA: a part that begins its item is its CTA's
// last, the others are their CTA's first.
MK_BOTH int64_t part_slot(Placed p, int k) { return 2 * ((int64_t)p.first + k) + (k == 0 ? 1 : 0); }

}  // namespace ops
}  // namespace mk
