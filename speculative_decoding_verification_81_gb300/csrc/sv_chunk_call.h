// sv_chunk_call.h -- which call of its workspace a call is, as arithmetic on
// host or device: what arrival counters it uses, and how it says that a wait
// gave up.
//
// A wait that runs out leaves the arrival counters of cut items anywhere, and
// nobody to put them right: a CTA cannot know that all others are done without
// waiting for them.  So each call counts in its own set, one of two by the
// parity of its number, and zeroes the other, which the call before it used
// and the next will; whatever a call leaves behind is gone two calls later,
// and no call looks at it before.
//
// The number is on the device, where a replayed graph finds it too.  The CTAs
// of a call, of any grid, add kCallShares to the workspace's word together,
// each its share as it begins: what a CTA reads as it adds lacks its own share
// at least, so that the quotient is the number of calls before, the same for
// every CTA.  The form for few rows, which has no counters to zero, counts its
// calls in words of its own.
//
// A wait that gave up concerns the whole call: its CTA may have left any item
// undone, and items shared with others unmerged.  The CTA sets gave_up to the
// call's tag, then writes SV_ERR_TIMEOUT for every sequence; a warp that has
// written another status looks at gave_up afterwards (a fence between on both
// sides), so that one of the two sees the other.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SV_CALL_HD __host__ __device__ __forceinline__
#else
#define SV_CALL_HD inline
#endif

namespace sv {
namespace chunk {

constexpr int kCallShares = 4096;     // CTAs of a call at most
constexpr int kCallBytes = 256;       // the workspace's first bytes: CallWords of the two forms
constexpr int kCtaCounters = 2 * 4;   // of a CTA in a set: [Q tile][quarter]

struct CallWords {
    unsigned long long shares;   // kCallShares for every call of the form that has begun
    unsigned long long gave_up;  // the tag of the last call in which a wait gave up, or 0
};

SV_CALL_HD unsigned long long call_share(int cta, int grid) { return cta == 0 ? kCallShares - grid + 1 : 1; }

// The number of the call whose CTA read `shares` as it added its own (or later, less its own).
SV_CALL_HD unsigned long long call_number(unsigned long long shares) { return shares / kCallShares; }

SV_CALL_HD unsigned long long call_tag(unsigned long long call) { return call + 1; }

// The first counter of the items cut from CTA `cta` on, in the set of the given call.
SV_CALL_HD int counters_of(unsigned long long call, int grid, int cta) {
    return ((int)(call & 1) * grid + cta) * kCtaCounters;
}

}  // namespace chunk
}  // namespace sv
