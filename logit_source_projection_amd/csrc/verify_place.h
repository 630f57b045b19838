// Where a sequence's drafts lie (plain C++: host and device).
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define SBK_ANYWHERE __host__ __device__ __forceinline__
#else
#define SBK_ANYWHERE inline
#endif

namespace sbk {

struct Place {
    int32_t first, count;
};

// Offsets are data of the device: whatever they hold, 0 <= first, 0 <= count <= K
// and first + count <= drafts, so that sequence i < N reads draft rows below
// drafts and target rows first + i + j, j <= count, below drafts + N.
SBK_ANYWHERE Place place_of(int32_t from, int32_t to, int32_t drafts, int32_t K)
{
    const int32_t first = from < 0 ? 0 : from > drafts ? drafts : from;
    const int32_t end = to < first ? first : to > drafts ? drafts : to;
    return {first, end - first < K ? end - first : K};
}

}  // namespace sbk
