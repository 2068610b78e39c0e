// Which part of a run of floats is copied in whole 16-byte lines.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SAF_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SAF_HOST_DEVICE inline
#endif

namespace saf {

// Entries [first, end) of a row, whole lines, cover the run lo .. hi of that row but for its entries below `first` and from
// `end` on: at most three at either end, and only where their line is not a part of the array. (Lines
// inside the array may hold entries of the rows beside.)
struct PatternRun {
    int first, end;   // first >= end: nothing
};

// row: address of the row's entry 0; before, behind: entries of the array before it, and from it on.
SAF_HOST_DEVICE PatternRun pattern_run(uintptr_t row, long long before, long long behind, int lo, int hi) {
    PatternRun x;
    x.first = lo - (int)(((row >> 2) + (uintptr_t)(intptr_t)lo) & 3);
    x.end = x.first + ((hi - x.first + 4) & ~3);
    if (x.first < -before) x.first += 4;
    if (x.end > behind) x.end -= 4;
    return x;
}

}  // namespace saf
