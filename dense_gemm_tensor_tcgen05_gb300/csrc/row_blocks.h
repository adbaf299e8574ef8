// row_blocks.h -- which aligned 16-byte blocks a copy of 16-bit rows may read.
// Rows that start anywhere are read in the aligned blocks they lie in; these
// conditions keep such a read inside the matrix [lo, hi).  Plain C++, so that
// they can be checked on the host for every alignment and row length.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define GB_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define GB_HOST_DEVICE inline
#endif

namespace gb300 {

// The two blocks that hold eight elements from `at` on.
GB_HOST_DEVICE bool pair_inside(uintptr_t at, uintptr_t lo, uintptr_t hi) {
    const uintptr_t block = at & ~static_cast<uintptr_t>(15);
    return block >= lo && block + 32 <= hi;
}

// The two blocks of every eight elements of a row of `cols` (at least one)
// from `at` on: the first ones and the last ones are.  A row need not be the
// matrix's first or last to fail: rows shorter than a block share blocks with
// several others.
GB_HOST_DEVICE bool row_inside(uintptr_t at, int64_t cols, uintptr_t lo, uintptr_t hi) {
    return pair_inside(at, lo, hi) && pair_inside(at + 2 * ((cols - 1) & ~static_cast<int64_t>(7)), lo, hi);
}

}  // namespace gb300
