// gdn_pages.h -- device helpers of the paged key/value cache: division by a constant of the
// call, the cache row of a position.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_attention_internal.h"

namespace gdn {
namespace dev {

// n / d for 0 <= n < 2^31 (see Divisor)
__device__ __forceinline__ unsigned divide(unsigned n, const Divisor& by) { return __umulhi(n << 1, by.m) >> by.l; }

// The pages of one sequence, in a table of at least one entry.  The entry is looked up apart from the row, so that its load can be in
// flight meanwhile.
struct Pages {
    const int32_t* table;
    int width;
    Divisor block;
    int64_t num_rows;
    // Entry of position p >= 0, or the last one where p lies past the table.
    __device__ __forceinline__ int entry(int p) const {
        const unsigned page = divide((unsigned)p, block);
        return table[page < (unsigned)width ? page : (unsigned)width - 1];
    }
    // Cache row of position p with that entry, or -1 where its page is absent or p is not below `end`.
    __device__ __forceinline__ int row(int p, int entry, int end) const {
        const unsigned page = divide((unsigned)p, block);
        const int64_t r = (int64_t)entry * block.d + ((unsigned)p - page * block.d);
        return p < end && page < (unsigned)width && entry >= 0 && r < num_rows ? (int)r : -1;
    }
};

}  // namespace dev
}  // namespace gdn
