// gdn_pages.h -- device helpers of the paged key/value cache: division by a constant of the
// call, the cache row of a position, values of a cache's formats.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_attention_internal.h"

namespace gdn {
namespace dev {

// n / d for 0 <= n < 2^31 (see Divisor)
__device__ __forceinline__ unsigned divide(unsigned n, const Divisor& by) { return __umulhi(n << 1, by.m) >> by.l; }

// The pages of one sequence.
struct Pages {
    const int32_t* table;
    int width;
    Divisor block;
    int64_t num_rows;
    // Cache row of position p >= 0, or -1 where its page is absent.
    __device__ __forceinline__ int64_t row(int p) const {
        const unsigned page = divide((unsigned)p, block);
        const int entry = page < (unsigned)width ? table[page] : -1;
        const int64_t r = (int64_t)entry * block.d + ((unsigned)p - page * block.d);
        return entry >= 0 && r < num_rows ? r : -1;
    }
};

}  // namespace dev
}  // namespace gdn
