// gdn_check.h -- host-side argument checks shared by the C ABI layers (defined in
// gdn_api.cpp): the thread-local error message and the checks that set it.
#pragma once

#include <initializer_list>
#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "gdn.h"

namespace gdn {

void clear_error();
gdn_status fail(gdn_status st, const char* fmt, ...);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

gdn_status check_shape(const gdn_shape* s);

struct Ptr {
    const char* name;
    const void* p;
    size_t align;
};
gdn_status check_ptrs(std::initializer_list<Ptr> ps);

gdn_status hip_status(hipError_t e, const char* what);

}  // namespace gdn
