// api_util.hpp -- host helpers shared by the translation units that hold the
// C ABI (api.hip, api_block.hip): workspace carving and argument checks.
#pragma once

#include "w4a8.h"

#include <stddef.h>
#include <stdint.h>

namespace w4a8 {
namespace api {

constexpr size_t kAlign = 256;

inline size_t round_up(size_t x)
{
    return (x + kAlign - 1) / kAlign * kAlign;
}
inline bool aligned16(const void* p)
{
    return ((uintptr_t)p & 15u) == 0;
}

// A bump allocator over the caller's workspace (or over nothing, to size it).
struct Carve {
    char* base;
    size_t used = 0;
    explicit Carve(void* b) : base((char*)b) {}
    template <typename T>
    T* take(size_t count)
    {
        T* p = base ? (T*)(base + used) : nullptr;
        used += round_up(count * sizeof(T));
        return p;
    }
};

inline int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

// products of non-negative sizes without int64 overflow (limit 2^62)
inline int64_t mul_sat(int64_t a, int64_t b)
{
    const int64_t cap = (int64_t)1 << 62;
    if (a <= 0 || b <= 0)
        return 0;
    return a > cap / b ? cap : a * b;
}

inline int check_workspace(void* ws, size_t* bytes, size_t need)
{
    if (bytes == nullptr)
        return W4A8_ERR_INVALID_ARG;
    if (ws == nullptr) {
        *bytes = need;
        return W4A8_OK;
    }
    if (*bytes < need)
        return W4A8_ERR_WORKSPACE;
    if (!aligned16(ws))
        return W4A8_ERR_UNSUPPORTED;
    return -1;  // proceed
}

inline int hip_status(hipError_t e)
{
    return e == hipSuccess ? W4A8_OK : W4A8_ERR_HIP;
}

}  // namespace api
}  // namespace w4a8
