// host.h — host-side helpers shared by the C ABI's translation units (api.hip,
// api_products.hip): error reporting, pointer checks, the device check.  Internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_ffn.h"

namespace moe {
namespace host {

// Sets this thread's error text (moe_ffn_last_error) and returns `status`.
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t err, const char *what);
void clear_error();

#define HIP_TRY(expr, what)                                                                        \
    do {                                                                                           \
        hipError_t e_ = (expr);                                                                    \
        if (e_ != hipSuccess)                                                                      \
            return hip_fail(e_, what);                                                             \
    } while (0)

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline size_t elem_size(int dtype) { return dtype == MOE_FFN_BF16 ? 2 : 4; }

int check_ptr(const void *ptr, const char *name, size_t align = 16);
// The current device must be a gfx950 GPU; its compute units, and the rate of
// its constant wall clock.
int check_device(int *num_cus = nullptr, int *clock_khz = nullptr);
// The limits of moe_ffn_problem.
int validate_problem(const moe_ffn_problem *p);

template <typename P> P *at(void *base, size_t off)
{
    return reinterpret_cast<P *>(static_cast<char *>(base) + off);
}

} // namespace host
} // namespace moe
