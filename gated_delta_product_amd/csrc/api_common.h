// api_common.h -- error reporting and small helpers shared by the C ABI's
// translation units (host side).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gdp.h"

namespace gdp {
namespace api {

// Sets this thread's message (gdp_last_error) and returns st.
gdp_status fail(gdp_status st, const char *fmt, ...);
// Clears it and returns GDP_OK.
gdp_status ok();
// GDP_OK, or GDP_ERR_HIP with the error's name after `what`.
gdp_status hip_status(hipError_t e, const char *what);

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Whether a launch of so many threads along x is allowed (HIP: under 2^32).
inline bool fits_launch(int64_t threads) { return threads <= 0xffffffffll; }
constexpr int64_t kAlign = 256;  // of a workspace and of the arrays in it
// A workspace of `bytes` where `need` (0: none) are used.
gdp_status check_space(const char *name, const void *ws, int64_t bytes, int64_t need);
inline size_t dsize(gdp_dtype d) { return d == GDP_BF16 ? 2 : 4; }

}  // namespace api
}  // namespace gdp
