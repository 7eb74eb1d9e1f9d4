// mx_host.h -- what the host sources behind include/mx.h share: argument
// checks, the gfx950 gate and the dispatch trace (defined in mx_api.cpp).
// Not part of the public ABI.
#pragma once

#include "../../include/mx.h"
#include "mx_kernels.h"

namespace mx {

constexpr int64_t kMaxRsrc = (int64_t(1) << 31) - 1;   // 32-bit buffer offsets

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }
inline mx_status launched(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_LAUNCH; }

// element, layout and shape rules of a weight of E experts x [N, K]
mx_status shape_ok(int elem, int layout, int64_t E, int64_t N, int64_t K);
// whether the current device is one the kernels are built for
mx_status device_ok();
// whether the batch-invariant mode is on (mx_set_batch_invariant)
bool batch_invariant();
// one line to stderr with MX_LOG=1
__attribute__((format(printf, 1, 2))) void log_dispatch(const char *fmt, ...);

}  // namespace mx
