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

// rows x [cols of ld] buffers of element size `size`
struct Span {
    const void *p;
    int64_t rows, ld, cols, size;
    uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t end() const { return begin() + (uintptr_t)(((rows - 1) * ld + cols) * size); }
};
inline bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.begin() >= b.end() || b.begin() >= a.end()) return false;
    // two column ranges of one wide buffer: rows of the same pitch whose columns
    // do not meet (b's start d bytes behind a's, counted round the pitch)
    const uintptr_t pitch = (uintptr_t)(a.ld * a.size);
    if (pitch == 0 || pitch != (uintptr_t)(b.ld * b.size)) return true;
    const uintptr_t d = (b.begin() % pitch + pitch - a.begin() % pitch) % pitch;
    return d < (uintptr_t)(a.cols * a.size) || pitch - d < (uintptr_t)(b.cols * b.size);
}
// an output that may stand exactly on an input (each value is read before its
// place is written) but not elsewhere in it
inline bool apart_or_same(const Span &out, const Span &in) {
    return !overlap(out, in) || (out.p == in.p && out.ld == in.ld);
}

// element, layout and shape rules of a weight of E experts x [N, K]
mx_status shape_ok(int elem, int layout, int64_t E, int64_t N, int64_t K);
// whether the current device is one the kernels are built for
mx_status device_ok();
// whether the batch-invariant mode is on (mx_set_batch_invariant)
bool batch_invariant();
// one line to stderr with MX_LOG=1
__attribute__((format(printf, 1, 2))) void log_dispatch(const char *fmt, ...);

}  // namespace mx
