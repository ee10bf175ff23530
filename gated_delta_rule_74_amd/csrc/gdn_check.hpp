// Argument checks shared by the C ABI's sources: status texts, sizes, and what
// is asked of a call's buffers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include "gdn_launch.hpp"

namespace gdn::check {

inline gdn_status_t fail(gdn_status_t st, const char *fmt, ...) {
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return gdn::fail_detail(st, text);
}
inline gdn_status_t ok() { return gdn::fail_detail(GDN_OK, ""); }
inline gdn_status_t hip_status(hipError_t e, const char *what) {
    return e == hipSuccess ? ok() : fail(GDN_EHIP, "%s: %s", what, hipGetErrorString(e));
}

inline size_t align_up(size_t x) { return (x + 255) & ~(size_t)255; }
inline size_t esize(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }
constexpr double LIMIT = 2147483648.0; // elements of a tensor
constexpr double THREADS = 4294967296.0; // threads of a launch
// What the kernels add to a position or a count (a few tiles ahead, a thread's
// run) must not pass int32: sizes that bound those stay so much below it.
constexpr double AHEAD = 2048.0;
constexpr int CUS = 256;               // compute units of the chip the kernels are built for

// One buffer of a call.
struct Buf {
    const void *p;
    size_t n;
    const char *name;
    size_t align;
    bool out, need;
};

// Required pointers, alignment, and no output over another buffer. `same`:
// index pair of an input and an output that may be one buffer (-1: none).
inline gdn_status_t check_bufs(const Buf *b, int n, const int (*same)[2] = nullptr, int nsame = 0) {
    for (int i = 0; i < n; ++i) {
        if (b[i].need && b[i].n && !b[i].p) return fail(GDN_EINVAL, "%s is NULL", b[i].name);
        if (b[i].p && (uintptr_t)b[i].p % b[i].align)
            return fail(GDN_EINVAL, "%s must be %zu-byte aligned", b[i].name, b[i].align);
    }
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            if (!b[i].out || i == j || (b[j].out && j > i)) continue;
            if (!b[i].p || !b[j].p || !b[i].n || !b[j].n) continue;
            bool may = false;
            for (int k = 0; k < nsame; ++k)
                may |= same[k][0] == j && same[k][1] == i && b[i].p == b[j].p;
            const char *x = (const char *)b[i].p, *y = (const char *)b[j].p;
            if (!may && x < y + b[j].n && y < x + b[i].n)
                return fail(GDN_EINVAL, "output %s overlaps %s", b[i].name, b[j].name);
        }
    return GDN_OK;
}

} // namespace gdn::check
