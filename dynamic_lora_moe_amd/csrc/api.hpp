// What the C ABI's implementations share: statuses with their texts, and checks of
// arguments (no GPU call before they pass).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <vector>

#include "dlm.h"
#include "internal.hpp"

namespace dlm {

// Text of the calling thread's last failure.
inline thread_local char g_err[512] = "";

inline int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

inline int ok() {
    g_err[0] = 0;
    return DLM_OK;
}

inline int hip_fail(hipError_t e, const char* what) {
    if (e == hipErrorInvalidConfiguration)  // the launchers' own refusal (grid_fits)
        return fail(DLM_ESHAPE, "%s: the sizes need a launch grid of more than 2^32 - 1 work-items", what);
    (void)hipGetLastError();  // reported here: the next launch must not find it
    if (e == hipErrorOutOfMemory) return fail(DLM_ENOMEM, "%s: %s", what, hipGetErrorString(e));
    return fail(DLM_EHIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline size_t esize(int dtype) { return dtype == DLM_F32 ? 4 : 2; }

inline bool valid_dtype(int dtype) { return dtype == DLM_F32 || dtype == DLM_BF16; }

constexpr int64_t kMaxDim = (int64_t)1 << 30;

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

// A byte range a launch reads or writes.  The kernels update buffers in place
// from many workgroups, so a written range that overlaps any other range of the
// same call gives a silent race: such calls are refused.
struct Span {
    uintptr_t lo, hi;  // [lo, hi)
    bool write;
    const char* what;
    int who;
};

inline Span span(const void* p, size_t bytes, bool write, const char* what, int who) {
    return Span{(uintptr_t)p, (uintptr_t)p + bytes, write, what, who};
}

// First pair of overlapping spans of which at least one is written, or false.
// Sorted by start; for each span, the span reaching furthest so far and the
// written span reaching furthest so far are the only candidates that can
// overlap it while some earlier written span overlaps it, so one pass finds a
// conflict whenever there is one.
inline bool write_conflict(std::vector<Span> v, Span* a, Span* b) {
    std::sort(v.begin(), v.end(), [](const Span& x, const Span& y) { return x.lo < y.lo; });
    int far = -1, farw = -1;
    for (int k = 0; k < (int)v.size(); ++k) {
        if (v[k].hi <= v[k].lo) continue;
        if (far >= 0 && v[far].hi > v[k].lo && (v[k].write || v[far].write)) {
            *a = v[far];
            *b = v[k];
            return true;
        }
        if (farw >= 0 && v[farw].hi > v[k].lo) {
            *a = v[farw];
            *b = v[k];
            return true;
        }
        if (far < 0 || v[k].hi > v[far].hi) far = k;
        if (v[k].write && (farw < 0 || v[k].hi > v[farw].hi)) farw = k;
    }
    return false;
}

// The same for the few spans of one call, pair by pair: it allocates nothing.
template <int N> bool pair_conflict(const Span (&v)[N], Span* a, Span* b) {
    for (int i = 0; i < N; ++i)
        for (int k = 0; k < i; ++k)
            if (v[k].hi > v[i].lo && v[i].hi > v[k].lo && (v[k].write || v[i].write)) {
                *a = v[k];
                *b = v[i];
                return true;
            }
    return false;
}

inline int conflict_fail(const char* call, const Span& a, const Span& b) {
    return fail(DLM_EINVAL, "%s: %s %d overlaps %s %d, and one of them is written in place", call, a.what, a.who,
                b.what, b.who);
}

// Bytes from the first to behind the last element of T rows of n, ld apart.
inline size_t rows_bytes(int64_t T, int64_t ld, int64_t n, size_t es) { return ((size_t)(T - 1) * ld + n) * es; }

}  // namespace dlm
