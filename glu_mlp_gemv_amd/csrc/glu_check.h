// Checks of a call's arrays, shared by the files of the C ABI.  Host only: nothing here makes a HIP call.
#pragma once

#include <stdint.h>

#include "../../include/glu_gemv.h"

namespace glu {

constexpr int64_t kMaxDim = (int64_t)1 << 30;  // rows and columns index in 32 bits, rounded up to tiles

inline bool bad_dim(int64_t v) { return v < 0 || v > kMaxDim; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// An array of `rows` rows of `len` elements at stride `ld`.
struct Array {
    const void* p;
    int64_t rows, len, ld;
    int size;  // bytes per element
    bool output;
};

// bytes from the first to past the last element; -1 if that does not fit
inline int64_t extent(const Array& a)
{
    if (a.rows == 0 || a.len == 0) return 0;
    const int64_t limit = INT64_MAX / a.size;
    if (a.rows > 1 && a.ld > (limit - a.len) / (a.rows - 1)) return -1;
    return ((a.rows - 1) * a.ld + a.len) * a.size;
}

constexpr int kMaxArrays = 16;

// NULL, strides, alignment and overlap of a call's arrays, in that order.  An output may coincide exactly
// (pointer and stride) with the inputs in `shared`, a bit per array.
inline glu_status check_arrays(const Array* a, int n, unsigned shared_out = 0, unsigned shared_in = 0)
{
    int64_t bytes[kMaxArrays];
    for (int i = 0; i < n; ++i) {
        if (a[i].rows > 1 && a[i].ld < a[i].len) return GLU_ERR_BAD_STRIDE;
        bytes[i] = extent(a[i]);
        if (bytes[i] < 0) return GLU_ERR_BAD_STRIDE;
    }
    for (int i = 0; i < n; ++i) {
        if (bytes[i] > 0 && !a[i].p) return GLU_ERR_NULL_POINTER;
    }
    for (int i = 0; i < n; ++i) {
        if (bytes[i] > 0 && ((uintptr_t)a[i].p & (uintptr_t)(a[i].size - 1))) return GLU_ERR_MISALIGNED;
    }
    for (int i = 0; i < n; ++i) {
        if (!a[i].output || bytes[i] == 0) continue;
        for (int j = 0; j < n; ++j) {
            if (j == i || bytes[j] == 0 || (a[j].output && j < i)) continue;
            const bool exact = a[i].p == a[j].p && a[i].len == a[j].len && (a[i].rows <= 1 || a[i].ld == a[j].ld);
            if (exact && (shared_out >> i & 1) && (shared_in >> j & 1)) continue;
            const uintptr_t p = (uintptr_t)a[i].p, q = (uintptr_t)a[j].p;
            if (p < q + (uintptr_t)bytes[j] && q < p + (uintptr_t)bytes[i]) return GLU_ERR_ALIASING;
        }
    }
    return GLU_OK;
}

}  // namespace glu
