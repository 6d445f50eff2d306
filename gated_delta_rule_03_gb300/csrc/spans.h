// spans.h -- host checks of pointer arguments: alignment and overlaps.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/gdr.h"

namespace gdr {

struct Bytes {
    const void *p;
    size_t n;
};
inline bool overlapping(const Bytes &a, const Bytes &b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const char *x = (const char *)a.p, *y = (const char *)b.p;
    return x < y + b.n && y < x + a.n;
}
// No output overlaps an input or another output.
inline bool outputs_apart(const Bytes *in, int ni, const Bytes *out, int no) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlapping(out[i], in[j])) return false;
        for (int j = 0; j < i; ++j)
            if (overlapping(out[i], out[j])) return false;
    }
    return true;
}
inline bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// Bytes that `tokens` rows of heads * d elements reach over with a stride between them.
inline size_t reach(int64_t tokens, int64_t stride, int64_t row, size_t e) {
    return tokens == 0 ? 0 : ((size_t)(tokens - 1) * stride + (size_t)row) * e;
}
// A token stride in elements (0: dense): at least dense, below 2^31, a multiple of 16 bytes.
inline int row_stride(int64_t given, int64_t dense, size_t e, int64_t *out) {
    *out = given == 0 ? dense : given;
    if (*out < dense || *out > INT32_MAX) return GDR_ERR_INVALID_ARG;
    return (*out * (int64_t)e) % 16 == 0 ? GDR_OK : GDR_ERR_ALIGNMENT;
}

// Rows of a tensor: `tokens` of them, `row` bytes each, `stride` bytes apart.
struct Rows {
    const void *p;
    int64_t tokens, stride, row;
};
// Whether two of them share a byte. Views of one buffer's rows lie within each other's reach without
// sharing one; those have the same stride, and their places in a row are compared.
inline bool sharing(const Rows &a, const Rows &b) {
    if (!a.p || !b.p || a.tokens == 0 || b.tokens == 0) return false;
    const Bytes x = {a.p, (size_t)((a.tokens - 1) * a.stride + a.row)}, y = {b.p, (size_t)((b.tokens - 1) * b.stride + b.row)};
    if (!overlapping(x, y)) return false;
    if (a.stride != b.stride || a.tokens == 1 || b.tokens == 1) return true;
    int64_t off = ((const char *)b.p - (const char *)a.p) % a.stride;
    if (off < 0) off += a.stride;
    return off < a.row || a.stride - off < b.row;
}

}  // namespace gdr
