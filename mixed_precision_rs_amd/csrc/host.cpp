// Checks of row-strided matrix arguments (host.hpp).
#include "host.hpp"

namespace tide {

tide_status matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t stride,
                   int32_t size, Mat* out) {
    *out = Mat{name, reinterpret_cast<uintptr_t>(p), 0, 0, 0};
    if (rows < 0 || cols < 0) return fail(TIDE_ERR_INVALID_ARG, "%s has a negative size", name);
    if (rows == 0 || cols == 0) return TIDE_OK;
    if (stride < cols)
        return fail(TIDE_ERR_INVALID_ARG, "%s: row stride %lld < %lld columns", name,
                    (long long)stride, (long long)cols);
    int64_t bytes;
    if (__builtin_mul_overflow(rows, stride, &bytes) || __builtin_mul_overflow(bytes, size, &bytes))
        return fail(TIDE_ERR_OVERFLOW, "%s: its extent overflows int64", name);
    if (!p) return fail(TIDE_ERR_INVALID_ARG, "%s is NULL", name);
    if (out->base & (uintptr_t)(size - 1))
        return fail(TIDE_ERR_ALIGNMENT, "%s is not %d-byte aligned", name, size);
    out->rows = rows;
    out->width = cols * size;
    out->stride = stride * size;
    return TIDE_OK;
}

namespace {
bool share(const Mat& a, const Mat& b) {
    if (a.rows == 0 || b.rows == 0) return false;
    const uintptr_t ae = a.base + (uintptr_t)((a.rows - 1) * a.stride + a.width);
    const uintptr_t be = b.base + (uintptr_t)((b.rows - 1) * b.stride + b.width);
    if (ae <= b.base || be <= a.base) return false;
    if (a.stride != b.stride) return true;
    const int64_t d = (int64_t)((b.base > a.base ? b.base - a.base : a.base - b.base) %
                                (uintptr_t)a.stride);
    const int64_t first = b.base > a.base ? a.width : b.width;
    const int64_t second = b.base > a.base ? b.width : a.width;
    return d < first || d + second > a.stride;
}
}  // namespace

tide_status no_overlap(const Mat* written, int nw, const Mat* read, int nr) {
    for (int i = 0; i < nw; ++i) {
        for (int j = 0; j < i; ++j)
            if (share(written[i], written[j]))
                return fail(TIDE_ERR_INVALID_ARG, "%s overlaps %s", written[i].name, written[j].name);
        for (int j = 0; j < nr; ++j)
            if (share(written[i], read[j]))
                return fail(TIDE_ERR_INVALID_ARG, "%s overlaps %s", written[i].name, read[j].name);
    }
    return TIDE_OK;
}

}  // namespace tide
