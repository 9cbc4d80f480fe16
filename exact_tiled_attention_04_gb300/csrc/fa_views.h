// Host-side checks of fa_rows_t views.  Not part of the public C ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"

namespace fa {
namespace host {

constexpr int64_t kMaxStride = int64_t{1} << 38;  // elements; a tensor map's strides are below 2^40 bytes

// A view with the strides that do not matter set to ones that do not disturb.
struct View {
    char* data;
    int64_t row, head;  // strides in elements
    int64_t rows, heads, d;
    bool by_row;        // all heads of a row lie before the next row

    size_t span() const { return rows == 0 ? 0 : static_cast<size_t>((rows - 1) * row + (heads - 1) * head + d) * 2; }
};

inline int make_view(const fa_rows_t* r, int64_t rows, int64_t heads, int64_t d, View* v) {
    if (r == nullptr || (r->data == nullptr && rows > 0)) return FA_ERR_INVALID_ARG;
    *v = View{static_cast<char*>(r->data), r->row_stride, r->head_stride, rows, heads, d, true};
    if (rows <= 1) v->row = (heads - 1) * (heads > 1 ? v->head : 0) + d;
    if (heads <= 1) v->head = d;
    if (v->row < 1 || v->head < 1) return FA_ERR_INVALID_ARG;
    if (v->row > kMaxStride || v->head > kMaxStride) return FA_ERR_UNSUPPORTED;
    if (v->row % 8 != 0 || v->head % 8 != 0) return FA_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(v->data) & 15u) return FA_ERR_ALIGNMENT;
    // (strides below 2^38 and counts below 2^31 may exceed 2^63 together)
    if ((rows > 1 && v->row > (int64_t{1} << 61) / rows) || (heads > 1 && v->head > (int64_t{1} << 61) / heads))
        return FA_ERR_INVALID_ARG;
    v->by_row = rows <= 1 || v->row >= (heads - 1) * v->head + d;
    if (v->head < d || v->row < d) return FA_ERR_INVALID_ARG;
    if (!v->by_row && heads > 1 && v->head < (rows - 1) * v->row + d) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// Elements at the addresses a + [0, wa) and b + [0, wb), each repeated every
// `period` bytes, have none in common.
inline bool apart(const View& a, int64_t wa, const View& b, int64_t wb, int64_t period) {
    int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.data) - reinterpret_cast<uintptr_t>(a.data)) % period;
    if (off < 0) off += period;
    return off >= wa && off + wb <= period;
}

// The distance in bytes that all of a view's strides are multiples of, where
// the smaller one is that (a stride that is not used counts as one), else 0.
inline int64_t step_of(const View& v) {
    if (v.rows <= 1 && v.heads <= 1) return 0;
    const int64_t row = v.rows <= 1 ? v.head : v.row, head = v.heads <= 1 ? v.row : v.head;
    const int64_t small = row < head ? row : head;
    return row % small == 0 && head % small == 0 ? small * 2 : 0;
}

// Views with no element in common: their spans do not meet; or both have rows
// equally far apart and their heads take different parts of a row's distance
// ([rows, heads of q, of k, of v]); or their rows of d elements take different
// parts of a distance that all their strides are multiples of ([rows, heads, 3, d]).
inline bool disjoint(const View& a, const View& b) {
    if (a.rows == 0 || b.rows == 0) return true;
    if (!overlaps(a.data, a.span(), b.data, b.span())) return true;
    if (a.by_row && b.by_row && a.row == b.row &&
        apart(a, ((a.heads - 1) * a.head + a.d) * 2, b, ((b.heads - 1) * b.head + b.d) * 2, a.row * 2))
        return true;
    const int64_t step = step_of(a);
    return step > 0 && step == step_of(b) && apart(a, a.d * 2, b, b.d * 2, step);
}

// A view and n bytes at p with any byte between them.
inline bool meets(const View& v, const void* p, size_t n) {
    return v.rows > 0 && p != nullptr && n > 0 && overlaps(v.data, v.span(), p, n);
}

}  // namespace host
}  // namespace fa
