// gdn_checks.cuh -- host-side checks of arguments that the C entry points of
// the layer's and the block's operators share: alignment, the bytes of strided
// tensors and where they meet, lengths.
#pragma once

#include <initializer_list>

#include "../../include/gdn.h"
#include "gdn_layer.cuh"

namespace gdn {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int elem_size(int dtype) { return dtype == GDN_BF16 ? 2 : dtype == GDN_E4M3 ? 1 : 4; }
inline bool dtype_ok(int t) { return t == GDN_F32 || t == GDN_BF16; }
inline uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
inline gdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }
inline bool ws_ok(const void *ws, size_t have, size_t need) { return ws && have >= need && addr(ws) % kAlign == 0; }
inline bool f32_ok(const void *p) { return addr(p) % 4 == 0; }

// Strided rows: the base on an element, no negative stride; `wide` stays set
// while every row starts on a boundary of `bytes` (0: element rows only).
struct Rows {
    bool ok = true, wide = true;
    void add(const void *p, int dtype, int64_t sb, int64_t st, int bytes = 16) {
        if (!p) return;
        const int64_t e = elem_size(dtype);
        ok = ok && addr(p) % e == 0 && sb >= 0 && st >= 0;
        wide = wide && addr(p) % bytes == 0 && sb * e % bytes == 0 && st * e % bytes == 0;
    }
};

// The bytes of a tensor: T rows of `row` bytes, `st` apart, in B lines, `sb`
// apart; none for a null pointer.
struct Area {
    int64_t at, sb, st, B, T, row;
    int elem;
    Area(const void *p, int dtype, int64_t sb_, int64_t st_, int64_t B_, int64_t T_, int64_t n)
        : at((int64_t)addr(p)), sb(sb_ * elem_size(dtype)), st(st_ * elem_size(dtype)), B(p ? B_ : 0), T(T_),
          row(n * elem_size(dtype)), elem(elem_size(dtype)) {
        if (sb == T * st) T *= B, B = B > 0, sb = 0;  // lines that continue one another
    }
    Area(const void *p, int dtype, int64_t n) : Area(p, dtype, 0, 0, 1, 1, n) {}  // contiguous
    bool empty() const { return B <= 0 || T <= 0 || row <= 0; }
    int64_t line_bytes() const { return (T - 1) * st + row; }
    int64_t bytes() const { return (B - 1) * sb + line_bytes(); }
};
inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }
// Whether a row of line a and one of line b share a byte; b begins d bytes after a.
inline bool lines_meet(const Area &a, const Area &b, int64_t d) {
    if (d >= a.line_bytes() || -d >= b.line_bytes()) return false;
    // some k >= k0 with k <= k1 and from + k step in (-b.row, a.row)
    auto hit = [&](int64_t from, int64_t step, int64_t k0, int64_t k1) {
        int64_t k = step > 0 ? floor_div(-b.row - from, step) + 1 : k0;
        if (k < k0) k = k0;
        return k <= k1 && from + k * step < a.row && from + k * step > -b.row;
    };
    if (a.st == b.st) return hit(d, a.st, -(a.T - 1), b.T - 1);
    if (a.T > b.T) return lines_meet(b, a, -d);
    for (int64_t t = 0; t < a.T; ++t)
        if (hit(d - t * a.st, b.st, 0, b.T - 1)) return true;
    return false;
}
inline bool meet(const Area &a, const Area &b) {
    const int64_t d = b.at - a.at;
    if (a.empty() || b.empty() || d >= a.bytes() || -d >= b.bytes()) return false;
    if (a.sb == b.sb) {  // (only the difference of the lines counts)
        for (int64_t k = 1 - a.B; k < b.B; ++k)
            if (lines_meet(a, b, d + k * a.sb)) return true;
        return false;
    }
    if (a.B * b.B > 1 << 20) return true;  // too many pairs of lines to tell them apart here
    for (int64_t i = 0; i < a.B; ++i)
        for (int64_t j = 0; j < b.B; ++j)
            if (lines_meet(a, b, d + j * b.sb - i * a.sb)) return true;
    return false;
}
inline bool rows_apart(const Area &a) {  // of an output
    if (a.empty()) return true;
    if (a.T > 1 && a.st < a.row) return false;
    for (int64_t k = 1; k < a.B && k * a.sb < a.line_bytes(); ++k)
        if (lines_meet(a, a, k * a.sb)) return false;
    return true;
}
// Outputs must have rows of their own and overlap nothing; those in `placed`
// may lie exactly on an input of the same layout in `same`, which is read
// there by the threads that write it.
inline gdn_status areas_ok(std::initializer_list<Area> placed, std::initializer_list<Area> other,
                    std::initializer_list<Area> same, std::initializer_list<Area> in) {
    const auto exact = [](const Area &a, const Area &b) {
        return a.at == b.at && a.elem == b.elem && a.row == b.row && a.B == b.B && a.T == b.T &&
               (a.B == 1 || a.sb == b.sb) && (a.T == 1 || a.st == b.st);
    };
    for (const auto *outs : {&placed, &other})
        for (const Area *o = outs->begin(); o != outs->end(); ++o) {
            if (!rows_apart(*o)) return GDN_ERR_LAYOUT;
            for (const Area *q = o + 1; q != outs->end(); ++q)
                if (meet(*o, *q)) return GDN_ERR_UNSUPPORTED;
            for (const Area &q : same)
                if (meet(*o, q) && !(outs == &placed && exact(*o, q))) return GDN_ERR_UNSUPPORTED;
            for (const Area &q : in)
                if (meet(*o, q)) return GDN_ERR_UNSUPPORTED;
        }
    for (const Area &o : placed)
        for (const Area &q : other)
            if (meet(o, q)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// Tokens or rows: with room for what kernels and sizes add to them (a tile, a run).
inline bool length_ok(int n) { return n >= 0 && n <= INT32_MAX - 65535; }
inline bool norm_shape_ok(int R, int D) { return length_ok(R) && D >= 1 && D <= kNormMaxD; }
inline bool dense_ok(int B, int T, int D) { return B >= 1 && B <= 65535 && length_ok(T) && D >= 1 && D <= (1 << 20); }
// shapes of a dense or packed batch
inline bool batch_ok(int B, int T, int D, const int32_t *cu, int n_seq) {
    return dense_ok(B, T, D) && (cu ? B == 1 && n_seq >= 1 : n_seq == B);
}

}  // namespace gdn
