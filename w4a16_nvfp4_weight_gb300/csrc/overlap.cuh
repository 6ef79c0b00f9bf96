// Host checks that a call's outputs do not lie over its inputs or each other.
#pragma once

#include <algorithm>
#include <cstdint>
#include <initializer_list>

namespace nvfp4 {

// `rows` rows of `bytes` bytes, `stride` bytes apart.
struct Span {
    const char* name;
    uintptr_t at;
    int64_t rows, stride, bytes;

    bool empty() const { return at == 0 || rows <= 0 || bytes <= 0; }
    bool dense() const { return rows <= 1 || stride == bytes; }
    int64_t extent() const { return (rows - 1) * stride + bytes; }
};

inline Span dense_span(const char* name, const void* p, int64_t bytes) { return {name, (uintptr_t)p, 1, 0, bytes}; }

// Rows of `bytes` bytes over dimensions of n elements, s bytes apart: the dimension of the
// largest step counts as rows, all others as filled.
struct Dim { int64_t n, s; };
inline Span strided_span(const char* name, const void* p, int64_t bytes, std::initializer_list<Dim> dims) {
    Dim most{1, 0};
    for (const Dim& d : dims) {
        if (d.n <= 0) return dense_span(name, p, 0);
        if (d.n > 1 && d.s > most.s) most = d;
    }
    bool taken = false;
    for (const Dim& d : dims) {
        if (!taken && most.n > 1 && d.n == most.n && d.s == most.s) taken = true;
        else bytes += (d.n - 1) * d.s;
    }
    return {name, (uintptr_t)p, most.n, most.s, bytes};
}

// Whether a dense `out` shares a byte with `in`.
inline bool overlaps(const Span& out, const Span& in) {
    if (out.empty() || in.empty()) return false;
    const int64_t lo = (int64_t)out.at - (int64_t)in.at, hi = lo + out.bytes;     // of `out`, from the first row on
    if (in.rows == 1 || in.stride == 0) return lo < in.bytes && hi > 0;
    if (hi <= 0 || lo >= in.extent()) return false;
    const int64_t last = std::min(in.rows - 1, (hi - 1) / in.stride);                 // row that begins below hi
    const int64_t first = lo < in.bytes ? 0 : (lo - in.bytes) / in.stride + 1;        // row that ends above lo
    return first <= last;
}

// Whether dense `out` is `in` itself, element for element.
inline bool same_place(const Span& out, const Span& in) { return out.at == in.at && in.dense() && out.bytes == in.rows * in.bytes; }

// The name of the first of `spans` that `out` overlaps, or null.
inline const char* met(const Span& out, std::initializer_list<Span> spans) {
    for (const Span& s : spans)
        if (overlaps(out, s)) return s.name;
    return nullptr;
}

}  // namespace nvfp4
