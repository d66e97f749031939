// What the library's translation units share on the host side.
#pragma once

#include <cstddef>
#include <cstdint>

constexpr size_t kErrorText = 512;

// The calling thread's message for its last nonzero return (zero_last_error).
__attribute__((visibility("hidden"))) char* zero_error_text();

namespace {

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }  // b > 0

// Where matrices are: `count` of them `stride` bytes apart, each `rows` runs of `width`
// bytes `ld` bytes apart (ld >= width, stride >= a matrix).
struct Place {
    const void* at;
    int64_t rows, width, ld, count, stride;
    int64_t span() const { return (rows - 1) * ld + width; }  // of one matrix
    Place(const void* p, int64_t r, int64_t w, int64_t l, int64_t c = 1, int64_t s = 0)
        : at(p), rows(r), width(w), ld(l), count(c), stride(s) {}
    Place(const void* p, int64_t bytes) : Place(p, 1, bytes, bytes) {}
};

// Whether runs of wa bytes at 0, la, .. (na of them) meet runs of wb bytes at d, d + lb, ..
// (nb of them): f(e) says so of two runs whose bytes' ranges do, e from the one's start
// to the other's.
template <class F>
bool runs_meet(int64_t na, int64_t wa, int64_t la, int64_t d, int64_t nb, int64_t wb, int64_t lb, F f) {
    if (na == 0 || nb == 0 || d >= (na - 1) * la + wa || d + (nb - 1) * lb + wb <= 0) return false;
    if (na == 1) la = lb;
    if (nb == 1) lb = la;
    if (na == 1 && nb == 1) return f(d);
    int64_t i = floor_div(d - wa, la);
    if (la == lb) {  // e = d - (run of the one - run of the other) la
        for (i = i > 1 - nb ? i : 1 - nb; i < na && i * la < d + wb; ++i)
            if (d - i * la < wa && f(d - i * la)) return true;
        return false;
    }
    for (i = i > 0 ? i : 0; i < na && i * la < d + (nb - 1) * lb + wb; ++i) {
        int64_t j = floor_div(i * la - d - wb, lb);
        for (j = j > 0 ? j : 0; j < nb && d + j * lb - i * la < wa; ++j)
            if (d + j * lb - i * la > -wb && f(d + j * lb - i * la)) return true;
    }
    return false;
}

// Whether two such places share a byte; null ones share none.
inline bool overlap(const Place& a, const Place& b) {
    if (a.at == nullptr || b.at == nullptr || a.width == 0 || b.width == 0 || a.rows == 0 || b.rows == 0) return false;
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at));
    return runs_meet(a.count, a.span(), a.stride, d, b.count, b.span(), b.stride, [&](int64_t e) {
        return runs_meet(a.rows, a.width, a.ld, e, b.rows, b.width, b.ld, [](int64_t) { return true; });
    });
}

}  // namespace
