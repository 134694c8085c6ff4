// kda_spans.h - the memory of strided tensors and whether two of them share any: plain arithmetic that the host's checks and a
// program on the CPU share.
#pragma once

#include <cstdint>

namespace kda {

// The memory of a tensor: `rows` rows `stride` bytes apart (not looked at for one), each of `parts` parts of `width` bytes,
// `part_stride` apart (the same).
struct Span {
    const char *name;
    uintptr_t at;
    int64_t rows, width, stride;
    int64_t parts = 1, part_stride = 0;
    bool empty() const { return !at || rows <= 0 || width <= 0 || parts <= 0; }
    int64_t row() const { return (parts - 1) * part_stride + width; }
    uintptr_t end() const { return at + static_cast<uintptr_t>((rows - 1) * stride + row()); }
};

// False only where no byte is in both: apart as a whole, or slices of one buffer that interleave.
inline bool overlap(const Span &a, const Span &b) {
    if (a.empty() || b.empty() || a.at >= b.end() || b.at >= a.end()) return false;
    // a single row lies in any distance of rows that holds it
    const int64_t s = a.rows > 1 ? a.stride : b.rows > 1 ? b.stride : int64_t{1} << 60;
    if ((b.rows > 1 && b.stride != s) || a.row() > s || b.row() > s) return true;
    // b's rows begin `off` bytes behind a's and may reach into a's next one
    const int64_t m = a.parts > 1 ? a.part_stride : b.part_stride;
    const int64_t off = ((static_cast<int64_t>(b.at - a.at) % s) + s) % s;
    // b's parts between a's, the rows this far apart
    auto between = [&](int64_t d) {
        if (m <= 0 || (a.parts > 1 && b.parts > 1 && a.part_stride != b.part_stride)) return false;
        const int64_t e = ((d % m) + m) % m;
        return e >= a.width && e + b.width <= m;
    };
    return !((off >= a.row() || between(off)) && (off + b.row() <= s || between(off - s)));
}

}  // namespace kda
