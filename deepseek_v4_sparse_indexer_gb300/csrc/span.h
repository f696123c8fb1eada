// Rows of a caller's buffer, and whether two buffers have a byte in common (host only).
#pragma once

#include <cstdint>

namespace ds4a {

// `rows` rows of `width` bytes, `stride` (>= width) bytes apart.
struct Span {
    const void *at;              // null: nothing
    long long rows, stride, width;
    int type;                    // of an element
};

inline bool overlap(const Span &a, const Span &b) {
    if (!a.at || !b.at) return false;
    // row i of a begins at i a.stride, row j of b at d + j b.stride
    const long long d = static_cast<long long>(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at));
    if (d >= (a.rows - 1) * a.stride + a.width || -d >= (b.rows - 1) * b.stride + b.width) return false;
    // Row i of a against b's: the last that begins no later, and the next.
    const auto meets = [&](long long i) {
        const long long at = i * a.stride;
        long long j = b.rows > 1 && at > d ? (at - d) / b.stride : 0;
        if (j > b.rows - 1) j = b.rows - 1;
        for (const long long end = j + 2 < b.rows ? j + 2 : b.rows; j < end; ++j) {
            const long long to = d + j * b.stride;
            if (to < at + a.width && at < to + b.width) return true;
        }
        return false;
    };
    if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {
        // Rows meet by the difference of their numbers alone: a's first row stands for b's
        // later ones, a's rows around b's first one for the others.
        const long long k = d > 0 ? d / a.stride : 0;
        return meets(0) || (k < a.rows && meets(k)) || (k + 1 < a.rows && meets(k + 1));
    }
    for (long long i = 0; i < a.rows; ++i)
        if (meets(i)) return true;
    return false;
}

// In place: element by element the same bytes.
inline bool same(const Span &a, const Span &b) {
    return a.at == b.at && a.type == b.type && a.width == b.width && a.rows == b.rows && (a.rows == 1 || a.stride == b.stride);
}

}  // namespace ds4a
