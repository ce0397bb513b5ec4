// rows_host.h -- whether two matrices of strided rows share memory, for the argument
// checks of the decoder-layer operators.
#pragma once

#include <cstdint>

namespace vlmce {

// `rows` rows of `bytes` bytes (<= ld), ld bytes apart.
struct RowsOf {
    const void *p;
    int64_t rows, bytes, ld;
};

// Columns side by side in one buffer (rows equally far apart, none reaching into
// another's) do not overlap, although the spans of memory do.  Rows of different
// strides whose spans meet count as overlapping.
inline bool rows_overlap(RowsOf a, RowsOf b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    if (pb >= pa + static_cast<uintptr_t>((a.rows - 1) * a.ld + a.bytes) ||
        pa >= pb + static_cast<uintptr_t>((b.rows - 1) * b.ld + b.bytes))
        return false;
    if (a.rows == 1 && b.rows == 1) return true;
    if (a.rows == 1) a.ld = b.ld;
    if (b.rows == 1) b.ld = a.ld;
    if (a.ld != b.ld || a.bytes > a.ld || b.bytes > b.ld) return true;
    const int64_t d = static_cast<int64_t>(pb - pa) % a.ld;
    const int64_t r = d < 0 ? d + a.ld : d;  // where b's rows start in a's
    return r < a.bytes || r + b.bytes > a.ld;
}

}  // namespace vlmce
