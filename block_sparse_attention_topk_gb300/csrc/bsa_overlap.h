// bsa_overlap.h -- whether two strided tensors share memory (host).
#pragma once

#include <stdint.h>

namespace bsa {

// T x H rows of `bytes` bytes, row (t, h) at p + t * ts + h * hs; strides in
// bytes, not negative.
struct Rows {
    const void* p;
    int64_t T, H, bytes, ts, hs;
};
inline Rows whole_rows(const void* p, int64_t bytes) { return Rows{p, 1, 1, bytes, 0, 0}; }

// Exact.  Tensors whose address ranges are apart, as separate allocations are, cost
// a comparison; parts of one buffer (the same token stride) one division for each
// pair of heads, or each difference of heads where their strides agree too.
inline bool rows_overlap(Rows a, Rows b) {
    if (a.T < 1 || a.H < 1 || a.bytes < 1 || b.T < 1 || b.H < 1 || b.bytes < 1) return false;
    const int64_t start = (int64_t)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p));
    if (start >= (a.T - 1) * a.ts + (a.H - 1) * a.hs + a.bytes) return false;
    if (-start >= (b.T - 1) * b.ts + (b.H - 1) * b.hs + b.bytes) return false;
    if (a.T == 1) a.ts = b.ts;
    if (b.T == 1) b.ts = a.ts;
    if (a.H == 1) a.hs = b.hs;
    if (b.H == 1) b.hs = a.hs;
    auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y != 0 && x < 0); };
    // a token of b that is `off` bytes from one of a, for any difference lo..hi of tokens
    auto meets = [&](int64_t off, int64_t ts, int64_t lo, int64_t hi) {
        if (ts == 0) return off < a.bytes && off > -b.bytes;
        const int64_t first = floor_div(-b.bytes - off, ts) + 1, last = -floor_div(off - a.bytes, ts) - 1;
        return (first > lo ? first : lo) <= (last < hi ? last : hi);
    };
    const bool tokens = a.ts == b.ts, heads = a.hs == b.hs;
    for (int64_t t = 0; t < (tokens ? 1 : b.T); ++t) {
        const int64_t at = start + t * (tokens ? 0 : b.ts);
        const int64_t lo = 1 - a.T, hi = tokens ? b.T - 1 : 0;
        if (heads) {
            for (int64_t h = 1 - a.H; h < b.H; ++h)
                if (meets(at + h * a.hs, a.ts, lo, hi)) return true;
        } else {
            for (int64_t g = 0; g < a.H; ++g)
                for (int64_t h = 0; h < b.H; ++h)
                    if (meets(at + h * b.hs - g * a.hs, a.ts, lo, hi)) return true;
        }
    }
    return false;
}

}  // namespace bsa
