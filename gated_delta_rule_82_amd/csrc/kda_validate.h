// kda_validate.h - host-side argument checks shared by the C ABI's entry points.
// None of them makes a HIP call.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {
namespace host {

inline bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool dtype_ok(kda_dtype dt) { return dt == KDA_F32 || dt == KDA_BF16; }
inline int elem_bytes(kda_dtype dt) { return dt == KDA_BF16 ? 2 : 4; }

// Checks a pointer that must be present; optional ones pass when NULL.
inline kda_status need(const void* p) {
    if (!p) return KDA_ERR_NULL;
    return aligned16(p) ? KDA_OK : KDA_ERR_ALIGN;
}
inline kda_status maybe(const void* p) { return (!p || aligned16(p)) ? KDA_OK : KDA_ERR_ALIGN; }

// Sizes the kernels index with 32-bit arithmetic: at most 2^24 (b, h) pairs,
// 2^30 tokens and 2^46 / 128 token rows.
inline bool sizes_ok(long long B, long long T, long long H) {
    if (B < 0 || T < 0 || H < 0) return false;
    const unsigned long long bh = (unsigned long long)B * (unsigned long long)H;
    return bh <= (1ull << 24) && T <= (1ll << 30) && bh * (unsigned long long)T * 128ull <= (1ull << 46);
}

// Byte ranges [a, a + na) and [b, b + nb) share a byte (both non-empty).
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

// Bytes [p, p + rows * ld) hold `rows` rows of `width` bytes, one every `ld`.
struct Rows {
    const void* p; size_t rows, ld, width;
    size_t extent() const { return rows ? (rows - 1) * ld + width : 0; }
};
// Two such sets of rows share a byte.  Rows of one stride that interleave (the
// q, k and v parts of one packed projection) are told apart; with different
// strides sharing the extent counts as sharing a byte.
inline bool overlaps(const Rows& a, const Rows& b) {
    if (!a.p || !b.p || !overlaps(a.p, a.extent(), b.p, b.extent())) return false;
    if (a.ld != b.ld) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const size_t d = y >= x ? (y - x) % a.ld : (a.ld - (x - y) % a.ld) % a.ld;  // b's row start within a's stride
    return d < a.width || a.ld - d < b.width;
}

}  // namespace host
}  // namespace kda

#define KDA_TRY(expr)                        \
    do {                                     \
        const kda_status st_ = (expr);       \
        if (st_ != KDA_OK) return st_;       \
    } while (0)

