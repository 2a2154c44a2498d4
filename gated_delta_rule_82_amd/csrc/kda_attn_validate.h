// kda_attn_validate.h - host-side argument checks shared by the entry points of the
// softmax attention and of its cache.  None of them makes a HIP call.
#pragma once

#include <math.h>

#include "kda_attn.h"
#include "kda_validate.h"

namespace kda {
namespace host {

constexpr double kLog2eD = 1.44269504088896340736;

inline bool heads_ok(int H, int HK) { return H >= 0 && HK >= 0 && (H == 0 || (HK > 0 && H % HK == 0)); }

inline bool rows_ok(int B, int Tq, int H, int HK) {
    if (!heads_ok(H, HK) || !sizes_ok(B, Tq, H)) return false;
    if (H == 0) return true;
    // packed rows of one key/value head, and less than 2^24 workgroups of 32 of them
    // (a grid holds less than 2^32 threads, a workgroup 256)
    const unsigned long long rows = (unsigned long long)(H / HK) * Tq;
    return rows <= (1ull << 29) && (unsigned long long)B * HK * (rows / 32 + 1) < (1ull << 24);
}

// A paged cache: its length only bounds a loop.
inline bool step_sizes_ok(int B, int Tq, int H, int HK, int max_len) {
    return max_len >= 0 && max_len <= (1 << 29) && rows_ok(B, Tq, H, HK);
}

// Row stride in elements, at most `most`: 0 selects contiguous tokens.
inline kda_status stride(int ld, int most, int heads, int D, kda_dtype dt, size_t* out) {
    const long long least = (long long)heads * D;
    if (ld < 0 || (ld > 0 && ld < least) || ld > most || least > kTileStride) return KDA_ERR_SHAPE;
    *out = ld ? (size_t)ld : (size_t)least;
    return (*out * elem_bytes(dt)) % 16 == 0 ? KDA_OK : KDA_ERR_ALIGN;
}

inline Rows rows_of(const void* p, size_t tokens, size_t ld, size_t heads, size_t D, kda_dtype dt) {
    const size_t e = (size_t)elem_bytes(dt);
    return Rows{p, tokens, ld * e, heads * D * e};
}
// n bytes in one piece, for comparison with strided rows
inline Rows bytes_of(const void* p, size_t n) { return Rows{p, n ? (size_t)1 : 0, n, n}; }

inline bool overlaps_any(const Rows& out, const Rows* in, size_t n) {
    for (size_t i = 0; i < n; ++i)
        if (overlaps(out, in[i])) return true;
    return false;
}

inline kda_status check_workspace(const void* ws, size_t have, size_t want) {
    if (want == 0) return KDA_OK;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || have < want) return KDA_ERR_WORKSPACE;
    return KDA_OK;
}

inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// Partial results of a key axis split over n workgroups: n x rows outputs of D
// floats, then as many (maximum, sum) pairs.
inline size_t split_bytes(int n, size_t rows, int D) {
    return n <= 1 ? 0 : round256((size_t)n * rows * D * 4) + round256((size_t)n * rows * 8);
}

// The kernels use it times log2 e, the backward lse over it.
inline bool scale_ok(float s) { return s >= 0x1p-64f && isfinite((float)(s * kLog2eD)); }

inline bool cache_sizes_ok(int n_pages, int max_pages, int B, int T, int HK, int D, int page) {
    if (!dim_ok(D) || (page != 16 && page != 32 && page != 64 && page != 128)) return false;
    if (n_pages < 0 || max_pages < 0 || !sizes_ok(B, T, HK)) return false;
    return (unsigned long long)n_pages * (unsigned)HK <= (1ull << 30) &&
           (unsigned long long)max_pages * (unsigned)page <= (1ull << 30) &&
           (unsigned long long)B * (unsigned)max_pages <= (1ull << 40);
}

}  // namespace host
}  // namespace kda
