// kda_cache_device.h - attention of packed query rows over pages of the 8-bit cache: the
// part that the decode step and the attention with a common prefix share.
#pragma once

#include "kda_attn_device.h"

namespace kda {

// Operands of an fp32 path as bf16 parts: x = sum of the parts to 24 bits.  The
// codes are exact in bf16, so three products give the fp32 one.  In bf16 queries are
// exact as they are, and a probability times its page's scale (a power of two) is rounded
// once, 2^-8 relative at most, as in the forward; the sum is over the unrounded ones.
template <typename T> struct Parts { static constexpr int N = sizeof(T) == 2 ? 1 : 3; };

template <int N>
__device__ __forceinline__ void split_parts(const float (&x)[8], Frag<bf16_t> (&f)[N]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float r = x[j];
#pragma unroll
        for (int p = 0; p < N; ++p) {
            const bf16_t h = (bf16_t)r;
            f[p].v[j] = h;
            r -= (float)h;
        }
    }
}

// Eight codes (two words) as a matrix operand.
__device__ __forceinline__ Frag<bf16_t> codes_frag(uint32_t a, uint32_t b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false), x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true);
    const bf16x2 y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false), z = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
    Frag<bf16_t> f;
    f.v = bf16x8{w[0], w[1], x[0], x[1], y[0], y[1], z[0], z[1]};
    return f;
}

// Bytes 0 .. n-1 of a 16-byte piece, the others zero.
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int n) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = n - 4 * i;
        w[i] = k >= 4 ? w[i] : k <= 0 ? 0u : w[i] & ((1u << (8 * k)) - 1u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes that are NaN become zeros; whether there were any.
__device__ __forceinline__ bool drop_nan_codes(uint4& v) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w}, any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t nan = ((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;    // 0x7f and 0xff only carry
        w[i] &= ~(nan | (nan - (nan >> 7)));
        any |= nan;
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
    return any != 0;
}

// NaN where bit i is set.
__device__ __forceinline__ float nan_if(float x, uint32_t bits, int i) {
    return __uint_as_float(__float_as_uint(x) | ((uint32_t)((int32_t)(bits << (31 - i)) >> 31) & 0x7fc00000u));
}

constexpr int kStepKeys = 64;   // keys of a wave's block: 16 for each lane group

// The pages of one sequence and one key/value head.
struct PagedKeys {
    const uint8_t* k_cache; const uint8_t* v_cache; const float* k_scale; const float* v_scale;
    const int* table;
    int n_pages, page, HK, hk;
    int kl;                     // cached tokens
    float scale_log2;

    __device__ __forceinline__ int page_log2() const { return 31 - __builtin_clz(page); }
    // 16-key pieces of a lane's V keys (piece g of block kb) and of its K rows (piece lr / 4);
    // those past the last token repeat the last one
    __device__ __forceinline__ int2 pieces(int kb, int lane) const {
        const int last = (kl - 1) >> 4, first = kb * (kStepKeys / 16);
        return make_int2(min(first + (lane >> 4), last), min(first + ((lane & 15) >> 2), last));
    }
    // their table entries, asked for a block ahead: one wait less a block (the decode step over 4096
    // tokens 220 -> 216 us, eight groups' 32-row tiles on 4001 common keys 28 -> 27; codes a block
    // ahead as well take registers that more waves need: 42)
    __device__ __forceinline__ int2 entries(int kb, int lane) const {
        const int2 p = pieces(kb, lane);
        const int shift = page_log2() - 4;
        return make_int2(table[p.x >> shift], table[p.y >> shift]);
    }
};

// A wave's 16 NR packed rows and what they have gathered.  It takes blocks of 64 keys: lane
// group g stands for keys 16 g .. 16 g + 15 of the block, which lie in one page, in the
// order in which its V bytes come.  Score tile i is formed with K rows ordered so that
// its accumulator rows of group g are keys 16 g + 4 i .. + 3: the exponentials of the four
// tiles are then the right operands of the product with V without moving.  Scales enter
// as one factor per lane.
template <typename T, int D, int NR> struct CacheRows {
    static constexpr int NP = Parts<T>::N, NS = (D + 31) / 32, ND = D / 16;
    static constexpr int KW = D / 16;          // words of K a lane holds per tile
    int lo[NR], hi[NR];                        // first and last key that this lane's rows see
    Frag<bf16_t> qf[NR][NS][NP];
    float m[NR], l[NR];
    floatx4 o[ND][NR];
    uint32_t nans[NR];                         // this lane's elements of o (bit 4 d + e) that met a NaN code of v

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            nans[n] = 0u;
            m[n] = kNegInf;
            l[n] = 0.f;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d][n] = floatx4{0.f, 0.f, 0.f, 0.f};
        }
    }

    // This lane's row n from its first element, g = lane / 16.
    __device__ __forceinline__ void load_query(int n, const T* qp, int g) {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.f;
            if constexpr (D >= 32) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = to_f<T>(qp[g * (D / 4) + 8 * s + e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = to_f<T>(qp[4 * g + e]);
            }
            split_parts<NP>(x, qf[n][s]);
        }
    }

    // Keys 64 kb .. 64 kb + 63 below the length, in the pages of these entries.
    __device__ __forceinline__ void attend(const PagedKeys& c, int kb, int2 entries, int lane) {
        const int g = lane >> 4, lr = lane & 15;
        const int k0 = kb * kStepKeys, kl = c.kl;
        const int2 piece = c.pieces(kb, lane);
        const int shift = c.page_log2(), subv = piece.x, subk = piece.y;
        int pv = entries.x, pk = entries.y;
        const bool seen = pv >= 0 && pv < c.n_pages;         // a missing page is masked and reads page 0
        pv = seen ? pv : 0;
        pk = pk >= 0 && pk < c.n_pages ? pk : 0;
        const size_t sv = (size_t)pv * c.HK + c.hk, sk = (size_t)pk * c.HK + c.hk;
        const float ksc = c.k_scale[sv] * c.scale_log2, vsc = c.v_scale[sv];
        const uint8_t* kp = c.k_cache + (sk << shift) * D + (size_t)((subk * 16 & (c.page - 1)) + (lr & 3)) * D + g * (D / 4);
        const uint8_t* vp = c.v_cache + (sv << shift) * D + ((size_t)lr << shift) + (subv * 16 & (c.page - 1));
        uint32_t kw[4][KW];
        uint4 vw[ND];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t* p = kp + 4 * i * D;
            if constexpr (KW >= 4) {
#pragma unroll
                for (int w = 0; w < KW / 4; ++w) {
                    const uint4 x = reinterpret_cast<const uint4*>(p)[w];
                    kw[i][4 * w] = x.x; kw[i][4 * w + 1] = x.y; kw[i][4 * w + 2] = x.z; kw[i][4 * w + 3] = x.w;
                }
            } else {
#pragma unroll
                for (int w = 0; w < KW; ++w) kw[i][w] = reinterpret_cast<const uint32_t*>(p)[w];
            }
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) vw[d] = *reinterpret_cast<const uint4*>(vp + ((size_t)(16 * d) << shift));
        const int key0 = k0 + 16 * g, valid = seen ? kl - key0 : 0;  // this group's keys below the length
        if (!__all(valid >= 16)) {  // bytes past the last token may be anything, NaN codes among them
#pragma unroll
            for (int d = 0; d < ND; ++d) vw[d] = keep_bytes(vw[d], valid);
        }
        // Zero times a NaN code is NaN too: where a row sees none of these keys, NaN codes are left out and noted for
        // the rows that see some.
        bool every = true;
#pragma unroll
        for (int n = 0; n < NR; ++n) every = every && (hi[n] < 0 || (lo[n] < k0 + kStepKeys && hi[n] >= k0));   // < 0: a row that is not there
        if (!__all(every)) {
            uint32_t mine = 0;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const uint64_t who = __ballot(drop_nan_codes(vw[d])), pair = who | who >> 32;
                mine |= ((uint32_t)(pair | pair >> 16) >> (4 * g) & 15u) << (4 * d);
            }
#pragma unroll
            for (int n = 0; n < NR; ++n) nans[n] |= lo[n] < k0 + kStepKeys && hi[n] >= k0 ? mine : 0u;
        }

        floatx4 st[4][NR];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int n = 0; n < NR; ++n) st[i][n] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const Frag<bf16_t> kf = codes_frag(kw[i][KW >= 2 ? 2 * s : 0], KW >= 2 ? kw[i][KW >= 2 ? 2 * s + 1 : 0] : 0u);
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int p = 0; p < NP; ++p) st[i][n] = mma(kf, qf[n][s][p], st[i][n]);
            }
        }
        Frag<bf16_t> pf[2][NR][NP];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float x = kNegInf;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + 4 * i + e;
                    const float y = st[i][n][e] * ksc;
                    st[i][n][e] = seen && key >= lo[n] && key <= hi[n] ? y : kNegInf;
                    x = fmaxf(x, st[i][n][e]);
                }
            x = fmaxf(m[n], group_max4(x));
            const float mu = x == kNegInf ? 0.f : x, alpha = exp2_fast(m[n] - mu);
            m[n] = x;
            l[n] *= alpha;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d][n] *= alpha;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float pr[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = exp2_fast(st[2 * u + e / 4][n][e % 4] - mu);
                    l[n] += y;
                    pr[e] = y == 0.f ? 0.f : y * vsc;  // an unread page's scale may be anything
                }
                split_parts<NP>(pr, pf[u][n]);
            }
        }
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const Frag<bf16_t> vf = u == 0 ? codes_frag(vw[d].x, vw[d].y) : codes_frag(vw[d].z, vw[d].w);
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int p = 0; p < NP; ++p) o[d][n] = mma(vf, pf[u][n][p], o[d][n]);
            }
    }

    // Blocks first, first + by, .. below end.
    __device__ __forceinline__ void attend(const PagedKeys& c, int first, int end, int by, int lane) {
        if (first >= end) return;
        int2 now = c.entries(first, lane);
        for (int kb = first; kb < end; kb += by) {
            const int2 next = c.entries(min(kb + by, end - 1), lane);
            attend(c, kb, now, lane);
            now = next;
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
            if (__any(nans[n] != 0)) {
#pragma unroll
                for (int i = 0; i < 4 * ND; ++i) o[i / 4][n][i % 4] = nan_if(o[i / 4][n][i % 4], nans[n], i);
            }
    }
};

}  // namespace kda
