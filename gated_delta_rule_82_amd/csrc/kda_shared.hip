// kda_shared.hip - attention of new tokens over the 8-bit cache where groups of sequences
// have a common prefix, on gfx950.
//
// The keys of a group's prefix are the same for all of its rows (N sequences of Tq tokens
// of G query heads for each key/value head), so they are read once a group instead of once
// a sequence; the keys behind the prefix are each sequence's own.  One launch does both:
// its first workgroups take tiles of a group's rows over parts of the prefix, the others a
// sequence's rows over parts of its own keys, and every part leaves its unnormalised
// output, maximum and sum for the join of split key axes,
//   o = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p.
#include <limits.h>

#include <type_traits>

#include "kda_branch.h"
#include "kda_cache_device.h"

namespace kda {

namespace {

constexpr int kSharedWaves = 4;

struct Group {
    int first, last, prefix;    // sequences [first, last), common tokens: whole pages
};
__device__ __forceinline__ Group group_at(const AttnSharedArgs& a, int g) {
    Group x;
    x.first = min(max(a.group_first[g], 0), a.B);
    x.last = min(max(a.group_first[g + 1], x.first), a.B);
    x.prefix = min(max(a.prefix_len[g], 0), a.max_pages * a.page) & -a.page;
    return x;
}

__device__ __forceinline__ Group from_lane(const Group& x, int i) {
    return Group{__builtin_amdgcn_readlane(x.first, i), __builtin_amdgcn_readlane(x.last, i), __builtin_amdgcn_readlane(x.prefix, i)};
}

// The group of sequence b (one of no tokens where there is none): the last that begins at or
// before it.  A wave looks at 64 groups at a time, evenly apart until they are next to
// each other.
__device__ __forceinline__ bool group_of(const AttnSharedArgs& a, int b, int lane, Group& found) {
    found = Group{0, 0, 0};
    int lo = 0, hi = a.n_groups;        // groups before lo begin at or before b, those from hi on behind it
    while (lo < hi) {
        const int apart = (hi - lo + 63) / 64, g = lo + lane * apart;
        Group x{0, 0, 0};
        if (g < hi) x = group_at(a, g);
        const int before = __popcll(__ballot(g < hi && x.first <= b));
        if (before == 0) break;
        found = from_lane(x, before - 1);
        const int last = lo + (before - 1) * apart;
        hi = min(hi, last + apart);
        lo = last + 1;
    }
    if (b >= found.first && b < found.last) return true;
    found = Group{b, b + 1, 0};
    return false;
}

// The group whose rows are in tile number `tile` of all groups' tiles, and the tile's
// number within it.  Four times 64 groups are on their way together.
__device__ __forceinline__ bool group_of_tile(const AttnSharedArgs& a, int& tile, int rows_per_tile, int lane, Group& found) {
    for (int g0 = 0; g0 < a.n_groups; g0 += 256) {
        Group x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int g = g0 + 64 * i + lane;
            x[i] = Group{0, 0, 0};
            if (g < a.n_groups) x[i] = group_at(a, g);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (g0 + 64 * i >= a.n_groups) break;
            const int n = (int)(((long long)(x[i].last - x[i].first) * a.Tq * a.G + rows_per_tile - 1) / rows_per_tile);
            int y = n;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int z = __shfl_up(y, o, 64);
                if (lane >= o) y += z;
            }
            const uint64_t who = __ballot(tile < y);
            if (who) {
                const int j = __builtin_ctzll(who);
                tile -= __builtin_amdgcn_readlane(y, j) - __builtin_amdgcn_readlane(n, j);
                found = from_lane(x[i], j);
                return true;
            }
            tile -= __builtin_amdgcn_readlane(y, 63);
        }
    }
    return false;
}

// The number of a workgroup among those of the prefixes (common) or of own keys.  Half of the
// latter go first and half last: all at once they are bound by memory, which the products
// of prefixes leave idle for the most part.  With all of them behind the prefixes, 64 sequences
// of up to 512 own keys on 32768 common ones take 74 us instead of 71, eight groups of eight 30
// instead of 26.
__device__ __forceinline__ int block_of(const AttnSharedArgs& a, bool& common) {
    const int bid = blockIdx.x, early = ((int)gridDim.x - a.prefix_blocks) / 2;
    common = bid >= early && bid < early + a.prefix_blocks;
    return common ? bid - early : bid < early ? bid : bid - a.prefix_blocks;
}

// What a workgroup of BR rows computes.
struct Work {
    int first, rows, r0;        // first sequence, rows of the group or sequence, first row here
    int hk, prefix, part, parts;
    bool common;                // keys of the prefix, for a group's rows
    int len;                    // tokens before the new ones, of own keys' sequence
};
template <int BR_COMMON, int BR_OWN, int TEAMS = 1>
__device__ __forceinline__ bool work_of(const AttnSharedArgs& a, int lane, Work& w, int team = 0) {
    const int each = a.Tq * a.G;
    int bid = block_of(a, w.common);
    if (w.common) {
        w.hk = bid % a.HK;
        bid /= a.HK;
        // tiles go slowest: the ones past the last, of which there may be as many as groups, come behind all
        // others; half of the own keys' workgroups come behind them, and wait while they look for a group
        w.part = bid % a.nprefix;
        int tile = bid / a.nprefix;
        w.parts = a.nprefix;
        Group x;
        if (!group_of_tile(a, tile, BR_COMMON, lane, x)) return false;
        w.first = x.first;
        w.prefix = x.prefix;
        w.rows = (x.last - x.first) * each;
        w.r0 = tile * BR_COMMON;
        return true;
    }
    bid = bid * TEAMS + team;
    const int nbh = a.B * a.HK, bh = bid % nbh;
    bid /= nbh;
    w.hk = bh % a.HK;
    w.first = bh / a.HK;
    w.part = bid % a.nown;
    w.parts = a.nown;
    w.rows = each;
    w.r0 = bid / a.nown * BR_OWN;
    if (w.r0 >= w.rows) return false;                   // a team without work
    w.len = a.cache_len[w.first];                        // on its way while the group is looked for
    Group x;
    const bool member = group_of(a, w.first, lane, x);
    w.prefix = x.prefix;
    if (!member && w.part == 0)                          // no group's tile has its rows
        for (int i = threadIdx.x % (blockDim.x / TEAMS); i < a.nprefix * min(BR_OWN, w.rows - w.r0); i += blockDim.x / TEAMS) {
            const size_t at = ((size_t)(i % a.nprefix) * a.B * a.HK + bh) * each + w.r0 + i / a.nprefix;
            *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(kNegInf, 0.f);
        }
    return true;
}

// Row r of the work: its sequence, token, first query element, and the keys that it sees.
template <typename T> struct Row {
    int b, t, lo, hi;
    const T* q;
};
template <typename T>
__device__ __forceinline__ Row<T> row_of(const AttnSharedArgs& a, const Work& w, int r, int D) {
    Row<T> x;
    r = min(r, w.rows - 1);
    const int tau = (int)fdiv((uint32_t)r, a.divG), s = (int)fdiv((uint32_t)tau, a.divT), h = w.hk * a.G + (r - tau * a.G);
    x.t = tau - s * a.Tq;
    x.b = w.first + s;
    const int ql = seq_len(a.new_len, x.b, a.Tq), cap = a.max_pages * a.page;
    const long long before = max(w.common ? a.cache_len[x.b] : w.len, 0), at = before + x.t;
    const int kl = (int)min(before + ql, (long long)cap);
    const int from = a.window ? (int)min((long long)cap, max(at - a.window + 1, 0ll)) : 0, to = (int)min(at, (long long)kl - 1);
    x.lo = w.common ? from : max(from, w.prefix);
    x.hi = x.t < ql ? (w.common ? min(to, w.prefix - 1) : to) : -1;
    // rows past the newest token are computed on a valid row and dropped
    const int tr = max(min(x.t, ql - 1), 0);
    x.q = reinterpret_cast<const T*>(a.q) + ((size_t)x.b * a.Tq + tr) * a.ldq + (size_t)h * D;
    return x;
}

// Where row r of the work leaves its part.
__device__ __forceinline__ size_t part_at(const AttnSharedArgs& a, const Work& w, int r) {
    const int each = a.Tq * a.G, s = (int)fdiv(fdiv((uint32_t)r, a.divG), a.divT);
    return (((size_t)(w.common ? w.part : a.nprefix + w.part) * a.B + w.first + s) * a.HK + w.hk) * each + (r - s * each);
}
// Whether it belongs to a token that there is.
__device__ __forceinline__ bool row_lives(const AttnSharedArgs& a, const Work& w, int r) {
    const int tau = (int)fdiv((uint32_t)r, a.divG), s = (int)fdiv((uint32_t)tau, a.divT);
    return tau - s * a.Tq < seq_len(a.new_len, w.first + s, a.Tq);
}
__device__ __forceinline__ size_t place_of(const uint2& x) { return (size_t)(x.y & ~(1u << 31)) << 32 | x.x; }
__device__ __forceinline__ void leave_sum(const AttnSharedArgs& a, bool live, size_t at, float m, float total) {
    *reinterpret_cast<float2*>(a.part_ml + 2 * at) = live ? make_float2(m, total) : make_float2(kNegInf, 0.f);
}

__device__ __forceinline__ PagedKeys keys_of(const AttnSharedArgs& a, const Work& w, int end) {
    return PagedKeys{a.k_cache, a.v_cache, a.k_scale, a.v_scale, a.block_table + (size_t)w.first * a.max_pages,
                     a.n_pages, a.page, a.HK, w.hk, end, a.scale_log2};
}

// 16-row blocks of a team of NW waves, every wave on other keys (CacheRows), joined in the
// team's `so` and `sml`.  All teams of a workgroup come here, also one without work.
template <typename T, int D, int NR, int NW>
__device__ __forceinline__ void narrow_rows(const AttnSharedArgs& a, const Work& w, bool work, float (*so)[16][D + 4], float (*sml)[16][2]) {
    constexpr int ND = D / 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % NW), g = lane >> 4, lr = lane & 15;
    CacheRows<T, D, NR> x;
    int lo = INT_MAX, hi = 0;           // keys that some row sees: [lo, hi)
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        if (!work) break;
        const Row<T> r = row_of<T>(a, w, w.r0 + 16 * n + lr, D);
        x.lo[n] = r.lo;
        x.hi[n] = r.hi;
        if (r.hi >= r.lo) {
            lo = min(lo, r.lo);
            hi = max(hi, r.hi + 1);
        }
        x.load_query(n, r.q, g);
    }
    x.clear();
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor(lo, o, 64));
        hi = max(hi, __shfl_xor(hi, o, 64));
    }
    if (lo < hi) {
        int kb0 = lo / kStepKeys, kb1 = (hi + kStepKeys - 1) / kStepKeys;
        const int per = (kb1 - kb0 + w.parts - 1) / w.parts;
        kb0 = min(kb1, kb0 + w.part * per);
        kb1 = min(kb1, kb0 + per);
        const PagedKeys keys = keys_of(a, w, hi);
        x.attend(keys, kb0 + wave, kb1, NW, lane);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const float sum = group_add4(x.l[n]);
        const float top = sum != sum ? -kNegInf : x.m[n];  // a NaN sum takes part whatever the other maxima are
        lds_barrier();
        if (g == 0) {
            sml[wave][lr][0] = top;
            sml[wave][lr][1] = sum;
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) *reinterpret_cast<floatx4*>(&so[wave][lr][16 * d + 4 * g]) = x.o[d][n];
        lds_barrier();
        for (int i = threadIdx.x % (64 * NW); i < 16 * D / 4; i += 64 * NW) {
            const int row = i / (D / 4), d = (i % (D / 4)) * 4, r = w.r0 + 16 * n + row;
            if (!work || r >= w.rows) continue;
            float mm = kNegInf;
#pragma unroll
            for (int v = 0; v < NW; ++v) mm = fmaxf(mm, sml[v][row][0]);
            const float mu = mm == kNegInf ? 0.f : mm;
            float total = 0.f;
            floatx4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int v = 0; v < NW; ++v) {
                const float f = exp2_fast(sml[v][row][0] - mu);
                if (f != 0.f) {
                    total = fmaf(f, sml[v][row][1], total);
                    y += f * *reinterpret_cast<const floatx4*>(&so[v][row][d]);
                }
            }
            const size_t at = part_at(a, w, r);
            *reinterpret_cast<floatx4*>(a.part_o + at * D + d) = y;
            if (d == 0) leave_sum(a, row_lives(a, w, r), at, mm, total);
        }
    }
}

// A row's maximum is kept until a score exceeds it by a factor 2: with none a rescaling of all outputs follows in
// most steps (four groups of 256 rows on 16384 keys, D = 64: 94 us; 88 with 2, 87 with 2^3 or 2^8).  The row's largest
// probability is then not 1, which needs no rounding, but anything up to 2; so that its rounding cancels, the sum is
// that of the rounded probabilities.  Root mean square error against softmax in 64 bits, the output's rounding
// included, of the decode step and of 1, 2, 2^3 and 2^8 here, scores of spread 3 over 4096 keys (D = 64): 1.73e-3; 1.73,
// 1.78, 1.86 and 2.01e-3; with the sum of unrounded ones and 2^8 2.21e-3.
constexpr float kSlack = 1.f;

// 32 RB rows of a wave on 32x32x16 products (bf16, D >= 32), over steps of 128 keys whose
// codes the workgroup has copied into LDS: K as rows of D bytes; V, where pages have at
// least 64 keys, as rows of 64 keys for each channel, two sets of them (whole rows are
// copied: single pieces of 16 keys cost four times as many addresses), else as rows of 16,
// eight sets.  The 16-byte granules of a row are exchanged so that reads of a column of
// them fill all banks.  The step is four blocks of 32 keys; in each, row r of the score product
// is key
//   16 ((r >> 2) & 1) + 8 (r >> 4) + 4 ((r >> 3) & 1) + (r & 3),
// so that a lane's 16 scores are 16 consecutive keys of one page, and its rounded
// probabilities are the operand of the product with V for the 16 bytes of channel l % 32
// that it reads.  Lane half h holds channels D/2 h .. of a key.  RB blocks of 32 rows use
// each converted code, because conversions are a third of what the vector unit does.
// Powers of two are what cache_append leaves as scales; they are applied by the
// conversions of the codes, exactly.  The rest of another scale multiplies scores and
// probabilities.
template <int D> struct StepCodes {
    static constexpr int kPiece = 16 * D;                   // bytes of 16 keys of K, or of V
    static constexpr int kBytes = 16 * kPiece;              // a step
    static constexpr int GR = D / 16;                       // granules of a K row
    static constexpr int kCopies = D >= 64 ? D / 64 : 1;    // wave instructions of a piece (D = 32: half a wave)
    static __device__ __forceinline__ int swizzle(int row) { return D == 128 ? row >> 1 : D == 64 ? row >> 2 : row >> 3; }
};
constexpr int kStepPieces = 8, kChunkPieces = 512;         // of a step; of page numbers in LDS together
struct Piece {
    uint32_t row;           // page * HK + head; kNoPage: none, or past the end; kPlain: see WideRows::soften
    float k_power, v_power, k_rest, v_rest;     // scales, as a power of two and what is left
    __device__ __forceinline__ bool there() const { return (row & kNoPage) == 0; }
    static constexpr uint32_t kNoPage = 1u << 31, kPlain = 1u << 30;    // n_pages * HK is at most 2^30
};

// The power of two in a scale (1 for what is none: zero, NaN of an unread page).
__device__ __forceinline__ float power(float x) {
    const uint32_t e = __float_as_uint(x) & 0x7f800000u;
    return e == 0u || e == 0x7f800000u ? 1.f : __uint_as_float(e);
}
// Eight codes (two words) times a power of two as a matrix operand.
__device__ __forceinline__ Frag<bf16_t> scaled_frag(uint32_t a, uint32_t b, float s) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false), x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true);
    const bf16x2 y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false), z = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true);
    Frag<bf16_t> f;
    f.v = bf16x8{w[0], w[1], x[0], x[1], y[0], y[1], z[0], z[1]};
    return f;
}

// Sum of eight bf16 values, and x.
__device__ __forceinline__ float sum_of(const Frag<bf16_t>& f, float x) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 one = {(__bf16)1.f, (__bf16)1.f};
#pragma unroll
    for (int i = 0; i < 8; i += 2) x = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{f.v[i], f.v[i + 1]}, one, x, false);
    return x;
}

// Queries of a workgroup's rows in LDS, granules of 16 bytes exchanged within a row so
// that 32 rows' reads of one column of them fill all banks.
template <int D> __device__ __forceinline__ uint32_t query_place(int row, int granule) {
    constexpr int GR = D / 8, RPL = 16 / GR;
    return row * (D * 2) + ((granule ^ (row / RPL & (GR - 1))) * 16);
}

template <int D, int RB> struct WideRows {
    static constexpr int ND = D / 32, kPiece = StepCodes<D>::kPiece;
    float m[RB], l[RB];
    floatx16 o[RB][ND];
    floatx16 st[RB];
    Frag<bf16_t> p[RB][2];

    // Products of a turn: VALUES, of the block whose probabilities are there (its step's V at
    // v_codes, this lane's 16 keys of channel l % 32 at v_place, 32 channels v_step bytes),
    // and SCORES, of the next step's block (K at k_codes), in turns of a quarter each.
    // Nobody else covers the latency of a wave's LDS reads in its matrix turn: the operands
    // of a quarter's scores are read before its values, those of the next values before
    // its scores, and reads are spread evenly (all of them take three quarters of the
    // turn).  between(k) runs in quarter k.
    template <bool VALUES, bool SCORES, typename Between>
    __device__ __forceinline__ void products(const unsigned char* v_codes, uint32_t v_place, uint32_t v_step, const Piece* v_pieces,
                                             int v_plain, int v_first, int end, const unsigned char* k_codes, const Piece* k_pieces,
                                             const unsigned char* queries, int b, const int2* bounds, uint32_t* nans, int lane, Between between) {
        const int h = lane >> 5, r = lane & 31, krow = 8 * (r >> 4) + 4 * ((r >> 3) & 1) + (r & 3), kp = 2 * b + ((r >> 2) & 1), vp = 2 * b + h;
        float v_scale = 1.f, k_scale = 1.f;
        // a granule's place is an exclusive or away from the first one's: two values are kept,
        // the others cost one instruction at their use
        uint32_t row = kp * kPiece + krow * D + (((ND * h) ^ StepCodes<D>::swizzle(krow)) * 16), query = query_place<D>(r, D / 16 * h);
        asm volatile("" : "+v"(row), "+v"(query));
        const unsigned char* col = v_codes + v_place;
        uint4 v[2];
        if constexpr (VALUES) {
            v[0] = *reinterpret_cast<const uint4*>(col);
            v_scale = v_pieces[vp].v_power;
        }
        if constexpr (SCORES) k_scale = k_pieces[kp].k_power;
        int valid = 16;
        int hidden = 0;         // some row that is there sees none of these keys
        if (VALUES && !v_plain) {
            valid = v_pieces[vp].there() ? end - v_first - 16 * h : 0;
            bool none = false;
#pragma unroll
            for (int n = 0; n < RB; ++n) {
                const int2 row = bounds[32 * n + r];
                none = none || (row.y >= 0 && (row.x >= v_first + 32 || row.y < v_first));
            }
            hidden = __any(none) ? 1 : 0;
        }
#pragma unroll
        for (int k = 0; k < ND; ++k) {
            uint4 kw;
            Frag<bf16_t> q[RB][2];
            if constexpr (SCORES) {
                kw = *reinterpret_cast<const uint4*>(k_codes + (row ^ (k * 16)));
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int n = 0; n < RB; ++n)
                        q[n][e].v = *reinterpret_cast<const bf16x8*>(queries + (query ^ ((2 * k + e) * 16)) + 32 * n * (D * 2));
            }
            if (VALUES && k + 1 < ND) v[(k + 1) & 1] = *reinterpret_cast<const uint4*>(col + v_step * (k + 1));
            between(k);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (VALUES) {
                uint4 x = v[k & 1];
                if (!v_plain) {     // bytes past the end may be anything, NaN codes among them
                    asm volatile("" : "+v"(valid));
                    x = keep_bytes(x, valid);
                    // Zero times a NaN code is NaN too: left out for rows that see none of these keys, and noted for those
                    // that see some.
                    if (hidden) {
                        const uint64_t who = __ballot(drop_nan_codes(x));
                        if (who != 0 && lane < 32) {
#pragma unroll
                            for (int n = 0; n < RB; ++n) {
                                const int2 row = bounds[32 * n + lane];
                                if (row.x < v_first + 32 && row.y >= v_first) atomicOr(nans + (32 * n + lane) * ND + k, (uint32_t)(who | who >> 32));
                            }
                        }
                    }
                }
                const Frag<bf16_t> v0 = scaled_frag(x.x, x.y, v_scale), v1 = scaled_frag(x.z, x.w, v_scale);
#pragma unroll
                for (int n = 0; n < RB; ++n) o[n][k] = mma32(v0, p[n][0], o[n][k]);
#pragma unroll
                for (int n = 0; n < RB; ++n) o[n][k] = mma32(v1, p[n][1], o[n][k]);
            }
            if constexpr (SCORES) {
                const Frag<bf16_t> k0 = scaled_frag(kw.x, kw.y, k_scale), k1 = scaled_frag(kw.z, kw.w, k_scale);
#pragma unroll
                for (int n = 0; n < RB; ++n) st[n] = mma32(k0, q[n][0], k == 0 ? splat16(0.f) : st[n]);
#pragma unroll
                for (int n = 0; n < RB; ++n) st[n] = mma32(k1, q[n][1], st[n]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Scores to probabilities: keys from `first` on, below `end`.  plain: every row sees
    // all of them, no page is missing and the scales are powers of two.
    __device__ __forceinline__ void soften(int plain, const Piece* pieces, int b, int first, int end, const int2* bounds, float scale_log2,
                                           int lane) {
        const Piece* mine = pieces + 2 * b + (lane >> 5);
        int key = first + 16 * (lane >> 5);
        if (!plain) {
            asm volatile("" : "+v"(key));   // a branch that stays one: computed for every step it would cost as much as the rest
            const bool there = mine->there();
            const float rest = mine->k_rest;
#pragma unroll
            for (int n = 0; n < RB; ++n) {
                const int2 row = bounds[32 * n + (lane & 31)];     // first and last key that it sees
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    st[n][i] = there && key + i < end && key + i >= row.x && key + i <= row.y ? st[n][i] * rest : kNegInf;
            }
        }
        float x[RB];
        bool grows = false;
#pragma unroll
        for (int n = 0; n < RB; ++n) {
            float y = kNegInf, z = kNegInf;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y = fmaxf(y, st[n][i]);
                z = fmaxf(z, st[n][8 + i]);
            }
            x[n] = pair_max(fmaxf(y, z)) * scale_log2;
            grows |= x[n] > m[n] + kSlack;
        }
        if (__any(grows)) {
#pragma unroll
            for (int n = 0; n < RB; ++n) {
                const float now = x[n] > m[n] + kSlack ? x[n] : m[n], alpha = exp2_fast(m[n] - (now == kNegInf ? 0.f : now));
                m[n] = now;
                l[n] *= alpha;
#pragma unroll
                for (int d = 0; d < ND; ++d) o[n][d] *= splat16(alpha);
            }
        }
#pragma unroll
        for (int n = 0; n < RB; ++n) {
            const float mu = m[n] == kNegInf ? 0.f : m[n];
#pragma unroll
            for (int i = 0; i < 16; ++i) st[n][i] = exp2_fast(fmaf(st[n][i], scale_log2, -mu));
        }
        if (!plain) {
            asm volatile("" : "+v"(key));
            const float rest = mine->there() ? mine->v_rest : 1.f;
#pragma unroll
            for (int n = 0; n < RB; ++n) {
                float y = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    y += st[n][i];
                    st[n][i] = st[n][i] == 0.f ? 0.f : st[n][i] * rest;  // an unread page's scale may be anything
                }
                // not what is rounded: the sum without rounding, as in the other tiles
                if (rest != 1.f) l[n] += y - (sum_of(frag_of(st[n], 0), 0.f) + sum_of(frag_of(st[n], 1), 0.f));
            }
        }
#pragma unroll
        for (int n = 0; n < RB; ++n) {
            p[n][0] = frag_of(st[n], 0);
            p[n][1] = frag_of(st[n], 1);
            l[n] += sum_of(p[n][0], 0.f) + sum_of(p[n][1], 0.f);
            settle(p[n]);
        }
    }
};

}  // namespace

// fp32, D = 16, and groups of few rows: bound by memory and, in few parts, by the latency of
// what four waves have in flight.  Eight groups of 8 sequences of 4 heads on 4001 common keys
// (8 key/value heads, 200 own keys each; 83 MB): 26 us with the join, 2 more with eight waves
// a workgroup.
template <typename T, int D, int NR>
__global__ __launch_bounds__(64 * kSharedWaves) void kda_attn_shared_kernel(const AttnSharedArgs a) {
    constexpr int NW = kSharedWaves;
    __shared__ __attribute__((aligned(16))) float so[NW][16][D + 4];
    __shared__ float sml[NW][16][2];
    Work w;
    if (!work_of<16 * NR, 16 * NR>(a, threadIdx.x & 63, w)) return;
    narrow_rows<T, D, NR, NW>(a, w, true, so, sml);
}

// Eight waves: two groups of 32 RB rows, four waves each, a block of 32 keys of a step for
// every wave.  A step's codes are copied straight into LDS, each piece of 16 keys by one
// wave, two steps ahead of their products; page numbers and scales of up to 8192 keys are
// there before, so that the loop has no load to wait for but those copies.  The waves of
// a SIMD, w and w + 4, take turns: between two barriers one forms products (values of the
// last step, scores of the next) while the other turns scores into probabilities.
// Own keys: two teams of four waves as above, each with a sequence of its own.
// Bound by issue: a step of 128 keys for 128 rows of D = 128 is 64 products (2048 cycles of a
// SIMD) beside as many cycles of conversions, exponentials and sums that the products of
// the other wave hide in part only; it takes about 5000.  64 sequences of 4 heads on 32768
// common keys (8 key/value heads, up to 512 own keys each): 68 us and 7 of the join (70 a call among
// others), of which the steps are 34 (the products alone would be 25 at the rate of a large product)
// and own keys 11.  On 32-row tiles 96 us.
// Two workgroups a compute unit where the LDS holds them (tiles of 64 rows, D = 32, and D = 64 with few own rows, which
// have 128 registers a lane then): 8 groups of 64 rows on 16384 keys, D = 64, 52 us instead of 60.
template <int D, int RB, int NR>
__global__ __launch_bounds__(512, RB == 1 && D * NR <= 64 ? 4 : 2) void kda_attn_shared_wide_kernel(const AttnSharedArgs a) {
    typedef bf16_t T;
    typedef StepCodes<D> S;
    constexpr int NW = 8, RW = 2, ND = D / 32, KW = NW / RW, NC = 2 * S::kCopies, BR = 32 * RB * RW, kChunk = kChunkPieces / kStepPieces;
    constexpr int kSide = S::kBytes / 2;            // K of a step, or V
    // bytes: codes of three steps, queries, page numbers; then what is joined, of two teams or of eight waves
    constexpr int kQueries = 3 * S::kBytes, kPieces = kQueries + BR * D * 2, kLoop = kPieces + kChunkPieces * (int)sizeof(Piece);
    constexpr int kTeam = 4 * 16 * (D + 4) * 4, kJoin = NW * 32 * (D + 4) * 4;
    constexpr int kBytes = kLoop > kJoin ? (kLoop > 2 * kTeam ? kLoop : 2 * kTeam) : (kJoin > 2 * kTeam ? kJoin : 2 * kTeam);
    __shared__ __attribute__((aligned(256))) unsigned char sm[kBytes];
    unsigned char* const queries = sm + kQueries;
    Piece* const pieces = reinterpret_cast<Piece*>(sm + kPieces);
    __shared__ float sml[NW][32][2];
    __shared__ int range[NW][2];
    __shared__ int2 bounds[BR];
    __shared__ uint32_t nans[BR][ND];               // channels of a row that met a NaN code of v
    __shared__ uint2 place[BR];                     // of a row's part, and whether the row is there
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
    Work w;
    bool common;
    block_of(a, common);
    if (!common) {
        const int team = wave / 4;
        const bool work = work_of<BR, 16 * NR, 2>(a, lane, w, team);
        narrow_rows<T, D, NR, 4>(a, w, work, reinterpret_cast<float(*)[16][D + 4]>(sm + team * kTeam),
                                 reinterpret_cast<float(*)[16][2]>(&sml[4 * team][0][0]));
        return;
    }
    if (!work_of<BR, 16 * NR, 2>(a, lane, w)) return;
    const int rg = wave % RW, kg = wave / RW, wr0 = 32 * RB * rg;
    const int shift = 31 - __clz(a.page);
    const int* table = a.block_table + (size_t)w.first * a.max_pages;
    // steps of this part: of the prefix, or of what a window leaves of it
    int s0 = 0, s1 = (w.prefix + 127) / 128, from, to;
    auto share = [&]() {
        s0 = __builtin_amdgcn_readfirstlane(s0);
        s1 = __builtin_amdgcn_readfirstlane(s1);
        const int per = s1 > s0 ? (s1 - s0 + w.parts - 1) / w.parts : 0;
        from = min(s1, s0 + w.part * per);
        to = min(s1, from + per);
    };
    share();
    auto page_of = [&](int c0, int i) {
        const int key = (c0 * kStepPieces + i) * 16;
        return key < w.prefix && i < (min(to, c0 + kChunk) - c0) * kStepPieces ? table[key >> shift] : -1;
    };
    auto piece_of = [&](int pg, float k, float v) {
        return pg >= 0 && pg < a.n_pages ? Piece{(uint32_t)pg * a.HK + w.hk, power(k), power(v), k / power(k), v / power(v)}
                                         : Piece{Piece::kNoPage, 1.f, 1.f, 1.f, 1.f};
    };
    auto scale_of = [&](const float* scale, int pg) { return pg >= 0 && pg < a.n_pages ? scale[(uint32_t)pg * a.HK + w.hk] : 1.f; };
    // Page numbers, queries, scales and lengths are each other's next loads or independent: they
    // are on their way together before anything waits.  With a window the steps are not known yet.
    int first_page = -1;
    if (!a.window) first_page = page_of(from, threadIdx.x);
    constexpr int NQ = (BR * D / 8 + 511) / 512;
    u32x4 first_q[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int at = i * 512 + threadIdx.x;
        first_q[i] = u32x4{0u, 0u, 0u, 0u};
        if (at < BR * D / 8) first_q[i] = *reinterpret_cast<const u32x4*>(row_of<T>(a, w, w.r0 + at / (D / 8), D).q + 8 * (at % (D / 8)));
    }
    const float first_k = scale_of(a.k_scale, first_page), first_v = scale_of(a.v_scale, first_page);
    WideRows<D, RB> x;
    // keys that some row sees, and that all of this wave's do
    int lo = INT_MAX, hi = 0, all_lo = 0, all_hi = INT_MAX;
#pragma unroll
    for (int n = 0; n < RB; ++n) {
        const Row<T> row = row_of<T>(a, w, w.r0 + wr0 + 32 * n + (lane & 31), D);
        if (kg == 0 && h == 0) {
            bounds[wr0 + 32 * n + lane] = make_int2(row.lo, row.hi);
#pragma unroll
            for (int d = 0; d < ND; ++d) nans[wr0 + 32 * n + lane][d] = 0u;
        }
        if (kg == 1 && h == 0) {
            const int r = min(w.r0 + wr0 + 32 * n + lane, w.rows - 1);
            const size_t at = part_at(a, w, r);
            place[wr0 + 32 * n + lane] = make_uint2((uint32_t)at, (uint32_t)(at >> 32) | (row_lives(a, w, r) ? 1u << 31 : 0u));
        }
        x.m[n] = kNegInf;
        x.l[n] = 0.f;
#pragma unroll
        for (int d = 0; d < ND; ++d) x.o[n][d] = splat16(0.f);
        if (row.hi >= row.lo) {
            lo = min(lo, row.lo);
            hi = max(hi, row.hi + 1);
        }
        all_lo = max(all_lo, row.lo);
        all_hi = min(all_hi, row.hi + 1);
    }
    const bool active = w.r0 + wr0 < w.rows;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor(lo, o, 64));
        hi = max(hi, __shfl_xor(hi, o, 64));
        all_lo = max(all_lo, __shfl_xor(all_lo, o, 64));
        all_hi = min(all_hi, __shfl_xor(all_hi, o, 64));
    }
    if (lane == 0) {
        range[wave][0] = lo;
        range[wave][1] = hi;
    }
    all_lo = __builtin_amdgcn_readfirstlane(all_lo);
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int at = i * 512 + threadIdx.x;
        if (at < BR * D / 8) *reinterpret_cast<u32x4*>(queries + query_place<D>(at / (D / 8), at % (D / 8))) = first_q[i];
    }
    if (a.window) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < NW; ++v) {
            lo = min(lo, range[v][0]);
            hi = max(hi, range[v][1]);
        }
        s0 = min(lo, w.prefix) / 128;
        s1 = (hi + 127) / 128;
        share();
    }
    // what this wave copies of a step: 16 keys of K; of V as much, as rows of 64 keys (a
    // quarter of the channels) or of 16
    const bool rows64 = a.page >= 64;
    const int vfirst = rows64 ? wave / 4 * 4 : wave, vchannel = rows64 ? wave % 4 * (D / 4) : 0;
    uint32_t koff[S::kCopies], voff[S::kCopies];
#pragma unroll
    for (int c = 0; c < S::kCopies; ++c) {
        const int n = c * 64 + lane, krow = n / S::GR, vrow = vchannel + (rows64 ? n / 4 : n);
        koff[c] = krow * D + ((n % S::GR) ^ S::swizzle(krow)) * 16;
        voff[c] = ((uint32_t)vrow << shift) + (rows64 ? ((n ^ (vrow >> 2)) & 3) * 16 : 0);
    }
    const uint32_t lds0 = lds_address(&sm[0]) + wave * S::kPiece;
    // this lane's first granule of V in a step: its keys 32 kg + 16 h .., channel l % 32
    const int vkey = 2 * kg + h, r32 = lane & 31;
    const uint32_t v_place = rows64 ? (vkey >> 2) * 4 * S::kPiece + r32 * 64 + ((vkey ^ (r32 >> 2)) & 3) * 16 : vkey * S::kPiece + r32 * 16;
    const uint32_t v_step = rows64 ? 32 * 64 : 32 * 16;
    const int page_log2 = shift + (D == 128 ? 7 : D == 64 ? 6 : 5);      // bytes of a page and head
    for (int c0 = from; c0 < to; c0 += kChunk) {
        const int c1 = min(to, c0 + kChunk);
        __syncthreads();
        {
            const int i = threadIdx.x;
            Piece p;
            if (c0 == from && !a.window) {
                p = piece_of(first_page, first_k, first_v);
            } else {
                const int pg = page_of(c0, i);
                p = piece_of(pg, scale_of(a.k_scale, pg), scale_of(a.v_scale, pg));
            }
            // plain steps: all pages there, scales powers of two
            const uint64_t fine = __ballot(p.there() && p.k_rest == 1.f && p.v_rest == 1.f);
            if ((fine >> (lane & 56) & 0xff) == 0xff) p.row |= Piece::kPlain;
            pieces[i] = p;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < NW; ++v) hi = max(hi, range[v][1]);
        hi = __builtin_amdgcn_readfirstlane(hi);        // no row sees a key from here on
        // where this wave's piece of a step's K or V is; one that is none reads page 0 and is masked
        auto source = [&](int s, uint32_t id, bool values) {
            const int within = (s * kStepPieces + (values ? vfirst : wave)) * 16 & (a.page - 1);
            const size_t base = id & Piece::kNoPage ? 0 : (size_t)(id & ~Piece::kPlain) << page_log2;
            return values ? tile_window(a.v_cache + base + within, D, a.page, rows64 ? 64 : 16)
                          : tile_window(a.k_cache + base + (size_t)within * D, 16, D, D);
        };
        auto copy = [&](const u32x4& window, int c, int place, bool values) {
            if (D >= 64 || lane < 32) copy_to_lds(window, values ? voff[c] : koff[c], lds0 + ((values ? 3 : 0) + place) * kSide + c * 1024);
        };
        auto stage = [&](int s, uint32_t id, int place, bool values) {
            const u32x4 window = source(s, id, values);
#pragma unroll
            for (int c = 0; c < S::kCopies; ++c) copy(window, c, place, values);
        };
        auto id_of = [&](int s, int piece) { return pieces[min(s - c0, c1 - c0 - 1) * kStepPieces + piece].row; };
        // a step is fine for this wave if it is plain and every row sees its keys
        auto seen = [&](int s, uint32_t id) {
            const int first = s * 128 + 32 * kg;
            return id & Piece::kPlain && first >= all_lo && first + 32 <= all_hi ? 1 : 0;
        };
        // Turn 2 s (even) brings the first half's products of step s, those of the other half
        // come a turn later.  In its products a wave copies its pieces of K of step s + 2
        // and V of step s + 1, an instruction in each quarter: together they keep the unit that
        // takes addresses busy for a fifth of a step, and issued at once they make all waves
        // wait for it.  Page numbers are read a step ahead; whether a step is fine goes along.
        const uint32_t id0 = __builtin_amdgcn_readfirstlane(id_of(c0, wave)), id1 = __builtin_amdgcn_readfirstlane(id_of(c0 + 1, wave));
        uint32_t ahead_k = id_of(c0 + 2, wave), ahead_v = id_of(c0 + 1, vfirst);
        int fine0 = seen(c0, id0), fine1 = seen(c0 + 1, id1), fine2 = 0;
        int place_k = 2, place_v = 1, place = 0;    // of K of step s + 2, V of step s + 1, K of step s
        const unsigned char* mine = queries + wr0 * D * 2;
        auto products = [&](auto values, auto scores, int s) {
            const uint32_t id = __builtin_amdgcn_readfirstlane(ahead_k);
            const bool more_k = s + 2 < c1, more_v = s + 1 < c1;
            const u32x4 kwin = source(s + 2, id, false), vwin = source(s + 1, __builtin_amdgcn_readfirstlane(ahead_v), true);
            fine2 = seen(s + 2, id);
            ahead_k = id_of(s + 3, wave);
            ahead_v = id_of(s + 2, vfirst);
            auto between = [&](int k) {
#pragma unroll
                for (int c = 0; c < S::kCopies; ++c) {
                    if (more_k && k == c % ND) copy(kwin, c, place_k, false);
                    if (more_v && k == (S::kCopies + c) % ND) copy(vwin, c, place_v, true);
                }
            };
            if (active) {
                const Piece* now = pieces + (s - c0) * kStepPieces;
                __builtin_amdgcn_s_setprio(2);
                x.template products<decltype(values)::value, decltype(scores)::value>(
                    sm + (3 + (place == 0 ? 2 : place - 1)) * kSide, v_place, v_step, now - kStepPieces, fine0, (s - 1) * 128 + 32 * kg, hi,
                    sm + place * kSide, now, mine, kg, bounds + wr0, &nans[wr0][0], lane, between);
                __builtin_amdgcn_s_setprio(0);
            } else {
#pragma unroll
                for (int k = 0; k < ND; ++k) between(k);
            }
            place_k = place_k == 2 ? 0 : place_k + 1;
            place_v = place_v == 2 ? 0 : place_v + 1;
            place = place == 2 ? 0 : place + 1;
        };
        auto landed = [&](int s) {      // K of step s and V of the step before
            if (s + 1 < c1) wait_vmcnt<NC>(); else wait_vmcnt<0>();
        };
        auto soften = [&](int s) {      // its flag is then fine0, for its values
            if (active) x.soften(fine0, pieces + (s - c0) * kStepPieces, kg, s * 128 + 32 * kg, hi, bounds + wr0, a.scale_log2, lane);
        };
        const std::integral_constant<bool, true> yes;
        const std::integral_constant<bool, false> no;
        const bool late = wave >= 4;
        stage(c0, id0, 0, false);
        stage(c0, __builtin_amdgcn_readfirstlane(id_of(c0, vfirst)), 0, true);
        if (c0 + 1 < c1) stage(c0 + 1, id1, 1, false);
        wait_vmcnt<0>();
        lds_barrier();
        if (late) lds_barrier();
        products(no, yes, c0);
        if (late) landed(c0 + 1);
        lds_barrier();
        for (int s = c0 + 1; s < c1; ++s) {
            const int after = fine1;    // of step s
            fine1 = fine2;
            soften(s - 1);
            if (!late) landed(s);
            lds_barrier();
            products(yes, yes, s);
            fine0 = after;
            if (late) landed(s + 1);
            lds_barrier();
        }
        soften(c1 - 1);
        if (!late) landed(c1);
        lds_barrier();
        products(yes, no, c1);
        lds_barrier();
        if (!late) lds_barrier();
    }
    // join the waves of each row group, 32 rows at a time: each wave's sums weighted, then added;
    // barriers that do not wait for the parts' way to memory
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));   // nothing of it is kept through the loop, where it would be spilled
    const int er = tid & 31, eh = tid >> 5 & 1;
    float(*buf)[32][D + 4] = reinterpret_cast<float(*)[32][D + 4]>(sm);
#pragma unroll
    for (int n = 0; n < RB; ++n) {
        const float sum = pair_add(x.l[n]);
        lds_barrier();
        if (eh == 0) {
            sml[wave][er][0] = sum != sum ? -kNegInf : x.m[n];  // a NaN sum takes part whatever the other maxima are
            sml[wave][er][1] = sum;
        }
        lds_barrier();
        float top[KW], total[KW], mm = kNegInf;
#pragma unroll
        for (int v = 0; v < KW; ++v) {
            top[v] = sml[v * RW + rg][er][0];
            total[v] = sml[v * RW + rg][er][1];
            mm = fmaxf(mm, top[v]);
        }
        const float mu = mm == kNegInf ? 0.f : mm, f = exp2_fast(sml[wave][er][0] - mu);
        if (kg == 0 && eh == 0 && w.r0 + wr0 + 32 * n + er < w.rows) {
            float l = 0.f;
#pragma unroll
            for (int v = 0; v < KW; ++v) {
                const float e = exp2_fast(top[v] - mu);
                if (e != 0.f) l = fmaf(e, total[v], l);
            }
            const uint2 there = place[wr0 + 32 * n + er];
            leave_sum(a, there.y >> 31, place_of(there), mm, l);
        }
        const bool all = __all(f != 0.f);           // a wave that saw nothing of a row takes no part in it
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                floatx4 y = {x.o[n][d][4 * e], x.o[n][d][4 * e + 1], x.o[n][d][4 * e + 2], x.o[n][d][4 * e + 3]};
                y *= f;
                if (!all) y = f == 0.f ? floatx4{0.f, 0.f, 0.f, 0.f} : y;
                *reinterpret_cast<floatx4*>(&buf[wave][er][32 * d + 8 * e + 4 * eh]) = y;
            }
        lds_barrier();
#pragma unroll
        for (int k = 0; k < RW * 32 * (D / 4) / (64 * NW); ++k) {
            const int i = k * (64 * NW) + tid;
            const int g = i / (8 * D), at32 = i / (D / 4) % 32, ch = i % (D / 4) * 4, local = 32 * (RB * g + n) + at32, row = w.r0 + local;
            if (row >= w.rows) continue;
            floatx4 y = *reinterpret_cast<const floatx4*>(&buf[g][at32][ch]);
#pragma unroll
            for (int v = 1; v < KW; ++v) y += *reinterpret_cast<const floatx4*>(&buf[v * RW + g][at32][ch]);
            const uint32_t bad = nans[local][ch / 32] >> (ch % 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = nan_if(y[e], bad, e);
            *reinterpret_cast<floatx4*>(a.part_o + place_of(place[local]) * D + ch) = y;
        }
    }
}

static unsigned shared_grid(const AttnSharedArgs& a, int br, int teams) {
    return (unsigned)(a.prefix_blocks + ((long long)a.B * a.HK * a.nown * (((long long)a.Tq * a.G + br - 1) / br) + teams - 1) / teams);
}
template <typename T, int D, int NR>
static hipError_t launch_shared_n(const AttnSharedArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((kda_attn_shared_kernel<T, D, NR>), dim3(shared_grid(a, 16 * NR, 1)), dim3(64 * kSharedWaves), 0, s, a);
    return hipGetLastError();
}
template <int D, int RB>
static hipError_t launch_shared_wide(const AttnSharedArgs& a, hipStream_t s) {
    if (a.own_blocks == 1) hipLaunchKernelGGL((kda_attn_shared_wide_kernel<D, RB, 1>), dim3(shared_grid(a, 16, 2)), dim3(512), 0, s, a);
    else hipLaunchKernelGGL((kda_attn_shared_wide_kernel<D, RB, 2>), dim3(shared_grid(a, 32, 2)), dim3(512), 0, s, a);
    return hipGetLastError();
}
template <typename T, int D>
static hipError_t launch_shared_t(const AttnSharedArgs& a, hipStream_t s) {
    hipError_t e = hipErrorInvalidValue;
    if constexpr (sizeof(T) == 2 && D >= 32) {
        if (a.wide == 2) e = launch_shared_wide<D, 1>(a, s);
        if (a.wide == 4) e = launch_shared_wide<D, 2>(a, s);
    }
    if (a.wide == 0) e = a.own_blocks == 1 ? launch_shared_n<T, D, 1>(a, s) : launch_shared_n<T, D, 2>(a, s);
    if (e != hipSuccess) return e;
    const JoinArgs j{a.part_o, a.part_ml, a.o, nullptr, a.nprefix + a.nown, a.B, a.Tq, a.H, a.HK, a.G, a.divG};
    return launch_attn_join(sizeof(T) == 2 ? 1 : 0, D, j, s);
}
template <typename T>
static hipError_t launch_shared_d(int D, const AttnSharedArgs& a, hipStream_t s) {
    switch (D) {
        case 16: return launch_shared_t<T, 16>(a, s);
        case 32: return launch_shared_t<T, 32>(a, s);
        case 64: return launch_shared_t<T, 64>(a, s);
        case 128: return launch_shared_t<T, 128>(a, s);
        default: return hipErrorInvalidValue;
    }
}
hipError_t launch_attn_shared(int dt, int D, const AttnSharedArgs& a, hipStream_t s) {
    return dt == 1 ? launch_shared_d<bf16_t>(D, a, s) : launch_shared_d<float>(D, a, s);
}

}  // namespace kda
