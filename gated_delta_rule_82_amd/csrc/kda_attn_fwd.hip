// kda_attn_fwd.hip - softmax attention forward on gfx950.
//
//   o_i = sum_j exp(c q_i.k_j - m_i) v_j / sum_j exp(c q_i.k_j - m_i)
//
// One pass over the keys with a running maximum and sum.  A wave owns 16 NQ
// packed rows (see kda_attn.h) as the COLUMNS of its products: S^T = K Q^T puts
// a row's scores into one lane column, so the maximum needs two lane swaps, the
// rescale is one factor per lane, and the exponentials are, as they stand, the
// right operand of O^T += V^T P^T.  Keys and values go through a two-deep LDS
// ring filled by direct loads while the previous tile is used.  Few query rows: the
// key axis is split over workgroups and joined.
//
// Long rows are bound by the matrix cores beside the vector unit (an exponential, a
// multiply-add, a maximum, a sum and half a rounding for every 4 D flops), few rows by
// the keys and values read.  bf16, D = 128: 4 x 16 heads (4 of keys) x 4096 causal 255 us,
// 1.08 PFLOP/s (a large matrix product reaches 1.14); 16 tokens of 32 heads behind
// 65 536 keys of 8 62 us with the join, 4.3 TB/s.  fp32, D = 64, 2 x 4 heads x 1023 with
// unequal lengths: 30 us, 42 TFLOP/s of 154 (workgroups that end early are not made up for).
#include "kda_attn_device.h"

namespace kda {

// The maximum that a row's exponentials are taken against is kept until a score
// exceeds it by a factor 2^8: sums and outputs stay far inside fp32 either way, and
// the rescaling of every accumulator becomes rare (with 32 rows to a wave some row's
// maximum grows in most tiles).
constexpr float kSlack = 8.f;

// Parts that one thread joins by itself.  8 184 rows of 3 parts (D = 64, fp32): 4 us,
// against 13 us with a workgroup per row; 512 rows of 64 parts the other way: 6 us
// against 46.
constexpr int kJoinFew = 8;

// T: element type; D: head dimension; NQ: 16-row column blocks of a wave; KB:
// keys per tile; NW: waves.
template <typename T, int D, int NQ, int KB, int NW>
__global__ __launch_bounds__(64 * NW, NW == 4 ? 2 : 1) void kda_attn_fwd_kernel(const AttnArgs a) {
    typedef TileGeom<T, D> G_;
    constexpr int NS = G_::NS, ND = G_::ND, NT = KB / 16, BQ = 16 * NQ * NW;
    constexpr int kTile = KB * D * (int)sizeof(T);
    __shared__ __attribute__((aligned(16))) unsigned char sm[4 * kTile];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
    // head fastest: the tiles of one key/value head run on one XCD when the
    // heads are a multiple of 8; late rows (the longest under a causal mask) first
    const int nbh = a.B * a.HK, rows = a.Tq * a.G;
    const int ntile = (rows + BQ - 1) / BQ;
    int bid = blockIdx.x;
    const int bh = head_of(a, bid, nbh);
    bid /= nbh;
    const int split = bid % a.nsplit;
    const int tile = ntile - 1 - bid / a.nsplit;
    const int b = bh / a.HK, hk = bh % a.HK;
    const int ql = seq_len(a.q_len, b, a.Tq), kl = seq_len(a.kv_len, b, a.Tk), off = kl - ql;
    const int r0 = tile * BQ, r1 = min(r0 + BQ, rows);
    const RowRange blk = row_range(a, r0, r1, ql, kl);
    int k_beg = blk.key_lo / KB, k_end = (blk.key_hi + KB - 1) / KB;  // tiles of KB keys
    if (blk.key_hi <= blk.key_lo) k_end = k_beg;
    if (a.nsplit > 1) {
        const int per = (k_end - k_beg + a.nsplit - 1) / a.nsplit;
        k_beg = min(k_end, k_beg + split * per);
        k_end = min(k_end, k_beg + per);
    }

    // this wave's rows
    const int w0 = r0 + wave * 16 * NQ;
    const RowRange mine = w0 < r1 ? row_range(a, w0, min(w0 + 16 * NQ, r1), ql, kl) : RowRange{0, -1, 0, 0};
    // every row of the wave sees the keys in [all_lo, all_hi)
    const int all_hi = a.causal ? min(kl, mine.t_first + off + 1) : kl;
    const int all_lo = a.window ? mine.t_last + off - a.window + 1 : 0;
    int t[NQ], lo[NQ], hi[NQ];   // token, first and last key of this lane's rows
    Frag<T> qf[NQ][NS];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int r = min(w0 + 16 * n + (lane & 15), rows - 1);
        t[n] = (int)fdiv((uint32_t)r, a.divG);
        const int h = hk * a.G + (r - t[n] * a.G), p = t[n] + off;
        hi[n] = a.causal ? min(kl - 1, p) : kl - 1;
        lo[n] = a.window ? p - a.window + 1 : 0;
        // rows past q_len are computed on the last valid token's values and dropped
        const int tr = max(min(t[n], ql - 1), 0);
        const T* qp = reinterpret_cast<const T*>(a.q) + ((size_t)b * a.Tq + tr) * a.ldq + (size_t)h * D;
#pragma unroll
        for (int s = 0; s < NS; ++s) qf[n][s] = row_frag_global<T, D>(qp, s, lane);
    }

    const T* kbase = reinterpret_cast<const T*>(a.k) + (size_t)b * a.Tk * a.ldk + (size_t)hk * D;
    const T* vbase = reinterpret_cast<const T*>(a.v) + (size_t)b * a.Tk * a.ldv + (size_t)hk * D;
    // keys past the length are past the windows and read as zeros
    Stage<T, D, KB, NW> kst, vst;
    kst.init(wave, lane, [&](int r) { return (uint32_t)(r * a.ldk * sizeof(T)); });
    vst.init(wave, lane, [&](int r) { return (uint32_t)(r * a.ldv * sizeof(T)); });
    const uint32_t lds0 = lds_address(&sm[0]);
    auto stage = [&](int kt, int buf) {
        const long long k0 = (long long)kt * KB, left = kl - 1 - k0;
        kst.issue(buffer_window(kbase + k0 * a.ldk, (left * (long long)a.ldk + D) * (long long)sizeof(T)), lds0 + buf * 2 * kTile, wave);
        vst.issue(buffer_window(vbase + k0 * a.ldv, (left * (long long)a.ldv + D) * (long long)sizeof(T)), lds0 + (buf * 2 + 1) * kTile, wave);
    };

    const TileLane<T, D> place(lane);
    const float c = a.scale_log2;
    float m[NQ], l[NQ];
    floatx4 o[ND][NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        m[n] = kNegInf;
        l[n] = 0.f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d][n] = floatx4{0.f, 0.f, 0.f, 0.f};
    }

    if (k_beg < k_end) stage(k_beg, 0);
    for (int kt = k_beg; kt < k_end; ++kt) {
        const int buf = (kt - k_beg) & 1, k0 = kt * KB;
        wait_vmcnt<0>();
        lds_barrier();  // tile kt has landed; every wave is done with the other buffer
        if (kt + 1 < k_end) stage(kt + 1, buf ^ 1);
        if (k0 >= mine.key_hi || k0 + KB <= mine.key_lo) continue;  // nothing for this wave's rows
        const uint32_t ks = buf * 2 * kTile, vs = ks + kTile;

        floatx4 st[NT][NQ];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int n = 0; n < NQ; ++n) st[i][n] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const Frag<T> kf = row_frag<D>(sm, ks, 16 * i, s, place, lane);
#pragma unroll
                for (int n = 0; n < NQ; ++n) st[i][n] = mma(kf, qf[n][s], st[i][n]);
            }
        if (k0 < all_lo || k0 + KB > all_hi) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const uint32_t span = max(hi[n] - lo[n] + 1, 0), first = k0 + 4 * g - lo[n];
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) st[i][n][e] = first + 16 * i + e < span ? st[i][n][e] : kNegInf;
            }
        }
        bool grew = false;
        float mu[NQ], top[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float x = kNegInf;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) x = fmaxf(x, st[i][n][e]);
            top[n] = group_max4(x) * c;
            grew |= top[n] > m[n] + kSlack;
        }
        if (__any(grew)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const float x = fmaxf(m[n], top[n]), alpha = exp2_fast(m[n] - (x == kNegInf ? 0.f : x));
                m[n] = x;
                l[n] *= alpha;
#pragma unroll
                for (int d = 0; d < ND; ++d) o[d][n] *= alpha;
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) mu[n] = m[n] == kNegInf ? 0.f : m[n];  // a row that has seen nothing yet
        // bf16 probabilities are rounded for the product (2^-8 relative each, as
        // the values beside them); the sum is over the unrounded ones
        Frag<T> pf[NT / 2][NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    st[i][n][e] = exp2_fast(fmaf(st[i][n][e], c, -mu[n]));
                    l[n] += st[i][n][e];
                }
#pragma unroll
            for (int i = 0; i < NT / 2; ++i) pf[i][n] = frag_from_c<T>(st[2 * i][n], st[2 * i + 1][n]);
        }
#pragma unroll
        for (int i = 0; i < NT / 2; ++i)
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const Frag<T> vf = col_frag<D>(sm, vs, 32 * i, d, place, lane);
#pragma unroll
                for (int n = 0; n < NQ; ++n) o[d][n] = mma(vf, pf[i][n], o[d][n]);
            }
    }

#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int r = w0 + 16 * n + (lane & 15);
        const float sum = group_add4(l[n]);
        if (r >= r1) continue;
        if (a.nsplit > 1) {
            const size_t row = ((size_t)split * nbh + bh) * rows + r;
#pragma unroll
            for (int d = 0; d < ND; ++d) store4(a.part_o + row * D + 16 * d + 4 * g, o[d][n]);
            // a NaN sum takes part whatever the other parts' maxima are
            const float top = sum != sum ? -kNegInf : m[n];
            if (g == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * row) = t[n] < ql ? make_float2(top, sum) : make_float2(kNegInf, 0.f);
        } else {
            const int h = hk * a.G + (r - t[n] * a.G);
            const float inv = 1.f / sum;
            const bool some = t[n] < ql && sum != 0.f;
            T* op = reinterpret_cast<T*>(a.o) + (((size_t)b * a.Tq + t[n]) * a.H + h) * D;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const floatx4 y = o[d][n] * inv;
                store4(op + 16 * d + 4 * g, some ? y : floatx4{0.f, 0.f, 0.f, 0.f});
            }
            if (a.lse && g == 0)
                a.lse[((size_t)b * a.H + h) * a.Tq + t[n]] =
                    some ? (m[n] + __builtin_amdgcn_logf(sum)) * kLn2 : kNegInf;
        }
    }
}

// The forward for grids that fill the card: eight waves share the tiles, two on each
// SIMD, and take turns.  Between two barriers one half forms products (O += V P of
// a tile and S = K Q of the next) while the other half, on the vector unit, turns its
// scores into probabilities; then they change over.  Left to themselves the two
// waves of a SIMD want the same unit at the same time.  Three tiles of keys and three
// of values: the copies for two tiles ahead are issued in the vector turn, so that the
// matrix turn holds nothing but fragment reads and products, and have a whole
// matrix turn to land.
template <int D>
__global__ __launch_bounds__(512, 2) void kda_attn_fwd_turns_kernel(const AttnArgs a) {
    typedef bf16_t T;
    constexpr int KB = 64, NW = 8, NS = D / 16, ND = D / 32, NT = KB / 32, BQ = 32 * NW;
    constexpr int kTile = KB * D * (int)sizeof(T);
    __shared__ __attribute__((aligned(16))) unsigned char sm[6 * kTile];   // three of K, three of V

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    const bool late = wave >= 4;   // the half that starts a turn later
    const int nbh = a.B * a.HK, rows = a.Tq * a.G;
    const int ntile = (rows + BQ - 1) / BQ;
    const int bh = head_of(a, blockIdx.x, nbh), tile = ntile - 1 - blockIdx.x / nbh;
    const int b = bh / a.HK, hk = bh % a.HK;
    const int ql = seq_len(a.q_len, b, a.Tq), kl = seq_len(a.kv_len, b, a.Tk), off = kl - ql;
    const int r0 = tile * BQ, r1 = min(r0 + BQ, rows);
    const RowRange blk = row_range(a, r0, r1, ql, kl);
    const int k_beg = blk.key_lo / KB, k_end = blk.key_hi > blk.key_lo ? (blk.key_hi + KB - 1) / KB : k_beg;

    const int w0 = r0 + wave * 32;
    const RowRange mine = w0 < r1 ? row_range(a, w0, min(w0 + 32, r1), ql, kl) : RowRange{0, -1, 0, 0};
    const int all_hi = a.causal ? min(kl, mine.t_first + off + 1) : kl;
    const int all_lo = a.window ? mine.t_last + off - a.window + 1 : 0;
    const int r = w0 + (lane & 31), t = (int)fdiv((uint32_t)min(r, rows - 1), a.divG);
    const int head = hk * a.G + (min(r, rows - 1) - t * a.G);
    Frag<T> qf[NS];
    {
        const int tr = max(min(t, ql - 1), 0);   // rows past q_len are dropped at the end
        const T* qp = reinterpret_cast<const T*>(a.q) + ((size_t)b * a.Tq + tr) * a.ldq + (size_t)head * D + 8 * half;
#pragma unroll
        for (int s = 0; s < NS; ++s) frag_load_row8(qf[s], qp + 16 * s);
    }

    const T* kbase = reinterpret_cast<const T*>(a.k) + (size_t)b * a.Tk * a.ldk + (size_t)hk * D;
    const T* vbase = reinterpret_cast<const T*>(a.v) + (size_t)b * a.Tk * a.ldv + (size_t)hk * D;
    Stage<T, D, KB, NW, true> kst, vst;
    kst.init(wave, lane, [&](int r) { return (uint32_t)(r * a.ldk * sizeof(T)); });
    vst.init(wave, lane, [&](int r) { return (uint32_t)(r * a.ldv * sizeof(T)); });
    const uint32_t lds0 = lds_address(&sm[0]);
    // the next tiles to copy, and the ring places they go to
    const uint32_t krow = (uint32_t)(a.ldk * sizeof(T)), vrow = (uint32_t)(a.ldv * sizeof(T));
    const T* knext = kbase + (size_t)k_beg * KB * a.ldk;
    const T* vnext = vbase + (size_t)k_beg * KB * a.ldv;
    int knum = k_beg, vnum = k_beg, kplace = 0, vplace = 0;
    auto load_k = [&]() {
        if (knum < k_end) kst.issue(tile_window(knext, min(kl - knum * KB, KB), krow, D * sizeof(T)), lds0 + kplace * kTile, wave);
        knext += KB * a.ldk;
        kplace = kplace == 2 ? 0 : kplace + 1;
        ++knum;
    };
    auto load_v = [&]() {
        if (vnum < k_end) vst.issue(tile_window(vnext, min(kl - vnum * KB, KB), vrow, D * sizeof(T)), lds0 + (3 + vplace) * kTile, wave);
        vnext += KB * a.ldv;
        vplace = vplace == 2 ? 0 : vplace + 1;
        ++vnum;
    };

    const WideLane<D> place(lane);
    const float c = a.scale_log2;
    float m = kNegInf, l = 0.f;
    floatx16 o[ND], st[NT];
    Frag<T> pf[NT][2];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = splat16(0.f);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        st[i] = splat16(0.f);
        pf[i][0].zero();
        pf[i][1].zero();
    }
    auto scores = [&](uint32_t ks) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < NT; ++i) st[i] = mma32(wide_row<D>(sm, ks, 32 * i, s, place), qf[s], s == 0 ? splat16(0.f) : st[i]);
    };
    auto values = [&](uint32_t vs) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int d = 0; d < ND; ++d) o[d] = mma32(wide_col<D>(sm, vs, 32 * i, u, d, place), pf[i][u], o[d]);
    };
    // both, in one stream of fragments read kAhead fragments before their products:
    // nobody else covers this wave's LDS latency in its matrix turn
    auto values_and_scores = [&](uint32_t vs, uint32_t ks) {
        constexpr int NV = NT * 2 * ND, NF = NV + NS * NT, kAhead = 6;
        Frag<T> ring[kAhead];
        auto fetch = [&](int f) {
            return f < NV ? wide_col<D>(sm, vs, 32 * (f / (2 * ND)), f / ND % 2, f % ND, place)
                          : wide_row<D>(sm, ks, 32 * ((f - NV) % NT), (f - NV) / NT, place);
        };
#pragma unroll
        for (int f = 0; f < kAhead; ++f) ring[f] = fetch(f);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const Frag<T> x = ring[f % kAhead];
            if (f + kAhead < NF) ring[f % kAhead] = fetch(f + kAhead);
            if (f < NV) {
                o[f % ND] = mma32(x, pf[f / (2 * ND)][f / ND % 2], o[f % ND]);
            } else {
                const int i = (f - NV) % NT, s = (f - NV) / NT;
                st[i] = mma32(x, qf[s], s == 0 ? splat16(0.f) : st[i]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto probabilities = [&](int kt) {
        const int k0 = kt * KB;
        if (k0 < all_lo || k0 + KB > all_hi) {
            const int p = t + off, hi = a.causal ? min(kl - 1, p) : kl - 1, lo = a.window ? p - a.window + 1 : 0;
            const uint32_t span = max(hi - lo + 1, 0), first = k0 + 4 * half - lo;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) st[i][e] = first + 32 * i + 8 * (e / 4) + e % 4 < span ? st[i][e] : kNegInf;
        }
        float x = kNegInf;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) x = fmaxf(x, st[i][e]);
        x = pair_max(x) * c;
        if (__any(x > m + kSlack)) {
            const float top = fmaxf(m, x), alpha = exp2_fast(m - (top == kNegInf ? 0.f : top));
            m = top;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] *= alpha;
        }
        const float mu = m == kNegInf ? 0.f : m;  // a row that has seen nothing yet
        // probabilities are rounded to bf16 for the product (2^-8 relative each, as the
        // values beside them); the sum is over the unrounded ones
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                st[i][e] = exp2_fast(fmaf(st[i][e], c, -mu));
                part[e % 4] += st[i][e];
            }
            pf[i][0] = frag_of(st[i], 0);
            pf[i][1] = frag_of(st[i], 1);
            settle(pf[i]);
        }
        l += (part[0] + part[1]) + (part[2] + part[3]);
    };

    if (k_beg < k_end) {
        load_k();
        load_k();
        load_v();
        load_k();
        load_v();
        wait_vmcnt<0>();
        lds_barrier();
        // the tiles [first, last) that this wave's rows see
        const bool any = mine.key_hi > mine.key_lo;
        const int first = any ? mine.key_lo / KB : k_end + 1, last = any ? (mine.key_hi + KB - 1) / KB : k_end + 1;
        if (first == k_beg) {
            scores(0);
            probabilities(k_beg);
        }
        // Before tile kt's products: keys up to kt + 2 and values up to kt + 1 are in LDS
        // or in flight.  Both halves wait for their copies at the end of a matrix turn;
        // the next ones go to the places of keys kt and values kt - 1, last read before it.
        uint32_t vs = 3 * kTile, ks = kTile;
        auto change_over = [&]() {
            __builtin_amdgcn_s_setprio(0);
            vs = vs == 5 * kTile ? 3 * kTile : vs + kTile;
            ks = ks == 2 * kTile ? 0 : ks + kTile;
            wait_vmcnt<0>();
            lds_barrier();
            load_k();
            load_v();
        };
        auto change_back = [&]() {
            lds_barrier();
            __builtin_amdgcn_s_setprio(1);
        };
        if (late) lds_barrier();
        int kt = k_beg;
        for (; kt + 1 < first && kt < k_end; ++kt) {
            change_over();
            change_back();
        }
        if (any && kt + 1 == first) {
            scores(ks);
            change_over();
            probabilities(first);
            change_back();
            ++kt;
        }
        for (; any && kt + 1 < last; ++kt) {
            values_and_scores(vs, ks);
            change_over();
            probabilities(kt + 1);
            change_back();
        }
        if (any && kt + 1 == last) {
            values(vs);
            change_over();
            change_back();
            ++kt;
        }
        for (; kt < k_end; ++kt) {
            change_over();
            change_back();
        }
        __builtin_amdgcn_s_setprio(0);
        if (!late) lds_barrier();
    }

    const float sum = pair_add(l);
    const bool some = t < ql && sum != 0.f;
    const float inv = some ? 1.f / sum : 0.f;
    if (a.lse && half == 0 && r < r1)
        a.lse[((size_t)b * a.H + head) * a.Tq + t] = some ? (m + __builtin_amdgcn_logf(sum)) * kLn2 : kNegInf;
    // rows without a sum get zeros; nobody reads tiles any more
    wide_rows_out<D>(o, inv, some, sm + wave * 64 * D, lane, [&](int row) -> T* {
        const int rr = w0 + row, tt = (int)fdiv((uint32_t)min(rr, rows - 1), a.divG), hh = hk * a.G + (rr - tt * a.G);
        return rr < r1 ? reinterpret_cast<T*>(a.o) + (((size_t)b * a.Tq + tt) * a.H + hh) * D : nullptr;
    });
}

// Few parts: a thread takes four channels of one packed row over all of them.
template <typename T, int D>
__global__ __launch_bounds__(256) void kda_attn_join_few_kernel(const JoinArgs a) {
    constexpr int L = D / 4;
    const int rows = a.Tq * a.G;
    const size_t n = (size_t)a.B * a.HK * rows, at = ((size_t)blockIdx.x * 256 + threadIdx.x) / L;
    const int d = (threadIdx.x % L) * 4;
    if (at >= n) return;
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
    float2 x[kJoinFew];
    floatx4 y[kJoinFew];
    float m = kNegInf;
#pragma unroll
    for (int s = 0; s < kJoinFew; ++s) {
        x[s] = make_float2(kNegInf, 0.f);
        y[s] = floatx4{0.f, 0.f, 0.f, 0.f};
        if (s < a.nsplit) {
            x[s] = ml[s * n + at];
            y[s] = *reinterpret_cast<const floatx4*>(a.part_o + (s * n + at) * D + d);
        }
        m = fmaxf(m, x[s].x);
    }
    const float mu = m == kNegInf ? 0.f : m;
    float sum = 0.f;
    floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kJoinFew; ++s) {
        const float w = exp2_fast(x[s].x - mu);
        if (w == 0.f) continue;  // a part that saw nothing takes no part
        sum = fmaf(w, x[s].y, sum);
        o += w * y[s];
    }
    const int r = (int)(at % rows), bh = (int)(at / rows), b = bh / a.HK, hk = bh % a.HK;
    const int t = (int)fdiv((uint32_t)r, a.divG), h = hk * a.G + (r - t * a.G);
    const float inv = 1.f / sum;
    store4(reinterpret_cast<T*>(a.o) + (((size_t)b * a.Tq + t) * a.H + h) * D + d, sum == 0.f ? floatx4{0.f, 0.f, 0.f, 0.f} : o * inv);
    if (a.lse && d == 0)
        a.lse[((size_t)b * a.H + h) * a.Tq + t] = sum == 0.f ? kNegInf : (m + __builtin_amdgcn_logf(sum)) * kLn2;
}

// Many parts: one workgroup per packed row.  The parts' maxima and sums are read one a
// thread, and at the same time their outputs: 256 / (D / 4) groups of threads take
// every so-manieth part, four channels a thread, all loads in flight before the weights
// are known, and are summed in LDS in a fixed order.  128 rows of 128 parts, D = 128
// (8 MB): 5.5 us, against 8.1 with the outputs read after the weights.
template <typename T, int D>
__global__ __launch_bounds__(256) void kda_attn_join_kernel(const JoinArgs a) {
    constexpr int L = D / 4, NG = 256 / L, P = kMaxSplits / NG;
    __shared__ float weight[kMaxSplits];
    __shared__ float red[2][4];
    __shared__ floatx4 part[NG][L];
    const int rows = a.Tq * a.G, tid = threadIdx.x;
    const size_t n = (size_t)a.B * a.HK * rows, at = blockIdx.x;
    const float2 x = tid < a.nsplit ? reinterpret_cast<const float2*>(a.part_ml)[tid * n + at] : make_float2(kNegInf, 0.f);
    const int grp = tid / L, d = (tid % L) * 4;
    floatx4 y[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int s = grp + i * NG;
        y[i] = s < a.nsplit ? *reinterpret_cast<const floatx4*>(a.part_o + (s * n + at) * D + d) : floatx4{0.f, 0.f, 0.f, 0.f};
    }
    float m = x.x;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    if ((tid & 63) == 0) red[0][tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float w = exp2_fast(x.x - (m == kNegInf ? 0.f : m));
    float sum = w == 0.f ? 0.f : w * x.y;  // a part that saw nothing takes no part
    if (tid < a.nsplit) weight[tid] = w;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if ((tid & 63) == 0) red[1][tid >> 6] = sum;
    __syncthreads();
    sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int s = grp + i * NG;
        if (s >= a.nsplit) break;
        const float f = weight[s];
        o += f == 0.f ? floatx4{0.f, 0.f, 0.f, 0.f} : f * y[i];
    }
    part[grp][tid % L] = o;
    __syncthreads();
    if (grp != 0) return;
    for (int i = 1; i < NG; ++i) o += part[i][tid];
    const int r = (int)(at % rows), bh = (int)(at / rows), b = bh / a.HK, hk = bh % a.HK;
    const int t = (int)fdiv((uint32_t)r, a.divG), h = hk * a.G + (r - t * a.G);
    const float inv = 1.f / sum;
    store4(reinterpret_cast<T*>(a.o) + (((size_t)b * a.Tq + t) * a.H + h) * D + d, sum == 0.f ? floatx4{0.f, 0.f, 0.f, 0.f} : o * inv);
    if (a.lse && tid == 0)
        a.lse[((size_t)b * a.H + h) * a.Tq + t] = sum == 0.f ? kNegInf : (m + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <typename T, int D>
static hipError_t launch_join_t(const JoinArgs& a, hipStream_t s) {
    const size_t rows = (size_t)a.B * a.HK * a.Tq * a.G;
    if (a.nsplit <= kJoinFew) {
        const size_t threads = rows * (D / 4);
        hipLaunchKernelGGL((kda_attn_join_few_kernel<T, D>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((kda_attn_join_kernel<T, D>), dim3((unsigned)rows), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <typename T>
static hipError_t launch_join_d(int D, const JoinArgs& a, hipStream_t s) {
    switch (D) {
        case 16: return launch_join_t<T, 16>(a, s);
        case 32: return launch_join_t<T, 32>(a, s);
        case 64: return launch_join_t<T, 64>(a, s);
        case 128: return launch_join_t<T, 128>(a, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_attn_join(int dt, int D, const JoinArgs& a, hipStream_t s) {
    return dt == 1 ? launch_join_d<bf16_t>(D, a, s) : launch_join_d<float>(D, a, s);
}

template <typename T, int D, int NQ, int KB, int NW>
static hipError_t launch_fwd_n(const AttnArgs& a, hipStream_t s) {
    constexpr int BQ = 16 * NQ * NW;
    const long long rows = (long long)a.Tq * a.G, tiles = (rows + BQ - 1) / BQ;
    hipLaunchKernelGGL((kda_attn_fwd_kernel<T, D, NQ, KB, NW>), dim3((unsigned)(tiles * a.B * a.HK * a.nsplit)), dim3(64 * NW), 0, s, a);
    return hipGetLastError();
}

template <typename T, int D>
static hipError_t launch_fwd_t(const AttnArgs& a, hipStream_t s) {
    constexpr int NQ = attn_rows_per_wave(sizeof(T)) / 16, KB = sizeof(T) == 2 ? 64 : 32;
    const long long rows = (long long)a.Tq * a.G;
    if constexpr (sizeof(T) == 2 && D == 128) {
        if (attn_fwd_turns(sizeof(T), D, a)) {
            hipLaunchKernelGGL((kda_attn_fwd_turns_kernel<D>), dim3((unsigned)turns_grid(a, rows, kTurnsRows)), dim3(512), 0, s, a);
            return hipGetLastError();
        }
    }
    const int nw = attn_waves(rows, 16 * NQ);
    hipError_t e = nw == 1 ? launch_fwd_n<T, D, NQ, KB, 1>(a, s)
                   : nw == 2 ? launch_fwd_n<T, D, NQ, KB, 2>(a, s)
                             : launch_fwd_n<T, D, NQ, KB, 4>(a, s);
    if (e != hipSuccess || a.nsplit == 1) return e;
    JoinArgs j{a.part_o, a.part_ml, a.o, a.lse, a.nsplit, a.B, a.Tq, a.H, a.HK, a.G, a.divG};
    return launch_attn_join(sizeof(T) == 2 ? 1 : 0, D, j, s);
}

template <typename T>
static hipError_t launch_fwd_d(int D, const AttnArgs& a, hipStream_t s) {
    switch (D) {
        case 16: return launch_fwd_t<T, 16>(a, s);
        case 32: return launch_fwd_t<T, 32>(a, s);
        case 64: return launch_fwd_t<T, 64>(a, s);
        case 128: return launch_fwd_t<T, 128>(a, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_attn_fwd(int dt, int D, const AttnArgs& a, hipStream_t s) {
    return dt == 1 ? launch_fwd_d<bf16_t>(D, a, s) : launch_fwd_d<float>(D, a, s);
}

}  // namespace kda
