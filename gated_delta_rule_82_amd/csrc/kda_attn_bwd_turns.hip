// kda_attn_bwd_turns.hip - the bf16 backward for grids that fill the card: dk with dv,
// and dq, on 32x32x16 products with the eight waves of a workgroup in two halves that
// take turns, as the forward's.
//
// Between two barriers one half forms products (the gradients of a tile and the scores
// of the next) while the other half, on the vector unit, turns its scores into P and
// dS; then they change over.  Copies are issued at the start of a vector turn and have
// until the end of the next matrix turn.  In dk and dv a turn takes 1470 cycles for 1024
// of products; fewer cycles have stopped paying, the clock falls as they do.
#include "kda_attn_device.h"

namespace kda {

namespace {

constexpr int kWaves = 8;
// Fragments are read this many ahead of their products: nobody else covers a wave's LDS
// latency in its matrix turn.  The first ones are read at the end of the vector turn,
// which has time to spare.
constexpr int kAhead = 6;

}  // namespace

// dk and dv of 128 keys, over the queries of all heads that share them.  Keys are the
// columns of S = Q K^T and dP = dO V^T.  Both halves hold the same keys, 32 a wave, and
// take every other tile of queries from rings of three tiles of their own; their sums
// are joined at the end.  (With 256 keys, 32 for each of the eight waves, causal masks
// left the card waiting for the workgroups with the earliest keys: 781 us for 16
// key/value heads of 4 query heads each, 4096 tokens, D = 128.)  A wave keeps both
// accumulators and its fragments of K in registers; those of V lie in LDS.
template <int D>
__global__ __launch_bounds__(512, 2) void kda_attn_dkv_turns_kernel(const AttnArgs a, int padded) {
    typedef bf16_t T;
    constexpr int RB = 32, NS = D / 16, ND = D / 32, NW = kWaves / 2, BK = 32 * NW, kRing = 3;
    constexpr int kTile = RB * D * (int)sizeof(T), kTiles = 2 * kRing * 2 * kTile;   // both halves' rings of Q and dO
    __shared__ __attribute__((aligned(16))) unsigned char sm[kTiles + NW * NS * 1024];   // and the fragments of V
    __shared__ __attribute__((aligned(16))) float srow[2 * kRing][256];  // RB pairs, and room for a whole wave's copy

    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % NW, late = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    const int nbh = a.B * a.HK;    // early keys are seen by most queries: they come first
    const int bh = head_of(a, blockIdx.x, nbh), tile = blockIdx.x / nbh;
    const int b = bh / a.HK, hk = bh % a.HK;
    const int ql = seq_len(a.q_len, b, a.Tq), kl = seq_len(a.kv_len, b, a.Tk), off = kl - ql;
    const int k0 = tile * BK, k1 = min(k0 + BK, kl);  // keys of the tile inside the length
    // queries that see some key of [k0, k1): t >= k0 - off if causal, t < k1 - 1 + window - off
    int t_lo = 0, t_hi = k0 < k1 ? ql : 0;
    if (a.causal) t_lo = max(0, k0 - off);
    if (a.window) t_hi = min(t_hi, max(0, k1 - 1 + a.window - off));
    const int beg = t_lo / RB, per = t_lo < t_hi ? (t_hi + RB - 1) / RB - beg : 0;  // tiles of a head
    const int steps = per * a.G, turns = (steps + 1) / 2, mine_n = late ? steps / 2 : turns;  // tiles of this half

    // the queries [seen_from(key), seen_to(key)) that see a key (lengths and the
    // window are below 2^29: no sum overflows)
    auto seen_from = [&](int key) { return a.causal ? min(max(key - off, 0), ql) : 0; };
    auto seen_to = [&](int key) { return key >= kl ? 0 : a.window ? min(max(key - off + a.window, 0), ql) : ql; };
    const int w0 = k0 + wave * 32, key = w0 + (lane & 31);
    const int lo = seen_from(key);
    const uint32_t span = max(seen_to(key) - lo, 0);
    // those that see all 32 keys of the wave
    const int all_lo = seen_from(w0 + 31), all_hi = w0 + 32 <= kl ? seen_to(w0) : 0;

    Frag<T> kf[NS];
    T* mine = reinterpret_cast<T*>(sm + kTiles) + wave * NS * 512;
    {
        const int kr = max(min(key, kl - 1), 0);
        const T* kp = reinterpret_cast<const T*>(a.k) + ((size_t)b * a.Tk + kr) * a.ldk + (size_t)hk * D + 8 * half;
        const T* vp = reinterpret_cast<const T*>(a.v) + ((size_t)b * a.Tk + kr) * a.ldv + (size_t)hk * D + 8 * half;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            frag_load_row8(kf[s], kp + 16 * s);
            if (!late) {
                Frag<T> x;
                frag_load_row8(x, vp + 16 * s);
                frag_store(x, mine + s * 512, lane);
            }
        }
    }

    const T* qbase = reinterpret_cast<const T*>(a.q) + (size_t)b * a.Tq * a.ldq + (size_t)hk * a.G * D;
    const size_t ldo = (size_t)a.H * D;
    const T* dobase = reinterpret_cast<const T*>(a.dout) + (size_t)b * a.Tq * ldo + (size_t)hk * a.G * D;
    const float* rbase = a.rows + ((size_t)b * a.H + (size_t)hk * a.G) * padded * 2;
    Stage<T, D, RB, NW, true> qst, dst;
    const int ring0 = late * kRing;   // this half's first place
    const uint32_t lds0 = lds_address(&sm[0]), lds_rows = lds_address(&srow[0][0]);
    qst.init(wave, lane, [&](int x) { return (uint32_t)(x * a.ldq * sizeof(T)); });
    dst.init(wave, lane, [&](int x) { return (uint32_t)(x * ldo * sizeof(T)); });
    auto advance = [&](int& h, int& t, int by) {
        for (t += by; t >= beg + per && h < a.G; ++h) t -= per;
    };
    // the next tile to copy
    const uint32_t qrow = (uint32_t)(a.ldq * sizeof(T)), drow = (uint32_t)(ldo * sizeof(T));
    const size_t qstep = 2 * RB * a.ldq, dstep = 2 * RB * ldo;
    const T *qnext, *dnext;
    const float* rnext;
    int next_h = 0, next_t = beg, next_place = ring0;
    auto seek = [&]() {
        qnext = qbase + (size_t)next_t * RB * a.ldq + (size_t)next_h * D;
        dnext = dobase + (size_t)next_t * RB * ldo + (size_t)next_h * D;
        rnext = rbase + 2 * ((size_t)next_h * padded + next_t * RB);
    };
    advance(next_h, next_t, late);
    seek();
    auto load = [&]() {
        if (next_h < a.G) {
            const int n = min(ql - next_t * RB, RB);  // queries past the last one are past the windows and read as zeros
            qst.issue(tile_window(qnext, n, qrow, D * sizeof(T)), lds0 + next_place * 2 * kTile, wave);
            dst.issue(tile_window(dnext, n, drow, D * sizeof(T)), lds0 + (next_place * 2 + 1) * kTile, wave);
            // the row array is padded to whole tiles; lanes past a tile's rows read zeros past the window, into the spare room
            if (wave == 0) copy_to_lds(tile_window(rnext, RB, 8, 8), lane * 16, lds_rows + next_place * 1024);
        }
        next_place = next_place == ring0 + kRing - 1 ? ring0 : next_place + 1;
        if (next_t + 2 < beg + per) {
            next_t += 2;
            qnext += qstep;
            dnext += dstep;
            rnext += 4 * RB;
        } else {
            advance(next_h, next_t, 2);
            seek();
        }
    };

    const WideLane<D> place(lane);
    const float c = a.scale_log2;
    floatx16 dk[ND], dv[ND], st, dp;
    Frag<T> pf[2], sf[2];
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        dk[d] = splat16(0.f);
        dv[d] = splat16(0.f);
    }
    // the initial accumulators of S - lse / c and dP - delta
    auto init_scores = [&](int at) {
        const float* rows = &srow[at][0];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const floatx4* rp = reinterpret_cast<const floatx4*>(rows + 8 * (2 * e + half));
            const floatx4 x = rp[0], y = rp[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                st[4 * e + j] = x[j];
                dp[4 * e + j] = y[j];
            }
        }
    };
    // One stream of fragments: with `grads` the columns of dO and Q at place p (products
    // with P and dS; the first kAhead are there), with `scores` the rows of Q and dO at
    // place p1, beside V's own.
    Frag<T> ring[kAhead];
    auto column = [&](int p, int f) { return wide_col<D>(sm, p * 2 * kTile + (f % 2 ? 0 : kTile), 0, f / (2 * ND), f / 2 % ND, place); };
    auto read_ahead = [&](int p) {
#pragma unroll
        for (int f = 0; f < kAhead; ++f) ring[f] = column(p, f);
    };
    auto products = [&](auto grads, auto scores, int p, int p1) {
        constexpr int NG = decltype(grads)::value ? 4 * ND : 0, NF = NG + (decltype(scores)::value ? 3 * NS : 0);
        const uint32_t qs1 = p1 * 2 * kTile, ds1 = qs1 + kTile;
        Frag<T> v;
        auto fetch = [&](int f) {
            if (f < NG) return column(p, f);
            const int s = (f - NG) / 3, kind = (f - NG) % 3;
            if (kind == 0) return wide_row<D>(sm, qs1, 0, s, place);
            if (kind == 2) return wide_row<D>(sm, ds1, 0, s, place);
            Frag<T> x;
            frag_load(x, mine + s * 512, lane);
            return x;
        };
        if (NG == 0) {
#pragma unroll
            for (int f = 0; f < kAhead; ++f) ring[f] = fetch(f);
            init_scores(p1);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const Frag<T> x = ring[f % kAhead];
            if (f + kAhead < NF) ring[f % kAhead] = fetch(f + kAhead);
            if (NG > 0 && NF > NG && f == NG - kAhead / 2) init_scores(p1);
            if (f < NG) {
                const int u = f / (2 * ND), d = f / 2 % ND;
                if (f % 2 == 0) dv[d] = mma32(x, pf[u], dv[d]);
                else dk[d] = mma32(x, sf[u], dk[d]);
            } else {
                const int s = (f - NG) / 3, kind = (f - NG) % 3;
                if (kind == 0) st = mma32(x, kf[s], st);
                else if (kind == 1) v = x;
                else dp = mma32(x, v, dp);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto probabilities = [&](int t0) {
        if (t0 < all_lo || t0 + RB > all_hi) {
            const uint32_t first = t0 + 4 * half - lo;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const bool seen = first + 8 * (e / 4) + e % 4 < span;
                st[e] = seen ? st[e] : kNegInf;
                dp[e] = seen ? dp[e] : 0.f;
            }
        }
        // P and dS are rounded for their products, 2^-8 relative each
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            st[e] = exp2_fast(st[e] * c);
            dp[e] *= st[e];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            pf[u] = frag_of(st, u);
            sf[u] = frag_of(dp, u);
        }
        settle(pf);
        settle(sf);
    };

    constexpr std::integral_constant<bool, true> yes{};
    constexpr std::integral_constant<bool, false> no{};
    if (steps > 0) {
        load();
        load();
        load();
        wait_vmcnt<0>();
        lds_barrier();
        int hh = 0, tt = beg, p = ring0;
        advance(hh, tt, late);
        auto after = [&](int at) { return at == ring0 + kRing - 1 ? ring0 : at + 1; };
        if (mine_n > 0) {
            products(no, yes, p, p);
            probabilities(tt * RB);
            read_ahead(p);
        }
        if (late) lds_barrier();
        for (int it = 1; it < mine_n; ++it) {
            products(yes, yes, p, after(p));
            __builtin_amdgcn_s_setprio(0);
            wait_vmcnt<0>();
            lds_barrier();
            load();   // to the place of the tile whose columns were just read
            p = after(p);
            advance(hh, tt, 2);
            probabilities(tt * RB);
            read_ahead(p);
            lds_barrier();
            __builtin_amdgcn_s_setprio(1);
        }
        if (mine_n > 0) products(yes, no, p, p);
        __builtin_amdgcn_s_setprio(0);
        lds_barrier();
        if (!late) lds_barrier();
        // the late half may have a tile less, but not a barrier
        if (mine_n < turns && mine_n > 0) {
            lds_barrier();
            lds_barrier();
        }
    } else {
        lds_barrier();   // the fragments of V are written
    }

    // The early half is left with the sum of dk, the late half with that of dv.
    unsigned char* other = sm + wave * (128 * D);
    floatx4* to = reinterpret_cast<floatx4*>(other + (late ? 0 : NW * 128 * D)) + lane;
    const floatx4* from = reinterpret_cast<const floatx4*>(other + (late ? NW * 128 * D : 0)) + lane;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const floatx16& x = late ? dk[d] : dv[d];
            to[(d * 4 + e) * 64] = floatx4{x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]};
        }
    lds_barrier();
    floatx16 sum[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        sum[d] = late ? dv[d] : dk[d];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const floatx4 y = from[(d * 4 + e) * 64];
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[d][4 * e + j] += y[j];
        }
    }
    T* grad = reinterpret_cast<T*>(late ? a.dv : a.dk);
    wide_rows_out<D>(sum, late ? 1.f : a.scale, true, other + (late ? NW * 128 * D : 0), lane, [&](int row) -> T* {
        const int at = w0 + row;
        return at < a.Tk ? grad + (((size_t)b * a.Tk + at) * a.HK + hk) * D : nullptr;
    });
}

// dq of 256 packed rows, 32 a wave: S^T = K Q^T and dP^T = V dO^T of 64 keys, then
// dQ^T += K^T dS^T.  A wave keeps its fragments of Q and dO and its accumulators.
template <int D>
__global__ __launch_bounds__(512, 2) void kda_attn_dq_turns_kernel(const AttnArgs a, int padded) {
    typedef bf16_t T;
    constexpr int KB = 64, NS = D / 16, ND = D / 32, NT = KB / 32, BQ = 32 * kWaves, kRing = 4;
    constexpr int kTile = KB * D * (int)sizeof(T);
    __shared__ __attribute__((aligned(16))) unsigned char sm[2 * kRing * kTile];   // K and V of every place

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    const bool late = wave >= 4;
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
    const int r = min(w0 + (lane & 31), rows - 1), t = (int)fdiv((uint32_t)r, a.divG), h = hk * a.G + (r - t * a.G);
    const int key_hi = a.causal ? min(kl - 1, t + off) : kl - 1, key_lo = a.window ? t + off - a.window + 1 : 0;
    const uint32_t span = max(key_hi - key_lo + 1, 0);
    Frag<T> qf[NS], df[NS];
    {
        const int tr = max(min(t, ql - 1), 0);   // rows past q_len are dropped at the end
        const T* qp = reinterpret_cast<const T*>(a.q) + ((size_t)b * a.Tq + tr) * a.ldq + (size_t)h * D + 8 * half;
        const T* dp = reinterpret_cast<const T*>(a.dout) + (((size_t)b * a.Tq + tr) * a.H + h) * D + 8 * half;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            frag_load_row8(qf[s], qp + 16 * s);
            frag_load_row8(df[s], dp + 16 * s);
        }
    }
    const float* row_values = a.rows + ((size_t)b * a.H + h) * padded * 2 + (t >> 2) * 8 + (t & 3);
    const float ls = row_values[0] * a.scale_log2, de = row_values[4];

    const T* kbase = reinterpret_cast<const T*>(a.k) + (size_t)b * a.Tk * a.ldk + (size_t)hk * D;
    const T* vbase = reinterpret_cast<const T*>(a.v) + (size_t)b * a.Tk * a.ldv + (size_t)hk * D;
    Stage<T, D, KB, kWaves, true> kst, vst;
    kst.init(wave, lane, [&](int x) { return (uint32_t)(x * a.ldk * sizeof(T)); });
    vst.init(wave, lane, [&](int x) { return (uint32_t)(x * a.ldv * sizeof(T)); });
    const uint32_t lds0 = lds_address(&sm[0]);
    // the next tile to copy
    const uint32_t krow = (uint32_t)(a.ldk * sizeof(T)), vrow = (uint32_t)(a.ldv * sizeof(T));
    const T* knext = kbase + (size_t)k_beg * KB * a.ldk;
    const T* vnext = vbase + (size_t)k_beg * KB * a.ldv;
    int next = k_beg, next_place = 0;
    auto load = [&]() {
        if (next < k_end) {
            const int n = min(kl - next * KB, KB);
            kst.issue(tile_window(knext, n, krow, D * sizeof(T)), lds0 + next_place * 2 * kTile, wave);
            vst.issue(tile_window(vnext, n, vrow, D * sizeof(T)), lds0 + (next_place * 2 + 1) * kTile, wave);
        }
        knext += KB * a.ldk;
        vnext += KB * a.ldv;
        next_place = (next_place + 1) % kRing;
        ++next;
    };

    const WideLane<D> place(lane);
    const float c = a.scale_log2;
    floatx16 dq[ND], st[NT], dp[NT];
    Frag<T> sf[NT][2];
#pragma unroll
    for (int d = 0; d < ND; ++d) dq[d] = splat16(0.f);
    // One stream of fragments: with `grads` the columns of K at place p (the first kAhead are
    // there), with `scores` the rows of K and V at place p1.
    Frag<T> ring[kAhead];
    auto column = [&](int p, int f) { return wide_col<D>(sm, p * 2 * kTile, 32 * (f / (2 * ND)), f / ND % 2, f % ND, place); };
    auto read_ahead = [&](int p) {
#pragma unroll
        for (int f = 0; f < kAhead; ++f) ring[f] = column(p, f);
    };
    auto products = [&](auto grads, auto scores, int p, int p1) {
        constexpr int NG = decltype(grads)::value ? 2 * NT * ND : 0, NF = NG + (decltype(scores)::value ? 2 * NT * NS : 0);
        const uint32_t ks1 = p1 * 2 * kTile, vs1 = ks1 + kTile;
        auto fetch = [&](int f) {
            if (f < NG) return column(p, f);
            const int s = (f - NG) / (2 * NT), i = (f - NG) / 2 % NT;
            return wide_row<D>(sm, (f - NG) % 2 ? vs1 : ks1, 32 * i, s, place);
        };
        if (NG == 0) {
#pragma unroll
            for (int f = 0; f < kAhead; ++f) ring[f] = fetch(f);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const Frag<T> x = ring[f % kAhead];
            if (f + kAhead < NF) ring[f % kAhead] = fetch(f + kAhead);
            if (f < NG) {
                dq[f % ND] = mma32(x, sf[f / (2 * ND)][f / ND % 2], dq[f % ND]);
            } else {
                const int s = (f - NG) / (2 * NT), i = (f - NG) / 2 % NT;
                if ((f - NG) % 2 == 0) st[i] = mma32(x, qf[s], s == 0 ? splat16(0.f) : st[i]);
                else dp[i] = mma32(x, df[s], s == 0 ? splat16(0.f) : dp[i]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto probabilities = [&](int kt) {
        const int k0 = kt * KB;
        if (k0 < all_lo || k0 + KB > all_hi) {
            const uint32_t first = k0 + 4 * half - key_lo;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const bool seen = first + 32 * i + 8 * (e / 4) + e % 4 < span;
                    st[i][e] = seen ? st[i][e] : kNegInf;
                    dp[i][e] = seen ? dp[i][e] : 0.f;
                }
        }
        // dS is rounded for its product, 2^-8 relative
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int e = 0; e < 16; ++e) dp[i][e] = exp2_fast(fmaf(st[i][e], c, ls)) * (dp[i][e] + de);
            sf[i][0] = frag_of(dp[i], 0);
            sf[i][1] = frag_of(dp[i], 1);
            settle(sf[i]);
        }
    };

    constexpr std::integral_constant<bool, true> yes{};
    constexpr std::integral_constant<bool, false> no{};
    if (k_beg < k_end) {
        load();
        load();
        load();
        wait_vmcnt<0>();
        lds_barrier();
        int p = 0;
        products(no, yes, 0, 0);
        probabilities(k_beg);
        read_ahead(0);
        if (late) lds_barrier();
        for (int kt = k_beg + 1; kt < k_end; ++kt) {
            products(yes, yes, p, (p + 1) % kRing);
            __builtin_amdgcn_s_setprio(0);
            wait_vmcnt<0>();
            lds_barrier();
            load();
            p = (p + 1) % kRing;
            probabilities(kt);
            read_ahead(p);
            lds_barrier();
            __builtin_amdgcn_s_setprio(1);
        }
        products(yes, no, p, p);
        __builtin_amdgcn_s_setprio(0);
        lds_barrier();
        if (!late) lds_barrier();
    }
    wide_rows_out<D>(dq, a.scale, t < ql, sm + wave * 64 * D, lane, [&](int row) -> T* {
        const int rr = w0 + row, tt = (int)fdiv((uint32_t)min(rr, rows - 1), a.divG), hh = hk * a.G + (rr - tt * a.G);
        return rr < r1 ? reinterpret_cast<T*>(a.dq) + (((size_t)b * a.Tq + tt) * a.H + hh) * D : nullptr;
    });
}

hipError_t launch_dkv_turns(const AttnArgs& a, int padded, hipStream_t s) {
    const dim3 grid((unsigned)turns_grid(a, a.Tk, kTurnsKeys));
    hipLaunchKernelGGL((kda_attn_dkv_turns_kernel<128>), grid, dim3(64 * kWaves), 0, s, a, padded);
    return hipGetLastError();
}

hipError_t launch_dq_turns(int D, const AttnArgs& a, int padded, hipStream_t s) {
    const dim3 grid((unsigned)turns_grid(a, (long long)a.Tq * a.G, kTurnsRows));
    if (D == 128) hipLaunchKernelGGL((kda_attn_dq_turns_kernel<128>), grid, dim3(64 * kWaves), 0, s, a, padded);
    else hipLaunchKernelGGL((kda_attn_dq_turns_kernel<64>), grid, dim3(64 * kWaves), 0, s, a, padded);
    return hipGetLastError();
}

}  // namespace kda
