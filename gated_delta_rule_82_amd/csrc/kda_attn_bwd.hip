// kda_attn_bwd.hip - softmax attention backward on gfx950.
//
//   P_ij = exp(c q_i.k_j - lse_i),  delta_i = dout_i.o_i
//   dv_j = sum_i P_ij dout_i,  dS_ij = P_ij (dout_i.v_j - delta_i)
//   dq_i = c sum_j dS_ij k_j,  dk_j = c sum_i dS_ij q_i
//
// Three kernels: the row values (lse, delta; formed in the dq kernel instead they cost
// it as much as this launch takes, 395 us against 362 for the first size below, o and dout
// arriving there with nothing else in flight); dk and dv, one workgroup per tile
// of keys, over the packed rows that see it (all query heads of the key/value
// head, so shared heads are summed in registers); dq, one workgroup per tile of
// packed rows.  Scores and dout.v are formed twice (7 products instead of 5):
// in exchange every sum stays in one workgroup's registers, in a fixed order,
// with no atomics and no partial results in memory (dS in bf16, written once and read
// once, would take 2.1 GB and 415 us for the first size below; the two products it
// saves take 240).
//
// Bound by the matrix cores: bf16, D = 128, 4 x 16 heads (4 of keys) x 4096 causal 846 us,
// what the 7 products alone would take at the rate of a large matrix product: row values
// 30 us (134 MB, 4.5 TB/s), dk and dv 500, dq 350 (kda_attn_bwd_turns.hip).
// fp32, D = 64, 2 x 4 heads (2) x 1024, window 256: 45 us for the three launches, one or two
// waves to a SIMD with little beside them while they wait.
#include "kda_attn_device.h"

namespace kda {

// P of a score q.k: in fp32 from -lse, in bf16 from -lse log2 e (see the row values).
template <typename T> __device__ __forceinline__ float row_lse(float lse) { return sizeof(T) == 4 ? -lse : -lse * kLog2e; }
template <typename T> __device__ __forceinline__ float probability(const AttnArgs& a, float score, float ls) {
    return sizeof(T) == 4 ? exp_carried(fmaf(score, a.scale, ls)) : exp2_fast(fmaf(score, a.scale_log2, ls));
}

// Row values where rows see few keys: delta = sum_j P_ij dP_ij / sum_j P_ij, from
// the very dP that the gradients are formed with (same products in the same order) and
// weights that add up to one.  dS is a difference that nearly vanishes there, and o's
// rounding (in fp32 that of the other order) shows in it: gradients of bf16 rows of two to
// five keys came out 1.3 to 2 times less precise, of fp32 ones up to eight times; in fp32
// lse is corrected by the sum's logarithm for the same reason.  For calls whose keys are
// whole (attn_few_keys, causal ones): the sum of a row does not tell, as a part with all
// but 10^-4 of the mass would lose just the 10^-4 that its dS is made of.  There the sum is
// one up to the rounding of scores about as large as lse (2^-24 of it, and as much for each
// of a few steps; eight times that is allowed); where it is not, delta is dout.o.  Packed
// rows r0 .. r0 + 15 by a wave, fragments straight from memory; wanted(t) says which are
// stored.
template <typename T, int D, typename Wanted>
__device__ __forceinline__ void rows_of_few_keys(const AttnArgs& a, int padded, int b, int hk, int r0, int lane, Wanted wanted) {
    constexpr int NS = TileGeom<T, D>::NS;
    const int g = lane >> 4, r = r0 + (lane & 15), t = (int)fdiv((uint32_t)r, a.divG), h = hk * a.G + (r - t * a.G);
    const int ql = seq_len(a.q_len, b, a.Tq), kl = seq_len(a.kv_len, b, a.Tk), off = kl - ql;
    const RowRange mine = row_range(a, r0, r0 + 16, ql, kl);
    const int hi = a.causal ? min(kl - 1, t + off) : kl - 1, lo = a.window ? t + off - a.window + 1 : 0;
    const int tr = max(min(t, ql - 1), 0);
    const T* qp = reinterpret_cast<const T*>(a.q) + ((size_t)b * a.Tq + tr) * a.ldq + (size_t)h * D;
    const size_t row = (((size_t)b * a.Tq + tr) * a.H + h) * D;
    Frag<T> qf[NS], df[NS];
    float delta_o = 0.f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        qf[s] = row_frag_global<T, D>(qp, s, lane);
        df[s] = row_frag_global<T, D>(reinterpret_cast<const T*>(a.dout) + row, s, lane);
        const Frag<T> of = row_frag_global<T, D>(reinterpret_cast<const T*>(a.o) + row, s, lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) delta_o = fmaf((float)df[s].v[j], (float)of.v[j], delta_o);
    }
    const float lse = t < ql ? a.lse[((size_t)b * a.H + h) * a.Tq + t] : kNegInf, ls = row_lse<T>(lse);
    float sum = 0.f, delta = 0.f;
    for (int k0 = mine.key_lo & ~15; k0 < mine.key_hi; k0 += 16) {
        const int kr = min(k0 + (lane & 15), kl - 1);
        const T* kp = reinterpret_cast<const T*>(a.k) + ((size_t)b * a.Tk + kr) * a.ldk + (size_t)hk * D;
        const T* vp = reinterpret_cast<const T*>(a.v) + ((size_t)b * a.Tk + kr) * a.ldv + (size_t)hk * D;
        floatx4 st = {0.f, 0.f, 0.f, 0.f}, dp = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            st = mma(row_frag_global<T, D>(kp, s, lane), qf[s], st);
            dp = mma(row_frag_global<T, D>(vp, s, lane), df[s], dp);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int key = k0 + 4 * g + e;
            if (key < lo || key > hi) continue;
            const float p = probability<T>(a, st[e], ls);
            sum += p;
            delta = fmaf(p, dp[e], delta);
        }
    }
    sum = group_add4(sum);
    delta = group_add4(delta);
    delta_o = group_add4(delta_o);
    if (g == 0 && wanted(t)) {
        const bool none = lse == kNegInf;
        const float d = sum - 1.f;
        const bool own = fabsf(d) < (8.f + fabsf(lse)) * 0x1p-20f;
        float* to = a.rows + ((size_t)b * a.H + h) * padded * 2 + (t >> 2) * 8 + (t & 3);
        to[0] = none ? kNegInf : sizeof(T) == 2 ? -lse / a.scale : own ? -(lse + (d - 0.5f * d * d)) : -lse;
        to[4] = none ? 0.f : own ? -delta / sum : -delta_o;
    }
}

// All rows, where none sees more.
template <typename T, int D>
__global__ __launch_bounds__(256) void kda_attn_rows_few_kernel(const AttnArgs a, int padded) {
    const size_t at = (size_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nbh = a.B * a.HK, bh = (int)(at % nbh);
    if (at / nbh >= (size_t)padded * a.G / 16) return;
    rows_of_few_keys<T, D>(a, padded, bh / a.HK, bh % a.HK, (int)(at / nbh) * 16, threadIdx.x & 63, [](int) { return true; });
}

// Row values of every query, padded per head to whole tiles with rows that
// contribute nothing (-inf makes P zero): -lse / c in bf16, the initial accumulators of
// the product that gives S - lse / c; in fp32 -lse, added after the product, where
// S c - lse is rounded once and small (as initial accumulators they doubled the gradients'
// error); and -delta.  Four queries' values of each kind lie together:
// rows[b][h][t / 4][kind][t % 4].
//
// Under a causal mask the first rows of a sequence see few keys, and their gradients are
// the largest: in bf16 the first `few` workgroups take the kFew tokens from the first that
// sees a key on as above (without it dq of 90 to 900 tokens was 1.6 times as far off as
// its rounding alone, with it 1.43, the square root of two: dS is rounded once more).
// fp32 gains nothing and would pay 3 us of 45 (2 x 4 heads x 1024, window 256).
constexpr int kFew = 32;
template <typename T, int D>
__global__ __launch_bounds__(256) void kda_attn_rows_kernel(const AttnArgs a, int padded, int few) {
    auto sees_few = [&](int t, int off) { return sizeof(T) == 2 && a.causal && t + off >= 0 && t + off < kFew && t - max(-off, 0) < kFew; };
    if (sizeof(T) == 2 && (int)blockIdx.x < few) {
        const size_t at = (size_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int nbh = a.B * a.HK, bh = (int)(at % nbh), b = bh / a.HK, i = (int)(at / nbh);
        const int ql = seq_len(a.q_len, b, a.Tq), off = seq_len(a.kv_len, b, a.Tk) - ql;
        if (i >= kFew / 16 * a.G || off >= kFew) return;
        rows_of_few_keys<T, D>(a, padded, b, bh % a.HK, max(-off, 0) * a.G + 16 * i, threadIdx.x & 63,
                               [&](int t) { return t < padded && sees_few(t, off); });
        return;
    }
    constexpr int N = Gran16<T>::N, L = D / N;   // elements and lanes per row
    const size_t at = ((size_t)(blockIdx.x - few) * 256 + threadIdx.x) / L;   // heads fastest, as the tensors lie
    const int part = threadIdx.x % L;
    const size_t n = (size_t)a.B * a.H * padded;
    const bool inside = at < n;
    const int h = (int)(at % a.H), t = (int)(at / a.H % padded), b = (int)(at / a.H / padded);
    const bool live = inside && t < seq_len(a.q_len, inside ? b : 0, a.Tq);
    float sum = 0.f, lse = kNegInf;
    if (live) {
        const size_t off = (((size_t)b * a.Tq + t) * a.H + h) * D + part * N;
        const uint4 x = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.o) + off);
        const uint4 y = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.dout) + off);
#pragma unroll
        for (int i = 0; i < N; ++i) sum = fmaf(Gran16<T>::get(x, i), Gran16<T>::get(y, i), sum);
        lse = a.lse[((size_t)b * a.H + h) * a.Tq + t];
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (inside && part == 0) {
        const int ql = seq_len(a.q_len, b, a.Tq);
        if (sees_few(t, seq_len(a.kv_len, b, a.Tk) - ql)) return;
        const bool none = !live || lse == kNegInf;
        float* to = a.rows + ((size_t)b * a.H + h) * padded * 2 + (t >> 2) * 8 + (t & 3);
        to[0] = none ? kNegInf : sizeof(T) == 4 ? -lse : -lse / a.scale;
        to[4] = none ? 0.f : -sum;
    }
}

// Adds the accumulators of the waves that took the other turns, through LDS, in
// the order of the turns; turn 0 is left with the sums.
template <int NG, int NT, int ND, int N>
__device__ __forceinline__ void join_turns(float* lds, floatx4 (&x)[ND][N], int group, int turn, int lane) {
    constexpr int kStride = (NT - 1) * NG * 64 * 4;   // floats between the fragments of one lane
    lds_barrier();  // the previous use of the LDS is over
    if (turn > 0) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int n = 0; n < N; ++n)
                *reinterpret_cast<floatx4*>(lds + (d * N + n) * kStride + (((turn - 1) * NG + group) * 64 + lane) * 4) = x[d][n];
    }
    lds_barrier();
    if (turn == 0) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int t = 0; t < NT - 1; ++t)
                    x[d][n] += *reinterpret_cast<const floatx4*>(lds + (d * N + n) * kStride + ((t * NG + group) * 64 + lane) * 4);
    }
}

// dk and dv of a tile of 16 NK NG keys.  Keys are the columns of S = Q K^T and
// dP = dO V^T, so the probabilities are right operands of dV^T += dO^T P and
// dK^T += Q^T dS as they stand.  The NW waves are NG groups of keys times NW / NG turns:
// a wave keeps its keys' fragments of K and V and both accumulators in registers
// and takes every (NW / NG)-th step of 32 queries from a two-deep LDS ring, head after
// head of those that share the keys; the turns are summed in LDS at the end, in order.
// Eight waves (fp32) take steps of 16 queries: the ring, which leaves room for no second
// workgroup, then feeds two waves on each SIMD.
template <typename T, int D, int NK, int NG, int NW>
__global__ __launch_bounds__(64 * NW, 2) void kda_attn_dkv_kernel(const AttnArgs a, int padded) {
    typedef TileGeom<T, D> G_;
    constexpr int NT = NW / NG, NS = G_::NS, ND = G_::ND, BK = 16 * NK * NG;
    constexpr int NI = NW == 8 ? 1 : 2, SR = 16 * NI, RB = SR * NT;   // 16-row blocks and rows of a step, rows of a tile
    // contraction steps whose K and V fragments stay in registers; at D = 128 those of the
    // fourth live in LDS (1 KiB a fragment), or two waves would not fit a SIMD
    constexpr int VR = sizeof(T) == 2 && D == 128 ? 3 : NS, VL = NS - VR;
    constexpr int kTile = RB * D * (int)sizeof(T);
    constexpr bool kInit = sizeof(T) == 2;   // the row values are initial accumulators
    static_assert(RB <= 128 && (NI == 2 || sizeof(T) == 4), "row values of a tile fit one copy; half a step is an fp32 product");
    constexpr int kSum = NT > 1 ? (NT - 1) * NG * 16 * NK * D * 4 : 0;   // the other turns' sums
    constexpr int kRing = 4 * kTile;
    __shared__ __attribute__((aligned(16))) unsigned char sm[kRing > kSum ? kRing : kSum];
    __shared__ __attribute__((aligned(16))) float srow[2][256];  // RB pairs, and room for a whole wave's copy
    __shared__ __attribute__((aligned(16))) T sv[VL > 0 ? NG * 2 * NK * VL * 512 : 1];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
    const int kgrp = wave % NG, turn = wave / NG;
    // Under a causal mask early keys are seen by most rows, and come first.  Where all
    // workgroups are there at once (NG = 4, two to a compute unit), those that share a
    // unit come half a grid apart: the second half runs backwards, so that a long
    // tile's neighbour is a short one (fp32, 16 heads x 2048, D = 128: 337 us, without 413).
    const int nbh = a.B * a.HK, ntile = (a.Tk + BK - 1) / BK, half = (ntile + 1) / 2, at_tile = blockIdx.x / nbh;
    const int bh = head_of(a, blockIdx.x, nbh), tile = NG < 4 || at_tile < half ? at_tile : ntile - 1 - (at_tile - half);
    const int b = bh / a.HK, hk = bh % a.HK;
    const int ql = seq_len(a.q_len, b, a.Tq), kl = seq_len(a.kv_len, b, a.Tk), off = kl - ql;
    const int k0 = tile * BK, k1 = min(k0 + BK, kl);  // keys of the tile inside the length
    // tokens that see some key of [k0, k1): t >= k0 - off if causal, t < k1 - 1 + window - off
    int t_lo = 0, t_hi = k0 < k1 ? ql : 0;
    if (a.causal) t_lo = max(0, k0 - off);
    if (a.window) t_hi = min(t_hi, max(0, k1 - 1 + a.window - off));
    // tiles of a head start at the 32 queries where the first one is seen, and nothing past
    // the last one is copied: small tiles of keys read 128 queries at a time
    const int beg = t_lo & ~31, per = t_lo < t_hi ? (t_hi - beg + RB - 1) / RB : 0;
    const int steps = per * a.G;

    // the tokens [seen_from(key), seen_to(key)) that see a key (lengths and the
    // window are below 2^29: no sum overflows)
    auto seen_from = [&](int key) { return a.causal ? min(max(key - off, 0), ql) : 0; };
    auto seen_to = [&](int key) { return key >= kl ? 0 : a.window ? min(max(key - off + a.window, 0), ql) : ql; };
    Frag<T> kf[NK][VR], vf[NK][VR];
    T* mine = sv + kgrp * 2 * NK * VL * 512;
    floatx4 dk[ND][NK], dv[ND][NK];
    const int w0 = k0 + kgrp * 16 * NK, w1 = min(w0 + 16 * NK, kl);
#pragma unroll
    for (int n = 0; n < NK; ++n) {
        const int kr = max(min(w0 + 16 * n + (lane & 15), kl - 1), 0);
        const T* kp = reinterpret_cast<const T*>(a.k) + ((size_t)b * a.Tk + kr) * a.ldk + (size_t)hk * D;
        const T* vp = reinterpret_cast<const T*>(a.v) + ((size_t)b * a.Tk + kr) * a.ldv + (size_t)hk * D;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const Frag<T> x = row_frag_global<T, D>(kp, s, lane), y = row_frag_global<T, D>(vp, s, lane);
            if (s < VR) {
                kf[n][s < VR ? s : 0] = x;
                vf[n][s < VR ? s : 0] = y;
            } else if (turn == 0) {
                frag_store(x, mine + ((s - VR) * 2 * NK + 2 * n) * 512, lane);
                frag_store(y, mine + ((s - VR) * 2 * NK + 2 * n + 1) * 512, lane);
            }
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            dk[d][n] = floatx4{0.f, 0.f, 0.f, 0.f};
            dv[d][n] = floatx4{0.f, 0.f, 0.f, 0.f};
        }
    }
    // queries that see some key of the wave, and those that see all 16 NK of them
    const int any_lo = w0 < w1 ? seen_from(w0) : 0, any_hi = w0 < w1 ? seen_to(w1 - 1) : 0;
    const int all_lo = seen_from(w0 + 16 * NK - 1), all_hi = w1 - w0 == 16 * NK ? seen_to(w0) : 0;

    const T* qbase = reinterpret_cast<const T*>(a.q) + (size_t)b * a.Tq * a.ldq + (size_t)hk * a.G * D;
    const size_t ldo = (size_t)a.H * D;
    const T* dobase = reinterpret_cast<const T*>(a.dout) + (size_t)b * a.Tq * ldo + (size_t)hk * a.G * D;
    const float* rbase = a.rows + ((size_t)b * a.H + (size_t)hk * a.G) * padded * 2;
    Stage<T, D, RB, NW> qst, dst;
    const uint32_t lds0 = lds_address(&sm[0]), lds_rows = lds_address(&srow[0][0]);
    qst.init(wave, lane, [&](int x) { return (uint32_t)(x * a.ldq * sizeof(T)); });
    dst.init(wave, lane, [&](int x) { return (uint32_t)(x * ldo * sizeof(T)); });
    auto stage = [&](int h, int t0, int buf) {
        const long long left = t_hi - 1 - t0;  // queries past the last one are past the windows and read as zeros
        qst.issue(buffer_window(qbase + t0 * a.ldq + (size_t)h * D, (left * (long long)a.ldq + D) * (long long)sizeof(T)),
                  lds0 + buf * 2 * kTile, wave);
        dst.issue(buffer_window(dobase + t0 * ldo + (size_t)h * D, (left * (long long)ldo + D) * (long long)sizeof(T)),
                  lds0 + (buf * 2 + 1) * kTile, wave);
        // a step's rows are within the padding; past it, and past the tile's rows, lanes read zeros past the
        // window, into rows of no step and the spare room
        if (wave == 0)
            copy_to_lds(buffer_window(rbase + 2 * ((size_t)h * padded + t0), min(RB, padded - t0) * 8), lane * 16, lds_rows + buf * 1024);
    };

    const TileLane<T, D> at(lane);
    const float c = a.scale_log2;
    auto step = [&](int rb, uint32_t qs, uint32_t ds, const float* rows, bool masked) {
        // bf16: P and dS are rounded for their products, 2^-8 relative each
        Frag<T> pf[NK], sf[NK];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (VL > 0) asm volatile("" ::: "memory");  // the second half reads its fragments again instead of keeping them
            const floatx4* rp = reinterpret_cast<const floatx4*>(rows + 2 * (16 * i + 4 * g));
            floatx4 st[NK], dp[NK];
#pragma unroll
            for (int n = 0; n < NK; ++n) st[n] = kInit ? rp[0] : floatx4{0.f, 0.f, 0.f, 0.f};
            if (kInit && masked) {  // -inf where the key is not seen: P and dS come out zero
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    const int key = w0 + 16 * n + (lane & 15), lo = seen_from(key);
                    const uint32_t span = max(seen_to(key) - lo, 0), first = rb + 16 * i + 4 * g - lo;
#pragma unroll
                    for (int e = 0; e < 4; ++e) st[n][e] = first + e < span ? st[n][e] : kNegInf;
                }
            }
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const Frag<T> qf = row_frag<D>(sm, qs, 16 * i, s, at, lane);
                const Frag<T> df = row_frag<D>(sm, ds, 16 * i, s, at, lane);
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    Frag<T> x, y;
                    if (s < VR) {
                        x = kf[n][s < VR ? s : 0];
                        y = vf[n][s < VR ? s : 0];
                    } else {
                        frag_load(x, mine + ((s - VR) * 2 * NK + 2 * n) * 512, lane);
                        frag_load(y, mine + ((s - VR) * 2 * NK + 2 * n + 1) * 512, lane);
                    }
                    st[n] = mma(qf, x, st[n]);
                    dp[n] = mma(df, y, s > 0 ? dp[n] : floatx4{0.f, 0.f, 0.f, 0.f});
                }
            }
            const floatx4 de = rp[1];
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                const int key = w0 + 16 * n + (lane & 15), lo = seen_from(key);
                const uint32_t span = max(seen_to(key) - lo, 0), first = rb + 16 * i + 4 * g - lo;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (kInit) {
                        st[n][e] = exp2_fast(st[n][e] * c);
                        dp[n][e] = (dp[n][e] + de[e]) * st[n][e];
                    } else {
                        const bool seen = !masked || first + e < span;
                        st[n][e] = seen ? probability<T>(a, st[n][e], rp[0][e]) : 0.f;
                        dp[n][e] = seen ? (dp[n][e] + de[e]) * st[n][e] : 0.f;
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NK; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pf[n].set(4 * i + e, st[n][e]);
                    sf[n].set(4 * i + e, dp[n][e]);
                }
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const Frag<T> dt = col_frag<D, 4 * NI>(sm, ds, 0, d, at, lane);
            const Frag<T> qt = col_frag<D, 4 * NI>(sm, qs, 0, d, at, lane);
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                dv[d][n] = mma_slots<4 * NI>(dt, pf[n], dv[d][n]);
                dk[d][n] = mma_slots<4 * NI>(qt, sf[n], dk[d][n]);
            }
        }
    };
    int h = 0, tt = beg;
    if (steps > 0) stage(0, beg, 0);
    for (int it = 0; it < steps; ++it) {
        const int buf = it & 1, t0 = tt + SR * turn;
        if ((tt += RB) >= t_hi) tt = beg, ++h;  // the next tile
        wait_vmcnt<0>();
        lds_barrier();
        if (it + 1 < steps) stage(h, tt, buf ^ 1);
        if (t0 >= any_hi || t0 + SR <= any_lo) continue;
        const uint32_t qs = buf * 2 * kTile + SR * turn * D * (int)sizeof(T), ds = qs + kTile;
        step(t0, qs, ds, &srow[buf][2 * SR * turn], t0 < all_lo || t0 + SR > all_hi);
    }

    if constexpr (NT > 1) {
        join_turns<NG, NT>(reinterpret_cast<float*>(sm), dk, kgrp, turn, lane);
        join_turns<NG, NT>(reinterpret_cast<float*>(sm), dv, kgrp, turn, lane);
        if (turn > 0) return;
    }
#pragma unroll
    for (int n = 0; n < NK; ++n) {
        const int key = w0 + 16 * n + (lane & 15);
        if (key >= a.Tk) continue;
        const size_t to = (((size_t)b * a.Tk + key) * a.HK + hk) * D + 4 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            store4(reinterpret_cast<T*>(a.dk) + to + 16 * d, dk[d][n] * a.scale);
            store4(reinterpret_cast<T*>(a.dv) + to + 16 * d, dv[d][n]);
        }
    }
}

// dq of a tile of packed rows: the forward's loop with the rows' lse in hand,
// S^T = K Q^T and dP^T = V dO^T, then dQ^T += K^T dS^T.  The NW waves are NG groups of
// rows times NW / NG turns over the steps of 32 keys (16 with eight waves), summed in LDS
// at the end.
template <typename T, int D, int NQ, int NG, int NW>
__global__ __launch_bounds__(64 * NW, NW == 8 ? 2 : 1) void kda_attn_dq_kernel(const AttnArgs a, int padded) {
    typedef TileGeom<T, D> G_;
    constexpr int NT = NW / NG, NS = G_::NS, ND = G_::ND, BQ = 16 * NQ * NG;
    constexpr int NI = NW == 8 ? 1 : 2, SR = 16 * NI;   // 16-key blocks and keys of a step
    static_assert(NI == 2 || sizeof(T) == 4, "half a step is an fp32 product");
    constexpr int KB = sizeof(T) == 2 && NT == 1 ? 64 : SR * NT;
    constexpr int kTile = KB * D * (int)sizeof(T);
    constexpr int kStep = SR * D * (int)sizeof(T);
    constexpr int kSum = (NT - 1) * NG * 16 * NQ * D * 4;   // the other turns' sums
    __shared__ __attribute__((aligned(16))) unsigned char sm[4 * kTile > kSum ? 4 * kTile : kSum];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
    const int nbh = a.B * a.HK, rows = a.Tq * a.G;
    const int ntile = (rows + BQ - 1) / BQ;
    const int bh = head_of(a, blockIdx.x, nbh), tile = ntile - 1 - blockIdx.x / nbh;
    const int b = bh / a.HK, hk = bh % a.HK;
    const int ql = seq_len(a.q_len, b, a.Tq), kl = seq_len(a.kv_len, b, a.Tk), off = kl - ql;
    const int r0 = tile * BQ, r1 = min(r0 + BQ, rows);
    const RowRange blk = row_range(a, r0, r1, ql, kl);
    const int k_beg = blk.key_lo & ~31, k_end = blk.key_hi > blk.key_lo ? blk.key_hi : k_beg;   // as the queries above

    const int rgrp = wave % NG, turn = wave / NG;
    const int w0 = r0 + rgrp * 16 * NQ;
    const RowRange mine = w0 < r1 ? row_range(a, w0, min(w0 + 16 * NQ, r1), ql, kl) : RowRange{0, -1, 0, 0};
    const int all_hi = a.causal ? min(kl, mine.t_first + off + 1) : kl;
    const int all_lo = a.window ? mine.t_last + off - a.window + 1 : 0;
    int t[NQ], lo[NQ], hi[NQ];
    float ls[NQ], de[NQ];
    Frag<T> qf[NQ][NS], df[NQ][NS];
    floatx4 dq[ND][NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int r = min(w0 + 16 * n + (lane & 15), rows - 1);
        t[n] = (int)fdiv((uint32_t)r, a.divG);
        const int h = hk * a.G + (r - t[n] * a.G), p = t[n] + off;
        hi[n] = a.causal ? min(kl - 1, p) : kl - 1;
        lo[n] = a.window ? p - a.window + 1 : 0;
        const int tr = max(min(t[n], ql - 1), 0);
        const T* qp = reinterpret_cast<const T*>(a.q) + ((size_t)b * a.Tq + tr) * a.ldq + (size_t)h * D;
        const T* dp = reinterpret_cast<const T*>(a.dout) + (((size_t)b * a.Tq + tr) * a.H + h) * D;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            qf[n][s] = row_frag_global<T, D>(qp, s, lane);
            df[n][s] = row_frag_global<T, D>(dp, s, lane);
        }
        const float* x = a.rows + ((size_t)b * a.H + h) * padded * 2 + (t[n] >> 2) * 8 + (t[n] & 3);
        ls[n] = sizeof(T) == 4 ? x[0] : x[0] * a.scale_log2;
        de[n] = x[4];
#pragma unroll
        for (int d = 0; d < ND; ++d) dq[d][n] = floatx4{0.f, 0.f, 0.f, 0.f};
    }

    const T* kbase = reinterpret_cast<const T*>(a.k) + (size_t)b * a.Tk * a.ldk + (size_t)hk * D;
    const T* vbase = reinterpret_cast<const T*>(a.v) + (size_t)b * a.Tk * a.ldv + (size_t)hk * D;
    Stage<T, D, KB, NW> kst, vst;
    kst.init(wave, lane, [&](int r) { return (uint32_t)(r * a.ldk * sizeof(T)); });
    vst.init(wave, lane, [&](int r) { return (uint32_t)(r * a.ldv * sizeof(T)); });
    const uint32_t lds0 = lds_address(&sm[0]);
    auto stage = [&](long long k0, int buf) {
        const long long left = k_end - 1 - k0;
        kst.issue(buffer_window(kbase + k0 * a.ldk, (left * (long long)a.ldk + D) * (long long)sizeof(T)), lds0 + buf * 2 * kTile, wave);
        vst.issue(buffer_window(vbase + k0 * a.ldv, (left * (long long)a.ldv + D) * (long long)sizeof(T)), lds0 + (buf * 2 + 1) * kTile, wave);
    };
    const TileLane<T, D> at(lane);
    if (k_beg < k_end) stage(k_beg, 0);
    for (int k0 = k_beg, buf = 0; k0 < k_end; k0 += KB, buf ^= 1) {
        wait_vmcnt<0>();
        lds_barrier();
        if (k0 + KB < k_end) stage(k0 + KB, buf ^ 1);
        if (k0 >= mine.key_hi || k0 + KB <= mine.key_lo) continue;
        const uint32_t ks = buf * 2 * kTile, vs = ks + kTile;
        const bool masked = k0 < all_lo || k0 + KB > all_hi;
#pragma unroll
        for (int v = 0; v < KB / SR / NT; ++v) {
            const int u = v * NT + turn;
            floatx4 st[NI][NQ], dp[NI][NQ];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    st[i][n] = floatx4{0.f, 0.f, 0.f, 0.f};
                    dp[i][n] = floatx4{0.f, 0.f, 0.f, 0.f};
                }
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const Frag<T> kf = row_frag<D>(sm, ks + turn * kStep, SR * v * NT + 16 * i, s, at, lane);
                    const Frag<T> vf = row_frag<D>(sm, vs + turn * kStep, SR * v * NT + 16 * i, s, at, lane);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        st[i][n] = mma(kf, qf[n][s], st[i][n]);
                        dp[i][n] = mma(vf, df[n][s], dp[i][n]);
                    }
                }
            }
            Frag<T> sf[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float p = probability<T>(a, st[i][n][e], ls[n]);
                        if (masked) {
                            const int key = k0 + SR * u + 16 * i + 4 * g + e;
                            p = key >= lo[n] && key <= hi[n] ? p : 0.f;
                        }
                        dp[i][n][e] = p == 0.f ? 0.f : p * (dp[i][n][e] + de[n]);
                    }
                sf[n] = frag_from_c<T>(dp[0][n], dp[NI - 1][n]);
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const Frag<T> kt_ = col_frag<D, 4 * NI>(sm, ks + turn * kStep, SR * v * NT, d, at, lane);
#pragma unroll
                for (int n = 0; n < NQ; ++n) dq[d][n] = mma_slots<4 * NI>(kt_, sf[n], dq[d][n]);
            }
        }
    }
    if constexpr (NT > 1) {
        join_turns<NG, NT>(reinterpret_cast<float*>(sm), dq, rgrp, turn, lane);
        if (turn > 0) return;
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int r = w0 + 16 * n + (lane & 15);
        if (r >= r1) continue;
        const int h = hk * a.G + (r - t[n] * a.G);
        T* p = reinterpret_cast<T*>(a.dq) + (((size_t)b * a.Tq + t[n]) * a.H + h) * D + 4 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d)
            store4(p + 16 * d, t[n] < ql ? dq[d][n] * a.scale : floatx4{0.f, 0.f, 0.f, 0.f});
    }
}

// Key or row groups of a workgroup.  Grids that fill the card with four groups take
// two, in two turns, so that there are workgroups left to even out a causal mask's long
// and short tiles: bf16, D = 64, dk and dv of 4 x 4 heads of 4 query heads, 4096 tokens,
// 294 us against 461, dq of 2 x 16 heads x 1024 19 us against 28.  Rows of more than 128
// bytes keep four: registers and LDS then leave room for one or two workgroups a unit
// either way (fp32, D = 128, dk and dv of 2 x 16 heads x 1024: 184 us against 205).
template <typename T, int D> constexpr int wide_groups() { return D * (int)sizeof(T) <= 128 ? 2 : 4; }
// Smaller grids share fewer keys or rows and take more turns, as far as the LDS ring
// reaches (its tiles hold 32 rows for each turn).
template <typename T, int D> constexpr int small_groups() { return D * (int)sizeof(T) >= 512 ? 2 : 1; }
// Grids of fewer workgroups of four groups are small.  256 leave no unit idle; rows of
// up to 64 bytes pay little for the turns and gain evenness up to 512 (bf16, D = 32, dk
// and dv of 2 x 4 heads of 4 query heads x 4096: 109 us against 184; D = 64, 2 x 16 heads x
// 1024: 32 us against 26).
template <typename T, int D> constexpr int small_grid() { return D * (int)sizeof(T) <= 64 ? 512 : 256; }

// Waves of a small grid's workgroup.  fp32, eight against four: dk and dv, D = 128, 1 x 4
// heads of 4 query heads x 512 156 us against 182, D = 64, 2 x 2 heads of 2 x 1024, window
// 256, 22 against 25 (the smallest, 2 x 4 heads x 64, 7.7 against 7.2); dq, D = 128, 8 heads
// x 1024 69 against 76, D = 64 29 against 30 and 4 x 8 heads x 256 15.4 against 14.1.
template <typename T> constexpr int dkv_small_waves() { return sizeof(T) == 4 ? 8 : 4; }
template <typename T, int D> constexpr int dq_small_waves() { return sizeof(T) == 4 && D == 128 ? 8 : 4; }

template <typename T, int D, int NG, int NW>
static hipError_t launch_dkv(const AttnArgs& a, int padded, hipStream_t s) {
    constexpr int NK = sizeof(T) == 2 ? 2 : 1, BK = 16 * NK * NG;
    const long long tiles = ((long long)a.Tk + BK - 1) / BK;
    hipLaunchKernelGGL((kda_attn_dkv_kernel<T, D, NK, NG, NW>), dim3((unsigned)(tiles * a.B * a.HK)), dim3(64 * NW), 0, s, a, padded);
    return hipGetLastError();
}
template <typename T, int D, int NG, int NW>
static hipError_t launch_dq(const AttnArgs& a, int padded, hipStream_t s) {
    constexpr int NQ = sizeof(T) == 2 ? 2 : 1, BQ = 16 * NQ * NG;
    const long long rows = (long long)a.Tq * a.G, tiles = (rows + BQ - 1) / BQ;
    hipLaunchKernelGGL((kda_attn_dq_kernel<T, D, NQ, NG, NW>), dim3((unsigned)(tiles * a.B * a.HK)), dim3(64 * NW), 0, s, a, padded);
    return hipGetLastError();
}

template <typename T, int D>
static hipError_t launch_bwd_t(const AttnArgs& a, hipStream_t s) {
    constexpr int kWide = sizeof(T) == 2 ? 128 : 64, kSmall = small_groups<T, D>();  // keys or rows of a workgroup
    const long long rows = (long long)a.Tq * a.G, nbh = (long long)a.B * a.HK;
    const int padded = (a.Tq + kAttnRowPad - 1) / kAttnRowPad * kAttnRowPad;
    hipError_t e = hipSuccess;
    if (rows > 0) {
        if (attn_few_keys(a)) {
            const size_t waves = (size_t)nbh * padded * a.G / 16;
            hipLaunchKernelGGL((kda_attn_rows_few_kernel<T, D>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, a, padded);
        } else {
            const size_t threads = (size_t)a.B * a.H * padded * (D * sizeof(T) / 16);
            const size_t few = sizeof(T) == 2 && a.causal ? ((size_t)nbh * (kFew / 16) * a.G + 3) / 4 : 0;
            hipLaunchKernelGGL((kda_attn_rows_kernel<T, D>), dim3((unsigned)(few + (threads + 255) / 256)), dim3(256), 0, s, a, padded, (int)few);
        }
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.Tk > 0) {
        const bool small = nbh * ((a.Tk + kWide - 1) / kWide) < small_grid<T, D>();
        e = attn_dkv_turns(sizeof(T), D, a) ? launch_dkv_turns(a, padded, s) : small ? launch_dkv<T, D, kSmall, dkv_small_waves<T>()>(a, padded, s) : launch_dkv<T, D, wide_groups<T, D>(), 4>(a, padded, s);
        if (e != hipSuccess) return e;
    }
    if (rows > 0) {
        const bool small = nbh * ((rows + kWide - 1) / kWide) < small_grid<T, D>();
        e = attn_dq_turns(sizeof(T), D, a) ? launch_dq_turns(D, a, padded, s) : small ? launch_dq<T, D, kSmall, dq_small_waves<T, D>()>(a, padded, s) : launch_dq<T, D, wide_groups<T, D>(), 4>(a, padded, s);
    }
    return e;
}

template <typename T>
static hipError_t launch_bwd_d(int D, const AttnArgs& a, hipStream_t s) {
    switch (D) {
        case 16: return launch_bwd_t<T, 16>(a, s);
        case 32: return launch_bwd_t<T, 32>(a, s);
        case 64: return launch_bwd_t<T, 64>(a, s);
        case 128: return launch_bwd_t<T, 128>(a, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_attn_bwd(int dt, int D, const AttnArgs& a, hipStream_t s) {
    return dt == 1 ? launch_bwd_d<bf16_t>(D, a, s) : launch_bwd_d<float>(D, a, s);
}

}  // namespace kda
