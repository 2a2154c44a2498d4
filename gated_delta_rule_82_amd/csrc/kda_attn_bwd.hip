// kda_attn_bwd.hip - softmax attention backward on gfx950.
//
//   P_ij = exp(c q_i.k_j - lse_i),  delta_i = dout_i.o_i
//   dv_j = sum_i P_ij dout_i,  dS_ij = P_ij (dout_i.v_j - delta_i)
//   dq_i = c sum_j dS_ij k_j,  dk_j = c sum_i dS_ij q_i
//
// Three kernels: the row values (lse, delta); dk and dv, one workgroup per tile
// of keys, over the packed rows that see it (all query heads of the key/value
// head, so shared heads are summed in registers); dq, one workgroup per tile of
// packed rows.  Scores and dout.v are formed twice (7 products instead of 5):
// in exchange every sum stays in one workgroup's registers, in a fixed order,
// with no atomics and no partial results in memory.
#include "kda_attn_device.h"

namespace kda {

// Row values of every packed row, padded per head to whole tiles with rows that
// contribute nothing (lse = +inf makes P zero): rows[bh][r] = (lse log2 e, delta).
template <typename T, int D>
__global__ __launch_bounds__(256) void kda_attn_rows_kernel(const AttnArgs a, int padded) {
    constexpr int N = Gran16<T>::N, L = D / N;   // elements and lanes per row
    const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) / L;
    const int part = threadIdx.x % L;
    const size_t n = (size_t)a.B * a.HK * padded;
    const bool inside = at < n;
    const int r = (int)(at % padded), bh = (int)(at / padded), b = bh / a.HK, hk = bh % a.HK;
    const int t = (int)fdiv((uint32_t)r, a.divG), h = hk * a.G + (r - t * a.G);
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
        const bool none = !live || lse == kNegInf;
        *reinterpret_cast<float2*>(a.rows + 2 * at) = none ? make_float2(-kNegInf, 0.f) : make_float2(lse * kLog2e, sum);
    }
}

// dk and dv of a tile of 16 NK NW keys.  Keys are the columns of S = Q K^T and
// dP = dO V^T, so the probabilities are right operands of dV^T += dO^T P and
// dK^T += Q^T dS as they stand; a wave keeps its keys' fragments of K and V and
// both accumulators in registers while 32 RB / 32 packed rows at a time pass through
// a two-deep LDS ring.
template <typename T, int D, int NK, int RB, int NW>
__global__ __launch_bounds__(64 * NW, 1) void kda_attn_dkv_kernel(const AttnArgs a, int padded) {
    typedef TileGeom<T, D> G_;
    constexpr int NS = G_::NS, ND = G_::ND, BK = 16 * NK * NW;
    constexpr int kTile = RB * D * (int)sizeof(T);
    __shared__ __attribute__((aligned(16))) unsigned char sm[2][2][kTile];
    __shared__ __attribute__((aligned(16))) float srow[2][256];  // RB pairs, and room for a whole wave's copy
    static_assert(RB <= 128, "row values fit");

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
    const int nbh = a.B * a.HK;
    const int bh = blockIdx.x % nbh, tile = blockIdx.x / nbh;  // early keys (seen by most rows) first
    const int b = bh / a.HK, hk = bh % a.HK;
    const int ql = seq_len(a.q_len, b, a.Tq), kl = seq_len(a.kv_len, b, a.Tk), off = kl - ql;
    const int k0 = tile * BK, k1 = min(k0 + BK, kl);  // keys of the tile inside the length
    // tokens that see some key of [k0, k1): t >= k0 - off if causal, t < k1 - 1 + window - off
    int t_lo = 0, t_hi = k0 < k1 ? ql : 0;
    if (a.causal) t_lo = max(0, k0 - off);
    if (a.window) t_hi = min((long long)t_hi, max(0ll, (long long)k1 - 1 + a.window - off));
    const int r_lo = t_lo < t_hi ? t_lo * a.G : 0, r_hi = t_lo < t_hi ? t_hi * a.G : 0;
    const int beg = r_lo / RB, end = (r_hi + RB - 1) / RB;

    // this lane's keys and the packed rows [rlo, rhi) that see them
    int rlo[NK], rhi[NK];
    Frag<T> kf[NK][NS], vf[NK][NS];
    floatx4 dk[ND][NK], dv[ND][NK];
    const int w0 = k0 + wave * 16 * NK;
    bool some = false;
#pragma unroll
    for (int n = 0; n < NK; ++n) {
        const int key = w0 + 16 * n + (lane & 15);
        long long tl = a.causal ? (long long)key - off : 0, th = a.window ? (long long)key + a.window - off : ql;
        tl = tl < 0 ? 0 : tl > ql ? ql : tl;
        th = th < 0 ? 0 : th > ql ? ql : th;
        if (key >= kl) th = 0;
        rlo[n] = (int)tl * a.G;
        rhi[n] = (int)th * a.G;
        some |= rlo[n] < rhi[n];
        const int kr = max(min(key, kl - 1), 0);
        const T* kp = reinterpret_cast<const T*>(a.k) + ((size_t)b * a.Tk + kr) * a.ldk + (size_t)hk * D;
        const T* vp = reinterpret_cast<const T*>(a.v) + ((size_t)b * a.Tk + kr) * a.ldv + (size_t)hk * D;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            kf[n][s] = row_frag_global<T, D>(kp, s, lane);
            vf[n][s] = row_frag_global<T, D>(vp, s, lane);
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            dk[d][n] = floatx4{0.f, 0.f, 0.f, 0.f};
            dv[d][n] = floatx4{0.f, 0.f, 0.f, 0.f};
        }
    }
    const bool active = __any(some);

    const T* qbase = reinterpret_cast<const T*>(a.q) + (size_t)b * a.Tq * a.ldq + (size_t)hk * a.G * D;
    const size_t ldo = (size_t)a.H * D;
    const T* dobase = reinterpret_cast<const T*>(a.dout) + (size_t)b * a.Tq * ldo + (size_t)hk * a.G * D;
    const float* rbase = a.rows + 2 * (size_t)bh * padded;
    Stage<T, D, RB, NW> qst, dst;
    const uint32_t lds0 = lds_address(&sm[0][0][0]), lds_rows = lds_address(&srow[0][0]);
    auto place = [&](int skip) {  // row x of a tile is packed row skip + x of the window's tokens
        qst.init(wave, lane, [&](int x) {
            const int t = (int)fdiv((uint32_t)(skip + x), a.divG);
            return (uint32_t)((t * a.ldq + (size_t)(skip + x - t * a.G) * D) * sizeof(T));
        });
        dst.init(wave, lane, [&](int x) {
            const int t = (int)fdiv((uint32_t)(skip + x), a.divG);
            return (uint32_t)((t * ldo + (size_t)(skip + x - t * a.G) * D) * sizeof(T));
        });
    };
    place(0);
    const bool whole_tokens = RB % a.G == 0;  // every tile starts with a token's first head
    auto stage = [&](int rt, int buf) {
        const int t0 = (int)fdiv((uint32_t)(rt * RB), a.divG);
        if (!whole_tokens) place(rt * RB - t0 * a.G);
        const long long left = ql - 1 - t0;  // rows past the last token's are past the windows and read as zeros
        qst.issue(buffer_window(qbase + t0 * a.ldq, (left * (long long)a.ldq + (long long)a.G * D) * (long long)sizeof(T)),
                  lds0 + buf * 2 * kTile, wave);
        dst.issue(buffer_window(dobase + t0 * ldo, (left * (long long)ldo + (long long)a.G * D) * (long long)sizeof(T)),
                  lds0 + (buf * 2 + 1) * kTile, wave);
        // the row array is padded to whole tiles; lanes past a tile's rows read zeros past the window, into the spare half
        if (wave == 0) copy_to_lds(buffer_window(rbase + 2 * (size_t)rt * RB, RB * 8), lane * 16, lds_rows + buf * 1024);
    };

    const float c = a.scale_log2;
    if (beg < end) stage(beg, 0);
    for (int rt = beg; rt < end; ++rt) {
        const int buf = (rt - beg) & 1;
        wait_vmcnt<0>();
        lds_barrier();
        if (rt + 1 < end) stage(rt + 1, buf ^ 1);
        if (!active) continue;
        const unsigned char* qs = sm[buf][0];
        const unsigned char* ds = sm[buf][1];
#pragma unroll
        for (int u = 0; u < RB / 32; ++u) {
            const int rb = rt * RB + 32 * u;
            floatx4 st[2][NK], dp[2][NK];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    st[i][n] = floatx4{0.f, 0.f, 0.f, 0.f};
                    dp[i][n] = floatx4{0.f, 0.f, 0.f, 0.f};
                }
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const Frag<T> qf = row_frag<D>(qs, 32 * u + 16 * i, s, lane, T());
                    const Frag<T> df = row_frag<D>(ds, 32 * u + 16 * i, s, lane, T());
#pragma unroll
                    for (int n = 0; n < NK; ++n) {
                        st[i][n] = mma(qf, kf[n][s], st[i][n]);
                        dp[i][n] = mma(df, vf[n][s], dp[i][n]);
                    }
                }
            }
            bool whole = true;  // every key of the wave is seen by every row of the step
#pragma unroll
            for (int n = 0; n < NK; ++n) whole &= rlo[n] <= rb && rb + 32 <= rhi[n];
            const bool masked = !__all(whole);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4* rp = reinterpret_cast<const float4*>(&srow[buf][2 * (32 * u + 16 * i + 4 * g)]);
                const float4 x = rp[0], y = rp[1];
                const float ls[4] = {x.x, x.z, y.x, y.z}, de[4] = {x.y, x.w, y.y, y.w};
#pragma unroll
                for (int n = 0; n < NK; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float p = exp2_fast(fmaf(st[i][n][e], c, -ls[e]));
                        if (masked) {
                            const int r = rb + 16 * i + 4 * g + e;
                            p = r >= rlo[n] && r < rhi[n] ? p : 0.f;
                        }
                        st[i][n][e] = p;
                        dp[i][n][e] = p == 0.f ? 0.f : p * (dp[i][n][e] - de[e]);
                    }
            }
            // bf16: P and dS are rounded for their products, 2^-9 relative each
            Frag<T> pf[NK], sf[NK];
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                pf[n] = frag_from_c<T>(st[0][n], st[1][n]);
                sf[n] = frag_from_c<T>(dp[0][n], dp[1][n]);
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const Frag<T> dt = col_frag<D>(ds, 32 * u, d, lane, T());
                const Frag<T> qt = col_frag<D>(qs, 32 * u, d, lane, T());
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    dv[d][n] = mma(dt, pf[n], dv[d][n]);
                    dk[d][n] = mma(qt, sf[n], dk[d][n]);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NK; ++n) {
        const int key = w0 + 16 * n + (lane & 15);
        if (key >= a.Tk) continue;
        const size_t at = (((size_t)b * a.Tk + key) * a.HK + hk) * D + 4 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            store4(reinterpret_cast<T*>(a.dk) + at + 16 * d, dk[d][n] * a.scale);
            store4(reinterpret_cast<T*>(a.dv) + at + 16 * d, dv[d][n]);
        }
    }
}

// dq of a tile of packed rows: the forward's loop with the rows' lse in hand,
// S^T = K Q^T and dP^T = V dO^T, then dQ^T += K^T dS^T.
template <typename T, int D, int NQ, int KB, int NW>
__global__ __launch_bounds__(64 * NW, 1) void kda_attn_dq_kernel(const AttnArgs a, int padded) {
    typedef TileGeom<T, D> G_;
    constexpr int NS = G_::NS, ND = G_::ND, BQ = 16 * NQ * NW;
    constexpr int kTile = KB * D * (int)sizeof(T);
    __shared__ __attribute__((aligned(16))) unsigned char sm[2][2][kTile];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
    const int nbh = a.B * a.HK, rows = a.Tq * a.G;
    const int ntile = (rows + BQ - 1) / BQ;
    const int bh = blockIdx.x % nbh, tile = ntile - 1 - blockIdx.x / nbh;
    const int b = bh / a.HK, hk = bh % a.HK;
    const int ql = seq_len(a.q_len, b, a.Tq), kl = seq_len(a.kv_len, b, a.Tk), off = kl - ql;
    const int r0 = tile * BQ, r1 = min(r0 + BQ, rows);
    const RowRange blk = row_range(a, r0, r1, ql, kl);
    const int k_beg = blk.key_lo / KB, k_end = blk.key_hi > blk.key_lo ? (blk.key_hi + KB - 1) / KB : k_beg;

    const int w0 = r0 + wave * 16 * NQ;
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
        const float2 x = *reinterpret_cast<const float2*>(a.rows + 2 * ((size_t)bh * padded + r));
        ls[n] = x.x;
        de[n] = x.y;
#pragma unroll
        for (int d = 0; d < ND; ++d) dq[d][n] = floatx4{0.f, 0.f, 0.f, 0.f};
    }

    const T* kbase = reinterpret_cast<const T*>(a.k) + (size_t)b * a.Tk * a.ldk + (size_t)hk * D;
    const T* vbase = reinterpret_cast<const T*>(a.v) + (size_t)b * a.Tk * a.ldv + (size_t)hk * D;
    Stage<T, D, KB, NW> kst, vst;
    kst.init(wave, lane, [&](int r) { return (uint32_t)(r * a.ldk * sizeof(T)); });
    vst.init(wave, lane, [&](int r) { return (uint32_t)(r * a.ldv * sizeof(T)); });
    const uint32_t lds0 = lds_address(&sm[0][0][0]);
    auto stage = [&](int kt, int buf) {
        const long long k0 = (long long)kt * KB, left = kl - 1 - k0;
        kst.issue(buffer_window(kbase + k0 * a.ldk, (left * (long long)a.ldk + D) * (long long)sizeof(T)), lds0 + buf * 2 * kTile, wave);
        vst.issue(buffer_window(vbase + k0 * a.ldv, (left * (long long)a.ldv + D) * (long long)sizeof(T)), lds0 + (buf * 2 + 1) * kTile, wave);
    };
    const float c = a.scale_log2;
    if (k_beg < k_end) stage(k_beg, 0);
    for (int kt = k_beg; kt < k_end; ++kt) {
        const int buf = (kt - k_beg) & 1, k0 = kt * KB;
        wait_vmcnt<0>();
        lds_barrier();
        if (kt + 1 < k_end) stage(kt + 1, buf ^ 1);
        if (k0 >= mine.key_hi || k0 + KB <= mine.key_lo) continue;
        const unsigned char* ks = sm[buf][0];
        const unsigned char* vs = sm[buf][1];
        const bool masked = k0 < all_lo || k0 + KB > all_hi;
#pragma unroll
        for (int u = 0; u < KB / 32; ++u) {
            floatx4 st[2][NQ], dp[2][NQ];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    st[i][n] = floatx4{0.f, 0.f, 0.f, 0.f};
                    dp[i][n] = floatx4{0.f, 0.f, 0.f, 0.f};
                }
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const Frag<T> kf = row_frag<D>(ks, 32 * u + 16 * i, s, lane, T());
                    const Frag<T> vf = row_frag<D>(vs, 32 * u + 16 * i, s, lane, T());
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
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float p = exp2_fast(fmaf(st[i][n][e], c, -ls[n]));
                        if (masked) {
                            const int key = k0 + 32 * u + 16 * i + 4 * g + e;
                            p = key >= lo[n] && key <= hi[n] ? p : 0.f;
                        }
                        dp[i][n][e] = p == 0.f ? 0.f : p * (dp[i][n][e] - de[n]);
                    }
                sf[n] = frag_from_c<T>(dp[0][n], dp[1][n]);
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const Frag<T> kt_ = col_frag<D>(ks, 32 * u, d, lane, T());
#pragma unroll
                for (int n = 0; n < NQ; ++n) dq[d][n] = mma(kt_, sf[n], dq[d][n]);
            }
        }
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

template <typename T, int D>
static hipError_t launch_bwd_t(const AttnArgs& a, hipStream_t s) {
    constexpr bool kWide = sizeof(T) == 2;
    constexpr int NK = kWide ? 2 : 1, RB = kWide ? 64 : 32, NQ = kWide ? 2 : 1, KB = kWide ? 64 : 32;
    const long long rows = (long long)a.Tq * a.G, nbh = (long long)a.B * a.HK;
    const int padded = (int)((rows + kAttnRowPad - 1) / kAttnRowPad * kAttnRowPad);
    if (rows > 0) {
        const size_t threads = (size_t)nbh * padded * (D * sizeof(T) / 16);
        hipLaunchKernelGGL((kda_attn_rows_kernel<T, D>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a, padded);
        if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
    }
    if (a.Tk > 0) {
        constexpr int BK = 16 * NK * 4;
        const long long tiles = ((long long)a.Tk + BK - 1) / BK;
        hipLaunchKernelGGL((kda_attn_dkv_kernel<T, D, NK, RB, 4>), dim3((unsigned)(tiles * nbh)), dim3(256), 0, s, a, padded);
        if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
    }
    if (rows > 0) {
        constexpr int BQ = 16 * NQ * 4;
        const long long tiles = (rows + BQ - 1) / BQ;
        hipLaunchKernelGGL((kda_attn_dq_kernel<T, D, NQ, KB, 4>), dim3((unsigned)(tiles * nbh)), dim3(256), 0, s, a, padded);
    }
    return hipGetLastError();
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
