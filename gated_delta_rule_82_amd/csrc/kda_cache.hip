// kda_cache.hip - the 8-bit paged key/value cache on gfx950: append, and the
// attention of the newest tokens over it (decode).
//
// Codes are e4m3; a page has one power-of-two scale per key/value head, so moving
// codes to a larger scale is exact down to the subnormals and no scale ever
// depends on how a division rounds.  K pages are [page][D], V pages [D][page]:
// both are then read along their contraction axis, 16 bytes a lane, straight into
// the matrix operands.
#include "kda_cache_device.h"

namespace kda {

namespace {

constexpr float kE4m3Max = 448.f;

// Smallest power of two s with amax <= 448 s, between 2^-100 and 2^120.
__device__ __forceinline__ float scale_for(float amax) {
    // 448 = 0.875 * 2^9
    int e;
    const float f = frexpf(amax, &e);
    int x = f <= 0.875f ? e - 9 : e - 8;
    x = amax > 0.f ? (x < -100 ? -100 : x > 120 ? 120 : x) : -100;
    return ldexpf(1.f, x);
}

__device__ __forceinline__ float finite_abs(float x) {
    const float y = fabsf(x);
    return y < __builtin_inff() ? y : 0.f;  // infinities and NaN set no scale
}

// x * inv within the codes' range: infinities saturate, NaN stays NaN.
__device__ __forceinline__ float to_range(float x, float inv) {
    const float y = x * inv;
    return y != y ? y : __builtin_amdgcn_fmed3f(y, -kE4m3Max, kE4m3Max);
}
// Codes of four values in range, nearest even, the first in the lowest byte.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}
__device__ __forceinline__ uint8_t encode(float x, float inv) {
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(to_range(x, inv), 0.f, 0, false) & 0xff);
}
__device__ __forceinline__ float decode(uint32_t code) { return __builtin_amdgcn_cvt_f32_fp8((int)code, 0); }

// Eight consecutive elements as loaded.
template <typename T> struct Raw8;
template <> struct Raw8<bf16_t> {
    uint4 v;
    __device__ __forceinline__ void load(const bf16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float get(int i) const { return Gran16<bf16_t>::get(v, i); }
};
template <> struct Raw8<float> {
    uint4 v[2];
    __device__ __forceinline__ void load(const float* p) {
        v[0] = reinterpret_cast<const uint4*>(p)[0];
        v[1] = reinterpret_cast<const uint4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float get(int i) const { return Gran16<float>::get(v[i >> 2], i & 3); }
};

// Threads of the append's workgroup: one for each four tokens by eight channels of
// a page, at most 256.
constexpr int append_items(int D, int page) { return (D / 8) * (page / 4); }
constexpr int append_threads(int D, int page) { return append_items(D, page) >= 256 ? 256 : append_items(D, page) >= 128 ? 128 : 64; }

}  // namespace

// One workgroup per (sequence, key/value head, page touched).  A thread holds four
// tokens by eight channels of K and of V, so every input is read once: the maxima
// of both are reduced together, K's codes leave as they are (8 bytes a token), V's
// are turned into words of four tokens and leave through LDS as whole 16-byte
// pieces of the page's rows (single bytes where tokens before or after them stay).
// Bound by the bytes: 4 x 4096 tokens of 8 heads x 128 in bf16 (101 MB) 20.5 us, 4.9 TB/s.
// That is without a scale that grows under older tokens: their codes are moved a byte at a
// time, each load waited for before its store.  256 sequences of 4 new tokens, every page's
// scale growing: 103 us with 32 older tokens in pages of 64, 177 with 60, 480 with 124 of
// 128; 20 to 27 us where none grows.
template <typename T, int D, int PAGE>
__global__ __launch_bounds__(append_threads(D, PAGE)) void kda_cache_append_kernel(const AppendArgs a, int touched) {
    constexpr int NTH = append_threads(D, PAGE), G8 = D / 8, ITEMS = append_items(D, PAGE), U = (ITEMS + NTH - 1) / NTH;
    constexpr int ROW = PAGE / 4 + 1;                       // words of an LDS row (odd: rows spread over the banks)
    __shared__ float red[2][NTH / 64];
    __shared__ uint32_t turned[D * ROW];
    const int tid = threadIdx.x;
    const int bh = blockIdx.x / touched, j = blockIdx.x % touched;
    const int b = bh / a.HK, hk = bh % a.HK;
    const long long before = max(a.cache_len[b], 0), fresh = seq_len(a.new_len, b, a.T);
    const long long pn = before / PAGE + j, p0 = pn * PAGE;  // page of the sequence and its first token
    const long long lo = max(before, p0), hi = min(before + fresh, p0 + PAGE);
    if (lo >= hi || pn >= a.max_pages) return;
    const int pg = a.block_table[(size_t)b * a.max_pages + pn];
    const int older = (int)(lo - p0), end = (int)(hi - p0);  // slots [older, end) of the page are written
    const size_t tok0 = (size_t)b * a.T + (size_t)(lo - before);

    Raw8<T> xk[U][4], xv[U][4];
    float top_k = 0.f, top_v = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int item = u * NTH + tid, dg = item % G8, s4 = item / G8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int slot = 4 * s4 + i;
            if (slot >= older && slot < end) {
                const size_t tok = tok0 + (slot - older);
                xk[u][i].load(reinterpret_cast<const T*>(a.k) + tok * a.ldk + (size_t)hk * D + dg * 8);
                xv[u][i].load(reinterpret_cast<const T*>(a.v) + tok * a.ldv + (size_t)hk * D + dg * 8);
            } else {
                xk[u][i].zero();
                xv[u][i].zero();
            }
        }
    }
    if (pg < 0 || pg >= a.n_pages) return;  // no page: the tokens are dropped
    const size_t slot0 = (size_t)pg * a.HK + hk;
    uint8_t* kc = a.k_cache + slot0 * (PAGE * D);
    uint8_t* vc = a.v_cache + slot0 * (PAGE * D);
    const float was_k = older > 0 ? a.k_scale[slot0] : 0.f, was_v = older > 0 ? a.v_scale[slot0] : 0.f;
    // this thread's four tokens hold none that is written
    auto idle = [&](int u) {
        const int s = 4 * ((u * NTH + tid) / G8);
        return s + 4 <= older || s >= end;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (idle(u)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                top_k = fmaxf(top_k, finite_abs(xk[u][i].get(e)));
                top_v = fmaxf(top_v, finite_abs(xv[u][i].get(e)));
            }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        top_k = fmaxf(top_k, __shfl_xor(top_k, o, 64));
        top_v = fmaxf(top_v, __shfl_xor(top_v, o, 64));
    }
    if ((tid & 63) == 0) {
        red[0][tid >> 6] = top_k;
        red[1][tid >> 6] = top_v;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NTH / 64; ++w) {
        top_k = fmaxf(top_k, red[0][w]);
        top_v = fmaxf(top_v, red[1][w]);
    }
    // never below the scale of the tokens there (one that is not a number counts as none)
    const float sk = fmaxf(scale_for(top_k), was_k), sv = fmaxf(scale_for(top_v), was_v);
    if (older > 0 && (sk > was_k || sv > was_v)) {  // those tokens move to the larger scale
        const float rk = was_k / sk, rv = was_v / sv;
        for (int i = tid; i < older * D; i += NTH) {
            if (sk > was_k) kc[i] = encode(decode(kc[i]), rk);
            if (sv > was_v) {
                uint8_t* p = vc + (size_t)(i % D) * PAGE + i / D;
                *p = encode(decode(*p), rv);
            }
        }
    }
    const float ik = 1.f / sk, iv = 1.f / sv;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int item = u * NTH + tid, dg = item % G8, s4 = item / G8;
        if (idle(u)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int slot = 4 * s4 + i;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = to_range(xk[u][i].get(e), ik);
            if (slot >= older && slot < end)
                *reinterpret_cast<uint2*>(kc + slot * D + dg * 8) = make_uint2(encode4(y[0], y[1], y[2], y[3]), encode4(y[4], y[5], y[6], y[7]));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            turned[(dg * 8 + e) * ROW + s4] = encode4(to_range(xv[u][0].get(e), iv), to_range(xv[u][1].get(e), iv),
                                                     to_range(xv[u][2].get(e), iv), to_range(xv[u][3].get(e), iv));
    }
    __syncthreads();
    constexpr int C = PAGE / 16;   // 16-byte pieces of a row
    for (int i = tid; i < D * C; i += NTH) {
        const int d = i / C, s0 = (i % C) * 16;
        if (s0 + 16 <= older || s0 >= end) continue;
        const uint32_t* w = turned + d * ROW + s0 / 4;
        uint8_t* p = vc + d * PAGE + s0;
        if (s0 >= older && s0 + 16 <= end) {
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int s = max(older - s0, 0); s < min(end - s0, 16); ++s) p[s] = (uint8_t)(w[s >> 2] >> (8 * (s & 3)));
        }
    }
    if (tid == 0) {
        a.k_scale[slot0] = sk;
        a.v_scale[slot0] = sv;
    }
}

// One token a sequence (decode): a lane holds eight channels of K or of V, D / 8 lanes
// each, a wave one (sequence, key/value head); no LDS and no barrier.  B = 256, 8 heads,
// D = 128, where no page's scale grows: 5 to 7 us, against 14 us with the workgroup above,
// whose registers for a whole page let only five of them share a compute unit.
// Where one grows, its lanes move the older tokens' codes a byte at a time, each load waited
// for before its store, and the slowest wave decides: 24 us behind 8 older tokens, 74 behind
// 32, 139 behind 63 of a page of 64, 719 behind 127 of 128.  In a decode of normal values
// (256 sequences of mixed lengths, pages of 64) some page's scale grows in every step: 76 us,
// 54 to 90 over 128 steps.  Codes moved in 16-byte pieces are the remedy; not done here.
template <typename T, int D>
__global__ __launch_bounds__(256) void kda_cache_append_one_kernel(const AppendArgs a) {
    constexpr int G8 = D / 8;
    const int lane = threadIdx.x & 63, bh = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (bh >= a.B * a.HK) return;
    const int b = bh / a.HK, hk = bh % a.HK;
    const bool kv = lane >= G8, mine = lane < 2 * G8;     // V's lanes follow K's
    const int dg = lane % G8;
    Raw8<T> x;
    x.zero();
    if (mine) x.load(reinterpret_cast<const T*>(kv ? a.v : a.k) + (size_t)b * (kv ? a.ldv : a.ldk) + (size_t)hk * D + dg * 8);
    const int before = max(a.cache_len[b], 0), pn = before / a.page, older = before % a.page;
    if (seq_len(a.new_len, b, 1) == 0 || pn >= a.max_pages) return;
    const int pg = a.block_table[(size_t)b * a.max_pages + pn];
    if (pg < 0 || pg >= a.n_pages) return;
    const size_t slot0 = (size_t)pg * a.HK + hk;
    uint8_t* codes = (kv ? a.v_cache : a.k_cache) + slot0 * a.page * D;
    float* scale = (kv ? a.v_scale : a.k_scale) + slot0;
    const float was = older > 0 ? *scale : 0.f;
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, finite_abs(x.get(e)));
#pragma unroll
    for (int o = G8 / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if (!mine) return;
    const float s = fmaxf(scale_for(top), was), inv = 1.f / s;
    if (older > 0 && s > was) {  // the tokens there move to the larger scale: each lane those of its channels
        const float r = was / s;
        for (int t = 0; t < older; ++t)
            for (int e = 0; e < 8; ++e) {
                const int d = dg * 8 + e;
                uint8_t* p = codes + (kv ? (size_t)d * a.page + t : (size_t)t * D + d);
                *p = encode(decode(*p), r);
            }
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = to_range(x.get(e), inv);
    const uint32_t w0 = encode4(y[0], y[1], y[2], y[3]), w1 = encode4(y[4], y[5], y[6], y[7]);
    if (!kv) {
        *reinterpret_cast<uint2*>(codes + (size_t)older * D + dg * 8) = make_uint2(w0, w1);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) codes[(size_t)(dg * 8 + e) * a.page + older] = (uint8_t)((e < 4 ? w0 : w1) >> (8 * (e & 3)));
    }
    if (dg == 0) *scale = s;
}

template <typename T, int D, int PAGE>
static hipError_t launch_append_p(const AppendArgs& a, hipStream_t s) {
    const int touched = (a.T + PAGE - 2) / PAGE + 1;
    hipLaunchKernelGGL((kda_cache_append_kernel<T, D, PAGE>), dim3((unsigned)((size_t)a.B * a.HK * touched)),
                       dim3(append_threads(D, PAGE)), 0, s, a, touched);
    return hipGetLastError();
}
template <typename T, int D>
static hipError_t launch_append_t(const AppendArgs& a, hipStream_t s) {
    if (a.T == 1) {
        hipLaunchKernelGGL((kda_cache_append_one_kernel<T, D>), dim3((unsigned)(((size_t)a.B * a.HK + 3) / 4)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    switch (a.page) {
        case 16: return launch_append_p<T, D, 16>(a, s);
        case 32: return launch_append_p<T, D, 32>(a, s);
        case 64: return launch_append_p<T, D, 64>(a, s);
        case 128: return launch_append_p<T, D, 128>(a, s);
        default: return hipErrorInvalidValue;
    }
}
template <typename T>
static hipError_t launch_append_d(int D, const AppendArgs& a, hipStream_t s) {
    switch (D) {
        case 16: return launch_append_t<T, 16>(a, s);
        case 32: return launch_append_t<T, 32>(a, s);
        case 64: return launch_append_t<T, 64>(a, s);
        case 128: return launch_append_t<T, 128>(a, s);
        default: return hipErrorInvalidValue;
    }
}
hipError_t launch_cache_append(int dt, int D, const AppendArgs& a, hipStream_t s) {
    return dt == 1 ? launch_append_d<bf16_t>(D, a, s) : launch_append_d<float>(D, a, s);
}

constexpr int kStepWaves = 4;

// A wave takes blocks of 64 keys (CacheRows).  The waves of a workgroup take blocks in
// turn and are joined in LDS; splits of a long cache are joined by kda_attn_join_kernel.  Nothing of the
// cache is staged: every byte is used by one wave, and loads straight into the operands
// leave the LDS and barriers out of the stream.  Bound by the bytes: 256 sequences of up
// to 4096 tokens, 8 heads of 128 channels (1.21 GB), 32 query heads 216 us, 5.6 TB/s; one
// sequence of 65 536, four new tokens (134 MB) 27 us and 5.5 for the join of 128 parts.
template <typename T, int D, int NR>
__global__ __launch_bounds__(64 * kStepWaves) void kda_attn_step_kernel(const AttnStepArgs a) {
    constexpr int ND = D / 16, NW = kStepWaves;
    __shared__ __attribute__((aligned(16))) float so[NW][16][D + 4];
    __shared__ float sml[NW][16][2];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, lr = lane & 15;
    const int nbh = a.B * a.HK, rows = a.Tq * a.G;
    int bid = blockIdx.x;
    const int bh = bid % nbh;
    bid /= nbh;
    const int split = bid % a.nsplit, r0 = (bid / a.nsplit) * 16 * NR;
    const int b = bh / a.HK, hk = bh % a.HK;
    const int cap = a.max_pages * a.page;
    const int ql = seq_len(a.new_len, b, a.Tq);
    // positions count from the length, which may lie past the table's end; cached tokens
    // are no more than the table has entries for
    const long long before = max(a.cache_len[b], 0);
    const int kl = (int)min(before + ql, (long long)cap);
    const int r1 = min(r0 + 16 * NR, min(rows, ql * a.G));   // valid rows of the block
    int kb0 = 0, kb1 = 0;                                    // blocks of 64 keys
    if (r0 < r1) {
        const int t0 = (int)fdiv((uint32_t)r0, a.divG), t1 = (int)fdiv((uint32_t)(r1 - 1), a.divG);
        const int hi = (int)min((long long)kl, before + t1 + 1);
        const int lo = a.window ? (int)min((long long)kl, max(0ll, before + t0 - a.window + 1)) : 0;
        if (lo < hi) {
            kb0 = lo / kStepKeys;
            kb1 = (hi + kStepKeys - 1) / kStepKeys;
            const int per = (kb1 - kb0 + a.nsplit - 1) / a.nsplit;
            kb0 = min(kb1, kb0 + split * per);
            kb1 = min(kb1, kb0 + per);
        }
    }

    CacheRows<T, D, NR> x;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int r = min(r0 + 16 * n + lr, rows - 1);
        const int t = (int)fdiv((uint32_t)r, a.divG), h = hk * a.G + (r - t * a.G);
        x.hi[n] = (int)min((long long)kl - 1, before + t);
        x.lo[n] = a.window ? (int)min((long long)kl, before + t - a.window + 1) : 0;
        // rows past the newest token are computed on a valid row and dropped
        const int tr = max(min(t, ql - 1), 0);
        x.load_query(n, reinterpret_cast<const T*>(a.q) + ((size_t)b * a.Tq + tr) * a.ldq + (size_t)h * D, g);
    }
    x.clear();
    const PagedKeys keys{a.k_cache, a.v_cache, a.k_scale, a.v_scale, a.block_table + (size_t)b * a.max_pages,
                         a.n_pages, a.page, a.HK, hk, kl, a.scale_log2};
    x.attend(keys, kb0 + wave, kb1, NW, lane);

    // join the waves, 16 rows at a time
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        if (r0 + 16 * n >= rows) break;
        const float sum = group_add4(x.l[n]);
        const float top = sum != sum ? -kNegInf : x.m[n];  // a NaN sum takes part whatever the other maxima are
        __syncthreads();
        if (g == 0) {
            sml[wave][lr][0] = top;
            sml[wave][lr][1] = sum;
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) *reinterpret_cast<floatx4*>(&so[wave][lr][16 * d + 4 * g]) = x.o[d][n];
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * D / 4; i += 64 * NW) {
            const int row = i / (D / 4), d = (i % (D / 4)) * 4, r = r0 + 16 * n + row;
            if (r >= rows) continue;
            float mm = kNegInf;
#pragma unroll
            for (int w = 0; w < NW; ++w) mm = fmaxf(mm, sml[w][row][0]);
            const float mu = mm == kNegInf ? 0.f : mm;
            float total = 0.f;
            floatx4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = exp2_fast(sml[w][row][0] - mu);
                if (f != 0.f) {
                    total = fmaf(f, sml[w][row][1], total);
                    y += f * *reinterpret_cast<const floatx4*>(&so[w][row][d]);
                }
            }
            const bool live = r < r1;
            if (a.nsplit > 1) {
                const size_t at = ((size_t)split * nbh + bh) * rows + r;
                *reinterpret_cast<floatx4*>(a.part_o + at * D + d) = y;
                if (d == 0)
                    *reinterpret_cast<float2*>(a.part_ml + 2 * at) = live ? make_float2(mm, total) : make_float2(kNegInf, 0.f);
            } else {
                const int t = (int)fdiv((uint32_t)r, a.divG), h = hk * a.G + (r - t * a.G);
                const float inv = 1.f / total;
                store4(reinterpret_cast<T*>(a.o) + (((size_t)b * a.Tq + t) * a.H + h) * D + d,
                       live && total != 0.f ? y * inv : floatx4{0.f, 0.f, 0.f, 0.f});
            }
        }
    }
}

template <typename T, int D, int NR>
static hipError_t launch_step_n(const AttnStepArgs& a, hipStream_t s) {
    const long long rows = (long long)a.Tq * a.G, blocks = (rows + 16 * NR - 1) / (16 * NR);
    hipLaunchKernelGGL((kda_attn_step_kernel<T, D, NR>), dim3((unsigned)(blocks * a.B * a.HK * a.nsplit)), dim3(64 * kStepWaves), 0, s, a);
    return hipGetLastError();
}
template <typename T, int D>
static hipError_t launch_step_t(const AttnStepArgs& a, hipStream_t s) {
    const hipError_t e = attn_step_row_blocks((long long)a.Tq * a.G) == 1 ? launch_step_n<T, D, 1>(a, s) : launch_step_n<T, D, 2>(a, s);
    if (e != hipSuccess || a.nsplit == 1) return e;
    const JoinArgs j{a.part_o, a.part_ml, a.o, nullptr, a.nsplit, a.B, a.Tq, a.H, a.HK, a.G, a.divG};
    return launch_attn_join(sizeof(T) == 2 ? 1 : 0, D, j, s);
}
template <typename T>
static hipError_t launch_step_d(int D, const AttnStepArgs& a, hipStream_t s) {
    switch (D) {
        case 16: return launch_step_t<T, 16>(a, s);
        case 32: return launch_step_t<T, 32>(a, s);
        case 64: return launch_step_t<T, 64>(a, s);
        case 128: return launch_step_t<T, 128>(a, s);
        default: return hipErrorInvalidValue;
    }
}
hipError_t launch_attn_step(int dt, int D, const AttnStepArgs& a, hipStream_t s) {
    return dt == 1 ? launch_step_d<bf16_t>(D, a, s) : launch_step_d<float>(D, a, s);
}

}  // namespace kda
