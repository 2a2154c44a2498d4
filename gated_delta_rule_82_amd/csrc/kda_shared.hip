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

// The group of sequence b, -1: none.  A wave looks at 64 groups at a time.
__device__ __forceinline__ int group_of(const AttnSharedArgs& a, int b, int lane) {
    for (int g0 = 0; g0 < a.n_groups; g0 += 64) {
        bool here = false;
        if (g0 + lane < a.n_groups) {
            const Group x = group_at(a, g0 + lane);
            here = x.first <= b && b < x.last;
        }
        const uint64_t who = __ballot(here);
        if (who) return g0 + __ffsll((unsigned long long)who) - 1;
    }
    return -1;
}

// The group and tile of its rows that are number `tile` of all groups' tiles.
__device__ __forceinline__ int group_of_tile(const AttnSharedArgs& a, int& tile, int rows_per_tile, int lane) {
    for (int g0 = 0; g0 < a.n_groups; g0 += 64) {
        int n = 0;
        if (g0 + lane < a.n_groups) {
            const Group x = group_at(a, g0 + lane);
            n = (int)(((long long)(x.last - x.first) * a.Tq * a.G + rows_per_tile - 1) / rows_per_tile);
        }
        int y = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int z = __shfl_up(y, o, 64);
            if (lane >= o) y += z;
        }
        const uint64_t who = __ballot(tile < y);
        if (who) {
            const int i = __ffsll((unsigned long long)who) - 1;
            tile -= __shfl(y, i, 64) - __shfl(n, i, 64);
            return g0 + i;
        }
        tile -= __shfl(y, 63, 64);
    }
    return -1;
}

}  // namespace

// Bound by the bytes: see launch_attn_shared.
template <typename T, int D, int NR>
__global__ __launch_bounds__(64 * kSharedWaves) void kda_attn_shared_kernel(const AttnSharedArgs a) {
    constexpr int ND = D / 16, NW = kSharedWaves;
    __shared__ __attribute__((aligned(16))) float so[NW][16][D + 4];
    __shared__ float sml[NW][16][2];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, lr = lane & 15;
    const int each = a.Tq * a.G;                        // rows of a sequence
    const size_t all_rows = (size_t)a.B * a.HK * each;
    int bid = blockIdx.x;
    const bool common = bid < a.prefix_blocks;
    int first, prefix, r0, rows, part, parts, hk;       // rows: of the group or sequence
    if (common) {
        hk = bid % a.HK;
        bid /= a.HK;
        int tile = bid % a.tiles;
        part = bid / a.tiles;
        parts = a.nprefix;
        const int gi = group_of_tile(a, tile, 16 * NR, lane);
        if (gi < 0) return;
        const Group x = group_at(a, gi);
        first = x.first;
        prefix = x.prefix;
        rows = (x.last - x.first) * each;
        r0 = tile * 16 * NR;
    } else {
        bid -= a.prefix_blocks;
        const int nbh = a.B * a.HK, bh = bid % nbh;
        bid /= nbh;
        hk = bh % a.HK;
        first = bh / a.HK;
        part = bid % a.nown;
        parts = a.nown;
        rows = each;
        r0 = bid / a.nown * 16 * NR;
        const int gi = group_of(a, first, lane);
        prefix = gi < 0 ? 0 : group_at(a, gi).prefix;
        if (gi < 0 && part == 0)                        // no group's tile has its rows
            for (int i = threadIdx.x; i < a.nprefix * min(16 * NR, rows - r0); i += 64 * NW) {
                const size_t at = (size_t)(i % a.nprefix) * all_rows + (size_t)bh * each + r0 + i / a.nprefix;
                *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(kNegInf, 0.f);
            }
    }
    const int cap = a.max_pages * a.page, r1 = min(r0 + 16 * NR, rows);
    const int out_part = common ? part : a.nprefix + part;

    // keys that some row sees: of the group's prefix, or behind it
    CacheRows<T, D, NR> x;
    int lo = cap, hi = 0;               // [lo, hi)
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int r = min(r0 + 16 * n + lr, rows - 1);
        const int tau = (int)fdiv((uint32_t)r, a.divG), s = tau / a.Tq, t = tau - s * a.Tq, b = first + s, h = hk * a.G + (r - tau * a.G);
        const int ql = seq_len(a.new_len, b, a.Tq);
        const long long before = max(a.cache_len[b], 0), at = before + t;
        const int kl = (int)min(before + ql, (long long)cap);
        const int from = a.window ? (int)min((long long)cap, max(at - a.window + 1, 0ll)) : 0;
        const int to = (int)min(at, (long long)kl - 1);
        x.lo[n] = common ? from : max(from, prefix);
        x.hi[n] = t < ql ? (common ? min(to, prefix - 1) : to) : -1;
        if (x.hi[n] >= x.lo[n]) {
            lo = min(lo, x.lo[n]);
            hi = max(hi, x.hi[n] + 1);
        }
        // rows past the newest token are computed on a valid row and dropped
        const int tr = max(min(t, ql - 1), 0);
        x.load_query(n, reinterpret_cast<const T*>(a.q) + ((size_t)b * a.Tq + tr) * a.ldq + (size_t)h * D, g);
    }
    x.clear();
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor(lo, o, 64));
        hi = max(hi, __shfl_xor(hi, o, 64));
    }
    if (lo < hi) {
        int kb0 = lo / kStepKeys, kb1 = (hi + kStepKeys - 1) / kStepKeys;
        const int per = (kb1 - kb0 + parts - 1) / parts;
        kb0 = min(kb1, kb0 + part * per);
        kb1 = min(kb1, kb0 + per);
        // nothing at or past hi is read: for a group it is the first sequence's own
        const PagedKeys keys{a.k_cache, a.v_cache, a.k_scale, a.v_scale, a.block_table + (size_t)first * a.max_pages,
                             a.n_pages, a.page, a.HK, hk, hi, a.scale_log2};
        for (int kb = kb0 + wave; kb < kb1; kb += NW) x.attend(keys, kb, lane);
    }

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
            if (r >= r1) continue;
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
            const int s = r / each, b = first + s;
            const size_t at = (size_t)out_part * all_rows + ((size_t)b * a.HK + hk) * each + (r - s * each);
            *reinterpret_cast<floatx4*>(a.part_o + at * D + d) = y;
            if (d == 0) {
                const bool live = (int)fdiv((uint32_t)(r - s * each), a.divG) < seq_len(a.new_len, b, a.Tq);
                *reinterpret_cast<float2*>(a.part_ml + 2 * at) = live ? make_float2(mm, total) : make_float2(kNegInf, 0.f);
            }
        }
    }
}

template <typename T, int D, int NR>
static hipError_t launch_shared_n(const AttnSharedArgs& a, hipStream_t s) {
    const long long own = (long long)a.B * a.HK * a.nown * (((long long)a.Tq * a.G + 16 * NR - 1) / (16 * NR));
    hipLaunchKernelGGL((kda_attn_shared_kernel<T, D, NR>), dim3((unsigned)(a.prefix_blocks + own)), dim3(64 * kSharedWaves), 0, s, a);
    return hipGetLastError();
}
template <typename T, int D>
static hipError_t launch_shared_t(const AttnSharedArgs& a, hipStream_t s) {
    const hipError_t e = a.row_blocks == 1 ? launch_shared_n<T, D, 1>(a, s) : launch_shared_n<T, D, 2>(a, s);
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
