// kda_beam.hip - beam search on gfx950: the best continuations of a request's beams
// over the whole vocabulary, and states that follow their parents.
//
// Selection.  s(b, w) = score_b + x_bw - lse_b, lse_b = ln sum_w exp x_bw, and the M
// largest of a request, ties to the lowest (b, w).  Within a beam the order is that of
// the logits, whatever lse_b is, so one pass over the logits gives both: workgroups
// take parts of a row and leave the part's maximum, its sum of exponentials and its M
// first logits; one workgroup a request joins them in 64 bits.
#include "kda_attn_device.h"
#include "kda_branch.h"

namespace kda {

namespace {

constexpr int kSegments = 8;      // of a part: each thread keeps the maximum of what it read of each
constexpr int kJoinThreads = 512;
constexpr int kUnroll = 4;        // 16-byte loads of a thread in flight; a segment is a multiple of them
constexpr int kFound = 1024;      // candidates of a part that are ranked
// A thread's sum of exponentials is relative to a value that its logits exceed by no more than this: sums of rows that
// rise slowly are not multiplied by a rounded factor for every group of loads.
constexpr float kRefSlack = 4.f;

// e^d for differences |d| of a few units: off by 2^-23 of itself (the instruction) and 1.3 |d| 2^-24 (the rounding of
// d log2 e, and kLog2e's own).
__device__ __forceinline__ float exp_term(float d) { return exp2_fast(d * kLog2e); }

// Order of values as that of unsigned integers; -0 is +0.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t order_key(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __longlong_as_double((long long)(k & 0x8000000000000000ull ? k ^ 0x8000000000000000ull : ~k));
}

// A t such that at least `most` of a wave's 2 x 64 keys are >= t (0 if fewer are): the largest
// one of 20 bits, for a float sign, exponent and 11 bits, because each bit costs a round of
// scalar work that nothing hides.
__device__ __forceinline__ uint32_t threshold(uint32_t key0, uint32_t key1, int most) {
    uint32_t t = 0;
    for (int bit = 31; bit >= 12; --bit) {
        const uint32_t c = t | 1u << bit;
        if (__popcll(__ballot(key0 >= c)) + __popcll(__ballot(key1 >= c)) >= most) t = c;
    }
    return t;
}

// 16 bytes of a row whose elements are aligned as such only.
template <typename T> struct Vec {
    static constexpr int N = 16 / (int)sizeof(T);
    struct __attribute__((packed, aligned(sizeof(T)))) Raw { uint32_t w[4]; } raw;
    __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const Raw*>(p); }
    // elements [at, at + N) of n; those at or past n are -infinity
    __device__ __forceinline__ void load(const T* row, int at, int n) {
        if (at + N <= n) {
            load(row + at);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x = at + i < n ? to_f<T>(row[at + i]) : kNegInf;
                if (sizeof(T) == 4) raw.w[i % 4] = __float_as_uint(x);
                else raw.w[(i / 2) % 4] = i & 1 ? raw.w[(i / 2) % 4] | (__float_as_uint(x) & 0xffff0000u) : __float_as_uint(x) >> 16;
            }
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        return __uint_as_float(sizeof(T) == 4 ? raw.w[i % 4] : i & 1 ? raw.w[(i / 2) % 4] & 0xffff0000u : raw.w[(i / 2) % 4] << 16);
    }
};

__device__ __forceinline__ bool beam_lives(const SelectArgs& a, int row) {
    return !a.scores || (a.scores[row] - a.scores[row] == 0.f);   // finite
}

}  // namespace

// One part of one beam's row.  Each thread keeps the maximum and the sum of exponentials
// of what it reads, and the maxima of its segments.  The M-th largest of the maxima of
// pairs of threads bounds the M first from below; only segments that reach it are read again (a
// few of 2048, from the cache nearby) and what reaches it there, usually little more
// than M values, is ranked by counting.  Sums are relative to a maximum of the thread's own, in 64
// bits beyond a group of loads: errors of equal terms do not cancel (one large logit above 2^20 equal
// ones: up to 9e-6 off with fp32 sums and one factor for all threads' terms, 3e-7 at most now).
// Bound by reading the logits: 512 rows of 131072 bf16 (134 MB) from memory take 34 us, 3.9 TB/s over all (30
// where part of them is in the last-level cache) and 26 us at the rate of a copy; the rest is the start and
// the selection, which all parts do at the same time.  An exponential with its argument's rounding carried along
// costs twice the instructions of one difference (41 us when the kernel took 34 like now), groups of eight loads
// a register too many for four workgroups a CU (48 us).  4 rows of 32000 fp32: 6.7 us.
template <typename T>
__global__ __launch_bounds__(kSelThreads) void kda_select_part_kernel(const SelectArgs a) {
    constexpr int N = Vec<T>::N, STEP = kSelThreads * N;
    __shared__ float seg[kSegments][kSelThreads];
    __shared__ float top[kSelThreads];
    __shared__ uint64_t found[kFound];
    __shared__ uint16_t todo[kSegments * kSelThreads];
    __shared__ double sums[kSelThreads / 64];
    __shared__ int counts[kSelThreads / 64], n_todo, n_found, n_above;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int row = blockIdx.x / a.nsplit, split = blockIdx.x % a.nsplit;
    const int per = select_part(a.V, a.nsplit, N), lo = min((long long)split * per, (long long)a.V), n = min(per, a.V - lo);
    const T* x = reinterpret_cast<const T*>(a.logits) + (size_t)row * a.ld + lo;
    // loads of a segment, groups of loads
    const int loads = (n + STEP - 1) / STEP, per_seg = max(1, (loads + kSegments * kUnroll - 1) / (kSegments * kUnroll)) * kUnroll;
    const int groups = (loads + kUnroll - 1) / kUnroll;
    const bool skip = (a.done && a.done[row]) || !beam_lives(a, row);

    // A group is loaded while the one before is summed.  Behind the last whole 16 bytes a
    // thread takes the row's last ones instead and drops those that are not its own.
    float m = kNegInf, ref = kNegInf, best = kNegInf;
    double l = 0.0;                 // sum of e^(x - ref)
    auto fetch = [&](Vec<T> (&v)[kUnroll], int g) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int at = ((g * kUnroll + u) * kSelThreads + tid) * N;
            if (n >= N) v[u].load(x + min(at, n - N));
            else v[u].load(x, at, n);
        }
    };
    auto reduce = [&](const Vec<T> (&v)[kUnroll], int g) {
        const bool whole = (g + 1) * kUnroll * STEP <= n || n < N;
        auto value = [&](int u, int e) {
            const int at = ((g * kUnroll + u) * kSelThreads + tid) * N;
            return whole || min(at, n - N) + e >= at ? v[u][e] : kNegInf;
        };
        auto both = [&](auto value) {
            float y[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                for (int e = 0; e < N; ++e) y[e % 4] = fmaxf(y[e % 4], value(u, e));
            const float z = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
            best = fmaxf(best, z);
            m = fmaxf(m, z);
            if (z > ref + kRefSlack) {
                l *= (double)exp_term(ref - z);
                ref = z;
            }
            const float mu = ref == kNegInf ? 0.f : ref;
            // pairs, pairs of pairs and so on: at most five roundings meet a term
            float part[kUnroll * N];
#pragma unroll
            for (int i = 0; i < kUnroll * N; ++i) part[i] = exp_term(value(i / N, i % N) - mu);
#pragma unroll
            for (int w = 1; w < kUnroll * N; w *= 2)
#pragma unroll
                for (int i = 0; i < kUnroll * N; i += 2 * w) part[i] += part[i + w];
            l += (double)part[0];
        };
        if (whole) both([&](int u, int e) { return v[u][e]; });
        else both(value);
        if ((g + 1) * kUnroll % per_seg == 0 || g + 1 == groups) {
            seg[g * kUnroll / per_seg][tid] = best;
            best = kNegInf;
        }
    };
    Vec<T> v0[kUnroll], v1[kUnroll];
    fetch(v0, 0);
    if (skip) return;    // the join does not ask for it
    for (int g = 0; g < groups; g += 2) {
        if (g + 1 < groups) fetch(v1, g + 1);
        reduce(v0, g);
        if (g + 1 < groups) {
            if (g + 2 < groups) fetch(v0, g + 2);
            reduce(v1, g + 1);
        }
    }
    const int segments = (groups * kUnroll + per_seg - 1) / per_seg;
    top[tid] = m;
    if (tid == 0) n_todo = n_found = n_above = 0;
    __syncthreads();

    // maxima of pairs of threads
    const float top0 = fmaxf(top[lane], top[lane + 64]), top1 = fmaxf(top[lane + 128], top[lane + 192]);
    float all = fmaxf(top0, top1);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor(all, o, 64));
    double sum = l == 0.0 ? 0.0 : l * exp((double)ref - (double)all);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (lane == 0) sums[wave] = sum;
    // candidates reach t; -infinity is none
    uint32_t t = max(threshold(order_key(top0), order_key(top1), a.M), order_key(kNegInf) + 1);

    auto collect = [&](uint32_t least, int* counter) {   // of the segments in `todo`
        for (int i = tid; i < n_todo * per_seg; i += kSelThreads) {
            const int which = todo[i / per_seg], at = ((which / kSelThreads * per_seg + i % per_seg) * kSelThreads + which % kSelThreads) * N;
            if (at >= n) continue;
            Vec<T> v;
            v.load(x, at, n);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const uint32_t k = order_key(v[e]);
                if (k < least || v[e] != v[e]) continue;
                const int p = atomicAdd(counter, 1);
                if (p < kFound) found[p] = (uint64_t)k << 32 | (uint32_t)~(uint32_t)(at + e);
            }
        }
    };
    for (int s = 0; s < segments; ++s)
        if (order_key(seg[s][tid]) >= t) todo[atomicAdd(&n_todo, 1)] = (uint16_t)(s * kSelThreads + tid);
    __syncthreads();
    collect(t, &n_found);
    __syncthreads();
    int held = n_found;
    if (held > kFound) {
        // many reach t: equal values (rows masked with one value), or rising ones.  What is
        // above t, and then the first that are equal to it in the order of the row.
        collect(t + 1, &n_above);
        __syncthreads();
        held = n_above;
        if (held > kFound) {
            // more than can be ranked: t becomes the M-th largest value of the part itself
            uint32_t exact = 0;
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t c = exact | 1u << bit;
                int mine = 0;
                for (int i = tid; i < n_todo * per_seg; i += kSelThreads) {
                    const int which = todo[i / per_seg], at = ((which / kSelThreads * per_seg + i % per_seg) * kSelThreads + which % kSelThreads) * N;
                    if (at >= n) continue;
                    Vec<T> v;
                    v.load(x, at, n);
#pragma unroll
                    for (int e = 0; e < N; ++e) mine += v[e] == v[e] && order_key(v[e]) >= c ? 1 : 0;
                }
#pragma unroll
                for (int o = 32; o > 0; o >>= 1) mine += __shfl_xor(mine, o, 64);
                __syncthreads();
                if (lane == 0) counts[wave] = mine;
                __syncthreads();
                int total = 0;
                for (int w = 0; w < kSelThreads / 64; ++w) total += counts[w];
                if (total >= a.M) exact = c;
            }
            t = exact;
            __syncthreads();
            if (tid == 0) n_above = 0;
            __syncthreads();
            collect(t + 1, &n_above);     // fewer than M
            __syncthreads();
            held = n_above;
        }
        for (int at0 = 0; at0 < n && held < a.M; at0 += STEP) {
            Vec<T> v;
            const int at = at0 + tid * N;
            int mine = 0;
            if (at < n) {
                v.load(x, at, n);
#pragma unroll
                for (int e = 0; e < N; ++e) mine += order_key(v[e]) == t ? 1 : 0;
            }
            int y = mine;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int z = __shfl_up(y, o, 64);
                if (lane >= o) y += z;
            }
            __syncthreads();
            if (lane == 63) counts[wave] = y;
            __syncthreads();
            int before = held, total = 0;
            for (int w = 0; w < kSelThreads / 64; ++w) {
                before += w < wave ? counts[w] : 0;
                total += counts[w];
            }
            before += y - mine;
            if (mine > 0) {
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (order_key(v[e]) == t) {
                        if (before < a.M) found[before] = (uint64_t)t << 32 | (uint32_t)~(uint32_t)(at + e);
                        ++before;
                    }
            }
            held = min(held + total, max(a.M, held));
        }
        __syncthreads();
    }

    const size_t part = blockIdx.x;
    for (int i = tid; i < held; i += kSelThreads) {
        const uint64_t k = found[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < held; ++j) rank += found[j] > k ? 1 : 0;
        if (rank < a.M) {
            a.part_x[part * a.M + rank] = key_value((uint32_t)(k >> 32));
            a.part_w[part * a.M + rank] = lo + (int)~(uint32_t)k;
        }
    }
    for (int i = held + tid; i < a.M; i += kSelThreads) a.part_w[part * a.M + i] = -1;
    if (tid == 0) {
        double total = 0.0;
        for (int w = 0; w < kSelThreads / 64; ++w) total += sums[w];
        a.stat[2 * part] = all;
        a.stat[2 * part + 1] = total;
    }
}

// One workgroup a request: each beam's lse from its parts, then its parts' candidates
// as scores in 64 bits, thinned by the M-th largest of the maxima of 128 sets (of the
// upper halves of their keys) and ranked by counting.  A wave has a beam: what a beam
// that lives no longer, or one at its end, has in the parts is whatever was there before.
// Bound by waits one after the other: 64 requests of 8 beams, 2 parts and 16 candidates
// take 5 us, 64 beams of 64 candidates 17.  Sets by thread were sets by rank, of which
// a few held all the best: a thousand candidates to rank instead of a hundred.
__global__ __launch_bounds__(kJoinThreads) void kda_select_join_kernel(const SelectArgs a) {
    __shared__ uint64_t key[kSelectHeld];
    __shared__ uint32_t token[kSelectHeld], logit[kSelectHeld];         // logit: the largest first
    // Order of equal scores: beam, then logit (a score rounds away what logits near zero differ by), then
    // candidate, which is by token where logits are equal: 6, 32 and 12 bits.
    __shared__ uint64_t list_key[kSelectHeld], list_id[kSelectHeld];
    static_assert(kSelectHeld == 1 << 12 && kSelectMost == 1 << 6, "bits of list_id");
    __shared__ uint32_t top[128];
    __shared__ int n_list;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = blockIdx.x;
    const int per = a.nsplit * a.M;
    if (tid == 0) n_list = 0;
    if (tid < 128) top[tid] = 0;
    __syncthreads();
    for (int k = wave; k < a.K; k += kJoinThreads / 64) {
        const int row = r * a.K + k;
        const size_t part = (size_t)row * a.nsplit;
        // independent of each other: one wait for all
        const bool mine = lane < a.nsplit;
        const double m0 = mine ? a.stat[2 * (part + lane)] : 0.0, l0 = mine ? a.stat[2 * (part + lane) + 1] : 0.0;
        const float score0 = a.scores ? a.scores[row] : 0.f;
        const bool done = a.done && a.done[row], lives = score0 - score0 == 0.f;
        int w0 = -1;
        float x0 = 0.f;
        if (lane < per) {
            w0 = a.part_w[part * a.M + lane];
            x0 = a.part_x[part * a.M + lane];
        }
        double lse = 0.0;
        if (lives && !done) {
            const float m = mine ? (float)m0 : kNegInf;
            float all = m;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor(all, o, 64));
            double sum = !mine || l0 == 0.0 ? 0.0 : l0 * exp((double)m - (double)all);
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
            lse = (double)all + log(sum);
        }
        for (int i = lane; i < per; i += 64) {
            uint64_t y = 0;
            uint32_t w = 0, x = 0;
            if (lives) {
                double s = -__builtin_inf();
                if (done) {
                    if (i == 0) {
                        s = (double)score0;
                        w = (uint32_t)a.end;
                    }
                } else {
                    const int next = i < 64 ? w0 : a.part_w[part * a.M + i];
                    if (next >= 0) {
                        const float value = i < 64 ? x0 : a.part_x[part * a.M + i];
                        s = (double)score0 + ((double)value - lse);
                        w = (uint32_t)next;
                        x = ~order_key(value);
                    }
                }
                const float rounded = (float)s;
                if (rounded - rounded == 0.f) y = order_key(s);   // what is not finite in fp32 is no continuation
            }
            key[k * per + i] = y;
            token[k * per + i] = w;
            logit[k * per + i] = x;
            // one of 128 sets, not by the rank in the part
            if (y) atomicMax(&top[((uint32_t)(k * per + i) * 0x9e3779b1u) >> 25], (uint32_t)(y >> 32));
        }
    }
    const int held = a.K * per;
    __syncthreads();
    const uint32_t t = max(threshold(top[lane], top[lane + 64], a.M), 1u);   // the key of no finite number is below 2^32
    for (int i = tid; i < held; i += kJoinThreads)
        if ((uint32_t)(key[i] >> 32) >= t) {
            const int p = atomicAdd(&n_list, 1);
            list_key[p] = key[i];
            list_id[p] = (uint64_t)(i / per) << 44 | (uint64_t)logit[i] << 12 | (uint32_t)i;
        }
    __syncthreads();
    const int n = n_list;
    for (int i = tid; i < n; i += kJoinThreads) {
        const uint64_t y = list_key[i], w = list_id[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) rank += (int)(list_key[j] > y) | ((int)(list_key[j] == y) & (int)(list_id[j] < w));
        if (rank < a.M) {
            const size_t at = (size_t)r * a.M + rank;
            a.scores_out[at] = (float)key_value(y);
            a.parent[at] = (int)(w >> 44);
            a.token[at] = (int)token[w & (kSelectHeld - 1)];
        }
    }
    for (int i = n + tid; i < a.M; i += kJoinThreads) {
        const size_t at = (size_t)r * a.M + i;
        a.scores_out[at] = kNegInf;
        a.parent[at] = a.token[at] = -1;
    }
}

template <typename T> static hipError_t launch_select_t(const SelectArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((kda_select_part_kernel<T>), dim3((unsigned)a.R * a.K * a.nsplit), dim3(kSelThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kda_select_join_kernel, dim3((unsigned)a.R), dim3(kJoinThreads), 0, s, a);
    return hipGetLastError();
}
hipError_t launch_beam_select(int dt, const SelectArgs& a, hipStream_t s) {
    return dt == 1 ? launch_select_t<bf16_t>(a, s) : launch_select_t<float>(a, s);
}

// ---------------------------------------------------------------- states

// Rows are not read again soon: they leave the caches at once.
template <typename P> __device__ __forceinline__ void store_once(void* p, const P& x) {
    typedef uint32_t Words __attribute__((ext_vector_type(sizeof(P) / 4)));
    __builtin_nontemporal_store(__builtin_bit_cast(Words, x), reinterpret_cast<Words*>(p));
}

// In place: a thread has the same 16 bytes of every row of a request, reads what
// moves and then writes it, so nothing is lost whatever the parents are, and rows that
// stay are not touched.  Bound by memory: 256 rows of 1 MB of which half move (about 240 MB)
// take 42 us, 5.8 TB/s (ordinary stores 44); 16 rows of 512 KB in 16 requests 21 (28); 64 in
// each of 4 requests reach 3.7 TB/s (3.2): their registers leave room for few waves.
template <int KM, typename P>
__global__ __launch_bounds__(256) void kda_reorder_kernel(const ReorderArgs a, unsigned blocks) {
    const unsigned r = blockIdx.x / blocks;
    const unsigned long long at = ((unsigned long long)(blockIdx.x % blocks) * 256 + threadIdx.x) * sizeof(P);
    if (at >= a.row_bytes) return;
    const int* parent = a.parent + (size_t)r * a.K_out;
    uint8_t* base = a.out + (size_t)r * a.K_out * a.row_bytes + at;
    P v[KM];
#pragma unroll
    for (int k = 0; k < KM; ++k) {
        v[k] = P{};
        if (k < a.K_out) {
            const int p = parent[k];
            if (p != k && p >= 0 && p < a.K_in) v[k] = *reinterpret_cast<const P*>(base + (size_t)p * a.row_bytes);
        }
    }
#pragma unroll
    for (int k = 0; k < KM; ++k)
        if (k < a.K_out && parent[k] != k) store_once(base + (size_t)k * a.row_bytes, v[k]);
}

// Into other memory: four 16-byte pieces a thread.  256 rows of 1 MB: 81 us (ordinary stores 87).
__global__ __launch_bounds__(256) void kda_gather_kernel(const ReorderArgs a, unsigned blocks) {
    const unsigned row = blockIdx.x / blocks, r = row / a.K_out;
    const unsigned long long first = (unsigned long long)(blockIdx.x % blocks) * 16384 + threadIdx.x * 16;
    const int p = a.parent[row];
    const bool child = p >= 0 && p < a.K_in;
    const uint8_t* from = a.state + ((size_t)r * a.K_in + (child ? p : 0)) * a.row_bytes;
    uint8_t* to = a.out + (size_t)row * a.row_bytes;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (child && first + i * 4096 < a.row_bytes) v[i] = *reinterpret_cast<const uint4*>(from + first + i * 4096);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (first + i * 4096 < a.row_bytes) store_once(to + first + i * 4096, v[i]);
}

template <int KM, typename P> static hipError_t launch_reorder_n(const ReorderArgs& a, hipStream_t s) {
    const unsigned blocks = (unsigned)((a.row_bytes / sizeof(P) + 255) / 256);
    hipLaunchKernelGGL((kda_reorder_kernel<KM, P>), dim3((unsigned)a.R * blocks), dim3(256), 0, s, a, blocks);
    return hipGetLastError();
}
hipError_t launch_state_reorder(const ReorderArgs& a, hipStream_t s) {
    if (a.out == a.state)
        return a.K_out <= 4   ? launch_reorder_n<4, uint4>(a, s)
               : a.K_out <= 8 ? launch_reorder_n<8, uint4>(a, s)
               : a.K_out <= 16 ? launch_reorder_n<16, uint4>(a, s)
               : a.K_out <= 32 ? launch_reorder_n<32, uint4>(a, s)
                               : launch_reorder_n<kReorderMost, uint2>(a, s);
    const unsigned blocks = (unsigned)((a.row_bytes + 16383) / 16384);
    hipLaunchKernelGGL(kda_gather_kernel, dim3((unsigned)a.R * a.K_out * blocks), dim3(256), 0, s, a, blocks);
    return hipGetLastError();
}

}  // namespace kda
