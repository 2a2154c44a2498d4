// kda_pages.hip - pages of the 8-bit cache on gfx950: sharing them between sequences,
// handing them out, taking them back, moving them to the front, copying them.
//
// Tables and references are a few thousand to a few hundred thousand ints: these
// kernels are bound by the latency of a handful of dependent loads, and everything is
// decided on the device in one launch each so that a decode loop needs no host in
// between and can be captured.  What a choice depends on (which free page, who keeps a
// shared one) follows the order of (sequence, page), never the order of threads:
// results do not vary from run to run.  Only the copies move data; they are apart from
// the bookkeeping because a stack has one set of tables and a cache in every layer.
#include "kda_branch.h"
#include "kda_device.h"

namespace kda {

namespace {

__device__ __forceinline__ int len_of(const int* len, int b) { return max(len[b], 0); }
__device__ __forceinline__ int fresh_of(const int* len, int b, int most) { return len ? min(max(len[b], 0), most) : most; }

// References are changed by atomics, which are performed behind the first-level cache:
// they are read there too.
__device__ __forceinline__ int load_refs(const int* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void store_refs(int* p, int x) { __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

constexpr int kBookThreads = 1024, kBookWaves = kBookThreads / 64;

// Sum of x over the threads before this one; `total` is that of all.  Two barriers.
__device__ __forceinline__ int prefix_sum(int x, int* waves, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int y = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int z = __shfl_up(y, o, 64);
        if (lane >= o) y += z;
    }
    if (lane == 63) waves[wave] = y;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kBookWaves; ++w) {
        const int t = waves[w];
        before += w < wave ? t : 0;
        total += t;
    }
    __syncthreads();
    return before + y - x;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store_once(void* p, const uint4& x) {
    __builtin_nontemporal_store(u32x4{x.x, x.y, x.z, x.w}, reinterpret_cast<u32x4*>(p));
}

// Four references from index i (a multiple of 4); those past the end count as in use.
__device__ __forceinline__ int4 four_refs(const int* refs, int i, int n) {
    if (i + 4 <= n) return *reinterpret_cast<const int4*>(refs + i);
    return make_int4(i < n ? refs[i] : 1, i + 1 < n ? refs[i + 1] : 1, i + 2 < n ? refs[i + 2] : 1, 1);
}

}  // namespace

// Threads for the entries of the old rows (references) and then of the new ones.
__global__ __launch_bounds__(256) void kda_cache_fork_kernel(const ForkArgs a, unsigned n_in, unsigned n_out, unsigned width) {
    unsigned i = blockIdx.x * 256u + threadIdx.x;
    if (i < n_in) {
        const int row = (int)(i / width), j = (int)(i % width), r = row / a.K_in, k = row % a.K_in;
        if (j >= a.max_pages) return;
        const int e = a.table[(size_t)row * a.max_pages + j];
        if (e < 0 || e >= a.n_pages) return;
        int delta = a.keep ? 0 : -1;
        if ((long long)j * a.page < len_of(a.cache_len, row))
            for (int c = 0; c < a.K_out; ++c) delta += a.parent[(size_t)r * a.K_out + c] == k;
        if (delta != 0) atomicAdd(a.refs + e, delta);
        return;
    }
    i -= n_in;
    if (i >= n_out) return;
    const int row = (int)(i / width), j = (int)(i % width), r = row / a.K_out;
    const int k = a.parent[row];
    const bool child = k >= 0 && k < a.K_in;
    const int from = r * a.K_in + (child ? k : 0), len = child ? len_of(a.cache_len, from) : 0;
    if (j == 0) a.len_out[row] = len;
    if (j < a.max_pages)
        a.table_out[(size_t)row * a.max_pages + j] = (long long)j * a.page < len ? a.table[(size_t)from * a.max_pages + j] : -1;
}

hipError_t launch_cache_fork(const ForkArgs& a, hipStream_t s) {
    const unsigned width = a.max_pages > 0 ? a.max_pages : 1;
    const unsigned n_in = a.max_pages > 0 ? (unsigned)a.R * a.K_in * width : 0, n_out = (unsigned)a.R * a.K_out * width;
    hipLaunchKernelGGL(kda_cache_fork_kernel, dim3((n_in + n_out + 255) / 256), dim3(256), 0, s, a, n_in, n_out, width);
    return hipGetLastError();
}

__global__ __launch_bounds__(256) void kda_cache_free_kernel(const FreeArgs a, unsigned n) {
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    if (i >= n) return;
    const int b = (int)(i / a.max_pages);
    const long long first = (long long)(i % a.max_pages) * a.page, last = first + a.page;
    const int e = a.table[i];
    const long long from = a.keep_from ? a.keep_from[b] : 0, to = a.keep_to ? a.keep_to[b] : 0;
    if (first < to && last > from && to > from) return;    // holds a token that is kept
    a.table[i] = -1;
    if (e >= 0 && e < a.n_pages) atomicAdd(a.refs + e, -1);
}

hipError_t launch_cache_free(const FreeArgs& a, hipStream_t s) {
    const unsigned n = (unsigned)a.B * a.max_pages;
    hipLaunchKernelGGL(kda_cache_free_kernel, dim3((n + 255) / 256), dim3(256), 0, s, a, n);
    return hipGetLastError();
}

// One workgroup.  Touched entries are taken 1024 at a time in order: which of them
// need a page, how many before them do (a prefix sum), and which holders of a shared
// page leave it (all but the last where nobody else holds it: holder k of those in
// order leaves while refs - k > 1).  Free pages come in order from a walk over the
// references, as many as are needed, through a ring in LDS.  Bound by loads that wait for
// each other (lengths, entries, references) and barriers: 4 sequences take 5 us; 256 of
// one new token that all leave a shared page take 11, of which finding their order among
// 256 holders is 4 (one compared at a time 6).
__global__ __launch_bounds__(kBookThreads) void kda_cache_reserve_kernel(const ReserveArgs a) {
    constexpr int RING = 8192, STEP = 4 * kBookThreads;   // a step adds up to 4096 to fewer than 1024 left
    __shared__ int ring[RING];
    __shared__ __align__(16) int claims[kBookThreads];   // whole groups of 16
    __shared__ int waves[kBookWaves];
    const int tid = threadIdx.x;
    const unsigned items = (unsigned)a.B * a.touched;
    const int page_log2 = 31 - __clz(a.page);
    int cursor = 0, lacking = 0;         // the same in every thread
    // What the next step of the walk reads, ahead of it: no page becomes free here, and those
    // handed out lie before the walk.
    int4 ahead = four_refs(a.refs, 4 * tid, a.n_pages);
    unsigned head = 0, tail = 0;
    for (unsigned base = 0; base < items; base += kBookThreads) {
        const unsigned item = base + tid;
        const int b = (int)(item / a.touched), jj = (int)(item % a.touched);
        bool need = false, claim = false, older = false;
        int e = -1, held = 0;
        size_t at = 0;
        if (item < items) {
            const long long before = len_of(a.cache_len, b), fresh = fresh_of(a.new_len, b, a.T), j = (before >> page_log2) + jj;
            if (fresh > 0 && j < a.max_pages && j << page_log2 < before + fresh) {
                at = (size_t)b * a.max_pages + j;
                e = a.table[at];
                older = jj == 0 && (before & (a.page - 1)) != 0;
                const bool has = e >= 0 && e < a.n_pages;
                if (has) held = load_refs(a.refs + e);
                claim = has && held > 1;
                need = !has && !older;
            }
        }
        int n_claims;
        const int rank = prefix_sum(claim ? 1 : 0, waves, n_claims);
        if (n_claims > 0) {
            if (claim) claims[rank] = e;
            __syncthreads();
            if (claim) {
                int k = 0;
                for (int i = 0; i < rank; i += 16) {
                    int4 c[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) c[u] = *reinterpret_cast<const int4*>(claims + i + 4 * u);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int left = rank - i - 4 * u;
                        k += (int)(left > 0 & c[u].x == e) + (int)(left > 1 & c[u].y == e) + (int)(left > 2 & c[u].z == e) +
                             (int)(left > 3 & c[u].w == e);
                    }
                }
                claim = held - k > 1;
                need = claim;
            }
        }
        int wanted;
        const int order = prefix_sum(need ? 1 : 0, waves, wanted);
        while ((int)(tail - head) < wanted && cursor < a.n_pages) {
            const int p = cursor + 4 * tid;
            const int4 r = ahead;
            ahead = four_refs(a.refs, p + STEP, a.n_pages);
            int found;
            unsigned to = tail + prefix_sum((r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0), waves, found);
            if (r.x == 0) ring[to++ % RING] = p;
            if (r.y == 0) ring[to++ % RING] = p + 1;
            if (r.z == 0) ring[to++ % RING] = p + 2;
            if (r.w == 0) ring[to++ % RING] = p + 3;
            tail += found;
            cursor = a.n_pages - cursor > STEP ? cursor + STEP : a.n_pages;
        }
        __syncthreads();
        const int have = min((int)(tail - head), wanted);
        int page = -1;
        if (need) {
            if (order < have) page = ring[(head + order) % RING];
            a.table[at] = page;
            if (page >= 0) store_refs(a.refs + page, 1);
            if (claim) atomicAdd(a.refs + e, -1);
        }
        if (item < items && jj == 0) {
            const bool copied = claim && older && page >= 0;
            a.src[b] = copied ? e : -1;
            a.dst[b] = copied ? page : -1;
        }
        head += have;
        lacking += wanted - have;
        if (items - base > kBookThreads) {
            // the next entries read these references: all are at the second-level cache then (a
            // fence for other workgroups too would write all of it back, 4 us)
            wait_vmcnt<0>();
            __syncthreads();
        }
    }
    // free pages left: those in the ring and those behind the walk
    int left = (ahead.x == 0) + (ahead.y == 0) + (ahead.z == 0) + (ahead.w == 0);
    for (int p = cursor + 4 * tid; p < a.n_pages - STEP; ) {
        p += STEP;
        const int4 r = four_refs(a.refs, p, a.n_pages);
        left += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    }
    int total;
    prefix_sum(left, waves, total);
    if (tid == 0) {
        a.info[0] = lacking;
        a.info[1] = total + (int)(tail - head);
    }
}

hipError_t launch_cache_reserve(const ReserveArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(kda_cache_reserve_kernel, dim3(1), dim3(kBookThreads), 0, s, a);
    return hipGetLastError();
}

// One workgroup, two walks over the references in order: how many pages are in use
// (U), then the free pages below U and the used ones from U on, as many of each, which
// are paired in order.  All free pages below U come before the first mover.
__global__ __launch_bounds__(kBookThreads) void kda_cache_compact_kernel(const CompactArgs a) {
    constexpr int STEP = 4 * kBookThreads;
    __shared__ int waves[kBookWaves];
    const int tid = threadIdx.x, n = a.n_pages;
    int mine = 0, used;
    for (int p = 4 * tid; p < n; p += STEP) {
        const int4 r = four_refs(a.refs, p, n);
        mine += (r.x != 0) + (r.y != 0) + (r.z != 0) + (r.w != 0) - (p + 4 > n ? p + 4 - n : 0);
    }
    prefix_sum(mine, waves, used);
    int holes = 0, movers = 0;          // before this step
    for (int base = 0; base < n; base += STEP) {
        const int p = base + 4 * tid;
        int r[4] = {0, 0, 0, 0};
        if (p < n) {
            const int4 q = four_refs(a.refs, p, n);
            r[0] = q.x; r[1] = q.y; r[2] = q.z; r[3] = q.w;
        }
        int count = 0, total;           // holes in the lower, movers in the upper half
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (p + i < n) count += r[i] == 0 ? (p + i < used ? 1 : 0) : (p + i >= used ? 1 << 16 : 0);
        const int before = prefix_sum(count, waves, total);
        int h = holes + (before & 0xffff), m = movers + (before >> 16), m0 = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (p + i >= n) continue;
            if (r[i] == 0) {
                a.remap[p + i] = -1;
                if (p + i < used) a.dst[h++] = p + i;
                else a.refs_out[p + i] = 0;
            } else if (p + i < used) {
                a.remap[p + i] = p + i;
                a.refs_out[p + i] = r[i];
            } else {
                a.src[m++] = p + i;
            }
        }
        __threadfence_block();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (p + i < n && p + i >= used && r[i] != 0) {
                const int to = a.dst[m0++];
                a.remap[p + i] = to;
                a.refs_out[p + i] = 0;
                a.refs_out[to] = r[i];
            }
        holes += total & 0xffff;
        movers += total >> 16;
        __syncthreads();
    }
    for (int i = movers + tid; i < n / 2; i += kBookThreads) a.src[i] = a.dst[i] = -1;
    if (tid == 0) {
        a.info[0] = movers;
        a.info[1] = used;
    }
}

__global__ __launch_bounds__(256) void kda_cache_remap_kernel(const CompactArgs a, unsigned n) {
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    if (i >= n) return;
    const int e = a.table[i];
    a.table_out[i] = e >= 0 && e < a.n_pages ? a.remap[e] : e;
}

hipError_t launch_cache_compact(const CompactArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(kda_cache_compact_kernel, dim3(1), dim3(kBookThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    const unsigned n = (unsigned)a.B * a.max_pages;
    if (e != hipSuccess || n == 0) return e;
    hipLaunchKernelGGL(kda_cache_remap_kernel, dim3((n + 255) / 256), dim3(256), 0, s, a, n);
    return hipGetLastError();
}

// A page's K, all heads, is one piece of memory, its V another.  A workgroup takes
// pieces of up to 16 KB, four loads a thread in flight.  512 pages of 64 tokens, 8 heads and
// D = 128 (134 MB read and written): 25 us, 5.4 TB/s, with stores that leave the caches at once;
// ordinary ones 38, loads of that kind as well 28; pieces of 8 KB 39, of 32 KB 50 (both with
// ordinary stores).
__global__ __launch_bounds__(256) void kda_cache_copy_kernel(const CopyArgs a, unsigned chunks) {
    constexpr unsigned U = 4, CHUNK = 256 * 16 * U;
    const int n = a.count ? min(max(a.count[0], 0), a.n) : a.n;
    const unsigned long long units = (unsigned long long)n * 2 * chunks;
    for (unsigned long long u = blockIdx.x; u < units; u += gridDim.x) {
        const unsigned c = (unsigned)(u % chunks), part = (unsigned)((u / chunks) & 1), entry = (unsigned)(u / (2 * chunks));
        const int from = a.src[entry], to = a.dst[entry];
        if (from < 0 || from >= a.n_src || to < 0 || to >= a.n_dst) continue;
        const uint8_t* p = (part ? a.v : a.k) + (size_t)from * a.bytes;
        uint8_t* q = (part ? a.v_to : a.k_to) + (size_t)to * a.bytes;
        uint4 x[U];
#pragma unroll
        for (unsigned i = 0; i < U; ++i) {
            const unsigned at = c * CHUNK + i * 4096 + threadIdx.x * 16;
            if (at < a.bytes) x[i] = *reinterpret_cast<const uint4*>(p + at);
        }
#pragma unroll
        for (unsigned i = 0; i < U; ++i) {
            const unsigned at = c * CHUNK + i * 4096 + threadIdx.x * 16;
            if (at < a.bytes) store_once(q + at, x[i]);
        }
        if (c == 0) {
            const float* s = (part ? a.vs : a.ks) + (size_t)from * a.HK;
            float* d = (part ? a.vs_to : a.ks_to) + (size_t)to * a.HK;
            for (int h = threadIdx.x; h < a.HK; h += 256) d[h] = s[h];
        }
    }
}

hipError_t launch_cache_copy(const CopyArgs& a, hipStream_t s) {
    const unsigned chunks = (a.bytes + 16383) / 16384;
    const unsigned long long units = (unsigned long long)a.n * 2 * chunks;
    hipLaunchKernelGGL(kda_cache_copy_kernel, dim3((unsigned)(units < 16384 ? units : 16384)), dim3(256), 0, s, a, chunks);
    return hipGetLastError();
}

}  // namespace kda
