// kda_branch.h - argument blocks and launchers of the operators that continue one
// prompt several times: pages of the cache, attention with a common prefix, selection
// over beams and vocabulary, states that follow their parents.
#pragma once

#include "kda_attn.h"

namespace kda {

struct ForkArgs {
    const int* table; const int* cache_len; const int* parent;
    int* table_out; int* len_out; int* refs;
    int R, K_in, K_out, max_pages, n_pages, page, keep;
};
hipError_t launch_cache_fork(const ForkArgs& a, hipStream_t s);

struct FreeArgs {
    int* table; int* refs; const int* keep_from; const int* keep_to;
    int B, max_pages, n_pages, page;
};
hipError_t launch_cache_free(const FreeArgs& a, hipStream_t s);

// Pages that T tokens of a sequence can touch.
inline int pages_touched(int T, int page) { return T > 0 ? (int)(((long long)T + page - 2) / page + 1) : 1; }

struct ReserveArgs {
    int* table; int* refs; const int* cache_len; const int* new_len;
    int* src; int* dst; int* info;
    int B, T, max_pages, n_pages, page, touched;
};
hipError_t launch_cache_reserve(const ReserveArgs& a, hipStream_t s);

struct CompactArgs {
    const int* table; const int* refs;
    int* table_out; int* refs_out; int* remap; int* src; int* dst; int* info;
    int B, max_pages, n_pages;
};
hipError_t launch_cache_compact(const CompactArgs& a, hipStream_t s);

struct CopyArgs {
    const uint8_t* k; const uint8_t* v; const float* ks; const float* vs;
    uint8_t* k_to; uint8_t* v_to; float* ks_to; float* vs_to;
    const int* src; const int* dst; const int* count;   // count nullable
    int n, n_src, n_dst, HK;
    unsigned bytes;                                     // of K (and of V) in a page, all heads: HK * page * D
};
hipError_t launch_cache_copy(const CopyArgs& a, hipStream_t s);

struct ReorderArgs {
    const uint8_t* state; uint8_t* out; const int* parent;
    int R, K_in, K_out;
    unsigned long long row_bytes;                       // a multiple of 16
};
constexpr int kReorderMost = 64;    // beams of a request that is reordered in place
hipError_t launch_state_reorder(const ReorderArgs& a, hipStream_t s);

struct AttnSharedArgs {
    const void* q; const uint8_t* k_cache; const uint8_t* v_cache; const float* k_scale; const float* v_scale;
    const int* block_table; const int* cache_len; const int* new_len; const int* group_first; const int* prefix_len;
    void* o; float* part_o; float* part_ml;
    int n_groups, n_pages, max_pages, B, Tq, H, HK, G, page, window;
    int wide, own_blocks;           // SharedPlan
    int tiles, nprefix, nown;       // tiles of all groups' rows (at most); parts of a prefix and of a sequence's own keys
    int prefix_blocks;              // HK * tiles * nprefix
    size_t ldq;
    float scale_log2;
    FastDiv divG, divT;
};
// How the rows and keys are cut, from what the host knows: tables of max_len tokens.
struct SharedPlan {
    int wide;               // groups of 32 rows of a workgroup on a prefix; 0: own_blocks of 16 there too
    int own_blocks;         // 16-row blocks of a workgroup on own keys
    int tiles, nprefix, nown;
    long long blocks;
};
inline SharedPlan shared_plan(int elem_bytes, int B, int Tq, int HK, int G, int D, int n_groups, int max_len) {
    SharedPlan p;
    const long long each = (long long)Tq * G, rows = each * B, average = n_groups > 0 ? rows / n_groups : rows;
    p.wide = elem_bytes == 4 || D < 32 || average <= 16 ? 0 : average <= 64 ? 2 : 4;
    p.own_blocks = (p.wide ? each : average) <= 16 ? 1 : 2;
    const int br = p.wide ? 32 * p.wide : 16 * p.own_blocks, bo = 16 * p.own_blocks;
    p.tiles = n_groups > 0 ? (int)(rows / br + n_groups) : 0;
    const long long own = (long long)B * HK * ((each + bo - 1) / bo), most = max_len / 256;
    const auto parts = [most](long long wgs, long long want, int limit) {
        long long n = wgs > 0 ? want / wgs : 1;
        n = n < most ? n : most;
        return n < 1 ? 1 : n > limit ? limit : (int)n;
    };
    // tiles that are there, if the groups are about as large as each other
    const long long tiles = (rows + br - 1) / br > n_groups ? (rows + br - 1) / br : n_groups;
    p.nprefix = parts(tiles * HK, p.wide ? 256 : 512, kMaxSplits / 2);
    p.nown = parts(own, 512, kMaxSplits / 2);
    p.blocks = (long long)HK * p.tiles * p.nprefix + own * p.nown;
    return p;
}
hipError_t launch_attn_shared(int dt, int D, const AttnSharedArgs& a, hipStream_t s);

// Beams of a request and candidates of a selection.
constexpr int kSelectMost = 64;
// Candidates that the joining workgroup holds.
constexpr int kSelectHeld = 4096;
struct SelectArgs {
    const void* logits; const float* scores; const uint8_t* done;
    float* scores_out; int* parent; int* token;
    double* stat;  float* part_x; int* part_w;           // of each part: (maximum, sum), M candidates, -1 behind the last
    int R, K, V, M, end, nsplit;
    size_t ld;
};
// Elements of a row's part of n: whole 16-byte loads of a workgroup's threads.
constexpr int kSelThreads = 256;
constexpr int select_part(int V, int n, int per_load) {
    const int step = kSelThreads * per_load, per = (V + n - 1) / n;
    return (per + step - 1) / step * step;
}
// Parts of a row: about 1024 workgroups (512 rows of 131072 bf16 take 54 us in 512, 43 in 1024,
// 45 in 2048), at least 4096 elements each (32 rows of 65536 fp32 take 12 us, 15 with
// twice as many parts of 2048), and no more
// candidates than the join holds (a wave joins a beam's parts).
inline int select_splits(int elem_bytes, int R, int K, int V, int M) {
    const long long rows = (long long)R * K;
    long long n = rows > 0 ? 1024 / rows : 1;
    if (n > V / 4096) n = V / 4096;
    if (n > kSelectHeld / (K * M)) n = kSelectHeld / (K * M);
    n = n < 1 ? 1 : n > 64 ? 64 : n;
    const int per = select_part(V, (int)n, 16 / elem_bytes);
    return (int)(((long long)V + per - 1) / per);   // none without elements
}
hipError_t launch_beam_select(int dt, const SelectArgs& a, hipStream_t s);

}  // namespace kda
