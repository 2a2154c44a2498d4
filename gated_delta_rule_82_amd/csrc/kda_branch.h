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
// How a call is divided: tiles of 64 or 128 rows of a group (bf16, D >= 32) over steps of
// 128 keys copied into LDS, or of 16 or 32 rows whose keys four waves read for
// themselves.  A wide tile reads and converts each key for more rows, but fills a
// compute unit alone (D = 128) and pays its start and end once a workgroup: its workgroups
// have to have enough steps.  Lengths are on the device: steps and parts are counted for
// prefixes that fill the table, and for groups as large as the average.  In us a call, 32-row /
// 64-row / 128-row tiles, 8 key/value heads, 200 own keys a sequence, tables as long as that:
//   groups of rows on keys     D = 128           D = 64            D = 32
//    8 of  32 on  4096       27   33            20   22           18   20
//    8 of  32 on 16384       65   73            46   47           38   42
//    4 of  64 on  4096       26   31   33       20   20   27      18   18   24
//    8 of  64 on  4096       47   47   51       29   24   37      23   21   32
//    8 of  64 on 16384       99   94  103       68   52   75      50   42   63
//    1 of 128 on 32768       49   48   45       39   30   35      37   28   31
//   16 of 128 on  4096      148  145  134       90   75   92      63   49   69
//    1 of 256 on  4096       25   30   33       20   20   27      18   18   23
//    1 of 256 on 16384       51   49   45       40   31   35      37   28   31
//    1 of 256 on 32768       86   75   62       68   47   47      64   43   41
//    4 of 256 on  4096       81   79   76       47   35   50      36   30   41
//    4 of 256 on 16384      160  158  129      118   84   87      89   74   73
// where the 64-row tiles' workgroups have 8, 32, 4, 8, 32, 16, 34, 4, 16, 32, 17 and 65 steps, 128-row tiles'
// half as many where groups have more rows (12 is between the 8 and 16 steps of the D = 128 lines:
// 8 would win up to 8 % there, and lose at D <= 64).  The rule is a compromise: 16 of 128 on 4096 at
// D = 64 and 32 would be quicker on 64-row tiles.  A table far longer than the prefixes is taken for long
// prefixes: 1 of 256 on 4096 takes 25 us with a table of 4608 tokens, 33 with one of 32768 or 131072.
// Own keys, and groups of 16 rows or fewer, have 16-row blocks: 8 groups of 16 rows on 4096 keys 22 us (32-row
// blocks 25), of 20 rows 28 (25); 64 samples of 20 own rows 96 (84).  Each part of a prefix is
// written and read again once, so there are only as many as give every
// compute unit a workgroup (8 groups of 32 rows on 4096 keys: 27 us with 4 parts, 33 with 8 or 2;
// on 16384 keys 65, 67 and 98); 32-row tiles that would have one or two get twice as many where each
// keeps 1024 keys (32 groups on 4096 keys, 60 own: 99 us with 1, 91 with 2, and 94 and 99 with 200 own; 16 on
// 16384, 60 own: 145 with 2, 123 with 4, and 122 and 127 with 200 own).  Own keys get parts of at least 256 keys up
// to two workgroups a compute unit: 512 own keys behind 32768 common ones 70 us, 71 with one workgroup, 76 with
// four; but 2 groups of 8 sequences with 2000 own keys 31, 25 with one workgroup.  Parts of 128 or 512 keys: no
// difference.
struct SharedPlan {
    int wide;           // 0, or blocks of 32 rows of a tile: 2, 4
    int own_blocks;     // blocks of 16 rows of a sequence's own keys (of a tile too, if not wide)
    int tiles, nprefix, nown;       // tiles: at most; one too many for each group whose rows fill its own
    long long blocks;   // workgroups, at most
};
inline SharedPlan shared_plan(int elem_bytes, int B, int Tq, int HK, int G, int D, int n_groups, int max_len) {
    SharedPlan p;
    const long long each = (long long)Tq * G, rows = each * B, average = n_groups > 0 ? rows / n_groups : rows;
    // tiles that are there, if the groups are about as large as each other
    const auto tiles_of = [rows, n_groups](int br) { const long long n = (rows + br - 1) / br; return n > n_groups ? n : n_groups; };
    const auto steps = [&](int br) {    // of a workgroup, where there are 256
        const long long n = tiles_of(br) * HK;
        return (n < 65536 ? n : 65536) * (max_len / 128) / 256;
    };
    const bool can = elem_bytes == 2 && D >= 32;
    p.wide = can && average > 64 && steps(128) >= 12 ? 4 : can && average > 32 && steps(64) >= 8 ? 2 : 0;
    p.own_blocks = (p.wide ? each : average) <= 16 ? 1 : 2;
    const int br = p.wide ? 32 * p.wide : 16 * p.own_blocks, bo = 16 * p.own_blocks;
    p.tiles = n_groups > 0 ? (int)(rows / br + n_groups) : 0;
    const long long own = (long long)B * HK * ((each + bo - 1) / bo);
    const auto parts = [max_len](long long wgs, int want, int keys) {
        long long n = wgs > 0 ? want / wgs : 1;
        n = n < max_len / keys ? n : max_len / keys;
        return n < 1 ? 1 : n > kMaxSplits / 2 ? kMaxSplits / 2 : (int)n;
    };
    const long long wgs = tiles_of(br) * HK;
    p.nprefix = parts(wgs, 256, 256);
    const int more = parts(wgs, 512, 1024);
    if (!p.wide && p.own_blocks == 2 && p.nprefix <= 2 && more > p.nprefix) p.nprefix = more;
    p.nown = parts(own, 512, 256);
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
// Parts of a row: about 1024 workgroups (512 rows of 131072 bf16 from memory take 53 us a call in 512, 40 in
// 1024, 44 in 2048 and 47 in 4096), at least 4096 elements each (32 rows of 65536 fp32 take 16 us a call, 19 with
// twice as many parts of 2048), and no more candidates than the join holds (a wave joins a beam's parts).
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
