// kda_attn.h - argument blocks and launchers of the softmax-attention operators.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// n / d for 0 <= n < 2^31 as a multiply and a shift (division by invariant integers using
// multiplication, Granlund and Montgomery 1994): with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(n, m) + n) >> s.
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.s) < d) ++f.s;
    f.m = (uint32_t)(((1ull << 32) * ((1ull << f.s) - d)) / d + 1);
    return f;
}

struct RotaryArgs {
    const void* q; const void* k; void* q_out; void* k_out;
    const int* positions; const double* inv_freq;
    size_t ldq, ldk, ldqo, ldko;   // elements between tokens
    size_t tokens;                 // B * T
    int T, H, HK, D, rot;
    float scale;
    int interleaved, inverse;
};
hipError_t launch_rotary(int dt, const RotaryArgs& a, hipStream_t s);

// Most elements between rows that are copied as tiles.  A tile's rows are addressed with
// unsigned 32-bit byte offsets from its first: 128 rows of 4-byte elements, the most that a
// kernel takes (Stage asserts it), start below 2^32 - 2^25.
constexpr int kTileStride = 1 << 23;

// The G query heads of a key/value head and their tokens are the packed rows
// r = t * G + g of one problem, 0 <= r < G * Tq, so a tile of rows shares the
// keys and values it streams.
struct AttnArgs {
    const void* q; const void* k; const void* v;
    const int* q_len; const int* kv_len;      // nullable
    void* o; float* lse;
    const void* dout; void* dq; void* dk; void* dv;
    float* rows;                // backward: (-lse / scale, in fp32 -lse, and -dout . o) of each query
    float* part_o; float* part_ml;  // split key axis: partial outputs and (maximum, sum)
    int B, Tq, Tk, H, HK, G;
    size_t ldq, ldk, ldv;       // elements between tokens
    float scale, scale_log2;    // scale, scale * log2 e
    int causal, window;         // window 0: none
    int whole;                  // backward: the keys are all that o and lse were formed with
    int nsplit;
    FastDiv divG;
};
// Packed rows of a wave (16-row column blocks: two in bf16, one in fp32), and
// waves of a workgroup: as many as the rows of a key/value head fill.
constexpr int attn_rows_per_wave(int elem_bytes) { return elem_bytes == 2 ? 32 : 16; }
inline int attn_waves(long long rows, int per_wave) { return rows <= per_wave ? 1 : rows <= 2 * per_wave ? 2 : 4; }
// Most parts a key axis is split into (the join reads their statistics at once).
constexpr int kMaxSplits = 128;
// Workgroups over the key axis (1: not split).  Two workgroups per compute unit
// fill the card; a split takes at least 256 keys (fp32, whose products cost 16 times
// as much: 128), so that its partial output stays small beside the keys it reads.
// fp32, 2 x 4 heads x 1023, D = 64: four parts 33 us with the join, three 37.
// Kernel and join in us with grids of 256 / 512 / 1024 workgroups, D = 128: 16 rows of 32
// heads over 65 536 keys of 8, bf16 54 / 54 / 62, fp32 221 / 190 / 206; 64 over 8192, bf16 26 /
// 31 / 31, fp32 107 / 96 / 105; 256 of 16 heads over 4096, bf16 25 / 33 / 33, fp32 104 / 93 /
// 103; 16 of 16 over 4096 (2 sequences), bf16 18 / 16 / 18.  Half the keys a split: fp32 16 over
// 65 536 204, 16 over 4096 25 against 22, one row over 1000 17 against 22; twice: bf16 16 over
// 4096 21 against 16, one over 1000 24 against 16, 256 over 4096 25 against 33.
inline int attn_fwd_splits(int elem_bytes, int B, int Tq, int Tk, int HK, int G) {
    const long long rows = (long long)Tq * G, per = attn_rows_per_wave(elem_bytes);
    const long long bq = per * attn_waves(rows, (int)per), wgs = (long long)B * HK * ((rows + bq - 1) / bq);
    const long long want = wgs > 0 ? 512 / wgs : 1, most = Tk / (elem_bytes == 2 ? 256 : 128), n = want < most ? want : most;
    return n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : (int)n;
}
hipError_t launch_attn_fwd(int dt, int D, const AttnArgs& a, hipStream_t s);
// The backward's row array holds a multiple of this many queries per head.
constexpr int kAttnRowPad = 64;
hipError_t launch_attn_bwd(int dt, int D, const AttnArgs& a, hipStream_t s);
// bf16 kernels whose eight waves take turns on the matrix cores.  A workgroup, of 256
// rows or 128 keys, has a compute unit to itself: they are taken where such workgroups
// fill the card's 256 units and what a row or key sees is long enough to pay for the
// slower start and, under a causal mask, for the whole tiles on the diagonal that both
// halves walk.  Measured, this kernel against the plain one (16 heads, D = 128 if not said):
//   forward  4 x 4096 causal, 4 heads of keys, 255 / 267 us, 2 x 2048 causal 57 / 56, window
//            2048 of 4096 125 / 115; 16 x 256 all keys 19 / 21; D = 64 4 x 4096 causal 175 / 158
//   dq       4 x 1024 causal 43 / 47, 8 x 512 causal 30 / 29; 16 x 256 all keys 23 / 25; D = 64
//            16 x 1024 causal, 4 heads of keys, 70 / 80, 2 x 2048 causal (256 workgroups, the
//            longest decides) 48 / 39, 16 x 256 all keys 12 / 16; D = 32 4 x 4096 167 / 157
//   dk, dv   4 x 4096 causal 488 / 735, 4 x 1024 causal 55 / 63, all keys 79 / 83; 8 x 512 43 / 39,
//            64 x 256 with 4 heads of keys 73 / 61, window 1024 of 4096 160 / 151, 2048 216 / 245;
//            D = 64 4 x 4096 causal 344 / 294
constexpr int kTurnsGrid = 256, kTurnsRows = 256, kTurnsKeys = 128;
inline long long turns_grid(const AttnArgs& a, long long n, int tile) { return (n + tile - 1) / tile * a.B * a.HK; }
inline bool attn_row_turns(const AttnArgs& a, int causal_from, int causal_grid) {
    const int keys = a.window > 0 && a.window < a.Tk ? a.window : a.Tk;
    const long long grid = turns_grid(a, (long long)a.Tq * a.G, kTurnsRows);
    return a.causal ? grid >= causal_grid && keys >= causal_from : grid >= kTurnsGrid && keys >= 256;
}
inline bool attn_fwd_turns(int elem_bytes, int D, const AttnArgs& a) {
    return elem_bytes == 2 && D == 128 && a.nsplit == 1 && attn_row_turns(a, 4096, kTurnsGrid);
}
inline bool attn_dq_turns(int elem_bytes, int D, const AttnArgs& a) {
    return elem_bytes == 2 && D >= 64 && attn_row_turns(a, 1024, D == 128 ? kTurnsGrid : 2 * kTurnsGrid);
}
inline bool attn_dkv_turns(int elem_bytes, int D, const AttnArgs& a) {
    const long long seen = a.window > 0 && a.window / 2 < a.Tq ? a.window / 2 : a.Tq;
    return elem_bytes == 2 && D == 128 && turns_grid(a, a.Tk, kTurnsKeys) >= kTurnsGrid && a.Tq >= 512 && seen * a.G >= 1024;
}
// Rows see so few keys that delta is summed over them (kda_attn_rows_few_kernel): no row
// more than 32, or 16 in windows of a long axis, where the kernel's 16 rows read 31 keys.
// Only where the call says that the keys are whole: a part of them that holds nearly all
// of a row's mass looks the same from here, and its dS is what the others leave of it.
// 64 x 16 heads x 64 of 128 channels, bf16: 22 us against 9 from o, with no gain in
// precision left; 4 x 16 heads x 4096, window 64: 102 us against 26.
inline bool attn_few_keys(const AttnArgs& a) { return a.whole && (a.Tk <= 32 || (a.causal && a.window > 0 && a.window <= 16)); }
hipError_t launch_dkv_turns(const AttnArgs& a, int padded, hipStream_t s);
hipError_t launch_dq_turns(int D, const AttnArgs& a, int padded, hipStream_t s);

struct AppendArgs {
    const void* k; const void* v;
    uint8_t* k_cache; uint8_t* v_cache; float* k_scale; float* v_scale;
    const int* block_table; const int* cache_len; const int* new_len;
    int n_pages, max_pages, B, T, HK, page;
    size_t ldk, ldv;
};
hipError_t launch_cache_append(int dt, int D, const AppendArgs& a, hipStream_t s);

struct AttnStepArgs {
    const void* q; const uint8_t* k_cache; const uint8_t* v_cache; const float* k_scale; const float* v_scale;
    const int* block_table; const int* cache_len; const int* new_len;
    void* o; float* part_o; float* part_ml;
    int n_pages, max_pages, B, Tq, H, HK, G, page, window, nsplit;
    size_t ldq;
    float scale_log2;
    FastDiv divG;
};
// 16-row blocks of a workgroup.
inline int attn_step_row_blocks(long long rows) { return rows <= 16 ? 1 : 2; }
// Workgroups over a cache of max_len tokens.  Four workgroups of four waves per
// compute unit keep enough loads in flight; a split takes at least 256 keys (one
// block for each wave).  Kernel and join in us with grids of 256 / 512 / 1024 / 2048
// workgroups, bf16, 32 heads (8 of keys), D = 128: 1 x 4 tokens over 65 536 31.7 / 30.2 / 31.9 /
// 31.7 (32 to 128 parts), 8 x 1 over 8192 28 / 29 / 28 / 28, 32 x 1 over 4096 42 / 47 / 47 / 48,
// 64 x 1 over 2048 43 / 43 / 48 / 48, 4 x 16 over 16 384 58 / 51 / 64 / 71.  At least 1024 keys
// a split: 30.2 for the first, 11 against 13 to 19 for one token over 1024.
inline int attn_step_splits(int B, int Tq, int HK, int G, int max_len) {
    const long long rows = (long long)Tq * G, br = 16 * attn_step_row_blocks(rows);
    const long long wgs = (long long)B * HK * ((rows + br - 1) / br);
    const long long want = wgs > 0 ? 1024 / wgs : 1, most = max_len / 256, n = want < most ? want : most;
    return n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : (int)n;
}
hipError_t launch_attn_step(int dt, int D, const AttnStepArgs& a, hipStream_t s);

// Joins the partial results of a split key axis: for packed row r of (b, hk),
// part_o [split][B*HK][rows][D] and part_ml [split][B*HK][rows][2] hold the
// unnormalised output, the maximum (log2 units) and the sum.
struct JoinArgs {
    const float* part_o; const float* part_ml; void* o; float* lse;  // lse nullable
    int nsplit, B, Tq, H, HK, G;
    FastDiv divG;
};
hipError_t launch_attn_join(int dt, int D, const JoinArgs& a, hipStream_t s);

}  // namespace kda
