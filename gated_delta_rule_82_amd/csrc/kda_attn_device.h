// kda_attn_device.h - device-side building blocks of the attention kernels.
//
// Tiles of token rows live in LDS as rows of D elements, cut into granules of 16
// bytes; granule c of row r is at position c ^ tile_swizzle(r), so that both ways a
// tile is read fill the 256 bytes a cycle of the 64 banks:
//   * row fragments (a lane reads 8 consecutive elements of its row): a 16-byte read
//     is served in phases of 16 lanes, {0-3, 12-15, 20-27} and {4-11, 16-19, 28-31} of
//     each half wave (measured): rows 0-3 and 12-15 at granule c, rows 4-11 at c ^ 1;
//   * column fragments of bf16 (four rows by 16 columns per 16 lanes through the
//     transposing LDS read): phases of 32 lanes, eight rows by two granules.
// Even swizzles 2 (r mod 8) (for 256-byte rows; one step per 256 bytes in general)
// meet both.  With a swizzle that serves only one of them every read of the other
// kind took twice as long.
// Contraction slots: row fragments hold elements 32 s + 8 (l / 16) + j of their
// row in slot j (any map serves as long as both operands share it), column
// fragments rows slot_index(l / 16, j), the map of frag_from_c, so that score
// tiles go from the accumulator into the next product without moving.
#pragma once

#include "kda_attn.h"
#include "kda_device.h"

namespace kda {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv& f) { return (__umulhi(n, f.m) + n) >> f.s; }

// Maximum / sum over the four lane groups that share lane % 16, on the vector
// unit (half-row swaps) rather than through LDS.
__device__ __forceinline__ float group_max4(float x) {
    const uint32_t u = __float_as_uint(x);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float y = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const uint32_t w = __float_as_uint(y);
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float group_add4(float x) {
    const uint32_t u = __float_as_uint(x);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float y = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const uint32_t w = __float_as_uint(y);
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Number of valid elements of sequence b, clamped to the tensor's range.
__device__ __forceinline__ int seq_len(const int* len, int b, int most) {
    if (!len) return most;
    const int n = len[b];
    return n < 0 ? 0 : n > most ? most : n;
}

// The (sequence, key/value head) of a workgroup, of nbh.  Heads go fastest, so that one
// head's tiles share an XCD's L2 where the heads are a multiple of 8.  Where sequences
// have lengths of their own and fewer than 8 heads each, that would leave the XCDs of the
// short ones idle: the head then moves on with every round of heads.  bf16, D = 128, 4 x 4
// heads of 4 query heads, 4096 down to 2560 tokens: forward 188 us against 223,
// backward 682 against 764, at the price of the L2 where all have 4096 (290 against 270);
// with rows below 8192 a head (1024 tokens) 57 us against 54.
__device__ __forceinline__ int head_of(const AttnArgs& a, int bid, int nbh) {
    const int i = bid % nbh;
    const bool move_on = (a.q_len || a.kv_len) && a.HK % 8 != 0 && a.Tq * a.G >= 8192;
    return move_on ? (i + bid / nbh) % nbh : i;
}

// Where a tile of packed rows starts and which keys its rows can see.
struct RowRange {
    int t_first, t_last;   // tokens of the first and last row (t_last < q_len)
    int key_lo, key_hi;    // keys seen by some row: [key_lo, key_hi)
};

__device__ __forceinline__ RowRange row_range(const AttnArgs& a, int r0, int r1, int ql, int kl) {
    RowRange x;
    x.t_first = (int)fdiv((uint32_t)r0, a.divG);
    x.t_last = min((int)fdiv((uint32_t)(r1 - 1), a.divG), ql - 1);
    const int off = kl - ql;
    x.key_hi = a.causal ? min(kl, x.t_last + off + 1) : kl;
    x.key_lo = a.window ? max(0, x.t_first + off - a.window + 1) : 0;
    if (x.t_first >= ql || x.key_hi < x.key_lo) x.key_hi = x.key_lo;
    return x;
}

template <typename T, int D> struct TileGeom {
    static constexpr int GR = D * (int)sizeof(T) / 16;      // granules per row
    static constexpr int NS = (D + 31) / 32;                // contraction steps over a row
    static constexpr int ND = D / 16;                       // 16-channel blocks
};

// Swizzle of a tile row (see the top of this file).  fp32 columns are read a word a
// lane, four rows at once: there the row number itself spreads them.
template <typename T, int D> __device__ __forceinline__ int tile_swizzle(int row) {
    constexpr int GR = TileGeom<T, D>::GR, RPL = GR < 16 ? 16 / GR : 1;   // rows per 256 bytes
    return sizeof(T) == 2 ? 2 * ((row / RPL) & (GR / 2 - 1) & 7) : (row / RPL) & (GR - 1) & 15;
}

// Swizzle of a tile that is read by 32x32x16 products (Wide fragments below): row
// fragments put rows {0-3, 12-15, 20-27} or {4-11, 16-19, 28-31} of one granule into a
// phase, column fragments four rows by four granules.
template <int D> __device__ __forceinline__ int wide_swizzle(int row) {
    constexpr int GR = TileGeom<bf16_t, D>::GR, RPL = GR < 16 ? 16 / GR : 1;
    return ((4 * (row / RPL)) & (GR - 1) & 12) | ((row >> 3) & 3);
}

// e^x for x <= about 0 with the rounding of x log2 e carried along (without it the result
// is off by up to |x| 2^-25 besides the instruction's own error).
__device__ __forceinline__ float exp_carried(float x) {
    constexpr float kLog2eLow = 1.92596299e-8f;   // log2 e - kLog2e
    const float hi = x * kLog2e, lo = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -hi)), y = exp2_fast(hi);
    return y == 0.f ? 0.f : fmaf(y, lo * kLn2, y);
}

// A window of memory for buffer loads: reads at or past `bytes` give zero.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4 buffer_window(const void* p, long long bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t n = bytes <= 0 ? 0u : bytes > 0xffffffffll ? 0xffffffffu : (uint32_t)bytes;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a), (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) & 0xffffu,
                 (uint32_t)__builtin_amdgcn_readfirstlane(n), 0x00020000u};
}

// The first `rows` of a tile's rows, which lie `step` bytes apart and are `width` wide (the
// tile spans less than 2^31 bytes; rows >= 1).  Loops that carry p and rows along leave
// little for the scalar unit: 64-bit products and clamps of whole tensors took half of a
// vector turn.
__device__ __forceinline__ u32x4 tile_window(const void* p, int rows, uint32_t step, uint32_t width) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a), (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) & 0xffffu,
                 (uint32_t)__builtin_amdgcn_readfirstlane((rows - 1) * step + width), 0x00020000u};
}

// 16 bytes a lane from window + off into LDS at lds + 16 * lane.  Written as
// assembly because the compiler, seeing the copy, would wait for all copies in
// flight (the next tile's) before the transposing reads of the current one.  It has
// no output registers; the kernels wait with wait_vmcnt and a barrier.  m0, which
// holds the LDS address, is set at every use and used by nothing else here.
__device__ __forceinline__ void copy_to_lds(const u32x4& window, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(window) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p);
}

// Copies of ROWS-row tiles into LDS by NW waves: one wave instruction moves 64
// granules.  row_off(r) is the byte offset of the tile's row r in the window.
template <typename T, int D, int ROWS, int NW, bool Wide = false> struct Stage {
    static constexpr int GR = TileGeom<T, D>::GR, N = ROWS * GR / 64, PER = (N + NW - 1) / NW;
    static_assert(ROWS * GR % 64 == 0, "whole wave instructions");
    static_assert((unsigned long long)ROWS * kTileStride * sizeof(T) <= 1ull << 32, "rows a largest stride apart fit 32-bit offsets");
    uint32_t off[PER];
    static __device__ __forceinline__ int swizzle(int r) { return Wide ? wide_swizzle<D>(r) : tile_swizzle<T, D>(r); }
    static __device__ __forceinline__ int row(int c, int wave, int lane) { return ((c * NW + wave) * 64 + lane) / GR; }
    // byte offset within its row of the granule that lands at this lane's place
    static __device__ __forceinline__ uint32_t col(int c, int wave, int lane) {
        return (uint32_t)(((lane % GR) ^ swizzle(row(c, wave, lane))) * 16);
    }
    template <typename RowOff> __device__ __forceinline__ void init(int wave, int lane, RowOff row_off) {
#pragma unroll
        for (int c = 0; c < PER; ++c) off[c] = row_off(row(c, wave, lane)) + col(c, wave, lane);
    }
    __device__ __forceinline__ void issue_one(const u32x4& window, uint32_t tile, int wave, int c) const {
        if (N % NW == 0 || c * NW + wave < N) copy_to_lds(window, off[c], tile + (c * NW + wave) * 1024);
    }
    __device__ __forceinline__ void issue(const u32x4& window, uint32_t tile, int wave) const {
#pragma unroll
        for (int c = 0; c < PER; ++c) issue_one(window, tile, wave, c);
    }
};

// A lane's place in a tile: byte offset of its granule of row l % 16 at
// contraction step 0 and, for column fragments of bf16, of the four columns it
// loads of row 4 (l / 16) + (l / 4) % 4 at column block 0.  Steps and blocks differ
// by an exclusive or within the row (`tile` and r0 move whole rows), so that only
// these two values are kept and the others cost one instruction at their use.
template <typename T, int D> struct TileLane {
    static constexpr int RB = D * (int)sizeof(T);   // bytes per row
    uint32_t row, col;
    __device__ __forceinline__ explicit TileLane(int lane) {
        const int r = lane & 15, g = lane >> 4, i = lane & 3;
        const int c = sizeof(T) == 2 ? (D >= 32 ? g : g & 1) : (D >= 32 ? 2 * g : 2 * (g & 1));
        row = r * RB + ((c ^ tile_swizzle<T, D>(r)) * 16);
        const int q = 4 * g + ((lane >> 2) & 3);
        col = q * RB + (((i >> 1) ^ tile_swizzle<T, D>(q)) * 16) + (i & 1) * 8;
    }
};

// Row fragment of rows [r0, r0 + 16) of the tile at byte `tile` of `sm`, contraction step s.
template <int D>
__device__ __forceinline__ Frag<bf16_t> row_frag(const unsigned char* sm, uint32_t tile, int r0, int s, const TileLane<bf16_t, D>& l,
                                                 int lane) {
    Frag<bf16_t> f;
    f.v = *reinterpret_cast<const bf16x8*>(sm + ((l.row + tile) ^ (64 * s)) + r0 * (D * 2));
    if (D < 32 && (lane >> 4) >= 2) f.zero();  // 16 channels fill half a step
    return f;
}
template <int D>
__device__ __forceinline__ Frag<float> row_frag(const unsigned char* sm, uint32_t tile, int r0, int s, const TileLane<float, D>& l,
                                                int lane) {
    const uint32_t o = (l.row + tile) ^ (128 * s);
    const float4 a = *reinterpret_cast<const float4*>(sm + o + r0 * (D * 4));
    const float4 b = *reinterpret_cast<const float4*>(sm + (o ^ 16) + r0 * (D * 4));
    Frag<float> f;
    f.v[0] = a.x; f.v[1] = a.y; f.v[2] = a.z; f.v[3] = a.w;
    f.v[4] = b.x; f.v[5] = b.y; f.v[6] = b.z; f.v[7] = b.w;
    if (D < 32 && (lane >> 4) >= 2) f.zero();
    return f;
}

// The same fragment straight from a row in memory (p: the row's first element).
template <typename T, int D>
__device__ __forceinline__ Frag<T> row_frag_global(const T* p, int s, int lane) {
    const int g = lane >> 4;
    Frag<T> f;
    if constexpr (D >= 32) {
        frag_load_row8(f, p + 32 * s + 8 * g);
    } else {
        frag_load_row8(f, p + 8 * (g & 1));
        if (g >= 2) f.zero();
    }
    return f;
}

// A product over the first N slots of each fragment (fp32: 4 of 8 are half a step).
template <int N, typename T> __device__ __forceinline__ floatx4 mma_slots(const Frag<T>& a, const Frag<T>& b, floatx4 c) {
    if constexpr (N == 8) {
        return mma(a, b, c);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
        return c;
    }
}

// Column fragment: column 16 c + l % 16 of the 32 rows from r0 of the tile; with N = 4
// (fp32) slots 0 .. 3 alone, the first 16 rows.
template <int D, int N = 8>
__device__ __forceinline__ Frag<bf16_t> col_frag(const unsigned char* sm, uint32_t tile, int r0, int c, const TileLane<bf16_t, D>& l,
                                                 int) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    typedef s16x4 __attribute__((address_space(3)))* lds4;
    // lane i of a 16-lane group loads 4 columns of row i / 4 and receives column i of the four rows
    const unsigned char* p = sm + ((l.col + tile) ^ (32 * c)) + r0 * (D * 2);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 16 * (D * 2)));
    Frag<bf16_t> f;
    f.v = __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
    return f;
}
template <int D, int N = 8>
__device__ __forceinline__ Frag<float> col_frag(const unsigned char* sm, uint32_t tile, int r0, int c, const TileLane<float, D>&,
                                                int lane) {
    const int col = 16 * c + (lane & 15), g = lane >> 4;
    Frag<float> f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int row = r0 + slot_index(g, j);
        f.v[j] = *reinterpret_cast<const float*>(sm + tile + row * (D * 4) +
                                                 (((col >> 2) ^ tile_swizzle<float, D>(row)) * 16) + (col & 3) * 4);
    }
    return f;
}

// ---------------------------------------------------------------- 32x32x16
// The same products on 32x32 tiles (bf16, D >= 32).  Per flop they hold the vector
// unit's issue for half as long: beside back-to-back 16x16x32 products another wave
// of the SIMD issues a vector instruction every 9.3 cycles, beside 32x32x16 ones
// every 6.0 (4.8 alone; exponentials 18.9, 11.2 and 8.5).
//   * accumulator: lane l, element i is row 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32;
//   * operand fragment of a 16-long step: lane l supplies row (column) l % 32 at 8 slots.
//     Row fragments hold elements 16 s + 8 (l / 32) + j; column fragments of 32 rows
//     hold, at step u, rows 16 u + 8 (j / 4) + 4 (l / 32) + j % 4: elements 8 u .. 8 u + 7
//     of an accumulator, rounded, are the matching operand.
typedef float floatx16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ floatx16 mma32(const Frag<bf16_t>& a, const Frag<bf16_t>& b, const floatx16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ floatx16 splat16(float x) {
    floatx16 v;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = x;
    return v;
}
// Operand of step u from an accumulator.
__device__ __forceinline__ Frag<bf16_t> frag_of(const floatx16& x, int u) {
    Frag<bf16_t> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = (bf16_t)x[8 * u + j];
    return f;
}

// Fragments whose computation ends here: without it the compiler moves their last
// instructions past the barrier that follows, in front of the next turn's products.
template <int N> __device__ __forceinline__ void settle(Frag<bf16_t> (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(f[i].v));
}

// Maximum / sum over the two lanes that share a column.
__device__ __forceinline__ float pair_max(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float pair_add(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// A lane's place in a tile, as TileLane.
template <int D> struct WideLane {
    static constexpr int RB = D * 2;
    uint32_t row, col;
    __device__ __forceinline__ explicit WideLane(int lane) {
        const int r = lane & 31, h = lane >> 5, i = lane & 3;
        row = r * RB + ((h ^ wide_swizzle<D>(r)) * 16);
        // lanes 16 .. 31 of a half take the upper 16 of 32 columns
        const int q = 4 * h + ((lane >> 2) & 3);
        col = q * RB + (((2 * ((lane >> 4) & 1) + (i >> 1)) ^ wide_swizzle<D>(q)) * 16) + (i & 1) * 8;
    }
};
// Row fragment of rows [r0, r0 + 32) (r0 a multiple of 32), step s.
template <int D>
__device__ __forceinline__ Frag<bf16_t> wide_row(const unsigned char* sm, uint32_t tile, int r0, int s, const WideLane<D>& l) {
    Frag<bf16_t> f;
    f.v = *reinterpret_cast<const bf16x8*>(sm + ((l.row + tile) ^ (32 * s)) + r0 * (D * 2));
    return f;
}
// Column fragment: columns 32 c + l % 32 at step u of the 32 rows from r0.
template <int D>
__device__ __forceinline__ Frag<bf16_t> wide_col(const unsigned char* sm, uint32_t tile, int r0, int u, int c, const WideLane<D>& l) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    typedef s16x4 __attribute__((address_space(3)))* lds4;
    // rows 16 u + 8 k + 4 h + .. differ from 4 h + .. in bits 3 and 4, the swizzle's low bits
    const unsigned char* base = sm + (r0 + 16 * u) * (D * 2);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(base + ((l.col + tile) ^ (64 * c) ^ (16 * (2 * u)))));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(base + 8 * (D * 2) + ((l.col + tile) ^ (64 * c) ^ (16 * (2 * u + 1)))));
    Frag<bf16_t> f;
    f.v = __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
    return f;
}

// Writes a wave's accumulators (rows: the D channels, columns: 32 tensor rows) times
// `scale` as bf16 rows, zeros for columns that are not live whatever the accumulators
// hold.  They go through the wave's 64 D bytes of LDS and leave as whole rows, 16 bytes
// a lane: straight from the accumulators a store would touch 32 rows, 16 bytes of each.
// dest(row) is the address of tensor row `row`, or null.
template <int D, typename Dest>
__device__ __forceinline__ void wide_rows_out(const floatx16 (&x)[D / 32], float scale, bool live, unsigned char* lds, int lane, Dest dest) {
    constexpr int GR = D / 8, RPI = 64 / GR;   // granules of a row, rows of a wave instruction
    auto place_of = [](int row, int granule) { return row * D * 2 + ((granule ^ wide_swizzle<D>(row)) * 16); };
    asm volatile("" ::: "memory");  // a wave's LDS accesses stay in order, and the compiler keeps that order
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const floatx4 y = {x[d][4 * e] * scale, x[d][4 * e + 1] * scale, x[d][4 * e + 2] * scale, x[d][4 * e + 3] * scale};
            store4(reinterpret_cast<bf16_t*>(lds + place_of(lane & 31, 4 * d + e) + 8 * (lane >> 5)), live ? y : floatx4{0.f, 0.f, 0.f, 0.f});
        }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32 / RPI; ++i) {
        const int row = i * RPI + lane / GR, granule = lane % GR;
        const uint4 y = *reinterpret_cast<const uint4*>(lds + place_of(row, granule));
        bf16_t* to = dest(row);
        if (to) *reinterpret_cast<uint4*>(to + granule * 8) = y;
    }
}

}  // namespace kda
