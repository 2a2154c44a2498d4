// Drives the softmax-attention entry points' host validation under
// AddressSanitizer and UndefinedBehaviorSanitizer: argument values up to INT_MAX in
// every slot, with counting stand-ins for the launchers.  A rejected call must
// reach no launcher, an accepted one exactly one, with sizes inside the limits
// the kernels index with.
#include <limits.h>
#include <math.h>
#include <stdio.h>

#include "../../include/kda.h"
#include "kda_attn.h"

static int g_launches = 0;
static int g_failures = 0;
static void expect(bool ok, const char* what) {
    if (ok) return;
    ++g_failures;
    printf("FAILED: %s\n", what);
}

namespace kda {
hipError_t launch_rotary(int, const RotaryArgs& a, hipStream_t) {
    ++g_launches;
    expect(a.rot <= a.D && a.ldq >= (size_t)a.H * a.D && a.tokens > 0 && a.tokens * a.D < (1ull << 32), "rotary sizes");
    return hipSuccess;
}
static void attn_sizes(const AttnArgs& a) {
    expect(a.G >= 1 && a.H == a.G * a.HK && a.nsplit >= 1, "attention sizes");
    expect((unsigned long long)a.Tq * a.G <= (1ull << 29) && a.Tk <= (1 << 29) && a.window >= 0 && (a.window == 0 || a.window < a.Tk), "attention rows");
    expect(a.nsplit == 1 || (a.part_o && a.part_ml), "attention partials");
    const unsigned long long bh = (unsigned long long)a.B * a.HK, rows = (unsigned long long)a.Tq * a.G;
    expect(bh * ((rows + 31) / 32) < (1ull << 24) && bh * (((unsigned long long)a.Tk + 31) / 32) < (1ull << 24), "attention grids");
}
static void row_pieces(int dt, int D, const AttnArgs& a) {
    const unsigned long long padded = ((unsigned long long)a.Tq + kAttnRowPad - 1) / kAttnRowPad * kAttnRowPad;
    expect(a.B * (unsigned long long)a.H * padded * (D * (dt == 1 ? 2 : 4) / 16) + 255 < (1ull << 32), "row pieces");
}
hipError_t launch_attn_fwd(int, int, const AttnArgs& a, hipStream_t) { ++g_launches; attn_sizes(a); return hipSuccess; }
hipError_t launch_attn_bwd(int dt, int D, const AttnArgs& a, hipStream_t) { ++g_launches; attn_sizes(a); row_pieces(dt, D, a); return hipSuccess; }
hipError_t launch_cache_append(int, int, const AppendArgs& a, hipStream_t) {
    ++g_launches;
    expect((unsigned long long)a.B * a.HK * ((unsigned long long)a.T / a.page + 2) < (1ull << 24), "append grid");
    return hipSuccess;
}
hipError_t launch_attn_step(int, int, const AttnStepArgs& a, hipStream_t) {
    ++g_launches;
    expect((long long)a.max_pages * a.page <= (1 << 29) && a.nsplit >= 1, "step sizes");
    expect((unsigned long long)a.B * a.HK * (((unsigned long long)a.Tq * a.G + 31) / 32) * a.nsplit < (1ull << 24), "step grid");
    return hipSuccess;
}
}  // namespace kda

static const int kInts[] = {INT_MIN, -1, 0, 1, 2, 3, 7, 16, 31, 64, 128, 4096, 1 << 20, 1 << 24, 1 << 30, INT_MAX};
constexpr int kN = sizeof(kInts) / sizeof(kInts[0]);

// Cheap deterministic choice of argument values.
static unsigned g_state = 1;
static unsigned draw(unsigned n) {
    g_state = g_state * 1664525u + 1013904223u;
    return (g_state >> 8) % n;
}
static int any_int() { return kInts[draw(kN)]; }
static int some(int usual) { return draw(4) ? usual : any_int(); }
template <typename P> static P* at(int i) {
    if (draw(40) == 0) return nullptr;
    return reinterpret_cast<P*>((uintptr_t)0x10000 + ((uintptr_t)i << 44) + (draw(40) == 0 ? 4 : 0));
}
static void one(kda_status st, int before) {
    expect(st == KDA_OK ? g_launches - before <= 1 : g_launches == before, "launches of a call");
    expect(kda_status(st) >= KDA_OK && st <= KDA_ERR_SCALE, "known status");
}

int main() {
    static const int dims[] = {16, 32, 64, 128}, pages[] = {16, 32, 64, 128};
    static const float scales[] = {1.f, 0.125f, 0.f, -1.f, INFINITY, NAN, 3e38f, 1e-40f};
    long accepted = 0;
    for (int i = 0; i < 400000; ++i) {
        const int B = some(2), T = some(64), Tk = some(4096), HK = some(2), H = draw(4) ? (HK > 0 && HK < 4096 ? HK * 4 : 4) : any_int();
        const int D = draw(6) ? dims[draw(4)] : any_int(), page = draw(6) ? pages[draw(4)] : any_int();
        const kda_dtype dt = (kda_dtype)(draw(12) ? draw(2) : 3);
        const float sc = draw(4) ? 0.125f : scales[draw(8)];
        const int ld = draw(4) ? 0 : any_int(), ld2 = draw(4) ? 0 : any_int(), win = draw(3) ? 0 : any_int();
        void* ws = at<void>(12);
        const size_t wsb = draw(4) ? (size_t)1 << 60 : draw(1000);
        const int before = g_launches;
        switch (i % 5) {
            case 0:
                one(kda_rotary(at<void>(1), at<void>(2), at<void>(3), at<void>(4), at<int>(5), at<double>(6), B, T, H, HK, D, some(16),
                               ld, ld2, ld, ld2, sc, draw(5), dt, nullptr), before);
                break;
            case 1:
                one(kda_attn_fwd(at<void>(1), at<void>(2), at<void>(3), at<int>(4), at<int>(5), at<void>(6), at<float>(7), B, T, Tk, H, HK,
                                 D, ld, ld2, ld2, sc, draw(2), win, dt, ws, wsb, nullptr), before);
                (void)kda_attn_fwd_workspace(B, T, Tk, H, HK, D, dt);
                break;
            case 2:
                one(kda_attn_bwd(at<void>(1), at<void>(2), at<void>(3), at<int>(4), at<int>(5), at<void>(6), at<float>(7), at<void>(8),
                                 at<void>(9), at<void>(10), at<void>(11), B, T, Tk, H, HK, D, ld, ld2, ld2, sc, draw(2), win, dt, ws, wsb,
                                 nullptr), before);
                (void)kda_attn_bwd_workspace(B, T, Tk, H, HK, D, dt);
                break;
            case 3:
                one(kda_cache_append(at<void>(1), at<void>(2), at<void>(3), at<void>(4), at<float>(5), at<float>(6), at<int>(7), at<int>(8),
                                     at<int>(9), some(8), some(4), B, T, HK, D, page, ld, ld2, dt, nullptr), before);
                break;
            default:
                one(kda_attn_step(at<void>(1), at<void>(2), at<void>(3), at<float>(4), at<float>(5), at<int>(6), at<int>(7), at<int>(8),
                                  at<void>(9), some(8), some(4), B, T, H, HK, D, page, ld, sc, win, dt, ws, wsb, nullptr), before);
                (void)kda_attn_step_workspace(B, T, H, HK, D, Tk);
        }
        accepted += g_launches - before;
    }
    expect(accepted > 10000, "enough accepted calls");
    for (int i = 0; i < 20000; ++i) {
        double f[64];
        float s;
        const double base = draw(4) ? 1e4 : draw(2) ? 1.0 : INFINITY, factor = draw(4) ? 4.0 : draw(2) ? 0.0 : NAN;
        const kda_status st = kda_rotary_freqs(draw(20) ? f : nullptr, draw(2) ? &s : nullptr, some(64), base, (int)draw(5), factor,
                                               some(4096), draw(4) ? 32.0 : NAN, draw(4) ? 1.0 : 40.0);
        expect(st >= KDA_OK && st <= KDA_ERR_SCALE, "frequencies' status");
    }
    // the division by a multiply and a shift, over small divisors and the range's ends
    for (uint32_t d = 1; d < 3000; d += d < 300 ? 1 : 37) {
        const kda::FastDiv f = kda::fast_div(d);
        for (int i = 0; i < 400; ++i) {
            uint32_t n = i < 100 ? (uint32_t)i : i < 200 ? (1u << 31) - 1 - (uint32_t)i : (uint32_t)(draw(1 << 24)) * 127u;
            n &= 0x7fffffffu;
            const uint32_t q = (uint32_t)(((uint64_t)n * f.m >> 32) + n) >> f.s;
            expect(q == n / d, "fast division");
        }
    }
    if (g_failures) return 1;
    printf("all expectations hold (%ld calls accepted)\n", accepted);
    return 0;
}
