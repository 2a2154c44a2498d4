// Drives the host validation of the operators that continue one prompt several times
// under AddressSanitizer and UndefinedBehaviorSanitizer: argument values up to INT_MAX in
// every slot, with counting stand-ins for the launchers.  A rejected call must reach no
// launcher, an accepted one at most one, with sizes inside the limits the kernels index
// with.
#include <limits.h>
#include <math.h>
#include <stdio.h>

#include "../../include/kda.h"
#include "kda_branch.h"

static int g_launches = 0;
static int g_failures = 0;
static void expect(bool ok, const char* what) {
    if (ok) return;
    ++g_failures;
    printf("FAILED: %s\n", what);
}

typedef unsigned long long u64;
namespace kda {
hipError_t launch_cache_fork(const ForkArgs& a, hipStream_t) {
    ++g_launches;
    const u64 w = a.max_pages > 0 ? a.max_pages : 1;
    expect((u64)a.R * a.K_in * w + (u64)a.R * a.K_out * w < (1ull << 31) && a.K_in <= 1024 && a.K_out <= 1024, "fork grid");
    return hipSuccess;
}
hipError_t launch_cache_free(const FreeArgs& a, hipStream_t) {
    ++g_launches;
    expect((u64)a.B * a.max_pages < (1ull << 31) && a.max_pages > 0, "free grid");
    return hipSuccess;
}
hipError_t launch_cache_reserve(const ReserveArgs& a, hipStream_t) {
    ++g_launches;
    expect((u64)a.B * a.touched < (1ull << 31) && a.touched >= 1 && a.n_pages <= (1 << 30), "reserve entries");
    return hipSuccess;
}
hipError_t launch_cache_compact(const CompactArgs& a, hipStream_t) {
    ++g_launches;
    expect((u64)a.B * a.max_pages < (1ull << 31) && a.n_pages <= (1 << 30), "compact grid");
    return hipSuccess;
}
hipError_t launch_cache_copy(const CopyArgs& a, hipStream_t) {
    ++g_launches;
    expect(a.bytes > 0 && a.bytes < (1u << 31) && a.bytes % 256 == 0 && a.n > 0, "copy sizes");
    return hipSuccess;
}
hipError_t launch_attn_shared(int, int, const AttnSharedArgs& a, hipStream_t) {
    ++g_launches;
    expect((long long)a.max_pages * a.page <= (1 << 29) && a.nprefix >= 1 && a.nown >= 1 && a.nprefix + a.nown <= kMaxSplits, "shared sizes");
    const u64 each = (u64)a.Tq * a.G, own = (u64)a.B * a.HK * a.nown * ((each + 16 * a.own_blocks - 1) / (16 * a.own_blocks));
    expect(a.prefix_blocks >= 0 && a.prefix_blocks + own < (1ull << 23) && (u64)a.B * each <= (1ull << 29), "shared grid");
    expect(a.part_o && a.part_ml, "shared partials");
    return hipSuccess;
}
hipError_t launch_state_reorder(const ReorderArgs& a, hipStream_t) {
    ++g_launches;
    const u64 pieces = a.out == a.state ? (u64)a.R * (a.row_bytes / 2048 + 1) : (u64)a.R * a.K_out * (a.row_bytes / 16384 + 1);
    expect(pieces < (1ull << 24) && a.row_bytes % 16 == 0 && (a.out != a.state || a.K_out <= kReorderMost), "reorder grid");
    return hipSuccess;
}
hipError_t launch_beam_select(int dt, const SelectArgs& a, hipStream_t) {
    ++g_launches;
    const int per = select_part(a.V, a.nsplit, dt == 1 ? 8 : 4);
    expect(a.nsplit >= 1 && a.nsplit <= 64 && a.K * a.nsplit * a.M <= kSelectHeld && (u64)a.R * a.K * a.nsplit < (1ull << 24), "select grid");
    expect((long long)(a.nsplit - 1) * per < a.V && (long long)a.nsplit * per >= a.V, "select parts");
    expect(a.ld >= (size_t)a.V && a.stat && a.part_x && a.part_w, "select buffers");
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
    expect(st >= KDA_OK && st <= KDA_ERR_SCALE, "known status");
}

int main() {
    static const int dims[] = {16, 32, 64, 128}, pages[] = {16, 32, 64, 128};
    static const float scales[] = {1.f, 0.125f, 0.f, -1.f, INFINITY, NAN, 3e38f, 1e-40f};
    long accepted = 0;
    for (int i = 0; i < 400000; ++i) {
        const int B = some(4), T = some(2), HK = some(2), H = draw(4) ? (HK > 0 && HK < 4096 ? HK * 4 : 4) : any_int();
        const int D = draw(6) ? dims[draw(4)] : any_int(), page = draw(6) ? pages[draw(4)] : any_int();
        const int np = some(64), mp = some(8), K = some(4), K2 = some(4), V = some(1000), M = some(8);
        const kda_dtype dt = (kda_dtype)(draw(12) ? draw(2) : 3);
        const float sc = draw(4) ? 0.125f : scales[draw(8)];
        const int ld = draw(4) ? 0 : any_int(), win = draw(3) ? 0 : any_int();
        void* ws = at<void>(14);
        const size_t wsb = draw(4) ? (size_t)1 << 60 : draw(1000);
        const int before = g_launches;
        switch (i % 8) {
            case 0:
                one(kda_cache_fork(at<int>(1), at<int>(2), at<int>(3), at<int>(4), at<int>(5), at<int>(6), B, K, K2, mp, np, page,
                                   draw(2), nullptr), before);
                break;
            case 1:
                one(kda_cache_reserve(at<int>(1), at<int>(2), at<int>(3), at<int>(4), at<int>(5), at<int>(6), at<int>(7), B, T, mp, np,
                                      page, nullptr), before);
                break;
            case 2:
                one(kda_cache_free(at<int>(1), at<int>(2), at<int>(3), at<int>(4), B, mp, np, page, nullptr), before);
                break;
            case 3:
                one(kda_cache_compact(at<int>(1), at<int>(2), at<int>(draw(3) ? 3 : 1), at<int>(draw(3) ? 4 : 2), at<int>(5), at<int>(6),
                                      at<int>(7), at<int>(8), B, mp, np, nullptr), before);
                break;
            case 4: {
                const int o = draw(3) ? 4 : 0;
                one(kda_cache_copy(at<void>(1), at<void>(2), at<float>(3), at<float>(4), at<void>(1 + o), at<void>(2 + o),
                                   at<float>(3 + o), at<float>(4 + o), at<int>(9), at<int>(10), at<int>(11), some(5), np,
                                   draw(2) ? np : some(64), HK, D, page, nullptr), before);
                break;
            }
            case 5:
                one(kda_attn_shared(at<void>(1), at<void>(2), at<void>(3), at<float>(4), at<float>(5), at<int>(6), at<int>(7), at<int>(8),
                                    at<int>(9), at<int>(10), at<void>(11), some(2), np, mp, B, T, H, HK, D, page, ld, sc, win, dt, ws, wsb,
                                    nullptr), before);
                (void)kda_attn_shared_workspace(B, T, H, HK, D, some(2), some(4096));
                break;
            case 6:
                one(kda_state_reorder(at<void>(1), at<void>(draw(3) ? 2 : 1), at<int>(3), B, K, draw(2) ? K : K2,
                                      (size_t)some(4096) * (draw(8) ? 16 : 1), nullptr), before);
                break;
            default:
                one(kda_beam_select(at<void>(1), at<float>(2), at<unsigned char>(3), at<float>(4), at<int>(5), at<int>(6), B, K, V, M, ld,
                                    some(3), dt, ws, wsb, nullptr), before);
                (void)kda_beam_select_workspace(B, K, V, M, dt);
        }
        accepted += g_launches - before;
    }
    expect(accepted > 10000, "enough accepted calls");
    if (g_failures) return 1;
    printf("all expectations hold (%ld calls accepted)\n", accepted);
    return 0;
}
