// kda_attn_api.cpp - the C ABI of the softmax-attention operators: host
// validation, sizing and dispatch.  As in kda_api.cpp, every argument is checked
// before anything is enqueued and a rejected call makes no HIP call.
#include <limits.h>
#include <math.h>

#include "kda_attn.h"
#include "kda_validate.h"

using namespace kda::host;

namespace {

constexpr double kPi = 3.14159265358979323846;
constexpr double kLog2eD = 1.44269504088896340736;

bool heads_ok(int H, int HK) { return H >= 0 && HK >= 0 && (H == 0 || (HK > 0 && H % HK == 0)); }

bool rows_ok(int B, int Tq, int H, int HK) {
    if (!heads_ok(H, HK) || !sizes_ok(B, Tq, H)) return false;
    if (H == 0) return true;
    // packed rows of one key/value head, and less than 2^24 workgroups of 32 of them
    // (a grid holds less than 2^32 threads, a workgroup 256)
    const unsigned long long rows = (unsigned long long)(H / HK) * Tq;
    return rows <= (1ull << 29) && (unsigned long long)B * HK * (rows / 32 + 1) < (1ull << 24);
}

// Keys in one piece: as many workgroups of them in the backward.
bool attn_sizes_ok(int B, int Tq, int Tk, int H, int HK) {
    if (!rows_ok(B, Tq, H, HK) || !sizes_ok(B, Tk, HK)) return false;
    return Tk <= (1 << 29) && (unsigned long long)B * HK * ((unsigned long long)Tk / 32 + 1) < (1ull << 24);
}

// The backward has a thread for each 16 bytes of a row of o, rows padded, and 128 more for
// each head (two waves for its first rows).
bool row_pieces_ok(int B, int Tq, int H, int D, kda_dtype dt) {
    return (unsigned long long)B * H * (((unsigned long long)Tq + kda::kAttnRowPad) * (D * elem_bytes(dt) / 16) + 256) < (1ull << 32);
}

// A paged cache: its length only bounds a loop.
bool step_sizes_ok(int B, int Tq, int H, int HK, int max_len) {
    return max_len >= 0 && max_len <= (1 << 29) && rows_ok(B, Tq, H, HK);
}

using kda::kTileStride;

// Row stride in elements, at most `most`: 0 selects contiguous tokens.
kda_status stride(int ld, int most, int heads, int D, kda_dtype dt, size_t* out) {
    const long long least = (long long)heads * D;
    if (ld < 0 || (ld > 0 && ld < least) || ld > most || least > kTileStride) return KDA_ERR_SHAPE;
    *out = ld ? (size_t)ld : (size_t)least;
    return (*out * elem_bytes(dt)) % 16 == 0 ? KDA_OK : KDA_ERR_ALIGN;
}

Rows rows_of(const void* p, size_t tokens, size_t ld, size_t heads, size_t D, kda_dtype dt) {
    const size_t e = (size_t)elem_bytes(dt);
    return Rows{p, tokens, ld * e, heads * D * e};
}
// n bytes in one piece, for comparison with strided rows
Rows bytes_of(const void* p, size_t n) { return Rows{p, n ? (size_t)1 : 0, n, n}; }

bool overlaps_any(const Rows& out, const Rows* in, size_t n) {
    for (size_t i = 0; i < n; ++i)
        if (overlaps(out, in[i])) return true;
    return false;
}

kda_status check_workspace(const void* ws, size_t have, size_t want) {
    if (want == 0) return KDA_OK;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || have < want) return KDA_ERR_WORKSPACE;
    return KDA_OK;
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// Partial results of a key axis split over n workgroups: n x rows outputs of D
// floats, then as many (maximum, sum) pairs.
size_t split_bytes(int n, size_t rows, int D) {
    return n <= 1 ? 0 : round256((size_t)n * rows * D * 4) + round256((size_t)n * rows * 8);
}

// Queries per head in the backward's row array.
size_t padded_rows(int Tq) { return ((size_t)Tq + kda::kAttnRowPad - 1) / kda::kAttnRowPad * kda::kAttnRowPad; }

// The kernels use it times log2 e, the backward lse over it.
bool scale_ok(float s) { return s >= 0x1p-64f && isfinite((float)(s * kLog2eD)); }

// A window as long as the key axis hides nothing.
int clamp_window(int w, int keys) { return w >= keys ? 0 : w; }

}  // namespace

extern "C" {

kda_status kda_rotary_freqs(double* inv_freq, float* scale, int rot, double base, int kind, double factor,
                            int trained, double beta_fast, double beta_slow) {
    if (rot < 2 || rot % 2 != 0 || rot > 128 || kind < KDA_ROTARY_NONE || kind > KDA_ROTARY_YARN) return KDA_ERR_SHAPE;
    if (!isfinite(base) || base <= 1.0) return KDA_ERR_SCALE;
    if (kind != KDA_ROTARY_NONE && (!isfinite(factor) || factor < 1.0)) return KDA_ERR_SCALE;
    if (kind == KDA_ROTARY_YARN) {
        if (trained < 1) return KDA_ERR_SHAPE;
        if (!isfinite(beta_fast) || !isfinite(beta_slow) || !(beta_fast > beta_slow) || !(beta_slow > 0.0))
            return KDA_ERR_SCALE;
    }
    if (!inv_freq) return KDA_ERR_NULL;
    if (kind == KDA_ROTARY_NTK && rot > 2) base *= pow(factor, (double)rot / (rot - 2));
    double lo = 0.0, hi = 0.0;
    if (kind == KDA_ROTARY_YARN) {
        // the index whose frequency turns n times within the trained length:
        // trained base^(-2i/rot) = 2 pi n
        const double per = rot / (2.0 * log(base));
        lo = floor(per * log(trained / (beta_fast * 2.0 * kPi)));
        hi = ceil(per * log(trained / (beta_slow * 2.0 * kPi)));
        if (lo < 0.0) lo = 0.0;
        if (hi > rot - 1) hi = rot - 1;
    }
    const double width = hi - lo > 1e-3 ? hi - lo : 1e-3;
    for (int i = 0; i < rot / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot);
        double r = 0.0;  // share of the frequency divided by factor
        if (kind == KDA_ROTARY_LINEAR) r = 1.0;
        if (kind == KDA_ROTARY_YARN) {
            r = (i - lo) / width;
            r = r < 0.0 ? 0.0 : r > 1.0 ? 1.0 : r;
        }
        inv_freq[i] = r == 0.0 ? f : f / factor * r + f * (1.0 - r);
    }
    if (scale) *scale = kind == KDA_ROTARY_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    return KDA_OK;
}

kda_status kda_rotary(const void* q, const void* k, void* q_out, void* k_out, const int* positions,
                      const double* inv_freq, int B, int T, int H, int HK, int D, int rot,
                      int ldq, int ldk, int ldqo, int ldko, float scale, unsigned mode, kda_dtype dt,
                      hipStream_t stream) {
    if (!dtype_ok(dt) || (mode & ~(KDA_ROTARY_INTERLEAVED | KDA_ROTARY_INVERSE))) return KDA_ERR_DTYPE;
    if (!k) HK = 0;
    if (!dim_ok(D) || rot < 2 || rot % 2 != 0 || rot > D || H < 0 || HK < 0 || !sizes_ok(B, T, (long long)H + HK))
        return KDA_ERR_SHAPE;
    if (!isfinite(scale)) return KDA_ERR_SCALE;
    kda::RotaryArgs a{};
    KDA_TRY(stride(ldq, INT_MAX, H, D, dt, &a.ldq)); KDA_TRY(stride(ldqo, INT_MAX, H, D, dt, &a.ldqo));
    if (HK) { KDA_TRY(stride(ldk, INT_MAX, HK, D, dt, &a.ldk)); KDA_TRY(stride(ldko, INT_MAX, HK, D, dt, &a.ldko)); }
    a.tokens = (size_t)B * T;
    if (a.tokens == 0 || H + HK == 0) return KDA_OK;
    // a grid holds less than 2^32 threads: at most one for each channel of a token
    if (a.tokens * (unsigned long long)D >= (1ull << 32)) return KDA_ERR_SHAPE;
    if (H) { KDA_TRY(need(q)); KDA_TRY(need(q_out)); }
    if (HK) { KDA_TRY(need(k)); KDA_TRY(need(k_out)); }
    KDA_TRY(need(inv_freq)); KDA_TRY(maybe(positions));
    const Rows rq = rows_of(q, H ? a.tokens : 0, a.ldq, H, D, dt), rk = rows_of(k, HK ? a.tokens : 0, a.ldk, HK, D, dt);
    const Rows qo = rows_of(q_out, H ? a.tokens : 0, a.ldqo, H, D, dt);
    const Rows ko = rows_of(k_out, HK ? a.tokens : 0, a.ldko, HK, D, dt);
    const Rows rest[] = {bytes_of(positions, a.tokens * 4), bytes_of(inv_freq, (size_t)rot * 4)};
    const bool q_same = q_out == q && a.ldqo == a.ldq, k_same = k_out == k && a.ldko == a.ldk;
    if ((!q_same && overlaps(qo, rq)) || (!k_same && overlaps(ko, rk)) || overlaps(qo, rk) || overlaps(ko, rq) ||
        overlaps(qo, ko) || overlaps_any(qo, rest, 2) || overlaps_any(ko, rest, 2))
        return KDA_ERR_SHAPE;
    a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out; a.positions = positions; a.inv_freq = inv_freq;
    a.T = T; a.H = H; a.HK = HK; a.D = D; a.rot = rot; a.scale = scale;
    a.interleaved = (mode & KDA_ROTARY_INTERLEAVED) != 0;
    a.inverse = (mode & KDA_ROTARY_INVERSE) != 0;
    return kda::launch_rotary(dt == KDA_BF16 ? 1 : 0, a, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_attn_fwd_workspace(int B, int Tq, int Tk, int H, int HK, int D, kda_dtype dt) {
    if (!dtype_ok(dt) || !dim_ok(D) || !attn_sizes_ok(B, Tq, Tk, H, HK) || B == 0 || H == 0 || Tq == 0) return 0;
    const int n = kda::attn_fwd_splits(elem_bytes(dt), B, Tq, Tk, HK, H / HK);
    return split_bytes(n, (size_t)B * Tq * H, D);
}

kda_status kda_attn_fwd(const void* q, const void* k, const void* v, const int* q_len, const int* kv_len,
                        void* o, float* lse, int B, int Tq, int Tk, int H, int HK, int D,
                        int ldq, int ldk, int ldv, float scale, int causal, int window, kda_dtype dt,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dtype_ok(dt)) return KDA_ERR_DTYPE;
    if (!dim_ok(D) || !attn_sizes_ok(B, Tq, Tk, H, HK) || window < 0) return KDA_ERR_SHAPE;
    if (!scale_ok(scale)) return KDA_ERR_SCALE;
    kda::AttnArgs a{};
    KDA_TRY(stride(ldq, INT_MAX, H, D, dt, &a.ldq)); KDA_TRY(stride(ldk, kTileStride, HK, D, dt, &a.ldk));
    KDA_TRY(stride(ldv, kTileStride, HK, D, dt, &a.ldv));
    if (B == 0 || H == 0 || Tq == 0) return KDA_OK;
    KDA_TRY(need(q)); KDA_TRY(need(o)); KDA_TRY(maybe(lse)); KDA_TRY(maybe(q_len)); KDA_TRY(maybe(kv_len));
    if (Tk > 0) { KDA_TRY(need(k)); KDA_TRY(need(v)); }
    const size_t want = kda_attn_fwd_workspace(B, Tq, Tk, H, HK, D, dt);
    KDA_TRY(check_workspace(workspace, workspace_bytes, want));
    const size_t nq = (size_t)B * Tq, nk = (size_t)B * Tk;
    const Rows in[] = {rows_of(q, nq, a.ldq, H, D, dt), rows_of(k, nk, a.ldk, HK, D, dt), rows_of(v, nk, a.ldv, HK, D, dt),
                       bytes_of(q_len, (size_t)B * 4), bytes_of(kv_len, (size_t)B * 4), bytes_of(workspace, want)};
    const Rows ro = rows_of(o, nq, (size_t)H * D, H, D, dt), rl = bytes_of(lse, nq * H * 4);
    if (overlaps_any(ro, in, 6) || overlaps_any(rl, in, 6) || overlaps(ro, rl)) return KDA_ERR_SHAPE;
    a.q = q; a.k = k; a.v = v; a.q_len = q_len; a.kv_len = kv_len; a.o = o; a.lse = lse;
    a.B = B; a.Tq = Tq; a.Tk = Tk; a.H = H; a.HK = HK; a.G = H / HK;
    a.scale = scale; a.scale_log2 = (float)(scale * kLog2eD);
    a.causal = causal ? 1 : 0; a.window = clamp_window(window, Tk);
    a.divG = kda::fast_div((uint32_t)a.G);
    a.nsplit = kda::attn_fwd_splits(elem_bytes(dt), B, Tq, Tk, HK, a.G);
    if (a.nsplit > 1) {
        a.part_o = reinterpret_cast<float*>(workspace);
        a.part_ml = a.part_o + round256((size_t)a.nsplit * nq * H * D * 4) / 4;
    }
    return kda::launch_attn_fwd(dt == KDA_BF16 ? 1 : 0, D, a, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_attn_bwd_workspace(int B, int Tq, int Tk, int H, int HK, int D, kda_dtype dt) {
    if (!dtype_ok(dt) || !dim_ok(D) || !attn_sizes_ok(B, Tq, Tk, H, HK) || B == 0 || H == 0 || Tq == 0 ||
        !row_pieces_ok(B, Tq, H, D, dt))
        return 0;
    return round256((size_t)B * H * padded_rows(Tq) * 8);
}

kda_status kda_attn_bwd(const void* q, const void* k, const void* v, const int* q_len, const int* kv_len,
                        const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                        int B, int Tq, int Tk, int H, int HK, int D, int ldq, int ldk, int ldv,
                        float scale, int causal, int window, kda_dtype dt,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dtype_ok(dt)) return KDA_ERR_DTYPE;
    if (!dim_ok(D) || !attn_sizes_ok(B, Tq, Tk, H, HK) || !row_pieces_ok(B, Tq, H, D, dt) || window < 0)
        return KDA_ERR_SHAPE;
    if (!scale_ok(scale)) return KDA_ERR_SCALE;
    kda::AttnArgs a{};
    KDA_TRY(stride(ldq, kTileStride, H, D, dt, &a.ldq)); KDA_TRY(stride(ldk, kTileStride, HK, D, dt, &a.ldk));
    KDA_TRY(stride(ldv, kTileStride, HK, D, dt, &a.ldv));
    if (B == 0 || H == 0 || (Tq == 0 && Tk == 0)) return KDA_OK;
    if (Tq > 0) { KDA_TRY(need(q)); KDA_TRY(need(o)); KDA_TRY(need(lse)); KDA_TRY(need(dout)); KDA_TRY(need(dq)); }
    if (Tk > 0) { KDA_TRY(need(k)); KDA_TRY(need(v)); KDA_TRY(need(dk)); KDA_TRY(need(dv)); }
    KDA_TRY(maybe(q_len)); KDA_TRY(maybe(kv_len));
    const size_t want = kda_attn_bwd_workspace(B, Tq, Tk, H, HK, D, dt);
    KDA_TRY(check_workspace(workspace, workspace_bytes, want));
    const size_t nq = (size_t)B * Tq, nk = (size_t)B * Tk, cq = (size_t)H * D, ck = (size_t)HK * D;
    const Rows in[] = {rows_of(q, nq, a.ldq, H, D, dt), rows_of(k, nk, a.ldk, HK, D, dt), rows_of(v, nk, a.ldv, HK, D, dt),
                       rows_of(o, nq, cq, H, D, dt), bytes_of(lse, nq * H * 4), rows_of(dout, nq, cq, H, D, dt),
                       bytes_of(q_len, (size_t)B * 4), bytes_of(kv_len, (size_t)B * 4), bytes_of(workspace, want)};
    const Rows rq = rows_of(dq, nq, cq, H, D, dt), rk = rows_of(dk, nk, ck, HK, D, dt), rv = rows_of(dv, nk, ck, HK, D, dt);
    if (overlaps_any(rq, in, 9) || overlaps_any(rk, in, 9) || overlaps_any(rv, in, 9) || overlaps(rq, rk) ||
        overlaps(rq, rv) || overlaps(rk, rv))
        return KDA_ERR_SHAPE;
    a.q = q; a.k = k; a.v = v; a.q_len = q_len; a.kv_len = kv_len;
    a.o = const_cast<void*>(o); a.lse = const_cast<float*>(lse);
    a.dout = dout; a.dq = dq; a.dk = dk; a.dv = dv; a.rows = reinterpret_cast<float*>(workspace);
    a.B = B; a.Tq = Tq; a.Tk = Tk; a.H = H; a.HK = HK; a.G = H / HK;
    a.scale = scale; a.scale_log2 = (float)(scale * kLog2eD);
    a.causal = causal ? 1 : 0; a.window = clamp_window(window, Tk);
    a.whole = causal || window > 0;   // parts of the keys come without either
    a.divG = kda::fast_div((uint32_t)a.G);
    a.nsplit = 1;
    return kda::launch_attn_bwd(dt == KDA_BF16 ? 1 : 0, D, a, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

static bool cache_sizes_ok(int n_pages, int max_pages, int B, int T, int HK, int D, int page) {
    if (!dim_ok(D) || (page != 16 && page != 32 && page != 64 && page != 128)) return false;
    if (n_pages < 0 || max_pages < 0 || !sizes_ok(B, T, HK)) return false;
    return (unsigned long long)n_pages * (unsigned)HK <= (1ull << 30) &&
           (unsigned long long)max_pages * (unsigned)page <= (1ull << 30) &&
           (unsigned long long)B * (unsigned)max_pages <= (1ull << 40);
}

kda_status kda_cache_append(const void* k, const void* v, void* k_cache, void* v_cache,
                            float* k_scale, float* v_scale, const int* block_table,
                            const int* cache_len, const int* new_len, int n_pages, int max_pages,
                            int B, int T, int HK, int D, int page, int ldk, int ldv, kda_dtype dt,
                            hipStream_t stream) {
    if (!dtype_ok(dt)) return KDA_ERR_DTYPE;
    if (HK < 0 || !cache_sizes_ok(n_pages, max_pages, B, T, HK, D, page)) return KDA_ERR_SHAPE;
    kda::AppendArgs a{};
    KDA_TRY(stride(ldk, INT_MAX, HK, D, dt, &a.ldk)); KDA_TRY(stride(ldv, INT_MAX, HK, D, dt, &a.ldv));
    if (B == 0 || T == 0 || HK == 0 || n_pages == 0 || max_pages == 0) return KDA_OK;
    // one workgroup of 256 threads for each page a sequence can touch
    if ((unsigned long long)B * HK * ((unsigned long long)T / page + 2) >= (1ull << 24)) return KDA_ERR_SHAPE;
    KDA_TRY(need(k)); KDA_TRY(need(v)); KDA_TRY(need(k_cache)); KDA_TRY(need(v_cache));
    KDA_TRY(need(k_scale)); KDA_TRY(need(v_scale)); KDA_TRY(need(block_table)); KDA_TRY(need(cache_len));
    KDA_TRY(maybe(new_len));
    const size_t nt = (size_t)B * T, nh = (size_t)n_pages * HK, nc = nh * page * D;
    const Rows in[] = {rows_of(k, nt, a.ldk, HK, D, dt), rows_of(v, nt, a.ldv, HK, D, dt),
                       bytes_of(block_table, (size_t)B * max_pages * 4), bytes_of(cache_len, (size_t)B * 4),
                       bytes_of(new_len, (size_t)B * 4)};
    const Rows out[] = {bytes_of(k_cache, nc), bytes_of(v_cache, nc), bytes_of(k_scale, nh * 4), bytes_of(v_scale, nh * 4)};
    for (int i = 0; i < 4; ++i)
        if (overlaps_any(out[i], in, 5) || overlaps_any(out[i], out + i + 1, 3 - i)) return KDA_ERR_SHAPE;
    a.k = k; a.v = v; a.k_cache = (uint8_t*)k_cache; a.v_cache = (uint8_t*)v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    a.block_table = block_table; a.cache_len = cache_len; a.new_len = new_len;
    a.n_pages = n_pages; a.max_pages = max_pages; a.B = B; a.T = T; a.HK = HK; a.page = page;
    return kda::launch_cache_append(dt == KDA_BF16 ? 1 : 0, D, a, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_attn_step_workspace(int B, int Tq, int H, int HK, int D, int max_len) {
    if (!dim_ok(D) || !step_sizes_ok(B, Tq, H, HK, max_len) || B == 0 || H == 0 || Tq == 0) return 0;
    return split_bytes(kda::attn_step_splits(B, Tq, HK, H / HK, max_len), (size_t)B * Tq * H, D);
}

kda_status kda_attn_step(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                         const float* v_scale, const int* block_table, const int* cache_len,
                         const int* new_len, void* o, int n_pages, int max_pages, int B, int Tq,
                         int H, int HK, int D, int page, int ldq, float scale, int window, kda_dtype dt,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dtype_ok(dt)) return KDA_ERR_DTYPE;
    if (HK < 0 || !cache_sizes_ok(n_pages, max_pages, B, Tq, HK, D, page) || window < 0) return KDA_ERR_SHAPE;
    const int max_len = max_pages * page;
    if (!step_sizes_ok(B, Tq, H, HK, max_len)) return KDA_ERR_SHAPE;
    if (!scale_ok(scale)) return KDA_ERR_SCALE;
    kda::AttnStepArgs a{};
    KDA_TRY(stride(ldq, INT_MAX, H, D, dt, &a.ldq));
    if (B == 0 || H == 0 || Tq == 0) return KDA_OK;
    KDA_TRY(need(q)); KDA_TRY(need(o)); KDA_TRY(need(cache_len)); KDA_TRY(maybe(new_len));
    if (n_pages > 0 && max_pages > 0) {
        KDA_TRY(need(k_cache)); KDA_TRY(need(v_cache)); KDA_TRY(need(k_scale)); KDA_TRY(need(v_scale));
        KDA_TRY(need(block_table));
    }
    const size_t want = kda_attn_step_workspace(B, Tq, H, HK, D, max_len);
    KDA_TRY(check_workspace(workspace, workspace_bytes, want));
    const size_t nq = (size_t)B * Tq, nh = (size_t)n_pages * HK, nc = nh * page * D;
    const Rows in[] = {rows_of(q, nq, a.ldq, H, D, dt), bytes_of(k_cache, nc), bytes_of(v_cache, nc),
                       bytes_of(k_scale, nh * 4), bytes_of(v_scale, nh * 4),
                       bytes_of(block_table, (size_t)B * max_pages * 4), bytes_of(cache_len, (size_t)B * 4),
                       bytes_of(new_len, (size_t)B * 4), bytes_of(workspace, want)};
    if (overlaps_any(rows_of(o, nq, (size_t)H * D, H, D, dt), in, 9)) return KDA_ERR_SHAPE;
    a.q = q; a.k_cache = (const uint8_t*)k_cache; a.v_cache = (const uint8_t*)v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    a.block_table = block_table; a.cache_len = cache_len; a.new_len = new_len; a.o = o;
    a.n_pages = n_pages; a.max_pages = n_pages > 0 ? max_pages : 0; a.B = B; a.Tq = Tq; a.H = H; a.HK = HK; a.G = H / HK;
    a.page = page; a.window = window;   // as it is: a query may stand past the table's last token
    a.scale_log2 = (float)(scale * kLog2eD);
    a.divG = kda::fast_div((uint32_t)a.G);
    a.nsplit = kda::attn_step_splits(B, Tq, HK, a.G, max_len);
    if (a.nsplit > 1) {
        a.part_o = reinterpret_cast<float*>(workspace);
        a.part_ml = a.part_o + round256((size_t)a.nsplit * nq * H * D * 4) / 4;
    }
    return kda::launch_attn_step(dt == KDA_BF16 ? 1 : 0, D, a, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
