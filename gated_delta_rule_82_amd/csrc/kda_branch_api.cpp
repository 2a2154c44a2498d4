// kda_branch_api.cpp - the C ABI of the operators that continue one prompt several
// times: host validation, sizing and dispatch.  As in kda_api.cpp, every argument is
// checked before anything is enqueued and a rejected call makes no HIP call.
#include <limits.h>
#include <math.h>

#include "kda_attn_validate.h"
#include "kda_branch.h"

using namespace kda::host;

namespace {

bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

// Rows of a table, one thread an entry (and one for a row without any).
bool table_ok(long long B, int max_pages, int n_pages) {
    return B >= 0 && max_pages >= 0 && n_pages >= 0 && n_pages <= (1 << 30) && B < (1ll << 30) &&
           B * (max_pages > 0 ? max_pages : 1) < (1ll << 30);
}

Rows ints(const int* p, unsigned long long n) { return bytes_of(p, (size_t)n * 4); }

// Outputs apart from each other and from the inputs.
bool apart(const Rows* out, size_t n_out, const Rows* in, size_t n_in) {
    for (size_t i = 0; i < n_out; ++i)
        if (overlaps_any(out[i], in, n_in) || overlaps_any(out[i], out + i + 1, n_out - i - 1)) return false;
    return true;
}

bool select_sizes_ok(int R, int K, int V, int M) {
    return R >= 0 && K >= 1 && K <= kda::kSelectMost && M >= 1 && M <= kda::kSelectMost && V >= 1 && V <= (1 << 30) &&
           (long long)R * K < (1 << 18);
}

kda_status status_of(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

}  // namespace

extern "C" {

kda_status kda_cache_fork(const int* table, const int* cache_len, const int* parent, int* table_out,
                          int* len_out, int* refs, int R, int K_in, int K_out, int max_pages,
                          int n_pages, int page, int keep, hipStream_t stream) {
    if (!page_ok(page) || R < 0 || K_in < 0 || K_in > 1024 || K_out < 0 || K_out > 1024 ||
        !table_ok((long long)R * K_in, max_pages, n_pages) || !table_ok((long long)R * K_out, max_pages, n_pages))
        return KDA_ERR_SHAPE;
    if (R == 0 || (K_out == 0 && (K_in == 0 || max_pages == 0))) return KDA_OK;    // no entry and no length to write
    const unsigned long long n_in = (unsigned long long)R * K_in, n_out = (unsigned long long)R * K_out;
    if (n_in > 0) KDA_TRY(need(cache_len));
    if (n_out > 0) { KDA_TRY(need(parent)); KDA_TRY(need(len_out)); }
    if (max_pages > 0) {
        if (n_in > 0) KDA_TRY(need(table));
        if (n_out > 0) KDA_TRY(need(table_out));
        if (n_pages > 0) KDA_TRY(need(refs));
    }
    const Rows in[] = {ints(table, n_in * max_pages), ints(cache_len, n_in), ints(parent, n_out)};
    const Rows out[] = {ints(table_out, n_out * max_pages), ints(len_out, n_out), ints(refs, n_pages)};
    if (!apart(out, 3, in, 3)) return KDA_ERR_SHAPE;
    const kda::ForkArgs a{table, cache_len, parent, table_out, len_out, refs, R, K_in, K_out, max_pages, n_pages, page, keep ? 1 : 0};
    return status_of(kda::launch_cache_fork(a, stream));
}

kda_status kda_cache_reserve(int* table, int* refs, const int* cache_len, const int* new_len,
                             int* src, int* dst, int* info, int B, int T, int max_pages, int n_pages,
                             int page, hipStream_t stream) {
    if (!page_ok(page) || T < 0 || !table_ok(B, max_pages, n_pages)) return KDA_ERR_SHAPE;
    const int pages = kda::pages_touched(T, page), width = max_pages > 0 ? max_pages : 1;
    if ((long long)B * pages >= (1ll << 30)) return KDA_ERR_SHAPE;
    const int touched = pages < width ? pages : width;      // entries of a row that there are
    KDA_TRY(need(info));
    if (B > 0) {
        KDA_TRY(need(cache_len)); KDA_TRY(maybe(new_len)); KDA_TRY(need(src)); KDA_TRY(need(dst));
        if (max_pages > 0) KDA_TRY(need(table));
    }
    if (n_pages > 0) KDA_TRY(need(refs));
    const Rows in[] = {ints(cache_len, B), ints(new_len, B)};
    const Rows out[] = {ints(table, (unsigned long long)B * max_pages), ints(refs, n_pages), ints(src, B), ints(dst, B), ints(info, 2)};
    if (!apart(out, 5, in, 2)) return KDA_ERR_SHAPE;
    const kda::ReserveArgs a{table, refs, cache_len, new_len, src, dst, info, B, T, max_pages, n_pages, page, touched};
    return status_of(kda::launch_cache_reserve(a, stream));
}

kda_status kda_cache_free(int* table, int* refs, const int* keep_from, const int* keep_to,
                          int B, int max_pages, int n_pages, int page, hipStream_t stream) {
    if (!page_ok(page) || !table_ok(B, max_pages, n_pages)) return KDA_ERR_SHAPE;
    if (B == 0 || max_pages == 0) return KDA_OK;
    KDA_TRY(need(table)); KDA_TRY(maybe(keep_from)); KDA_TRY(maybe(keep_to));
    if (n_pages > 0) KDA_TRY(need(refs));
    const Rows in[] = {ints(keep_from, B), ints(keep_to, B)};
    const Rows out[] = {ints(table, (unsigned long long)B * max_pages), ints(refs, n_pages)};
    if (!apart(out, 2, in, 2)) return KDA_ERR_SHAPE;
    const kda::FreeArgs a{table, refs, keep_from, keep_to, B, max_pages, n_pages, page};
    return status_of(kda::launch_cache_free(a, stream));
}

kda_status kda_cache_compact(const int* table, const int* refs, int* table_out, int* refs_out,
                             int* remap, int* src, int* dst, int* info, int B, int max_pages,
                             int n_pages, hipStream_t stream) {
    if (!table_ok(B, max_pages, n_pages)) return KDA_ERR_SHAPE;
    const unsigned long long entries = (unsigned long long)B * max_pages;
    KDA_TRY(need(info));
    if (entries > 0) { KDA_TRY(need(table)); KDA_TRY(need(table_out)); }
    if (n_pages > 0) { KDA_TRY(need(refs)); KDA_TRY(need(refs_out)); KDA_TRY(need(remap)); }
    if (n_pages > 1) { KDA_TRY(need(src)); KDA_TRY(need(dst)); }
    const Rows in[] = {ints(table, entries), ints(refs, n_pages)};
    const Rows out[] = {ints(remap, n_pages), ints(src, n_pages / 2), ints(dst, n_pages / 2), ints(info, 2),
                        ints(table_out, entries), ints(refs_out, n_pages)};
    if (!apart(out, 6, nullptr, 0) || !apart(out, 4, in, 2) || overlaps(out[4], in[1]) || overlaps(out[5], in[0]) ||
        (table_out != table && overlaps(out[4], in[0])) || (refs_out != refs && overlaps(out[5], in[1])))
        return KDA_ERR_SHAPE;
    const kda::CompactArgs a{table, refs, table_out, refs_out, remap, src, dst, info, B, max_pages, n_pages};
    return status_of(kda::launch_cache_compact(a, stream));
}

kda_status kda_cache_copy(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                          void* k_to, void* v_to, float* k_scale_to, float* v_scale_to,
                          const int* src, const int* dst, const int* count, int n, int n_src, int n_dst,
                          int HK, int D, int page, hipStream_t stream) {
    if (HK < 0 || n < 0 || !cache_sizes_ok(n_src, 0, 0, 0, HK, D, page) || !cache_sizes_ok(n_dst, 0, 0, 0, HK, D, page) ||
        (long long)HK * page * D >= (1ll << 31))
        return KDA_ERR_SHAPE;
    if (n == 0 || n_src == 0 || n_dst == 0 || HK == 0) return KDA_OK;
    KDA_TRY(need(k_cache)); KDA_TRY(need(v_cache)); KDA_TRY(need(k_scale)); KDA_TRY(need(v_scale));
    KDA_TRY(need(k_to)); KDA_TRY(need(v_to)); KDA_TRY(need(k_scale_to)); KDA_TRY(need(v_scale_to));
    KDA_TRY(need(src)); KDA_TRY(need(dst)); KDA_TRY(maybe(count));
    const bool same = k_cache == k_to && v_cache == v_to && k_scale == k_scale_to && v_scale == v_scale_to;
    if (same && n_src != n_dst) return KDA_ERR_SHAPE;
    const size_t bytes = (size_t)HK * page * D, hs = (size_t)n_src * HK * 4, hd = (size_t)n_dst * HK * 4;
    const Rows lists[] = {ints(src, n), ints(dst, n), ints(count, 1)};
    const Rows from[] = {bytes_of(k_cache, n_src * bytes), bytes_of(v_cache, n_src * bytes), bytes_of(k_scale, hs), bytes_of(v_scale, hs)};
    const Rows to[] = {bytes_of(k_to, n_dst * bytes), bytes_of(v_to, n_dst * bytes), bytes_of(k_scale_to, hd), bytes_of(v_scale_to, hd)};
    if (!apart(to, 4, lists, 3) || (!same && !apart(to, 4, from, 4))) return KDA_ERR_SHAPE;
    const kda::CopyArgs a{(const uint8_t*)k_cache, (const uint8_t*)v_cache, k_scale, v_scale, (uint8_t*)k_to, (uint8_t*)v_to,
                          k_scale_to, v_scale_to, src, dst, count, n, n_src, n_dst, HK, (unsigned)bytes};
    return status_of(kda::launch_cache_copy(a, stream));
}

static bool shared_sizes_ok(int B, int Tq, int H, int HK, int D, int n_groups, int max_len) {
    if (n_groups < 0 || n_groups > (1 << 16) || !step_sizes_ok(B, Tq, H, HK, max_len)) return false;
    // packed rows of all sequences, the workgroups of one launch, and the threads of the join behind it (four
    // channels each where there are few parts; with many there are few rows)
    if (H == 0) return true;
    return (unsigned long long)B * Tq * H * (D / 4) + 255 < (1ull << 32) && (unsigned long long)B * Tq * (H / HK) <= (1ull << 29) &&
           kda::shared_plan(4, B, Tq, HK, H / HK, D, n_groups, max_len).blocks < (1ll << 23) &&
           kda::shared_plan(2, B, Tq, HK, H / HK, D, n_groups, max_len).blocks < (1ll << 23);
}

size_t kda_attn_shared_workspace(int B, int Tq, int H, int HK, int D, int n_groups, int max_len) {
    if (!dim_ok(D) || !shared_sizes_ok(B, Tq, H, HK, D, n_groups, max_len) || B == 0 || H == 0 || Tq == 0) return 0;
    int parts = 0;      // as many as either type needs
    for (int e = 2; e <= 4; e += 2) {
        const kda::SharedPlan p = kda::shared_plan(e, B, Tq, HK, H / HK, D, n_groups, max_len);
        if (p.nprefix + p.nown > parts) parts = p.nprefix + p.nown;
    }
    return split_bytes(parts, (size_t)B * Tq * H, D);
}

kda_status kda_attn_shared(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int* block_table, const int* cache_len,
                           const int* new_len, const int* group_first, const int* prefix_len, void* o,
                           int n_groups, int n_pages, int max_pages, int B, int Tq, int H, int HK, int D,
                           int page, int ldq, float scale, int window, kda_dtype dt,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dtype_ok(dt)) return KDA_ERR_DTYPE;
    if (HK < 0 || !cache_sizes_ok(n_pages, max_pages, B, Tq, HK, D, page) || window < 0) return KDA_ERR_SHAPE;
    const int max_len = max_pages * page;
    if (!shared_sizes_ok(B, Tq, H, HK, D, n_groups, max_len)) return KDA_ERR_SHAPE;
    if (!scale_ok(scale)) return KDA_ERR_SCALE;
    kda::AttnSharedArgs a{};
    KDA_TRY(stride(ldq, INT_MAX, H, D, dt, &a.ldq));
    if (B == 0 || H == 0 || Tq == 0) return KDA_OK;
    KDA_TRY(need(q)); KDA_TRY(need(o)); KDA_TRY(need(cache_len)); KDA_TRY(maybe(new_len));
    if (n_groups > 0) { KDA_TRY(need(group_first)); KDA_TRY(need(prefix_len)); }
    if (n_pages > 0 && max_pages > 0) {
        KDA_TRY(need(k_cache)); KDA_TRY(need(v_cache)); KDA_TRY(need(k_scale)); KDA_TRY(need(v_scale));
        KDA_TRY(need(block_table));
    }
    const size_t want = kda_attn_shared_workspace(B, Tq, H, HK, D, n_groups, max_len);
    KDA_TRY(check_workspace(workspace, workspace_bytes, want));
    const size_t nq = (size_t)B * Tq, nh = (size_t)n_pages * HK, nc = nh * page * D;
    const Rows in[] = {rows_of(q, nq, a.ldq, H, D, dt), bytes_of(k_cache, nc), bytes_of(v_cache, nc),
                       bytes_of(k_scale, nh * 4), bytes_of(v_scale, nh * 4), ints(block_table, (size_t)B * max_pages),
                       ints(cache_len, B), ints(new_len, B), ints(group_first, n_groups > 0 ? n_groups + 1 : 0),
                       ints(prefix_len, n_groups), bytes_of(workspace, want)};
    const Rows ro = rows_of(o, nq, (size_t)H * D, H, D, dt);
    if (overlaps_any(ro, in, 11) || overlaps_any(in[10], in, 10)) return KDA_ERR_SHAPE;
    const kda::SharedPlan p = kda::shared_plan(elem_bytes(dt), B, Tq, HK, H / HK, D, n_groups, max_len);
    a.q = q; a.k_cache = (const uint8_t*)k_cache; a.v_cache = (const uint8_t*)v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    a.block_table = block_table; a.cache_len = cache_len; a.new_len = new_len; a.group_first = group_first;
    a.prefix_len = prefix_len; a.o = o;
    a.n_groups = n_groups; a.n_pages = n_pages; a.max_pages = n_pages > 0 ? max_pages : 0;
    a.B = B; a.Tq = Tq; a.H = H; a.HK = HK; a.G = H / HK; a.page = page; a.window = window;
    a.wide = p.wide; a.own_blocks = p.own_blocks; a.tiles = p.tiles; a.nprefix = p.nprefix; a.nown = p.nown;
    a.prefix_blocks = HK * p.tiles * p.nprefix;
    a.scale_log2 = (float)(scale * kLog2eD);
    a.divG = kda::fast_div((uint32_t)a.G);
    a.divT = kda::fast_div((uint32_t)Tq);
    const size_t parts = (size_t)p.nprefix + p.nown;
    a.part_o = reinterpret_cast<float*>(workspace);
    a.part_ml = a.part_o + round256(parts * nq * H * D * 4) / 4;
    return status_of(kda::launch_attn_shared(dt == KDA_BF16 ? 1 : 0, D, a, stream));
}

kda_status kda_state_reorder(const void* state, void* out, const int* parent, int R, int K_in, int K_out,
                             size_t row_bytes, hipStream_t stream) {
    if (R < 0 || K_in < 0 || K_out < 0 || (long long)R * K_in > (1 << 24) || (long long)R * K_out > (1 << 24) ||
        row_bytes > ((size_t)1 << 40))
        return KDA_ERR_SHAPE;
    if (row_bytes % 16 != 0) return KDA_ERR_ALIGN;
    if (R == 0 || K_out == 0 || row_bytes == 0) return KDA_OK;
    const size_t n_in = (size_t)R * K_in, n_out = (size_t)R * K_out;
    if (n_in > 0) KDA_TRY(need(state));
    KDA_TRY(need(out)); KDA_TRY(need(parent));
    const bool same = out == state;
    if (same ? K_in != K_out || K_out > kda::kReorderMost : overlaps(out, n_out * row_bytes, state, n_in * row_bytes)) return KDA_ERR_SHAPE;
    if (overlaps(out, n_out * row_bytes, parent, n_out * 4)) return KDA_ERR_SHAPE;
    if ((same ? (size_t)R * (row_bytes / 2048 + 1) : n_out * (row_bytes / 16384 + 1)) >= (size_t)1 << 24) return KDA_ERR_SHAPE;
    const kda::ReorderArgs a{(const uint8_t*)state, (uint8_t*)out, parent, R, K_in, K_out, row_bytes};
    return status_of(kda::launch_state_reorder(a, stream));
}

size_t kda_beam_select_workspace(int R, int K, int V, int M, kda_dtype dt) {
    if (!dtype_ok(dt) || !select_sizes_ok(R, K, V, M)) return 0;
    const size_t parts = (size_t)R * K * kda::select_splits(elem_bytes(dt), R, K, V, M);
    return round256(parts * 16) + 2 * round256(parts * M * 4);
}

kda_status kda_beam_select(const void* logits, const float* scores, const unsigned char* done,
                           float* scores_out, int* parent, int* token, int R, int K, int V, int M,
                           int ld, int end, kda_dtype dt, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
    if (!dtype_ok(dt)) return KDA_ERR_DTYPE;
    if (!select_sizes_ok(R, K, V, M) || ld < 0 || (ld > 0 && ld < V) || (done && (end < 0 || end >= V))) return KDA_ERR_SHAPE;
    if (R == 0) return KDA_OK;
    KDA_TRY(need(logits)); KDA_TRY(maybe(scores)); KDA_TRY(maybe(done));
    KDA_TRY(need(scores_out)); KDA_TRY(need(parent)); KDA_TRY(need(token));
    const size_t want = kda_beam_select_workspace(R, K, V, M, dt);
    KDA_TRY(check_workspace(workspace, workspace_bytes, want));
    kda::SelectArgs a{};
    a.ld = ld ? ld : V;
    const size_t rows = (size_t)R * K, picks = (size_t)R * M;
    const Rows in[] = {rows_of(logits, rows, a.ld, 1, V, dt), bytes_of(scores, rows * 4), bytes_of(done, rows), bytes_of(workspace, want)};
    const Rows out[] = {bytes_of(scores_out, picks * 4), ints(parent, picks), ints(token, picks)};
    if (!apart(out, 3, in, 4) || overlaps_any(in[3], in, 3)) return KDA_ERR_SHAPE;
    a.logits = logits; a.scores = scores; a.done = done; a.scores_out = scores_out; a.parent = parent; a.token = token;
    a.R = R; a.K = K; a.V = V; a.M = M; a.end = end;
    a.nsplit = kda::select_splits(elem_bytes(dt), R, K, V, M);
    const size_t parts = rows * a.nsplit;
    a.stat = reinterpret_cast<double*>(workspace);
    a.part_x = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + round256(parts * 16));
    a.part_w = reinterpret_cast<int*>(reinterpret_cast<char*>(a.part_x) + round256(parts * M * 4));
    return status_of(kda::launch_beam_select(dt == KDA_BF16 ? 1 : 0, a, stream));
}

}  // extern "C"
