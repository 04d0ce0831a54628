// beam_api.cpp - the C ABI of the calls for 4-bit caches, beams and their pages
// (declared in include/gdn.h): argument validation.
#include "../../include/gdn.h"

#include <climits>
#include <cmath>

#include "serving.h"

using namespace gdn;

namespace {

int launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? GDN_OK : set_error(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int check_dtype(int dtype, const char *what) {
    if (dtype != GDN_F32 && dtype != GDN_BF16)
        return set_error(GDN_ERR_UNSUPPORTED, "%s: activation dtype %d not supported (bf16 or fp32)", what, dtype);
    return GDN_OK;
}

int check_stride(int64_t stride, int64_t least, int64_t rows, const char *name) {
    if (stride < least)
        return set_error(GDN_ERR_SHAPE, "%s=%lld is below the row width %lld", name, (long long)stride, (long long)least);
    if (stride > (int64_t(1) << 40) / (rows > 0 ? rows : 1))
        return set_error(GDN_ERR_OVERFLOW, "%s=%lld is out of range", name, (long long)stride);
    return GDN_OK;
}

int check_workspace(const void *ws, size_t have, size_t need, const char *what) {
    if (!ws || ((uintptr_t)ws & 255) != 0)
        return set_error(GDN_ERR_WORKSPACE, "%s: workspace must be a non-NULL 256-byte aligned device pointer", what);
    if (have < need) return set_error(GDN_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", what, have, need);
    return GDN_OK;
}

// Two buffers that overlap without beginning together.
bool apart_or_same(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x == y || x + a_bytes <= y || y + b_bytes <= x;
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// Heads, pages and lengths that both kv4 calls take.
int check_kv4(int N, int HKV, int D, int page_size, int num_pages, const char *what) {
    if (N < 0) return set_error(GDN_ERR_SHAPE, "%s: N=%d is negative", what, N);
    if (HKV < 1 || D < 1) return set_error(GDN_ERR_SHAPE, "%s: head geometry must be positive (HKV=%d D=%d)", what, HKV, D);
    if (D > 256) return set_error(GDN_ERR_SHAPE, "%s: head width D=%d exceeds 256", what, D);
    if (D % 16 != 0) return set_error(GDN_ERR_UNSUPPORTED, "%s: head width D=%d is not a multiple of 16", what, D);
    if (page_size < 1 || num_pages < 1)
        return set_error(GDN_ERR_SHAPE, "%s: page_size=%d and num_pages=%d must be positive", what, page_size, num_pages);
    if (page_size % 16 != 0)
        return set_error(GDN_ERR_UNSUPPORTED, "%s: page_size=%d is not a multiple of 16", what, page_size);
    // (places within a page's block of a head fit 32 bits)
    if (page_size > 1 << 20) return set_error(GDN_ERR_OVERFLOW, "%s: page_size=%d exceeds 2^20", what, page_size);
    if (N > INT_MAX - 1024 || HKV > 32767 || (long)page_size * num_pages > INT_MAX - 1024 ||
        (long)N * HKV > (1L << 40) / (D * 2))
        return set_error(GDN_ERR_OVERFLOW, "%s: N, HKV or page_size * num_pages out of range", what);
    return GDN_OK;
}

int check_pages(int B, int page_size, int max_pages, int num_pages, const char *what) {
    if (B < 1) return set_error(GDN_ERR_SHAPE, "%s: B=%d must be positive", what, B);
    if (B > kPagePlanMaxB) return set_error(GDN_ERR_UNSUPPORTED, "%s: B=%d exceeds %d rows", what, B, kPagePlanMaxB);
    if (page_size < 1 || page_size > 65536 || max_pages < 1 || num_pages < 1)
        return set_error(GDN_ERR_SHAPE, "%s: page_size=%d (1..65536), max_pages=%d and num_pages=%d (>= 1)", what, page_size,
                         max_pages, num_pages);
    if ((long)B * max_pages > INT_MAX || (long)page_size * max_pages > INT_MAX - page_size || num_pages > INT_MAX - 65536)
        return set_error(GDN_ERR_OVERFLOW, "%s: block table, its tokens or num_pages exceed int32", what);
    return GDN_OK;
}

int check_beams(int G, int K, int V, int n) {
    if (G < 1 || K < 1 || V < 1 || n < 1)
        return set_error(GDN_ERR_SHAPE, "beam select: G=%d, K=%d, V=%d and n=%d must be positive", G, K, V, n);
    if (K > kBeamMaxK || n > kBeamMaxN)
        return set_error(GDN_ERR_UNSUPPORTED, "beam select: K=%d beams (at most %d), n=%d selected (at most %d)", K, kBeamMaxK, n,
                         kBeamMaxN);
    if ((long)K * V < n) return set_error(GDN_ERR_SHAPE, "beam select: n=%d exceeds the K * V=%ld candidates", n, (long)K * V);
    if ((long)K * V > INT_MAX || (long)G * K > INT_MAX / 256 || !beam_select_fits(G, K, V, n))
        return set_error(GDN_ERR_OVERFLOW, "beam select: G=%d, K=%d, V=%d are out of range", G, K, V);
    return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_kv4_write(const void *k, const void *v, int64_t k_stride, int64_t v_stride, const int32_t *slots, const float *k_scale,
                  const float *v_scale, void *k_cache, void *v_cache, void *k_out, void *v_out, int N, int HKV, int D,
                  int page_size, int num_pages, int dtype, void *stream) {
    set_error(GDN_OK, "%s", "");
    int rc = check_kv4(N, HKV, D, page_size, num_pages, "kv4 write");
    if (rc) return rc;
    if ((rc = check_dtype(dtype, "kv4 write"))) return rc;
    if ((rc = check_stride(k_stride, (int64_t)HKV * D, N, "k_stride")) || (rc = check_stride(v_stride, (int64_t)HKV * D, N, "v_stride")))
        return rc;
    if (N == 0) return GDN_OK;
    if (!k || !v || !slots || !k_cache || !v_cache) return set_error(GDN_ERR_NULL, "kv4 write: a required pointer is NULL");
    if (!k_out != !v_out) return set_error(GDN_ERR_NULL, "kv4 write: k_out and v_out come together");
    if ((((uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)k_out | (uintptr_t)v_out) & 15) != 0)
        return set_error(GDN_ERR_UNSUPPORTED, "kv4 write: caches and outputs must be 16-byte aligned");
    const Kv4Write p{k, v, (long)k_stride, (long)v_stride, slots, k_scale, v_scale, k_cache, v_cache, k_out, v_out, N, HKV, D,
                     page_size, num_pages, 0, 0};
    return launched(launch_kv4_write(p, dtype, static_cast<cudaStream_t>(stream)), "kv4 write kernel launch");
}

size_t gdn_attention_paged_kv4_workspace_bytes(int B, int N, int H, int HKV, int D, int max_q) {
    if (B < 1 || N < 0 || max_q < 0 || H < 1 || HKV < 1 || H % HKV != 0 || D < 1 || D > 256 || D % 16 != 0 || HKV > 32767) return 0;
    return round256(attention_kv4_workspace(B, N, H, HKV, D, max_q < N ? max_q : N));
}

int gdn_attention_paged_kv4(const void *q, const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                            const int32_t *block_table, const int32_t *kv_lens, const int32_t *offsets, void *out, int B, int N,
                            int H, int HKV, int D, int page_size, int max_pages, int num_pages, int max_q, int64_t q_stride,
                            float scale, int dtype, void *workspace, size_t ws_bytes, void *stream) {
    set_error(GDN_OK, "%s", "");
    int rc = check_kv4(N, HKV, D, page_size, num_pages, "kv4 attention");
    if (rc) return rc;
    if (B < 1) return set_error(GDN_ERR_SHAPE, "kv4 attention: B=%d must be positive", B);
    if (H < 1 || H % HKV != 0)
        return set_error(GDN_ERR_SHAPE, "kv4 attention: query heads H=%d not a multiple of key-value heads HKV=%d", H, HKV);
    if (max_pages < 1 || max_q < 0)
        return set_error(GDN_ERR_SHAPE, "kv4 attention: max_pages=%d must be positive, max_q=%d not negative", max_pages, max_q);
    if ((rc = check_dtype(dtype, "kv4 attention"))) return rc;
    if ((long)N * (H / HKV) > INT_MAX - 1024 || (long)H * D > INT_MAX / 2 || (long)page_size * max_pages > INT_MAX - 1024 ||
        (long)B * HKV > INT_MAX / 4)
        return set_error(GDN_ERR_OVERFLOW, "kv4 attention: rows, heads or page_size * max_pages out of range");
    if ((rc = check_stride(q_stride, (int64_t)H * D, N, "q_stride"))) return rc;
    if (!std::isfinite(scale)) return set_error(GDN_ERR_SHAPE, "kv4 attention: scale must be finite");
    if (N == 0 || max_q == 0) return GDN_OK;
    if (!q || !k_cache || !v_cache || !block_table || !kv_lens || !offsets || !out)
        return set_error(GDN_ERR_NULL, "kv4 attention: a required pointer is NULL");
    if ((((uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out) & 15) != 0)
        return set_error(GDN_ERR_UNSUPPORTED, "kv4 attention: caches and output must be 16-byte aligned");
    rc = check_workspace(workspace, ws_bytes, gdn_attention_paged_kv4_workspace_bytes(B, N, H, HKV, D, max_q), "kv4 attention");
    if (rc) return rc;
    Attn a{};
    a.q = q, a.k = k_cache, a.v = v_cache, a.out = out, a.offsets = offsets;
    a.kv_lens = kv_lens, a.block_table = block_table;
    a.B = B, a.N = N, a.H = H, a.HKV = HKV, a.D = D;
    a.page_size = page_size, a.max_pages = max_pages, a.num_pages = num_pages;
    a.max_q = max_q < N ? max_q : N;
    a.qs = (long)q_stride;
    a.scale = scale == 0.f ? 1.f / std::sqrt((float)D) : scale;
    return launched(launch_attention_kv4(a, k_scale, v_scale, dtype, workspace, static_cast<cudaStream_t>(stream)),
                    "kv4 attention kernel launch");
}

size_t gdn_beam_select_workspace_bytes(int G, int K, int V, int n) {
    return check_beams(G, K, V, n) ? 0 : round256(beam_select_workspace(G, K, V, n));
}

int gdn_beam_select(const void *logits, int64_t row_stride, const float *scores, const uint8_t *finished, int end_token,
                    int keep_rows, int32_t *tokens, int32_t *parents, float *scores_out, uint8_t *finished_out, int G, int K, int V,
                    int n, int dtype, void *workspace, size_t ws_bytes, void *stream) {
    set_error(GDN_OK, "%s", "");
    int rc = check_beams(G, K, V, n);
    if (rc) return rc;
    if ((rc = check_dtype(dtype, "beam select"))) return rc;
    if ((rc = check_stride(row_stride, V, (int64_t)G * K, "row_stride"))) return rc;
    if (keep_rows && n != K)
        return set_error(GDN_ERR_SHAPE, "beam select: keep_rows needs as many selected (n=%d) as beams (K=%d)", n, K);
    if ((finished || finished_out) && (end_token < 0 || end_token >= V))
        return set_error(GDN_ERR_SHAPE, "beam select: end_token=%d outside [0, V=%d)", end_token, V);
    if (!logits || !scores || !tokens || !parents || !scores_out)
        return set_error(GDN_ERR_NULL, "beam select: a required pointer is NULL");
    const int64_t in = (int64_t)G * K, out = (int64_t)G * n;
    if ((n != K && (scores_out == scores || (finished && finished_out == finished))) ||
        !apart_or_same(scores, in * 4, scores_out, out * 4) ||
        (finished && finished_out && !apart_or_same(finished, in, finished_out, out)))
        return set_error(GDN_ERR_SHAPE, "beam select: outputs lie over scores or flags that are still read");
    rc = check_workspace(workspace, ws_bytes, gdn_beam_select_workspace_bytes(G, K, V, n), "beam select");
    if (rc) return rc;
    const BeamSelect p{logits, (long)row_stride, scores, finished, end_token, keep_rows != 0, tokens, parents, scores_out,
                       finished_out, G, K, V, n};
    return launched(launch_beam_select(p, dtype, workspace, static_cast<cudaStream_t>(stream)), "beam select kernel launch");
}

int gdn_state_reorder(void *const *states, const int64_t *row_bytes, int count, const int32_t *parents, int B, void *stream) {
    set_error(GDN_OK, "%s", "");
    if (count < 0 || B < 1) return set_error(GDN_ERR_SHAPE, "state reorder: count=%d, B=%d", count, B);
    if (count > kStateMaxTensors || B > kStateMaxRows)
        return set_error(GDN_ERR_UNSUPPORTED, "state reorder: %d tensors (at most %d) of %d rows (at most %d)", count, kStateMaxTensors,
                         B, kStateMaxRows);
    if (count == 0) return GDN_OK;
    if (!states || !row_bytes || !parents) return set_error(GDN_ERR_NULL, "state reorder: a required pointer is NULL");
    StateReorder r{};
    r.count = count, r.B = B, r.parents = parents;
    for (int i = 0; i < count; ++i) {
        if (row_bytes[i] < 0) return set_error(GDN_ERR_SHAPE, "state reorder: row_bytes[%d] is negative", i);
        if (row_bytes[i] > (int64_t(1) << 40) / B) return set_error(GDN_ERR_OVERFLOW, "state reorder: row_bytes[%d] is out of range", i);
        if (!states[i] && row_bytes[i] > 0) return set_error(GDN_ERR_NULL, "state reorder: states[%d] is NULL", i);
        for (int j = 0; j < i; ++j)
            if (row_bytes[i] > 0 && row_bytes[j] > 0 &&
                (states[i] == states[j] || !apart_or_same(states[i], row_bytes[i] * B, states[j], row_bytes[j] * B)))
                return set_error(GDN_ERR_SHAPE, "state reorder: states[%d] and states[%d] overlap", j, i);
        r.states[i] = states[i], r.row_bytes[i] = (long)row_bytes[i];
    }
    return launched(launch_state_reorder(r, static_cast<cudaStream_t>(stream)), "state reorder kernel launch");
}

size_t gdn_page_fork_workspace_bytes(int B, int max_pages, int num_pages) {
    return check_pages(B, 1, max_pages, num_pages, "page fork") ? 0 : round256(page_fork_workspace(B, max_pages, num_pages));
}

int gdn_page_fork(const int32_t *parents, const int32_t *kv_lens, const int32_t *block_table, int32_t *free_pages,
                  const int32_t *cursor, int32_t *table_out, int32_t *kv_lens_out, int32_t *copies, int32_t *cursor_out,
                  int32_t *status, int B, int B_out, int page_size, int max_pages, int num_pages, int n_free, void *workspace,
                  size_t ws_bytes, void *stream) {
    set_error(GDN_OK, "%s", "");
    int rc = check_pages(B, page_size, max_pages, num_pages, "page fork");
    if (rc || (rc = check_pages(B_out, page_size, max_pages, num_pages, "page fork"))) return rc;
    if (n_free < 0) return set_error(GDN_ERR_SHAPE, "page fork: n_free=%d is negative", n_free);
    if (!parents || !kv_lens || !block_table || (n_free > 0 && !free_pages) || !cursor || !table_out || !kv_lens_out || !copies ||
        !cursor_out || !status)
        return set_error(GDN_ERR_NULL, "page fork: a required pointer is NULL");
    if (((uintptr_t)copies & 7) != 0) return set_error(GDN_ERR_UNSUPPORTED, "page fork: copies must be 8-byte aligned");
    const int64_t in = (int64_t)B * max_pages * 4, out = (int64_t)B_out * max_pages * 4;
    if ((B != B_out && (table_out == block_table || kv_lens_out == kv_lens)) || !apart_or_same(block_table, in, table_out, out) ||
        !apart_or_same(kv_lens, B * 4L, kv_lens_out, B_out * 4L))
        return set_error(GDN_ERR_SHAPE, "page fork: outputs lie over a table or lengths that are still read");
    rc = check_workspace(workspace, ws_bytes, gdn_page_fork_workspace_bytes(B, max_pages, num_pages), "page fork");
    if (rc) return rc;
    const PageFork p{parents, kv_lens, block_table, free_pages, cursor, table_out, kv_lens_out, copies, cursor_out, status, B, B_out,
                     page_size, max_pages, num_pages, n_free};
    return launched(launch_page_fork(p, workspace, static_cast<cudaStream_t>(stream)), "page fork kernel launch");
}

size_t gdn_page_compact_workspace_bytes(int num_pages) {
    return num_pages < 1 || num_pages > INT_MAX - 65536 ? 0 : round256(page_compact_workspace(num_pages));
}

int gdn_page_compact(const int32_t *kv_lens, const int32_t *block_table, int32_t *table_out, int32_t *copies, int32_t *free_pages,
                     int32_t *cursor_out, int32_t *status, int B, int page_size, int max_pages, int num_pages, void *workspace,
                     size_t ws_bytes, void *stream) {
    set_error(GDN_OK, "%s", "");
    int rc = check_pages(B, page_size, max_pages, num_pages, "page compact");
    if (rc) return rc;
    if (!kv_lens || !block_table || !table_out || (num_pages > 1 && !copies) || !free_pages || !cursor_out || !status)
        return set_error(GDN_ERR_NULL, "page compact: a required pointer is NULL");
    if (((uintptr_t)copies & 7) != 0) return set_error(GDN_ERR_UNSUPPORTED, "page compact: copies must be 8-byte aligned");
    const int64_t table = (int64_t)B * max_pages * 4;
    if (!apart_or_same(block_table, table, table_out, table))
        return set_error(GDN_ERR_SHAPE, "page compact: table_out lies over a part of block_table");
    rc = check_workspace(workspace, ws_bytes, gdn_page_compact_workspace_bytes(num_pages), "page compact");
    if (rc) return rc;
    const PageCompact p{kv_lens, block_table, table_out, copies, free_pages, cursor_out, status, B, page_size, max_pages, num_pages};
    return launched(launch_page_compact(p, workspace, static_cast<cudaStream_t>(stream)), "page compact kernel launch");
}

int gdn_page_copy(void *const *caches, const int64_t *page_bytes, int count, const int32_t *copies, int n, int num_pages,
                  void *stream) {
    set_error(GDN_OK, "%s", "");
    if (count < 0 || n < 0 || num_pages < 0)
        return set_error(GDN_ERR_SHAPE, "page copy: count=%d, n=%d and num_pages=%d must not be negative", count, n, num_pages);
    if (count > kPageMaxCaches) return set_error(GDN_ERR_UNSUPPORTED, "page copy: %d caches (at most %d)", count, kPageMaxCaches);
    if (count == 0 || n == 0 || num_pages == 0) return GDN_OK;
    if (!caches || !page_bytes || !copies) return set_error(GDN_ERR_NULL, "page copy: a required pointer is NULL");
    if (((uintptr_t)copies & 7) != 0) return set_error(GDN_ERR_UNSUPPORTED, "page copy: copies must be 8-byte aligned");
    PageCopy c{};
    c.count = count, c.n = n, c.num_pages = num_pages, c.copies = copies;
    for (int i = 0; i < count; ++i) {
        if (page_bytes[i] < 0) return set_error(GDN_ERR_SHAPE, "page copy: page_bytes[%d] is negative", i);
        if (page_bytes[i] > (int64_t(1) << 32)) return set_error(GDN_ERR_OVERFLOW, "page copy: page_bytes[%d] is out of range", i);
        if (!caches[i] && page_bytes[i] > 0) return set_error(GDN_ERR_NULL, "page copy: caches[%d] is NULL", i);
        c.caches[i] = caches[i], c.page_bytes[i] = (long)page_bytes[i];
    }
    return launched(launch_page_copy(c, static_cast<cudaStream_t>(stream)), "page copy kernel launch");
}

}  // extern "C"
