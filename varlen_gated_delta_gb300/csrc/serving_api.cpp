// serving_api.cpp - the C ABI of the softmax-attention serving calls (declared
// in include/gdn.h): argument validation and kernel choice.
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

int check_geometry(int N, int H, int HKV, int D, const char *what) {
    if (N < 0) return set_error(GDN_ERR_SHAPE, "%s: N=%d is negative", what, N);
    if (N > INT_MAX - 1024) return set_error(GDN_ERR_OVERFLOW, "%s: N=%d is out of range", what, N);
    if (H < 1 || HKV < 1 || D < 1)
        return set_error(GDN_ERR_SHAPE, "%s: head geometry must be positive (H=%d HKV=%d D=%d)", what, H, HKV, D);
    if (D > 256) return set_error(GDN_ERR_SHAPE, "%s: head width D=%d exceeds 256", what, D);
    if (H % HKV != 0)
        return set_error(GDN_ERR_SHAPE, "%s: query heads H=%d not a multiple of key-value heads HKV=%d", what, H, HKV);
    if ((long)N * (H / HKV) > INT_MAX - 1024)
        return set_error(GDN_ERR_OVERFLOW, "%s: N*H/HKV rows exceed int32", what);
    if (HKV > 65535) return set_error(GDN_ERR_OVERFLOW, "%s: HKV=%d exceeds 65535", what, HKV);
    if ((long)H * D > INT_MAX / 2) return set_error(GDN_ERR_OVERFLOW, "%s: H*D exceeds its range", what);
    return GDN_OK;
}

int check_stride(int64_t stride, int64_t least, int N, const char *name) {
    if (stride < least)
        return set_error(GDN_ERR_SHAPE, "%s=%lld is below the row width %lld", name, (long long)stride, (long long)least);
    if (stride > (int64_t(1) << 40) / (N > 0 ? N : 1))
        return set_error(GDN_ERR_OVERFLOW, "%s=%lld is out of range", name, (long long)stride);
    return GDN_OK;
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

extern "C" {

int gdn_page_plan(const int32_t *new_lens, const int32_t *cached_lens, int32_t *block_table,
                  const int32_t *free_pages, const int32_t *cursor, int32_t *offsets,
                  int32_t *kv_lens, int32_t *positions, int32_t *slots, int32_t *cursor_out,
                  int32_t *status, int B, int N, int page_size, int max_pages, int n_free,
                  void *stream) {
    set_error(GDN_OK, "%s", "");
    if (B < 1 || N < 0) return set_error(GDN_ERR_SHAPE, "page plan: B=%d, N=%d", B, N);
    if (B > kPagePlanMaxB)
        return set_error(GDN_ERR_UNSUPPORTED, "page plan: B=%d exceeds %d requests", B, kPagePlanMaxB);
    if (page_size < 1 || page_size > 65536 || max_pages < 1 || n_free < 0)
        return set_error(GDN_ERR_SHAPE, "page plan: page_size=%d (1..65536), max_pages=%d (>= 1), n_free=%d (>= 0)",
                         page_size, max_pages, n_free);
    if (!new_lens || !cached_lens || !block_table || (n_free > 0 && !free_pages) || !cursor || !offsets ||
        !kv_lens || (N > 0 && (!positions || !slots)) || !cursor_out || !status)
        return set_error(GDN_ERR_NULL, "page plan: a required pointer is NULL");
    const PagePlan p{new_lens, cached_lens, block_table, free_pages, cursor, offsets, kv_lens, positions, slots,
                     cursor_out, status, B, N, page_size, max_pages, n_free, 0};
    return launched(launch_page_plan(p, static_cast<cudaStream_t>(stream)), "page plan kernel launch");
}

int gdn_qk_norm_rope(const void *qkv, int64_t row_stride, const float *q_weight,
                     const float *k_weight, float eps, const float *cos_sin,
                     const int32_t *positions, int max_pos, const int32_t *slots, void *q_out,
                     void *k_out, void *k_cache, void *v_cache, int num_slots, int N, int H,
                     int HKV, int D, int R, int style, int dtype, void *stream) {
    set_error(GDN_OK, "%s", "");
    int rc = check_geometry(N, H, HKV, D, "qk norm rope");
    if (rc) return rc;
    if ((rc = check_dtype(dtype, "qk norm rope"))) return rc;
    if (R < 0 || R > D || R % 2 != 0)
        return set_error(GDN_ERR_SHAPE, "qk norm rope: R=%d must be even and in [0, D=%d]", R, D);
    if (style != GDN_ROPE_HALF && style != GDN_ROPE_PAIRS)
        return set_error(GDN_ERR_UNSUPPORTED, "qk norm rope: unknown rotation style %d", style);
    if ((rc = check_stride(row_stride, ((int64_t)H + 2 * HKV) * D, N, "row_stride"))) return rc;
    if (!(eps >= 0.f)) return set_error(GDN_ERR_SHAPE, "qk norm rope: eps must not be negative");
    if (R > 0 && max_pos < 1) return set_error(GDN_ERR_SHAPE, "qk norm rope: max_pos=%d", max_pos);
    if (slots && num_slots < 0) return set_error(GDN_ERR_SHAPE, "qk norm rope: num_slots=%d", num_slots);
    if (N == 0) return GDN_OK;
    if (!qkv || !q_out || (R > 0 && (!cos_sin || !positions)) ||
        (slots && num_slots > 0 && (!k_cache || !v_cache)))
        return set_error(GDN_ERR_NULL, "qk norm rope: a required pointer is NULL");
    const NormRope p{qkv, (long)row_stride, q_weight, k_weight, eps, cos_sin, positions, max_pos, slots, q_out,
                     k_out, k_cache, v_cache, slots ? num_slots : 0, N, H, HKV, D, R, style};
    return launched(launch_qk_norm_rope(p, dtype, static_cast<cudaStream_t>(stream)), "qk norm rope kernel launch");
}

int gdn_attention_varlen(const void *q, const void *k, const void *v, const int32_t *offsets,
                         void *out, int B, int N, int H, int HKV, int D, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, float scale, int dtype,
                         void *stream) {
    set_error(GDN_OK, "%s", "");
    int rc = check_geometry(N, H, HKV, D, "attention");
    if (rc) return rc;
    if (B < 1) return set_error(GDN_ERR_SHAPE, "attention: B=%d must be positive", B);
    if ((rc = check_dtype(dtype, "attention"))) return rc;
    if ((rc = check_stride(q_stride, (int64_t)H * D, N, "q_stride")) ||
        (rc = check_stride(k_stride, (int64_t)HKV * D, N, "k_stride")) ||
        (rc = check_stride(v_stride, (int64_t)HKV * D, N, "v_stride")))
        return rc;
    if (!std::isfinite(scale)) return set_error(GDN_ERR_SHAPE, "attention: scale must be finite");
    if (N == 0) return GDN_OK;
    if (!q || !k || !v || !offsets || !out) return set_error(GDN_ERR_NULL, "attention: a required pointer is NULL");
    Attn a{};
    a.q = q, a.k = k, a.v = v, a.out = out, a.offsets = offsets;
    a.B = B, a.N = N, a.H = H, a.HKV = HKV, a.D = D;
    a.max_q = N;
    a.qs = (long)q_stride, a.ks = (long)k_stride, a.vs = (long)v_stride;
    a.scale = scale == 0.f ? 1.f / std::sqrt((float)D) : scale;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launched(attention_prompt_supported(a, dtype) ? launch_attention_prompt(a, 0, st)
                                                         : launch_attention_f32(a, dtype, st),
                    "attention kernel launch");
}

int gdn_attention_status(void *stream) {
    set_error(GDN_OK, "%s", "");
    cudaError_t e;
    const int late = attention_timeouts(static_cast<cudaStream_t>(stream), &e);
    if (e != cudaSuccess) return launched(e, "attention status");
    return late ? set_error(GDN_ERR_TIMEOUT, "a wait inside an attention kernel gave up") : GDN_OK;
}

int gdn_selftest_attention_timeout(int limit_us, void *stream) {
    set_error(GDN_OK, "%s", "");
    if (limit_us < 1 || limit_us > 1000000)
        return set_error(GDN_ERR_SHAPE, "limit_us=%d outside [1, 1000000]", limit_us);
    return launched(launch_attention_wait_probe(limit_us / 4 + 1, static_cast<cudaStream_t>(stream)), "self-test launch");
}

size_t gdn_attention_paged_workspace_bytes(int B, int N, int H, int HKV, int D, int max_q) {
    if (B < 1 || max_q < 0 || check_geometry(N, H, HKV, D, "attention")) return 0;
    const size_t wide = attention_f32_part_floats(N, H, D) * 4;
    const size_t split = attention_split_workspace(B, H, HKV, D, max_q);
    const size_t prompt = (long)max_q * (H / HKV) > kSplitRows ? attention_prompt_part_floats(B, N, H, HKV, D, max_q < N ? max_q : N) * 4 : 0;
    const size_t most = wide > split ? wide : split;
    return round256(most > prompt ? most : prompt);
}

int gdn_attention_paged(const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *block_table, const int32_t *kv_lens,
                        const int32_t *offsets, void *out, int B, int N, int H, int HKV, int D,
                        int page_size, int max_pages, int num_pages, int max_q, int64_t q_stride,
                        float scale, int dtype, void *workspace, size_t ws_bytes, void *stream) {
    set_error(GDN_OK, "%s", "");
    int rc = check_geometry(N, H, HKV, D, "paged attention");
    if (rc) return rc;
    if (B < 1) return set_error(GDN_ERR_SHAPE, "paged attention: B=%d must be positive", B);
    if ((rc = check_dtype(dtype, "paged attention"))) return rc;
    if (page_size < 1 || max_pages < 1 || num_pages < 1 || max_q < 0)
        return set_error(GDN_ERR_SHAPE, "paged attention: page_size=%d, max_pages=%d, num_pages=%d must be positive, max_q=%d not negative",
                         page_size, max_pages, num_pages, max_q);
    // (room for a tile of keys past the end)
    if ((long)page_size * num_pages > INT_MAX - 1024 || (long)page_size * max_pages > INT_MAX - 1024)
        return set_error(GDN_ERR_OVERFLOW, "paged attention: page_size * num_pages and page_size * max_pages must fit int32");
    if ((rc = check_stride(q_stride, (int64_t)H * D, N, "q_stride"))) return rc;
    if (!std::isfinite(scale)) return set_error(GDN_ERR_SHAPE, "paged attention: scale must be finite");
    if (N == 0 || max_q == 0) return GDN_OK;
    if (!q || !k_cache || !v_cache || !block_table || !kv_lens || !offsets || !out)
        return set_error(GDN_ERR_NULL, "paged attention: a required pointer is NULL");
    const size_t need = gdn_attention_paged_workspace_bytes(B, N, H, HKV, D, max_q);
    if (!workspace || ((uintptr_t)workspace & 255) != 0)
        return set_error(GDN_ERR_WORKSPACE, "paged attention: workspace must be a non-NULL 256-byte aligned device pointer");
    if (ws_bytes < need)
        return set_error(GDN_ERR_WORKSPACE, "paged attention: workspace has %zu bytes, needs %zu", ws_bytes, need);
    Attn a{};
    a.q = q, a.k = k_cache, a.v = v_cache, a.out = out, a.offsets = offsets;
    a.kv_lens = kv_lens, a.block_table = block_table;
    a.B = B, a.N = N, a.H = H, a.HKV = HKV, a.D = D;
    a.page_size = page_size, a.max_pages = max_pages, a.num_pages = num_pages;
    a.max_q = max_q < N ? max_q : N;
    a.qs = (long)q_stride, a.ks = a.vs = (long)HKV * D;
    a.scale = scale == 0.f ? 1.f / std::sqrt((float)D) : scale;
    a.part = static_cast<float *>(workspace);
    a.part_floats = attention_f32_part_floats(N, H, D);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Sequences of few rows run split over their keys, longer ones as prompt slices; a call
    // that may hold both launches both, and each kernel takes its own.
    const bool some_long = (long)a.max_q * (H / HKV) > kSplitRows;
    const bool split = attention_split_supported(a, dtype);
    if (some_long ? !attention_prompt_supported(a, dtype) : !split)
        return launched(launch_attention_f32(a, dtype, st), "paged attention kernel launch");
    if (split) rc = launched(launch_attention_split(a, workspace, st), "split attention kernel launch");
    if (!rc && some_long)
        rc = launched(launch_attention_prompt(a, split ? kSplitRows : 0, st), "prompt attention kernel launch");
    return rc;
}

}  // extern "C"
