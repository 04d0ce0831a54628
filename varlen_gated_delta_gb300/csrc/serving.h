// serving.h - host-side interface of the kernels that serve softmax-attention
// layers and beams (page_plan.cu, page_fork.cu, qk_norm_rope.cu, kv4_write.cu,
// attention_*.cu, beam_select.cu, state_reorder.cu), called by serving_api.cpp
// and beam_api.cpp.  Not installed; the public ABI is include/gdn.h.
#pragma once

#include "internal.h"

namespace gdn {

constexpr int kPagePlanMaxB = 8192;  // three ints a request in shared memory

struct PagePlan {
    const int32_t *new_lens, *cached_lens;
    int32_t *block_table;
    const int32_t *free_pages, *cursor;
    int32_t *offsets, *kv_lens, *positions, *slots, *cursor_out, *status;
    int B, N, page_size, max_pages, n_free;
    int wide;  // positions and slots lie on 16-byte boundaries (set by the launcher)
};
cudaError_t launch_page_plan(const PagePlan &p, cudaStream_t s);

struct NormRope {
    const void *qkv;
    long row_stride;  // elements
    const float *qw, *kw;
    float eps;
    const float *cos_sin;
    const int32_t *positions;
    int max_pos;
    const int32_t *slots;
    void *q, *k, *k_cache, *v_cache;
    int num_slots, N, H, HKV, D, R, style;
};
cudaError_t launch_qk_norm_rope(const NormRope &p, int dtype, cudaStream_t s);

// Attention of packed queries over packed keys (block_table NULL: the queries'
// own tokens) or over a paged cache.
struct Attn {
    const void *q, *k, *v;
    void *out;
    const int32_t *offsets;
    const int32_t *kv_lens, *block_table;  // paged only
    int B, N, H, HKV, D;
    int page_size, max_pages, num_pages, max_q;
    long qs, ks, vs;  // token strides in elements (paged: HKV * D for k and v)
    float scale;
    float *part;  // parts of key splits (paged only): [N][H][splits][D], then [N][H][splits][2]
    size_t part_floats;
    const float *out_scale;  // of the joined outputs of each key-value head, or NULL
};

// Whether base and row stride suit 16-byte accesses of every head's row.
inline bool rows_aligned(const void *base, long stride_elems, int D, size_t esz) {
    return ((uintptr_t)base & 15) == 0 && (size_t)stride_elems * esz % 16 == 0 &&
           (size_t)D * esz % 16 == 0;
}

// Any type, head width and alignment, with fp32 accuracy.
size_t attention_f32_part_floats(int N, int H, int D);
cudaError_t launch_attention_f32(const Attn &a, int dtype, cudaStream_t s);

// The output of rows whose keys were split into parts (Attn::part, see attention.cuh) of sequences
// with more than min_rows (query, head of a group) rows.
cudaError_t launch_attention_join(const Attn &a, int splits, int min_rows, int dtype, cudaStream_t s);

// bf16, few rows over long paged histories: sequences of at most kSplitRows
// (query, head of a group) rows, the others are left out.
constexpr int kSplitRows = 64;
bool attention_split_supported(const Attn &a, int dtype);
size_t attention_split_workspace(int B, int H, int HKV, int D, int max_q);
cudaError_t launch_attention_split(const Attn &a, void *ws, cudaStream_t s);

// bf16 on the tensor cores, one item per (query tile pair, head): prompts and
// prompt slices.  Sequences of at most min_rows (query, head of a group) rows
// are left out.
bool attention_prompt_supported(const Attn &a, int dtype);
size_t attention_prompt_part_floats(int B, int N, int H, int HKV, int D, int max_q);
cudaError_t launch_attention_prompt(const Attn &a, int min_rows, cudaStream_t s);
// Synchronises s; non-zero when a bounded wait gave up since the last call for this stream.
int attention_timeouts(cudaStream_t s, cudaError_t *e);
// A kernel whose only wait gives up.
cudaError_t launch_attention_wait_probe(int tries, cudaStream_t s);

// ---------------------------------------------------------------- 4-bit cache (kv4.cuh)

struct Kv4Write {
    const void *k, *v;
    long k_stride, v_stride;  // elements
    const int32_t *slots;
    const float *k_scale, *v_scale;
    void *k_cache, *v_cache, *k_out, *v_out;
    int N, HKV, D, page_size, num_pages;
    int tokens, page_shift;  // of a CTA; log2 of page_size or -1 (set by the launcher)
};
cudaError_t launch_kv4_write(const Kv4Write &p, int dtype, cudaStream_t s);

// bf16 sequences of more than min_rows rows over a 4-bit cache.
cudaError_t launch_attention_prompt_kv4(const Attn &a, const float *ks, int min_rows, cudaStream_t s);

// Any rows; a.k and a.v are the 4-bit caches.
size_t attention_kv4_workspace(int B, int N, int H, int HKV, int D, int max_q);
cudaError_t launch_attention_kv4(const Attn &a, const float *k_scale, const float *v_scale, int dtype, void *ws,
                                 cudaStream_t s);

// ---------------------------------------------------------------- beams

constexpr int kBeamMaxK = 128, kBeamMaxN = 128;  // beams of a group, selected of a group
struct BeamSelect {
    const void *logits;
    long stride;  // elements
    const float *scores;
    const uint8_t *finished;
    int end_token, keep_rows;
    int32_t *tokens, *parents;
    float *scores_out;
    uint8_t *finished_out;
    int G, K, V, n;
};
size_t beam_select_workspace(int G, int K, int V, int n);
bool beam_select_fits(int G, int K, int V, int n);  // in the kernels' integers
cudaError_t launch_beam_select(const BeamSelect &p, int dtype, void *ws, cudaStream_t s);

constexpr int kStateMaxTensors = 64, kStateMaxRows = 4096;  // kernel parameters; 24 bytes a row in shared memory
struct StateReorder {
    void *states[kStateMaxTensors];
    long row_bytes[kStateMaxTensors];
    int count, B;
    const int32_t *parents;
};
cudaError_t launch_state_reorder(const StateReorder &r, cudaStream_t s);

struct PageFork {
    const int32_t *parents, *kv_lens, *block_table;
    int32_t *free_pages;
    const int32_t *cursor;
    int32_t *table_out, *kv_lens_out, *copies, *cursor_out, *status;
    int B, B_out, page_size, max_pages, num_pages, n_free;
};
size_t page_fork_workspace(int B, int max_pages, int num_pages);
cudaError_t launch_page_fork(const PageFork &p, void *ws, cudaStream_t s);

struct PageCompact {
    const int32_t *kv_lens, *block_table;
    int32_t *table_out, *copies, *free_pages, *cursor_out, *status;
    int B, page_size, max_pages, num_pages;
};
size_t page_compact_workspace(int num_pages);
cudaError_t launch_page_compact(const PageCompact &p, void *ws, cudaStream_t s);

constexpr int kPageMaxCaches = 128;
struct PageCopy {
    void *caches[kPageMaxCaches];
    long page_bytes[kPageMaxCaches];
    int count, n, num_pages;
    const int32_t *copies;
};
cudaError_t launch_page_copy(const PageCopy &c, cudaStream_t s);

}  // namespace gdn
