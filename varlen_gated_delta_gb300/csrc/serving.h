// serving.h - host-side interface of the kernels that serve softmax-attention
// layers (page_plan.cu, qk_norm_rope.cu, attention_*.cu), called by
// serving_api.cpp.  Not installed; the public ABI is include/gdn.h.
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

}  // namespace gdn
