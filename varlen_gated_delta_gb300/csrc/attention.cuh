// attention.cuh - device helpers shared by the attention kernels.
#pragma once

#include "common.cuh"
#include "serving.h"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x on the special-function unit (relative error about 2^-22; 0 for -inf).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Rows [start, start + len) of sequence b and its key count; false for a
// malformed sequence.
__device__ __forceinline__ bool attn_seq(const Attn &a, int b, int &start, int &len, int &kv) {
    start = __ldg(a.offsets + b);
    len = __ldg(a.offsets + b + 1) - start;
    kv = len;
    if (start < 0 || len < 0 || start > a.N - len) return false;
    if (a.block_table == nullptr) return true;
    kv = __ldg(a.kv_lens + b);
    return kv >= 0 && kv <= (long long)a.max_pages * a.page_size && len <= a.max_q;
}

// Element offset of key j of sequence b in a row of k (or v) with token stride
// `stride`, or -1 when its page is not one of the cache's.
__device__ __forceinline__ long attn_key_row(const Attn &a, int b, int start, int j, long stride) {
    if (a.block_table == nullptr) return (long)(start + j) * stride;
    const int page = __ldg(a.block_table + (size_t)b * a.max_pages + j / a.page_size);
    if (page < 0 || page >= a.num_pages) return -1;
    return ((long)page * a.page_size + j % a.page_size) * stride;
}

// Where split `i` of `splits` of a (token, head) row leaves its part: an unscaled output o, and ml =
// {maximum in base 2, sum}.
struct Part {
    float *o, *ml;
    __device__ __forceinline__ Part(const Attn &a, int splits, size_t row, int i) {
        const size_t at = row * splits + i;
        o = a.part + at * a.D;
        ml = a.part + (size_t)a.N * a.H * splits * a.D + at * 2;
    }
};

// Warp-wide: the idx-th tile of `rows` rows over all sequences, whose row
// counts are len * per_token; false past the last one.  Malformed sequences
// have no tiles.
__device__ __forceinline__ bool attn_find_tile(const Attn &a, int per_token, int rows, long idx,
                                               int &b, int &tile) {
    const int lane = threadIdx.x & 31;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        int start, len, kv;
        long n = 0;
        if (b0 + lane < a.B && attn_seq(a, b0 + lane, start, len, kv))
            n = ((long)len * per_token + rows - 1) / rows;
        long sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long x = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += x;
        }
        const long all = __shfl_sync(0xffffffffu, sum, 31);
        if (idx < all) {
            const int at = __ffs(__ballot_sync(0xffffffffu, idx < sum)) - 1;
            b = b0 + at;
            tile = (int)(idx - __shfl_sync(0xffffffffu, sum - n, at));
            return true;
        }
        idx -= all;
    }
    return false;
}

}  // namespace gdn
