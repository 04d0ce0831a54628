// state_reorder.cu - gdn_state_reorder: rows of states follow the chosen beams,
// row i <- row parents[i], in place, for several state tensors in one launch.
//
// Nothing is computed: bound by HBM at one read of every row that is a parent of another
// and one write of every row that changes.  In place, a row may be read by one and written by
// another: so a CTA owns a strip of columns of all rows, brings the strips of all changed rows'
// parents into shared memory, and writes them after a barrier; strips of different CTAs do not touch.
// The strip is as wide as shared memory allows for B rows, which keeps the accesses long (256
// rows: 256 bytes).  Rows that keep their place are neither read nor written.
#include <algorithm>

#include "common.cuh"
#include "serving.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kStrip = 64 * 1024;  // bytes of all strips of a CTA: three CTAs to an SM

struct ReorderParams {
    StateReorder r;
    long first[kStateMaxTensors + 1];  // first strip of each tensor
    int strip;                         // bytes, a multiple of 16
    int vec[kStateMaxTensors];         // bytes of an access: 16, 8, 4, 2 or 1
};

template <typename T>
__device__ __forceinline__ void move_strip(unsigned char *base, long row_bytes, long from, int bytes, int strip, int moved,
                                           const int2 *s_move, unsigned char *s_data) {
    const int per = bytes / (int)sizeof(T), all = moved * per;
    for (int i = threadIdx.x; i < all; i += kThreads) {
        const int m = i / per, c = i % per;
        const void *src = base + s_move[m].x * row_bytes + from + c * (long)sizeof(T);
        T *dst = reinterpret_cast<T *>(s_data + (size_t)m * strip) + c;
        if constexpr (sizeof(T) >= 4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                         "n"((int)sizeof(T))
                         : "memory");
        else
            *dst = *static_cast<const T *>(src);
    }
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    for (int i = threadIdx.x; i < all; i += kThreads) {
        const int m = i / per, c = i % per;
        *reinterpret_cast<T *>(base + s_move[m].y * row_bytes + from + c * (long)sizeof(T)) =
            reinterpret_cast<const T *>(s_data + (size_t)m * strip)[c];
    }
}

__global__ void __launch_bounds__(kThreads) state_reorder_kernel(const __grid_constant__ ReorderParams p) {
    extern __shared__ __align__(16) unsigned char s_data[];
    __shared__ int s_n;
    int2 *s_move = reinterpret_cast<int2 *>(s_data + (size_t)p.r.B * p.strip);  // (parent, row)
    pdl_wait_primary();
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.r.B; i += kThreads) {
        const int from = __ldg(p.r.parents + i);
        if (from != i && from >= 0 && from < p.r.B) s_move[atomicAdd(&s_n, 1)] = make_int2(from, i);
    }
    __syncthreads();
    const int moved = s_n;
    if (moved == 0) return;
    for (long strip = blockIdx.x; strip < p.first[p.r.count]; strip += gridDim.x) {
        int t = 0;
        while (strip >= p.first[t + 1]) ++t;
        const long from = (strip - p.first[t]) * p.strip, row = p.r.row_bytes[t];
        const int bytes = (int)min((long)p.strip, row - from);
        unsigned char *base = static_cast<unsigned char *>(p.r.states[t]);
        switch (p.vec[t]) {
        case 16: move_strip<uint4>(base, row, from, bytes, p.strip, moved, s_move, s_data); break;
        case 8: move_strip<uint2>(base, row, from, bytes, p.strip, moved, s_move, s_data); break;
        case 4: move_strip<uint32_t>(base, row, from, bytes, p.strip, moved, s_move, s_data); break;
        case 2: move_strip<uint16_t>(base, row, from, bytes, p.strip, moved, s_move, s_data); break;
        default: move_strip<uint8_t>(base, row, from, bytes, p.strip, moved, s_move, s_data);
        }
        __syncthreads();  // the strips are read before the next ones come
    }
}

}  // namespace

cudaError_t launch_state_reorder(const StateReorder &r, cudaStream_t s) {
    ReorderParams p{};
    p.r = r;
    p.strip = std::max(16, std::min(4096, kStrip / r.B / 16 * 16));
    p.first[0] = 0;
    for (int t = 0; t < r.count; ++t) {
        p.first[t + 1] = p.first[t] + (r.row_bytes[t] + p.strip - 1) / p.strip;
        const uintptr_t at = (uintptr_t)r.states[t] | (uintptr_t)r.row_bytes[t];
        p.vec[t] = at % 16 == 0 ? 16 : at % 8 == 0 ? 8 : at % 4 == 0 ? 4 : at % 2 == 0 ? 2 : 1;
    }
    if (p.first[r.count] == 0) return cudaSuccess;
    const size_t smem = (size_t)r.B * (p.strip + sizeof(int2));
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(state_reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    std::max(kStrip + kStateMaxRows * 8, kStateMaxRows * 24));
    });
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long grid = std::min(p.first[r.count], 3L * sms);
    e = launch_kernel(state_reorder_kernel, dim3((unsigned)grid), dim3(kThreads), smem, s, true, p);
    note_launch();
    return e;
}

}  // namespace gdn
