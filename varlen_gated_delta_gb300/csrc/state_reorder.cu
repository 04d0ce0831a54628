// state_reorder.cu - gdn_state_reorder: rows of states follow the chosen beams,
// row i <- row parents[i], in place, for several state tensors in one launch.
//
// Nothing is computed: bound by HBM at one read of every row that is a parent of another
// and one write of every row that changes.  Rows that keep their place are neither read nor written.
//
// A row that takes the content of one that keeps its place, and that nobody else takes anything from, is
// copied in long pieces (so all of them, when gdn_beam_select keeps rows).  Among the others a row may be
// read by one and written by another: for these a CTA owns a strip of columns of all rows, brings the
// strips of all their parents into shared memory, and writes them after a barrier; strips of different
// CTAs do not touch.  The strip is as wide as shared memory allows for B rows: 256 bytes for 256 rows, 32 for 2048, 16, half
// a sector, for 4096.  268 MB in a random permutation: 96 us for 256 rows (79 at the measured copy's rate), 121 for 1024, 181
// for 2048, 467 for 4096.
//
// 32 x 8 beams, two layers' states (2.1 MB a row and layer), rows kept: 141 us, 6.0 TB/s, 0.88 of the measured copy (strips for
// all rows: 159); one request's four beams, one layer: 3.4 us.
#include <algorithm>

#include "common.cuh"
#include "copy.cuh"
#include "serving.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kStrip = 64 * 1024;  // bytes of all strips of a CTA: three CTAs to an SM

constexpr int kPiece = kThreads * 16 * 8;  // bytes of a row that a CTA copies at a time

struct ReorderParams {
    StateReorder r;
    long first_piece[kStateMaxTensors + 1];  // first piece of each tensor's rows
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
    // (parent, row) of the rows that change: the simple ones from the back, the others from the front; which rows are read
    // by others and which change, a byte to each
    __shared__ int2 s_count[kThreads / 32];
    int2 *s_move = reinterpret_cast<int2 *>(s_data + (size_t)p.r.B * p.strip);
    uint8_t *s_read = reinterpret_cast<uint8_t *>(s_move + p.r.B), *s_changes = s_read + p.r.B;
    const int B = p.r.B;
    pdl_wait_primary();
    for (int i = threadIdx.x; i < B; i += kThreads) s_read[i] = 0;
    __syncthreads();
    const auto parent = [&](int i) {
        const int from = __ldg(p.r.parents + i);
        return from >= 0 && from < B ? from : i;
    };
    for (int i = threadIdx.x; i < B; i += kThreads) {
        const int from = parent(i);
        s_changes[i] = from != i;
        if (from != i) s_read[from] = 1;
    }
    __syncthreads();
    // (in the order of rows: all CTAs have to agree on who copies which)
    int moved = 0, simple = 0;
    for (int i0 = 0; i0 < B; i0 += kThreads) {
        const int i = i0 + threadIdx.x, from = i < B ? parent(i) : i;
        const bool is_simple = from != i && !s_changes[from] && !s_read[i], other = from != i && !is_simple;
        const unsigned a = __ballot_sync(0xffffffffu, is_simple), b = __ballot_sync(0xffffffffu, other);
        const unsigned before = (1u << (threadIdx.x & 31)) - 1;
        if ((threadIdx.x & 31) == 0) s_count[threadIdx.x >> 5] = make_int2(__popc(a), __popc(b));
        __syncthreads();
        int at_simple = simple + __popc(a & before), at_other = moved + __popc(b & before);
        for (int w = 0; w < kThreads / 32; ++w) {
            const int2 c = s_count[w];
            if (w < threadIdx.x >> 5) at_simple += c.x, at_other += c.y;
            simple += c.x, moved += c.y;
        }
        if (is_simple) s_move[B - 1 - at_simple] = make_int2(from, i);
        if (other) s_move[at_other] = make_int2(from, i);
        __syncthreads();
    }
    // (the rows of a piece follow one another, so that children of one parent find it in L2)
    if (simple > 0)
        for (long item = blockIdx.x; item < p.first_piece[p.r.count] * simple; item += gridDim.x) {
            const long piece = item / simple;
            const int2 move = s_move[B - 1 - (int)(item - piece * simple)];
            int t = 0;
            while (piece >= p.first_piece[t + 1]) ++t;
            const long row = p.r.row_bytes[t], from = (piece - p.first_piece[t]) * kPiece, bytes = min((long)kPiece, row - from);
            unsigned char *base = static_cast<unsigned char *>(p.r.states[t]) + from;
            copy_bytes<kThreads, 8>(base + move.y * row, base + move.x * row, bytes, p.vec[t]);
        }
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
    for (int t = 0; t < r.count; ++t) {
        p.first_piece[t + 1] = p.first_piece[t] + (r.row_bytes[t] + kPiece - 1) / kPiece;
        p.first[t + 1] = p.first[t] + (r.row_bytes[t] + p.strip - 1) / p.strip;
        p.vec[t] = copy_width((uintptr_t)r.states[t], (uintptr_t)r.row_bytes[t]);
    }
    if (p.first[r.count] == 0) return cudaSuccess;
    const size_t smem = (size_t)r.B * (p.strip + sizeof(int2) + 2);
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(state_reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    std::max(kStrip + kStateMaxRows * 10, kStateMaxRows * 26));
    });
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long grid = std::min(std::max(p.first[r.count], p.first_piece[r.count] * r.B), 3L * sms);
    e = launch_kernel(state_reorder_kernel, dim3((unsigned)grid), dim3(kThreads), smem, s, true, p);
    note_launch();
    return e;
}

}  // namespace gdn
