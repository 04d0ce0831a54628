// page_fork.cu - gdn_page_fork, gdn_page_compact and gdn_page_copy: block tables follow the chosen beams, live
// pages move to the front of the pool, and the pages' contents are copied.
//
// Who owns a page is read off the block table itself: a page is live while a row holds it among its first
// ceil(len / page_size) entries.  So both plans are marks on the pool's pages (one byte each, plain
// stores of the same value), prefix sums over the marks and over the rows, and independent rewriting of the entries:
// a few hundred kilobytes at most, bound by the launch and by the latency of some dependent steps.  One launch
// each: a thread-block cluster, whose barrier parts the steps (one CTA for small pools).  Order comes from
// page numbers and row numbers alone, so results do not depend on timing.
//
// 64 x 4 rows of up to 4096 tokens in pages of 64: the plan of a fork takes some 15 us (launch, four cluster barriers, ten
// dependent loads; 28 with a cluster of four, 48 in one CTA, copies included), the copies of its last pages 8; a compaction's
// plan 15 (19 before its copies), its copies 51 (350 MB at 6.8 TB/s, the measured copy's rate).
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "copy.cuh"
#include "serving.h"

namespace gdn {
namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;
static_assert(kThreads == 32 * 32, "the scan's last step is one warp's");

// Exclusive sum over the block; returns the block's total in `all`.
__device__ __forceinline__ int block_scan(int x, int &all, int *s_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, x0 = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();  // an earlier scan's sums have been read
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = s_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += y;
        }
        s_sum[lane] = w;
    }
    __syncthreads();
    all = s_sum[31];
    return x - x0 + (warp ? s_sum[warp - 1] : 0);
}

// The part of n things that thread `i` of `of` takes: [lo, hi), in whole multiples of 16.
__device__ __forceinline__ void share(int n, int i, int of, int &lo, int &hi) {
    const int per = ((n + of - 1) / of + 15) / 16 * 16;
    lo = (int)min((long)n, (long)i * per), hi = min(n, lo + per);
}

// f(i) for the pages of [lo, hi) (lo a multiple of 16) whose mark in `a` is set and whose mark in `b`, if given, is not;
// neither(i) for the others.
template <typename F, typename G>
__device__ __forceinline__ void for_marks(const uint8_t *a, const uint8_t *b, int lo, int hi, F f, G neither) {
    for (int i = lo; i < hi; i += 16) {
        const uint4 x = __ldcg(reinterpret_cast<const uint4 *>(a + i));
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
        if (b != nullptr) {
            const uint4 y = __ldcg(reinterpret_cast<const uint4 *>(b + i));
            w[0] &= ~y.x, w[1] &= ~y.y, w[2] &= ~y.z, w[3] &= ~y.w;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if (i + k >= hi) break;
            if (w[k / 4] >> (k % 4 * 8) & 1) f(i + k);
            else neither(i + k);
        }
    }
}

struct ForkSpace {  // in the workspace; every part on a 16-byte boundary
    int *total;     // [kCluster] a CTA's sum
    int *error;     // [kCluster]
    int *old;       // [B][max_pages] a table that is written in place, before the call
    uint8_t *was, *is;  // [num_pages] live before and after
};

// f(row, column) for the first width(row) of `columns` columns of each row, shared out among the grid's warps: a warp takes 128
// entries of a row at a time.
template <typename W, typename F>
__device__ __forceinline__ void for_entries(int rows, int columns, W width, F f) {
    const int lane = threadIdx.x & 31, warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kThreads / 32);
    const int parts = (columns + 127) / 128;
    for (int item = warp; item < rows * parts; item += warps) {  // (rows * columns fits)
        const int row = item / parts, first = (item - row * parts) * 128 + lane, n = width(row);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (first + 32 * k < n) f(row, first + 32 * k);
    }
}

__global__ void __launch_bounds__(kThreads) page_fork_kernel(const PageFork p, ForkSpace w) {
    extern __shared__ int s_fork[];
    // [B]: tokens of an old row, its first child; [B_out]: parent of a new row, and its place among the rows that need a page
    // of their own for their last, partly filled one (all children but the first), or -1
    int *s_len = s_fork, *s_first = s_len + p.B, *s_parent = s_first + p.B, *s_rank = s_parent + p.B_out;
    __shared__ int s_sum[32], s_bad;
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int tid = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x, ps = p.page_size, M = p.max_pages;
    const long t0 = (long)rank * kThreads + tid, step = (long)ranks * kThreads;
    const bool same_table = p.table_out == p.block_table, same_lens = p.kv_lens_out == p.kv_lens;
    const auto pages = [&](int b) { return (s_len[b] + ps - 1) / ps; };
    const auto child_pages = [&](int i) { return s_parent[i] < 0 ? 0 : pages(s_parent[i]); };
    pdl_wait_primary();

    // ---- clear the marks; copy a table that is written in place; look for what is wrong
    for (long i = t0 * 16; i < p.num_pages; i += step * 16)  // (the marks' rooms are multiples of 16)
        *reinterpret_cast<uint4 *>(w.was + i) = *reinterpret_cast<uint4 *>(w.is + i) = make_uint4(0, 0, 0, 0);
    if (tid == 0) s_bad = 0;
    const int cursor = *p.cursor;  // (not as read-only data: cursor_out may be the same word)
    bool bad = cursor < 0 || cursor > p.n_free;
    for (int b = tid; b < p.B; b += kThreads) {
        const int len = p.kv_lens[b];
        const bool fits = len >= 0 && len <= (long)M * ps;
        bad |= !fits;
        s_len[b] = fits ? len : 0;
        s_first[b] = p.B_out;
    }
    for (int i = tid; i < p.B_out; i += kThreads) {
        const int parent = __ldg(p.parents + i);
        bad |= parent >= p.B;
        s_parent[i] = parent < p.B ? parent : -1;
    }
    __syncthreads();
    for (int i = tid; i < p.B_out; i += kThreads)
        if (s_parent[i] >= 0) atomicMin(s_first + s_parent[i], i);
    for_entries(p.B, M, pages, [&](int b, int j) {
        const int page = p.block_table[(long)b * M + j];
        bad |= page < 0 || page >= p.num_pages;
        if (same_table) w.old[(long)b * M + j] = page;
    });
    if (bad) s_bad = 1;
    __syncthreads();
    if (tid == 0) w.error[rank] = s_bad;
    int copies = 0, mine = 0;
    {
        const int per = (p.B_out + kThreads - 1) / kThreads, i0 = min(p.B_out, tid * per), i1 = min(p.B_out, i0 + per);
        for (int i = i0; i < i1; ++i) {
            const int parent = s_parent[i];
            const bool own = parent >= 0 && s_len[parent] % ps != 0 && s_first[parent] != i;
            s_rank[i] = own ? mine++ : -1;
        }
        const int at = block_scan(mine, copies, s_sum);
        for (int i = i0; i < i1; ++i)
            if (s_rank[i] >= 0) s_rank[i] += at;
    }
    cluster.sync();
    bad = false;
    for (int r = 0; r < ranks; ++r) bad |= __ldcg(w.error + r) != 0;
    const int *old = same_table ? w.old : p.block_table;

    // ---- marks
    if (!bad) {
        for_entries(p.B, M, pages, [&](int b, int j) { w.was[__ldcg(old + (long)b * M + j)] = 1; });
        for_entries(p.B_out, M, [&](int i) { return child_pages(i) - (s_rank[i] >= 0); },
                    [&](int i, int j) { w.is[__ldcg(old + (long)s_parent[i] * M + j)] = 1; });
    }
    cluster.sync();

    // ---- pages that go back to the list, in their order
    int lo, hi;
    share(p.num_pages, (int)t0, (int)step, lo, hi);
    int back = 0, all = 0;
    for (int i = lo; i < hi; i += 16) {
        const uint4 a = __ldcg(reinterpret_cast<const uint4 *>(w.was + i)), b = __ldcg(reinterpret_cast<const uint4 *>(w.is + i));
        back += __popc(a.x & ~b.x) + __popc(a.y & ~b.y) + __popc(a.z & ~b.z) + __popc(a.w & ~b.w);
    }
    int at = block_scan(back, all, s_sum);
    if (tid == 0) w.total[rank] = all;
    cluster.sync();
    int freed = 0;
    for (int r = 0; r < ranks; ++r) {
        const int x = __ldcg(w.total + r);
        if (r < rank) at += x;
        freed += x;
    }
    const long start = (long)cursor - freed;  // the list's place of the first page that goes back
    const int status = bad || start < 0 ? GDN_ERR_SHAPE : start + copies > p.n_free ? GDN_ERR_CAPACITY : GDN_OK;
    const bool ok = status == GDN_OK;

    if (ok && back > 0) for_marks(w.was, w.is, lo, hi, [&](int i) { p.free_pages[start + at++] = i; }, [](int) {});
    cluster.sync();

    // ---- the new rows
    if (ok || !same_table)
        for_entries(p.B_out, M, [&](int) { return M; }, [&](int i, int j) {
            const int n = ok ? child_pages(i) : 0;
            int page = -1;
            if (j < n) page = j == n - 1 && s_rank[i] >= 0 ? __ldcg(p.free_pages + start + s_rank[i]) : __ldcg(old + (long)s_parent[i] * M + j);
            p.table_out[(long)i * M + j] = page;
        });
    for (int i = (int)t0; i < p.B_out; i += (int)step) {
        const int parent = s_parent[i];
        if (ok || !same_lens) p.kv_lens_out[i] = ok && parent >= 0 ? s_len[parent] : 0;
        if (ok && s_rank[i] >= 0)
            reinterpret_cast<int2 *>(p.copies)[s_rank[i]] =
                make_int2(__ldcg(old + (long)parent * M + s_len[parent] / ps), __ldcg(p.free_pages + start + s_rank[i]));
        if (!ok || i >= copies) reinterpret_cast<int2 *>(p.copies)[i] = make_int2(-1, -1);
    }
    if (t0 == 0) {
        *p.cursor_out = ok ? (int)(start + copies) : cursor;
        *p.status = status;
    }
}

struct CompactSpace {
    int *total, *error, *below;  // [kCluster], [kCluster], [1]: live pages among the first `live`
    uint8_t *is;                 // [num_pages]
    int *list;                   // [num_pages] holes from the front, pages that fill them from the back
    int *to;                     // [num_pages] where such a page goes
};

__global__ void __launch_bounds__(kThreads) page_compact_kernel(const PageCompact p, CompactSpace w) {
    extern __shared__ int s_used[];  // [B]: pages of a row
    __shared__ int s_sum[32], s_bad;
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int tid = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x, ps = p.page_size, M = p.max_pages;
    const long t0 = (long)rank * kThreads + tid, step = (long)ranks * kThreads;
    pdl_wait_primary();
    for (long i = t0 * 16; i < p.num_pages; i += step * 16) *reinterpret_cast<uint4 *>(w.is + i) = make_uint4(0, 0, 0, 0);
    if (tid == 0) s_bad = 0;
    bool bad = false;
    for (int b = tid; b < p.B; b += kThreads) {
        const int len = __ldg(p.kv_lens + b);
        const bool fits = len >= 0 && len <= (long)M * ps;
        bad |= !fits;
        s_used[b] = fits ? (len + ps - 1) / ps : 0;
    }
    __syncthreads();
    const auto used = [&](int b) { return s_used[b]; };
    for_entries(p.B, M, used, [&](int b, int j) {
        const int page = p.block_table[(long)b * M + j];
        bad |= page < 0 || page >= p.num_pages;
    });
    if (bad) s_bad = 1;
    __syncthreads();
    if (tid == 0) w.error[rank] = s_bad;
    cluster.sync();
    bad = false;
    for (int r = 0; r < ranks; ++r) bad |= __ldcg(w.error + r) != 0;
    if (!bad) for_entries(p.B, M, used, [&](int b, int j) { w.is[p.block_table[(long)b * M + j]] = 1; });
    cluster.sync();

    int lo, hi;
    share(p.num_pages, (int)t0, (int)step, lo, hi);
    int mine = 0, all = 0;
    for (int i = lo; i < hi; i += 16) {
        const uint4 a = __ldcg(reinterpret_cast<const uint4 *>(w.is + i));
        mine += __popc(a.x) + __popc(a.y) + __popc(a.z) + __popc(a.w);
    }
    int before = block_scan(mine, all, s_sum);  // live pages before lo
    if (tid == 0) w.total[rank] = all;
    cluster.sync();
    int live = 0;
    for (int r = 0; r < ranks; ++r) {
        const int x = __ldcg(w.total + r);
        if (r < rank) before += x;
        live += x;
    }
    // holes among the first `live` pages by their rank from the front, the live ones behind them by their rank
    // among all live ones from the back: with H holes, H <= num_pages - live, and those fill the last `live` places at
    // most, so the two lists do not meet
    if (!bad) {
        if (lo <= live && live < hi) {  // (this thread meets the page numbered `live`)
            int n = before;
            for_marks(w.is, nullptr, lo, live, [&](int) { ++n; }, [](int) {});
            *w.below = n;
        }
        for_marks(w.is, nullptr, lo, hi, [&](int i) {
            if (i >= live) w.list[p.num_pages - 1 - before] = i;
            ++before;
        }, [&](int i) {
            if (i < live) w.list[i - before] = i;
        });
    }
    cluster.sync();
    const int below = bad ? 0 : live < p.num_pages ? __ldcg(w.below) : live, moved = bad ? 0 : live - below;
    for (long i = t0; i < p.num_pages / 2; i += step) {
        int2 pair = make_int2(-1, -1);
        if (i < moved) {
            pair = make_int2(__ldcg(w.list + p.num_pages - 1 - below - i), __ldcg(w.list + i));
            w.to[pair.x] = pair.y;
        }
        reinterpret_cast<int2 *>(p.copies)[i] = pair;
    }
    cluster.sync();
    const bool same = p.table_out == p.block_table;
    if (!bad || !same)
        for_entries(p.B, M, [&](int) { return M; }, [&](int b, int j) {
            int page = -1;
            if (!bad && j < used(b)) {
                page = p.block_table[(long)b * M + j];
                if (page >= live) page = __ldcg(w.to + page);
            }
            p.table_out[(long)b * M + j] = page;
        });
    if (!bad)
        for (long i = t0; i < p.num_pages; i += step) p.free_pages[i] = (int)i;
    if (t0 == 0) {
        if (!bad) *p.cursor_out = live;
        *p.status = bad ? GDN_ERR_SHAPE : GDN_OK;
    }
}

constexpr int kCopyThreads = 256, kCopyBytes = kCopyThreads * 16 * 4;  // of a CTA's turn

struct CopyParams {
    PageCopy c;
    int first[kPageMaxCaches + 1];  // first piece of each cache's page
    int vec[kPageMaxCaches];
};

// CTAs take (pair, piece) items in turn.  Lists may be mostly empty: the threads of a CTA look at the pairs of its next 256
// items at once, and only those with something to copy are gone through.
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ CopyParams p) {
    __shared__ unsigned s_have[kCopyThreads / 32];
    const int pieces = p.first[p.c.count], tid = threadIdx.x;
    const long items = (long)p.c.n * pieces;
    pdl_wait_primary();
    const auto pair_of = [&](long item) { return __ldg(reinterpret_cast<const int2 *>(p.c.copies) + item / pieces); };
    for (long first = blockIdx.x; first < items; first += (long)gridDim.x * kCopyThreads) {
        const long mine = first + (long)tid * gridDim.x;
        bool have = false;
        if (mine < items) {
            const int2 pair = pair_of(mine);
            have = pair.x >= 0 && pair.x < p.c.num_pages && pair.y >= 0 && pair.y < p.c.num_pages && pair.x != pair.y;
        }
        const unsigned bits = __ballot_sync(0xffffffffu, have);
        __syncthreads();  // the last items' words have been read
        if ((tid & 31) == 0) s_have[tid >> 5] = bits;
        __syncthreads();
        for (int w = 0; w < kCopyThreads / 32; ++w)
            for (unsigned left = s_have[w]; left != 0; left &= left - 1) {
                const long item = first + (long)(w * 32 + __ffs(left) - 1) * gridDim.x;
                const int2 pair = pair_of(item);
                const int piece = (int)(item % pieces);
                int t = 0;
                while (piece >= p.first[t + 1]) ++t;
                const long page = p.c.page_bytes[t], from = (long)(piece - p.first[t]) * kCopyBytes;
                const long bytes = min((long)kCopyBytes, page - from);
                unsigned char *base = static_cast<unsigned char *>(p.c.caches[t]) + from;
                unsigned char *dst = base + pair.y * page;
                const unsigned char *src = base + pair.x * page;
                copy_bytes<kCopyThreads, 4>(dst, src, bytes, p.vec[t]);
            }
    }
}

size_t round16(size_t x) { return (x + 15) & ~size_t(15); }

template <typename K, typename P, typename W>
cudaError_t launch_plan(K kernel, size_t smem, long work, const P &p, const W &w, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    const int ctas = work <= 2 * kThreads ? 1 : kCluster;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, w);
    note_launch();
    return e;
}

}  // namespace

size_t page_fork_workspace(int B, int max_pages, int num_pages) {
    return 64 + round16((size_t)B * max_pages * 4) + 2 * round16(num_pages);
}

cudaError_t launch_page_fork(const PageFork &p, void *ws, cudaStream_t s) {
    ForkSpace w;
    char *at = static_cast<char *>(ws);
    w.total = reinterpret_cast<int *>(at), w.error = w.total + kCluster;
    w.old = reinterpret_cast<int *>(at += 64);
    w.was = reinterpret_cast<uint8_t *>(at += round16((size_t)p.B * p.max_pages * 4));
    w.is = reinterpret_cast<uint8_t *>(at + round16(p.num_pages));
    static std::atomic<uint64_t> attr_set{0};
    const cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(page_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kPagePlanMaxB * 4);
    });
    if (e != cudaSuccess) return e;
    const long work = std::max(std::max((long)p.B, (long)p.B_out) * p.max_pages, p.num_pages / 4L);
    return launch_plan(page_fork_kernel, 2 * ((size_t)p.B + p.B_out) * 4, work, p, w, s);
}

size_t page_compact_workspace(int num_pages) { return 128 + round16(num_pages) + 8 * (size_t)num_pages; }

cudaError_t launch_page_compact(const PageCompact &p, void *ws, cudaStream_t s) {
    CompactSpace w;
    char *at = static_cast<char *>(ws);
    w.total = reinterpret_cast<int *>(at), w.error = w.total + kCluster, w.below = w.error + kCluster;
    w.is = reinterpret_cast<uint8_t *>(at += 128);
    w.list = reinterpret_cast<int *>(at += round16(p.num_pages));
    w.to = w.list + p.num_pages;
    static std::atomic<uint64_t> attr_set{0};
    const cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(page_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPagePlanMaxB * 4);
    });
    if (e != cudaSuccess) return e;
    return launch_plan(page_compact_kernel, (size_t)p.B * 4, std::max((long)p.B * p.max_pages, p.num_pages / 4L), p, w, s);
}

cudaError_t launch_page_copy(const PageCopy &c, cudaStream_t s) {
    CopyParams p{};
    p.c = c;
    for (int t = 0; t < c.count; ++t) {
        p.first[t + 1] = p.first[t] + (int)((c.page_bytes[t] + kCopyBytes - 1) / kCopyBytes);
        p.vec[t] = copy_width((uintptr_t)c.caches[t], (uintptr_t)c.page_bytes[t]);
    }
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long grid = std::min((long)c.n * p.first[c.count], 8L * sms);
    if (grid == 0) return cudaSuccess;
    const cudaError_t e = launch_kernel(page_copy_kernel, dim3((unsigned)grid), dim3(kCopyThreads), 0, s, true, p);
    note_launch();
    return e;
}

}  // namespace gdn
