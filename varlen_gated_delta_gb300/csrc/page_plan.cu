// page_plan.cu - gdn_page_plan: block tables, slots and positions of a step's
// new tokens, built on the GPU from request lengths.
//
// With ps tokens to a page, request b owns ceil(cached_b / ps) pages and needs
// ceil((cached_b + new_b) / ps); the difference comes from the free list at
// cursor + (the needs of requests before b).  So the whole plan is two prefix
// sums over the requests and one independent computation per new token and per
// new page.  There is next to nothing to read or write: the call is bound by
// its launch and by the latency of the scan.  One launch: every CTA computes both
// prefix sums for itself in shared memory (B is small), and the CTAs share the
// tokens and pages.  Where an output lies over an input (the lengths or the cursor
// carried in place), the CTAs form one thread-block cluster, whose barrier between
// the last read and the first write keeps them apart.  One CTA for small steps (64
// requests of one token: 4.6 us); 107781 tokens of 32 requests: 11.8 us carried in
// place, 6.6 us otherwise.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "serving.h"

namespace gdn {
namespace {

constexpr int kThreads = 1024;

// Exclusive sums of (a, c) over the block; returns the block's totals in ta, tc.
__device__ __forceinline__ void block_scan2(long long &a, long long &c, long long &ta,
                                            long long &tc, long long (*s_sum)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long a0 = a, c0 = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long xa = __shfl_up_sync(0xffffffffu, a, d), xc = __shfl_up_sync(0xffffffffu, c, d);
        if (lane >= d) a += xa, c += xc;
    }
    if (lane == 31) s_sum[warp][0] = a, s_sum[warp][1] = c;
    __syncthreads();
    if (warp == 0) {
        long long wa = s_sum[lane][0], wc = s_sum[lane][1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long xa = __shfl_up_sync(0xffffffffu, wa, d), xc = __shfl_up_sync(0xffffffffu, wc, d);
            if (lane >= d) wa += xa, wc += xc;
        }
        s_sum[lane][0] = wa, s_sum[lane][1] = wc;
    }
    __syncthreads();
    ta = s_sum[31][0], tc = s_sum[31][1];
    a += (warp ? s_sum[warp - 1][0] : 0) - a0;
    c += (warp ? s_sum[warp - 1][1] : 0) - c0;
}

// Largest b with ofs[b] <= x (ofs[0] = 0 <= x < ofs[B]).
__device__ __forceinline__ int find(const int *ofs, int B, int x) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ofs[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(const PagePlan p) {
    extern __shared__ int s_plan[];
    int *s_ofs = s_plan, *s_page = s_plan + p.B + 1, *s_cached = s_plan + 2 * (p.B + 1);
    __shared__ long long s_sum[32][2];
    __shared__ int s_bad;
    const int tid = threadIdx.x;
    const int rank = blockIdx.x, ranks = gridDim.x;
    const int ps = p.page_size;
    pdl_wait_primary();

    if (tid == 0) s_bad = 0;
    __syncthreads();
    const int cursor = *p.cursor;  // (this and the cached lengths not as read-only data: outputs may be the same words)
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    long long tok = 0, pages = 0;
    int bad = 0;  // the most severe finding: shape, then capacity
    for (int b = b0; b < b1; ++b) {
        int n = __ldg(p.new_lens + b), c = p.cached_lens[b];
        if (n < 0 || c < 0) {
            bad = GDN_ERR_SHAPE;
            n = 0, c = max(c, 0);
        }
        if ((long long)c + n > (long long)p.max_pages * ps || (long long)c + n > INT32_MAX - ps)
            bad = bad ? bad : GDN_ERR_CAPACITY;
        s_cached[b] = c;
        tok += n;
        pages += ((long long)c + n + ps - 1) / ps - ((long long)c + ps - 1) / ps;
    }
    if (bad) atomicMax(&s_bad, bad == GDN_ERR_SHAPE ? 2 : 1);
    long long all_tok, all_pages;
    block_scan2(tok, pages, all_tok, all_pages, s_sum);
    int status = s_bad == 2 || cursor < 0      ? GDN_ERR_SHAPE
                 : all_tok > p.N               ? GDN_ERR_OFFSETS
                 : s_bad || cursor + all_pages > p.n_free ? GDN_ERR_CAPACITY
                                               : GDN_OK;
    const bool ok = status == GDN_OK;
    if (ok)
        for (int b = b0; b < b1; ++b) {  // every sum fits: at most N tokens and n_free pages
            const int n = __ldg(p.new_lens + b), c = s_cached[b];
            s_ofs[b] = (int)tok;
            s_page[b] = (int)pages;
            tok += n;
            pages += (c + n + ps - 1) / ps - (c + ps - 1) / ps;
        }
    const int total = ok ? (int)all_tok : 0, fresh = ok ? (int)all_pages : 0;
    if (tid == 0) s_ofs[p.B] = total, s_page[p.B] = fresh;
    // Every CTA has read what the outputs may overwrite (in a cluster), and this CTA's sums are in place.
    cooperative_groups::this_cluster().sync();

    const int t0 = rank * kThreads + tid, step = ranks * kThreads;
    for (int b = t0; b <= p.B; b += step) {
        p.offsets[b] = ok ? s_ofs[b] : 0;
        if (b < p.B && (ok || p.kv_lens != p.cached_lens))
            p.kv_lens[b] = ok ? s_cached[b] + s_ofs[b + 1] - s_ofs[b] : p.cached_lens[b];
    }
    if (t0 == 0) {
        *p.cursor_out = cursor + fresh;
        *p.status = status;
    }
    for (int i = t0; i < fresh; i += step) {
        const int b = find(s_page, p.B, i), old = (s_cached[b] + ps - 1) / ps;
        p.block_table[(size_t)b * p.max_pages + old + i - s_page[b]] = __ldg(p.free_pages + cursor + i);
    }
    // With many tokens a thread takes four neighbouring ones: one search, and mostly one page.
    const int run = p.N > 4 * kThreads ? 4 : 1;
    for (long t4 = (long)run * t0; t4 < p.N; t4 += (long)run * step) {
        int pos[4], slot[4], b = t4 < total ? find(s_ofs, p.B, (int)t4) : 0, page = -1;
        long long base = -1;  // the first slot of `page`
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = (int)t4 + i;
            pos[i] = 0, slot[i] = -1;
            if (i >= run || t >= total) continue;
            while (t >= s_ofs[b + 1]) ++b, page = -1;
            const int c = s_cached[b], old = (c + ps - 1) / ps;
            pos[i] = c + t - s_ofs[b];
            if (pos[i] / ps != page) {
                page = pos[i] / ps;
                // a page of before this step, or the one that the loop above hands out
                base = page < old ? p.block_table[(size_t)b * p.max_pages + page]
                                  : __ldg(p.free_pages + cursor + s_page[b] + page - old);
                base *= ps;
            }
            const long long at = base + pos[i] - (long long)page * ps;
            slot[i] = base < 0 || at > INT32_MAX ? -1 : (int)at;
        }
        if (p.wide && run == 4 && t4 + 4 <= p.N) {
            *reinterpret_cast<int4 *>(p.positions + t4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4 *>(p.slots + t4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < run && t4 + i < p.N) p.positions[t4 + i] = pos[i], p.slots[t4 + i] = slot[i];
        }
    }
}

}  // namespace

cudaError_t launch_page_plan(const PagePlan &plan, cudaStream_t s) {
    PagePlan p = plan;
    p.wide = (((uintptr_t)p.positions | (uintptr_t)p.slots) & 15) == 0;
    static std::atomic<uint64_t> attr_set{0};
    const size_t smem = 3 * ((size_t)p.B + 1) * 4;
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    3 * (kPagePlanMaxB + 1) * 4);
    });
    if (e != cudaSuccess) return e;
    // Does an output lie over an input that every CTA reads?
    const auto over = [](const int *out, long n, const int *in, long m) {
        return (uintptr_t)out < (uintptr_t)(in + m) && (uintptr_t)in < (uintptr_t)(out + n);
    };
    const auto over_input = [&](const int *out, long n) {
        return over(out, n, p.new_lens, p.B) || over(out, n, p.cached_lens, p.B) || over(out, n, p.cursor, 1);
    };
    const bool in_place = over_input(p.offsets, p.B + 1L) || over_input(p.kv_lens, p.B) || over_input(p.positions, p.N) ||
                          over_input(p.slots, p.N) || over_input(p.cursor_out, 1) || over_input(p.status, 1);
    const long work = (long)p.N + p.B;
    const int ctas = work <= 2 * kThreads ? 1 : in_place ? 8 : (int)std::min(64L, (work + 4 * kThreads - 1) / (4 * kThreads));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = in_place ? ctas : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, page_plan_kernel, p);
    note_launch();
    return e;
}

}  // namespace gdn
