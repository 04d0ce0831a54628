// beam_select.cu - gdn_beam_select: the best continuations of each group of beams.
//
//   total[g, k, t] = score[g, k] + x[g, k, t] - log sum_t' exp x[g, k, t'],
// and of a group's K V totals the n largest, ties to the lowest k V + t.  The logits are read once, in two
// launches.
//
// The first cuts every row into pieces, one CTA each, held in registers: the piece's maximum m and sum of
// exp(x - m), and its n largest logits.  For these, the CTA's threads form at least n groups whose maxima are at
// hand: at least n values reach the least of them, and few more do (8 groups: some 22 of 8192 values), so
// those go into a list and are ranked by counting.  A list that overflows (many equal logits) is left for n
// rounds of the CTA-wide largest value below the last one.
//
// The second, a CTA to a group of beams, joins the pieces' sums, and takes the n best of their candidates the
// same way.  Totals and their comparison are in 64 bits: only the error of the row's sum (fp32 terms) is left
// in the order of beams.
#include <climits>
#include <cmath>

#include "common.cuh"
#include "serving.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kList = 1024;  // candidates that are ranked by counting

struct Pieces {  // in the workspace
    float *m;    // [rows][pieces]: maximum
    float *sum;  // [rows][pieces]: sum of exp(x - m), 0 for a piece of nothing but -inf
    float *x;    // [rows][pieces][n]: the largest logits, descending; -inf past the last
    int *token;  // [rows][pieces][n]
};

// A value in the order of its bits as an unsigned number, and the position behind it: of equal values the
// lowest position is the largest key.
__device__ __forceinline__ unsigned long long key_of(float x, int at) {
    const uint32_t b = __float_as_uint(x);
    return (unsigned long long)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xffffffffu - (uint32_t)at);
}

template <typename T>
__device__ __forceinline__ T warp_max(T x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const T y = __shfl_xor_sync(0xffffffffu, x, d);
        x = y > x ? y : x;
    }
    return x;
}

// The least of the maxima of `groups` (8, 32, 128 or 256) equal sets of neighbouring threads.
template <typename T>
__device__ __forceinline__ T least_of_maxima(T x, int groups, T *s_warp, T most) {
    const int width = kThreads / groups;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const T y = __shfl_xor_sync(0xffffffffu, x, d);
        if (d < width && y > x) x = y;
    }
    // (the least over the warp's groups)
    T least = x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const T y = __shfl_xor_sync(0xffffffffu, least, d);
        if (y < least) least = y;
    }
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = least;
    __syncthreads();
    least = most;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) least = s_warp[w] < least ? s_warp[w] : least;
    return least;
}

__device__ __forceinline__ int groups_for(int n) { return n <= 8 ? 8 : n <= 32 ? 32 : n <= 128 ? 128 : 256; }

template <typename T, int ELEMS>
__global__ void __launch_bounds__(kThreads)
    beam_pieces_kernel(const T *__restrict__ logits, long stride, const uint8_t *__restrict__ finished, Pieces out, int V,
                       int n, int pieces) {
    constexpr int VEC = 16 / sizeof(T), VECS = ELEMS / VEC;
    __shared__ float s_warp[kThreads / 32], s_least[kThreads / 32];
    __shared__ double s_sum[kThreads / 32];
    __shared__ unsigned long long s_list[kList], s_top[kThreads / 32];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long row = blockIdx.x / pieces;
    const int piece = blockIdx.x % pieces;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (finished != nullptr && __ldg(finished + row) != 0) return;  // (nothing of it is looked at)
    const T *x = logits + row * stride;
    // Vectors lie on 16-byte boundaries: the first may begin before the row.
    const int skew = (int)(((uintptr_t)x / sizeof(T)) % VEC);
    const long first = (long)piece * (ELEMS * kThreads) - skew;

    float v[ELEMS];
    if (tid == 0) s_n = 0;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
        const long at = first + (long)(j * kThreads + tid) * VEC;
        if (at >= 0 && at + VEC <= V) {
            Vec16<T> w;
            w.u = __ldg(reinterpret_cast<const uint4 *>(x + at));
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j * VEC + i] = to_f32(w.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j * VEC + i] = at + i >= 0 && at + i < V ? to_f32(x[at + i]) : -INFINITY;
        }
    }
    float mine = -INFINITY;
#pragma unroll
    for (int i = 0; i < ELEMS; ++i) {
        v[i] = v[i] != v[i] ? -INFINITY : v[i] + 0.f;  // (NaN is no candidate; no negative zeros)
        mine = fmaxf(mine, v[i]);
    }
    const float wm = warp_max(mine);
    if (lane == 0) s_warp[warp] = wm;
    const float least = least_of_maxima(mine, groups_for(n), s_least, INFINITY);  // (a barrier)
    float m = s_warp[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, s_warp[w]);

    // ---- sum, and the list of what reaches `least`
    const float base = m == -INFINITY ? 0.f : m;
    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ELEMS; ++i) {
        part[i & 3] += __expf(v[i] - base);
        if (v[i] >= least && v[i] != -INFINITY) {
            const int k = atomicAdd(&s_n, 1);
            const int at = (int)(first + (long)(i / VEC * kThreads + tid) * VEC + i % VEC);
            if (k < kList) s_list[k] = key_of(v[i], at);
        }
    }
    double sum = ((double)part[0] + part[1]) + ((double)part[2] + part[3]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    const long o = row * pieces + piece;
    if (tid == 0) {
        sum = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) sum += s_sum[w];
        out.m[o] = m, out.sum[o] = (float)sum;
    }
    auto put = [&](int rank, unsigned long long key) {
        const uint32_t b = (uint32_t)(key >> 32);
        out.x[o * n + rank] = __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
        out.token[o * n + rank] = (int)(0xffffffffu - (uint32_t)key);
    };
    int found = s_n;
    if (found <= kList) {
        for (int i = tid; i < found; i += kThreads) {
            const unsigned long long key = s_list[i];
            int rank = 0;
            for (int j = 0; j < found && rank < n; ++j) rank += s_list[j] > key;
            if (rank < n) put(rank, key);
        }
    } else {
        unsigned long long last = ~0ull;
        for (found = 0; found < n; ++found) {
            unsigned long long best = 0;
#pragma unroll
            for (int i = 0; i < ELEMS; ++i) {
                const unsigned long long key = key_of(v[i], (int)(first + (long)(i / VEC * kThreads + tid) * VEC + i % VEC));
                if (v[i] != -INFINITY && key < last && key > best) best = key;
            }
            best = warp_max(best);
            if (lane == 0) s_top[warp] = best;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) best = s_top[w] > best ? s_top[w] : best;
            __syncthreads();
            if (best == 0) break;
            if (tid == 0) put(found, best);
            last = best;
        }
    }
    for (int i = min(found, n) + tid; i < n; i += kThreads) out.x[o * n + i] = -INFINITY, out.token[o * n + i] = -1;
}

struct Beam {
    double total;
    int at;  // k V + t
};
__device__ __forceinline__ bool before(double a, int ia, double b, int ib) { return a > b || (a == b && ia < ib); }

__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamSelect p, Pieces in, int pieces) {
    __shared__ double s_lse[kBeamMaxK], s_least[kThreads / 32];
    __shared__ float s_score[kBeamMaxK];
    __shared__ uint8_t s_done[kBeamMaxK];
    __shared__ double s_total[kList];
    __shared__ int s_at[kList];
    __shared__ Beam s_pick[kBeamMaxN];
    __shared__ int s_place[kBeamMaxN];
    __shared__ Beam s_top[kThreads / 32];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.x, K = p.K, n = p.n;
    // scores and flags may be written over below, by this CTA alone
    pdl_wait_primary();
    if (tid == 0) s_n = 0;
    for (int k = tid; k < K; k += kThreads) {
        const float s = p.scores[(long)g * K + k];
        s_score[k] = s != s ? -INFINITY : s;
        s_done[k] = p.finished != nullptr && p.finished[(long)g * K + k] != 0;
    }
    __syncthreads();
    for (int k = warp; k < K; k += kThreads / 32) {
        double lse = -INFINITY;
        if (!s_done[k]) {
            const long o = ((long)g * K + k) * pieces;
            float m = -INFINITY;
            for (int i = lane; i < pieces; i += 32) m = fmaxf(m, __ldcg(in.m + o + i));
            m = warp_max(m);
            double sum = 0;
            for (int i = lane; i < pieces; i += 32) {
                const float mi = __ldcg(in.m + o + i);
                if (mi != -INFINITY) sum += (double)__ldcg(in.sum + o + i) * exp((double)mi - (double)m);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            lse = m == -INFINITY ? -INFINITY : (double)m + log(sum);
        }
        if (lane == 0) s_lse[k] = lse;
    }
    __syncthreads();

    // Candidate c of the group: its total (NaN: none) and place.
    const int per_beam = pieces * n, all = K * per_beam;
    auto candidate = [&](int c, double &total, int &at) {
        const int k = c / per_beam, i = c % per_beam;
        if (s_done[k]) {  // it goes on as it is, once
            total = i == 0 && s_score[k] != -INFINITY ? (double)s_score[k] : NAN;
            at = k * p.V + p.end_token;
            return;
        }
        const long o = ((long)g * K + k) * per_beam + i;
        const float x = __ldcg(in.x + o);
        total = (double)s_score[k] + ((double)x - s_lse[k]);
        at = k * p.V + __ldcg(in.token + o);
        if (x == -INFINITY || !(total > -INFINITY)) total = NAN;
    };
    double mine = -INFINITY;
    for (int c = tid; c < all; c += kThreads) {
        double t;
        int at;
        candidate(c, t, at);
        if (t > mine) mine = t;
    }
    const double least = least_of_maxima(mine, groups_for(n), s_least, (double)INFINITY);
    for (int c = tid; c < all; c += kThreads) {
        double t;
        int at;
        candidate(c, t, at);
        if (t >= least) {
            const int i = atomicAdd(&s_n, 1);
            if (i < kList) s_total[i] = t, s_at[i] = at;
        }
    }
    __syncthreads();
    int found = s_n;
    if (found <= kList) {
        for (int i = tid; i < found; i += kThreads) {
            const double t = s_total[i];
            const int at = s_at[i];
            int rank = 0;
            for (int j = 0; j < found && rank < n; ++j) rank += before(s_total[j], s_at[j], t, at);
            if (rank < n) s_pick[rank] = Beam{t, at};
        }
    } else {
        double lt = INFINITY;
        int la = -1;
        for (found = 0; found < n; ++found) {
            double bt = -INFINITY;
            int ba = INT_MAX;
            for (int c = tid; c < all; c += kThreads) {
                double t;
                int at;
                candidate(c, t, at);
                if (t == t && before(lt, la, t, at) && before(t, at, bt, ba)) bt = t, ba = at;
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const double t = __shfl_xor_sync(0xffffffffu, bt, d);
                const int at = __shfl_xor_sync(0xffffffffu, ba, d);
                if (before(t, at, bt, ba)) bt = t, ba = at;
            }
            if (lane == 0) s_top[warp] = Beam{bt, ba};
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w)
                if (before(s_top[w].total, s_top[w].at, bt, ba)) bt = s_top[w].total, ba = s_top[w].at;
            __syncthreads();
            if (ba == INT_MAX) break;
            if (tid == 0) s_pick[found] = Beam{bt, ba};
            lt = bt, la = ba;
        }
    }
    found = min(found, n);
    __syncthreads();
    if (tid == 0) {
        // too few: the lowest places of those that are left, all of them at -inf
        for (int at = 0; found < n; ++at) {
            bool have = false;
            for (int i = 0; i < found; ++i) have |= s_pick[i].at == at;
            if (!have) s_pick[found++] = Beam{-INFINITY, at};
        }
        for (int i = 0; i < n; ++i) s_place[i] = i;
        if (p.keep_rows) {  // a beam's best child takes its row, the others take the rows that are left in order
            for (int i = 0; i < n; ++i) s_place[i] = -1;
            for (int i = 0; i < n; ++i) {
                const int k = s_pick[i].at / p.V;
                if (s_place[k] < 0) s_place[k] = i, s_at[i] = 1;
                else s_at[i] = 0;
            }
            int row = 0;
            for (int i = 0; i < n; ++i)
                if (!s_at[i]) {
                    while (s_place[row] >= 0) ++row;
                    s_place[row] = i;
                }
        }
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const Beam b = s_pick[s_place[i]];
        const int k = b.at / p.V, token = b.at % p.V;
        const long o = (long)g * n + i;
        p.tokens[o] = token;
        p.parents[o] = g * K + k;
        p.scores_out[o] = (float)b.total;
        if (p.finished_out != nullptr) p.finished_out[o] = s_done[k] || token == p.end_token;
    }
}

// A piece of 8 values a thread while that leaves SMs without a CTA, 32 otherwise.
int piece_size(int rows, int V, int dtype) {
    return (long)rows * ((V + 8191) / 8192) < 4 * 152 ? 2048 : 8192;
}
int piece_count(int rows, int V, int dtype) {
    const int size = piece_size(rows, V, dtype);
    return (int)(((long)V + 7 + size - 1) / size);  // (up to 7 values of the first vector lie before the row)
}

template <typename T, int ELEMS>
cudaError_t launch_pieces(const BeamSelect &p, const Pieces &w, int pieces, cudaStream_t s) {
    const cudaError_t e =
        launch_kernel(beam_pieces_kernel<T, ELEMS>, dim3((unsigned)(p.G * p.K * pieces)), dim3(kThreads), 0, s, true,
                      static_cast<const T *>(p.logits), p.stride, p.finished, w, p.V, p.n, pieces);
    note_launch();
    return e;
}

}  // namespace

size_t beam_select_workspace(int G, int K, int V, int n) {
    // (of the two piece sizes the one that asks for more)
    const size_t rows = (size_t)G * K, pieces = (size_t)piece_count(G * K, V, 0);
    return rows * pieces * (8 + 8 * (size_t)n);
}

bool beam_select_fits(int G, int K, int V, int n) {
    return (long)G * K * piece_count(G * K, V, 0) <= INT_MAX && (long)K * piece_count(G * K, V, 0) * n <= INT_MAX;
}

cudaError_t launch_beam_select(const BeamSelect &p, int dtype, void *ws, cudaStream_t s) {
    const int rows = p.G * p.K, pieces = piece_count(rows, p.V, dtype);
    const size_t all = (size_t)rows * pieces;
    Pieces w;
    w.m = static_cast<float *>(ws), w.sum = w.m + all, w.x = w.sum + all;
    w.token = reinterpret_cast<int *>(w.x + all * p.n);
    const bool small = piece_size(rows, p.V, dtype) == 2048;
    cudaError_t e;
    if (dtype == GDN_BF16)
        e = small ? launch_pieces<__nv_bfloat16, 8>(p, w, pieces, s) : launch_pieces<__nv_bfloat16, 32>(p, w, pieces, s);
    else
        e = small ? launch_pieces<float, 8>(p, w, pieces, s) : launch_pieces<float, 32>(p, w, pieces, s);
    if (e != cudaSuccess) return e;
    e = launch_kernel(beam_join_kernel, dim3((unsigned)p.G), dim3(kThreads), 0, s, true, p, w, pieces);
    note_launch();
    return e;
}

}  // namespace gdn
