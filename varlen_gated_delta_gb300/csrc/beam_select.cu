// beam_select.cu - gdn_beam_select: the best continuations of each group of beams.
//
//   total[g, k, t] = score[g, k] + x[g, k, t] - log sum_t' exp x[g, k, t'],
// and of a group's K V totals the n largest.  Of equal ones the lowest beam comes first, within a beam the largest logit (a
// score of -1e30 leaves nothing of the logits in 64 bits), then the lowest token.  The logits are read once, in two launches.
//
// The first gives a CTA a span of a row, which it goes through in pieces that fit its registers, with the largest logit m, the
// sum of exp(x - m), and the n largest logits so far.  In a first piece (with at least n values above -inf, else in the
// next too) the threads form groups whose maxima are at hand: at least n values reach the n-th largest of them, and few
// more do (n = 8 of 32 groups: some 9 of 16384 values).  Later pieces have few values above the n-th largest so far.  Those
// go into a list and are ranked by counting, together with the ones before.  A list that overflows (equal or rising
// logits) is left for n rounds of the CTA-wide largest value below the last one.
//
// The second, a CTA to a group of beams, joins the spans' sums, and takes the n best of their candidates the
// same way.  Totals and their comparison are in 64 bits: only the error of the row's sum (fp32 terms, a thread's of a
// piece added in fp32, all after that in two values) is left in the order of beams.  Measured against 64 bits, the logarithm of
// the sum is off by at most 4e-8 where no few terms dominate (normal logits of deviation 0.5 and 1, 1000 to 200000 of
// them; most of it the same for all rows), and by at most 4.9e-7 where one does.
//
// 64 x 8 beams of 131072 bf16 logits, a tenth of the beams at their end: 46 us, 2.6 TB/s.  Reading is not what bounds it: 20
// million warp instructions at two a clock (two fifths of them exponentials and the conversions before them), and warps that wait
// for a piece's ranking.  One launch's pieces without the next one's loads in flight: 55 us; one piece to a CTA: 57.
// One group of 4 x 32768: 9 us, two launches and chains of dependent steps.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "serving.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kList = 512;  // candidates that are ranked by counting
constexpr int kSpanTarget = 8 * 152;  // spans to go for
constexpr int kNear = 2560;  // candidates of a group that are kept in shared memory

struct Spans {   // in the workspace
    float *m;    // [rows][spans]: the largest; -inf: nothing but -inf
    float2 *sum;  // [rows][spans]: sum of exp(x - m), in two values
    float *x;    // [rows][spans][n]: the largest logits, descending; -inf past the last
    int *token;  // [rows][spans][n]
};

// A value in the order of its bits as an unsigned number, and the position behind it: of equal values the
// lowest position is the largest key.
__device__ __forceinline__ unsigned long long key_of(float x, int at) {
    const uint32_t b = __float_as_uint(x + 0.f);  // (no negative zeros)
    return (unsigned long long)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xffffffffu - (uint32_t)at);
}
// The same for 64 bits, and back.  Keys are compared as whole numbers: the 64-bit pipe takes two lanes a clock.
__device__ __forceinline__ unsigned long long key_of(double x) {
    const unsigned long long b = __double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double of_key(unsigned long long k) { return __longlong_as_double(k >> 63 ? k & ~(1ull << 63) : ~k); }

template <typename T>
__device__ __forceinline__ T warp_max(T x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const T y = __shfl_xor_sync(0xffffffffu, x, d);
        x = y > x ? y : x;
    }
    return x;
}

// A sum held in two values: x + y = hi + lo exactly, added to lo.
__device__ __forceinline__ void add_two(float &hi, float &lo, float y, float y_lo) {
    const float s = __fadd_rn(hi, y), back = __fsub_rn(s, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, back)), __fsub_rn(y, back)) + y_lo;
    hi = s;
}
// hi + lo times e^-d, d >= 0: d = n ln 2 + r (the product n ln 2 exact in two values), e^-r from its series, whose terms past
// r^8 are below 2^-31 for |r| <= 0.35.  2^-27 off at most.
__device__ __forceinline__ void scale_two(float &hi, float &lo, float d) {
    if (d == 0.f) return;
    if (d > 80.f) {  // (nothing beside the largest; a NaN goes on)
        hi = lo = 0.f;
        return;
    }
    constexpr float kLn2 = 0.69314718246f, kLn2Lo = -1.9046543e-9f;  // ln 2 in two values
    const float n = rintf(d * 1.44269504f), p = __fmul_rn(n, kLn2);
    const float r = __fsub_rn(p, d), r_lo = __fmaf_rn(n, kLn2, -p) + n * kLn2Lo;  // e^-d = 2^-n e^(r + r_lo)
    float q = 1.f / 40320;
    q = fmaf(q, r, 1.f / 5040), q = fmaf(q, r, 1.f / 720), q = fmaf(q, r, 1.f / 120), q = fmaf(q, r, 1.f / 24);
    q = fmaf(q, r, 1.f / 6), q = fmaf(q, r, 0.5f);
    const float one = __fadd_rn(1.f, r), rest = q * (r * r);
    const float tail = __fadd_rn(__fsub_rn(1.f, one), r) + fmaf(r_lo, one + rest, rest);
    const float both = __fadd_rn(one, tail), power = __int_as_float((127 - (int)n) << 23);
    const float f = both * power, f_lo = __fsub_rn(tail, __fsub_rn(both, one)) * power;
    const float x = __fmul_rn(hi, f);
    lo = __fmaf_rn(hi, f, -x) + fmaf(hi, f_lo, lo * f);
    hi = x;
}
__device__ __forceinline__ void warp_sum_two(float &hi, float &lo) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, hi, d), y_lo = __shfl_xor_sync(0xffffffffu, lo, d);
        add_two(hi, lo, y, y_lo);
    }
}

// The n-th largest (any of them, if there are fewer) of the maxima of `groups` (32 or 256) equal sets of neighbouring
// threads, and the largest.
__device__ __forceinline__ float nth_maximum(float x, int n, int groups, float *s_all, float2 *s_nth, float &top) {
    const int tid = threadIdx.x;
    if (groups == 32) {  // (one warp ranks them)
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        if (tid % 8 == 0) s_all[tid / 8] = x;
    } else {
        s_all[tid] = x;
    }
    __syncthreads();
    if (tid < groups) {
        x = s_all[tid];
        int larger = 0;
#pragma unroll 8
        for (int i = 0; i < groups; i += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(s_all + i);
            larger += (y.x > x) + (y.y > x) + (y.z > x) + (y.w > x);
        }
        float nth = larger < n ? x : INFINITY;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            nth = fminf(nth, __shfl_xor_sync(0xffffffffu, nth, d));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        }
        if ((tid & 31) == 0) s_nth[tid >> 5] = make_float2(nth, x);
    }
    __syncthreads();
    float2 y = s_nth[0];
    for (int w = 1; w < groups / 32; ++w) y.x = fminf(y.x, s_nth[w].x), y.y = fmaxf(y.y, s_nth[w].y);
    top = y.y;
    return y.x;
}

__device__ __forceinline__ float of_key(uint32_t high) {
    return __uint_as_float(high & 0x80000000u ? high & 0x7fffffffu : ~high);
}

// Vectors of a warp in a row of its stage.  SKEWED: some rows do not begin on 16-byte boundaries, and values are shifted
// into their places when they come from the stage (64 x 8 beams of 131071: 55 us; 51 with sums in the order of
// addresses, which differ from row to row).
constexpr int warp_row(bool skewed) { return skewed ? 33 : 32; }

template <typename T, int ELEMS, bool SKEWED>
__global__ void __launch_bounds__(kThreads, ELEMS <= 8 ? 6 : 3)
    beam_spans_kernel(const T *__restrict__ logits, long stride, const uint8_t *__restrict__ finished, Spans out, int V,
                      int n, int spans, int pieces) {
    constexpr int VEC = 16 / sizeof(T), VECS = ELEMS / VEC;
    using Key = unsigned long long;
    // [2 stages][VECS][8 warps][32 or 33]: each warp's vectors of a piece and of the next (SKEWED: and the one behind them)
    extern __shared__ uint4 s_data[];
    constexpr int kWarp = warp_row(SKEWED), kRow = kThreads / 32 * kWarp, kStage = VECS * kRow;
    __shared__ __align__(16) float s_all[kThreads];
    __shared__ Key s_list[kList], s_top[kThreads / 32], s_best[2][kBeamMaxN];
    __shared__ float2 s_nth[kThreads / 32];
    __shared__ int s_n[3];  // of a piece; cleared a piece before its turn, when nobody looks at it
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long row = blockIdx.x / spans;
    const int span = blockIdx.x % spans;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (finished != nullptr && __ldg(finished + row) != 0) return;  // (nothing of it is looked at)
    const T *x = logits + row * stride;
    // Copied vectors lie on 16-byte boundaries, which a row may begin `skew` values behind.  A thread's values are the same wherever
    // a row begins, so that equal rows have equal sums.  (Places up to a piece past V fit: beam_select_fits)
    const int skew = SKEWED ? (int)(((uintptr_t)x / sizeof(T)) % VEC) : 0;
    const int from = span * pieces * (ELEMS * kThreads);
    if (tid < 3) s_n[tid] = 0;

    constexpr float kL = 1.4426950408889634f;
    float sum = 0.f, sum_lo = 0.f;  // of this thread
    float base = -INFINITY;         // m
    float least = -INFINITY;        // the n-th largest so far
    int have = 0;                   // best ones so far, in s_best[piece & 1]
    const auto fetch = [&](int piece) {
        const int first = from + piece * (ELEMS * kThreads);
        if (piece < pieces && first < V) {
            uint4 *stage = s_data + (piece & 1) * kStage + warp * kWarp;
            const auto copy = [&](int j, int i) {  // the warp's vector i of row j
                const int at = first - skew + (j * kThreads + warp * 32 + i) * VEC;
                if (at >= 0 && at <= V - VEC) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(stage + j * kRow + i)),
                                 "l"(x + at)
                                 : "memory");
                } else {
                    Vec16<T> w;
#pragma unroll
                    for (int k = 0; k < VEC; ++k) w.v[k] = at + k >= 0 && at + k < V ? x[at + k] : from_f32<T>(-INFINITY);
                    stage[j * kRow + i] = w.u;
                }
            };
#pragma unroll
            for (int j = 0; j < VECS; ++j) copy(j, lane);
            if (SKEWED && lane < VECS) copy(lane, 32);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
#pragma unroll 1
    for (int piece = 0; piece < pieces; ++piece) {
        const int first = from + piece * (ELEMS * kThreads);
        if (first >= V) break;
        fetch(piece + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();  // (the warp's vectors are here: its lanes read each other's, also below)
        const uint4 *stage = s_data + (piece & 1) * kStage + warp * kWarp;
        // value i of a lane
        const auto held = [&](int lane, int i) { return to_f32(reinterpret_cast<const T *>(stage + i / VEC * kRow + lane)[skew + i % VEC]); };
        Vec16<T> w[VECS];
        if constexpr (!SKEWED) {
#pragma unroll
            for (int j = 0; j < VECS; ++j) w[j].u = stage[j * kRow + lane];
        } else {
            const auto shifted = [&](auto words) {  // by so many words, and half a one
                constexpr int k = decltype(words)::value;
                const int bits = sizeof(T) == 2 && (skew & 1) ? 16 : 0;
#pragma unroll
                for (int j = 0; j < VECS; ++j) {
                    const uint4 a = stage[j * kRow + lane], b = stage[j * kRow + lane + 1];
                    const uint32_t c[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                    w[j].u = make_uint4(__funnelshift_r(c[k], c[k + 1], bits), __funnelshift_r(c[k + 1], c[k + 2], bits),
                                        __funnelshift_r(c[k + 2], c[k + 3], bits), __funnelshift_r(c[k + 3], c[k + 4], bits));
                }
            };
            switch (skew * (int)sizeof(T) / 4) {
            case 0: shifted(std::integral_constant<int, 0>()); break;
            case 1: shifted(std::integral_constant<int, 1>()); break;
            case 2: shifted(std::integral_constant<int, 2>()); break;
            default: shifted(std::integral_constant<int, 3>());
            }
        }
        const auto value = [&](int i) { return to_f32(w[i / VEC].v[i % VEC]); };
        const auto token = [&](int i) { return first + (i / VEC * kThreads + tid) * VEC + i % VEC; };
        // (NaN is passed over: it is no candidate)
        float mine = -INFINITY;
        if constexpr (sizeof(T) == 2) {
            __nv_bfloat162 top = __float2bfloat162_rn(-INFINITY);
#pragma unroll
            for (int j = 0; j < VECS; ++j)
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) top = __hmax2(top, reinterpret_cast<const __nv_bfloat162 *>(w + j)[i]);
            mine = fmaxf(__low2float(top), __high2float(top));
        } else {
#pragma unroll
            for (int i = 0; i < ELEMS; ++i) mine = fmaxf(mine, value(i));
        }

        // ---- the list of what may be among the n largest: values from this piece's n-th largest on (or near it), or above the
        // n-th largest of earlier pieces, whose places are lower
        bool some;
        float reach;
        if (have < n) {
            float top;
            reach = nth_maximum(mine, n, n <= 32 ? 32 : kThreads, s_all, s_nth, top);  // (barriers)
            some = mine >= reach && mine != -INFINITY;
        } else {
            reach = nextafterf(least, INFINITY);
            some = mine > least;
        }
        // Few threads have such values: the warp looks at those of one of them at a time.
        for (unsigned left = __ballot_sync(0xffffffffu, some); left != 0; left &= left - 1)
#pragma unroll
            for (int e = lane; e < ELEMS; e += 32) {
                const int of = __ffs(left) - 1, at = first + (e / VEC * kThreads + warp * 32 + of) * VEC + e % VEC;
                const float v = fmaxf(held(of, e), -INFINITY);
                if (v >= reach && v != -INFINITY) {
                    const int k = atomicAdd(&s_n[piece % 3], 1);
                    if (k < kList) s_list[k] = key_of(v, at);
                }
            }
        const bool any = __syncthreads_or(some);
        if (tid == 0) s_n[(piece + 2) % 3] = 0;
        if (any) {
            const Key *best = s_best[piece & 1];
            Key *next = s_best[(piece & 1) ^ 1];
            int found = s_n[piece % 3];
            if (found <= kList) {
                for (int i = tid; i < have + found; i += kThreads) {
                    const Key key = i < have ? best[i] : s_list[i - have];
                    int rank = 0;
#pragma unroll 8
                    for (int j = 0; j < have; ++j) rank += best[j] > key;
#pragma unroll 8
                    for (int j = 0; j < found; ++j) rank += s_list[j] > key;
                    if (rank < n) next[rank] = key;
                }
                have = min(n, have + found);
            } else {
                Key last = ~0ull;
                for (found = 0; found < n; ++found) {
                    Key top = tid < have && best[tid] < last ? best[tid] : 0;
#pragma unroll 4
                    for (int i = 0; i < ELEMS; ++i) {
                        const float v = fmaxf(held(lane, i), -INFINITY);
                        const Key key = key_of(v, token(i));
                        if (v != -INFINITY && key < last && key > top) top = key;
                    }
                    top = warp_max(top);
                    if (lane == 0) s_top[warp] = top;
                    __syncthreads();
#pragma unroll
                    for (int w = 0; w < kThreads / 32; ++w) top = s_top[w] > top ? s_top[w] : top;
                    __syncthreads();
                    if (top == 0) break;
                    if (tid == 0) next[found] = top;
                    last = top;
                }
                have = found;
            }
            __syncthreads();
            // (have > 0: some value was above -inf)
            const float top = of_key((uint32_t)(next[0] >> 32));
            if (have == n) least = of_key((uint32_t)(next[n - 1] >> 32));
            if (top > base) {
                if (base != -INFINITY) scale_two(sum, sum_lo, top - base);
                base = top;
            }
        } else {  // the best ones stay: in the place where the next piece looks for them
            if (tid < have) s_best[(piece & 1) ^ 1][tid] = s_best[piece & 1][tid];
        }

        // ---- sum of exp(x - m) = 2^(x L - m L), L = log2(e): a product and a sum in one rounding, and the rounding of m L, which
        // all terms share, is taken back at the end (2^-t = 1 - t ln 2 + ..., t < 2^-10).  Large m, or a NaN: x - m first.
        if (base != -INFINITY) {
            const float mL = __fmul_rn(base, kL);
            const auto sum_of = [&](auto term) {
                float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int i = 0; i < ELEMS; i += 2) {
                    float2 e = term(make_float2(value(i), value(i + 1)));
                    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
                    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
                    part[i / 2 & 1] = __fadd2_rn(part[i / 2 & 1], e);
                }
                const float2 both = __fadd2_rn(part[0], part[1]);
                return both.x + both.y;
            };
            float more_lo = 0.f, more = sum_of([&](float2 x) { return __ffma2_rn(x, make_float2(kL, kL), make_float2(-mL, -mL)); });
            const float t = 0.69314718f * __fmaf_rn(base, kL, -mL);
            if (more != more || fabsf(base) > 8192.f)
                more = sum_of([&](float2 x) {
                    return make_float2((fmaxf(x.x, -INFINITY) - base) * kL, (fmaxf(x.y, -INFINITY) - base) * kL);
                });
            else
                more_lo = more * (t * (0.5f * t - 1.f));
            add_two(sum, sum_lo, more, more_lo);
        }
        if (piece + 1 == pieces || first + ELEMS * kThreads >= V) {  // the span's end
            warp_sum_two(sum, sum_lo);
            __syncthreads();
            if (lane == 0) s_nth[warp] = make_float2(sum, sum_lo);
            __syncthreads();
            const long o = row * spans + span;
            if (tid == 0) {
#pragma unroll
                for (int w = 1; w < kThreads / 32; ++w) add_two(sum, sum_lo, s_nth[w].x, s_nth[w].y);
                out.m[o] = base, out.sum[o] = make_float2(sum, sum_lo);
            }
            const Key *best = s_best[(piece & 1) ^ 1];
            for (int i = tid; i < n; i += kThreads) {
                out.x[o * n + i] = i < have ? of_key((uint32_t)(best[i] >> 32)) : -INFINITY;
                out.token[o * n + i] = i < have ? (int)(0xffffffffu - (uint32_t)best[i]) : -1;
            }
        }
    }
    // (a span that begins past V: rounding up may leave one)
    if (from >= V) {
        const long o = row * spans + span;
        if (tid == 0) out.m[o] = -INFINITY, out.sum[o] = make_float2(0.f, 0.f);
        for (int i = tid; i < n; i += kThreads) out.x[o * n + i] = -INFINITY, out.token[o * n + i] = -1;
    }
}

// A continuation: the larger key comes first, of equal totals the larger place (the lowest beam, in it the largest logit, of
// equal ones the lowest token).
struct Pick {
    unsigned long long total;  // key_of
    unsigned long long place;  // K - 1 - k; the logit's key; 2^bits - 1 - t
};
__device__ __forceinline__ bool before(unsigned long long a, unsigned long long ia, unsigned long long b, unsigned long long ib) {
    return a > b || (a == b && ia > ib);
}

__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamSelect p, Spans in, int spans) {
    __shared__ double s_lse[kBeamMaxK];
    __shared__ __align__(16) float s_all[kThreads];
    __shared__ float2 s_least[kThreads / 32];
    __shared__ float s_score[kBeamMaxK], s_m[kBeamMaxK], s_lse32[kBeamMaxK];
    __shared__ float2 s_sum[kBeamMaxK];
    __shared__ uint8_t s_done[kBeamMaxK];
    __shared__ unsigned long long s_total[kList];
    __shared__ unsigned long long s_key[kList];
    __shared__ int s_first[kBeamMaxN], s_place[kBeamMaxN], s_rest[kBeamMaxN];
    __shared__ Pick s_pick[kBeamMaxN], s_top[kThreads / 32];
    __shared__ float s_x[kNear];
    __shared__ int s_token[kNear];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.x, K = p.K, n = p.n;
    const int per_beam = spans * n, all = K * per_beam;
    pdl_wait_primary();
    // All that is read comes at once: the candidates (as many as there is room for), scores and flags (which may be written
    // over below, by this CTA alone), and the spans' sums.
#pragma unroll 4
    for (int c = tid; c < min(all, kNear); c += kThreads) {
        s_x[c] = __ldcg(in.x + (long)g * all + c);
        s_token[c] = __ldcg(in.token + (long)g * all + c);
    }
    if (tid == 0) s_n = 0;
    for (int k = tid; k < K; k += kThreads) {
        const float s = p.scores[(long)g * K + k];
        s_score[k] = s != s ? -INFINITY : s;
        s_done[k] = p.finished != nullptr && p.finished[(long)g * K + k] != 0;
    }
    for (int k = warp; k < K; k += kThreads / 32) {  // (of a beam at its end: of no meaning)
        const long o = ((long)g * K + k) * spans;
        float m = -INFINITY, sum = 0.f, lo = 0.f;
        for (int i0 = 0; i0 < spans; i0 += 32) {
            const int i = i0 + lane;
            const float mi = i < spans ? __ldcg(in.m + o + i) : -INFINITY;
            float2 si = i < spans ? __ldcg(in.sum + o + i) : make_float2(0.f, 0.f);
            const float top = fmaxf(m, warp_max(mi));
            if (top > m && m != -INFINITY) scale_two(sum, lo, top - m);
            m = top;
            if (mi != -INFINITY) {
                scale_two(si.x, si.y, m - mi);
                add_two(sum, lo, si.x, si.y);
            }
        }
        warp_sum_two(sum, lo);
        if (lane == 0) s_m[k] = m, s_sum[k] = make_float2(sum, lo);
    }
    __syncthreads();
    for (int k = tid; k < K; k += kThreads) {
        const double lse = s_done[k] || s_m[k] == -INFINITY ? -INFINITY : (double)s_m[k] + log((double)s_sum[k].x + s_sum[k].y);
        s_lse[k] = lse, s_lse32[k] = (float)lse;
    }
    __syncthreads();

    // Candidate c of the group: beam and logit; -inf: none.  (A beam at its end goes on as it is, once.)
    auto logit = [&](int c, int k) {
        if (s_done[k]) return c - k * per_beam == 0 ? 0.f : -INFINITY;
        return c < kNear ? s_x[c] : __ldcg(in.x + (long)g * all + c);
    };
    // Its total in 32 bits, near enough to leave most of them out.
    auto about = [&](float x, int k) { return s_done[k] ? s_score[k] + x : s_score[k] + (x - s_lse32[k]); };
    auto total = [&](int c, int k, float x) {
        return key_of(s_done[k] ? (double)s_score[k] : (double)s_score[k] + ((double)x - s_lse[k]));
    };
    // How far that may be off: the row's term, the two sums and this bound's own are rounded to 2^-24 of these sizes each.
    auto off = [&](float x, int k) { return (fabsf(x) + (s_done[k] ? 0.f : fabsf(s_lse32[k])) + fabsf(s_score[k])) * 0x1p-21f; };
    const int bits = p.V > 1 ? 32 - __clz(p.V - 1) : 0;  // of a token (bits of K and V together: at most 32)
    const uint32_t mask = (1u << bits) - 1u;
    auto place = [&](int c, int k, float x) {
        const uint32_t t = s_done[k] ? p.end_token : c < kNear ? s_token[c] : __ldcg(in.token + (long)g * all + c);
        return (unsigned long long)(K - 1 - k) << (32 + bits) | (key_of(x, 0) >> 32) << bits | (mask - t);
    };
    auto beam_of = [&](const Pick &b) { return K - 1 - (int)(b.place >> (32 + bits)); };
    auto token_of = [&](const Pick &b) { return (int)(mask - ((uint32_t)b.place & mask)); };
    float mine = -INFINITY;
    for (int c = tid; c < all; c += kThreads) {
        const int k = c / per_beam;
        const float x = logit(c, k), t = about(x, k);
        if (x != -INFINITY && t > -INFINITY) mine = fmaxf(mine, t - off(x, k));  // (passes over inf - inf)
    }
    float best;  // (barriers)
    const float reach = nth_maximum(mine, n, kThreads, s_all, s_least, best);
    for (int c = tid; c < all; c += kThreads) {
        const int k = c / per_beam;
        const float x = logit(c, k), t = about(x, k);
        if (x != -INFINITY && t > -INFINITY && t + off(x, k) >= reach) {
            const int i = atomicAdd(&s_n, 1);
            if (i < kList) s_total[i] = total(c, k, x), s_key[i] = place(c, k, x);
        }
    }
    __syncthreads();
    int found = s_n;
    if (found <= kList) {
        for (int i = tid; i < found; i += kThreads) {
            const unsigned long long t = s_total[i], at = s_key[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < found; ++j) rank += before(s_total[j], s_key[j], t, at);
            if (rank < n) s_pick[rank] = Pick{t, at};
        }
    } else {
        Pick last{~0ull, ~0ull};
        for (found = 0; found < n; ++found) {
            Pick top{0, 0};
            for (int c = tid; c < all; c += kThreads) {
                const int k = c / per_beam;
                const float x = logit(c, k);
                if (x == -INFINITY || !(about(x, k) > -INFINITY)) continue;
                const unsigned long long t = total(c, k, x), at = place(c, k, x);
                if (before(last.total, last.place, t, at) && before(t, at, top.total, top.place)) top = Pick{t, at};
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const unsigned long long t = __shfl_xor_sync(0xffffffffu, top.total, d), at = __shfl_xor_sync(0xffffffffu, top.place, d);
                if (before(t, at, top.total, top.place)) top = Pick{t, at};
            }
            if (lane == 0) s_top[warp] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w)
                if (before(s_top[w].total, s_top[w].place, top.total, top.place)) top = s_top[w];
            __syncthreads();
            if (top.total == 0) break;
            if (tid == 0) s_pick[found] = top;
            last = top;
        }
    }
    found = min(found, n);
    __syncthreads();
    if (tid == 0 && found < n) {
        // too few: the lowest places of those that are left, all of them at -inf
        const int had = found;
        for (int k = 0, t = 0; found < n; t + 1 < p.V ? ++t : (t = 0, ++k)) {
            bool have = false;
            for (int i = 0; i < had; ++i) have |= beam_of(s_pick[i]) == k && token_of(s_pick[i]) == t;
            if (!have) s_pick[found++] = Pick{key_of(-(double)INFINITY), (unsigned long long)(K - 1 - k) << (32 + bits) | (mask - t)};
        }
    }
    __syncthreads();
    // With keep_rows a beam's best child takes its row; the others, in order, the rows that are left.
    if (p.keep_rows) {
        for (int i = tid; i < n; i += kThreads) s_rest[i] = -1;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            const int k = beam_of(s_pick[i]);
            bool best = true;
            for (int j = 0; j < i; ++j) best &= beam_of(s_pick[j]) != k;
            s_first[i] = best ? k : -1;
            if (best) s_rest[k] = i;
        }
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            if (s_rest[i] >= 0) s_place[i] = s_rest[i];
            if (s_first[i] >= 0) continue;
            int others = 0, row = -1;  // the others before this one, and the row that many are left before
            for (int j = 0; j < i; ++j) others += s_first[j] < 0;
            while (others >= 0) others -= s_rest[++row] < 0;
            s_place[row] = i;
        }
        __syncthreads();
    }
    for (int i = tid; i < n; i += kThreads) {
        const Pick b = s_pick[p.keep_rows ? s_place[i] : i];
        const int k = beam_of(b), token = token_of(b);
        const long o = (long)g * n + i;
        p.tokens[o] = token;
        p.parents[o] = g * K + k;
        p.scores_out[o] = (float)of_key(b.total);
        if (p.finished_out != nullptr) p.finished_out[o] = s_done[k] || token == p.end_token;
    }
}

// How rows are cut: pieces of 128 bytes to a thread, several to a span where there are spans enough for all SMs; 8 values to a
// thread while that leaves SMs without work.
struct Cut {
    int elems, spans, pieces;  // of a thread; of a row; of a span
};
Cut cut_rows(int rows, int V, int dtype) {
    const auto pieces = [&](int elems) { return (int)(((long)V + elems * kThreads - 1) / (elems * kThreads)); };
    Cut c;
    c.elems = dtype == GDN_BF16 ? 64 : 32;
    int all = pieces(c.elems);
    if ((long)rows * all < 4 * 152) return Cut{8, pieces(8), 1};
    const int spans = std::max(1, std::min(all, (kSpanTarget + rows - 1) / rows));
    c.pieces = (all + spans - 1) / spans;
    c.spans = (all + c.pieces - 1) / c.pieces;
    return c;
}
int most_spans(int rows, int V) { return std::max(cut_rows(rows, V, GDN_BF16).spans, cut_rows(rows, V, GDN_F32).spans); }

template <typename T, int ELEMS, bool SKEWED>
cudaError_t launch_spans(const BeamSelect &p, const Spans &w, const Cut &c, cudaStream_t s) {
    constexpr int kBytes = 2 * (ELEMS * sizeof(T)) * (kThreads / 32 * warp_row(SKEWED));
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(beam_spans_kernel<T, ELEMS, SKEWED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    });
    if (e != cudaSuccess) return e;
    e = launch_kernel(beam_spans_kernel<T, ELEMS, SKEWED>, dim3((unsigned)(p.G * p.K * c.spans)), dim3(kThreads), kBytes, s, true,
                      static_cast<const T *>(p.logits), p.stride, p.finished, w, p.V, p.n, c.spans, c.pieces);
    note_launch();
    return e;
}
template <typename T, int ELEMS>
cudaError_t launch_spans(const BeamSelect &p, const Spans &w, const Cut &c, cudaStream_t s) {
    const bool aligned = (uintptr_t)p.logits % 16 == 0 && (p.G * p.K == 1 || p.stride * sizeof(T) % 16 == 0);
    return aligned ? launch_spans<T, ELEMS, false>(p, w, c, s) : launch_spans<T, ELEMS, true>(p, w, c, s);
}

}  // namespace

size_t beam_select_workspace(int G, int K, int V, int n) {
    return (size_t)G * K * most_spans(G * K, V) * (12 + 8 * (size_t)n);
}

bool beam_select_fits(int G, int K, int V, int n) {
    if (V > INT_MAX - 4 * 64 * kThreads) return false;
    const long spans = most_spans(G * K, V);
    return (long)G * K * spans <= INT_MAX && K * spans * n <= INT_MAX;
}

cudaError_t launch_beam_select(const BeamSelect &p, int dtype, void *ws, cudaStream_t s) {
    const int rows = p.G * p.K;
    const Cut c = cut_rows(rows, p.V, dtype);
    const size_t all = (size_t)rows * c.spans;
    Spans w;
    w.sum = static_cast<float2 *>(ws), w.m = reinterpret_cast<float *>(w.sum + all), w.x = w.m + all;
    w.token = reinterpret_cast<int *>(w.x + all * p.n);
    cudaError_t e;
    if (dtype == GDN_BF16)
        e = c.elems == 8 ? launch_spans<__nv_bfloat16, 8>(p, w, c, s) : launch_spans<__nv_bfloat16, 64>(p, w, c, s);
    else
        e = c.elems == 8 ? launch_spans<float, 8>(p, w, c, s) : launch_spans<float, 32>(p, w, c, s);
    if (e != cudaSuccess) return e;
    e = launch_kernel(beam_join_kernel, dim3((unsigned)p.G), dim3(kThreads), 0, s, true, p, w, c.spans);
    note_launch();
    return e;
}

}  // namespace gdn
