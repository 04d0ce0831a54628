// attention_f32.cu - softmax attention with fp32 accuracy: fp32 activations, and
// any head width and alignment that the bf16 kernels do not take.
//
// The query heads of one key-value head share its keys, so a tile holds ROWS
// (token, head) pairs of one key-value head, token-major: row r is token r / G,
// head r % G.  Keys go by in tiles of 64 with the running maximum m and sum l
// of the softmax, in base 2: with x = scale log2(e) q k,
//   m' = max(m, max x),  l' = l 2^(m - m') + sum 2^(x - m'),  o' likewise,
// and o / l at the end.
//
// The products run on the tensor cores as sums of tf32 products: x = hi + lo, each
// with 10 explicit bits, leaves out less than 2^-21 |x|, and a b is taken as hi hi'
// + (hi lo' + lo hi'), which leaves out another 2^-22 |a b|.  The large and
// the small terms of a score have accumulators of their own, and the output of
// a key tile is summed apart and then added in fp32, so that few additions
// round inside the tensor cores.  Infinities, and what rounds up to one, have no such
// split: scores that come out NaN are taken again as plain sums, and a tile whose output
// is not finite goes by a second time, without the non-finite values, which then join the
// rows that see them.  Bound by these products (mma.sync in tf32, three for
// each one wanted) and their latency: the tensor pipe is 50% active, and the two warps
// of a scheduler mostly wait for it or for a product's result.  471 us, 35 TFLOP/s, for 4 x 1000 tokens, 16
// heads of 128 on 4, where multiply-adds on the fp32 pipe in the same tiles took
// 558 us, and 301 against 445 us for 2 histories of up to 101321 tokens.
//
// Tiles sit in shared memory as fp32, the next one on its way under the products.
// The k index of both products is permuted (t <-> 2 t, t + 4 <-> 2 t + 1 within
// eight), so that q and k fragments are 8-byte loads and the accumulators of the
// scores are the operand of the second product as they are.  Eight warps are MT
// row groups of 16 times WK key groups, which join at the end.  Over a paged cache
// the keys of a tile are split `splits` ways (grid z) when tiles are few; each
// split leaves m, l and an unscaled o for a second kernel.
#include "attention.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kKeys = 64;
constexpr int kMaxSplits = 128;

template <int DP, int MT>
struct F32 {
    static constexpr int ROWS = 16 * MT, WK = 8 / MT, KW = kKeys / WK;
    static constexpr int LD = DP + 8, LDV = DP + 4;  // floats a row: fragment loads meet every bank once
    static constexpr size_t SMEM = (size_t)(ROWS * LD + kKeys * LD + kKeys * LDV) * 4;
    static_assert(WK == 1 || ROWS * DP <= kKeys * LD + kKeys * LDV, "the join uses the key tiles' place");
};

// x = hi + lo: hi is x rounded to the 10 explicit bits of tf32 (by an integer addition: the
// conversion instruction runs at a fraction of its rate), lo is exact, and the product reads the
// upper 10 of its bits.  NaN stays in lo, whatever the addition makes of hi.
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma1688(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes to shared memory, or zeros
__device__ __forceinline__ void copy16(float *dst, const void *src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(read ? 16 : 0)
                 : "memory");
}

// `rows` rows of D values (row r at off(r), or zeros when off(r) < 0) into
// shared memory, LD floats apart, columns from D on zero; aligned fp32 rows by
// copies that are in flight until copies_landed().
template <typename T, int DP, int LD, typename Off>
__device__ __forceinline__ void load_rows(float *dst, const T *src, int rows, int D, bool vec,
                                          Off off) {
    if (std::is_same_v<T, float> && vec) {
        constexpr int CH = DP / 4;
        for (int i = threadIdx.x; i < rows * CH; i += kThreads) {
            const int r = i / CH, d = (i % CH) * 4;
            const long at = off(r);
            const bool read = at >= 0 && d < D;
            copy16(dst + r * LD + d, src + (read ? at + d : 0), read);
        }
    } else if (vec) {
        constexpr int V = Vec16<T>::N, CH = DP / V;
        for (int i = threadIdx.x; i < rows * CH; i += kThreads) {
            const int r = i / CH, d = (i % CH) * V;
            const long at = off(r);
            Vec16<T> x;
            x.u = make_uint4(0, 0, 0, 0);
            if (at >= 0 && d < D) x.u = __ldg(reinterpret_cast<const uint4 *>(src + at + d));
#pragma unroll
            for (int j = 0; j < V; ++j) dst[r * LD + d + j] = to_f32(x.v[j]);
        }
    } else {
        for (int i = threadIdx.x; i < rows * DP; i += kThreads) {
            const int r = i / DP, d = i % DP;
            const long at = off(r);
            dst[r * LD + d] = at >= 0 && d < D ? to_f32(src[at + d]) : 0.f;
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the newest `N` load_rows() of this thread have landed.
template <int N>
__device__ __forceinline__ void copies_landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int DP, int MT>
__global__ void __launch_bounds__(kThreads) attn_f32_kernel(const Attn a, int splits, bool vec) {
    using C = F32<DP, MT>;
    constexpr int ROWS = C::ROWS, WK = C::WK, KW = C::KW, LD = C::LD, LDV = C::LDV;
    extern __shared__ __align__(16) float smem[];
    __shared__ float s_ml[8][2][16];
    __shared__ int s_bad;
    float *sq = smem, *sk = sq + ROWS * LD, *sv = sk + kKeys * LD;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int mt = warp / WK, wk = warp % WK;
    const int G = a.H / a.HKV, D = a.D, kvh = blockIdx.y;
    pdl_wait_primary();

    int b, tile;
    if (!attn_find_tile(a, G, ROWS, blockIdx.x, b, tile)) return;
    int start, len, kv;
    attn_seq(a, b, start, len, kv);
    tile = (len * G + ROWS - 1) / ROWS - 1 - tile;  // the tiles with the most keys first
    const int r0 = tile * ROWS, rows = min(ROWS, len * G - r0);
    const int shift = kv - len;  // query i sees keys [0, shift + i]
    const int most = min(kv, shift + (r0 + rows - 1) / G + 1);  // keys the tile sees
    const int least = shift + r0 / G + 1;                        // keys every row sees

    // this split's key tiles
    const int tiles = most > 0 ? (most + kKeys - 1) / kKeys : 0;
    const int per = (tiles + splits - 1) / splits;
    const int k0 = blockIdx.z * per, k1 = min(tiles, k0 + per);

    if (threadIdx.x == 0) s_bad = 0;
    load_rows<T, DP, LD>(sq, static_cast<const T *>(a.q), ROWS, D, vec, [&](int r) -> long {
        if (r >= rows) return -1;
        return (long)(start + (r0 + r) / G) * a.qs + (long)(kvh * G + (r0 + r) % G) * D;
    });
    auto load_keys = [&](auto ld, float *dst, const void *src, int kt, long stride) {
        load_rows<T, DP, decltype(ld)::value>(dst, static_cast<const T *>(src), kKeys, D, vec, [&](int r) -> long {
            const int j = kt * kKeys + r;
            const long at = kt < k1 && j < most ? attn_key_row(a, b, start, j, stride) : -1;
            return at < 0 ? -1 : at + (long)kvh * D;
        });
    };
    constexpr std::integral_constant<int, LD> kLd{};
    constexpr std::integral_constant<int, LDV> kLdv{};

    float o[DP / 8][4], m[2], l[2];
    int seen[2];  // keys that rows g and g + 8 see
#pragma unroll
    for (int z = 0; z < 2; ++z) seen[z] = min(kv, shift + (r0 + mt * 16 + g + 8 * z) / G + 1);
    const float c = a.scale * kLog2e;

    // The keys' way past the rows.  Where it leaves an output that is not finite it is taken again, and then
    // looks at all values: the non-finite ones become 0, the others are halved, so that none rounds up to inf.
    auto pass = [&](auto looks) {
        constexpr bool careful = decltype(looks)::value;
        load_keys(kLd, sk, a.k, k0, a.ks);
        load_keys(kLdv, sv, a.v, k0, a.vs);
        m[0] = m[1] = -INFINITY, l[0] = l[1] = 0.f;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        // The next tile's keys are on their way under the values' product, its values under the scores.
        for (int kt = k0; kt < k1; ++kt) {
            const int j0 = kt * kKeys;
            copies_landed<1>();
            __syncthreads();
            const bool edge = j0 + kKeys > least;  // some row does not see the whole tile
            // ---- scores of 16 rows and KW keys
            float s[KW / 8][4], small[KW / 8][4];
#pragma unroll
            for (int n = 0; n < KW / 8; ++n)
#pragma unroll
                for (int z = 0; z < 4; ++z) s[n][z] = small[n][z] = 0.f;
#pragma unroll 2
            for (int ks = 0; ks < DP; ks += 8) {
                const float2 q0 = *reinterpret_cast<const float2 *>(sq + (mt * 16 + g) * LD + ks + 2 * t4);
                const float2 q1 = *reinterpret_cast<const float2 *>(sq + (mt * 16 + g + 8) * LD + ks + 2 * t4);
                uint32_t qh[4], ql[4];
                split(q0.x, qh[0], ql[0]), split(q1.x, qh[1], ql[1]);
                split(q0.y, qh[2], ql[2]), split(q1.y, qh[3], ql[3]);
#pragma unroll
                for (int n = 0; n < KW / 8; ++n) {
                    const float2 kk = *reinterpret_cast<const float2 *>(sk + (wk * KW + n * 8 + g) * LD + ks + 2 * t4);
                    uint32_t h0, l0, h1, l1;
                    split(kk.x, h0, l0), split(kk.y, h1, l1);
                    mma1688(small[n], ql, h0, h1);
                    mma1688(small[n], qh, l0, l1);
                    mma1688(s[n], qh, h0, h1);
                }
            }
            bool odd = false;
#pragma unroll
            for (int n = 0; n < KW / 8; ++n)
#pragma unroll
                for (int z = 0; z < 4; ++z) s[n][z] += small[n][z], odd |= s[n][z] != s[n][z];
            if (__any_sync(0xffffffffu, odd)) {
                // inf has no split: take the scores of this warp as plain sums
#pragma unroll
                for (int n = 0; n < KW / 8; ++n)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const float *qr = sq + (mt * 16 + g + 8 * (z >> 1)) * LD, *kr = sk + (wk * KW + n * 8 + 2 * t4 + (z & 1)) * LD;
                        float x = 0.f;
#pragma unroll 1
                        for (int d = 0; d < D; ++d) x = fmaf(qr[d], kr[d], x);
                        s[n][z] = x;
                    }
            }
            __syncthreads();
            load_keys(kLd, sk, a.k, kt + 1, a.ks);
            // ---- running softmax of rows g and g + 8
            float mx[2] = {m[0], m[1]};
#pragma unroll
            for (int n = 0; n < KW / 8; ++n)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    s[n][z] *= c;
                    if (edge && j0 + wk * KW + n * 8 + 2 * t4 + (z & 1) >= seen[z >> 1]) s[n][z] = -INFINITY;
                    mx[z >> 1] = fmaxf(mx[z >> 1], s[n][z]);
                }
            float ref[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                mx[z] = fmaxf(mx[z], __shfl_xor_sync(0xffffffffu, mx[z], 1));
                mx[z] = fmaxf(mx[z], __shfl_xor_sync(0xffffffffu, mx[z], 2));
                ref[z] = mx[z] == -INFINITY ? 0.f : mx[z];  // (a row that has seen nothing yet)
            }
            if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
                const float f0 = exp2_fast(m[0] - ref[0]), f1 = exp2_fast(m[1] - ref[1]);
                l[0] *= f0, l[1] *= f1;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) o[i][0] *= f0, o[i][1] *= f0, o[i][2] *= f1, o[i][3] *= f1;
                m[0] = mx[0], m[1] = mx[1];
            }
            // probabilities as operand fragments: k index t is key 2 t, t + 4 is key 2 t + 1
            uint32_t ph[KW / 8][4], pl[KW / 8][4];
#pragma unroll
            for (int n = 0; n < KW / 8; ++n) {
                float e[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) e[z] = exp2_fast(s[n][z] - ref[z >> 1]), l[z >> 1] += e[z];
                split(e[0], ph[n][0], pl[n][0]), split(e[2], ph[n][1], pl[n][1]);
                split(e[1], ph[n][2], pl[n][2]), split(e[3], ph[n][3], pl[n][3]);
            }
            copies_landed<1>();
            __syncthreads();
            if (edge || careful) {
                // values that some row must not see: non-finite ones become 0 and join their rows at the end
                for (int i = threadIdx.x; i < kKeys * DP; i += kThreads) {
                    float &v = sv[(i / DP) * LDV + i % DP];
                    if (!isfinite(v)) v = 0.f, s_bad = 1;
                    else if (careful) v *= 0.5f;
                }
                __syncthreads();
            }
            // ---- o += P V, two blocks of eight channels at a time
#pragma unroll
            for (int i = 0; i < DP / 8; i += 2) {
                float big[2][4] = {}, rest[2][4] = {};
#pragma unroll
                for (int n = 0; n < KW / 8; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float *v = sv + (wk * KW + n * 8 + 2 * t4) * LDV + (i + y) * 8 + g;
                        uint32_t h0, l0, h1, l1;
                        split(v[0], h0, l0), split(v[LDV], h1, l1);
                        mma1688(rest[y], pl[n], h0, h1);
                        mma1688(rest[y], ph[n], l0, l1);
                        mma1688(big[y], ph[n], h0, h1);
                    }
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int z = 0; z < 4; ++z) o[i + y][z] += big[y][z] + rest[y][z];
            }
            __syncthreads();
            load_keys(kLdv, sv, a.v, kt + 1, a.vs);
        }
        copies_landed<0>();
    };
    pass(std::false_type{});
    float finite = 0.f;  // NaN when an output is not
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
        for (int z = 0; z < 4; ++z) finite = fmaf(o[i][z], 0.f, finite);
    const bool careful = __syncthreads_or(finite != 0.f);
    if (careful) pass(std::true_type{});
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        l[z] += __shfl_xor_sync(0xffffffffu, l[z], 1);
        l[z] += __shfl_xor_sync(0xffffffffu, l[z], 2);
    }
    if constexpr (WK > 1) {  // warps that share rows join, in turn
        if (t4 == 0)
#pragma unroll
            for (int z = 0; z < 2; ++z) s_ml[warp][0][g + 8 * z] = m[z], s_ml[warp][1][g + 8 * z] = l[z];
        __syncthreads();
        float f[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < WK; ++w) M = fmaxf(M, s_ml[mt * WK + w][0][g + 8 * z]);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < WK; ++w) L += s_ml[mt * WK + w][1][g + 8 * z] * exp2_fast(s_ml[mt * WK + w][0][g + 8 * z] - ref);
            f[z] = exp2_fast(m[z] - ref);
            m[z] = M, l[z] = L;
        }
#pragma unroll 1
        for (int w = 0; w < WK; ++w) {
            if (wk == w)
#pragma unroll
                for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        float2 *at = reinterpret_cast<float2 *>(sk + (mt * 16 + g + 8 * z) * DP + i * 8 + 2 * t4);
                        float2 x = make_float2(o[i][2 * z] * f[z], o[i][2 * z + 1] * f[z]);
                        if (w > 0) x.x += at->x, x.y += at->y;
                        o[i][2 * z] = x.x, o[i][2 * z + 1] = x.y;
                        *at = x;
                    }
            __syncthreads();
        }
        if (wk != WK - 1 && !careful) return;
    }
    if (careful) {
        // the values that were taken out, to the rows that see them
        for (int kt = k0; kt < k1; ++kt) {
            __syncthreads();
            load_keys(kLdv, sv, a.v, kt, a.vs);
            copies_landed<0>();
            __syncthreads();
            bool odd = false;
            for (int i = threadIdx.x; i < kKeys * DP; i += kThreads) odd |= !isfinite(sv[(i / DP) * LDV + i % DP]);
            if (!__syncthreads_or(odd)) continue;
#pragma unroll 1
            for (int j = 0; j < kKeys; ++j)
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    if (kt * kKeys + j < seen[z])
#pragma unroll
                        for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float v = sv[j * LDV + i * 8 + 2 * t4 + y];
                                if (!isfinite(v)) o[i][2 * z + y] += v;
                            }
        }
        if (wk != WK - 1) return;
    }
    const float unit = careful ? 2.f : 1.f;  // of o
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        const int r = mt * 16 + g + 8 * z;
        if (r >= rows) continue;
        if (s_bad && !careful)
            for (int j = max(0, min(least, k1 * kKeys) / kKeys) * kKeys; j < min(seen[z], k1 * kKeys); ++j) {
                const long at = j >= k0 * kKeys ? attn_key_row(a, b, start, j, a.vs) : -1;
                if (at < 0) continue;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int d = i * 8 + 2 * t4 + y;
                        const float v = d < D ? to_f32(static_cast<const T *>(a.v)[at + (long)kvh * D + d]) : 0.f;
                        if (!isfinite(v)) o[i][2 * z + y] += v;
                    }
            }
        const size_t row = (size_t)(start + (r0 + r) / G) * a.H + kvh * G + (r0 + r) % G;
        const float inv = l[z] > 0.f ? 1.f / l[z] : l[z];  // (0 gives 0, NaN stays)
        if (splits == 1) {
            T *out = static_cast<T *>(a.out) + row * D;
#pragma unroll
            for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    if (i * 8 + 2 * t4 + y < D) out[i * 8 + 2 * t4 + y] = from_f32<T>(l[z] != 0.f ? o[i][2 * z + y] * inv * unit : 0.f);
        } else {
            const Part part(a, splits, row, blockIdx.z);
            if (t4 == 0) part.ml[0] = m[z], part.ml[1] = l[z];
#pragma unroll
            for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    if (i * 8 + 2 * t4 + y < D) part.o[i * 8 + 2 * t4 + y] = o[i][2 * z + y] * unit;
        }
    }
}

// Joins the splits of each row: one warp a (token, head).  Sequences of at most min_rows (query, head
// of a group) rows have none.
template <typename T>
__global__ void __launch_bounds__(128) attn_join_kernel(const Attn a, int splits, int min_rows) {
    const int lane = threadIdx.x & 31, D = a.D;
    const long row = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait_primary();
    if (row >= (long)a.N * a.H) return;
    // The row's sequence.  Each sequence is judged by itself, as where the parts were left: past a malformed
    // one the offsets may go down, and the binary search then misses sound ones.
    const int t = (int)(row / a.H);
    int start, len, kv;
    auto holds = [&](int b) { return attn_seq(a, b, start, len, kv) && t >= start && t < start + len; };
    if (!holds(seq_of_token(a.offsets, a.B, t))) {
        int b0 = 0;
        unsigned found = 0;
        for (; found == 0 && b0 < a.B; b0 += 32) found = __ballot_sync(0xffffffffu, b0 + lane < a.B && holds(b0 + lane));
        if (found == 0) return;
        holds(b0 - 32 + __ffs(found) - 1);
    }
    if ((long)len * (a.H / a.HKV) <= min_rows) return;
    const Part first(a, splits, row, 0);
    float m = -INFINITY, l = 0.f;
    for (int s = lane; s < splits; s += 32) m = fmaxf(m, first.ml[2 * s]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float ref = m == -INFINITY ? 0.f : m;
    for (int s = lane; s < splits; s += 32) l += first.ml[2 * s + 1] * exp2_fast(first.ml[2 * s] - ref);
    l = group_sum<32>(l);
    const float inv = l > 0.f ? 1.f / l : l;  // (0 gives 0, NaN stays)
    const float scale = a.out_scale ? __ldg(a.out_scale + row % a.H / (a.H / a.HKV)) : 1.f;
    T *out = static_cast<T *>(a.out) + row * D;
    for (int d = lane; d < D; d += 32) {
        float o = 0.f;
#pragma unroll 8
        for (int s = 0; s < splits; ++s) {
            const float c = exp2_fast(first.ml[2 * s] - ref), v = first.o[(size_t)s * D + d];
            o += c > 0.f ? v * c : 0.f;  // (a split that counts for nothing may hold inf)
        }
        out[d] = from_f32<T>(l != 0.f ? o * inv * scale : 0.f);
    }
}

template <typename T, int DP, int MT>
cudaError_t launch_tile(const Attn &a, bool vec, cudaStream_t s) {
    using C = F32<DP, MT>;
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(attn_f32_kernel<T, DP, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    });
    if (e != cudaSuccess) return e;
    const int G = a.H / a.HKV;
    const long tiles = (long)a.N * G / C::ROWS + a.B;
    if (tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
    // Splits until every SM has tiles to choose from (histories differ), but not below four key tiles.
    int splits = 1;
    if (a.part != nullptr)
        while (splits < kMaxSplits && tiles * a.HKV * splits < 4 * 152 &&
               (long)a.max_pages * a.page_size >= 8L * splits * kKeys &&
               (size_t)a.N * a.H * (splits * 2) * (a.D + 2) <= a.part_floats)
            splits *= 2;
    e = launch_kernel(attn_f32_kernel<T, DP, MT>, dim3((unsigned)tiles, a.HKV, splits), dim3(kThreads), C::SMEM, s, true,
                      a, splits, vec);
    note_launch();
    if (e != cudaSuccess || splits == 1) return e;
    return launch_attention_join(a, splits, 0, std::is_same_v<T, float> ? GDN_F32 : GDN_BF16, s);
}

template <typename T>
cudaError_t launch_typed(const Attn &a, cudaStream_t s) {
    const bool vec = rows_aligned(a.q, a.qs, a.D, sizeof(T)) && rows_aligned(a.k, a.ks, a.D, sizeof(T)) &&
                     rows_aligned(a.v, a.vs, a.D, sizeof(T));
    // Rows a tile: sequences of few rows leave most of a wide tile's work unused, long ones load less
    // for each product with it.
    const long G = a.H / a.HKV;
    const long rows = a.block_table != nullptr && a.max_q * G <= 16 ? a.max_q * G : (long)a.N * G / a.B;
    if (a.D <= 64)
        return rows <= 16 ? launch_tile<T, 64, 1>(a, vec, s) : rows <= 64 ? launch_tile<T, 64, 4>(a, vec, s)
                                                                         : launch_tile<T, 64, 8>(a, vec, s);
    if (a.D <= 128)
        return rows <= 16 ? launch_tile<T, 128, 1>(a, vec, s) : rows <= 64 ? launch_tile<T, 128, 4>(a, vec, s)
                                                                          : launch_tile<T, 128, 8>(a, vec, s);
    return rows <= 16 ? launch_tile<T, 256, 1>(a, vec, s) : launch_tile<T, 256, 4>(a, vec, s);
}

}  // namespace

size_t attention_f32_part_floats(int N, int H, int D) {
    // Splits are chosen while tiles * HKV * splits < 4 * 152 tiles of at most 128 rows; doubled once more.
    const size_t rows = (size_t)N * H, most = rows * kMaxSplits, cap = 2 * 4 * 152 * 128;
    return (most < cap ? most : cap) * (D + 2);
}

cudaError_t launch_attention_join(const Attn &a, int splits, int min_rows, int dtype, cudaStream_t s) {
    const dim3 ctas((unsigned)(((long)a.N * a.H + 3) / 4));
    const cudaError_t e =
        dtype == GDN_BF16
            ? launch_kernel(attn_join_kernel<__nv_bfloat16>, ctas, dim3(128), 0, s, true, a, splits, min_rows)
            : launch_kernel(attn_join_kernel<float>, ctas, dim3(128), 0, s, true, a, splits, min_rows);
    note_launch();
    return e;
}

cudaError_t launch_attention_f32(const Attn &a, int dtype, cudaStream_t s) {
    return dtype == GDN_BF16 ? launch_typed<__nv_bfloat16>(a, s) : launch_typed<float>(a, s);
}

}  // namespace gdn
