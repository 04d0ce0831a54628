// attention_simt.cu - softmax attention on the fp32 pipe: fp32 activations, and
// any head width and alignment the tensor-core kernels do not take.
//
// The query heads of one key-value head share its keys, so a tile holds ROWS
// (token, head) pairs of one key-value head, token-major: row r is token r / G,
// head r % G.  Keys go by in tiles of 64 with the running maximum m and sum l
// of the softmax, in base 2: with x = scale log2(e) q k,
//   m' = max(m, max x),  l' = l 2^(m - m') + sum 2^(x - m'),  o' likewise,
// and o / l at the end.  Everything is held in shared memory as fp32; 256
// threads form a 16 x 16 grid that computes the scores (ROWS/16 x 4 each) and
// the output (ROWS/16 x DP/16 each).  Bound by the fp32 pipe: 2 D
// multiply-adds for each (row, key); the 16-row variant wastes less of it on
// decode steps, whose rows are few.
// Over a paged cache the keys of a tile are split `splits` ways (grid z) when
// tiles are few; each split leaves m, l and an unscaled o for a second kernel.
#include "attention.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kKeys = 64;
constexpr int kMaxSplits = 32;

template <int DP, int RPT>
constexpr size_t smem_bytes() {
    return (size_t)(RPT * 16 * (DP + 4) + 2 * kKeys * (DP + 4) + RPT * 16 * (kKeys + 4)) * 4;
}

// 16 bytes to shared memory, or zeros
__device__ __forceinline__ void copy16(float *dst, const void *src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(read ? 16 : 0)
                 : "memory");
}

// `rows` rows of D values (row r at off(r), or zeros when off(r) < 0) into
// shared memory, DP + 4 floats apart, columns from D on zero; aligned fp32 rows by
// copies that are in flight until copies_landed().
template <typename T, int DP, typename Off>
__device__ __forceinline__ void load_rows(float *dst, const T *src, int rows, int D, bool vec,
                                          Off off) {
    if (std::is_same_v<T, float> && vec) {
        constexpr int CH = DP / 4;
        for (int i = threadIdx.x; i < rows * CH; i += kThreads) {
            const int r = i / CH, d = (i % CH) * 4;
            const long at = off(r);
            const bool read = at >= 0 && d < D;
            copy16(dst + r * (DP + 4) + d, src + (read ? at + d : 0), read);
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
            for (int j = 0; j < V; ++j) dst[r * (DP + 4) + d + j] = to_f32(x.v[j]);
        }
    } else {
        for (int i = threadIdx.x; i < rows * DP; i += kThreads) {
            const int r = i / DP, d = i % DP;
            const long at = off(r);
            dst[r * (DP + 4) + d] = at >= 0 && d < D ? to_f32(src[at + d]) : 0.f;
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the newest `N` load_rows() of this thread have landed.
template <int N>
__device__ __forceinline__ void copies_landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int DP, int RPT>
__global__ void __launch_bounds__(kThreads) attn_simt_kernel(const Attn a, int splits, bool vec) {
    constexpr int ROWS = 16 * RPT, LD = DP + 4, LP = kKeys + 4, OC = DP / 64;
    extern __shared__ __align__(16) float smem[];
    float *sq = smem, *sk = sq + ROWS * LD, *sv = sk + kKeys * LD, *sp = sv + kKeys * LD;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
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

    load_rows<T, DP>(sq, static_cast<const T *>(a.q), ROWS, D, vec, [&](int r) -> long {
        if (r >= rows) return -1;
        return (long)(start + (r0 + r) / G) * a.qs + (long)(kvh * G + (r0 + r) % G) * D;
    });
    float m[RPT], l[RPT];
    float2 o[RPT][OC][2];  // channels c 64 + tx 4 + {0, 1}, {2, 3}
    int last[RPT];  // keys this row sees
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
        last[i] = min(kv, shift + (r0 + ty * RPT + i) / G + 1);
#pragma unroll
        for (int c = 0; c < OC; ++c) o[i][c][0] = o[i][c][1] = make_float2(0.f, 0.f);
    }
    const float sl = a.scale * kLog2e;
    auto load_keys = [&](float *dst, const void *src, int kt, long stride) {
        load_rows<T, DP>(dst, static_cast<const T *>(src), kKeys, D, vec, [&](int r) -> long {
            const int j = kt * kKeys + r;
            const long at = kt < k1 && j < most ? attn_key_row(a, b, start, j, stride) : -1;
            return at < 0 ? -1 : at + (long)kvh * D;
        });
    };
    load_keys(sk, a.k, k0, a.ks);
    load_keys(sv, a.v, k0, a.vs);

    // The next tile's keys are on their way under the values' product, its values under the scores.
    for (int kt = k0; kt < k1; ++kt) {
        const int j0 = kt * kKeys;
        copies_landed<1>();
        __syncthreads();
        // scores of rows ty RPT + i, keys tx + 16 j: even and odd channels apart on the packed
        // fp32 pipe, and in runs of 32 channels, whose short sums round less than one long one
        float x[RPT][4];
#pragma unroll
        for (int i = 0; i < RPT; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll 1
        for (int e = 0; e < DP; e += 32) {
            float2 y[RPT][4];
#pragma unroll
            for (int i = 0; i < RPT; ++i) y[i][0] = y[i][1] = y[i][2] = y[i][3] = make_float2(0.f, 0.f);
#pragma unroll
            for (int d = e; d < e + 32; d += 4) {
                float4 kk[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * LD + d);
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float4 qq = *reinterpret_cast<const float4 *>(sq + (ty * RPT + i) * LD + d);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[i][j] = __ffma2_rn(make_float2(qq.x, qq.y), make_float2(kk[j].x, kk[j].y), y[i][j]);
                        y[i][j] = __ffma2_rn(make_float2(qq.z, qq.w), make_float2(kk[j].z, kk[j].w), y[i][j]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < RPT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] += y[i][j].x + y[i][j].y;
        }
        __syncthreads();
        load_keys(sk, a.k, kt + 1, a.ks);
        const bool edge = j0 + kKeys > least;  // some row does not see the whole tile
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] *= sl;
                if (edge && j0 + tx + 16 * j >= last[i]) x[i][j] = -INFINITY;
                mx = fmaxf(mx, x[i][j]);
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float ref = mx == -INFINITY ? 0.f : mx;  // a row that has seen nothing yet
            const float c = exp2_fast(m[i] - ref);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = exp2_fast(x[i][j] - ref);
                sum += e;
                // a masked key is marked, so that its value is left out and not multiplied by 0
                const bool off = edge && j0 + tx + 16 * j >= last[i];
                sp[(ty * RPT + i) * LP + tx + 16 * j] = off ? -1.f : e;
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            m[i] = mx;
            l[i] = l[i] * c + sum;
#pragma unroll
            for (int q = 0; q < OC; ++q)
#pragma unroll
                for (int z = 0; z < 2; ++z) o[i][q][z] = __fmul2_rn(o[i][q][z], make_float2(c, c));
        }
        copies_landed<1>();
        __syncthreads();
#pragma unroll 2
        for (int j = 0; j < kKeys; j += 4) {
            float pr[RPT][4];
#pragma unroll
            for (int i = 0; i < RPT; ++i)
                *reinterpret_cast<float4 *>(pr[i]) =
                    *reinterpret_cast<const float4 *>(sp + (ty * RPT + i) * LP + j);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                for (int c = 0; c < OC; ++c) {
                    const float4 v = *reinterpret_cast<const float4 *>(sv + (j + jj) * LD + c * 64 + tx * 4);
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        if (edge && pr[i][jj] < 0.f) continue;
                        const float2 pp = make_float2(pr[i][jj], pr[i][jj]);
                        o[i][c][0] = __ffma2_rn(pp, make_float2(v.x, v.y), o[i][c][0]);
                        o[i][c][1] = __ffma2_rn(pp, make_float2(v.z, v.w), o[i][c][1]);
                    }
                }
        }
        __syncthreads();
        load_keys(sv, a.v, kt + 1, a.vs);
    }
    copies_landed<0>();

#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = ty * RPT + i;
        if (r >= rows) continue;
        const size_t row = (size_t)(start + (r0 + r) / G) * a.H + kvh * G + (r0 + r) % G;
        if (splits == 1) {
            const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);  // (NaN stays)
            T *out = static_cast<T *>(a.out) + row * D;
#pragma unroll
            for (int c = 0; c < OC; ++c)
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (c * 64 + tx * 4 + z < D) out[c * 64 + tx * 4 + z] = from_f32<T>((z & 1 ? o[i][c][z >> 1].y : o[i][c][z >> 1].x) * inv);
        } else {
            float *part = a.part + (row * splits + blockIdx.z) * (D + 2);
            if (tx == 0) part[0] = m[i], part[1] = l[i];
#pragma unroll
            for (int c = 0; c < OC; ++c)
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (c * 64 + tx * 4 + z < D) part[2 + c * 64 + tx * 4 + z] = z & 1 ? o[i][c][z >> 1].y : o[i][c][z >> 1].x;
        }
    }
}

// Joins the splits of each row: one warp a (token, head).
template <typename T>
__global__ void __launch_bounds__(128) attn_simt_join_kernel(const Attn a, int splits) {
    const int lane = threadIdx.x & 31, D = a.D;
    const long row = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait_primary();
    if (row >= (long)a.N * a.H) return;
    const int t = (int)(row / a.H), total = __ldg(a.offsets + a.B);
    if (t >= total || total > a.N) return;
    int start, len, kv;
    const int b = seq_of_token(a.offsets, a.B, t);
    if (!attn_seq(a, b, start, len, kv) || t < start || t >= start + len) return;
    const float *part = a.part + row * splits * (D + 2);
    float m = -INFINITY, l = 0.f;
    for (int s = 0; s < splits; ++s) m = fmaxf(m, part[s * (D + 2)]);
    const float ref = m == -INFINITY ? 0.f : m;
    for (int s = 0; s < splits; ++s) l += part[s * (D + 2) + 1] * exp2_fast(part[s * (D + 2)] - ref);
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    T *out = static_cast<T *>(a.out) + row * D;
    for (int d = lane; d < D; d += 32) {
        float o = 0.f;
        for (int s = 0; s < splits; ++s) {
            const float c = exp2_fast(part[s * (D + 2)] - ref);
            o += c > 0.f ? part[s * (D + 2) + 2 + d] * c : 0.f;
        }
        out[d] = from_f32<T>(o * inv);
    }
}

template <typename T, int DP, int RPT>
cudaError_t launch_tile(const Attn &a, bool vec, cudaStream_t s) {
    constexpr int ROWS = 16 * RPT;
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(attn_simt_kernel<T, DP, RPT>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)smem_bytes<DP, RPT>());
    });
    if (e != cudaSuccess) return e;
    const int G = a.H / a.HKV;
    const long tiles = (long)a.N * G / ROWS + a.B;
    if (tiles > INT32_MAX || a.HKV > 65535) return cudaErrorInvalidConfiguration;
    int splits = 1;
    if (a.part != nullptr)
        while (splits < kMaxSplits && tiles * a.HKV * splits < 2 * 152 &&
               (size_t)a.N * a.H * (splits * 2) * (a.D + 2) <= a.part_floats)
            splits *= 2;
    e = launch_kernel(attn_simt_kernel<T, DP, RPT>, dim3((unsigned)tiles, a.HKV, splits),
                      dim3(kThreads), smem_bytes<DP, RPT>(), s, true, a, splits, vec);
    note_launch();
    if (e != cudaSuccess || splits == 1) return e;
    const long ctas = ((long)a.N * a.H + 3) / 4;
    e = launch_kernel(attn_simt_join_kernel<T>, dim3((unsigned)ctas), dim3(128), 0, s, true, a, splits);
    note_launch();
    return e;
}

template <typename T>
cudaError_t launch_typed(const Attn &a, cudaStream_t s) {
    const bool vec = rows_aligned(a.q, a.qs, a.D, sizeof(T)) && rows_aligned(a.k, a.ks, a.D, sizeof(T)) &&
                     rows_aligned(a.v, a.vs, a.D, sizeof(T));
    // Rows a tile: sequences of few rows would leave most of a wide tile's work unused, long ones
    // load less for each product with it (4 x 1000 tokens, 16 heads of 128 on 4: 806 us with 64 rows, 558 with 128).
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

size_t attention_simt_part_floats(int B, int N, int H, int HKV, int D) {
    // up to kMaxSplits partial rows while the split tiles are few
    const long rows = (long)N * H;
    const long cap = 2L * 152 * 64 * 2;  // rows of a split launch: below two waves of 64-row tiles, doubled
    const long n = rows * kMaxSplits < cap ? rows * kMaxSplits : cap;
    (void)B, (void)HKV;
    return (size_t)n * (D + 2);
}

cudaError_t launch_attention_simt(const Attn &a, int dtype, cudaStream_t s) {
    return dtype == GDN_BF16 ? launch_typed<__nv_bfloat16>(a, s) : launch_typed<float>(a, s);
}

}  // namespace gdn
