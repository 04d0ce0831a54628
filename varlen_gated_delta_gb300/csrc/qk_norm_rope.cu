// qk_norm_rope.cu - gdn_qk_norm_rope: per-head RMS norm of q and k, position
// rotation, and the write of k and v into the paged cache, in one pass.
//
// Per head x of D channels: y = x w / sqrt(mean(x^2) + eps), then (a, b) -> (a c
// - b s, b c + a s) for each rotated pair.  Some ten operations for every value
// read and written: bound by HBM at 2 N (H + 2 HKV) D values.
//
// Vector kernel: a head takes D / VEC neighbouring lanes of 16 bytes each, so a
// warp holds one or several heads; it stays with one token and walks its heads.
// A lane's channels are then the same in every step, and with rs = 1 / sqrt(mean
// + eps) an output is rs (x A + x' B) with A = w cos and B = +- w' sin, x' and w'
// the partner channel's: A and B are computed once and stay in registers.  In the
// half style x' sits in the lane R / 2 channels away, at a fixed xor distance when
// R is a power of two, and comes over in the packed type.  The rows stream
// through with UNROLL loads in flight (more of them cost more warps, by their
// registers, than they bring) behind a prefetch of the whole row to L2: 32768 bf16
// tokens, 32 + 8 + 8 heads of 128, into the cache, 137 us, 5.9 TB/s, 0.89 of the
// measured copy (149 us without the prefetch).  All arithmetic is fp32 with one
// rounding at the store.
#include "common.cuh"
#include "serving.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;

// N (a multiple of 2) floats from an address on a boundary of min(N, 4) of them.
template <int N>
__device__ __forceinline__ void load_floats(const float *src, float *dst) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(src + i));
            dst[i] = v.x, dst[i + 1] = v.y, dst[i + 2] = v.z, dst[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 v = __ldg(reinterpret_cast<const float2 *>(src + i));
            dst[i] = v.x, dst[i + 1] = v.y;
        }
    }
}

// The factors A and B of a lane's VEC channels from d0 on, for weight w (NULL: 1).
template <int VEC, bool HALVES>
__device__ __forceinline__ void factors(const float *w, const float *row, int d0, int R, float (&a)[VEC], float (&b)[VEC]) {
    const int half = R >> 1, e0 = d0 < half ? d0 + half : d0 - half;  // (halves: the partner channels)
    float other[VEC], c[VEC], sn[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) a[i] = other[i] = 1.f, b[i] = 0.f;
    if (w != nullptr) load_floats<VEC>(w + d0, a);
    if (d0 >= R) return;  // (R is a multiple of VEC)
    if constexpr (HALVES) {
        const int j0 = min(d0, e0);
        if (w != nullptr) load_floats<VEC>(w + e0, other);
        load_floats<VEC>(row + j0, c), load_floats<VEC>(row + half + j0, sn);
#pragma unroll
        for (int i = 0; i < VEC; ++i) b[i] = (d0 < half ? -sn[i] : sn[i]) * other[i], a[i] *= c[i];
    } else {
        load_floats<VEC / 2>(row + d0 / 2, c), load_floats<VEC / 2>(row + half + d0 / 2, sn);
#pragma unroll
        for (int i = 0; i < VEC; ++i) b[i] = (i & 1 ? sn[i / 2] : -sn[i / 2]) * a[i ^ 1];
#pragma unroll
        for (int i = 0; i < VEC; ++i) a[i] *= c[i / 2];
    }
}

// LPH lanes to a head, a lane's channels from (lane % LPH) VEC on.
template <typename T, int LPH, bool HALVES, int UNROLL>
__global__ void __launch_bounds__(kThreads, 8) norm_rope_vec_kernel(const NormRope p, int splits) {
    constexpr int VEC = Vec16<T>::N, HPW = 32 / LPH, D = LPH * VEC;
    const int lane = threadIdx.x & 31;
    const long wid = (long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(wid / splits), part = (int)(wid % splits);
    if (t >= p.N) return;
    const int d0 = (lane % LPH) * VEC, R = p.R;
    pdl_wait_primary();
    const int pos = R > 0 ? __ldg(p.positions + t) : 0;
    if (R > 0 && (pos < 0 || pos >= p.max_pos)) return;
    const float *row = p.cos_sin + (size_t)pos * R;
    const int slot = p.slots ? __ldg(p.slots + t) : -1;
    const bool cached = slot >= 0 && slot < p.num_slots;
    const T *x = static_cast<const T *>(p.qkv) + (size_t)t * p.row_stride + d0;
    // the rest of the row is on its way to L2 while its first heads are worked on
    if (splits == 1) {
        const char *from = reinterpret_cast<const char *>(static_cast<const T *>(p.qkv) + (size_t)t * p.row_stride);
        const int bytes = (p.H + p.HKV + (cached ? p.HKV : 0)) * D * (int)sizeof(T);
        for (int i = lane * 128; i < bytes; i += 32 * 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + i));
    }
    const bool turned = d0 < R;
    const int apart = HALVES ? (R >> 1) / VEC : 0;

    // heads [first, last) of the row, this warp's share, through put(head - first, raw, result)
    float a[VEC], b[VEC];
    auto walk = [&](int first, int last, bool norm, auto put) {
        for (int g0 = first + part * HPW + lane / LPH; g0 - lane / LPH < last; g0 += splits * HPW * UNROLL) {
            Vec16<T> in[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int h = g0 + u * splits * HPW;
                if (h < last) in[u].u = __ldcs(reinterpret_cast<const uint4 *>(x + (size_t)h * D));
                else in[u].u = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int h = g0 + u * splits * HPW;
                float f[VEC], ss = 0.f;
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] = to_f32(in[u].v[i]), ss += f[i] * f[i];
                ss = group_sum<LPH>(ss);  // (all lanes take part, whatever their head is)
                const float r = norm ? rsqrtf(ss * (1.f / D) + p.eps) : 1.f;
                Vec16<T> other = in[u], o;
                if (HALVES) {
                    other.u.x = __shfl_xor_sync(0xffffffffu, in[u].u.x, apart);
                    other.u.y = __shfl_xor_sync(0xffffffffu, in[u].u.y, apart);
                    other.u.z = __shfl_xor_sync(0xffffffffu, in[u].u.z, apart);
                    other.u.w = __shfl_xor_sync(0xffffffffu, in[u].u.w, apart);
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float y = f[i] * a[i];
                    if (turned) y = fmaf(to_f32(other.v[HALVES ? i : i ^ 1]), b[i], y);
                    o.v[i] = from_f32<T>(y * r);
                }
                if (h < last) put(h - first, in[u].u, o.u);
            }
        }
    };
    auto at = [&](void *base, size_t token, int heads, int h) {
        return reinterpret_cast<uint4 *>(static_cast<T *>(base) + (token * heads + h) * D + d0);
    };
    factors<VEC, HALVES>(p.qw, row, d0, R, a, b);
    walk(0, p.H, p.qw != nullptr, [&](int h, uint4, uint4 y) { *at(p.q, t, p.H, h) = y; });
    factors<VEC, HALVES>(p.kw, row, d0, R, a, b);
    walk(p.H, p.H + p.HKV, p.kw != nullptr, [&](int h, uint4, uint4 y) {
        if (p.k) *at(p.k, t, p.HKV, h) = y;
        if (cached) *at(p.k_cache, slot, p.HKV, h) = y;
    });
    if (cached)
        for (int h = part * HPW + lane / LPH; h < p.HKV; h += splits * HPW)
            *at(p.v_cache, slot, p.HKV, h) = __ldcs(reinterpret_cast<const uint4 *>(x + (size_t)(p.H + p.HKV + h) * D));
}

// Any width and alignment: one warp per (token, head), channels 32 lanes apart.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const NormRope p) {
    const int lane = threadIdx.x & 31, D = p.D, R = p.R, half = R >> 1;
    const long wid = (long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int heads = p.H + 2 * p.HKV;
    const int t = (int)(wid / heads), h = (int)(wid % heads);
    if (t >= p.N) return;
    pdl_wait_primary();
    const int pos = R > 0 ? __ldg(p.positions + t) : 0;
    if (R > 0 && (pos < 0 || pos >= p.max_pos)) return;
    const int slot = p.slots ? __ldg(p.slots + t) : -1;
    const bool cached = slot >= 0 && slot < p.num_slots;
    const T *x = static_cast<const T *>(p.qkv) + (size_t)t * p.row_stride + (size_t)h * D;
    if (h >= p.H + p.HKV) {
        if (!cached) return;
        T *vc = static_cast<T *>(p.v_cache) + ((size_t)slot * p.HKV + h - p.H - p.HKV) * D;
        for (int d = lane; d < D; d += 32) vc[d] = x[d];
        return;
    }
    const bool is_q = h < p.H;
    const float *w = is_q ? p.qw : p.kw;
    float r = 1.f;
    if (w != nullptr) {
        float ss = 0.f;
        for (int d = lane; d < D; d += 32) {
            const float f = to_f32(x[d]);
            ss += f * f;
        }
        r = rsqrtf(group_sum<32>(ss) / D + p.eps);
    }
    T *q = is_q ? static_cast<T *>(p.q) + ((size_t)t * p.H + h) * D : nullptr;
    T *k = !is_q && p.k ? static_cast<T *>(p.k) + ((size_t)t * p.HKV + h - p.H) * D : nullptr;
    T *kc = !is_q && cached ? static_cast<T *>(p.k_cache) + ((size_t)slot * p.HKV + h - p.H) * D : nullptr;
    const float *row = R > 0 ? p.cos_sin + (size_t)pos * R : nullptr;
    for (int d = lane; d < D; d += 32) {
        float y = to_f32(x[d]) * r * (w ? __ldg(w + d) : 1.f);
        if (d < R) {
            const bool halves = p.style == GDN_ROPE_HALF;
            const int j = halves ? (d < half ? d : d - half) : d >> 1;
            const bool first = halves ? d < half : (d & 1) == 0;
            const int e = halves ? (first ? d + half : d - half) : d ^ 1;
            const float other = to_f32(x[e]) * r * (w ? __ldg(w + e) : 1.f);
            const float s = __ldg(row + half + j);
            y = y * __ldg(row + j) + other * (first ? -s : s);
        }
        const T o = from_f32<T>(y);
        if (q) q[d] = o;
        if (k) k[d] = o;
        if (kc) kc[d] = o;
    }
}

template <typename T, int LPH>
cudaError_t launch_vec(const NormRope &p, cudaStream_t s) {
    // (16 channels a lane in flight: with 32, the registers of bf16 rows cost more warps than they bring)
    constexpr int kUnroll = 16 / Vec16<T>::N, kGroup = 32 / LPH * kUnroll;
    // one warp a token when tokens abound; for few, its heads go over more warps
    const int heads = p.H + 2 * p.HKV;
    int splits = 1;
    while (splits * kGroup < heads && (long)p.N * splits < 4 * 152 * 8) splits *= 2;
    const long warps = (long)p.N * splits, ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    const cudaError_t e =
        p.style == GDN_ROPE_HALF
            ? launch_kernel(norm_rope_vec_kernel<T, LPH, true, kUnroll>, dim3((unsigned)ctas), dim3(kThreads), 0, s, true, p, splits)
            : launch_kernel(norm_rope_vec_kernel<T, LPH, false, kUnroll>, dim3((unsigned)ctas), dim3(kThreads), 0, s, true, p, splits);
    note_launch();
    return e;
}

template <typename T>
cudaError_t launch_typed(const NormRope &p, cudaStream_t s) {
    constexpr int VEC = Vec16<T>::N;
    auto at16 = [](const void *x) { return ((uintptr_t)x & 15) == 0; };
    const int lph = p.D / VEC, half_lanes = p.R / 2 / VEC;
    const bool aligned = p.D % VEC == 0 && rows_aligned(p.qkv, p.row_stride, p.D, sizeof(T)) &&
                         at16(p.q) && at16(p.k) && at16(p.k_cache) && at16(p.v_cache) &&
                         at16(p.qw) && at16(p.kw) && at16(p.cos_sin);
    // whole lanes turn or do not; the half style reaches a partner lane by xor: R / 2 a power of two of them
    const bool reach = p.style == GDN_ROPE_PAIRS ? p.R % 8 == 0
                                                 : p.R % (2 * VEC) == 0 && (half_lanes & (half_lanes - 1)) == 0;
    if (aligned && reach) {
        if (lph == 8) return launch_vec<T, 8>(p, s);
        if (lph == 16) return launch_vec<T, 16>(p, s);
        if (lph == 32) return launch_vec<T, 32>(p, s);
    }
    const long warps = (long)p.N * (p.H + 2 * p.HKV), ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_kernel(norm_rope_any_kernel<T>, dim3((unsigned)ctas), dim3(kThreads), 0,
                                        s, true, p);
    note_launch();
    return e;
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRope &p, int dtype, cudaStream_t s) {
    return dtype == GDN_BF16 ? launch_typed<__nv_bfloat16>(p, s) : launch_typed<float>(p, s);
}

}  // namespace gdn
