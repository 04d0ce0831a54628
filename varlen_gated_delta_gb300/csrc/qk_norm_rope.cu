// qk_norm_rope.cu - gdn_qk_norm_rope: per-head RMS norm of q and k, position
// rotation, and the write of k and v into the paged cache, in one pass.
//
// Per head x of D channels: y = x w / sqrt(mean(x^2) + eps), then (a, b) -> (a c
// - b s, b c + a s) for each rotated pair.  Some ten operations for every value
// read and written: bound by HBM at 2 N (H + 2 HKV) D values.
//
// Vector kernel: a head takes D / VEC neighbouring lanes of 16 bytes each, so a
// warp holds one or several heads; it stays with one token and walks its heads.
// A lane's channels are then the same in every step: its weights, cosines and
// sines are loaded once and stay in registers, and the rows stream through
// with UNROLL loads in flight.  The partner of a channel in the half style sits
// in the lane R / 2 channels away, at a fixed xor distance when R is a power of
// two.  All arithmetic is fp32 with one rounding at the store.
#include "common.cuh"
#include "serving.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;

// One lane's channels d0 .. d0 + VEC of a head (LPH lanes to a head).
template <typename T, int LPH, int UNROLL>
__global__ void __launch_bounds__(kThreads) norm_rope_vec_kernel(const NormRope p, int splits) {
    constexpr int VEC = Vec16<T>::N, HPW = 32 / LPH, D = LPH * VEC;
    const int lane = threadIdx.x & 31;
    const long wid = (long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(wid / splits), part = (int)(wid % splits);
    if (t >= p.N) return;
    const int d0 = (lane % LPH) * VEC, R = p.R, half = R >> 1;
    const bool halves = p.style == GDN_ROPE_HALF;
    pdl_wait_primary();

    float cs[VEC], sn[VEC];  // the rotation y = x cs + partner sn (sn holds the sign)
#pragma unroll
    for (int i = 0; i < VEC; ++i) cs[i] = 1.f, sn[i] = 0.f;
    if (R > 0) {
        const int pos = __ldg(p.positions + t);
        if (pos < 0 || pos >= p.max_pos) return;
        const float *row = p.cos_sin + (size_t)pos * R;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int d = d0 + i;
            if (d >= R) continue;
            const int j = halves ? (d < half ? d : d - half) : d >> 1;
            const bool first = halves ? d < half : (d & 1) == 0;
            cs[i] = __ldg(row + j);
            sn[i] = first ? -__ldg(row + half + j) : __ldg(row + half + j);
        }
    }
    const int slot = p.slots ? __ldg(p.slots + t) : -1;
    const bool cached = slot >= 0 && slot < p.num_slots;
    const T *x = static_cast<const T *>(p.qkv) + (size_t)t * p.row_stride;
    T *q = static_cast<T *>(p.q) + (size_t)t * p.H * D;
    T *k = p.k ? static_cast<T *>(p.k) + (size_t)t * p.HKV * D : nullptr;
    T *kc = cached ? static_cast<T *>(p.k_cache) + (size_t)slot * p.HKV * D : nullptr;
    T *vc = cached ? static_cast<T *>(p.v_cache) + (size_t)slot * p.HKV * D : nullptr;
    // the warps of a token share its heads: groups of HPW heads, splits apart
    const int heads = p.H + p.HKV + (cached ? p.HKV : 0);
    const int lane_head = lane / LPH;

    for (int g0 = part * HPW; g0 < heads; g0 += splits * HPW * UNROLL) {
        Vec16<T> in[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int h = g0 + u * splits * HPW + lane_head;
            if (h < heads) in[u].u = __ldcs(reinterpret_cast<const uint4 *>(x + (size_t)h * D + d0));
            else in[u].u = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int h = g0 + u * splits * HPW + lane_head;
            const bool is_q = h < p.H, is_k = !is_q && h < p.H + p.HKV;
            const float *w = is_q ? p.qw : p.kw;
            float f[VEC], ss = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = to_f32(in[u].v[i]), ss += f[i] * f[i];
            ss = group_sum<LPH>(ss);  // (all lanes take part, whatever their head is)
            if (w != nullptr) {
                const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                for (int i = 0; i < VEC; i += 4) {
                    const float4 ww = __ldg(reinterpret_cast<const float4 *>(w + d0 + i));
                    f[i] *= r * ww.x, f[i + 1] *= r * ww.y, f[i + 2] *= r * ww.z, f[i + 3] *= r * ww.w;
                }
            }
            Vec16<T> o;
            if (halves) {
                const int apart = half / VEC;  // lanes (0: no rotation)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float other = __shfl_xor_sync(0xffffffffu, f[i], apart);
                    o.v[i] = from_f32<T>(d0 < R ? f[i] * cs[i] + other * sn[i] : f[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    o.v[i] = from_f32<T>(d0 + i < R ? f[i] * cs[i] + f[i ^ 1] * sn[i] : f[i]);
            }
            if (is_q) {
                *reinterpret_cast<uint4 *>(q + (size_t)h * D + d0) = o.u;
            } else if (is_k) {
                const size_t at = (size_t)(h - p.H) * D + d0;
                if (k) *reinterpret_cast<uint4 *>(k + at) = o.u;
                if (kc) *reinterpret_cast<uint4 *>(kc + at) = o.u;
            } else if (h < heads) {
                *reinterpret_cast<uint4 *>(vc + (size_t)(h - p.H - p.HKV) * D + d0) = in[u].u;
            }
        }
    }
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
    constexpr int kUnroll = 4, kGroup = 32 / LPH * kUnroll;
    // one warp a token when tokens abound; for few, its heads go over more warps
    const int heads = p.H + 2 * p.HKV;
    int splits = 1;
    while (splits * kGroup < heads && (long)p.N * splits < 4 * 152 * 8) splits *= 2;
    const long warps = (long)p.N * splits, ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_kernel(norm_rope_vec_kernel<T, LPH, kUnroll>, dim3((unsigned)ctas),
                                        dim3(kThreads), 0, s, false, p, splits);
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
                         at16(p.qw) && at16(p.kw);
    // the half style reaches a partner lane by xor: R a power of two of whole lanes
    const bool reach = p.style == GDN_ROPE_PAIRS || p.R == 0 ||
                       (p.R % (2 * VEC) == 0 && (half_lanes & (half_lanes - 1)) == 0);
    if (aligned && reach) {
        if (lph == 8) return launch_vec<T, 8>(p, s);
        if (lph == 16) return launch_vec<T, 16>(p, s);
        if (lph == 32) return launch_vec<T, 32>(p, s);
    }
    const long warps = (long)p.N * (p.H + 2 * p.HKV), ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_kernel(norm_rope_any_kernel<T>, dim3((unsigned)ctas), dim3(kThreads), 0,
                                        s, false, p);
    note_launch();
    return e;
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRope &p, int dtype, cudaStream_t s) {
    return dtype == GDN_BF16 ? launch_typed<__nv_bfloat16>(p, s) : launch_typed<float>(p, s);
}

}  // namespace gdn
