// kv4_write.cu - gdn_kv4_write: keys and values into a paged cache of 4-bit values (kv4.cuh).
//
// Per 16 channels x of a head: s = e4m3(max |x| / (6 ts)), u = s ts, code = e2m1(x (1 / u)), all but the last step in fp32
// with one rounding each, so that the bytes do not depend on who computes them.  If asked for, the values held, u c, are
// written as rows of T too.
//
// Bound by HBM: each value read once (2 or 4 bytes), 9/16 byte written, and T again for the values.  A thread takes
// one group: 16 values are two or four 16-byte loads, its codes one 8-byte store.  A CTA takes neighbouring tokens of one
// head, so that its stores cover whole sectors where slots follow one another.  32768 tokens, 8 heads of 128, bf16, with the
// values: 54 us, 5.6 TB/s (0.83 of the measured copy; 67 us with four tokens to a head at a time); 64 tokens: 2.1 us.
#include "kv4.cuh"
#include "serving.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const Kv4Write p) {
    constexpr int VEC = 16 / sizeof(T);
    const int groups = p.D / 16, tid = threadIdx.x;
    pdl_wait_primary();
    const int in = tid / groups, g = tid - in * groups, kv = blockIdx.y & 1, h = blockIdx.y >> 1;
    const long token = (long)blockIdx.x * p.tokens + in;
    if (in >= p.tokens || token >= p.N) return;
    const int slot = __ldg(p.slots + token);
    const bool held = slot >= 0 && slot < (long)p.num_pages * p.page_size;
    T *out = static_cast<T *>(kv ? p.v_out : p.k_out);
    if (!held && out == nullptr) return;
    const T *src = static_cast<const T *>(kv ? p.v : p.k) + token * (kv ? p.v_stride : p.k_stride) + (long)h * p.D + g * 16;
    float x[16];
    if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < 16 / VEC; ++j) {
            Vec16<T> w;
            w.u = __ldg(reinterpret_cast<const uint4 *>(src) + j);
#pragma unroll
            for (int k = 0; k < VEC; ++k) x[j * VEC + k] = to_f32(w.v[k]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = to_f32(src[j]);
    }
    const float *scale = kv ? p.v_scale : p.k_scale;
    const float ts = scale ? __ldg(scale + h) : 1.f;
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(x[j]));  // (passes over NaN)
    float unit;
    const uint32_t byte = kv4_unit(amax, ts, unit);
    // (the reciprocal of a unit below 2^-128 leaves the range: both factors of the quotient are moved by a power of two, which
    // changes none of its bits otherwise)
    const float up = unit < 0x1p-64f ? 0x1p64f : 1.f, r = unit > 0.f ? __fdiv_rn(1.f, unit * up) : 0.f;
    uint32_t code[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = __fmul_rn(x[half * 8 + j] * up, r);
        code[half] = kv4_encode(t);
    }
    if (held) {
        const int page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size, at = slot - page * p.page_size;
        uint8_t *block = static_cast<uint8_t *>(kv ? p.v_cache : p.k_cache) +
                         ((long)page * p.HKV + h) * ((long)p.page_size * groups * 9);
        *reinterpret_cast<uint2 *>(block + ((long)at * groups + g) * 8) = make_uint2(code[0], code[1]);
        block[(long)p.page_size * groups * 8 + at * groups + g] = (uint8_t)byte;
    }
    if (out == nullptr) return;
    out += (token * p.HKV + h) * p.D + g * 16;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t d[4];
        kv4_codes(code[half], d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = f16x2_to_f32(d[j]);
            x[half * 8 + 2 * j] = f.x * unit, x[half * 8 + 2 * j + 1] = f.y * unit;
        }
    }
#pragma unroll
    for (int j = 0; j < 16 / VEC; ++j) {
        Vec16<T> w;
#pragma unroll
        for (int k = 0; k < VEC; ++k) w.v[k] = from_f32<T>(x[j * VEC + k]);
        reinterpret_cast<uint4 *>(out)[j] = w.u;
    }
}

template <typename T>
cudaError_t launch(const Kv4Write &p, cudaStream_t s) {
    Kv4Write w = p;
    w.tokens = kThreads / (p.D / 16);
    w.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (p.page_size == 1 << i) w.page_shift = i;
    const bool wide = rows_aligned(p.k, p.k_stride, p.D, sizeof(T)) && rows_aligned(p.v, p.v_stride, p.D, sizeof(T));
    const dim3 grid((unsigned)((p.N + w.tokens - 1) / w.tokens), (unsigned)(2 * p.HKV));
    const cudaError_t e = wide ? launch_kernel(kv4_write_kernel<T, true>, grid, dim3(kThreads), 0, s, true, w)
                               : launch_kernel(kv4_write_kernel<T, false>, grid, dim3(kThreads), 0, s, true, w);
    note_launch();
    return e;
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4Write &p, int dtype, cudaStream_t s) {
    return dtype == GDN_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}

}  // namespace gdn
