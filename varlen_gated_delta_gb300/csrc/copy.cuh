// copy.cuh - block-wide copies within global memory.
#pragma once

#include <stdint.h>

namespace gdn {

template <typename T, int THREADS, int N>  // N accesses in flight
__device__ __forceinline__ void copy_as(unsigned char *dst, const unsigned char *src, long bytes) {
    const int n = (int)(bytes / (long)sizeof(T));
    for (int i0 = threadIdx.x; i0 < n; i0 += N * THREADS) {
        T x[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (i0 + k * THREADS < n) x[k] = reinterpret_cast<const T *>(src)[i0 + k * THREADS];
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (i0 + k * THREADS < n) reinterpret_cast<T *>(dst)[i0 + k * THREADS] = x[k];
    }
}

// `bytes` (less than 2^31) from src to dst, both on boundaries of `vec` bytes (16, 8, 4, 2 or 1), and a multiple of it.
template <int THREADS, int N>
__device__ __forceinline__ void copy_bytes(unsigned char *dst, const unsigned char *src, long bytes, int vec) {
    switch (vec) {
    case 16: copy_as<uint4, THREADS, N>(dst, src, bytes); break;
    case 8: copy_as<uint2, THREADS, N>(dst, src, bytes); break;
    case 4: copy_as<uint32_t, THREADS, N>(dst, src, bytes); break;
    case 2: copy_as<uint16_t, THREADS, N>(dst, src, bytes); break;
    default: copy_as<uint8_t, THREADS, N>(dst, src, bytes);
    }
}

// The widest such access for a base address and row size in bytes.
inline int copy_width(uintptr_t base, uintptr_t row) {
    const uintptr_t at = base | row;
    return at % 16 == 0 ? 16 : at % 8 == 0 ? 8 : at % 4 == 0 ? 4 : at % 2 == 0 ? 2 : 1;
}

}  // namespace gdn
