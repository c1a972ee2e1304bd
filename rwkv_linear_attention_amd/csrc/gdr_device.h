// gdr_device.h -- device helpers shared by the gated delta rule kernels (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wkv7_device.h"

namespace gdr {

using wkv7::bf16x8;
using wkv7::f32x4;
using wkv7::f32_to_bf16_bits;
using wkv7::load_elem;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// n consecutive elements (n a multiple of 4, the first 8- or 16-byte aligned), widened.
template <int N>
__device__ __forceinline__ void load_row(const float *p, float (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const f32x4 u = *reinterpret_cast<const f32x4 *>(p + i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[i + e] = u[e];
    }
}
template <int N>
__device__ __forceinline__ void load_row(const uint16_t *p, float (&x)[N])
{
    if constexpr (N % 8 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const u32x4 u = *reinterpret_cast<const u32x4 *>(p + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[i + 2 * e] = bf16_lo(u[e]);
                x[i + 2 * e + 1] = bf16_hi(u[e]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x2 u = *reinterpret_cast<const u32x2 *>(p + i);
            x[i] = bf16_lo(u[0]);
            x[i + 1] = bf16_hi(u[0]);
            x[i + 2] = bf16_lo(u[1]);
            x[i + 3] = bf16_hi(u[1]);
        }
    }
}

// Four consecutive outputs (fp32, or bf16 rounded to nearest even).
__device__ __forceinline__ void store4(float *p, const f32x4 x) { *reinterpret_cast<f32x4 *>(p) = x; }
__device__ __forceinline__ void store4(uint16_t *p, const f32x4 x)
{
    const uint32_t lo = f32_to_bf16_bits(x[0]) | (static_cast<uint32_t>(f32_to_bf16_bits(x[1])) << 16);
    const uint32_t hi = f32_to_bf16_bits(x[2]) | (static_cast<uint32_t>(f32_to_bf16_bits(x[3])) << 16);
    *reinterpret_cast<u32x2 *>(p) = u32x2{lo, hi};
}

// `rows` rows of a tensor as a buffer: offsets from the first element are 32-bit, a load behind
// the last row gives 0 and a store there does nothing, so the last rows of a sequence take no
// path of their own.
typedef __amdgpu_buffer_rsrc_t Buffer;
template <typename T>
__device__ __forceinline__ Buffer rows_buffer(T *p, int rows, size_t stride)
{
    const unsigned bytes = static_cast<unsigned>(rows) * static_cast<unsigned>(stride * sizeof(T));
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(static_cast<const void *>(p)), static_cast<short>(0),
                                             static_cast<int>(bytes), 0x00027000);
}
__device__ __forceinline__ u32x4 fetch4(Buffer b, unsigned at)
{
    return __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0);
}

// Workgroup index to work item: consecutive workgroups go round the 8 XCDs, so each XCD
// gets one contiguous run of items, and items that share inputs meet in its L2.
__device__ __forceinline__ unsigned xcd_item(unsigned bid, unsigned n)
{
    const unsigned x = bid & 7, per = n >> 3, rest = n & 7;
    return x * per + (x < rest ? x : rest) + (bid >> 3);
}

}  // namespace gdr
