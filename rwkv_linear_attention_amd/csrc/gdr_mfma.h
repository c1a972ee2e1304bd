// gdr_mfma.h -- matrix-core helpers of the gated delta rule kernels (gfx950 only).
//
// All products run on v_mfma_f32_16x16x32_{f16,bf16} with fp32 accumulation.  An fp32 operand
// is split into pieces, x = x0 + x1 [+ x2], each the rounded remainder of the ones before, and
// the piece products are summed.  A piece rounds to half a step, 2^-8 (bf16) or 2^-11 (fp16)
// of it, so two fp16 pieces keep x to 2^-22 and three bf16 pieces to 2^-24, two to 2^-16.
// fp16 needs x near 1: its last piece reaches down to 2^-25 only and 65504 is the most, so
// those operands carry a power of two apart (a row's, or a state column's).  bf16 pieces
// need none.
#pragma once

#include "gdr_device.h"

namespace gdr {

// Two fp32 values to a packed pair of bf16 (round to nearest even), element 0 low.
__device__ __forceinline__ uint32_t pk_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Eight fp32 values to NP fragment planes of eight bf16 pieces.
template <int NP>
__device__ __forceinline__ void split8(const f32x4 a, const f32x4 b, s16x8 (&out)[NP])
{
    float r[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = pk_bf16(r[2 * e], r[2 * e + 1]);
        out[p] = __builtin_bit_cast(s16x8, u32x4{w[0], w[1], w[2], w[3]});
        if (p + 1 < NP) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                r[2 * e] -= bf16_lo(w[e]);
                r[2 * e + 1] -= bf16_hi(w[e]);
            }
        }
    }
}
template <int NP>
__device__ __forceinline__ void split4(const f32x4 a, u32x2 (&out)[NP])
{
    float r[4] = {a[0], a[1], a[2], a[3]};
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        out[p] = u32x2{pk_bf16(r[0], r[1]), pk_bf16(r[2], r[3])};
        if (p + 1 < NP) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                r[2 * e] -= bf16_lo(out[p][e]);
                r[2 * e + 1] -= bf16_hi(out[p][e]);
            }
        }
    }
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// -1 as a value the compiler does not see through: x - float(h) is then one v_fma_mix_f32
// on the packed half instead of a conversion and a subtraction.
__device__ __forceinline__ float minus_one()
{
    float m = -1.f;
    asm("" : "+s"(m));
    return m;
}

// Eight fp32 values to NP planes of eight fp16 pieces.
template <int NP>
__device__ __forceinline__ void split8h(const f32x4 a, const f32x4 b, s16x8 (&out)[NP], float m1)
{
    float r[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        f16x2 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = __builtin_convertvector(f32x2{r[2 * e], r[2 * e + 1]}, f16x2);
        out[p] = __builtin_bit_cast(s16x8, u32x4{__builtin_bit_cast(uint32_t, w[0]), __builtin_bit_cast(uint32_t, w[1]),
                                                 __builtin_bit_cast(uint32_t, w[2]), __builtin_bit_cast(uint32_t, w[3])});
        if (p + 1 < NP) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e] = fmaf(static_cast<float>(w[e / 2][e % 2]), m1, r[e]);
        }
    }
}

// As mma below, of fp16 pieces.
template <int NPA, int NPB>
__device__ __forceinline__ void mmah(f32x4 &acc, const s16x8 (&A)[NPA], const s16x8 (&B)[NPB])
{
    constexpr int NPM = NPA > NPB ? NPA : NPB;
#pragma unroll
    for (int s = NPM - 1; s >= 0; --s)
#pragma unroll
        for (int p = 0; p < NPA; ++p) {
            const int r = s - p;
            if (r >= 0 && r < NPB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, A[p]),
                                                             __builtin_bit_cast(f16x8, B[r]), acc, 0, 0, 0);
        }
}

// acc += sum over the pieces p + r < max(NPA, NPB) of A_p B_r, smallest first.
template <int NPA, int NPB>
__device__ __forceinline__ void mma(f32x4 &acc, const s16x8 (&A)[NPA], const s16x8 (&B)[NPB])
{
    constexpr int NPM = NPA > NPB ? NPA : NPB;
#pragma unroll
    for (int s = NPM - 1; s >= 0; --s)
#pragma unroll
        for (int p = 0; p < NPA; ++p) {
            const int r = s - p;
            if (r >= 0 && r < NPB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, A[p]),
                                                              __builtin_bit_cast(bf16x8, B[r]), acc, 0, 0, 0);
        }
}

__device__ __forceinline__ s16x8 lds8(const uint16_t *p) { return *reinterpret_cast<const s16x8 *>(p); }

// LDS transpose load of a 16x16 bf16 tile stored row-major as X[k][n]: lane 16 q + i passes
// the address of X[4 q + i/4][4 (i%4)] (four consecutive n), and lane (n = l%16, q = l/16)
// receives X[4 q + e][n], e = 0..3.  The four n-groups of a row may sit anywhere.
__device__ __forceinline__ s16x4 tr4(const uint16_t *p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
}
__device__ __forceinline__ s16x8 cat(const s16x4 a, const s16x4 b)
{
    return s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Two accumulators at once, with the same right operand: their chains of dependent products
// alternate.  TURN: the products transposed (the pieces change places; both operands have the
// same layout).
template <int NPA, int NPB, bool TURN = false>
__device__ __forceinline__ void mma2(f32x4 &acc0, f32x4 &acc1, const s16x8 (&A0)[NPA], const s16x8 (&A1)[NPA],
                                     const s16x8 (&B)[NPB])
{
    constexpr int NPM = NPA > NPB ? NPA : NPB;
#pragma unroll
    for (int s = NPM - 1; s >= 0; --s)
#pragma unroll
        for (int p = 0; p < NPA; ++p) {
            const int r = s - p;
            if (r >= 0 && r < NPB) {
                const bf16x8 b = __builtin_bit_cast(bf16x8, B[r]);
                const bf16x8 a0 = __builtin_bit_cast(bf16x8, A0[p]), a1 = __builtin_bit_cast(bf16x8, A1[p]);
                acc0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(TURN ? b : a0, TURN ? a0 : b, acc0, 0, 0, 0);
                acc1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(TURN ? b : a1, TURN ? a1 : b, acc1, 0, 0, 0);
            }
        }
}
template <int NPA, int NPB, bool TURN = false>
__device__ __forceinline__ void mmah2(f32x4 &acc0, f32x4 &acc1, const s16x8 (&A0)[NPA], const s16x8 (&A1)[NPA],
                                      const s16x8 (&B)[NPB])
{
    constexpr int NPM = NPA > NPB ? NPA : NPB;
#pragma unroll
    for (int s = NPM - 1; s >= 0; --s)
#pragma unroll
        for (int p = 0; p < NPA; ++p) {
            const int r = s - p;
            if (r >= 0 && r < NPB) {
                const f16x8 b = __builtin_bit_cast(f16x8, B[r]);
                const f16x8 a0 = __builtin_bit_cast(f16x8, A0[p]), a1 = __builtin_bit_cast(f16x8, A1[p]);
                acc0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(TURN ? b : a0, TURN ? a0 : b, acc0, 0, 0, 0);
                acc1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(TURN ? b : a1, TURN ? a1 : b, acc1, 0, 0, 0);
            }
        }
}

// Maximum over the four lanes that share lane % 16, to all of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t x)
{
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(x, x, false, false));
    x = max(a[0], a[1]);
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(x, x, false, false));
    return max(b[0], b[1]);
}

// LDS written by some lanes of this wave is read by others of it: the wave's LDS
// operations complete in order, so the compiler only has to keep theirs.
__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace gdr
