// gdr_chain.hip -- the gated delta rule over whole sequences, chunk by chunk on the matrix
// cores: the parallel forward pass, and the backward pass's walk of the state's gradient.
//
// CHUNK FORM.  Over a chunk of C = 32 tokens entered by state S, with alpha_i = exp(g_i),
// P_ij = alpha_{j+1} .. alpha_i, gamma_i = alpha_first .. alpha_i and gamma_C its last,
//     Z  = V - diag(gamma) K S                      the residuals if the chunk wrote nothing
//     R  = (I + X B)^-1 Z,     X_ij = P_ij k_i.k_j for j < i, B = diag(beta)
//     O  = scale diag(gamma) Q S + A R,  A_ij = scale P_ij q_i.k_j beta_j for j <= i
//     S' = gamma_C S + K^T diag(beta_j P_Cj) R.
// Backward, from the gradient G of the state behind the chunk (dO the gradient of O):
//     D  = A'^T dO + diag(P_C) K G,                 A' = A without beta
//     Y  = (I + B X)^-T D                           (Y is the gradient of beta R; dV = beta Y)
//     G' = gamma_C G + Q^T diag(scale gamma) dO - K^T diag(gamma beta) Y.
// Both walks have the same shape: two products with the state, a triangular 32 x 32
// product, and an update of the state; value columns never meet.  The decays enter as
// products of alphas (a column of P per lane), so no exponent range limits them and
// alpha = 0 is exact.
//
// MAPPING.  A workgroup takes 64 value columns of one head (fewer where there are few heads)
// and walks its chunks in order, with one barrier per chunk.  Four (two, one) consumer waves
// keep 16 columns of the state each, in the accumulator layout of the matrix cores, and do the
// products above; four producer waves prepare what does not depend on the state, up to three
// chunks ahead:
//     decay wave  (s + 3)  P, gamma and the vectors derived from them
//     K wave      (s + 2)  the rows of K, X = P o K K^T
//     Q wave      (s + 1)  the rows of Q, A = P o Q K^T (K from LDS)
//     inverse     (s + 1)  (I + X B)^-1 - I: two 16 x 16 blocks by substitution in fp32,
//                          the block below by fp32 matrix products.
// (Substitution, not products of powers of X: with equal keys the powers grow to 3000 and
// cancel.)  A row of K serves twice from one copy in LDS, as 16-byte fragments for K S and
// through the transpose load for K^T R: state tile t holds the channels
// 32 (t/2) + 8 (row/4) + 4 (t%2) + row%4, so the eight channels of a lane's fragment are
// consecutive, and the state's own registers are the operand of the next product.
//
// PRECISION.  The products with the state run on fp16 pieces: K and Q in one (bf16 inputs,
// exact) or two (fp32), the state and what is added to it in two, 2^-22 each.  A row of K or
// Q carries a power of two that brings its largest entry into [1/2, 1); a column of the state
// is kept in registers multiplied by a power of two (up), which changes only when the column
// leaves [2^-2, 2^13] or an added term 2^8: 32 terms below 2^8 then stay below the fp16
// limit of 65504.  (Rows of norms in [1/8, 2], as normalised keys are, go without a power:
// their squares are on the diagonal of K K^T.)  Where a column is zero or the chunk's decay is
// below 1/4, the added terms decide its power.  The 32 x 32 products run on three bf16 pieces
// (A R on two where o is bf16, whose own rounding is 2^-8); the unit diagonal of the inverse is
// added in fp32.
//
// WHAT BOUNDS IT.  4 x 8192 tokens of 32 heads of 128 x 128 take 465 us (0.83 GB of inputs and
// outputs, 1.8 TB/s): vector instructions fill 55% of the SIMDs' cycles, matrix instructions
// 31%, and a chunk is one dependent path through a consumer (about 3500 cycles at K = 128, 2500
// at K = 64) beside which the producer on the same SIMD has to fit.  8 x 4096 tokens of 12 heads
// of 64 x 64, 128 chunks in a row on 96 to 192 workgroups, take 150 us.
#include <type_traits>

#include "gdr_launch.h"
#include "gdr_mfma.h"

namespace gdr {
namespace {

constexpr int C = 32;          // tokens of a chunk
constexpr int LDT = C + 8;     // pitch (bf16) of the 32 x 32 matrices: 16-byte reads without conflicts

enum Mode { FWD, CKPT, BWD };

struct ChainArgs {
    const void *q, *k, *v;     // v: forward
    const float *g, *beta, *first;  // first: state_in / d_state_out or nullptr
    const float *d_o;          // backward
    void *o;                   // forward
    float *last;               // state_out / d_state_in
    float *saved;              // ckpt / work
    float *rows;               // resid / Y
    const int *lengths;
    float scale;
    int B, T, Hk, H, V;
};

// fp16 pieces of an input row.
template <typename Tin> constexpr int input_pieces() { return std::is_same<Tin, float>::value ? 2 : 1; }

template <int K, int NP, int NA>
struct Smem {
    alignas(16) uint16_t k[3][NP][C][K + 16];
    alignas(16) uint16_t q[2][NP][C][K + 16];
    // inverse - I and A as [row][token slot] (backward: transposed); token t < 16 has slot
    // 8 (t/4) + t%4, token 16 + t four more: a fragment's eight tokens are consecutive
    alignas(16) uint16_t t[2][3][C][LDT];
    alignas(16) uint16_t a[2][NA][C][LDT];
    alignas(16) float x[2][C][36];   // x[j][i] = the triangular matrix at (i, j)
    alignas(16) float d[2][16][20];  // the inverse's diagonal blocks, [column][row]
    alignas(16) float vec[4][4][C];  // gamma | beta P_C (backward: P_C) | beta | gamma beta
    alignas(16) float con[4][3][C];  // vec 0, 1 (backward: 1, -3) with K's row factors; scale gamma with Q's
    alignas(16) float kf[C];         // row factors: K's (K wave)
    alignas(16) float qf[C];         // Q's (Q wave)
    alignas(16) float bk[4][C];      // beta with K's row factors (backward: these alone)
    alignas(16) float head[4][C];    // P from the start of a token's half chunk to the token
    alignas(16) float tail[4][C];    // P from behind the token to the end of its half
    float p[4][2][16][17];           // P inside the halves
};

// One element, widened or as it is.
__device__ __forceinline__ void fetch(float &x, Buffer b, unsigned at)
{
    x = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0));
}
__device__ __forceinline__ void fetch(uint16_t &x, Buffer b, unsigned at)
{
    x = __builtin_amdgcn_raw_buffer_load_b16(b, at, 0, 0);
}
// Eight input elements of a row.
template <typename Tin> struct Raw;
template <> struct Raw<uint16_t> {
    u32x4 x;
    __device__ void load(Buffer b, unsigned at) { x = __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0); }
    // the largest magnitude, as fp32 bits
    __device__ uint32_t top() const
    {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        u16x2 m = __builtin_bit_cast(u16x2, x[0] & 0x7fff7fffu);
#pragma unroll
        for (int e = 1; e < 4; ++e)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x[e] & 0x7fff7fffu));
        return static_cast<uint32_t>(m[0] > m[1] ? m[0] : m[1]) << 16;
    }
    __device__ void planes(float m1, s16x8 (&out)[1]) const
    {
        split8h<1>(f32x4{bf16_lo(x[0]), bf16_hi(x[0]), bf16_lo(x[1]), bf16_hi(x[1])},
                   f32x4{bf16_lo(x[2]), bf16_hi(x[2]), bf16_lo(x[3]), bf16_hi(x[3])}, out, m1);
    }
    __device__ void planes(float f, float m1, s16x8 (&out)[1]) const
    {
        split8h<1>(f32x4{bf16_lo(x[0]) * f, bf16_hi(x[0]) * f, bf16_lo(x[1]) * f, bf16_hi(x[1]) * f},
                   f32x4{bf16_lo(x[2]) * f, bf16_hi(x[2]) * f, bf16_lo(x[3]) * f, bf16_hi(x[3]) * f}, out, m1);
    }
    __device__ void bf16(s16x8 (&out)[1]) const { out[0] = __builtin_bit_cast(s16x8, x); }
};
template <> struct Raw<float> {
    f32x4 x, y;
    __device__ void load(Buffer b, unsigned at)
    {
        x = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0));
        y = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, at + 16, 0, 0));
    }
    __device__ uint32_t top() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            m = max(m, max(__float_as_uint(x[e]) & 0x7fffffffu, __float_as_uint(y[e]) & 0x7fffffffu));
        return m;
    }
    __device__ void planes(float f, float m1, s16x8 (&out)[2]) const { split8h<2>(x * f, y * f, out, m1); }
};

// The exponent e of a row or column whose largest magnitude has these fp32 bits: 2^-e brings
// it into [1/2, 1).  0 for a largest of 0, infinity or NaN; kept to what 2^e and 2^-e hold.
__device__ __forceinline__ int exponent(uint32_t bits)
{
    const int e = static_cast<int>(bits >> 23);
    return bits == 0 || e == 255 ? 0 : min(max(e - 126, -120), 120);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Four consecutive values.
__device__ __forceinline__ void put4(const float *, Buffer b, unsigned at, const f32x4 x)
{
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), b, at, 0, 0);
}
__device__ __forceinline__ void put4(const uint16_t *, Buffer b, unsigned at, const f32x4 x)
{
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3])}, b, at, 0, 0);
}

// What every wave of a workgroup knows.
struct Place {
    int lane, row, quad;  // lane % 16, lane / 16
    int b, h, kh;
    int L, n;             // tokens and chunks of this row
    size_t tok0;
};

// x of lane `J` of this lane's row of 16.
template <int J>
__device__ __forceinline__ float row_lane(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + J, 0xf, 0xf, true));
}

// Walk down the columns of a half's decays: lane (half, row) holds alpha of its token; on
// return p = P(last, row), all the product of all and from = that up to the token.
template <int I>
__device__ __forceinline__ void walk(float alpha, int row, float &p, float &all, float &from, float (*out)[17])
{
    if constexpr (I < 16) {
        const float x = row_lane<I>(alpha), next = p * x;
        const bool here = I == row;
        all *= x;
        p = here ? 1.f : next;
        from = here ? all : from;
        out[I][row] = p;
        walk<I + 1>(alpha, row, p, all, from, out);
    }
}

// Decays of chunk s + 3.
template <bool BACK, typename SM>
__device__ __forceinline__ void decay_wave(SM &sm, const ChainArgs &a, const Place &w)
{
    float g[2], be[2];
    auto load = [&](int s, int at) {
        const int c = BACK ? w.n - 1 - s : s, t = c * C + (w.lane & (C - 1));
        g[at] = be[at] = 0.f;  // behind the end: no decay, nothing written
        if (s < w.n && t < w.L) {
            const size_t i = (w.tok0 + t) * a.H + w.h;
            g[at] = a.g[i];
            be[at] = a.beta[i];
        }
    };
    auto body = [&](int s, auto at) {
        if (s < w.n) {
            const float alpha = expf(g[at]), beta = be[at];
            load(s + 2, at);
            const int half = w.quad & 1;  // the upper 32 lanes repeat the lower
            float tail = 0.f, all = 1.f, from = 0.f;
            walk<0>(alpha, w.row, tail, all, from, sm.p[s & 3][half]);
            const float first = wkv7::lane_bcast(all, 0), second = wkv7::lane_bcast(all, 16);
            const float gamma = half ? first * from : from, toend = half ? tail : tail * second;
            if (w.lane < C) {
                sm.head[s & 3][w.lane] = from;
                sm.tail[s & 3][w.lane] = tail;
                sm.vec[s & 3][0][w.lane] = gamma;
                sm.vec[s & 3][1][w.lane] = BACK ? toend : toend * beta;
                sm.vec[s & 3][2][w.lane] = beta;
                sm.vec[s & 3][3][w.lane] = gamma * beta;
            }
        }
        __syncthreads();
    };
    load(0, 0);
    load(1, 1);
    for (int s = 0;;) {
        body(s, std::integral_constant<int, 0>{});
        if (++s == w.n + 3)
            break;
        body(s, std::integral_constant<int, 1>{});
        if (++s == w.n + 3)
            break;
    }
}

// One step of the substitution: c[i] -= M(i, J) c[J] for i > J, then the next.  Lane (column
// of the inverse) r of a row of 16 holds M(i, r) in m[i]; the broadcast of lane J's is part of
// the multiply-add.  (m must not have been written by the vector unit in the two cycles before:
// the s_nop.)
template <int J>
__device__ __forceinline__ void eliminate(float (&c)[16], const float (&m)[16])
{
    if constexpr (J < 15) {
        const float x = -c[J];
        asm volatile("s_nop 1");
#pragma unroll
        for (int i = J + 1; i < 16; ++i)
            asm volatile("v_fmac_f32_dpp %0, %1, %2 row_newbcast:%3 row_mask:0xf bank_mask:0xf"
                         : "+v"(c[i])
                         : "v"(m[i]), "v"(x), "n"(J));
        eliminate<J + 1>(c, m);
    }
}

// The inverse of chunk s + 1, less the unit diagonal.
template <bool BACK, typename SM>
__device__ __forceinline__ void inverse_wave(SM &sm, const Place &w)
{
    const int row = w.row, quad = w.quad, blk = quad & 1;
    float unit[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        unit[i] = i == row ? 1.f : 0.f;
        asm volatile("" : "+v"(unit[i]));  // kept in a register: 16 lane masks would not be
    }
    for (int it = -3; it < w.n; ++it) {
        const int s = it + 1;
        if (s >= 0 && s < w.n) {
            const float(*x)[36] = sm.x[s & 1];
            // lanes 16 blk + r (and the upper 32 again): column r of diagonal block blk
            float c[16], m[16];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const f32x4 u = *reinterpret_cast<const f32x4 *>(&x[16 * blk + row][16 * blk + i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    m[i + e] = u[e];
                    c[i + e] = unit[i + e];
                }
            }
            // the block below, read ahead
            float low[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                low[e] = BACK ? x[4 * e + quad][16 + row] : x[row][16 + 4 * e + quad];
            eliminate<0>(c, m);
            if (w.lane < 32)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<f32x4 *>(&sm.d[blk][row][i]) = f32x4{c[i], c[i + 1], c[i + 2], c[i + 3]};
            wave_lds_fence();
            // the block below the diagonal, -D1 M D0 (backward: its rows; forward: transposed)
            f32x4 acc = {0.f, 0.f, 0.f, 0.f}, below = acc, right, diag[2];
            float left[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                left[e] = BACK ? sm.d[0][row][4 * e + quad] : sm.d[1][4 * e + quad][row];
            if constexpr (BACK) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    right[e] = sm.d[1][4 * quad + e][row];
                diag[0] = *reinterpret_cast<const f32x4 *>(&sm.d[0][row][4 * quad]);
                diag[1] = *reinterpret_cast<const f32x4 *>(&sm.d[1][row][4 * quad]);
            } else {
                right = *reinterpret_cast<const f32x4 *>(&sm.d[0][row][4 * quad]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    diag[0][e] = sm.d[0][4 * quad + e][row];
                    diag[1][e] = sm.d[1][4 * quad + e][row];
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(low[e], left[e], acc, 0, 0, 0);
            u32x2 out[3];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f32x4 dd = diag[e];
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    dd[f] = 4 * quad + f == row ? 0.f : dd[f];
                split4<3>(dd, out);
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<u32x2 *>(&sm.t[s & 1][p][16 * e + row][8 * quad + 4 * e]) = out[p];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                below = __builtin_amdgcn_mfma_f32_16x16x4f32(right[e], -acc[e], below, 0, 0, 0);
            split4<3>(below, out);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<u32x2 *>(&sm.t[s & 1][p][BACK ? row : 16 + row][8 * quad + (BACK ? 4 : 0)]) = out[p];
        }
        __syncthreads();
    }
}

// Rows of a tensor [b, :, kh, :] in tile fragments: lane (row, quad) takes eight channels.
template <typename Tin, int K, bool BACK>
struct Rows {
    static constexpr int NP = input_pieces<Tin>(), NM = K / 32;
    static constexpr int DEPTH = std::is_same<Tin, float>::value ? 1 : 2;  // chunks in flight
    const Place &w;
    const Tin *base;
    size_t stride;
    unsigned at0;  // this lane's place in the first tile, bytes
    Raw<Tin> raw[DEPTH][2][NM];
    __device__ __forceinline__ Rows(const void *p, const ChainArgs &a, const Place &w_) : w(w_)
    {
        stride = static_cast<size_t>(a.Hk) * K;
        base = static_cast<const Tin *>(p) + (w.tok0 * a.Hk + w.kh) * K;
        at0 = static_cast<unsigned>((w.row * stride + 8 * w.quad) * sizeof(Tin));
    }
    __device__ __forceinline__ int first(int s) const { return (BACK ? w.n - 1 - s : s) * C; }
    __device__ __forceinline__ void load(int s, int at)
    {
        if (s >= w.n)
            return;
        const int f = first(s);
        const Buffer b = rows_buffer(base + f * stride, min(w.L - f, C), stride);
#pragma unroll
        for (int tau = 0; tau < 2; ++tau)
#pragma unroll
            for (int m = 0; m < NM; ++m)
                raw[at][tau][m].load(b, at0 + static_cast<unsigned>((16 * tau * stride + 32 * m) * sizeof(Tin)));
    }
    // fp16 fragments of the rows with their power of two; fac undoes it.  `self`: the diagonal
    // tiles of the rows' products with themselves (bf16 inputs).
    __device__ __forceinline__ void convert(int at, const f32x4 (&self)[2], float m1, s16x8 (&f)[2][NM][NP],
                                            float (&fac)[2]) const
    {
        fac[0] = fac[1] = 1.f;
        if constexpr (NP == 1) {
            // |x|^2 of this lane's rows, from the lanes that hold the diagonal
            bool plain = true;
#pragma unroll
            for (int tau = 0; tau < 2; ++tau) {
                const f32x4 &d = self[tau];
                const float lo = w.row & 1 ? d[1] : d[0], hi = w.row & 1 ? d[3] : d[2];
                const float sq = __shfl(w.row & 2 ? hi : lo, 16 * (w.row >> 2) + w.row);
                plain = plain && ((sq >= 0x1p-6f && sq <= 4.f) || sq == 0.f);
            }
            if (__all(plain)) {  // rows of norms in [1/8, 2]: fp16 holds them as they are
#pragma unroll
                for (int tau = 0; tau < 2; ++tau)
#pragma unroll
                    for (int m = 0; m < NM; ++m)
                        raw[at][tau][m].planes(m1, f[tau][m]);
                return;
            }
        }
#pragma unroll
        for (int tau = 0; tau < 2; ++tau) {
            uint32_t top = 0;
#pragma unroll
            for (int m = 0; m < NM; ++m)
                top = max(top, raw[at][tau][m].top());
            const int e = exponent(quad_max(top));
            const float down = pow2(-e);
#pragma unroll
            for (int m = 0; m < NM; ++m)
                raw[at][tau][m].planes(down, m1, f[tau][m]);
            fac[tau] = pow2(e);
        }
    }
    // to LDS, [piece][row][channel]
    __device__ __forceinline__ void put(const s16x8 (&f)[2][NM][NP], uint16_t (*to)[C][K + 16]) const
    {
#pragma unroll
        for (int tau = 0; tau < 2; ++tau)
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    *reinterpret_cast<s16x8 *>(&to[p][16 * tau + w.row][32 * m + 8 * w.quad]) = f[tau][m][p];
    }
};

// The rows of K and X of chunk s + 2.
template <typename Tin, int K, bool BACK, typename SM>
__device__ __forceinline__ void k_wave(SM &sm, const ChainArgs &a, const Place &w)
{
    constexpr int NP = input_pieces<Tin>(), NM = K / 32;
    using R = Rows<Tin, K, BACK>;
    const int row = w.row, quad = w.quad;
    const float m1 = minus_one();
    R rows(a.k, a, w);
    int slot = 0;  // s % 3
    auto body = [&](int it, auto at) {
        const int s = it + 2;
        if (s >= 0 && s < w.n) {
            f32x4 acc[3];
#pragma unroll
            for (int e = 0; e < 3; ++e)
                acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
            s16x8 f[2][NM][NP];
            float fac[2];
            if constexpr (NP == 1) {
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    s16x8 kb[2][1];
#pragma unroll
                    for (int tau = 0; tau < 2; ++tau)
                        rows.raw[at][tau][m].bf16(kb[tau]);
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        mma<1, 1>(acc[e], kb[e > 0], kb[e > 1]);
                }
            }
            const f32x4 self[2] = {acc[0], acc[2]};
            rows.convert(at, self, m1, f, fac);
            rows.load(s + R::DEPTH, at);
            rows.put(f, sm.k[slot]);
            slot = slot == 2 ? 0 : slot + 1;
            if (quad == 0) {
                sm.kf[row] = fac[0];
                sm.kf[16 + row] = fac[1];
            }
            if constexpr (NP != 1)
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        mmah<NP, NP>(acc[e], f[e > 0][m], f[e > 1][m]);
            wave_lds_fence();
            if constexpr (NP != 1)
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    acc[e] *= fac[e > 1] * *reinterpret_cast<const f32x4 *>(&sm.kf[16 * (e > 0) + 4 * quad]);
            const float *head = sm.head[s & 3], *tail = sm.tail[s & 3];
            const float *beta = sm.vec[s & 3][2];
            if (w.lane < C) {
                const int l = w.lane;
                const float kf = sm.kf[l];
                sm.con[s & 3][0][l] = (BACK ? sm.vec[s & 3][1][l] : sm.vec[s & 3][0][l]) * kf;
                sm.con[s & 3][1][l] = (BACK ? -sm.vec[s & 3][3][l] : sm.vec[s & 3][1][l]) * kf;
                sm.bk[s & 3][l] = BACK ? kf : beta[l] * kf;
            }
            // lane: column j; registers: rows i
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                const int ti = e > 0, tj = e > 1, i0 = 16 * ti + 4 * quad, j = 16 * tj + row;
                f32x4 v, x;
                if constexpr (BACK)
                    x = *reinterpret_cast<const f32x4 *>(&beta[i0]) * acc[e];
                else
                    x = beta[j] * acc[e];
                if (e == 1) {
                    v = x * (tail[j] * *reinterpret_cast<const f32x4 *>(&head[i0]));
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float y = sm.p[s & 3][ti][4 * quad + r][row] * x[r];
                        v[r] = row < 4 * quad + r ? y : 0.f;
                    }
                }
                *reinterpret_cast<f32x4 *>(&sm.x[s & 1][j][i0]) = v;
            }
        }
        __syncthreads();
    };
#pragma unroll
    for (int i = 0; i < R::DEPTH; ++i)
        rows.load(i, i);
    // the buffer in use alternates from chunk 0, which iteration -2 takes
    for (int it = -3;;) {
        body(it, std::integral_constant<int, R::DEPTH - 1>{});
        if (++it == w.n)
            break;
        body(it, std::integral_constant<int, 0>{});
        if (++it == w.n)
            break;
    }
}

// The rows of Q and A of chunk s + 1, with the rows of K that the K wave has left in LDS.
template <typename Tin, int K, int NA, bool BACK, typename SM>
__device__ __forceinline__ void q_wave(SM &sm, const ChainArgs &a, const Place &w)
{
    constexpr int NP = input_pieces<Tin>(), NM = K / 32;
    using R = Rows<Tin, K, BACK>;
    const int row = w.row, quad = w.quad;
    const float m1 = minus_one();
    R rows(a.q, a, w);
    int slot = 0;  // s % 3
    auto body = [&](int it, auto at) {
        const int s = it + 1;
        if (s >= 0 && s < w.n) {
            s16x8 kh[2][NM][NP];
#pragma unroll
            for (int tau = 0; tau < 2; ++tau)
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        kh[tau][m][p] = lds8(&sm.k[slot][p][16 * tau + row][32 * m + 8 * quad]);
            slot = slot == 2 ? 0 : slot + 1;
            f32x4 acc[3], self[2];
#pragma unroll
            for (int e = 0; e < 3; ++e)
                acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
            self[0] = self[1] = acc[0];
            s16x8 f[2][NM][NP];
            float fac[2];
            if constexpr (NP == 1)
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int tau = 0; tau < 2; ++tau) {
                        s16x8 qb[1];
                        rows.raw[at][tau][m].bf16(qb);
                        mma<1, 1>(self[tau], qb, qb);
                    }
            rows.convert(at, self, m1, f, fac);
            rows.load(s + R::DEPTH, at);
            rows.put(f, sm.q[s & 1]);
            if (quad == 0) {
                sm.qf[row] = fac[0];
                sm.qf[16 + row] = fac[1];
            }
            // forward: lane: row i of A; registers: columns j.  Backward: transposed.
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    if constexpr (BACK)
                        mmah<NP, NP>(acc[e], f[e > 0][m], kh[e > 1][m]);
                    else
                        mmah<NP, NP>(acc[e], kh[e > 1][m], f[e > 0][m]);
                }
            wave_lds_fence();
            const float *head = sm.head[s & 3], *tail = sm.tail[s & 3], *bk = sm.bk[s & 3];
            if (w.lane < C)
                sm.con[s & 3][2][w.lane] = a.scale * sm.vec[s & 3][0][w.lane] * sm.qf[w.lane];
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                const int ti = e > 0, tj = e > 1;
                f32x4 v;
                if constexpr (!BACK) {
                    const int i = 16 * ti + row, j0 = 16 * tj + 4 * quad;
                    const f32x4 x = ((a.scale * fac[ti]) * *reinterpret_cast<const f32x4 *>(&bk[j0])) * acc[e];
                    if (e == 1) {
                        v = x * (head[i] * *reinterpret_cast<const f32x4 *>(&tail[j0]));
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float y = sm.p[s & 3][ti][row][4 * quad + r] * x[r];
                            v[r] = 4 * quad + r <= row ? y : 0.f;
                        }
                    }
                } else {
                    const int i0 = 16 * ti + 4 * quad, j = 16 * tj + row;
                    const f32x4 x = ((a.scale * bk[j]) * *reinterpret_cast<const f32x4 *>(&sm.qf[i0])) * acc[e];
                    if (e == 1) {
                        v = x * (tail[j] * *reinterpret_cast<const f32x4 *>(&head[i0]));
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float y = sm.p[s & 3][ti][4 * quad + r][row] * x[r];
                            v[r] = row <= 4 * quad + r ? y : 0.f;
                        }
                    }
                }
                u32x2 out[NA];
                split4<NA>(v, out);
#pragma unroll
                for (int p = 0; p < NA; ++p)
                    *reinterpret_cast<u32x2 *>(
                        &sm.a[s & 1][p][16 * (BACK ? tj : ti) + row][8 * quad + 4 * (BACK ? ti : tj)]) = out[p];
            }
        }
        __syncthreads();
    };
#pragma unroll
    for (int i = 0; i < R::DEPTH; ++i)
        rows.load(i, i);
    // the buffer in use alternates from chunk 0, which iteration -1 takes
    for (int it = -3;;) {
        body(it, std::integral_constant<int, 0>{});
        if (++it == w.n)
            break;
        body(it, std::integral_constant<int, R::DEPTH - 1>{});
        if (++it == w.n)
            break;
    }
}

// Workgroup index to (row, head, columns): the workgroups that read the same query / key head
// (`share` of them, next to each other) go to one XCD and its L2, the next such group to the
// next XCD.  (Consecutive workgroups go round the 8 XCDs.)
__device__ __forceinline__ unsigned chain_item(unsigned bid, unsigned n, unsigned share)
{
    const unsigned rounds = n / (8 * share) * 8 * share;
    if (bid >= rounds)
        return bid;
    const unsigned x = bid & 7, i = bid >> 3;
    return (i / share * 8 + x) * share + i % share;
}

// The row of rank r by length, the longest first: workgroups start in this order, so the long
// rows do not wait for a compute unit while short ones hold them.
__device__ __forceinline__ int by_length(const int *lengths, int B, int T, int r, int lane)
{
    const int own = lane < B ? min(max(lengths[lane], 0), T) : -1;
    int rank = 0;
    for (int i = 0; i < B; ++i) {
        const int x = __builtin_amdgcn_readlane(own, i);
        rank += x > own || (x == own && i < lane);
    }
    return __builtin_amdgcn_readfirstlane(__ffsll(__ballot(lane < B && rank == r)) - 1);
}

template <typename Tin, typename Tout, int K, int MODE>
__global__ __launch_bounds__(512) void gdr_chain_kernel(ChainArgs a)
{
    constexpr bool BACK = MODE == BWD;
    constexpr int NP = input_pieces<Tin>(), NM = K / 32, NT = K / 16;
    constexpr int NA = !BACK && std::is_same<Tout, uint16_t>::value ? 2 : 3;  // bf16 pieces in A R
    __shared__ Smem<K, NP, NA> sm;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int consumers = (blockDim.x >> 6) - 4, cols = 16 * consumers;
    const unsigned nblk = a.V / cols;
    const unsigned item = chain_item(blockIdx.x, gridDim.x, nblk * (a.H / a.Hk));
    Place w;
    w.lane = threadIdx.x & 63;
    w.row = w.lane & 15;
    w.quad = w.lane >> 4;
    w.b = item / nblk / a.H;
    w.h = item / nblk % a.H;
    if (a.lengths && a.B <= 64)
        w.b = by_length(a.lengths, a.B, a.T, w.b, w.lane);
    const unsigned head = w.b * a.H + w.h;
    w.kh = w.h / (a.H / a.Hk);
    w.L = a.lengths ? min(max(a.lengths[w.b], 0), a.T) : a.T;
    w.n = (w.L + C - 1) / C;
    w.tok0 = static_cast<size_t>(w.b) * a.T;

    for (unsigned i = threadIdx.x; i < sizeof(sm.t) / 4; i += blockDim.x)
        reinterpret_cast<uint32_t *>(sm.t)[i] = 0;  // the blocks above the diagonal stay 0
    for (unsigned i = threadIdx.x; i < sizeof(sm.a) / 4; i += blockDim.x)
        reinterpret_cast<uint32_t *>(sm.a)[i] = 0;
    __syncthreads();

    if (wave >= consumers) {
        // Wave i runs on SIMD i % 4: with two consumers the heavier two producers get the SIMDs
        // that these leave free.
        const int role = (wave - consumers) ^ (consumers == 2 ? 2 : 0);
        if (role == 0)
            k_wave<Tin, K, BACK>(sm, a, w);
        else if (role == 1)
            consumers == 2 ? decay_wave<BACK>(sm, a, w) : q_wave<Tin, K, NA, BACK>(sm, a, w);
        else if (role == 2)
            inverse_wave<BACK>(sm, w);
        else
            consumers == 2 ? q_wave<Tin, K, NA, BACK>(sm, a, w) : decay_wave<BACK>(sm, a, w);
        return;
    }

    // -------------------------------------------------------------------- consumers
    const int lane = w.lane, row = w.row, quad = w.quad, n = w.n, L = w.L;
    const float m1 = minus_one();
    const int col = (item % nblk) * cols + 16 * wave + row;
    const size_t vs = static_cast<size_t>(a.H) * a.V;
    // [b, 0, h, 0] of v, o, resid, d_o, and this lane's place in the rows of a chunk
    const size_t row0 = (w.tok0 * a.H + w.h) * a.V;
    unsigned at[2][4];
#pragma unroll
    for (int tau = 0; tau < 2; ++tau)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            at[tau][r] = static_cast<unsigned>((16 * tau + 4 * quad + r) * vs + col);
    // and of four columns of a token
    const unsigned turned[2] = {static_cast<unsigned>(row * vs + (col - row) + 4 * quad),
                                static_cast<unsigned>((16 + row) * vs + (col - row) + 4 * quad)};
    const size_t st0 = static_cast<size_t>(head) * K * a.V + col;  // [b, h, 0, col] of a state
    auto channel = [&](int t, int r) { return 32 * (t >> 1) + 8 * quad + 4 * (t & 1) + r; };
    using Trow = typename std::conditional<BACK, float, Tin>::type;
    const Trow *in = static_cast<const Trow *>(BACK ? static_cast<const void *>(a.d_o) : a.v) + row0;

    f32x4 S[NT];  // the state (backward: its gradient) times up
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[t][r] = a.first ? a.first[st0 + static_cast<size_t>(channel(t, r)) * a.V] : 0.f;
    float up = 1.f, down = 1.f;  // 2^e and 2^-e, one e for each column
    f32x4 down4 = {1.f, 1.f, 1.f, 1.f};  // down of the columns 4 quad .. 4 quad + 3
    int scale_e = 0;
    // Bring the column's scale back if an entry of S or an added term (in its true size) asks for it.
    // A column's entries and terms sit in four lanes: too large in one of them, or too small in
    // all four, is seen in the lanes' votes; maxima are formed only then.
    auto largest_entry = [&]() {
        float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; r += 2)
                top[t & 3] = fmaxf(fmaxf(fabsf(S[t][r]), fabsf(S[t][r + 1])), top[t & 3]);
        return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    };
    // columns in which one lane at least says yes: all sixteen?
    auto every_column = [](bool yes) {
        unsigned long long m = __ballot(yes);
        m |= m >> 32;
        m |= m >> 16;
        return (m & 0xffffu) == 0xffffu;
    };
    auto column_max = [](float x) { return __uint_as_float(quad_max(__float_as_uint(x))); };
    bool zero = false;  // the column is zero: what is added alone decides its scale
    // asks, and so the column's new scale, depends on that column alone: results are the same
    // whichever columns share the wave
    auto rescale = [&](bool asks, float top, float term) {
        int e = 0;
        if (asks && (top > 0.f || term > 0.f) && top < __builtin_huge_valf() && term < __builtin_huge_valf()) {
            const int of_top = top > 0.f ? exponent(__float_as_uint(top)) - scale_e : -1000;
            const int of_term = term > 0.f ? exponent(__float_as_uint(term)) - 3 : -1000;
            e = min(max(3 - max(of_top, of_term), -120), 120) - scale_e;  // to [4, 8)
        }
        scale_e += e;
        up = pow2(scale_e);
        down = pow2(-scale_e);
        if (!BACK)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                down4[r] = __shfl(down, 4 * quad + r);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[t][r] = ldexpf(S[t][r], e);
    };
    auto check_entries = [&]() {
        float top = largest_entry();
        zero = false;
        if (!every_column(top >= 0x1p-2f) || __any(!(top <= 0x1p13f))) {
            top = column_max(top);
            zero = top == 0.f;
            rescale(!(top >= 0x1p-2f && top <= 0x1p13f), top, 0.f);
        }
    };
    // The terms of a chunk, formed under the columns' scales and about to be added; S has decayed
    // already.  Small ones are looked at only where the column may be smaller still: it was zero or
    // has fallen below 1/4.
    auto check_terms = [&](auto form, const f32x4(&x)[2], const f32x4(&y)[2], bool fell) {
        auto largest = [&]() {
            form();
            float term = 0.f;
#pragma unroll
            for (int tau = 0; tau < 2; ++tau)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    term = fmaxf(fmaxf(fabsf(x[tau][r]), fabsf(y[tau][r])), term);
            return term;
        };
        float term = largest();
        const bool low = fell || zero;
        if (__any(!(term <= 0x1p8f)) || (__any(low) && !every_column(!low || term >= 0x1p-3f))) {
            term = column_max(term);
            up = 1.f;  // in their true size: a scale may be 2^120 off
            const float bare = column_max(largest());
            rescale(!(term <= 0x1p8f) || (low && term < 0x1p-3f), column_max(largest_entry()), bare);
            form();
        }
    };

    Trow next[2][4];
    auto load = [&](int s) {
        const int first = (BACK ? n - 1 - s : s) * C;
        const Buffer b = rows_buffer(in + first * vs, min(L - first, C), vs);
#pragma unroll
        for (int tau = 0; tau < 2; ++tau)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                fetch(next[tau][r], b, at[tau][r] * static_cast<unsigned>(sizeof(Trow)));
    };
    // The residuals of a chunk: a column a lane, as the products with them need it.
    auto store_rows = [&](int first, const f32x4(&x)[2]) {
        const Buffer b = rows_buffer(a.rows + row0 + first * vs, min(L - first, C), vs);
#pragma unroll
        for (int tau = 0; tau < 2; ++tau)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[tau][r]), b, at[tau][r] * 4, 0, 0);
    };
    // The outputs: their products are formed transposed, a token a lane, so that four columns go
    // in one store (8 x 4096 x 12 heads 153 -> 150 us).
    auto store_out = [&](int first, const f32x4(&x)[2]) {
        Tout *out = static_cast<Tout *>(a.o);
        const Buffer b = rows_buffer(out + row0 + first * vs, min(L - first, C), vs);
#pragma unroll
        for (int tau = 0; tau < 2; ++tau)
            put4(out, b, turned[tau] * static_cast<unsigned>(sizeof(Tout)), x[tau]);
    };
    if (n > 0)
        load(0);
    __syncthreads();
    __syncthreads();
    __syncthreads();
    // The plain forward pass stores a chunk's outputs at the top of the next: addresses and stores
    // then run while the first operands are on their way (8 x 4096 x 12 heads 155 -> 150 us; beside
    // the checkpoints' and residuals' stores it gives nothing).
    f32x4 O[2], R[2];
    auto store_chunk = [&](int c) {
        if constexpr (MODE != BWD)
            store_out(c * C, O);
        if constexpr (MODE != FWD)
            store_rows(c * C, R);
    };
    int kslot = 0;  // s % 3
    bool fell = false, again = false;  // the last chunk's decay was below 1/4; that, or above 1
    for (int s = 0; s < n; ++s) {
        const int slot = s & 1, c = BACK ? n - 1 - s : s;
        const auto &kr = sm.k[kslot];
        kslot = kslot == 2 ? 0 : kslot + 1;
        f32x4 v[2];
#pragma unroll
        for (int tau = 0; tau < 2; ++tau)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[tau][r] = load_elem(&next[tau][r], 0);
        if (s + 1 < n)
            load(s + 1);
        // the state on entering a block of 64 tokens (backward: the gradient behind it), in tile order
        if (MODE == CKPT ? (c & 1) == 0 : MODE == BWD && ((c & 1) == 1 || c == n - 1)) {
            const int nsaved = (a.T + kBlock - 1) / kBlock;
            float *to = a.saved + ((static_cast<size_t>(w.b) * nsaved + c / 2) * a.H + w.h) * K * a.V +
                        static_cast<size_t>(col / 16) * (16 * K) + 4 * lane;
#pragma unroll
            for (int t = 0; t < NT; ++t)
                *reinterpret_cast<f32x4 *>(to + 256 * t) = S[t] * down;
        }
        // Operands are asked for well before the products that use them: a wave alone on its SIMD
        // has nothing else to hide the LDS behind.
        f32x4 con[BACK ? 3 : 2][2];
        float scaled[2];  // scale gamma and Q's row factor of this lane's tokens
#pragma unroll
        for (int x = 0; x < (BACK ? 3 : 2); ++x)
#pragma unroll
            for (int tau = 0; tau < 2; ++tau)
                con[x][tau] = *reinterpret_cast<const f32x4 *>(&sm.con[s & 3][x][16 * tau + 4 * quad]);
        if (!BACK)
#pragma unroll
            for (int tau = 0; tau < 2; ++tau)
                scaled[tau] = sm.con[s & 3][2][16 * tau + row];
        const float gC = sm.vec[s & 3][0][C - 1];
        auto rows_of = [&](const uint16_t(&x)[NP][C][K + 16], int m, s16x8(&f)[2][NP]) {
#pragma unroll
            for (int tau = 0; tau < 2; ++tau)
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    f[tau][p] = lds8(&x[p][16 * tau + row][32 * m + 8 * quad]);
        };
        s16x8 kf[NM][2][NP], qf[NM][2][NP];
#pragma unroll
        for (int m = 0; m < NM; ++m)
            rows_of(kr, m, kf[m]);
        __builtin_amdgcn_sched_barrier(0);
        if (MODE == FWD && s > 0)
            store_chunk(c - 1);
        // A chunk adds at most 2^14 (backward: twice that), which twice over still fits on top of
        // 2^13 unless the chunk's "decay" was a growth.
        if (BACK || (s & 1) == 0 || again)
            check_entries();
        const unsigned decay = __builtin_amdgcn_readfirstlane(__float_as_uint(gC));
        fell = decay < 0x3e800000u;
        again = fell || decay > 0x3f800000u;
        if constexpr (!BACK && NP == 1)
#pragma unroll
            for (int m = 0; m < NM; ++m)
                rows_of(sm.q[slot], m, qf[m]);
        __builtin_amdgcn_sched_barrier(0);

        // products with the state
        f32x4 ks[2], qs[2];
        s16x8 Sp[NM][2];
#pragma unroll
        for (int tau = 0; tau < 2; ++tau)
            ks[tau] = qs[tau] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            split8h<2>(S[2 * m], S[2 * m + 1], Sp[m], m1);
            mmah2<NP, 2>(ks[0], ks[1], kf[m][0], kf[m][1], Sp[m]);
        }
        // the 32 x 32 matrices
        auto matrix = [&](const auto &x, auto &f) {
            constexpr int NZ = std::extent<std::remove_reference_t<decltype(x)>>::value;
#pragma unroll
            for (int tau = 0; tau < 2; ++tau)
#pragma unroll
                for (int p = 0; p < NZ; ++p)
                    f[tau][p] = lds8(&x[p][16 * tau + row][8 * quad]);
        };
        s16x8 tf[2][3], af[2][NA];
        matrix(sm.t[slot], tf);
        if constexpr (BACK)
            matrix(sm.a[slot], af);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!BACK)
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                if constexpr (NP != 1)
                    rows_of(sm.q[slot], m, qf[m]);
                mmah2<NP, 2, true>(qs[0], qs[1], qf[m][0], qf[m][1], Sp[m]);
            }
        // K^T or Q^T of state tile t
        auto transposed = [&](const uint16_t(&x)[NP][C][K + 16], int t, s16x8(&f)[NP]) {
            const int at = 32 * (t >> 1) + 8 * (lane & 3) + 4 * (t & 1), r = 4 * quad + (row >> 2);
#pragma unroll
            for (int p = 0; p < NP; ++p)
                f[p] = cat(tr4(&x[p][r][at]), tr4(&x[p][16 + r][at]));
        };
        f32x4 u[2];
        s16x8 zp[3], up2[2];
        if constexpr (!BACK) {
            const f32x4 qdown = down4;  // qs was formed under this scale
#pragma unroll
            for (int tau = 0; tau < 2; ++tau) {
                const f32x4 c = con[0][tau] * down;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    R[tau][r] = fmaf(-c[r], ks[tau][r], v[tau][r]);
            }
            split8<3>(R[0], R[1], zp);
            s16x8 kt[NT][NP];
            if constexpr (NP == 1)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    transposed(kr, t, kt[t]);
            __builtin_amdgcn_sched_barrier(0);
            mma2<3, 3>(R[0], R[1], tf[0], tf[1], zp);
            matrix(sm.a[slot], af);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                S[t] *= gC;
            check_terms(
                [&]() {
#pragma unroll
                    for (int tau = 0; tau < 2; ++tau)
                        u[tau] = con[1][tau] * (R[tau] * up);
                },
                u, u, fell);
            split8h<2>(u[0], u[1], up2, m1);
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                if constexpr (NP != 1) {
                    transposed(kr, t, kt[t]);
                    transposed(kr, t + 1, kt[t + 1]);
                }
                mmah2<NP, 2>(S[t], S[t + 1], kt[t], kt[t + 1], up2);
            }
            s16x8 rp[NA];
            split8<NA>(R[0], R[1], rp);
#pragma unroll
            for (int tau = 0; tau < 2; ++tau)
                O[tau] = (scaled[tau] * qdown) * qs[tau];
            mma2<NA, NA, true>(O[0], O[1], af[0], af[1], rp);
        } else {
            f32x4 y[2];
            s16x8 yp[2];
            split8<3>(v[0], v[1], zp);
#pragma unroll
            for (int tau = 0; tau < 2; ++tau)
                R[tau] = (con[0][tau] * down) * ks[tau];
            mma2<3, 3>(R[0], R[1], af[0], af[1], zp);
            split8<3>(R[0], R[1], zp);
            mma2<3, 3>(R[0], R[1], tf[0], tf[1], zp);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                S[t] *= gC;
            check_terms(
                [&]() {
#pragma unroll
                    for (int tau = 0; tau < 2; ++tau) {
                        u[tau] = con[1][tau] * (R[tau] * up);
                        y[tau] = con[2][tau] * (v[tau] * up);
                    }
                },
                u, y, fell);
            split8h<2>(u[0], u[1], up2, m1);
            split8h<2>(y[0], y[1], yp, m1);
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                s16x8 x[2][NP];
                transposed(sm.q[slot], t, x[0]);
                transposed(sm.q[slot], t + 1, x[1]);
                mmah2<NP, 2>(S[t], S[t + 1], x[0], x[1], yp);
                transposed(kr, t, x[0]);
                transposed(kr, t + 1, x[1]);
                mmah2<NP, 2>(S[t], S[t + 1], x[0], x[1], up2);
            }
        }
        if (MODE != FWD)
            store_chunk(c);
        __syncthreads();
    }
    if (MODE == FWD && n > 0)
        store_chunk(n - 1);
    if (n > 0 || a.first != a.last)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                a.last[st0 + static_cast<size_t>(channel(t, r)) * a.V] = S[t][r] * down;
}

template <typename Tin, typename Tout, int MODE>
hipError_t launch_k(const ChainArgs &a, int K, hipStream_t stream)
{
    // Consumer waves of a workgroup: four (64 columns), or two or one while that many more
    // workgroups still fit the 256 compute units side by side.  A consumer with its SIMD to
    // itself walks faster (2048 tokens, 64 x 64 heads: 32 heads 96 us with four, 79 with two, 71
    // with one; 96 heads 96, 85 and, in two rounds, 145; 128 wide columns of 128 channels 126,
    // 113 and 194), at the price of preparing the same chunk in each workgroup.
    const long long units = static_cast<long long>(a.B) * a.H * (a.V / 64);
    const int consumers = units * 4 <= 256 ? 1 : units * 2 <= 256 ? 2 : 4;
    const dim3 grid(static_cast<unsigned>(units * (4 / consumers))), block(64 * (4 + consumers));
    if (K == 64)
        hipLaunchKernelGGL((gdr_chain_kernel<Tin, Tout, 64, MODE>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((gdr_chain_kernel<Tin, Tout, 128, MODE>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_chain(const SeqArgs &p, hipStream_t stream)
{
    ChainArgs a = {};
    a.q = p.q; a.k = p.k; a.v = p.v; a.g = p.g; a.beta = p.beta; a.first = p.state_in;
    a.o = p.o; a.last = p.state_out; a.saved = p.ckpt; a.rows = p.resid; a.lengths = p.lengths;
    a.scale = p.scale;
    a.B = p.B; a.T = p.T; a.Hk = p.Hk; a.H = p.H; a.V = p.V;
    if (p.ckpt)
        return p.in_bf16 ? launch_k<uint16_t, float, CKPT>(a, p.K, stream) : launch_k<float, float, CKPT>(a, p.K, stream);
    if (p.in_bf16)
        return p.o_bf16 ? launch_k<uint16_t, uint16_t, FWD>(a, p.K, stream) : launch_k<uint16_t, float, FWD>(a, p.K, stream);
    return p.o_bf16 ? launch_k<float, uint16_t, FWD>(a, p.K, stream) : launch_k<float, float, FWD>(a, p.K, stream);
}

hipError_t launch_backward_chain(const BwdArgs &p, hipStream_t stream)
{
    ChainArgs a = {};
    a.q = p.q; a.k = p.k; a.g = p.g; a.beta = p.beta; a.first = p.d_state_out; a.d_o = p.d_o;
    a.last = p.d_state_in; a.saved = p.work; a.rows = p.dv;
    a.scale = p.scale;
    a.B = p.B; a.T = p.T; a.Hk = p.Hk; a.H = p.H; a.V = p.V;
    return p.in_bf16 ? launch_k<uint16_t, float, BWD>(a, p.K, stream) : launch_k<float, float, BWD>(a, p.K, stream);
}

}  // namespace gdr
