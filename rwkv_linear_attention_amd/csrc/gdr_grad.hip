// gdr_grad.hip -- the gradients of the gated delta rule, block by block of 64 tokens.
//
// The backward chain (gdr_chain.hip) has left, for every value head, Y (the gradient of
// beta R) in dv and the gradient G of the state behind each block in work; the forward pass
// kept the state S entering the block and the residuals R.  With U = beta R, dV = beta Y and
// decays P_ij, gamma_i, P_Cj as in the chain but over the block, nothing couples two blocks:
//     E1 = scale P o tril(dO U^T),   E2 = -P o tril(dV U^T, -1)
//     dq = diag(scale gamma) dO S^T + E1 K
//     dk = -diag(gamma) dV S^T + diag(P_C) U G^T + E1^T Q + (E2 + E2^T) K
//     dv = dV,   dbeta_i = R_i . Y_i
//     dg_t = sum_{j < t <= i} W_ij + sum_{i >= t} e_i + sum_{j < t} f_j + gamma_C <G, S>
// where W = E1 o Q K^T + E2 o K K^T, e_i = q_i . (diag(scale gamma) dO S^T)_i -
// k_i . (diag(gamma) dV S^T)_i and f_j = k_j . (diag(P_C) U G^T)_j: what the decay of token t
// multiplies, term by term.  (Sums over i of the derivative by the decays from the block's
// start to i would need no W, but cancel: ten times the error.)  No division by beta or by a
// decay: both may be 0.
//
// MAPPING.  A workgroup of four waves takes one block of one query / key head and goes over
// the value heads of its group in order, so dq and dk are summed in a fixed order.  Wave w
// owns the rows 16 w .. 16 w + 15.  Per 32 value columns, the 32 columns of S and G are
// staged in LDS as three bf16 pieces and read through the transpose load; rows of dO, Y and R
// come straight from memory in fragment layout; U's fragments are shared through LDS.  Then
// E1 and E2 go to LDS once (they replace the staged states) and serve as they are and
// transposed.  Everything is on three bf16 pieces: products of magnitudes no scale is known of.
//
// WHAT BOUNDS IT.  2 x 4096 tokens of 32 heads of 128 x 128 on 16 key heads take 395 us for
// 1.65 GB (S, G, dO, Y, R in, five gradients out, dq and dk twice): 4.2 TB/s, against 4.8 of a
// plain copy.  8 x 1024 tokens of 12 heads of 64 x 64 take 67 us.
#include <type_traits>

#include "gdr_launch.h"
#include "gdr_mfma.h"

namespace gdr {
namespace {

constexpr int TB = kBlock;   // tokens of a block
constexpr int VB = 32;       // value columns of a step
constexpr int LDE = TB + 8;  // pitch (bf16) of E1 and E2

template <typename Tin> constexpr int row_pieces() { return std::is_same<Tin, float>::value ? 3 : 1; }

template <int K, int NB>
struct Smem {
    union {
        uint16_t st[2][3][VB][K + 16];  // S and G: [value column][channel]
        uint16_t m[2][3][TB][LDE];      // E1 and E2: [i][slot of j]
    };
    union {
        uint16_t rows[NB][TB][K + 16];  // K, then Q
        uint16_t u[4][3][64][8];        // U's fragments by row tile
    };
    float diag[4][16][17];  // P inside a tile of 16 tokens
    float a[TB], b[TB];     // P from a tile's start to its token; from behind the token to its end
    float gamma[TB], pc[TB], beta[TB], bp[4];
    float e[TB], f[TB], pair[4][TB], sums[4];
};

__device__ __forceinline__ float quad_sum(float x)
{
    const u32x2 a = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const u32x2 b = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int J>
__device__ __forceinline__ float row_lane(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + J, 0xf, 0xf, true));
}

// Walk down the columns of a tile's decays: lane (tile, row) holds alpha of its token; on
// return p = P(last, row) and from = P(before the tile, row).
template <int I>
__device__ __forceinline__ void walk(float alpha, int row, float &p, float &all, float &from, float (*diag)[17])
{
    if constexpr (I < 16) {
        const float x = row_lane<I>(alpha), next = p * x;
        all *= x;
        p = I == row ? 1.f : next;
        from = I == row ? all : from;
        diag[I][row] = p;
        walk<I + 1>(alpha, row, p, all, from, diag);
    }
}

// Eight elements of a row as bf16 pieces.
template <typename Tin, int NB>
__device__ __forceinline__ void fragment(Buffer b, unsigned at, s16x8 (&f)[NB])
{
    if constexpr (NB == 1)
        f[0] = __builtin_bit_cast(s16x8, fetch4(b, at));
    else
        split8<NB>(__builtin_bit_cast(f32x4, fetch4(b, at)), __builtin_bit_cast(f32x4, fetch4(b, at + 16)), f);
}

// Waves per SIMD: two workgroups share a compute unit with bf16 inputs (80 KB of LDS each).
template <typename Tin> constexpr int grad_waves() { return std::is_same<Tin, float>::value ? 1 : 2; }

template <typename Tin, int K>
__global__ __launch_bounds__(256, grad_waves<Tin>()) void gdr_grad_kernel(BwdArgs p, int nblk)
{
    constexpr int NB = row_pieces<Tin>(), NT = K / 16;
    constexpr int UNITS = VB * K / 4 / 256;  // 16-byte units of a staged state, per thread
    __shared__ Smem<K, NB> sm;

    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned item = xcd_item(blockIdx.x, gridDim.x);
    const int kh = item % p.Hk, blk = (item / p.Hk) % nblk, b = item / p.Hk / nblk;
    const int group = p.H / p.Hk, t0 = blk * TB, live = min(p.T - t0, TB);  // tokens of this block
    const size_t tok0 = static_cast<size_t>(b) * p.T + t0;
    const size_t qk0 = (tok0 * p.Hk + kh) * K, qs = static_cast<size_t>(p.Hk) * K;
    for (int hh = 0; hh < group; ++hh) {
        const int h = kh * group + hh;
        // Addresses are formed per head: hoisted out of this loop, a few hundred of them, they
        // would spill.
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        int lane = tid & 63, row = lane & 15, quad = lane >> 4;
        int mine = 16 * w + row;  // this lane's token as a fragment row
        bool on = mine < live;

        // The rows of K or Q to LDS, in bf16 pieces; rows behind the end are 0.
        const unsigned qrow = static_cast<unsigned>(qs * sizeof(Tin));  // bytes of a row of q or k
        const Buffer qb = rows_buffer(static_cast<const Tin *>(p.q) + qk0, live, qs);
        const Buffer kb = rows_buffer(static_cast<const Tin *>(p.k) + qk0, live, qs);
        auto stage_rows = [&](Buffer src) {
            constexpr int N = TB * (K / 8) / 256, STEP = N < 4 ? N : 4;
#pragma unroll
            for (int i0 = 0; i0 < N; i0 += STEP) {
                s16x8 f[STEP][NB];
#pragma unroll
                for (int i = 0; i < STEP; ++i) {
                    const int u = tid + 256 * (i0 + i), t = u / (K / 8), c = 8 * (u % (K / 8));
                    fragment<Tin>(src, t * qrow + c * static_cast<unsigned>(sizeof(Tin)), f[i]);
                }
#pragma unroll
                for (int i = 0; i < STEP; ++i) {
                    const int u = tid + 256 * (i0 + i), t = u / (K / 8), c = 8 * (u % (K / 8));
#pragma unroll
                    for (int y = 0; y < NB; ++y)
                        *reinterpret_cast<s16x8 *>(&sm.rows[y][t][c]) = f[i][y];
                }
            }
        };
        // staged rows 16 w + 4 quad + r (r = 0..3), channel 16 t + row
        auto staged = [&](int t) {
            f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = NB - 1; i >= 0; --i) {
                const s16x4 x = tr4(&sm.rows[i][16 * w + 4 * quad + (row >> 2)][16 * t + 4 * (lane & 3)]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    y[r] += bf16_lo(static_cast<uint16_t>(x[r]));
            }
            return y;
        };

        if (w == 0) {  // decays
            float g = 0.f, beta = 0.f;
            if (lane < live) {
                g = p.g[(tok0 + lane) * p.H + h];
                beta = p.beta[(tok0 + lane) * p.H + h];
            }
            float last = 0.f, all = 1.f, from = 0.f;
            walk<0>(expf(g), row, last, all, from, sm.diag[quad]);
            float before = 1.f, behind = 1.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = wkv7::lane_bcast(all, 16 * i);
                before = i < quad ? before * x : before;
                behind = i > quad ? behind * x : behind;
                if (lane == 0)
                    sm.bp[i] = x;
            }
            sm.a[lane] = from;
            sm.b[lane] = last;
            sm.gamma[lane] = before * from;
            sm.pc[lane] = last * behind;
            sm.beta[lane] = beta;
        }
        const size_t v0 = (tok0 * p.H + h) * p.V, vs = static_cast<size_t>(p.H) * p.V;
        const Buffer bo = rows_buffer(p.d_o + v0, live, vs), by = rows_buffer(p.dv + v0, live, vs);
        const Buffer br = rows_buffer(p.resid + v0, live, vs);
        const unsigned mrow = static_cast<unsigned>(mine * vs + 4 * quad) * 4;
        const float *sp = p.ckpt + ((static_cast<size_t>(b) * nblk + blk) * p.H + h) * K * p.V + 4 * tid;
        const float *gp = p.work + ((static_cast<size_t>(b) * nblk + blk) * p.H + h) * K * p.V + 4 * tid;

        f32x4 dq[NT], dr[NT], dc[NT], e1[4], e2[4];  // dr, dc: the two parts of dk; e1, e2 transposed
#pragma unroll
        for (int t = 0; t < NT; ++t)
            dq[t] = dr[t] = dc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 4; ++t)
            e1[t] = e2[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        float gs = 0.f, db = 0.f;
        __syncthreads();
        const float beta = sm.beta[mine];

        for (int v = 0; v < p.V; v += VB) {
            // (two workgroups share a compute unit: one multiplies while the other loads)
            f32x4 s4[UNITS], g4[UNITS], x4[3][2];  // units of S and G; dO, Y, R at columns 4 quad and 16 + 4 quad
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const unsigned at = mrow + 4 * (v + 16 * e);
                x4[0][e] = __builtin_bit_cast(f32x4, fetch4(bo, at));
                x4[1][e] = __builtin_bit_cast(f32x4, fetch4(by, at));
                x4[2][e] = __builtin_bit_cast(f32x4, fetch4(br, at));
            }
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                s4[i] = *reinterpret_cast<const f32x4 *>(sp + static_cast<size_t>(v) * K + 1024 * i);
                g4[i] = *reinterpret_cast<const f32x4 *>(gp + static_cast<size_t>(v) * K + 1024 * i);
            }
            s16x8 fo[3], fv[3], fu[3];
            split8<3>(x4[0][0], x4[0][1], fo);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    db = fmaf(x4[1][e][r], x4[2][e][r], db);
                x4[1][e] *= beta;
                x4[2][e] *= beta;
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x4[1][e]), by, mrow + 4 * (v + 16 * e), 0, 0);
            }
            split8<3>(x4[1][0], x4[1][1], fv);
            split8<3>(x4[2][0], x4[2][1], fu);
#pragma unroll
            for (int x = 0; x < 3; ++x)
                *reinterpret_cast<s16x8 *>(&sm.u[w][x][lane][0]) = fu[x];
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const int u = tid + 256 * i, jt = u / (4 * K), t = (u >> 6) % NT;
                const int vr = 16 * jt + row, c = 32 * (t >> 1) + 8 * quad + 4 * (t & 1);
                u32x2 f[3];
                split4<3>(s4[i], f);
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    *reinterpret_cast<u32x2 *>(&sm.st[0][x][vr][c]) = f[x];
                split4<3>(g4[i], f);
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    *reinterpret_cast<u32x2 *>(&sm.st[1][x][vr][c]) = f[x];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    gs = fmaf(s4[i][r], g4[i][r], gs);
            }
            __syncthreads();
            const int r0 = 4 * quad + (row >> 2);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                s16x8 f[3];
                const int c = 16 * t + 4 * (lane & 3);
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    f[x] = cat(tr4(&sm.st[0][x][r0][c]), tr4(&sm.st[0][x][16 + r0][c]));
                mma<3, 3>(dq[t], fo, f);
                mma<3, 3>(dr[t], fv, f);
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    f[x] = cat(tr4(&sm.st[1][x][r0][c]), tr4(&sm.st[1][x][16 + r0][c]));
                mma<3, 3>(dc[t], fu, f);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t <= w) {
                    s16x8 f[3];
#pragma unroll
                    for (int x = 0; x < 3; ++x)
                        f[x] = lds8(&sm.u[t][x][lane][0]);
                    mma<3, 3>(e1[t], f, fo);
                    mma<3, 3>(e2[t], f, fv);
                }
            __syncthreads();
        }

        db = quad_sum(db);
        tid = threadIdx.x;
        asm volatile("" : "+v"(tid));  // as above: nothing of this phase is formed before the columns' loop
        lane = tid & 63;
        row = lane & 15;
        quad = lane >> 4;
        mine = 16 * w + row;
        on = mine < live;
        if (quad == 0 && on)
            p.dbeta[(tok0 + mine) * p.H + h] = db;
        // decays on E1, E2 (lane: i = mine; registers: j = 16 t + 4 quad + r), to LDS
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t > (w | 1))
                continue;  // never read
            if (t <= w) {
                f32x4 P;
                if (t == w) {
                    P = f32x4{sm.diag[w][row][4 * quad], sm.diag[w][row][4 * quad + 1], sm.diag[w][row][4 * quad + 2],
                              sm.diag[w][row][4 * quad + 3]};
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        e1[t][r] = 4 * quad + r <= row ? P[r] * (p.scale * e1[t][r]) : 0.f;
                        e2[t][r] = 4 * quad + r < row ? -P[r] * e2[t][r] : 0.f;
                    }
                } else {
                    float mid = sm.a[mine];
#pragma unroll
                    for (int i = 1; i < 3; ++i)
                        mid *= i > t && i < w ? sm.bp[i] : 1.f;
                    P = mid * *reinterpret_cast<const f32x4 *>(&sm.b[16 * t + 4 * quad]);
                    e1[t] *= p.scale * P;
                    e2[t] *= -P;
                }
            }
            const int slot = 32 * (t >> 1) + 8 * quad + 4 * (t & 1);
            u32x2 f[3];
            split4<3>(e1[t], f);
#pragma unroll
            for (int x = 0; x < 3; ++x)
                *reinterpret_cast<u32x2 *>(&sm.m[0][x][mine][slot]) = f[x];
            split4<3>(e2[t], f);
#pragma unroll
            for (int x = 0; x < 3; ++x)
                *reinterpret_cast<u32x2 *>(&sm.m[1][x][mine][slot]) = f[x];
        }
        f32x4 gam = *reinterpret_cast<const f32x4 *>(&sm.gamma[16 * w + 4 * quad]);
        const f32x4 pc = *reinterpret_cast<const f32x4 *>(&sm.pc[16 * w + 4 * quad]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            dq[t] *= p.scale * gam;
            dr[t] *= -gam;
            dc[t] *= pc;
        }
        stage_rows(kb);
        __syncthreads();

        // out += E (rows 16 w ..) or E^T (columns 16 w ..) times the staged rows
        auto apply = [&](int which, bool trans, f32x4(&out)[NT]) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (trans ? s == 0 && w >= 2 : s == 1 && w < 2)
                    continue;  // zeros above the diagonal
                const int r0 = 32 * s + 4 * quad + (row >> 2);
                s16x8 f[3];
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    const int at = 32 * (w >> 1) + 8 * (lane & 3) + 4 * (w & 1);  // slot of j = 16 w + 4 (lane % 4)
                    f[x] = trans ? cat(tr4(&sm.m[which][x][r0][at]), tr4(&sm.m[which][x][16 + r0][at]))
                                 : lds8(&sm.m[which][x][mine][32 * s + 8 * quad]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    s16x8 g[NB];
                    const int c = 16 * t + 4 * (lane & 3);
#pragma unroll
                    for (int x = 0; x < NB; ++x)
                        g[x] = cat(tr4(&sm.rows[x][r0][c]), tr4(&sm.rows[x][16 + r0][c]));
                    mma<3, NB>(out[t], f, g);
                }
            }
        };
        // e and f, while dq, dr and dc hold the states' parts only
        f32x4 ei = {0.f, 0.f, 0.f, 0.f}, fj = ei;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4 k = staged(t);
            ei += k * dr[t];
            fj += k * dc[t];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
            fj[r] = wkv7::group16_sum(fj[r]);
        if (row == 0)
            *reinterpret_cast<f32x4 *>(&sm.f[16 * w + 4 * quad]) = fj;
        const float state = wkv7::wave_sum(gs) * sm.gamma[TB - 1];
        if (lane == 0)
            sm.sums[w] = state;
        // W of this lane's row i: prefix sums over j, then over the rows i > j of the wave
        {
            s16x8 qf[K / 32][NB], kf[K / 32][NB];
#pragma unroll
            for (int m = 0; m < K / 32; ++m) {
                fragment<Tin>(qb, mine * qrow + static_cast<unsigned>((32 * m + 8 * quad) * sizeof(Tin)), qf[m]);
#pragma unroll
                for (int x = 0; x < NB; ++x)
                    kf[m][x] = lds8(&sm.rows[x][mine][32 * m + 8 * quad]);
            }
            float before = 0.f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t <= w) {
                    f32x4 qk = {0.f, 0.f, 0.f, 0.f}, kk = qk;
#pragma unroll
                    for (int m = 0; m < K / 32; ++m) {
                        s16x8 x[NB];
#pragma unroll
                        for (int y = 0; y < NB; ++y)
                            x[y] = lds8(&sm.rows[y][16 * t + row][32 * m + 8 * quad]);
                        mma<NB, NB>(qk, x, qf[m]);
                        mma<NB, NB>(kk, x, kf[m]);
                    }
                    f32x4 run;
                    float sum = before;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const bool in = on && (t < w || 4 * quad + r < row);
                        run[r] = in ? fmaf(e1[t][r], qk[r], e2[t][r] * kk[r]) : 0.f;
                        if (r)
                            run[r] += run[r - 1];
                    }
                    // the quads before this one, of the same row, and all four
                    const uint32_t own = __float_as_uint(run[3]);
                    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(own, own, false, false));
                    const float pair = __uint_as_float(a[0]) + __uint_as_float(a[1]);
                    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(
                                                                  __float_as_uint(pair), __float_as_uint(pair), false, false));
                    sum += (quad >= 2 ? __uint_as_float(b[0]) : 0.f) + (quad & 1 ? __uint_as_float(a[0]) : 0.f);
                    before += __uint_as_float(b[0]) + __uint_as_float(b[1]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const bool past = t < w || 4 * quad + r < row;  // i >= j + 1
                        const float x = wkv7::group16_sum(past ? sum + run[r] : 0.f);
                        const int at = 16 * t + 4 * quad + r + 1;
                        if (row == 0 && at < TB)
                            sm.pair[w][at] = x;
                    }
                }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            dr[t] += dc[t];  // dk
            dc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        apply(0, false, dc);  // dq's other part, apart until dq has been used
        apply(1, false, dr);
        apply(1, true, dr);
        __syncthreads();
        stage_rows(qb);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            ei += staged(t) * dq[t];
            dq[t] += dc[t];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
            ei[r] = wkv7::group16_sum(ei[r]);
        if (row == 0)
            *reinterpret_cast<f32x4 *>(&sm.e[16 * w + 4 * quad]) = ei;
        apply(0, true, dr);
        __syncthreads();
        if (w == 0) {
            float x = sm.e[lane], y = sm.f[lane], z = 0.f;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const float u = __shfl_down(x, off), v = __shfl_up(y, off);
                x += lane + off < 64 ? u : 0.f;
                y += lane >= off ? v : 0.f;
            }
            const float ahead = __shfl_up(y, 1);
            // waves whose rows reach behind token `lane`
            for (int i = 0; i < 4; ++i)
                z += lane > 0 && 16 * i + 15 >= lane ? sm.pair[i][lane] : 0.f;
            x += (lane ? ahead : 0.f) + z + ((sm.sums[0] + sm.sums[1]) + (sm.sums[2] + sm.sums[3]));
            if (lane < live)
                p.dg[(tok0 + lane) * p.H + h] = x;
        }
        // dq, dk: the first head of a group writes, the others add
        const Buffer dqb = rows_buffer(p.dq + qk0, live, qs), dkb = rows_buffer(p.dk + qk0, live, qs);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * w + 4 * quad + r;
            const unsigned at = static_cast<unsigned>(t * qs + row) * 4;
            float x[NT], y[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                x[i] = dq[i][r];
                y[i] = dr[i][r];
            }
            if (hh) {
                float x0[NT], y0[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    x0[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(dqb, at + 64 * i, 0, 0));
                    y0[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(dkb, at + 64 * i, 0, 0));
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    x[i] += x0[i];
                    y[i] += y0[i];
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[i]), dqb, at + 64 * i, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[i]), dkb, at + 64 * i, 0, 0);
            }
        }
        __syncthreads();
    }
}

template <typename Tin>
hipError_t launch_typed(const BwdArgs &p, hipStream_t stream)
{
    const int nblk = (p.T + TB - 1) / TB;
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(p.B) * nblk * p.Hk)), block(256);
    if (p.K == 64)
        hipLaunchKernelGGL((gdr_grad_kernel<Tin, 64>), grid, block, 0, stream, p, nblk);
    else
        hipLaunchKernelGGL((gdr_grad_kernel<Tin, 128>), grid, block, 0, stream, p, nblk);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_backward(const BwdArgs &p, hipStream_t stream)
{
    const hipError_t e = launch_backward_chain(p, stream);
    if (e != hipSuccess)
        return e;
    return p.in_bf16 ? launch_typed<uint16_t>(p, stream) : launch_typed<float>(p, stream);
}

}  // namespace gdr
