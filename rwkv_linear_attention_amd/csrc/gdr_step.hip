// gdr_step.hip -- the recurrent gated delta rule (decode, verify, short prompts).
//
// Per head and token, with alpha = exp(g):
//     R = v - alpha S^T k,   S <- alpha S + beta k R^T,   o = scale S^T q.
// Value columns are independent, so a wave takes CW columns of one head and keeps
// their K x CW state in registers for all its tokens: no LDS, no barrier, and the
// state crosses HBM once each way.  A lane holds 4 columns (one 16-byte unit of a
// state row) and K / RG consecutive rows, RG = 256 / CW row groups; S^T k and S^T q
// are sums inside the lane, then across the row groups.
//
// What bounds it: the states' bytes.  32 rows of 40 heads of 128 x 128 take 36.9 us for 169 MB
// (4.6 TB/s; a plain copy reaches 4.8); 16 rows of 32 heads that keep the states after five
// tokens 48.0 us for 237 MB, mostly writes.
// A few heads alone wait for memory once (5 us).  Inputs of four tokens in flight instead of
// one gave nothing at T = 5 and cost 42 us against 37 at T = 1.
#include "gdr_device.h"
#include "gdr_launch.h"

namespace gdr {
namespace {

constexpr int CW = 32;        // value columns of a wave
constexpr int RG = 256 / CW;  // lanes (row groups) that share a column
constexpr int WAVES = 4;      // waves of a workgroup (independent of each other)

// Sum over the 8 row groups (lane bits 3, 4 and 5), to every lane.
__device__ __forceinline__ float group_sum(float x)
{
    x += wkv7::row_dpp<0x128>(x);  // row_ror:8, the other half of the 16-lane row
    const u32x2 a = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const u32x2 b = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int RPL>
struct Token {
    float q[RPL], k[RPL], v[4], g, beta;
};

template <typename Tin, typename Tout, int K>
__global__ __launch_bounds__(WAVES * 64) void gdr_step_kernel(SeqArgs p, unsigned nwaves)
{
    constexpr int RPL = K / RG;  // state rows of a lane
    const unsigned wave = xcd_item(blockIdx.x, gridDim.x) * WAVES + (threadIdx.x >> 6);
    if (wave >= nwaves)
        return;
    const int lane = threadIdx.x & 63;
    const unsigned nblk = p.V / CW;
    const unsigned head = wave / nblk;  // b * H + h
    const int b = head / p.H, h = head % p.H, kh = h / (p.H / p.Hk);
    const int row0 = (lane >> 3) * RPL, col0 = (wave % nblk) * CW + (lane & 7) * 4;
    int L = p.T;
    if (p.lengths)
        L = min(max(p.lengths[b], 0), p.T);

    const size_t tok0 = static_cast<size_t>(b) * p.T;
    const Tin *q = static_cast<const Tin *>(p.q) + (tok0 * p.Hk + kh) * K + row0;
    const Tin *k = static_cast<const Tin *>(p.k) + (tok0 * p.Hk + kh) * K + row0;
    const Tin *v = static_cast<const Tin *>(p.v) + (tok0 * p.H + h) * p.V + col0;
    const float *g = p.g + tok0 * p.H + h, *beta = p.beta + tok0 * p.H + h;
    Tout *o = static_cast<Tout *>(p.o) + (tok0 * p.H + h) * p.V + col0;
    const size_t qs = static_cast<size_t>(p.Hk) * K, vs = static_cast<size_t>(p.H) * p.V;

    auto load = [&](Token<RPL> &t, int at) {
        load_row(q + at * qs, t.q);
        load_row(k + at * qs, t.k);
        load_row(v + at * vs, t.v);
        t.g = g[static_cast<size_t>(at) * p.H];
        t.beta = beta[static_cast<size_t>(at) * p.H];
    };
    Token<RPL> now;
    if (L > 0)
        load(now, 0);
    const size_t sbase = (static_cast<size_t>(head) * K + row0) * p.V + col0;
    f32x4 S[RPL];
#pragma unroll
    for (int i = 0; i < RPL; ++i)
        S[i] = p.state_in ? *reinterpret_cast<const f32x4 *>(p.state_in + sbase + static_cast<size_t>(i) * p.V)
                          : f32x4{0.f, 0.f, 0.f, 0.f};

    for (int t = 0; t < L; ++t) {
        Token<RPL> next;
        if (t + 1 < L)
            load(next, t + 1);
        const float alpha = expf(now.g);
        f32x4 R, O;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < RPL; ++i)
                s = fmaf(now.k[i], S[i][c], s);
            R[c] = now.beta * (now.v[c] - alpha * group_sum(s));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < RPL; ++i) {
                S[i][c] = fmaf(now.k[i], R[c], alpha * S[i][c]);
                s = fmaf(now.q[i], S[i][c], s);
            }
            O[c] = p.scale * group_sum(s);
        }
        if (lane < 8)
            store4(o + t * vs, O);
        if (p.state_pos) {
            const size_t at = ((tok0 + t) * p.H + h) * K * p.V + static_cast<size_t>(row0) * p.V + col0;
#pragma unroll
            for (int i = 0; i < RPL; ++i)
                *reinterpret_cast<f32x4 *>(p.state_pos + at + static_cast<size_t>(i) * p.V) = S[i];
        }
        now = next;
    }
    if (p.state_out)
#pragma unroll
        for (int i = 0; i < RPL; ++i)
            *reinterpret_cast<f32x4 *>(p.state_out + sbase + static_cast<size_t>(i) * p.V) = S[i];
}

template <typename Tin, typename Tout>
hipError_t launch_typed(const SeqArgs &p, hipStream_t stream)
{
    const unsigned nwaves = static_cast<unsigned>(static_cast<long long>(p.B) * p.H * (p.V / CW));
    const dim3 grid((nwaves + WAVES - 1) / WAVES), block(WAVES * 64);
    if (p.K == 64)
        hipLaunchKernelGGL((gdr_step_kernel<Tin, Tout, 64>), grid, block, 0, stream, p, nwaves);
    else
        hipLaunchKernelGGL((gdr_step_kernel<Tin, Tout, 128>), grid, block, 0, stream, p, nwaves);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_step(const SeqArgs &p, hipStream_t stream)
{
    if (p.in_bf16)
        return p.o_bf16 ? launch_typed<uint16_t, uint16_t>(p, stream) : launch_typed<uint16_t, float>(p, stream);
    return p.o_bf16 ? launch_typed<float, uint16_t>(p, stream) : launch_typed<float, float>(p, stream);
}

}  // namespace gdr
