// draft.hip -- verification of drafted tokens (include/draft.h).
//
// One workgroup of 16 waves per batch row.  The drafts are tested side by side (a handful of
// gathered probabilities); then the waves sum the weights of the one vocabulary row the token
// is drawn from -- max(p - q, 0), or p -- in 64 bits, one sum for each of 64 segments of the
// row.  A scan over these sums (one per lane) finds the segment in which the running sum passes
// u times the total; there every lane of wave 0 sums a run of neighbouring tokens, a second scan
// finds the lane, and that lane walks its run.  The order of all sums is fixed.
//
// What bounds it: one compute unit reads the two rows, 64 bytes a cycle at best (0.5 MB of a
// 65536-token fp32 vocabulary in 3.6 us), behind a chain of four dependent memory latencies
// (tokens, their probabilities, the row, the segment again): 13.2 us for one row of 65536 fp32
// tokens, 16.4 us for 64 rows (33 MB, 2.0 TB/s).
#include <type_traits>

#include "gdr_device.h"
#include "gdr_launch.h"

namespace gdr {
namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr int SEGS = 64;  // segments of a vocabulary row: a lane each in the scan
constexpr int RUN = 16;   // tokens of a lane in the last scan that are read at once

// What a probability weighs: nothing unless it is a positive finite number.
__device__ __forceinline__ float clean(float x) { return x > 0.f && x < __builtin_huge_valf() ? x : 0.f; }

template <typename Tin>
struct Weights {
    const Tin *p, *q;  // rows of target and draft (q may be null)
    int sure;          // the token a sure drafter holds all mass on, or -1
    __device__ static double of(float p, float q)
    {
        const float x = clean(p), y = clean(q);
        return x > y ? static_cast<double>(x) - static_cast<double>(y) : 0.0;
    }
    // RUN weights from x on, 0 from hi on, with all loads in flight at once
    __device__ void some(size_t x, size_t hi, double (&y)[RUN]) const
    {
        float a[RUN], b[RUN];
#pragma unroll
        for (int e = 0; e < RUN; ++e) {
            a[e] = b[e] = 0.f;
            if (x + e < hi) {
                a[e] = load_elem(p, x + e);
                if (q)
                    b[e] = load_elem(q, x + e);
                else
                    b[e] = static_cast<int>(x) + e == sure ? 1.f : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < RUN; ++e)
            y[e] = of(a[e], b[e]);
    }
};

// Sum over the lanes up to this one.
__device__ __forceinline__ double wave_scan(double x, int lane)
{
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const double y = __shfl_up(x, off);
        if (lane >= off)
            x += y;
    }
    return x;
}

// This lane's share of the weights of [lo, hi): units of 16 bytes where rows are aligned so.
template <typename Tin, bool WIDE, bool PAIR>
__device__ __forceinline__ double share(const Weights<Tin> &w, size_t lo, size_t hi, int lane)
{
    constexpr int N = WIDE ? 16 / sizeof(Tin) : 1, U = WIDE ? 16 / N : 8;  // elements of a load, loads in flight
    double sum = 0.0;
    for (size_t base = lo; base < hi; base += 64 * N * U) {
        float p[U][N], q[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const size_t x = base + 64 * N * u + N * lane;
#pragma unroll
            for (int e = 0; e < N; ++e)
                p[u][e] = q[u][e] = 0.f;
            if (x < hi) {
                if constexpr (WIDE) {
                    load_row(w.p + x, p[u]);
                    if constexpr (PAIR)
                        load_row(w.q + x, q[u]);
                } else {
                    p[u][0] = load_elem(w.p, x);
                    if constexpr (PAIR)
                        q[u][0] = load_elem(w.q, x);
                }
                if constexpr (!PAIR)
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        q[u][e] = static_cast<int>(x) + e == w.sure ? 1.f : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < N; ++e)
                sum += Weights<Tin>::of(p[u][e], q[u][e]);
    }
    return sum;
}

template <typename Tin, bool WIDE>
__global__ __launch_bounds__(THREADS) void draft_verify_kernel(DraftArgs a)
{
    __shared__ double seg[SEGS];
    __shared__ int first_refused;
    const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const size_t vocab = a.vocab;
    const Tin *target = static_cast<const Tin *>(a.target) + static_cast<size_t>(b) * (a.N + 1) * vocab;
    const Tin *draft = a.draft ? static_cast<const Tin *>(a.draft) + static_cast<size_t>(b) * a.N * vocab : nullptr;
    const int *tokens = a.tokens + static_cast<size_t>(b) * a.N;
    const int given = a.n_draft ? min(max(a.n_draft[b], 0), a.N) : a.N;

    if (threadIdx.x == 0)
        first_refused = given;
    __syncthreads();
    for (int j = threadIdx.x; j < a.N; j += THREADS) {
        const int x = tokens[j];
        bool ok = x >= 0 && x < a.vocab;
        if (ok) {
            const double p = clean(load_elem(target, j * vocab + x));
            const double q = draft ? clean(load_elem(draft, j * vocab + x)) : 1.f;
            ok = static_cast<double>(a.u[static_cast<size_t>(b) * a.N + j]) * q < p;
        }
        if (!ok && j < given)
            atomicMin(&first_refused, j);
    }
    __syncthreads();
    const int n = first_refused;

    Weights<Tin> w = {target + n * vocab, nullptr, -1};
    if (n < given) {
        if (draft)
            w.q = draft + n * vocab;
        else
            w.sure = tokens[n];
    }
    // tokens of a segment: whole 16-byte units
    const size_t len = ((vocab + SEGS - 1) / SEGS + 7) / 8 * 8;
    double upto, total;
    for (;;) {
        double sum[SEGS / WAVES];
#pragma unroll
        for (int i = 0; i < SEGS / WAVES; ++i) {
            const size_t lo = min((wave + WAVES * i) * len, vocab), hi = min(lo + len, vocab);
            sum[i] = w.q ? share<Tin, WIDE, true>(w, lo, hi, lane) : share<Tin, WIDE, false>(w, lo, hi, lane);
        }
#pragma unroll
        for (int off = 32; off; off >>= 1)
#pragma unroll
            for (int i = 0; i < SEGS / WAVES; ++i)
                sum[i] += __shfl_xor(sum[i], off);
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < SEGS / WAVES; ++i)
                seg[wave + WAVES * i] = sum[i];
        __syncthreads();
        upto = wave_scan(seg[lane], lane);
        total = __shfl(upto, 63);
        if (total > 0.0 || (!w.q && w.sure < 0))
            break;
        w.q = nullptr;  // nothing left of max(p - q, 0): p itself
        w.sure = -1;
        __syncthreads();
    }
    if (wave != 0)
        return;

    int drawn = -1;
    if (total > 0.0) {
        const double mark = static_cast<double>(a.u_draw[b]) * total, own = seg[lane];
        // the first segment whose running sum passes the mark, or the last with any weight
        unsigned long long any = __ballot(own > 0.0), past = __ballot(own > 0.0 && upto > mark);
        const int s = past ? __ffsll(past) - 1 : 63 - __clzll(any);
        const double before = __shfl(upto - own, s);
        // this lane's run of the segment
        const size_t run = len / 64 + (len % 64 != 0), end = min((s + 1) * len, vocab);
        const size_t lo = min(s * len + lane * run, end), hi = min(lo + run, end);
        double y[RUN], mine = 0.0;
        for (size_t x = lo; x < hi; x += RUN) {
            w.some(x, hi, y);
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                mine += y[e];
        }
        const double sum = before + wave_scan(mine, lane);
        any = __ballot(mine > 0.0);
        past = __ballot(mine > 0.0 && sum > mark);
        const int owner = past ? __ffsll(past) - 1 : 63 - __clzll(any);
        if (lane == owner) {
            double x = sum - mine;
            bool found = false;
            for (size_t i = lo; i < hi && !found; i += RUN) {
                if (hi - lo > RUN)
                    w.some(i, hi, y);
#pragma unroll
                for (int e = 0; e < RUN; ++e) {
                    x += y[e];
                    if (y[e] > 0.0 && !found) {
                        drawn = static_cast<int>(i) + e;
                        found = x > mark;
                    }
                }
            }
        }
        drawn = __shfl(drawn, owner);
    }
    int *out = a.out + static_cast<size_t>(b) * (a.N + 1);
    for (int j = lane; j <= a.N; j += 64)
        out[j] = j < n ? tokens[j] : j == n ? drawn : -1;
    if (lane == 0)
        a.kept[b] = n + 1;
}

template <typename Tin>
hipError_t launch_typed(const DraftArgs &a, hipStream_t stream)
{
    if (a.vocab % (16 / static_cast<int>(sizeof(Tin))) == 0)
        hipLaunchKernelGGL((draft_verify_kernel<Tin, true>), dim3(a.B), dim3(THREADS), 0, stream, a);
    else
        hipLaunchKernelGGL((draft_verify_kernel<Tin, false>), dim3(a.B), dim3(THREADS), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_draft(const DraftArgs &a, hipStream_t stream)
{
    return a.bf16 ? launch_typed<uint16_t>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace gdr
