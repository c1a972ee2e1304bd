// draft.hip -- verification of drafted tokens (include/draft.h).
//
// One workgroup of 16 waves per batch row.  The drafts are tested side by side (a handful of
// gathered probabilities); then the waves sum the weights of the one vocabulary row the token
// is drawn from -- max(p - q, 0), or p -- in 64 bits, one sum for each of 64 segments of the
// row, 16 lanes a segment.  A scan over these sums (one per lane) finds the segment in which the
// running sum passes u times the total; there every lane of wave 0 sums a run of neighbouring
// tokens, a second scan finds the lane, and that lane walks its run.  The order of all sums is
// fixed.
//
// What bounds it: the one compute unit of a row.  Its two rows (0.5 MB of a 65536-token fp32
// vocabulary) come in at 64 bytes a cycle at best, 3.6 us, beside 64-bit sums of about as long,
// behind a chain of four dependent memory latencies (tokens, their probabilities, the row, the
// segment again): 9.5 us for one row, 11.7 us for 64 rows (33 MB, 2.9 TB/s).  One test for
// infinities and NaN per 16 probabilities in the place of one for each took 13.3 us to 11.8,
// the segment's wide loads 11.8 to 10.2, scans without LDS 10.2 to 9.5.
#include <type_traits>

#include "gdr_device.h"
#include "gdr_launch.h"

namespace gdr {
namespace {

constexpr int THREADS = 1024;  // 16 waves
constexpr int SEGS = 64;  // segments of a vocabulary row: a lane each in the scan
constexpr int RUN = 16;   // tokens of a lane in the last scan that are read at once

// What a probability weighs: nothing unless it is a positive finite number, whose bits are below
// infinity's.
constexpr uint32_t INFINITE = 0x7f800000u;
__device__ __forceinline__ float clean(float x) { return __float_as_uint(x) < INFINITE ? x : 0.f; }
// max(x - y, 0) in 64 bits, of such
__device__ __forceinline__ double above(float x, float y)
{
    return static_cast<double>(x) - static_cast<double>(y < x ? y : x);
}

template <typename Tin>
struct Weights {
    const Tin *p, *q;  // rows of target and draft (q may be null)
    int sure;          // the token a sure drafter holds all mass on, or -1
};

// N consecutive elements as they are.
template <typename Tin, int N>
struct Unit {
    u32x4 x;
    __device__ __forceinline__ void zero() { x = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void load(const Tin *p) { x = *reinterpret_cast<const u32x4 *>(p); }
    __device__ __forceinline__ void clear(int e)
    {
        x[N == 4 ? e : e / 2] &= N == 4 ? 0u : e & 1 ? 0xffffu : 0xffff0000u;
    }
    __device__ __forceinline__ float at(int e) const
    {
        if constexpr (N == 4)
            return __uint_as_float(x[e]);
        else
            return e & 1 ? bf16_hi(x[e / 2]) : bf16_lo(x[e / 2]);
    }
};
template <typename Tin>
struct Unit<Tin, 1> {
    float x;
    __device__ __forceinline__ void zero() { x = 0.f; }
    __device__ __forceinline__ void load(const Tin *p) { x = load_elem(p, 0); }
    __device__ __forceinline__ void clear(int) { x = 0.f; }
    __device__ __forceinline__ float at(int) const { return x; }
};

// RUN weights from x on, 0 from hi on, with all loads in flight at once.
template <typename Tin, bool WIDE>
__device__ __forceinline__ void some(const Weights<Tin> &w, size_t x, size_t hi, double (&y)[RUN])
{
    constexpr int N = WIDE ? 16 / sizeof(Tin) : 1;
    Unit<Tin, N> a[RUN / N], b[RUN / N];
#pragma unroll
    for (int i = 0; i < RUN / N; ++i) {
        a[i].zero();
        b[i].zero();
        if (x + N * i < hi) {
            a[i].load(w.p + x + N * i);
            if (w.q)
                b[i].load(w.q + x + N * i);
        }
    }
#pragma unroll
    for (int e = 0; e < RUN; ++e) {
        const float q = !w.q && static_cast<int>(x) + e == w.sure ? 1.f : b[e / N].at(e % N);
        y[e] = above(clean(a[e / N].at(e % N)), clean(q));
    }
}

// x moved along its row of 16 lanes by a DPP control; lanes that nothing reaches get 0.
template <int CTRL>
__device__ __forceinline__ double row_move(double x)
{
    const u32x2 u = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, u[0], CTRL, 0xf, 0xf, true)),
                                            static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, u[1], CTRL, 0xf, 0xf, true))});
}
__device__ __forceinline__ double read_lane(double x, int lane)
{
    const u32x2 u = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{static_cast<uint32_t>(__builtin_amdgcn_readlane(u[0], lane)),
                                            static_cast<uint32_t>(__builtin_amdgcn_readlane(u[1], lane))});
}

// Sum over a row of 16 lanes, to its first.
__device__ __forceinline__ double row_sum(double x)
{
    x += row_move<0x128>(x);  // row_ror:8, 4, 2, 1
    x += row_move<0x124>(x);
    x += row_move<0x122>(x);
    return x + row_move<0x121>(x);
}

// Sum over the lanes up to this one.
__device__ __forceinline__ double wave_scan(double x, int lane)
{
    x += row_move<0x111>(x);  // row_shr:1, 2, 4, 8
    x += row_move<0x112>(x);
    x += row_move<0x114>(x);
    x += row_move<0x118>(x);
    // the rows before this one
    const double first = read_lane(x, 15), second = first + read_lane(x, 31), third = second + read_lane(x, 47);
    return x + (lane < 16 ? 0.0 : lane < 32 ? first : lane < 48 ? second : third);
}

// This lane's share of the weights of [lo, hi), a segment that 16 lanes read: units of 16 bytes
// where rows are aligned so.
template <typename Tin, bool WIDE, bool PAIR>
__device__ __forceinline__ double share(const Weights<Tin> &w, size_t lo, size_t hi, int row)
{
    constexpr int N = WIDE ? 16 / sizeof(Tin) : 1, U = WIDE ? 16 / N : 8;  // elements of a load, loads in flight
    double sum = 0.0;
    for (size_t base = lo; base < hi; base += 16 * N * U) {
        Unit<Tin, N> p[U], q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const size_t x = base + 16 * N * u + N * row;
            p[u].zero();
            if constexpr (PAIR)
                q[u].zero();
            if (x < hi) {
                p[u].load(w.p + x);
                if constexpr (PAIR)
                    q[u].load(w.q + x);
            }
        }
        if constexpr (!PAIR)
            // the token a sure drafter holds all mass on: in one stretch of many
            if (static_cast<size_t>(w.sure) - base < 16 * N * U)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (base + 16 * N * u + N * row + e == static_cast<size_t>(w.sure)) {
                            sum += above(clean(p[u].at(e)), 1.f);
                            p[u].clear(e);
                        }
        // One test for the stretch in the place of one for each probability: the sums' vector
        // instructions are what the kernel's time is made of.
        uint32_t most = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                most = max(most, __float_as_uint(p[u].at(e)));
                if constexpr (PAIR)
                    most = max(most, __float_as_uint(q[u].at(e)));
            }
        auto add = [&](auto of) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    sum += of(p[u].at(e), PAIR ? q[u].at(e) : 0.f);
        };
        if (most < INFINITE)
            add([](float x, float y) { return PAIR ? above(x, y) : static_cast<double>(x); });
        else
            add([](float x, float y) { return above(clean(x), clean(y)); });
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
        // a wave takes four segments, 16 lanes each
        const int s = 4 * wave + (lane >> 4), row = lane & 15;
        const size_t lo = min(s * len, vocab), hi = min(lo + len, vocab);
        double sum = w.q ? share<Tin, WIDE, true>(w, lo, hi, row) : share<Tin, WIDE, false>(w, lo, hi, row);
        sum = row_sum(sum);
        if (row == 0)
            seg[s] = sum;
        __syncthreads();
        upto = wave_scan(seg[lane], lane);
        total = read_lane(upto, 63);
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
        const double before = read_lane(upto - own, s);
        // this lane's run of the segment
        const size_t run = WIDE ? (len + 511) / 512 * 8 : (len + 63) / 64;  // whole units
        const size_t end = min((s + 1) * len, vocab);
        const size_t lo = min(s * len + lane * run, end), hi = min(lo + run, end);
        double y[RUN], mine = 0.0;
        for (size_t x = lo; x < hi; x += RUN) {
            some<Tin, WIDE>(w, x, hi, y);
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
                    some<Tin, WIDE>(w, i, hi, y);
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
        drawn = __builtin_amdgcn_readlane(drawn, owner);
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
