// draft.hip -- verification of drafted tokens (include/draft.h).
//
// One workgroup per batch row.  Wave 0 tests the drafts (a handful of gathered
// probabilities), then all waves sum the weights of the one vocabulary row the token
// is drawn from -- max(p - q, 0), or p -- in 64 bits: SEGS segments of the row, one
// sum each in LDS.  A scan of these finds the segment in which the running sum passes
// u times the total; the wave that owns it walks it again, 64 tokens at a time.
#include "gdr_device.h"
#include "gdr_launch.h"

namespace gdr {
namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr int SEGS = 64;  // segments of a vocabulary row

// What a probability weighs: nothing unless it is a positive finite number.
__device__ __forceinline__ float clean(float x) { return x > 0.f && x < __builtin_huge_valf() ? x : 0.f; }

struct Weights {
    const void *p, *q;  // rows of target and draft (q may be null)
    int sure;           // the token a sure drafter holds all mass on, or -1
};

template <typename Tin>
__device__ __forceinline__ double weight(const Weights &w, size_t x)
{
    const double p = clean(load_elem(static_cast<const Tin *>(w.p), x));
    double q = 0.0;
    if (w.q)
        q = clean(load_elem(static_cast<const Tin *>(w.q), x));
    else if (static_cast<int>(x) == w.sure)
        q = 1.0;
    return p > q ? p - q : 0.0;
}

__device__ __forceinline__ double wave_sum(double x)
{
#pragma unroll
    for (int off = 32; off; off >>= 1)
        x += __shfl_xor(x, off);
    return x;
}

template <typename Tin>
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
    for (int j = threadIdx.x; j < given; j += THREADS) {
        const int x = tokens[j];
        bool ok = x >= 0 && x < a.vocab;
        if (ok) {
            const double p = clean(load_elem(target, j * vocab + x));
            const double q = draft ? clean(load_elem(draft, j * vocab + x)) : 1.f;
            ok = static_cast<double>(a.u[static_cast<size_t>(b) * a.N + j]) * q < p;
        }
        if (!ok)
            atomicMin(&first_refused, j);
    }
    __syncthreads();
    const int n = first_refused;

    Weights w = {target + n * vocab, nullptr, -1};
    if (n < given) {
        if (draft)
            w.q = draft + n * vocab;
        else
            w.sure = tokens[n];
    }
    const size_t len = (vocab + SEGS - 1) / SEGS;  // tokens of a segment
    double total = 0.0;
    for (;;) {
        for (int s = wave; s < SEGS; s += WAVES) {
            const size_t lo = s * len, hi = min(lo + len, vocab);
            double sum = 0.0;
            for (size_t x = lo + lane; x < hi; x += 64)
                sum += weight<Tin>(w, x);
            sum = wave_sum(sum);
            if (lane == 0)
                seg[s] = sum;
        }
        __syncthreads();
        total = 0.0;
        for (int s = 0; s < SEGS; ++s)
            total += seg[s];
        if (total > 0.0 || (!w.q && w.sure < 0))
            break;
        w.q = nullptr;  // nothing left of max(p - q, 0): p itself
        w.sure = -1;
        __syncthreads();
    }

    int drawn = -1;
    if (wave == 0 && total > 0.0) {
        // The first segment whose running sum passes the mark, or the last with any weight.
        const double mark = static_cast<double>(a.u_draw[b]) * total;
        double before = 0.0, run = 0.0;
        int at = -1;
        for (int s = 0; s < SEGS; ++s) {
            if (seg[s] > 0.0) {
                at = s;
                before = run;
                run += seg[s];
                if (run > mark)
                    break;
            }
        }
        const size_t lo = at * len, hi = min(lo + len, vocab);
        run = before;
        for (size_t base = lo; base < hi; base += 64) {
            const size_t x = base + lane;
            const double own = x < hi ? weight<Tin>(w, x) : 0.0;
            double upto = own;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const double y = __shfl_up(upto, off);
                if (lane >= off)
                    upto += y;
            }
            const unsigned long long past = __ballot(own > 0.0 && run + upto > mark), any = __ballot(own > 0.0);
            if (any)
                drawn = static_cast<int>(base) + 63 - __clzll(any);
            if (past) {
                drawn = static_cast<int>(base) + __ffsll(past) - 1;
                break;
            }
            run += __shfl(upto, 63);
        }
    }
    int *out = a.out + static_cast<size_t>(b) * (a.N + 1);
    drawn = __shfl(drawn, 0);
    if (wave == 0) {
        for (int j = lane; j <= a.N; j += 64)
            out[j] = j < n ? tokens[j] : j == n ? drawn : -1;
        if (lane == 0)
            a.kept[b] = n + 1;
    }
}

}  // namespace

hipError_t launch_draft(const DraftArgs &a, hipStream_t stream)
{
    if (a.bf16)
        hipLaunchKernelGGL(draft_verify_kernel<uint16_t>, dim3(a.B), dim3(THREADS), 0, stream, a);
    else
        hipLaunchKernelGGL(draft_verify_kernel<float>, dim3(a.B), dim3(THREADS), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdr
