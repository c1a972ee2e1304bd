// Drives csrc/gdr_api.hip (built for the host with sanitizers, against the stubs below)
// through accepted and refused calls, sizes up to INT_MAX included.  Pointers are never
// dereferenced by the layer under test, so made-up addresses do.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "../../include/draft.h"
#include "../../include/gdr.h"
#include "../../rwkv_linear_attention_amd/csrc/gdr_launch.h"
#include "../../rwkv_linear_attention_amd/csrc/wkv7_launch.h"

static const char *last = "none";

namespace gdr {
hipError_t launch_step(const SeqArgs &, hipStream_t) { last = "step"; return hipSuccess; }
hipError_t launch_chain(const SeqArgs &, hipStream_t) { last = "chain"; return hipSuccess; }
hipError_t launch_backward(const BwdArgs &, hipStream_t) { last = "backward"; return hipSuccess; }
hipError_t launch_draft(const DraftArgs &, hipStream_t) { last = "draft"; return hipErrorInvalidValue; }
}  // namespace gdr
namespace wkv7 {
hipError_t launch_state_copy(const float *, float *, long long n, hipStream_t)
{
    last = "copy";
    return n > 0 ? hipSuccess : hipErrorInvalidValue;
}
}  // namespace wkv7

template <typename T = float>
static T *at(int i) { return reinterpret_cast<T *>((static_cast<uintptr_t>(1) << 50) + (static_cast<uintptr_t>(i) << 40)); }

static int fails = 0;
static void want(const char *what, int got, int status, const char *launch)
{
    bool ok = got == status;
    for (const char *x = last, *y = launch; ok && (*x || *y); ++x, ++y)
        ok = *x == *y;
    if (!ok) {
        std::printf("%s: status %d (want %d), launch %s (want %s)\n", what, got, status, last, launch);
        ++fails;
    }
    last = "none";
}

static int fwd(int B, int T, int Hk, int H, int K, int V)
{
    return gdr_forward(at(0), at(1), at(2), at(3), at(4), WKV7_BF16, at(5), at(6), WKV7_F32, at(7), nullptr, 1.f, B, T,
                       Hk, H, K, V, nullptr);
}
static int train(int B, int T, int Hk, int H, int K, int V)
{
    return gdr_forward_ckpt(at(0), at(1), at(2), at(3), at(4), WKV7_BF16, at(5), at(6), at(7), at(8), at(9), 1.f, B, T,
                            Hk, H, K, V, nullptr);
}
static int back(int B, int T, int Hk, int H, int K, int V)
{
    return gdr_backward_ckpt(at(0), at(1), at(2), at(3), WKV7_BF16, at(4), at(5), at(6), at(7), at(8), at(9), at(10),
                             at(11), at(12), at(13), at(14), 1.f, B, T, Hk, H, K, V, nullptr);
}
static int step(int B, int T, int Hk, int H, int K, int V, float *out, float *pos)
{
    return gdr_step(at(0), at(1), at(2), at(3), at(4), WKV7_F32, nullptr, at(6), WKV7_BF16, out, pos, 1.f, B, T, Hk, H,
                    K, V, nullptr);
}
static int draft(int B, int N, int vocab)
{
    return draft_verify(at(0), at(1), WKV7_F32, at<int>(2), at<int>(3), at(4), at(5), at<int>(6), at<int>(7), B, N, vocab,
                        nullptr);
}

int main()
{
    want("8 tokens", fwd(2, 8, 2, 4, 64, 64), WKV7_OK, "step");
    want("9 tokens", fwd(2, 9, 2, 4, 128, 512), WKV7_OK, "chain");
    want("no tokens", fwd(2, 0, 2, 4, 64, 64), WKV7_OK, "copy");
    want("step", step(1, 1, 1, 1, 64, 64, at(7), nullptr), WKV7_OK, "step");
    want("step states only", step(1, 5, 1, 1, 64, 64, nullptr, at(8)), WKV7_OK, "step");
    want("step nothing", step(1, 5, 1, 1, 64, 64, nullptr, nullptr), WKV7_ERR_NULL, "none");
    want("train", train(1, 1, 1, 1, 64, 64), WKV7_OK, "chain");
    want("train no tokens", train(1, 0, 1, 1, 64, 64), WKV7_OK, "copy");
    want("back", back(1, 100, 1, 1, 64, 64), WKV7_OK, "backward");
    want("back no tokens", back(1, 0, 1, 1, 64, 64), WKV7_OK, "copy");
    want("draft (launch refused)", draft(1, 3, 100), WKV7_ERR_HIP, "draft");
    const int sizes[] = {INT_MIN, -1, 0, 1, 63, 64, 128, 1 << 16, 1 << 24, 1 << 30, INT_MAX};
    for (int B : sizes)
        for (int T : sizes)
            for (int H : sizes)
                for (int V : sizes) {
                    for (int got : {fwd(B, T, H, H, 128, V), train(B, T, 1, H, 64, V), back(B, T, H, H, 64, V),
                                    step(B, T, 1, H, 128, V, at(7), at(8)), fwd(B, T, H, H, V, 64), draft(B, T, V)})
                        if (got > 0 || got < WKV7_ERR_HIP) {
                            std::printf("unknown status %d\n", got);
                            ++fails;
                        }
                }
    std::printf("%d failures\n", fails);
    return fails != 0;
}
