// gdr_api.hip -- the C ABI of the gated delta rule (include/gdr.h) and of draft
// verification (include/draft.h).
//
// Every argument is validated here, before any HIP call, so each error path can be
// exercised without a GPU.  The entry points only enqueue work on the caller's stream:
// no allocation, no synchronisation, no global state.
#include <stdint.h>

#include "../../include/draft.h"
#include "../../include/gdr.h"
#include "gdr_launch.h"
#include "wkv7_launch.h"

namespace {

// Sequences shorter than this go to the step kernel in gdr_forward.
constexpr int kChainMinT = 9;

static_assert(GDR_MAX_COLUMNS / 64 * 512ll < (1ll << 32) && GDR_MAX_COLUMNS / 32 * 64ll < (1ll << 32) &&
                  GDR_MAX_BLOCKS * 512ll < (1ll << 32) &&
                  DRAFT_MAX_ROWS * 1024ll < (1ll << 32),
              "a launch must hold fewer than 2^32 threads");

// The buffers of one call: every output must lie apart from every other buffer.
struct Buffers {
    struct Item {
        uintptr_t lo, hi;
        bool out;
    } item[20];
    int n = 0;
    bool aligned = true;
    void add(const void *p, int64_t bytes, bool out, uintptr_t align = 16)
    {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (!p)
            return;
        if (lo % align)
            aligned = false;
        if (bytes > 0)
            item[n++] = Item{lo, lo + static_cast<uintptr_t>(bytes), out};
    }
    void in(const void *p, int64_t bytes, uintptr_t align = 16) { add(p, bytes, false, align); }
    void out(const void *p, int64_t bytes, uintptr_t align = 16) { add(p, bytes, true, align); }
    int check() const
    {
        if (!aligned)
            return WKV7_ERR_ALIGN;
        for (int x = 0; x < n; ++x)
            for (int y = x + 1; y < n; ++y)
                if ((item[x].out || item[y].out) && item[x].lo < item[y].hi && item[y].lo < item[x].hi)
                    return WKV7_ERR_ALIAS;
        return WKV7_OK;
    }
};

bool is_dtype(int d) { return d == WKV7_F32 || d == WKV7_BF16; }
int64_t elem(int dtype) { return dtype == WKV7_BF16 ? 2 : 4; }

int check_shape(int B, int T, int Hk, int H, int K, int V)
{
    if ((K != 64 && K != 128) || V < 64 || V % 64 != 0)
        return WKV7_ERR_UNSUPPORTED;
    if (B < 1 || T < 0 || Hk < 1 || H < 1 || H % Hk != 0 || V > GDR_MAX_V)
        return WKV7_ERR_SHAPE;
    const int64_t heads = static_cast<int64_t>(B) * H;
    if (T > GDR_MAX_T || H > GDR_MAX_ROW / (K > V ? K : V) || heads > GDR_MAX_COLUMNS / V)
        return WKV7_ERR_SHAPE;
    // B T H K V 4 bytes (the per-position states, the largest buffer) within int64
    if (T > 0 && heads > INT64_MAX / (static_cast<int64_t>(K) * V * 8) / T)
        return WKV7_ERR_SHAPE;
    return WKV7_OK;
}

// The training pair's blocks of 64 tokens.
bool blocks_ok(int B, int T, int H)
{
    const int64_t blocks = (static_cast<int64_t>(T) + gdr::kBlock - 1) / gdr::kBlock;
    return blocks == 0 || static_cast<int64_t>(B) * H <= GDR_MAX_BLOCKS / blocks;
}

struct Sizes {
    int64_t qk, v, gate, state, ckpt;  // elements
    Sizes(int B, int T, int Hk, int H, int K, int V)
    {
        const int64_t tok = static_cast<int64_t>(B) * T;
        qk = tok * Hk * K;
        v = tok * H * V;
        gate = tok * H;
        state = static_cast<int64_t>(B) * H * K * V;
        ckpt = static_cast<int64_t>((static_cast<int64_t>(T) + gdr::kBlock - 1) / gdr::kBlock) * state;
    }
};

int check_seq(const gdr::SeqArgs &a, int in_dtype, int o_dtype, bool out_optional, bool training = false)
{
    if (!is_dtype(in_dtype) || !is_dtype(o_dtype))
        return WKV7_ERR_UNSUPPORTED;
    const int st = check_shape(a.B, a.T, a.Hk, a.H, a.K, a.V);
    if (st != WKV7_OK)
        return st;
    if (training && !blocks_ok(a.B, a.T, a.H))
        return WKV7_ERR_SHAPE;
    if (!a.state_out && !(out_optional && a.state_pos && a.T > 0))
        return WKV7_ERR_NULL;
    if (a.T > 0 && (!a.q || !a.k || !a.v || !a.g || !a.beta || !a.o))
        return WKV7_ERR_NULL;
    const Sizes n(a.B, a.T, a.Hk, a.H, a.K, a.V);
    Buffers bufs;
    bufs.in(a.q, n.qk * elem(in_dtype));
    bufs.in(a.k, n.qk * elem(in_dtype));
    bufs.in(a.v, n.v * elem(in_dtype));
    bufs.in(a.g, n.gate * 4);
    bufs.in(a.beta, n.gate * 4);
    if (a.state_in != a.state_out)
        bufs.in(a.state_in, n.state * 4);
    if (a.lengths)
        bufs.in(a.lengths, static_cast<int64_t>(a.B) * 4, 4);
    bufs.out(a.o, n.v * elem(o_dtype));
    bufs.out(a.state_out, n.state * 4);
    bufs.out(a.state_pos, a.T > 0 ? n.state * a.T * 4 : 0);
    bufs.out(a.ckpt, n.ckpt * 4);
    bufs.out(a.resid, n.v * 4);
    return bufs.check();
}

gdr::SeqArgs make_args(const void *q, const void *k, const void *v, const float *g, const float *beta,
                       int in_dtype, const float *state_in, void *o, int o_dtype, float *state_out, float scale,
                       int B, int T, int Hk, int H, int K, int V)
{
    gdr::SeqArgs a = {};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.state_in = state_in; a.o = o; a.state_out = state_out;
    a.scale = scale;
    a.B = B; a.T = T; a.Hk = Hk; a.H = H; a.K = K; a.V = V;
    a.in_bf16 = in_dtype == WKV7_BF16;
    a.o_bf16 = o_dtype == WKV7_BF16;
    return a;
}

int done(hipError_t e) { return e == hipSuccess ? WKV7_OK : WKV7_ERR_HIP; }

// A call without tokens: the state passes through.
int pass_through(const float *src, float *dst, int64_t n, hipStream_t s)
{
    return src == dst ? WKV7_OK : done(wkv7::launch_state_copy(src, dst, n, s));
}

}  // namespace

extern "C" {

int gdr_forward(const void *q, const void *k, const void *v, const float *g, const float *beta, int in_dtype,
                const float *state_in, void *o, int o_dtype, float *state_out, const int *lengths, float scale,
                int B, int T, int Hk, int H, int K, int V, void *stream)
{
    gdr::SeqArgs a = make_args(q, k, v, g, beta, in_dtype, state_in, o, o_dtype, state_out, scale, B, T, Hk, H, K, V);
    a.lengths = lengths;
    const int st = check_seq(a, in_dtype, o_dtype, false);
    if (st != WKV7_OK)
        return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0)
        return pass_through(state_in, state_out, Sizes(B, T, Hk, H, K, V).state, s);
    return done(T < kChainMinT ? gdr::launch_step(a, s) : gdr::launch_chain(a, s));
}

int gdr_step(const void *q, const void *k, const void *v, const float *g, const float *beta, int in_dtype,
             const float *state_in, void *o, int o_dtype, float *state_out, float *state_pos, float scale,
             int B, int T, int Hk, int H, int K, int V, void *stream)
{
    gdr::SeqArgs a = make_args(q, k, v, g, beta, in_dtype, state_in, o, o_dtype, state_out, scale, B, T, Hk, H, K, V);
    a.state_pos = state_pos;
    const int st = check_seq(a, in_dtype, o_dtype, true);
    if (st != WKV7_OK)
        return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0)
        return pass_through(state_in, state_out, Sizes(B, T, Hk, H, K, V).state, s);
    return done(gdr::launch_step(a, s));
}

int gdr_forward_ckpt(const void *q, const void *k, const void *v, const float *g, const float *beta, int in_dtype,
                     const float *state_in, float *o, float *state_out, float *ckpt, float *resid, float scale,
                     int B, int T, int Hk, int H, int K, int V, void *stream)
{
    gdr::SeqArgs a = make_args(q, k, v, g, beta, in_dtype, state_in, o, WKV7_F32, state_out, scale, B, T, Hk, H, K, V);
    a.ckpt = ckpt;
    a.resid = resid;
    const int st = check_seq(a, in_dtype, WKV7_F32, false, true);
    if (st != WKV7_OK)
        return st;
    if (T > 0 && (!ckpt || !resid))
        return WKV7_ERR_NULL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0)
        return pass_through(state_in, state_out, Sizes(B, T, Hk, H, K, V).state, s);
    return done(gdr::launch_chain(a, s));
}

int gdr_backward_ckpt(const void *q, const void *k, const float *g, const float *beta, int in_dtype,
                      const float *ckpt, const float *resid, const float *d_o, const float *d_state_out,
                      float *dq, float *dk, float *dv, float *dg, float *dbeta, float *d_state_in, float *work,
                      float scale, int B, int T, int Hk, int H, int K, int V, void *stream)
{
    if (!is_dtype(in_dtype))
        return WKV7_ERR_UNSUPPORTED;
    int st = check_shape(B, T, Hk, H, K, V);
    if (st != WKV7_OK)
        return st;
    if (!blocks_ok(B, T, H))
        return WKV7_ERR_SHAPE;
    if (!d_state_in)
        return WKV7_ERR_NULL;
    if (T > 0 && (!q || !k || !g || !beta || !ckpt || !resid || !d_o || !dq || !dk || !dv || !dg || !dbeta || !work))
        return WKV7_ERR_NULL;
    const Sizes n(B, T, Hk, H, K, V);
    Buffers bufs;
    bufs.in(q, n.qk * elem(in_dtype));
    bufs.in(k, n.qk * elem(in_dtype));
    bufs.in(g, n.gate * 4);
    bufs.in(beta, n.gate * 4);
    bufs.in(ckpt, n.ckpt * 4);
    bufs.in(resid, n.v * 4);
    bufs.in(d_o, n.v * 4);
    if (d_state_out != d_state_in)
        bufs.in(d_state_out, n.state * 4);
    bufs.out(dq, n.qk * 4);
    bufs.out(dk, n.qk * 4);
    bufs.out(dv, n.v * 4);
    bufs.out(dg, n.gate * 4);
    bufs.out(dbeta, n.gate * 4);
    bufs.out(d_state_in, n.state * 4);
    bufs.out(work, n.ckpt * 4);
    st = bufs.check();
    if (st != WKV7_OK)
        return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0)
        return pass_through(d_state_out, d_state_in, n.state, s);
    gdr::BwdArgs a = {};
    a.q = q; a.k = k; a.g = g; a.beta = beta; a.ckpt = ckpt; a.resid = resid; a.d_o = d_o;
    a.d_state_out = d_state_out;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.d_state_in = d_state_in; a.work = work;
    a.scale = scale;
    a.B = B; a.T = T; a.Hk = Hk; a.H = H; a.K = K; a.V = V;
    a.in_bf16 = in_dtype == WKV7_BF16;
    return done(gdr::launch_backward(a, s));
}

int draft_verify(const void *target, const void *draft, int dtype, const int *tokens, const int *n_draft,
                 const float *u, const float *u_draw, int *out, int *kept, int B, int N, int vocab, void *stream)
{
    if (!is_dtype(dtype))
        return WKV7_ERR_UNSUPPORTED;
    if (B < 1 || B > DRAFT_MAX_ROWS || N < 0 || N > DRAFT_MAX_DRAFTS || vocab < 1 || vocab > DRAFT_MAX_VOCAB)
        return WKV7_ERR_SHAPE;
    if (!target || !u_draw || !out || !kept || (N > 0 && (!tokens || !u)))
        return WKV7_ERR_NULL;
    const int64_t rows = static_cast<int64_t>(B) * N;
    Buffers bufs;
    bufs.in(target, (rows + B) * vocab * elem(dtype));
    bufs.in(draft, rows * vocab * elem(dtype));
    bufs.in(tokens, rows * 4, 4);
    bufs.in(n_draft, static_cast<int64_t>(B) * 4, 4);
    bufs.in(u, rows * 4, 4);
    bufs.in(u_draw, static_cast<int64_t>(B) * 4, 4);
    bufs.out(out, (rows + B) * 4, 4);
    bufs.out(kept, static_cast<int64_t>(B) * 4, 4);
    const int st = bufs.check();
    if (st != WKV7_OK)
        return st;
    gdr::DraftArgs a = {};
    a.target = target; a.draft = draft; a.tokens = tokens; a.n_draft = n_draft; a.u = u; a.u_draw = u_draw;
    a.out = out; a.kept = kept;
    a.B = B; a.N = N; a.vocab = vocab;
    a.bf16 = dtype == WKV7_BF16;
    return done(gdr::launch_draft(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
