// gdr_launch.h -- internal launch entry points of the gated delta rule and of draft
// verification.  Arguments are validated by gdr_api.hip before these run.
#pragma once

#include <hip/hip_runtime.h>

namespace gdr {

constexpr int kBlock = 64;  // tokens between two checkpoints

struct SeqArgs {
    const void *q, *k, *v;     // [B,T,Hk,K], [B,T,Hk,K], [B,T,H,V], in_dtype
    const float *g, *beta;     // [B,T,H]
    const float *state_in;     // [B,H,K,V] or nullptr (zeros)
    void *o;                   // [B,T,H,V], o_dtype
    float *state_out;          // [B,H,K,V] or nullptr (step with state_pos)
    float *state_pos;          // [B,T,H,K,V] or nullptr
    float *ckpt;               // [B,ceil(T/64),H,K*V] or nullptr
    float *resid;              // [B,T,H,V] with ckpt
    const int *lengths;        // [B] or nullptr
    float scale;
    int B, T, Hk, H, K, V;
    int in_bf16, o_bf16;
};

struct BwdArgs {
    const void *q, *k;         // [B,T,Hk,K], in_dtype
    const float *g, *beta;     // [B,T,H]
    const float *ckpt, *resid; // as gdr_forward_ckpt wrote them
    const float *d_o;          // [B,T,H,V]
    const float *d_state_out;  // [B,H,K,V] or nullptr (zeros)
    float *dq, *dk;            // [B,T,Hk,K]
    float *dv;                 // [B,T,H,V]
    float *dg, *dbeta;         // [B,T,H]
    float *d_state_in;         // [B,H,K,V]
    float *work;               // [B,ceil(T/64),H,K*V]
    float scale;
    int B, T, Hk, H, K, V;
    int in_bf16;
};

struct DraftArgs {
    const void *target, *draft;
    const int *tokens, *n_draft;
    const float *u, *u_draw;
    int *out, *kept;
    int B, N, vocab;
    int bf16;
};

hipError_t launch_step(const SeqArgs &a, hipStream_t stream);
hipError_t launch_chain(const SeqArgs &a, hipStream_t stream);
hipError_t launch_backward_chain(const BwdArgs &a, hipStream_t stream);
hipError_t launch_backward(const BwdArgs &a, hipStream_t stream);
hipError_t launch_draft(const DraftArgs &a, hipStream_t stream);

}  // namespace gdr
