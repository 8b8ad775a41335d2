// vla_decay.cuh -- linear attention with a decay per head, what its kernels
// share (include/vla_layer.h).
//
// Forward and gradients are one operation with its three sequences renamed:
//
//   out_i = w_in sum_{j <= i} l^(i-j) (a_i . b_j) c_j + w_st l^(i+1) S a_i,
//   S     <- l^n S + k_st sum_j l^(n-1-j) c_j b_j^T
//
// in the order of time (j <= i) or against it (j >= i, and the state is kept
// already decayed to the next token it meets, so that its weights are l^i and
// k_st l^(n-j) with i, j counted from the sequence's last token):
//
//            a    b   c   time      S starts as      ends as
//   o        q    k   v   forward   S0               S_T
//   dq       dO   v   k   forward   S0^T
//   dk       v    dO  q   backward  dS_T^T           (dS0^T)
//   dv       k    q   dO  backward  dS_T             dS0
//
// S is d x d with a row per value of c and a column per value of b.
#pragma once

#include "vla_layer.cuh"

namespace vla_layer {

constexpr int MAX_ROLES = 3;

struct Role {
    Seq a, b, c, out;
    const float* init;  // start of S per (b, h), or null for 0
    float* fin;         // end of S per (b, h), or null
    int init_t;         // init holds S^T
    int reverse;        // against the order of time
    float w_in, w_st, k_st;
    int map_a, map_b, map_c;  // of the tensor-core kernel's tensor maps
};

struct DecayArgs {
    Role role[MAX_ROLES];
    const float* log_decay;
    const int* lengths;
    vla::DeviceStatus* status;
    float* seg;    // states of segments [state role][bhs][nseg][d][d], in place of init and fin where nseg > 1
    int seg_role[MAX_ROLES];  // which of them a role starts from
    int seg_t[MAX_ROLES];     // ... transposed
    int B, H, T;
    int bh0, bhs;       // the launch's heads: [bh0, bh0 + bhs) of the B x H
    int nseg, seg_len;  // segments of the sequence and their tokens (a multiple of 64)
    unsigned long long wait_ns;
};

// Tokens [t0, t0 + n) of segment s of sequence b.
struct Span {
    int t0, n;
};
__device__ __forceinline__ int seq_len(const DecayArgs& p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}
// State of segment s of head bh for state role `role`.
__device__ __forceinline__ float* seg_of(const DecayArgs& p, int role, int bh, int s, int d) {
    return p.seg + (((size_t)role * p.bhs + (bh - p.bh0)) * p.nseg + s) * d * d;
}
__device__ __forceinline__ Span span_of(const DecayArgs& p, int b, int s) {
    const int t0 = s * p.seg_len;
    return Span{t0, max(0, min(p.seg_len, seq_len(p, b) - t0))};
}

}  // namespace vla_layer
