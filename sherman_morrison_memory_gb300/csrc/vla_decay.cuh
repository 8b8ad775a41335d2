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
    int stall;          // testing: the last chunk's loads are kept back
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

// Start of a role's S (null for 0; `init_t`: transposed) and where its end goes (or null).
template <int D, bool STATE>
__device__ __forceinline__ const float* start_of(const DecayArgs& p, int role, int bh, int seg, int& init_t) {
    const Role& r = p.role[role];
    init_t = p.nseg > 1 ? p.seg_t[role] : r.init_t;
    if (p.nseg > 1) return STATE ? nullptr : seg_of(p, p.seg_role[role], bh, seg, D);
    return r.init ? r.init + (size_t)bh * D * D : nullptr;
}
template <int D, bool STATE>
__device__ __forceinline__ float* end_of(const DecayArgs& p, int role, int bh, int seg) {
    if (STATE) return seg_of(p, role, bh, seg, D);
    return p.nseg > 1 || !p.role[role].fin ? nullptr : p.role[role].fin + (size_t)bh * D * D;
}

// Whether the powers of a growing head's factor over a chunk of C tokens are too
// large to be formed apart from what they multiply (2^64, half of the exponent's
// range): a block then goes token by token.
__device__ __forceinline__ bool outgrows(float g, int C) { return g * (float)C > 44.f; }

// A block whose outputs are not all finite asks whether they are that before their
// time: a chunk's pairs, zero above the diagonal, carry an Inf or NaN in c to the
// tokens that come before it in its chunk of C (zero times Inf). True if a
// column's first such value has any. `first`: D ints of shared memory.
template <int D, typename T, int THREADS, int C>
__device__ __forceinline__ bool seen_too_early(const DecayArgs& p, const Role& r, int b, int h, const Span sp, int* first) {
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += THREADS) first[i] = sp.n;
    __syncthreads();
    for (int i = threadIdx.x; i < sp.n * (D / 8); i += THREADS) {
        const int j = i / (D / 8), col = i % (D / 8) * 8;
        float v[8];
        load8(row_of<T>(r.c, b, h, sp.t0 + j) + col, v);
        for (int e = 0; e < 8; ++e)
            if (!(fabsf(v[e]) < __int_as_float(0x7F800000))) atomicMin(first + col + e, r.reverse ? sp.n - 1 - j : j);
    }
    __syncthreads();
    bool early = false;
    for (int i = threadIdx.x; i < D; i += THREADS) {
        // against time a segment's first chunk in order is the one that may be shorter
        const int f = first[i], head = r.reverse ? (sp.n - 1) % C + 1 : C;
        early |= f < sp.n && (f < head ? f > 0 : (f - head) % C != 0);
    }
    return __syncthreads_or(early);
}

// The operation a token at a time, as the recurrence has it:
//   S <- l S + k_st c b^T,  out = w_st S a        (in the order of time)
//   S <- S + k_st c b^T,  out = w_st S a,  S <- l S   (against it)
// for the tokens of a block whose chunks cannot give it (seen_too_early(), outgrows()). S is in
// shared memory, with LN lanes a row, which nobody else reads; tokens come in 8 at a
// time. (152 heads of 4,096 tokens, d = 128, an Inf in the middle of each: 6.6 ms, 0.15 without.)
template <int D, typename T, int THREADS, bool STATE>
__device__ __noinline__ void by_token(const DecayArgs& p, int role, int bh, int seg, float* sm) {
    constexpr int LN = THREADS >= 4 * D ? 4 : 2, LD = D + 4, TOK = 8;
    static_assert(THREADS >= LN * D && LN * D % 32 == 0, "whole warps of rows");
    float *S = sm, *rows = sm + D * LD;  // [D][LD] and a, b, c of TOK tokens, D * LD + 3 * TOK * D floats
    const Role& r = p.role[role];
    const int tid = threadIdx.x, lane = tid % LN, x = tid / LN, b = bh / p.H, h = bh % p.H;
    const bool rev = r.reverse;
    const float g = p.log_decay[h];
    const Span sp = span_of(p, b, seg);
    int init_t;
    const float* init = start_of<D, STATE>(p, role, bh, seg, init_t);
    if (x < D)
        for (int y = lane; y < D; y += LN) S[x * LD + y] = !init ? 0.f : init_t ? init[y * D + x] : init[x * D + y];
    float bad = 0.f;
    SlowDecay slow(g, 1);
    const bool steep = g > 1.f;  // roundings that add up matter for a slow decay alone
    const float once = expf(g);
    for (int m = 0; m < sp.n; m += TOK) {
        const int k = min(TOK, sp.n - m);
        auto token = [&](int j) { return sp.t0 + (rev ? sp.n - 1 - (m + j) : m + j); };
        __syncthreads();
        for (int i = tid; i < 3 * TOK * (D / 8); i += THREADS) {
            const int q = i / (TOK * (D / 8)), j = i / (D / 8) % TOK, col = i % (D / 8) * 8;
            if (j >= k || (STATE && q == 0)) continue;
            float v[8];
            load8(row_of<T>(q == 0 ? r.a : q == 1 ? r.b : r.c, b, h, token(j)) + col, v);
            store8(rows + (q * TOK + j) * D + col, v);
        }
        __syncthreads();
        if (x >= D) continue;
        for (int j = 0; j < k; ++j) {
            const float l = steep ? once : slow.next(), c = r.k_st * rows[(2 * TOK + j) * D + x];
            const float *av = rows + j * D, *bv = rows + (TOK + j) * D;
            float acc = 0.f;
            for (int y = lane; y < D; y += LN) {
                const float s = fmaf(c, bv[y], rev ? S[x * LD + y] : l * S[x * LD + y]);
                if (!STATE) acc = fmaf(s, av[y], acc);
                S[x * LD + y] = rev ? l * s : s;
            }
            if constexpr (!STATE) {
#pragma unroll
                for (int i = 1; i < LN; i <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, i);
                acc *= r.w_st;
                bad = fmaf(acc, 0.f, bad);
                if (lane == 0) row_of<T>(r.out, b, h, token(j))[x] = (T)acc;
            }
        }
    }
    if (!STATE) {  // rows behind the sequence's last token
        const int behind = min(p.seg_len, p.T - sp.t0) - sp.n;
        const float zero[8] = {};
        for (int i = tid; i < behind * (D / 8); i += THREADS)
            store8(row_of<T>(r.out, b, h, sp.t0 + sp.n + i / (D / 8)) + (i % (D / 8)) * 8, zero);
    }
    float* fin = end_of<D, STATE>(p, role, bh, seg);
    if (fin && x < D)
        for (int y = lane; y < D; y += LN) {
            fin[x * D + y] = S[x * LD + y];
            bad = fmaf(S[x * LD + y], 0.f, bad);
        }
    if (bad != bad && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, sp.t0);
}

}  // namespace vla_layer
