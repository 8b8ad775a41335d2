// vla_decay_fma.cuh -- the operation of vla_decay.cuh on the FP32 pipes, for fp32
// inputs and for the shortest bf16 calls: a block per (role, head, segment) goes through its tokens 32 at a time
// with S and the tiles of a, b, c and the decayed c in shared memory. The next
// 32 tokens' rows are on their way to registers meanwhile.
//
// Bound by shared memory: a value read there feeds 4 to 16 multiply-adds. (d =
// 64, 40 heads of up to 1,021 tokens: 63 us for the outputs' launch, of 84 us.)
//
// STATE: only the segment's own state, from zero, is formed (of b and c).
#pragma once

#include "vla_decay.cuh"

namespace vla_layer {

template <int D>
struct FmaLay {
    static constexpr int C = 32, THREADS = 256;
    static constexpr int LD = D + 4;  // row pitch: rows of a column of float4s lie in different banks
    static constexpr int PP = C + 4;  // of the pairs
    static constexpr int S = 0;
    static constexpr int A = S + D * LD, B = A + C * LD, CC = B + C * LD, CW = CC + C * LD, P = CW + C * LD;
    static constexpr int W = P + C * PP;  // weights: by lag, of the state to tokens
    static constexpr int FLOATS = W + 2 * C;
    static constexpr int SMEM = FLOATS * 4;
    static constexpr int CG = D / 4;                               // groups of four columns
    static constexpr int RG = D == 128 || D == 96 ? 8 : 1024 / D;  // row groups of the output tile
    static constexpr int RPT = C / RG;
    static constexpr int NPT = (C * (D / 8) + THREADS - 1) / THREADS;  // 8-value pieces of a tile a thread moves
};

__device__ __forceinline__ float dot4(float4 x, float4 y, float s) {
    return fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
}

// bf16 calls of up to this many tokens run here too: their rows have so few
// terms that the tensor cores' bf16 pairs do not average out and would show in
// the result. (One token, 32 heads, d = 128: 12 us against the tensor cores' 10.)
constexpr int FMA_T = 8;

template <int D, typename T, bool STATE>
__global__ void __launch_bounds__(256, 2) vla_decay_fma_kernel(const __grid_constant__ DecayArgs p) {
    using L = FmaLay<D>;
    extern __shared__ __align__(16) float fma_sm[];
    float* sm = fma_sm;
    const int tid = threadIdx.x;
    const int seg = blockIdx.x % p.nseg, bh = p.bh0 + blockIdx.x / p.nseg, b = bh / p.H, h = bh % p.H;
    const Role& r = p.role[blockIdx.y];
    const float g = p.log_decay[h];
    const Span sp = span_of(p, b, seg);
    const bool rev = r.reverse;
    float bad = 0.f;  // NaN once an output or a final state is not finite

    const int chunks = (sp.n + L::C - 1) / L::C;
    // first token (within the segment) of the m-th 32 in the role's order
    auto chunk0 = [&](int m) { return (rev ? chunks - 1 - m : m) * L::C; };
    using Raw = decltype(raw8((const T*)nullptr));
    Raw ra[L::NPT], rb[L::NPT], rc[L::NPT];
    auto fetch = [&](int m) {
        const int c0 = chunk0(m), n = min(L::C, sp.n - c0), t0 = sp.t0 + c0;
#pragma unroll
        for (int k = 0; k < L::NPT; ++k) {
            const int i = tid + k * L::THREADS, row = i / (D / 8), col = (i % (D / 8)) * 8;
            ra[k] = rb[k] = rc[k] = Raw{};
            if (row < n) {
                if (!STATE) ra[k] = raw8(row_of<T>(r.a, b, h, t0 + row) + col);
                rb[k] = raw8(row_of<T>(r.b, b, h, t0 + row) + col);
                rc[k] = raw8(row_of<T>(r.c, b, h, t0 + row) + col);
            }
        }
    };
    if (chunks > 0) fetch(0);

    const float* init = r.init ? r.init + (size_t)bh * D * D : nullptr;
    int init_t = r.init_t;
    if (p.nseg > 1) {
        init = STATE ? nullptr : seg_of(p, p.seg_role[blockIdx.y], bh, seg, D);
        init_t = p.seg_t[blockIdx.y];
    }
#pragma unroll 4
    for (int i = tid * 4; i < D * D; i += L::THREADS * 4) {
        const int x = i / D, y = i % D;
        const float4 v = init ? *reinterpret_cast<const float4*>(init + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (init_t) {
            float* to = sm + L::S + y * L::LD + x;
            to[0] = v.x, to[L::LD] = v.y, to[2 * L::LD] = v.z, to[3 * L::LD] = v.w;
        } else {
            *reinterpret_cast<float4*>(sm + L::S + x * L::LD + y) = v;
        }
    }
    if (tid < L::C) sm[L::W + tid] = r.w_in * decay_pow(g, tid);
    SlowDecay slow(g, L::C);

    for (int ci = 0; ci < chunks; ++ci) {
        const int c0 = chunk0(ci), n = min(L::C, sp.n - c0), t0 = sp.t0 + c0;
        const int n8 = (n + 7) & ~7;  // rows from n on are zero in c and the pairs
        __syncthreads();
#pragma unroll
        for (int k = 0; k < L::NPT; ++k) {
            const int i = tid + k * L::THREADS, row = i / (D / 8), col = (i % (D / 8)) * 8;
            if (row < L::C) {
                float x[8];
                if (!STATE) {
                    open8(ra[k], x);
                    store8(sm + L::A + row * L::LD + col, x);
                }
                open8(rb[k], x);
                store8(sm + L::B + row * L::LD + col, x);
                open8(rc[k], x);
                if (!STATE) store8(sm + L::CC + row * L::LD + col, x);
                // token to state
                const float w = row < n ? r.k_st * decay_pow(g, rev ? row + 1 : n - 1 - row) : 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= w;
                store8(sm + L::CW + row * L::LD + col, x);
            }
        }
        if (tid < L::C)  // state to token
            sm[L::W + L::C + tid] = tid < n ? r.w_st * decay_pow(g, rev ? n - 1 - tid : tid + 1) : 0.f;
        __syncthreads();
        if (ci + 1 < chunks) fetch(ci + 1);
        if (!STATE) {
            {
                const int i = tid / 8, j0 = tid % 8;
                float acc[4] = {};
#pragma unroll 8
                for (int k = 0; k < D; k += 4) {
                    const float4 a = *reinterpret_cast<float4*>(sm + L::A + i * L::LD + k);
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        acc[m] = dot4(a, *reinterpret_cast<float4*>(sm + L::B + (j0 + 8 * m) * L::LD + k), acc[m]);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int j = j0 + 8 * m, lag = rev ? j - i : i - j;
                    sm[L::P + i * L::PP + j] = lag >= 0 && i < n && j < n ? acc[m] * sm[L::W + max(lag, 0)] : 0.f;
                }
            }
            __syncthreads();
            if (tid < L::CG * L::RG && tid / L::CG * L::RPT < n) {
                // columns c, c + CG, ...: neighbouring lanes read neighbouring rows of S, whose pitch
                // puts them in different banks, and write neighbouring values
                const int c = tid % L::CG, i0 = (tid / L::CG) * L::RPT;
                float acc[L::RPT][4] = {};
#pragma unroll 4
                for (int k = 0; k < D; k += 4) {
                    float4 s[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) s[m] = *reinterpret_cast<float4*>(sm + L::S + (c + m * L::CG) * L::LD + k);
#pragma unroll
                    for (int i = 0; i < L::RPT; ++i) {
                        const float4 a = *reinterpret_cast<float4*>(sm + L::A + (i0 + i) * L::LD + k);
#pragma unroll
                        for (int m = 0; m < 4; ++m) acc[i][m] = dot4(a, s[m], acc[i][m]);
                    }
                }
#pragma unroll
                for (int i = 0; i < L::RPT; ++i)
#pragma unroll
                    for (int m = 0; m < 4; ++m) acc[i][m] *= sm[L::W + L::C + i0 + i];
#pragma unroll 2
                for (int j = 0; j < n8; j += 4) {
                    float v[4][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int m = 0; m < 4; ++m) v[q][m] = sm[L::CC + (j + q) * L::LD + c + m * L::CG];
#pragma unroll
                    for (int i = 0; i < L::RPT; ++i) {
                        const float4 w = *reinterpret_cast<float4*>(sm + L::P + (i0 + i) * L::PP + j);
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            acc[i][m] = fmaf(w.x, v[0][m], fmaf(w.y, v[1][m], fmaf(w.z, v[2][m], fmaf(w.w, v[3][m], acc[i][m]))));
                    }
                }
#pragma unroll
                for (int i = 0; i < L::RPT; ++i) {
                    if (i0 + i >= n) continue;
                    T* o = row_of<T>(r.out, b, h, t0 + i0 + i) + c;
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        o[m * L::CG] = (T)acc[i][m];
                        bad = fmaf(acc[i][m], 0.f, bad);
                    }
                }
            }
            __syncthreads();
        }
        const float whole = n < L::C ? decay_pow(g, n) : slow.next();
        for (int blk = tid; blk < L::CG * L::CG; blk += L::THREADS) {
            const int x = (blk / L::CG) * 4, y = (blk % L::CG) * 4;
            float acc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = *reinterpret_cast<float4*>(sm + L::S + (x + i) * L::LD + y);
                acc[i][0] = whole * v.x, acc[i][1] = whole * v.y, acc[i][2] = whole * v.z, acc[i][3] = whole * v.w;
            }
#pragma unroll 8
            for (int j = 0; j < n8; ++j) {
                const float4 cv = *reinterpret_cast<float4*>(sm + L::CW + j * L::LD + x);
                const float4 bv = *reinterpret_cast<float4*>(sm + L::B + j * L::LD + y);
                const float cw[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[i][0] = fmaf(cw[i], bv.x, acc[i][0]);
                    acc[i][1] = fmaf(cw[i], bv.y, acc[i][1]);
                    acc[i][2] = fmaf(cw[i], bv.z, acc[i][2]);
                    acc[i][3] = fmaf(cw[i], bv.w, acc[i][3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(sm + L::S + (x + i) * L::LD + y) =
                    make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        }
    }
    __syncthreads();
    // rows behind the sequence's last token
    if (!STATE) {
        const int behind = min(p.seg_len, p.T - sp.t0) - sp.n;
        const float zero[8] = {};
        for (int i = tid; i < behind * (D / 8); i += L::THREADS)
            store8(row_of<T>(r.out, b, h, sp.t0 + sp.n + i / (D / 8)) + (i % (D / 8)) * 8, zero);
    }
    float* fin = STATE ? seg_of(p, blockIdx.y, bh, seg, D)
                       : (p.nseg > 1 || !r.fin ? nullptr : r.fin + (size_t)bh * D * D);
    if (fin) {
#pragma unroll 4
        for (int i = tid * 4; i < D * D; i += L::THREADS * 4) {
            const float4 v = *reinterpret_cast<float4*>(sm + L::S + (i / D) * L::LD + i % D);
            *reinterpret_cast<float4*>(fin + i) = v;
            bad = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, fmaf(v.w, 0.f, bad))));
        }
    }
    if (bad != bad && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, sp.t0);
}

}  // namespace vla_layer
