// vla_decay_fma.cuh -- the operation of vla_decay.cuh on the FP32 pipes, for fp32
// inputs and for bf16 calls of a few tokens: a block per (role, head, segment) goes
// through its tokens 32 at a time with S and the tiles of a, b, c and the decayed c
// in shared memory. The next 32 tokens' rows are on their way to registers meanwhile.
//
// Bound by shared memory: its pipe gives a warp one value a lane a cycle, against
// four multiply-adds, so a thread's tiles are as large as its registers allow: of S
// 8 x 8 at d = 128, 6 x 6 at 96, 4 x 4 at 64, of the output 4 rows of d/32 columns.
// (fp32, 4 x 16 heads of 4,096 tokens: d = 128 966 us, 1,139 with half as large
// tiles; d = 64 343 against 399; gradients of d = 128 2,090 against 3,210.) At d =
// 32 two warps a block give a thread four times as much of each tile (4 x 32 heads:
// 220 us, 355 with eight); at d = 64 they leave too few warps an SM (355 us, eight
// 343), and short bf16 calls want the threads for their latency (4 tokens, d = 64:
// 5.0 us, 7.3 with two warps).
//
// STATE: only the segment's own state, from zero, is formed (of b and c).
#pragma once

#include "vla_decay.cuh"

namespace vla_layer {

template <int D, typename T>
struct FmaLay {
    static constexpr int C = 32, THREADS = D == 32 && sizeof(T) == 4 ? 64 : 256;
    static constexpr int LD = D + 4;  // row pitch: rows of a column of float4s lie in different banks
    static constexpr int PP = C + 4;  // of the pairs
    static constexpr int S = 0;
    static constexpr int A = S + D * LD, B = A + C * LD, CC = B + C * LD, CW = CC + C * LD, P = CW + C * LD;
    static constexpr int W = P + C * PP;  // weights: by lag, of the state to tokens
    static constexpr int FLOATS = W + 2 * C;
    static constexpr int SMEM = FLOATS * 4;
    static constexpr int OCC = D == 128 ? 1 : D == 96 ? 2 : D == 64 ? 3 : THREADS == 64 ? 7 : 4;  // blocks an SM holds
    static_assert(OCC * (SMEM + 1024) <= 228 * 1024, "shared memory");
    static constexpr int NPT = (C * (D / 8) + THREADS - 1) / THREADS;  // 8-value pieces of a tile a thread moves
    // tiles of a thread: pairs, PR rows of columns j, j + PJ, ..; output, 4 rows
    // of columns c, c + CG, ..; state, NG x NG squares of GW values, TW GW apart
    static constexpr int PJ = THREADS == 64 ? 8 : 16, PC = C / PJ, PR = C * PJ / THREADS;
    static constexpr int CG = THREADS / 8, OC = D / CG;
    static constexpr int TW = THREADS == 64 ? 8 : 16, GW = D % (4 * TW) ? 2 : 4, NG = D / (GW * TW);
    static_assert(NG * GW * TW == D && TW * TW == THREADS, "tiles");
};

__device__ __forceinline__ float dot4(float4 x, float4 y, float s) {
    return fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
}

// bf16 calls of up to this many tokens run here too (never cut into segments): a
// chunk's fixed costs on the tensor cores are as large as all their arithmetic. Here
// against there, us, forward | gradients, 1 to 8 tokens (the same within a tenth):
//   heads      d = 32                   d = 64                   d = 96                   d = 128
//      32   3.7,  4.6 |  3.8,  5.5   5.4,  5.1 |  5.5,  5.8   7.4,  9.3 |  7.9,  9.7    9.9, 10.9 |  12.2,  11.3
//     256   4.4,  9.1 |  8.5, 24.0   7.1,  9.8 | 16.1, 25.7    10, 18.3 | 29.9, 40.8   19.0, 21.3 |  60.6,  46.8
//     512   5.8, 16.4 | 13.4, 42.9  12.3, 17.7 | 28.7, 46.3    19, 34.3 | 55.2, 74.9   36.7, 40.2 | 117.8, 110.5
// (At d = 128 gradients pay for one block an SM.) Their pairs and states stay in fp32
// as well, so that o is rounded once, where the tensor-core kernel's rows meet one
// more rounding to bf16, however many tokens there are: its errors are about 1.4
// times as large (2.3e-3 of a row's size against 1.65e-3).
constexpr int FMA_T = 8;

template <int D, typename T, bool STATE>
__global__ void __launch_bounds__(FmaLay<D, T>::THREADS, FmaLay<D, T>::OCC)
    vla_decay_fma_kernel(const __grid_constant__ DecayArgs p) {
    using L = FmaLay<D, T>;
    extern __shared__ __align__(16) float fma_sm[];
    float* sm = fma_sm;
    const int tid = threadIdx.x;
    const int seg = blockIdx.x % p.nseg, bh = p.bh0 + blockIdx.x / p.nseg, b = bh / p.H, h = bh % p.H;
    const Role& r = p.role[blockIdx.y];
    const float g = p.log_decay[h];
    const Span sp = span_of(p, b, seg);
    const bool rev = r.reverse;
    float bad = 0.f;  // NaN once an output or a final state is not finite

    static_assert(L::FLOATS >= D * (D + 4) + 24 * D, "by_token's floats");
    if (outgrows(g, L::C)) {
        by_token<D, T, L::THREADS, STATE>(p, blockIdx.y, bh, seg, sm);
        return;
    }

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

    int init_t;
    const float* init = start_of<D, STATE>(p, blockIdx.y, bh, seg, init_t);
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
                const int i0 = tid / L::PJ * L::PR, j0 = tid % L::PJ;
                float acc[L::PR][L::PC] = {};
#pragma unroll 4
                for (int k = 0; k < D; k += 4) {
                    float4 a[L::PR];
#pragma unroll
                    for (int i = 0; i < L::PR; ++i) a[i] = *reinterpret_cast<float4*>(sm + L::A + (i0 + i) * L::LD + k);
#pragma unroll
                    for (int m = 0; m < L::PC; ++m) {
                        const float4 v = *reinterpret_cast<float4*>(sm + L::B + (j0 + L::PJ * m) * L::LD + k);
#pragma unroll
                        for (int i = 0; i < L::PR; ++i) acc[i][m] = dot4(a[i], v, acc[i][m]);
                    }
                }
#pragma unroll
                for (int i = 0; i < L::PR; ++i)
#pragma unroll
                    for (int m = 0; m < L::PC; ++m) {
                        const int j = j0 + L::PJ * m, lag = rev ? j - (i0 + i) : i0 + i - j;
                        sm[L::P + (i0 + i) * L::PP + j] =
                            lag >= 0 && i0 + i < n && j < n ? acc[i][m] * sm[L::W + max(lag, 0)] : 0.f;
                    }
            }
            __syncthreads();
            const int c = tid % L::CG, i0 = tid / L::CG * 4;
            if (i0 < n) {
                // columns c, c + CG, ...: neighbouring lanes read neighbouring rows of S, whose pitch
                // puts them in different banks, and write neighbouring values
                float acc[4][L::OC] = {};
#pragma unroll 2
                for (int k = 0; k < D; k += 4) {
                    float4 a[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<float4*>(sm + L::A + (i0 + i) * L::LD + k);
#pragma unroll
                    for (int m = 0; m < L::OC; ++m) {
                        const float4 v = *reinterpret_cast<float4*>(sm + L::S + (c + m * L::CG) * L::LD + k);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[i][m] = dot4(a[i], v, acc[i][m]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int m = 0; m < L::OC; ++m) acc[i][m] *= sm[L::W + L::C + i0 + i];
#pragma unroll 1
                for (int j = 0; j < n8; j += 4) {
                    float4 w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<float4*>(sm + L::P + (i0 + i) * L::PP + j);
#pragma unroll
                    for (int m = 0; m < L::OC; ++m) {
                        const float* v = sm + L::CC + j * L::LD + c + m * L::CG;
                        const float4 x = make_float4(v[0], v[L::LD], v[2 * L::LD], v[3 * L::LD]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[i][m] = dot4(w[i], x, acc[i][m]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i0 + i >= n) continue;
                    T* o = row_of<T>(r.out, b, h, t0 + i0 + i) + c;
#pragma unroll
                    for (int m = 0; m < L::OC; ++m) {
                        o[m * L::CG] = (T)acc[i][m];
                        bad = fmaf(acc[i][m], 0.f, bad);
                    }
                }
            }
            __syncthreads();
        }
        {
            constexpr int N = L::NG * L::GW;
            const float whole = n < L::C ? decay_pow(g, n) : slow.next();
            const int x0 = tid / L::TW * L::GW, y0 = tid % L::TW * L::GW;
            // GW values of each of NG groups
            auto values = [&](const float* from, float (&v)[N]) {
#pragma unroll
                for (int q = 0; q < L::NG; ++q) {
                    const float* at = from + q * L::TW * L::GW;
                    if constexpr (L::GW == 4) {
                        const float4 t = *reinterpret_cast<const float4*>(at);
                        v[4 * q] = t.x, v[4 * q + 1] = t.y, v[4 * q + 2] = t.z, v[4 * q + 3] = t.w;
                    } else {
                        const float2 t = *reinterpret_cast<const float2*>(at);
                        v[2 * q] = t.x, v[2 * q + 1] = t.y;
                    }
                }
            };
            float acc[N][N];
            auto row = [&](int i) { return sm + L::S + (x0 + i / L::GW * L::TW * L::GW + i % L::GW) * L::LD + y0; };
#pragma unroll
            for (int i = 0; i < N; ++i) {
                values(row(i), acc[i]);
#pragma unroll
                for (int m = 0; m < N; ++m) acc[i][m] *= whole;
            }
#pragma unroll 2
            for (int j = 0; j < n8; ++j) {
                float cv[N], bv[N];
                values(sm + L::CW + j * L::LD + x0, cv);
                values(sm + L::B + j * L::LD + y0, bv);
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int m = 0; m < N; ++m) acc[i][m] = fmaf(cv[i], bv[m], acc[i][m]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int q = 0; q < L::NG; ++q) {
                    float* to = row(i) + q * L::TW * L::GW;
                    if constexpr (L::GW == 4)
                        *reinterpret_cast<float4*>(to) =
                            make_float4(acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]);
                    else
                        *reinterpret_cast<float2*>(to) = make_float2(acc[i][2 * q], acc[i][2 * q + 1]);
                }
        }
    }
    __syncthreads();
    if constexpr (!STATE) {
        // fin, which may be init, is not written yet
        if (__syncthreads_or(bad != bad) &&
            seen_too_early<D, T, L::THREADS, L::C>(p, r, b, h, sp, reinterpret_cast<int*>(sm + L::A))) {
            by_token<D, T, L::THREADS, STATE>(p, blockIdx.y, bh, seg, sm);
            return;
        }
        // rows behind the sequence's last token
        const int behind = min(p.seg_len, p.T - sp.t0) - sp.n;
        const float zero[8] = {};
        for (int i = tid; i < behind * (D / 8); i += L::THREADS)
            store8(row_of<T>(r.out, b, h, sp.t0 + sp.n + i / (D / 8)) + (i % (D / 8)) * 8, zero);
    }
    if (float* fin = end_of<D, STATE>(p, blockIdx.y, bh, seg)) {
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
