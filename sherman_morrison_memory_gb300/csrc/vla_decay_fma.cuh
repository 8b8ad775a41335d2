// vla_decay_fma.cuh -- the operation of vla_decay.cuh on the FP32 pipes, for
// any input type: a block per (role, head, segment) goes through its tokens 32
// at a time with S and the three tiles in shared memory as fp32.
//
// STATE: only the segment's own state, from zero, is formed (of b and c).
#pragma once

#include "vla_decay.cuh"

namespace vla_layer {

template <int D>
struct FmaLay {
    static constexpr int C = 32, THREADS = 256;
    static constexpr int LD = D + 4;  // row pitch: rows of a column of float4s lie in different banks
    static constexpr int S = 0;
    static constexpr int A = S + D * LD, B = A + C * LD, CC = B + C * LD, P = CC + C * LD;
    static constexpr int W = P + C * (C + 1);
    static constexpr int FLOATS = W + 3 * C;
    static constexpr int SMEM = FLOATS * 4;
    static constexpr int CG = D / 4;                           // groups of four columns
    static constexpr int RG = D == 128 || D == 96 ? 8 : 1024 / D;  // row groups of the output tile
    static constexpr int RPT = C / RG;
};

template <int D, typename T>
__device__ __forceinline__ void load_tile(float* dst, const Seq& s, int b, int h, int t0, int n) {
    using L = FmaLay<D>;
    for (int i = threadIdx.x; i < L::C * (D / 8); i += L::THREADS) {
        const int r = i / (D / 8), c = (i % (D / 8)) * 8;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < n) load8(row_of<T>(s, b, h, t0 + r) + c, x);
        store8(dst + r * L::LD + c, x);
    }
}

__device__ __forceinline__ float dot4(float4 x, float4 y, float s) {
    return fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
}

template <int D, typename T, bool STATE>
__global__ void __launch_bounds__(256, 2) vla_decay_fma_kernel(const __grid_constant__ DecayArgs p) {
    using L = FmaLay<D>;
    extern __shared__ __align__(16) float fma_sm[];
    float* sm = fma_sm;
    const int tid = threadIdx.x;
    const int seg = blockIdx.x % p.nseg, bh = blockIdx.x / p.nseg, b = bh / p.H, h = bh % p.H;
    const Role& r = p.role[blockIdx.y];
    const float g = p.log_decay[h];
    const Span sp = span_of(p, b, seg);
    const bool rev = r.reverse;
    float bad = 0.f;  // NaN once an output or a final state is not finite

    const float* init = r.init ? r.init + (size_t)bh * D * D : nullptr;
    int init_t = r.init_t;
    if (p.nseg > 1) {
        init = STATE ? nullptr : p.seg + (((size_t)p.seg_role[blockIdx.y] * p.B * p.H + bh) * p.nseg + seg) * D * D;
        init_t = p.seg_t[blockIdx.y];
    }
    for (int i = tid; i < D * D; i += L::THREADS) {
        const int x = i / D, y = i % D;
        const float v = init ? init[i] : 0.f;
        sm[L::S + (init_t ? y * L::LD + x : x * L::LD + y)] = v;
    }
    const int chunks = (sp.n + L::C - 1) / L::C;
    for (int ci = 0; ci < chunks; ++ci) {
        const int c0 = (rev ? chunks - 1 - ci : ci) * L::C;  // first token within the segment
        const int n = min(L::C, sp.n - c0), t0 = sp.t0 + c0;
        __syncthreads();
        if (!STATE) load_tile<D, T>(sm + L::A, r.a, b, h, t0, n);
        load_tile<D, T>(sm + L::B, r.b, b, h, t0, n);
        load_tile<D, T>(sm + L::CC, r.c, b, h, t0, n);
        if (tid < L::C) {
            const int back = n - 1 - tid;  // tokens behind this one
            const bool in = tid < n;
            sm[L::W + tid] = decay_pow(g, tid);                                              // l^lag
            sm[L::W + L::C + tid] = in ? r.w_st * decay_pow(g, rev ? back : tid + 1) : 0.f;   // state to output
            sm[L::W + 2 * L::C + tid] = in ? r.k_st * decay_pow(g, rev ? tid + 1 : back) : 0.f;  // token to state
        }
        __syncthreads();
        if (!STATE) {
            {
                const int i = tid / 8;
                for (int j = tid % 8; j < L::C; j += 8) {
                    float s = 0.f;
#pragma unroll
                    for (int k = 0; k < D; k += 4)
                        s = dot4(*reinterpret_cast<float4*>(sm + L::A + i * L::LD + k),
                                 *reinterpret_cast<float4*>(sm + L::B + j * L::LD + k), s);
                    const int lag = rev ? j - i : i - j;
                    sm[L::P + i * (L::C + 1) + j] = lag >= 0 && i < n && j < n ? r.w_in * s * sm[L::W + lag] : 0.f;
                }
            }
            __syncthreads();
            if (tid < L::CG * L::RG) {
                // columns c, c + CG, ...: neighbouring lanes read neighbouring rows of S, whose pitch
                // puts them in different banks, and write neighbouring values
                const int c = tid % L::CG, i0 = (tid / L::CG) * L::RPT;
                float acc[L::RPT][4] = {};
#pragma unroll 2
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
#pragma unroll 4
                for (int j = 0; j < n; ++j) {
                    float v[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) v[m] = sm[L::CC + j * L::LD + c + m * L::CG];
#pragma unroll
                    for (int i = 0; i < L::RPT; ++i) {
                        const float w = sm[L::P + (i0 + i) * (L::C + 1) + j];
#pragma unroll
                        for (int m = 0; m < 4; ++m) acc[i][m] = fmaf(w, v[m], acc[i][m]);
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
        const float whole = decay_pow(g, n);
        for (int blk = tid; blk < L::CG * L::CG; blk += L::THREADS) {
            const int x = (blk / L::CG) * 4, y = (blk % L::CG) * 4;
            float acc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int m = 0; m < 4; ++m) acc[i][m] = whole * sm[L::S + (x + i) * L::LD + y + m];
#pragma unroll 4
            for (int j = 0; j < n; ++j) {
                const float w = sm[L::W + 2 * L::C + j];
                const float4 cv = *reinterpret_cast<float4*>(sm + L::CC + j * L::LD + x);
                const float4 bv = *reinterpret_cast<float4*>(sm + L::B + j * L::LD + y);
                const float cw[4] = {cv.x * w, cv.y * w, cv.z * w, cv.w * w};
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
    float* fin = STATE ? p.seg + (((size_t)blockIdx.y * p.B * p.H + bh) * p.nseg + seg) * D * D
                       : (p.nseg > 1 || !r.fin ? nullptr : r.fin + (size_t)bh * D * D);
    if (fin) {
        for (int i = tid; i < D * D; i += L::THREADS) {
            const float v = sm[L::S + (i / D) * L::LD + i % D];
            fin[i] = v;
            bad = fmaf(v, 0.f, bad);
        }
    }
    if (bad != bad && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, sp.t0);
}

}  // namespace vla_layer
