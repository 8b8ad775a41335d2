// vla_delta_forward.cuh -- the gated delta rule over a sequence (vla_delta.cuh):
// outputs and final state, or (TAPE) what its gradients need of it.
#pragma once

#include "vla_delta.cuh"

namespace vla_layer {

template <int D, typename T, bool TAPE>
struct DeltaForward {
    static constexpr int NP = PARTS<T>;
    static constexpr int TILES = TAPE && NP == 1 ? 4 : 3;         // K, Q, V and dO (fp32: read where it is used)
    static constexpr bool FULL = TAPE || NP == 3;                 // o as an fp32 result
    static constexpr int PP = FULL ? 3 : 1, UP = FULL ? 3 : 2;    // parts of P and of b E on their way to o
    using L = DeltaLay<D, T, TILES, PP>;
};

template <int D, typename T, bool TAPE>
__global__ void __launch_bounds__(D * 2 + HELPERS) vla_delta_forward_kernel(const __grid_constant__ DeltaArgs p) {
    using F = DeltaForward<D, T, TAPE>;
    using L = typename F::L;
    constexpr int NP = F::NP, PP = F::PP, LD = L::LD, SPAN = BLOCK<T>;
    extern __shared__ __align__(128) char sm[];
    const int splits = D / p.rows, bh = blockIdx.x / splits, row0 = (blockIdx.x % splits) * p.rows;
    const int b = bh / p.H, h = bh % p.H;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, workers = p.rows / 16;
    const long long n = delta_len(p, b);
    const int chunks = (int)((n + DC - 1) / DC);
    auto tile = [&](int c, int i) { return sm + L::IN + ((c % L::STAGES) * F::TILES + i) * L::TILE; };
    auto prep = [&](int c) { return sm + L::PREPS + (c & 1) * L::PREP; };

    if (warp >= workers) {
        const int tid = threadIdx.x - workers * 32, hw = warp - workers;
        // bf16: the last helper warp loads; fp32: all, as values are cut into parts on the way
        constexpr int LOADERS = NP == 1 ? 32 : HELPERS;
        auto load = [&](int c) {
            const int at = tid & (LOADERS - 1);
            const long long t0 = (long long)c * DC;
            load_tile<LD, LOADERS, T>(tile(c, 0), p.k, b, h, t0, 0, D, n, at);
            load_tile<LD, LOADERS, T>(tile(c, 1), p.q, b, h, t0, 0, D, n, at);
            load_tile<LD, LOADERS, T>(tile(c, 2), p.v, b, h, t0, row0, p.rows, n, at);
            if constexpr (F::TILES == 4) load_tile<LD, LOADERS, T>(tile(c, 3), p.dO, b, h, t0, row0, p.rows, n, at);
            cp_async_commit();
        };
        Whole whole;
        float g = 0.f, beta = 0.f;
        auto gates = [&](int c) {
            const long long t = (long long)c * DC + lane;
            g = t < n && p.g.p ? *p.g.at(b, h, t) : 0.f;
            beta = t < n ? *p.beta.at(b, h, t) : 0.f;
        };
        gates(0);
        if (NP == 1 && hw == 3 && chunks) load(0);
        if constexpr (NP == 1) {
            cp_async_wait<0>();
            vla::named_bar(1, HELPERS);
        }
        for (int c = 0; c <= chunks; ++c) {  // chunk c is prepared while chunk c - 1 is computed
            if (c < chunks) {
                if constexpr (NP > 1) {
                    load(c);
                    vla::named_bar(1, HELPERS);
                }
                if (hw < 3) {
                    const float gc = g, bc = beta;
                    gates(c + 1);
                    prepare_chunk<L, D, NP, PP, false>(sm, tile(c, 0), tile(c, 1), prep(c), gc, bc, p.scale, whole, hw, lane);
                } else if (NP == 1 && c + 1 < chunks) {
                    load(c + 1);
                    cp_async_wait<0>();
                }
            }
            __syncthreads();
        }
        if constexpr (!TAPE) zero_tokens<T>(p.out, b, h, (long long)chunks * DC, p.T, row0, p.rows);
        return;
    }

    const int r = lane >> 2, t2 = (lane & 3) * 2, my_row = row0 + warp * 16;
    float s[D / 8][4];
    load_rows<D>(s, p.S0 ? p.S0 + (size_t)bh * D * D + my_row * D : nullptr, lane);
    float bad = 0.f;
    char* stage = sm + L::OUT + warp * DC * L::OUT_LD * 2;
    __syncthreads();
    for (int c = 0; c < chunks; ++c) {
        const long long t0 = (long long)c * DC;
        if constexpr (TAPE) {
            if (t0 % SPAN == 0)
                store_rows<D>(s, p.before + ((size_t)bh * (p.blocks + 1) + t0 / SPAN) * D * D + my_row * D, lane);
        }
        const uint32_t kt = vla::smem_u32(tile(c, 0)), qt = vla::smem_u32(tile(c, 1));
        const uint32_t vt = vla::smem_u32(tile(c, 2)) + (across_down<LD>(lane) + warp * 16) * 2;
        const char* pr = prep(c);
        const float* gates = reinterpret_cast<const float*>(pr + L::GATES);
        float x[4][4], o[4][4];
        if constexpr (F::FULL) {
            times_rows<D, LD, NP, 0, L::PLANE>(x, o, s, kt + across_down<LD>(lane) * 2, 0);
            times_rows<D, LD, NP, 0, L::PLANE>(o, x, s, qt + across_down<LD>(lane) * 2, 0);
        } else {
            times_rows<D, LD, NP, 1, L::PLANE>(x, o, s, kt + across_down<LD>(lane) * 2, qt + across_down<LD>(lane) * 2);
        }
        // what the state gets wrong about the tokens' values, each token on its own
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 near = *reinterpret_cast<const float2*>(gates + GATE_NEAR + i * 8 + t2);
            if (i % 2 == 0) {
                float v0[4], v1[4];
                columns_of<NP, L::PLANE>(v0, v1, vt + (i / 2) * 16 * LD * 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][e] = fmaf(-(e & 1 ? near.y : near.x), x[i][e], v0[e]);
                const float2 next = *reinterpret_cast<const float2*>(gates + GATE_NEAR + i * 8 + 8 + t2);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i + 1][e] = fmaf(-(e & 1 ? next.y : next.x), x[i + 1][e], v1[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] *= p.scale * (e & 1 ? near.y : near.x);
        }
        // ... and after the tokens before it in the chunk
        float u[4][4] = {}, low[4][4] = {};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            uint32_t a[3][4];
            to_operand<3>(a, x[2 * ks], x[2 * ks + 1]);
            times_triangle<INV_PARTS, 3, L::PAIR, true, true>(u, low, a, ks, vla::smem_u32(pr + L::INV) + down_across<PLD>(lane) * 2);
        }
        join(u, low);
        if constexpr (TAPE) {
            float* E = p.E + ((size_t)bh * p.T + t0) * D + my_row;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = i * 8 + t2 + e;
                    if (t0 + j >= n) continue;
                    E[(size_t)j * D + r] = u[i][e];
                    E[(size_t)j * D + r + 8] = u[i][2 + e];
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 beta = *reinterpret_cast<const float2*>(gates + GATE_BETA + i * 8 + t2);
#pragma unroll
            for (int e = 0; e < 4; ++e) u[i][e] *= e & 1 ? beta.y : beta.x;
        }
        {
            float ol[4][4] = {};
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                uint32_t a[F::UP][4];
                to_operand<F::UP>(a, u[2 * ks], u[2 * ks + 1]);
                times_triangle<PP, F::UP, L::PAIR, true, false>(o, F::FULL ? ol : o, a, ks, vla::smem_u32(pr + L::P) + across_down<PLD>(lane) * 2);
            }
            if constexpr (F::FULL) join(o, ol);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 far = *reinterpret_cast<const float2*>(gates + GATE_FAR + i * 8 + t2);
#pragma unroll
            for (int e = 0; e < 4; ++e) u[i][e] *= e & 1 ? far.y : far.x;
        }
        add_outer<D, LD, NP, L::PLANE>(s, gates[GATE_WHOLE], u, kt + down_across<LD>(lane) * 2);
        if constexpr (TAPE) {
            float od[8];
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                float d0[4], d1[4];
                if constexpr (NP == 1) {
                    columns_of<1, L::PLANE>(d0, d1, vla::smem_u32(tile(c, 3)) + (across_down<LD>(lane) + warp * 16 + (i / 2) * 16 * LD) * 2);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const long long t = t0 + i * 8 + (e >> 2) * 8 + t2 + (e & 1);
                        const float v = t < n ? row_of<float>(p.dO, b, h, t)[my_row + r + (e & 2) * 4] : 0.f;
                        (e < 4 ? d0 : d1)[e & 3] = v;
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    od[2 * i + e] = over_rows(fmaf(o[i][e], d0[e], o[i][2 + e] * d0[2 + e]));
                    od[2 * i + 2 + e] = over_rows(fmaf(o[i + 1][e], d1[e], o[i + 1][2 + e] * d1[2 + e]));
                }
            }
            if (lane < 4) {
                float* out = p.od + ((size_t)bh * (D / 16) + my_row / 16) * p.T + t0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = (i >> 1) * 8 + t2 + (i & 1);
                    if (t0 + j < n) out[j] = od[i];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t0 + i * 8 + t2 + (e & 1) < n) bad = fmaf(o[i][e], 0.f, bad);
            store_tokens<T, L::OUT_LD>(o, stage, p.out, b, h, t0, my_row, n, p.T, lane);
        }
        __syncthreads();
    }
    if constexpr (TAPE) {
        const long long last = (n + SPAN - 1) / SPAN;
        store_rows<D>(s, p.before + ((size_t)bh * (p.blocks + 1) + last) * D * D + my_row * D, lane);
    } else {
        store_rows<D>(s, p.S + (size_t)bh * D * D + my_row * D, lane);
#pragma unroll
        for (int m = 0; m < D / 8; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) bad = fmaf(s[m][e], 0.f, bad);
        zero_tokens<T>(p.out, b, h, (long long)chunks * DC, p.T, row0, p.rows);
        if (bad != bad && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, 0);
    }
}

}  // namespace vla_layer
