// vla_delta_forward.cuh -- the gated delta rule over a sequence (vla_delta.cuh):
// outputs and final state, or (TAPE) what its gradients need of it. fp32, and
// bf16 of few tokens.
//
// What bounds it: the chain of a chunk's products in the workers and, beside it,
// the helpers' next chunk. fp32, 5 x 8 heads of 1,021 tokens, d = 64: 106 us, 3.3 us
// a chunk, for 6.4 us of memory traffic; 8 x 16 heads of 4,096 tokens: 336, 497,
// 820 and 1,450 us for d = 32, 64, 96 and 128 (the last in two rounds of blocks).
// The products of one fp32 part with another are six where bf16 inputs take three,
// and a warp's product waits 21 cycles for the one before it on the same sum.
#pragma once

#include "vla_delta.cuh"

namespace vla_layer {

template <int D, typename T, bool TAPE>
struct DeltaForward {
    static constexpr int NP = PARTS<T>;
    static constexpr int TILES = TAPE && NP == 1 ? 4 : 3;         // K, Q, V and dO (fp32: read where it is used)
    static constexpr bool FULL = TAPE || NP == 3;                 // o as an fp32 result
    static constexpr int OP = FULL ? 3 : 2;                       // parts of S, P and b E on their way to o
    using L = DeltaLay<D, T, TILES, OP>;
};

template <int D, typename T, bool TAPE>
__global__ void __launch_bounds__(DELTA_THREADS<D>, D == 32 ? 2 : 1) vla_delta_forward_kernel(const __grid_constant__ DeltaArgs p) {
    using F = DeltaForward<D, T, TAPE>;
    using L = typename F::L;
    constexpr int NP = F::NP, OP = F::OP, LD = L::LD, SPAN = BLOCK<T>;
    extern __shared__ __align__(128) char sm[];
    const int splits = D / p.rows, bh = blockIdx.x / splits, row0 = (blockIdx.x % splits) * p.rows;
    const int b = bh / p.H, h = bh % p.H;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, workers = p.rows / 8;
    const long long n = delta_len(p, b);
    const int chunks = (int)((n + DC - 1) / DC);
    auto tile = [&](int c, int i) { return sm + L::IN + ((c % L::STAGES) * F::TILES + i) * L::TILE; };
    auto prep = [&](int c) { return sm + L::PREPS + (c & 1) * L::PREP; };

    if (warp >= workers) {
        const int tid = threadIdx.x - workers * 32, hw = warp - workers;
        // bf16: the last helper warp loads; fp32: all, as values are cut into parts on the way
        auto load = [&](int c) {
            const long long t0 = (long long)c * DC;
            if constexpr (NP == 1) {
                load_tile<LD, T>(tile(c, 0), p.k, b, h, t0, 0, D, n, lane);
                load_tile<LD, T>(tile(c, 1), p.q, b, h, t0, 0, D, n, lane);
                load_tile<LD, T>(tile(c, 2), p.v, b, h, t0, row0, p.rows, n, lane);
                if constexpr (F::TILES == 4) load_tile<LD, T>(tile(c, 3), p.dO, b, h, t0, row0, p.rows, n, lane);
                cp_async_commit();
            }
        };
        // fp32: a chunk's rows are loaded while the one before it is prepared, where registers hold them (304 heads of 1,024
        // tokens, d = 64: 412 us with a tile loaded and cut after the other, 268 with the loads under way together, 258 ahead
        // too; d = 128: 834, 750, and 875 ahead, which spills)
        Rows32<NP == 1 ? 32 : D> x, y, z;
        constexpr bool AHEAD = D <= 64;
        auto fetch = [&](int c) {
            const long long t0 = (long long)c * DC;
            x.load(p.k, b, h, t0, 0, D, n, tid, DC);
            y.load(p.q, b, h, t0, 0, D, n, tid, DC);
            if constexpr (AHEAD) z.load(p.v, b, h, t0, row0, p.rows, n, tid, DC);
        };
        auto put = [&](int c) {
            x.template put<LD>(tile(c, 0));
            if constexpr (!AHEAD) x.load(p.v, b, h, (long long)c * DC, row0, p.rows, n, tid, DC);
            y.template put<LD>(tile(c, 1));
            if constexpr (AHEAD)
                z.template put<LD>(tile(c, 2));
            else
                x.template put<LD>(tile(c, 2));
        };
        Whole whole;
        float g = 0.f, beta = 0.f;
        auto gates = [&](int c) {
            const long long t = (long long)c * DC + lane;
            g = t < n && p.g.p ? *p.g.at(b, h, t) : 0.f;
            beta = t < n ? *p.beta.at(b, h, t) : 0.f;
        };
        gates(0);
        if constexpr (NP > 1 && AHEAD)
            if (chunks) fetch(0);
        if (NP == 1 && hw == 3 && chunks) load(0);
        if constexpr (NP == 1) {
            cp_async_wait<0>();
            vla::named_bar(1, HELPERS);
        }
        for (int c = 0; c <= chunks; ++c) {  // chunk c is prepared while chunk c - 1 is computed
            if (c < chunks) {
                if constexpr (NP > 1) {
                    if (!AHEAD) fetch(c);
                    put(c);
                    vla::named_bar(1, HELPERS);
                    if (AHEAD && c + 1 < chunks) fetch(c + 1);
                }
                if (NP == 1 && hw == 3 && c + 1 < chunks) load(c + 1);
                const float gc = g, bc = beta;
                gates(c + 1);
                prepare_chunk<L, D, NP, OP, false>(sm, tile(c, 0), tile(c, 1), prep(c), gc, bc, p.scale, whole, hw, lane);
                cp_async_wait<0>();
            }
            __syncthreads();
        }
        if constexpr (!TAPE) zero_tokens<T>(p.out, b, h, (long long)chunks * DC, p.T, row0, p.rows);
        return;
    }

    constexpr int W = D / 2;  // columns of a warp
    const int r = lane >> 2, t2 = (lane & 3) * 2, pair = warp >> 1, half = warp & 1, my_row = row0 + pair * 16;
    const size_t at = (size_t)my_row * D + half * W;
    float s[W / 8][4];
    load_rows<D, W>(s, p.S0 ? p.S0 + (size_t)bh * D * D + at : nullptr, lane);
    float bad = 0.f;
    char* stage = sm + L::OUT + warp * L::OUTS;
    char *mine = sm + L::SWAP + warp * L::SWAPS, *other = sm + L::SWAP + (warp ^ 1) * L::SWAPS;
    __syncthreads();
    for (int c = 0; c < chunks; ++c) {
        const long long t0 = (long long)c * DC, h0 = t0 + half * 16;  // the chunk's tokens, those whose results it writes
        if constexpr (TAPE) {
            if (t0 % SPAN == 0) store_rows<D, W>(s, p.before + ((size_t)bh * (p.blocks + 1) + t0 / SPAN) * D * D + at, lane);
        }
        const uint32_t kt = vla::smem_u32(tile(c, 0)) + half * W * 2, qt = vla::smem_u32(tile(c, 1)) + half * W * 2;
        const uint32_t vt = vla::smem_u32(tile(c, 2)) + (across_down<LD>(lane) + pair * 16) * 2;
        const char* pr = prep(c);
        const uint32_t inv = vla::smem_u32(pr + L::INV) + down_across<PLD>(lane) * 2;
        const float* gates = reinterpret_cast<const float*>(pr + L::GATES);
        float x[4][4], o[2][4];
        {
            float all[4][4], away[2][4];
            if constexpr (F::FULL) {
                times_rows<W, LD, NP, 0, L::PLANE>(x, all, s, kt + across_down<LD>(lane) * 2, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) give(mine, i, x[i], lane);
                times_rows<W, LD, NP, 0, L::PLANE>(all, x, s, qt + across_down<LD>(lane) * 2, 0);
            } else {
                times_rows<W, LD, NP, OP, L::PLANE>(x, all, s, kt + across_down<LD>(lane) * 2, qt + across_down<LD>(lane) * 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) give(mine, i, x[i], lane);
            }
            half_of(away, all, !half);
            give(mine, 4, away[0], lane);
            give(mine, 5, away[1], lane);
            half_of(o, all, half);
        }
        vla::named_bar(3 + pair, 64);
#pragma unroll
        for (int i = 0; i < 4; ++i) take(other, i, x[i], lane);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            take(other, 4 + i, o[i], lane);
            const float2 near = *reinterpret_cast<const float2*>(gates + GATE_NEAR + (half * 2 + i) * 8 + t2);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] *= p.scale * (e & 1 ? near.y : near.x);
        }
        // what the state gets wrong about the tokens' values, each token on its own
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            float v[2][4];
            columns_of<NP, L::PLANE>(v[0], v[1], vt + (i / 2) * 16 * LD * 2);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 near = *reinterpret_cast<const float2*>(gates + GATE_NEAR + (i + k) * 8 + t2);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i + k][e] = fmaf(-(e & 1 ? near.y : near.x), x[i + k][e], v[k][e]);
            }
        }
        // ... and after the tokens before it in the chunk
        float u[4][4] = {};
        {
            float low[4][4] = {};
            uint32_t a[2][3][4];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) to_operand<3>(a[ks], x[2 * ks], x[2 * ks + 1]);
            times_triangle<INV_PARTS, 3, L::PAIR, true, true>(u, low, a, inv);
            join(u, low);
        }
        if constexpr (TAPE) {
            float e[2][4];
            half_of(e, u, half);
            float* E = p.E + ((size_t)bh * p.T + h0) * D + my_row + r;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int j = i * 8 + t2 + k;
                    if (h0 + j >= n) continue;
                    E[(size_t)j * D] = e[i][k];
                    E[(size_t)j * D + 8] = e[i][2 + k];
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 beta = *reinterpret_cast<const float2*>(gates + GATE_BETA + i * 8 + t2);
#pragma unroll
            for (int e = 0; e < 4; ++e) u[i][e] *= e & 1 ? beta.y : beta.x;
        }
        {
            float low[2][4] = {};
            const uint32_t pairs = vla::smem_u32(pr + L::P) + (half * 16 * PLD + across_down<PLD>(lane)) * 2;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                if (ks > half) break;
                uint32_t a[OP][4];
                to_operand<OP>(a, u[2 * ks], u[2 * ks + 1]);
                times_block<OP, OP, L::PAIR, false>(o, low, a, pairs + ks * 32);
            }
            join(o, low);
        }
        if constexpr (TAPE) {
            float d[2][4];
            if constexpr (NP == 1) {
                columns_of<1, L::PLANE>(d[0], d[1], vla::smem_u32(tile(c, 3)) + (half * 16 * LD + across_down<LD>(lane) + pair * 16) * 2);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const long long t = h0 + i * 8 + t2 + (e & 1);
                        d[i][e] = t < n ? row_of<float>(p.dO, b, h, t)[my_row + r + (e & 2) * 4] : 0.f;
                    }
            }
            float* od = p.od + ((size_t)bh * (D / 16) + my_row / 16) * p.T + h0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float y = over_rows(fmaf(o[i][e], d[i][e], o[i][2 + e] * d[i][2 + e]));
                    if (lane < 4 && h0 + i * 8 + t2 + e < n) od[i * 8 + t2 + e] = y;
                }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (h0 + i * 8 + t2 + (e & 1) < n) bad = fmaf(o[i][e], 0.f, bad);
            store_tokens<T, L::OUT_LD>(o, stage, p.out, b, h, h0, my_row, n, p.T, lane);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 far = *reinterpret_cast<const float2*>(gates + GATE_FAR + i * 8 + t2);
#pragma unroll
            for (int e = 0; e < 4; ++e) u[i][e] *= e & 1 ? far.y : far.x;
        }
        add_outer<W, LD, NP, L::PLANE>(s, gates[GATE_WHOLE], u, kt + down_across<LD>(lane) * 2);
        __syncthreads();
    }
    if constexpr (TAPE) {
        const long long last = (n + SPAN - 1) / SPAN;
        store_rows<D, W>(s, p.before + ((size_t)bh * (p.blocks + 1) + last) * D * D + at, lane);
    } else {
        store_rows<D, W>(s, p.S + (size_t)bh * D * D + at, lane);
#pragma unroll
        for (int m = 0; m < W / 8; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) bad = fmaf(s[m][e], 0.f, bad);
        zero_tokens<T>(p.out, b, h, (long long)chunks * DC, p.T, row0, p.rows);
        if (bad != bad && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, 0);
    }
}

}  // namespace vla_layer
