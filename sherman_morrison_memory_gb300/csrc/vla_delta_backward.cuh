// vla_delta_backward.cuh -- gradients of the gated delta rule (vla_delta.cuh), in
// three launches: the forward recurrence again, which keeps S before every block
// of tokens, E and o . dO; the reverse recurrence, which gives dV and keeps R
// behind every block; and, all blocks side by side, dQ, dK and the gates'
// gradients. With i, j tokens of a block, S before and R behind it, u = b e:
//
//   X[i][j] = scale exp(G_i - G_j) dO_i . u_j  (j <= i),   M[i][j] = -exp(G_i - G_j) dV_i . u_j  (j < i)
//   dQ = scale diag(exp(G)) dO S + X K
//   dK = diag(exp(G_C - G)) U R - diag(exp(G)) dV S + X^T Q + M K + M^T K
//
// A log decay touches q exp(G), v exp(-G) and the state behind a block alone, so
//   dg_t = sum over the block's i >= t of (o_i . dO_i - v_i . dV_i) + <R, S> behind the block,
// of fp32 results of the two recurrences. Before a first token without a state
// nothing decays: its dg is 0, where the sum would leave its roundings. So it would
// where exp(g_t) is small: the terms do not get smaller with it, what they leave does
// (2e-5 of dg is lost at g = -3, 8% at -12, all of it at -16). Tokens whose decay is
// below DeltaGrads::STRONG take what lies across it instead, every term of which has
// the factor exp(g_t) in it:
//   dg_t = sum i >= t of (scale exp(G_i) q_i . S^T dO_i - exp(G_i) k_i . S^T dV_i) + sum j < t of exp(G_C - G_j) k_j . R^T u_j
//          + sum i >= t > j of (X_ij q_i . k_j + M_ij k_i . k_j) + exp(G_C) <R, S> of S before the block.
// Only sums of such terms are formed, no differences: of 16 x 16 blocks of pairs their
// rows' and columns' sums. A block of tokens without such a one does nothing of it (bf16
// gradients of 8 x 16 heads of 4,096 tokens, d = 64: 710 us, 806 with one in every block).
//
// What bounds them: the recurrences' chains, as forward; the third launch moves two
// fp32 states of every 64 tokens (fp32: 32), E and seven sequences. bf16, 4 x 8 heads
// of 4,096 tokens, d = 64: 493 us, of which 207, 206 and 79; 2 x 32 heads of 2,048, d =
// 128: 140, 137 and 213 (542 MB of DRAM, 80 us at the memory's rate; one block an SM,
// whose loads, products and barriers follow each other, its shared memory 54% busy).
// States every 64 tokens and not 32: half the bytes, and the pairs' products still are
// a small part. Of 2 x 32 heads of 4,095 tokens, d = 128, in all: 1,620 us with the states
// loaded as they are used, 1,474 through a ring of shared memory, 32 rows at a time; 1,253
// with register loads first and X and M of a block together; 1,017 with the reverse
// recurrence on tcgen05; 946 with <R, S> in the third launch, where R passes anyway (in the
// reverse recurrence the loads of S stood in the chain); 921 with stores off the chain; 947
// with S and R in two parts for dQ and dK, 953 with dg of strong decays apart.
#pragma once

#include "vla_delta.cuh"

namespace vla_layer {

template <int D, typename T>
struct DeltaReverse {
    static constexpr int NP = PARTS<T>;
    static constexpr int TILES = NP == 1 ? 4 : 3;  // K, Q, dO and V (fp32: read where it is used)
    using L = DeltaLay<D, T, TILES, 3>;
};

template <int D, typename T>
__global__ void __launch_bounds__(DELTA_THREADS<D>, D == 32 ? 2 : 1) vla_delta_reverse_kernel(const __grid_constant__ DeltaArgs p) {
    using F = DeltaReverse<D, T>;
    using L = typename F::L;
    constexpr int NP = F::NP, LD = L::LD, SPAN = BLOCK<T>;
    extern __shared__ __align__(128) char sm[];
    const int splits = D / p.rows, bh = blockIdx.x / splits, row0 = (blockIdx.x % splits) * p.rows;
    const int b = bh / p.H, h = bh % p.H;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, workers = p.rows / 8;
    const long long n = delta_len(p, b);
    const int chunks = (int)((n + DC - 1) / DC);
    // the m-th chunk in the order of work
    auto tile = [&](int m, int i) { return sm + L::IN + ((m % L::STAGES) * F::TILES + i) * L::TILE; };
    auto prep = [&](int m) { return sm + L::PREPS + (m & 1) * L::PREP; };

    if (warp >= workers) {
        const int tid = threadIdx.x - workers * 32, hw = warp - workers;
        // bf16: the last helper warp loads; fp32: all, as values are cut into parts on the way
        auto load = [&](int m) {
            const long long t0 = (long long)(chunks - 1 - m) * DC;
            if constexpr (NP == 1) {
                load_tile<LD, T>(tile(m, 0), p.k, b, h, t0, 0, D, n, lane);
                load_tile<LD, T>(tile(m, 1), p.q, b, h, t0, 0, D, n, lane);
                load_tile<LD, T>(tile(m, 2), p.dO, b, h, t0, row0, p.rows, n, lane);
                if constexpr (F::TILES == 4) load_tile<LD, T>(tile(m, 3), p.v, b, h, t0, row0, p.rows, n, lane);
                cp_async_commit();
            }
        };
        // fp32: as in the forward kernel
        Rows32<NP == 1 ? 32 : D> x, y, z;
        constexpr bool AHEAD = D <= 64;
        auto fetch = [&](int m) {
            const long long t0 = (long long)(chunks - 1 - m) * DC;
            x.load(p.k, b, h, t0, 0, D, n, tid, -DC);
            y.load(p.q, b, h, t0, 0, D, n, tid, -DC);
            if constexpr (AHEAD) z.load(p.dO, b, h, t0, row0, p.rows, n, tid, -DC);
        };
        auto put = [&](int m) {
            x.template put<LD>(tile(m, 0));
            if constexpr (!AHEAD) x.load(p.dO, b, h, (long long)(chunks - 1 - m) * DC, row0, p.rows, n, tid, -DC);
            y.template put<LD>(tile(m, 1));
            if constexpr (AHEAD)
                z.template put<LD>(tile(m, 2));
            else
                x.template put<LD>(tile(m, 2));
        };
        Whole whole;
        float g = 0.f, beta = 0.f;
        auto gates = [&](int m) {
            const long long t = (long long)(chunks - 1 - m) * DC + lane;
            const bool on = t >= 0 && t < n;
            g = on && p.g.p ? *p.g.at(b, h, t) : 0.f;
            beta = on ? *p.beta.at(b, h, t) : 0.f;
        };
        gates(0);
        if constexpr (NP > 1 && AHEAD)
            if (chunks) fetch(0);
        if (NP == 1 && hw == 3 && chunks) load(0);
        if constexpr (NP == 1) {
            cp_async_wait<0>();
            vla::named_bar(1, HELPERS);
        }
        for (int m = 0; m <= chunks; ++m) {  // chunk m is prepared while chunk m - 1 is computed
            if (m < chunks) {
                if constexpr (NP > 1) {
                    if (!AHEAD) fetch(m);
                    put(m);
                    vla::named_bar(1, HELPERS);
                    if (AHEAD && m + 1 < chunks) fetch(m + 1);
                }
                if (NP == 1 && hw == 3 && m + 1 < chunks) load(m + 1);
                const float gm = g, bm = beta;
                gates(m + 1);
                prepare_chunk<L, D, NP, 3, true>(sm, tile(m, 0), tile(m, 1), prep(m), gm, bm, p.scale, whole, hw, lane);
                cp_async_wait<0>();
            }
            __syncthreads();
        }
        zero_tokens<T>(p.dv, b, h, (long long)chunks * DC, p.T, row0, p.rows);
        return;
    }

    constexpr int W = D / 2;  // columns of a warp
    const int r = lane >> 2, t2 = (lane & 3) * 2, pair = warp >> 1, half = warp & 1, my_row = row0 + pair * 16;
    const size_t own = (size_t)my_row * D + half * W;
    float s[W / 8][4];
    load_rows<D, W>(s, p.dS_T ? p.dS_T + (size_t)bh * D * D + own : nullptr, lane);
    float bad = 0.f;
    char* stage = sm + L::OUT + warp * L::OUTS;
    char *mine = sm + L::SWAP + warp * L::SWAPS, *other = sm + L::SWAP + (warp ^ 1) * L::SWAPS;
    __syncthreads();
    for (int m = 0; m < chunks; ++m) {
        const long long t0 = (long long)(chunks - 1 - m) * DC, h0 = t0 + half * 16;
        const uint32_t kt = vla::smem_u32(tile(m, 0)) + half * W * 2, qt = vla::smem_u32(tile(m, 1)) + half * W * 2;
        const uint32_t ot = vla::smem_u32(tile(m, 2)) + (across_down<LD>(lane) + pair * 16) * 2;
        const char* pr = prep(m);
        const float* gates = reinterpret_cast<const float*>(pr + L::GATES);
        float e[2][4], v[2][4];
        {
            const float* E = p.E + ((size_t)bh * p.T + h0) * D + my_row + r;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = i * 8 + t2 + (k & 1);
                    e[i][k] = h0 + j < n ? E[(size_t)j * D + (k & 2) * 4] : 0.f;
                    if constexpr (NP > 1) v[i][k] = h0 + j < n ? row_of<float>(p.v, b, h, h0 + j)[my_row + r + (k & 2) * 4] : 0.f;
                }
        }
        if (m == 0 || (t0 + DC) % SPAN == 0) {
            const long long blk = t0 / SPAN;
            const size_t at = ((size_t)bh * (p.blocks + 1) + blk) * D * D + own;
            store_rows<D, W>(s, p.behind + at, lane);
        }
        float x[4][4];
        {
            float none[4][4];
            times_rows<W, LD, NP, 0, L::PLANE>(x, none, s, kt + across_down<LD>(lane) * 2, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) give(mine, i, x[i], lane);
        vla::named_bar(3 + pair, 64);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            take(other, i, x[i], lane);
            const float2 far = *reinterpret_cast<const float2*>(gates + GATE_FAR + i * 8 + t2);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i][k] *= k & 1 ? far.y : far.x;
        }
        {
            float low[4][4] = {};
            uint32_t a[2][NP][4];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int q = 0; q < NP; ++q) ldsm_t(a[ks][q], ot + q * L::PLANE + ks * 16 * LD * 2);
            times_triangle<3, NP, L::PAIR, false, true>(x, low, a, vla::smem_u32(pr + L::P) + down_across<PLD>(lane) * 2);
            join(x, low);
        }
        float u[4][4] = {};
        {
            float low[4][4] = {};
            uint32_t a[2][3][4];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) to_operand<3>(a[ks], x[2 * ks], x[2 * ks + 1]);
            times_triangle<INV_PARTS, 3, L::PAIR, false, false>(u, low, a, vla::smem_u32(pr + L::INV) + across_down<PLD>(lane) * 2);
            join(u, low);
        }
        // the half of the tokens whose results it writes
        float y[2][4];
        half_of(y, u, half);
        if constexpr (NP == 1)
            columns_of<1, L::PLANE>(v[0], v[1], vla::smem_u32(tile(m, 3)) + (half * 16 * LD + across_down<LD>(lane) + pair * 16) * 2);
        {
            const size_t at = ((size_t)bh * (D / 16) + my_row / 16) * p.T + h0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 beta = *reinterpret_cast<const float2*>(gates + GATE_BETA + (half * 2 + i) * 8 + t2);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float bd = over_rows(fmaf(y[i][k], e[i][k], y[i][2 + k] * e[i][2 + k]));
                    y[i][k] *= k ? beta.y : beta.x;
                    y[i][2 + k] *= k ? beta.y : beta.x;
                    const float vd = over_rows(fmaf(y[i][k], v[i][k], y[i][2 + k] * v[i][2 + k]));
                    const int j = i * 8 + t2 + k;
                    if (h0 + j < n) {
                        if (lane < 4) p.bd[at + j] = bd, p.vd[at + j] = vd;
                        bad = fmaf(y[i][k], 0.f, fmaf(y[i][2 + k], 0.f, bad));
                    }
                }
            }
        }
        store_tokens<T, L::OUT_LD>(y, stage, p.dv, b, h, h0, my_row, n, p.T, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 near = *reinterpret_cast<const float2*>(gates + GATE_NEAR + i * 8 + t2);
            const float2 beta = *reinterpret_cast<const float2*>(gates + GATE_BETA + i * 8 + t2);
#pragma unroll
            for (int k = 0; k < 4; ++k) u[i][k] *= -((k & 1 ? near.y : near.x) * (k & 1 ? beta.y : beta.x));
        }
        add_outer<W, LD, NP, L::PLANE>(s, gates[GATE_WHOLE], u, kt + down_across<LD>(lane) * 2);
#pragma unroll
        for (int i = 0; i < 4; i += 2) columns_of<NP, L::PLANE>(x[i], x[i + 1], ot + (i / 2) * 16 * LD * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 near = *reinterpret_cast<const float2*>(gates + GATE_NEAR + i * 8 + t2);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i][k] *= p.scale * (k & 1 ? near.y : near.x);
        }
        add_outer<W, LD, NP, L::PLANE>(s, 1.f, x, qt + down_across<LD>(lane) * 2);
        __syncthreads();
    }
    if (p.dS0) {
        store_rows<D, W>(s, p.dS0 + (size_t)bh * D * D + own, lane);
#pragma unroll
        for (int i = 0; i < W / 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) bad = fmaf(s[i][k], 0.f, bad);
    }
    zero_tokens<T>(p.dv, b, h, (long long)chunks * DC, p.T, row0, p.rows);
    if (bad != bad && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, 0);
}

// exp(x) as two factors, for blocks of 64 tokens: a head that grows by less than float32 holds in 32 tokens grows by up to the
// square of that in 64, of values so small that the results are finite. Where exp(x) is small enough it is the first alone.
__device__ __forceinline__ float grow_first(float x) { return expf(x > 64.f ? 0.5f * x : x); }
__device__ __forceinline__ float grow_second(float x) { return x > 64.f ? expf(0.5f * x) : 1.f; }

// dQ, dK and the gates' gradients of a block of tokens: two warps for 16 columns of d, a half of the tokens each. bf16 calls
// take dV as it was written, the one rounding of a term to bf16 on its way (dk 2.0e-3 off where rounding the exact result
// gives 1.65e-3); S, R, U, X and M are two parts, 2^-16 off. (One part of S against dO and of R against U: 2.2e-3 for dq and
// dk. dV in two parts, the second in E's low bits: 1.65e-3 for dk, but 1,043 us for 948 of 2 x 32 heads of 4,095 tokens, d =
// 128, and 541 for 485 of 4 x 8 heads, d = 64.)
template <int D, typename T>
struct DeltaGrads {
    static constexpr int NP = PARTS<T>, TB = BLOCK<T>, MT = TB / 16;
    static constexpr int UP = NP == 1 ? 2 : 3, XP = UP, MP = UP;
    // the log decay below which dg_t is the sum of what lies across it: as exact as the parts are (fp32 2e-7; bf16 4e-5 to 2e-4,
    // by dV as it was written), where the difference of sums loses 1e-6 at -1, 2e-5 at -3 and 4e-5 at -5
    static constexpr float STRONG = NP == 1 ? -6.f : -2.f;
    static constexpr int UNITS = MT * (MT + 1) / 2;  // 16 x 16 blocks of pairs
    static constexpr int LD = D + 8, PLANE = TB * LD * 2, XLD = TB + 8, XPLANE = TB * XLD * 2;
    static constexpr int Q = 0, K = Q + NP * PLANE, O = K + NP * PLANE, V = O + NP * PLANE, U = V + NP * PLANE,
                         X = U + UP * PLANE, M = X + XP * XPLANE, GATES = M + MP * XPLANE, RING = GATES + 5 * TB * 4;
    // the states, 32 rows at a time, two of them under way, or (bf16, d = 64) one, which leaves room for two blocks on an
    // SM (all gradients of 8 x 16 heads of 4,096 tokens: 795 us with two under way, 706 with one); the rows' shares of the
    // gates' gradients
    static constexpr int SLD = D + 4, SLICE = 32 * SLD * 4, SLICES = NP == 1 && D == 64 ? 2 : 3, SHARES = RING + SLICES * SLICE,
                         ENDS = SHARES + (D / 16) * TB * 8, FLAGS = ENDS + D / 8 * 8, PAIRS = FLAGS + 16,
                         BYTES = PAIRS + UNITS * 128;
    static constexpr int THREADS = D * 4, MH = MT / 2;  // a warp's tiles of 16 tokens
};

// Two values of a tile, their parts added up.
template <int NP, int PLANE>
__device__ __forceinline__ float2 two_of(const char* at) {
    float2 x = make_float2(0.f, 0.f);
#pragma unroll
    for (int q = NP - 1; q >= 0; --q) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(at + q * PLANE);
        x.x += low_of(w), x.y += high_of(w);
    }
    return x;
}

// dg's terms of a 16 x 16 block of pairs, X_ij q_i . k_j + M_ij k_i . k_j for j < i: below the diagonal the sums of rows from
// each one on in out[0..16) and of columns up to each one in out[16..32); on it out[t], of the pairs that lie across its token
// t. By the warp that wrote X and M there.
template <typename L, int D>
__device__ __noinline__ void sums_across(float* out, const char* sm, int mt, int np, int lane) {
    constexpr int NP = L::NP, LD = L::LD;
    float z[2][2][4] = {}, zl[2][2][4] = {};  // q_i . k_j, k_i . k_j
    const uint32_t base = vla::smem_u32(sm), a_at = base + (mt * 16 * LD + down_across<LD>(lane)) * 2, b_at = base + L::K + (np * 16 * LD + across_down<LD>(lane)) * 2;
#pragma unroll 2
    for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t a[NP][4], b[2][NP][2];
#pragma unroll
        for (int q = 0; q < NP; ++q) ldsm_pair(b, 0, q, b_at + q * L::PLANE + ks * 32);
#pragma unroll
        for (int q = 0; q < NP; ++q) ldsm(a[q], a_at + L::Q + q * L::PLANE + ks * 32);
        mma_tiles<NP>(z[0], zl[0], a, b);
#pragma unroll
        for (int q = 0; q < NP; ++q) ldsm(a[q], a_at + L::K + q * L::PLANE + ks * 32);
        mma_tiles<NP>(z[1], zl[1], a, b);
    }
    join(z[0], zl[0]);
    join(z[1], zl[1]);
    const int r = lane >> 2, t2 = (lane & 3) * 2;
    float row[2] = {}, col[4] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int at = ((mt * 16 + hf * 8 + r) * L::XLD + np * 16 + k * 8 + t2) * 2;
            const float2 x = two_of<L::XP, L::XPLANE>(sm + L::X + at), m = two_of<L::MP, L::XPLANE>(sm + L::M + at);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int e = 2 * hf + q;
                const bool on = mt != np || k * 8 + t2 + q < hf * 8 + r;
                z[0][k][e] = on ? fmaf(q ? x.y : x.x, z[0][k][e], (q ? m.y : m.x) * z[1][k][e]) : 0.f;
                row[hf] += z[0][k][e], col[2 * k + q] += z[0][k][e];
            }
        }
    if (mt == np) {
        float s[16] = {};
#pragma unroll
        for (int t = 1; t < 16; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (k * 8 + t2 + (e & 1) < t && (e >> 1) * 8 + r >= t) s[t] += z[0][k][e];
        // over all lanes: a half of the sums goes to the other half of the lanes each time
#pragma unroll
        for (int m = 16; m > 1; m >>= 1)
#pragma unroll
            for (int t = 0; t < m / 2; ++t) {
                const bool upper = lane & m;
                const float keep = upper ? s[t + m / 2] : s[t], give = upper ? s[t] : s[t + m / 2];
                s[t] = keep + __shfl_xor_sync(0xffffffffu, give, m);
            }
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
        if (!(lane & 1)) out[lane >> 1] = s[0];
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        row[i] += __shfl_xor_sync(0xffffffffu, row[i], 1);
        row[i] += __shfl_xor_sync(0xffffffffu, row[i], 2);
        if (t2 == 0) out[i * 8 + r] = row[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        col[i] = over_rows(col[i]);
        if (r == 0) out[16 + (i >> 1) * 8 + t2 + (i & 1)] = col[i];
    }
    __syncwarp();
    float s = out[lane];
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) {
        const float on = __shfl_down_sync(0xffffffffu, s, m, 16), back = __shfl_up_sync(0xffffffffu, s, m, 16);
        if (lane < 16 ? lane + m < 16 : lane - 16 >= m) s += lane < 16 ? on : back;
    }
    out[lane] = s;
}

// dg of a block's tokens as the sums of what lies across their decays, in lane l those of tokens 31 - l and 63 - l: the states'
// terms of the rows (shares: with S, with R), the pairs' sums, and the two states' product. By a warp.
template <int TB, int D>
__device__ __noinline__ float2 sums_of_decays(const float2* shares, const float* pairs, float whole, int lane) {
    constexpr int MT = TB / 16, N = TB / 32;
    float by_s[N] = {}, by_r[N] = {}, dg[2] = {};
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int w = 0; w < D / 16; ++w) {
            const float2 y = shares[w * TB + k * 32 + 31 - lane];
            by_s[k] += y.x, by_r[k] += y.y;
        }
    float later = 0.f, earlier = 0.f;  // of the other groups
#pragma unroll
    for (int k = N - 1; k >= 0; --k) {
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, by_s[k], m);
            if (lane >= m) by_s[k] += x;
        }
        by_s[k] += later;
        later = __shfl_sync(0xffffffffu, by_s[k], 31);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const float x = __shfl_down_sync(0xffffffffu, by_r[k], m);
            if (lane + m < 32) by_r[k] += x;
        }
        const float all = __shfl_sync(0xffffffffu, by_r[k], 0), before = __shfl_down_sync(0xffffffffu, by_r[k], 1);
        const int j = k * 32 + 31 - lane, at = j / 16, t = j % 16;
        float x = by_s[k] + (lane < 31 ? before : 0.f) + earlier + whole;
        earlier += all;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int np = 0; np <= mt; ++np) {
                // rows from t on, or (on the diagonal) the pairs across t; all of it; columns before t
                const int i = mt == at ? t : np < at ? 31 : 15 + t;
                const float s = pairs[(mt * (mt + 1) / 2 + np) * 32 + i];
                if (mt >= at && np <= at && (mt == at || i != 15)) x += s;
            }
        dg[k] = x;
    }
    return make_float2(dg[0], dg[1]);
}

// A thread's share of <R, S> of two states in memory (in the L2 cache, as the block has read both).
template <int D, int THREADS>
__device__ __noinline__ float dot_of(const float* R, const float* S, int tid) {
    float sum = 0.f;
#pragma unroll 2
    for (int i = tid * 4; i < D * D; i += THREADS * 4) {
        const float4 x = *reinterpret_cast<const float4*>(R + i), s = *reinterpret_cast<const float4*>(S + i);
        sum = fmaf(x.x, s.x, fmaf(x.y, s.y, fmaf(x.z, s.z, fmaf(x.w, s.w, sum))));
    }
    return sum;
}

template <int D, typename T>
__global__ void __launch_bounds__(D * 4) vla_delta_grads_kernel(const __grid_constant__ DeltaArgs p) {
    using L = DeltaGrads<D, T>;
    constexpr int NP = L::NP, TB = L::TB, MT = L::MT, MH = L::MH, LD = L::LD, XLD = L::XLD, UP = L::UP, THREADS = L::THREADS;
    extern __shared__ __align__(128) char sm[];
    const int bh = blockIdx.x / p.blocks, blk = blockIdx.x % p.blocks, b = bh / p.H, h = bh % p.H;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const long long t0 = (long long)blk * TB, n = delta_len(p, b);
    const int rows = (int)min((long long)TB, p.T - t0), live = (int)max(0LL, min((long long)TB, n - t0));
    if (live == 0) {
        const float zero[8] = {};
        for (int i = tid; i < rows * (D / 8); i += THREADS) {
            store8(row_of<T>(p.dq, b, h, t0 + i / (D / 8)) + i % (D / 8) * 8, zero);
            store8(row_of<T>(p.dk, b, h, t0 + i / (D / 8)) + i % (D / 8) * 8, zero);
        }
        for (int i = tid; i < rows; i += THREADS) {
            if (p.dg.p) *p.dg.at(b, h, t0 + i) = 0.f;
            *p.dbeta.at(b, h, t0 + i) = 0.f;
        }
        return;
    }
    // what goes through registers is under way first
    constexpr int EK = TB / 32;  // groups of eight values of E a thread
    Raw8F e_raw[EK];
    float e_beta[EK], share[3] = {}, g_in[TB / 32], b_in[TB / 32];
#pragma unroll
    for (int k = 0; k < EK; ++k) {
        const int i = tid + k * THREADS, row = i / (D / 8), c = i % (D / 8) * 8;
        e_raw[k] = {}, e_beta[k] = 0.f;
        if (row < live) {
            e_raw[k] = raw8(p.E + ((size_t)bh * p.T + t0 + row) * D + c);
            e_beta[k] = *p.beta.at(b, h, t0 + row);
        }
    }
    const int sj = tid % TB, sw = tid / TB;  // the thread's share: a token of 16 rows
    if (sw < D / 16 && sj < live) {
        const size_t i = ((size_t)bh * (D / 16) + sw) * p.T + t0 + sj;
        share[0] = p.od[i], share[1] = p.vd[i], share[2] = p.bd[i];
    }
    if (warp == 0)
#pragma unroll
        for (int k = 0; k < TB / 32; ++k) {
            const int j = k * 32 + lane;
            g_in[k] = j < live && p.g.p ? *p.g.at(b, h, t0 + j) : 0.f;
            b_in[k] = j < live ? *p.beta.at(b, h, t0 + j) : 0.f;
        }
    auto load = [&](int at, const Seq& s) {
#pragma unroll 4
        for (int i = tid; i < TB * (D / 8); i += THREADS) {
            const int row = i / (D / 8), c = i % (D / 8) * 8;
            char* dst = sm + at + (row * LD + c) * 2;
            const T* src = row_of<T>(s, b, h, row < live ? t0 + row : 0) + c;
            if constexpr (NP == 1) {
                cp_async16(vla::smem_u32(dst), src, row < live ? 16 : 0);
            } else {
                float x[8] = {};
                if (row < live) load8(src, x);
                uint32_t w[4][NP];
#pragma unroll
                for (int j = 0; j < 4; ++j) split<NP>(x[2 * j], x[2 * j + 1], w[j]);
#pragma unroll
                for (int q = 0; q < NP; ++q) *reinterpret_cast<uint4*>(dst + q * L::PLANE) = make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
            }
        }
    };
    load(L::O, p.dO);
    load(L::V, p.dv);
    load(L::K, p.k);
    load(L::Q, p.q);
    cp_async_commit();
    const size_t at = ((size_t)bh * (p.blocks + 1) + blk) * D * D;
    auto slice = [&](int i) {  // the i-th 32 rows of S, then of R: 32 bytes a thread
        if (i < D / 16) {
            const float* from = (i < D / 32 ? p.before : p.behind) + at + (size_t)(i % (D / 32)) * 32 * D;
            const uint32_t to = vla::smem_u32(sm + L::RING + i % L::SLICES * L::SLICE);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = tid / (D / 4) + k * 16, c = tid % (D / 4) * 4;
                cp_async16(to + (row * L::SLD + c) * 4, from + row * D + c, 16);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < L::SLICES - 1; ++i) slice(i);
    // the rows' shares of the gates' gradients: o . dO - v . dV and U' . E
    float2* shares = reinterpret_cast<float2*>(sm + L::SHARES);
    if (sw < D / 16) shares[sw * TB + sj] = make_float2(share[0] - share[1], share[2]);
    // gates: the sums of g as two floats, b, exp(G), exp(G_C - G)
    float* gates = reinterpret_cast<float*>(sm + L::GATES);
    if (warp == 0) {
        float hi[TB / 32], lo[TB / 32];
        float all = 0.f, rest = 0.f, up = 0.f;
#pragma unroll
        for (int k = 0; k < TB / 32; ++k) {
            up += fmaxf(g_in[k], 0.f);
            sums_of(g_in[k], lane, hi[k], lo[k]);
            const float s = all + hi[k], d = s - all;
            lo[k] += rest + ((all - (s - d)) + (hi[k] - d));
            hi[k] = s;
            all = __shfl_sync(0xffffffffu, hi[k], 31), rest = __shfl_sync(0xffffffffu, lo[k], 31);
        }
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) up += __shfl_xor_sync(0xffffffffu, up, m);
        const bool grows = TB > 32 && up > 64.f;  // no two tokens are further apart than that
        bool any = false;
#pragma unroll
        for (int k = 0; k < TB / 32; ++k) any |= p.dg.p && g_in[k] < L::STRONG;
        any = __any_sync(0xffffffffu, any);
        if (lane == 0) *reinterpret_cast<int2*>(sm + L::FLAGS) = make_int2(grows, any);
#pragma unroll
        for (int k = 0; k < TB / 32; ++k) {
            const int j = k * 32 + lane;
            const float near = hi[k] + lo[k], far = (all - hi[k]) + (rest - lo[k]);
            gates[j] = hi[k], gates[TB + j] = lo[k], gates[2 * TB + j] = b_in[k];
            gates[3 * TB + j] = grows ? grow_first(near) : expf(near);
            gates[4 * TB + j] = grows ? grow_first(far) : expf(far);
        }
    }
#pragma unroll
    for (int k = 0; k < EK; ++k) {
        const int i = tid + k * THREADS, row = i / (D / 8), c = i % (D / 8) * 8;
        float x[8];
        open8(e_raw[k], x);
        uint32_t w[4][UP];
#pragma unroll
        for (int j = 0; j < 4; ++j) split<UP>(x[2 * j] * e_beta[k], x[2 * j + 1] * e_beta[k], w[j]);
#pragma unroll
        for (int q = 0; q < UP; ++q)
            *reinterpret_cast<uint4*>(sm + L::U + q * L::PLANE + (row * LD + c) * 2) = make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
    }
    cp_async_wait<L::SLICES - 1>();
    __syncthreads();

    const int r = lane >> 2, t2 = (lane & 3) * 2;
    const uint32_t base = vla::smem_u32(sm);
    const bool grows = TB > 32 && reinterpret_cast<const int*>(sm + L::FLAGS)[0], strong = reinterpret_cast<const int*>(sm + L::FLAGS)[1];
    // X and M, a 16 x 16 block of both at a time
    for (int unit = warp; unit < L::UNITS; unit += THREADS / 32) {
        int mt = 0, np = unit;
        while (np > mt) np -= ++mt;
        float c[2][2][4] = {}, cl[2][2][4] = {};
        const uint32_t a_at = base + (mt * 16 * LD + down_across<LD>(lane)) * 2;
        const uint32_t b_at = base + L::U + (np * 16 * LD + across_down<LD>(lane)) * 2;
#pragma unroll 2
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t a[NP][4], v[NP][4], u[2][UP][2];
#pragma unroll
            for (int q = 0; q < NP; ++q) ldsm(a[q], a_at + L::O + q * L::PLANE + ks * 32);
#pragma unroll
            for (int q = 0; q < NP; ++q) ldsm(v[q], a_at + L::V + q * L::PLANE + ks * 32);
#pragma unroll
            for (int q = 0; q < UP; ++q) ldsm_pair(u, 0, q, b_at + q * L::PLANE + ks * 32);
            mma_tiles<NP>(c[0], cl[0], a, u);
            mma_tiles<NP>(c[1], cl[1], v, u);
        }
        join(c[0], cl[0]);
        join(c[1], cl[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = mt * 16 + hf * 8 + r, j = np * 16 + k * 8 + t2;
                float x[2], m[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float w = expf((gates[i] - gates[j + q]) + (gates[TB + i] - gates[TB + j + q]));
                    x[q] = j + q <= i ? c[0][k][2 * hf + q] * w * p.scale : 0.f;
                    m[q] = j + q < i ? -c[1][k][2 * hf + q] * w : 0.f;
                }
                if (grows)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float a = (gates[i] - gates[j + q]) + (gates[TB + i] - gates[TB + j + q]);
                        x[q] = j + q <= i ? c[0][k][2 * hf + q] * grow_first(a) * p.scale * grow_second(a) : 0.f;
                        m[q] = j + q < i ? -c[1][k][2 * hf + q] * grow_first(a) * grow_second(a) : 0.f;
                    }
                uint32_t w[L::XP], y[L::MP];
                split<L::XP>(x[0], x[1], w);
                split<L::MP>(m[0], m[1], y);
#pragma unroll
                for (int q = 0; q < L::XP; ++q) *reinterpret_cast<uint32_t*>(sm + L::X + q * L::XPLANE + (i * XLD + j) * 2) = w[q];
#pragma unroll
                for (int q = 0; q < L::MP; ++q) *reinterpret_cast<uint32_t*>(sm + L::M + q * L::XPLANE + (i * XLD + j) * 2) = y[q];
            }
        if (__builtin_expect(strong, false)) sums_across<L, D>(reinterpret_cast<float*>(sm + L::PAIRS) + unit * 32, sm, mt, np, lane);
    }
    // The gates' gradients, the sums of the rows' shares: dbeta, and dlog_decay's sums from the last token of a 32 on. The
    // last warp has no pairs, or few.
    float dg_hi[TB / 32] = {}, dg_lo[TB / 32] = {}, bad = 0.f;
    if (warp == THREADS / 32 - 1) {
#pragma unroll
        for (int k = 0; k < TB / 32; ++k) {
            const int j = k * 32 + 31 - lane;
            float db = 0.f;
#pragma unroll
            for (int w = 0; w < D / 16; ++w) {
                const float2 y = shares[w * TB + j];
                dg_hi[k] += y.x;
                db += y.y;
            }
            running_sums(dg_hi[k], dg_lo[k], lane);
            if (j >= rows) continue;
            bad = fmaf(db, 0.f, bad);
            *p.dbeta.at(b, h, t0 + j) = db;
        }
    }

    // dq and dk of the warp's 16 columns at its tokens: first the states
    const int col0 = warp % (D / 16) * 16, m0 = warp / (D / 16) * MH;
    // <R, S> behind the block: R as it passes, S from memory, where the next block's S is the same
    float4 behind[2];
    float dot = 0.f, across = 0.f;  // ... and of S before the block
    const int own_row = tid / (D / 4), own_col = tid % (D / 4) * 4;
    auto load_behind = [&](int i) {
#pragma unroll
        for (int k = 0; k < 2; ++k) behind[k] = *reinterpret_cast<const float4*>(p.before + at + (size_t)(D + i * 32 + own_row + k * 16) * D + own_col);
    };
    load_behind(0);
    float dq[MH][2][4] = {}, dk[MH][2][4] = {}, small[3][MH][2][4] = {};
    float(&ql)[MH][2][4] = NP > 1 ? small[0] : dq;  // fp32 results: the small products apart
    float(&kl)[MH][2][4] = NP > 1 ? small[1] : dk;
    // the parts of the i-th 16 rows of the states at the warp's columns, as B operands
    auto state_of = [&](int i, auto& w) {
        constexpr int N = sizeof(w) / 16;
        if (i % 2 == 0) {
            cp_async_wait<L::SLICES - 2>();
            __syncthreads();
            slice(i / 2 + L::SLICES - 1);  // in the place of the one before, which everyone has read
        }
        const float* S = reinterpret_cast<const float*>(sm + L::RING + i / 2 % L::SLICES * L::SLICE) + i % 2 * 16 * L::SLD + col0 + r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float* at = S + ((k & 1) * 8 + t2) * L::SLD + (k >> 1) * 8;
            uint32_t x[N];
            split<N>(at[0], at[L::SLD], x);
#pragma unroll
            for (int q = 0; q < N; ++q) w[q][k] = x[q];
        }
    };
    const uint32_t rows_at = base + (m0 * 16 * LD + down_across<LD>(lane)) * 2;
#pragma unroll 2
    for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t w[UP][4];
        state_of(ks, w);
#pragma unroll
        for (int m = 0; m < MH; ++m) {
            uint32_t a[NP][4];
#pragma unroll
            for (int q = 0; q < NP; ++q) ldsm(a[q], rows_at + L::O + q * L::PLANE + (m * 16 * LD + ks * 16) * 2);
            mma_parts<NP>(dq[m][0], ql[m][0], a, w, 0);
            mma_parts<NP>(dq[m][1], ql[m][1], a, w, 1);
#pragma unroll
            for (int q = 0; q < NP; ++q) ldsm(a[q], rows_at + L::V + q * L::PLANE + (m * 16 * LD + ks * 16) * 2);
            mma_parts<NP>(dk[m][0], kl[m][0], a, w, 0);
            mma_parts<NP>(dk[m][1], kl[m][1], a, w, 1);
        }
    }
    {
        float y[MH][2][4] = {};
        float(&yl)[MH][2][4] = NP > 1 ? small[2] : y;
#pragma unroll 2
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t w[UP][4];
            state_of(D / 16 + ks, w);
            if (ks % 2 == 0) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 x = *reinterpret_cast<const float4*>(
                        sm + L::RING + (D / 32 + ks / 2) % L::SLICES * L::SLICE + ((own_row + k * 16) * L::SLD + own_col) * 4);
                    dot = fmaf(x.x, behind[k].x, fmaf(x.y, behind[k].y, fmaf(x.z, behind[k].z, fmaf(x.w, behind[k].w, dot))));
                }
                if (ks / 2 + 1 < D / 32) load_behind(ks / 2 + 1);
            }
#pragma unroll
            for (int m = 0; m < MH; ++m) {
                uint32_t a[UP][4];
#pragma unroll
                for (int q = 0; q < UP; ++q) ldsm(a[q], rows_at + L::U + q * L::PLANE + (m * 16 * LD + ks * 16) * 2);
                mma_parts<UP>(y[m][0], yl[m][0], a, w, 0);
                mma_parts<UP>(y[m][1], yl[m][1], a, w, 1);
            }
        }
        if constexpr (NP > 1)
#pragma unroll
            for (int m = 0; m < MH; ++m)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dq[m][k][e] += ql[m][k][e], dk[m][k][e] += kl[m][k][e], y[m][k][e] += yl[m][k][e];
                        ql[m][k][e] = kl[m][k][e] = 0.f;
                    }
        if (grows)
#pragma unroll
            for (int m = 0; m < MH; ++m)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int i = (m0 + m) * 16 + hf * 8 + r;
                    const float near = grow_second(gates[i] + gates[TB + i]),
                                far = grow_second((gates[TB - 1] - gates[i]) + (gates[2 * TB - 1] - gates[TB + i]));
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 2 * hf; e < 2 * hf + 2; ++e) dq[m][k][e] *= near, dk[m][k][e] *= near, y[m][k][e] *= far;
                }
        if (__builtin_expect(strong, false)) {  // the states' terms of a token, for the decays that they lie across
#pragma unroll
            for (int m = 0; m < MH; ++m)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int i = (m0 + m) * 16 + hf * 8 + r;
                    const float near = gates[3 * TB + i], far = gates[4 * TB + i];
                    float by_s = 0.f, by_r = 0.f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int e = 2 * hf;
                        const float2 qv = two_of<NP, L::PLANE>(sm + L::Q + (i * LD + col0 + k * 8 + t2) * 2),
                                     kv = two_of<NP, L::PLANE>(sm + L::K + (i * LD + col0 + k * 8 + t2) * 2);
                        by_s = fmaf(qv.x, p.scale * near * dq[m][k][e], fmaf(qv.y, p.scale * near * dq[m][k][e + 1], by_s));
                        by_s = fmaf(-kv.x, near * dk[m][k][e], fmaf(-kv.y, near * dk[m][k][e + 1], by_s));
                        by_r = fmaf(kv.x, far * y[m][k][e], fmaf(kv.y, far * y[m][k][e + 1], by_r));
                    }
#pragma unroll
                    for (int x = 1; x < 4; x <<= 1) by_s += __shfl_xor_sync(0xffffffffu, by_s, x), by_r += __shfl_xor_sync(0xffffffffu, by_r, x);
                    if (t2 == 0) shares[col0 / 16 * TB + i] = make_float2(by_s, by_r);
                }
        }
#pragma unroll
        for (int m = 0; m < MH; ++m)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = (m0 + m) * 16 + (e >> 1) * 8 + r;
                    dq[m][k][e] *= p.scale * gates[3 * TB + i];
                    dk[m][k][e] = fmaf(gates[4 * TB + i], y[m][k][e], -gates[3 * TB + i] * dk[m][k][e]);
                }
    }
    if (__builtin_expect(strong, false)) across = dot_of<D, THREADS>(p.behind + at, p.before + at, tid);
    float* ends = reinterpret_cast<float*>(sm + L::ENDS);
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m), across += __shfl_xor_sync(0xffffffffu, across, m);
    if (lane == 0) ends[warp] = dot, ends[D / 8 + warp] = across;
    __syncthreads();  // X and M are complete
    if (warp == THREADS / 32 - 1) {  // dlog_decay: what is behind the block and the tokens' sums
        float end_in = lane < THREADS / 32 ? ends[lane] : 0.f;
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) end_in += __shfl_xor_sync(0xffffffffu, end_in, m);
        float after = __shfl_sync(0xffffffffu, end_in, 0), rest = 0.f;
        float2 sums = make_float2(0.f, 0.f);
        if (strong) {
            float whole = lane < D / 8 ? ends[D / 8 + lane] : 0.f;
#pragma unroll
            for (int m = 1; m < 16; m <<= 1) whole += __shfl_xor_sync(0xffffffffu, whole, m);
            whole = __shfl_sync(0xffffffffu, whole, 0) * gates[4 * TB - 1];
            if (grows) whole *= grow_second(gates[TB - 1] + gates[2 * TB - 1]);
            sums = sums_of_decays<TB, D>(shares, reinterpret_cast<const float*>(sm + L::PAIRS), whole, lane);
        }
#pragma unroll
        for (int k = TB / 32 - 1; k >= 0; --k) {
            const int j = k * 32 + 31 - lane;
            const float s = after + dg_hi[k], d = s - after, lo = dg_lo[k] + (rest + ((after - (s - d)) + (dg_hi[k] - d)));
            float x = s + lo;
            after = __shfl_sync(0xffffffffu, s, 31), rest = __shfl_sync(0xffffffffu, lo, 31);
            if (j >= rows || !p.dg.p) continue;
            if (strong && j < live && *p.g.at(b, h, t0 + j) < L::STRONG) x = k ? sums.y : sums.x;
            if (j >= live || (!p.S0 && t0 + j == 0)) x = 0.f;
            bad = fmaf(x, 0.f, bad);
            *p.dg.at(b, h, t0 + j) = x;
        }
    }
    // ... then the pairs
#pragma unroll 1
    for (int ks = 0; ks < MT; ++ks) {
        uint32_t kk[NP][4], qq[NP][4];
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            ldsm_t(kk[q], base + L::K + q * L::PLANE + (ks * 16 * LD + col0 + down_across<LD>(lane)) * 2);
            ldsm_t(qq[q], base + L::Q + q * L::PLANE + (ks * 16 * LD + col0 + down_across<LD>(lane)) * 2);
        }
#pragma unroll
        for (int m = 0; m < MH; ++m) {
            const int mt = m0 + m;
            uint32_t x[L::XP][4], y[L::MP][4];
            if (mt >= ks) {  // rows mt of X and M, columns ks
#pragma unroll
                for (int q = 0; q < L::XP; ++q) ldsm(x[q], base + L::X + q * L::XPLANE + (mt * 16 * XLD + ks * 16 + down_across<XLD>(lane)) * 2);
#pragma unroll
                for (int q = 0; q < L::MP; ++q) ldsm(y[q], base + L::M + q * L::XPLANE + (mt * 16 * XLD + ks * 16 + down_across<XLD>(lane)) * 2);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    mma_parts<L::XP>(dq[m][k], ql[m][k], x, kk, k);
                    mma_parts<L::MP>(dk[m][k], kl[m][k], y, kk, k);
                }
            }
            if (mt <= ks) {  // rows ks, columns mt, transposed
#pragma unroll
                for (int q = 0; q < L::XP; ++q) ldsm_t(x[q], base + L::X + q * L::XPLANE + (ks * 16 * XLD + mt * 16 + across_down<XLD>(lane)) * 2);
#pragma unroll
                for (int q = 0; q < L::MP; ++q) ldsm_t(y[q], base + L::M + q * L::XPLANE + (ks * 16 * XLD + mt * 16 + across_down<XLD>(lane)) * 2);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    mma_parts<L::XP>(dk[m][k], kl[m][k], x, qq, k);
                    mma_parts<L::MP>(dk[m][k], kl[m][k], y, kk, k);
                }
            }
        }
    }
    if constexpr (NP > 1) {
#pragma unroll
        for (int m = 0; m < MH; ++m) join(dq[m], ql[m]), join(dk[m], kl[m]);
    }
#pragma unroll
    for (int m = 0; m < MH; ++m)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int i = (m0 + m) * 16 + hf * 8 + r;
            if (i >= rows) continue;
            T *yq = row_of<T>(p.dq, b, h, t0 + i) + col0 + t2, *yk = row_of<T>(p.dk, b, h, t0 + i) + col0 + t2;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float2 vq = make_float2(dq[m][k][2 * hf], dq[m][k][2 * hf + 1]), vk = make_float2(dk[m][k][2 * hf], dk[m][k][2 * hf + 1]);
                if (i >= live) vq = vk = make_float2(0.f, 0.f);
                bad = fmaf(vq.x, 0.f, fmaf(vq.y, 0.f, fmaf(vk.x, 0.f, fmaf(vk.y, 0.f, bad))));
                if constexpr (NP == 1) {
                    *reinterpret_cast<uint32_t*>(yq + k * 8) = pack_bf16(vq.x, vq.y);
                    *reinterpret_cast<uint32_t*>(yk + k * 8) = pack_bf16(vk.x, vk.y);
                } else {
                    *reinterpret_cast<float2*>(yq + k * 8) = vq;
                    *reinterpret_cast<float2*>(yk + k * 8) = vk;
                }
            }
        }
    if (bad != bad && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, (int)t0);
}

}  // namespace vla_layer
