// vla_delta.cuh -- the gated delta rule, what its kernels share
// (include/vla_layer.h).
//
//   S_t = a_t S_{t-1} + b_t e_t k_t^T,  e_t = v_t - a_t S_{t-1} k_t,  o_t = scale S_t q_t,  a_t = exp(g_t).
//
// C = 32 tokens at a time, G_i the sum of g up to token i of the chunk, S the
// state before it, rows of K, Q, V, E its tokens:
//
//   N[i][j] = exp(G_i - G_j) k_i . k_j  (j < i),   P[i][j] = scale exp(G_i - G_j) q_i . k_j  (j <= i)
//   E   = (1 + N diag(b))^-1 (V - diag(exp(G)) K S^T)
//   O   = scale diag(exp(G)) Q S^T + P diag(b) E
//   S  <- exp(G_C) S + (diag(b exp(G_C - G)) E)^T K
//
// and against the order of time, R the gradient of the state behind the chunk:
//
//   U'  = (1 + diag(b) N)^-T (P^T dO + diag(exp(G_C - G)) K R^T),   dV = diag(b) U',   db_i = U'_i . E_i
//   R  <- exp(G_C) R + (scale diag(exp(G)) dO)^T Q - (diag(exp(G)) dV)^T K
//
// The rows of S and R (coordinates of v) need nothing of each other. So a warp
// keeps 16 of them in registers, as sums of warp-level products whose fragments
// are, cut into bf16 parts, the next product's operands: S to K S^T to E to S
// without shared memory or a barrier between. Three parts hold an fp32 value's 24
// bits and bf16 inputs are one part as they are, so states, E and gates' gradients
// are fp32 results. Blocks of fewer rows than d use more SMs for few heads.
// Four helper warps work a chunk ahead: loads, N, P and the inverse, of which the
// two 16 x 16 blocks on the diagonal are solved a lane a column and joined.
#pragma once

#include "vla_mma.cuh"

namespace vla_layer {

constexpr int DC = 32;            // tokens of a chunk
constexpr int HELPERS = 128;      // threads that work a chunk ahead
constexpr int PLD = DC + 8;       // elements of a row of P's and the inverse's parts
constexpr int NLD = DC + 4;       // floats of a row of N
constexpr int INV_PARTS = 3;

// a [B, H, T] float32 sequence of gates; data null: none
struct Gate {
    float* p;
    long long sb, sh, st;
    __device__ __forceinline__ float* at(int b, int h, long long t) const { return p + (b * sb + h * sh + t * st); }
};

struct DeltaArgs {
    Seq q, k, v, dO;        // inputs
    Seq out, dq, dk, dv;    // o; the gradients
    Gate g, beta, dg, dbeta;
    const int* lengths;
    const float *S0, *dS_T;
    float *S, *dS0;
    float scale;
    int B, H, T;
    int rows;               // rows of S of a block
    vla::DeviceStatus* status;
    // kept between the launches of a backward call
    float* E;               // [BH][T][d]
    float *before, *behind; // [BH][blocks + 1][d][d]: S before a block of tokens (the last one behind all), R behind it
    float *od, *vd, *bd;    // [BH][d / 16][T]: o . dO, v . dV and U' . E of 16 rows
    float* ends;            // [BH][blocks][d / 16]: <R, S> behind a block, of 16 rows
    int blocks;             // blocks of tokens of a sequence of T
};

__device__ __forceinline__ int delta_len(const DeltaArgs& p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}

// parts of an input value, and tokens of a block that S and R are kept for
template <typename T>
constexpr int PARTS = sizeof(T) == 2 ? 1 : 3;
template <typename T>
constexpr int BLOCK = sizeof(T) == 2 ? 64 : 32;

// Shared memory of a block: stages of input tiles, and two chunks' pairs and gates.
template <int D, typename T, int TILES, int PP>
struct DeltaLay {
    static constexpr int NP = PARTS<T>;
    static constexpr int LD = D + 8;                       // elements of a tile's row
    static constexpr int PLANE = DC * LD * 2, TILE = NP * PLANE;
    static constexpr int STAGES = NP == 1 ? 3 : 2;
    static constexpr int PAIR = DC * PLD * 2;              // bytes of a part of P or of the inverse
    static constexpr int INV = 0, P = INV_PARTS * PAIR, GATES = P + PP * PAIR, PREP = GATES + 5 * DC * 4;
    static constexpr int IN = 0, PREPS = STAGES * TILES * TILE, N = PREPS + 2 * PREP, OUT = N + DC * NLD * 4;
    static constexpr int OUT_LD = 24;                      // elements of a row of a warp's staged outputs
    static constexpr int BYTES = OUT + (D / 16) * DC * OUT_LD * 2;
};
// gates of a chunk: exp(G), exp(G_C - G), b of each token, then exp(G_C)
enum { GATE_NEAR = 0, GATE_FAR = DC, GATE_BETA = 2 * DC, GATE_WHOLE = 3 * DC };

// Rows [t0, t0 + DC) of a sequence's `cols` columns to a tile; those from `n` on are zero.
template <int LD, typename T>
__device__ __forceinline__ void load_tile(char* tile, const Seq& s, int b, int h, long long t0, int col0, int cols, long long n,
                                          int tid) {
    constexpr int NP = PARTS<T>, PLANE = DC * LD * 2;
    const int per = cols / 8;
    for (int i = tid; i < DC * per; i += HELPERS) {
        const int r = i / per, c = i % per * 8;
        char* dst = tile + (r * LD + c) * 2;
        const bool on = t0 + r < n;
        const T* src = row_of<T>(s, b, h, on ? t0 + r : 0) + col0 + c;
        if constexpr (NP == 1) {
            cp_async16(vla::smem_u32(dst), src, on ? 16 : 0);
        } else {
            float x[8] = {};
            if (on) load8(src, x);
            uint32_t w[4][NP];
#pragma unroll
            for (int j = 0; j < 4; ++j) split<NP>(x[2 * j], x[2 * j + 1], w[j]);
#pragma unroll
            for (int p = 0; p < NP; ++p) *reinterpret_cast<uint4*>(dst + p * PLANE) = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
        }
    }
}

// A decay over a chunk that multiplies a state again and again: what the
// roundings of the factors add up to is put right by the next ones (SlowDecay of
// vla_layer.cuh, for factors that differ).
struct Whole {
    float owed = 0.f;
    __device__ __forceinline__ float next(float x) {
        const float m = expm1f(x), w = 1.f + m;
        if (!(w > 0.5f && w < 2.f)) {
            const float v = fmaf(expf(x), owed, expf(x));
            owed = 0.f;
            return v;
        }
        const float inv = 1.f / w;
        owed = fmaf(m - (w - 1.f), inv, owed);
        const float v = fmaf(w, owed, w);
        owed = fmaf(w - v, inv, owed);
        return v;
    }
};

// The helpers' part of a chunk: gates, P and the inverse. Warps 0 and 1 form the rows 0-15 and 16-31 of N, 2 and
// 3 those of P; then warp 0 inverts. ROWS: 1 + diag(b) N, else 1 + N diag(b).
template <typename L, int D, int NP, int PP, bool ROWS>
__device__ __forceinline__ void prepare_chunk(char* sm, const char* kt, const char* qt, char* prep, float g, float beta, float scale,
                                              Whole& whole, int hw, int lane) {
    // the sum of g in 64 bits, as two floats: a difference of sums far from zero keeps its precision
    double G = g < -256.f ? -256.0 : (double)g;  // exp(-256) is 0
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, G, m);
        if (lane >= m) G += x;
    }
    const float Gh = (float)G, Gl = (float)(G - (double)Gh);
    const double all = __shfl_sync(0xffffffffu, G, 31);
    if (hw == 0) {
        float* gates = reinterpret_cast<float*>(prep + L::GATES);
        gates[GATE_NEAR + lane] = expf(Gh);
        gates[GATE_FAR + lane] = expf((float)(all - G));
        gates[GATE_BETA + lane] = beta;
        const float w = whole.next((float)all);
        if (lane == 0) gates[GATE_WHOLE] = w;
    }
    const int mt = hw & 1;
    const bool of_q = hw >= 2;
    float c[4][4] = {}, cl[4][4] = {};
    const uint32_t a_at = vla::smem_u32(of_q ? qt : kt) + (mt * 16 * L::LD + down_across<L::LD>(lane)) * 2;
    const uint32_t b_at = vla::smem_u32(kt) + across_down<L::LD>(lane) * 2;
#pragma unroll 2
    for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t a[NP][4];
#pragma unroll
        for (int p = 0; p < NP; ++p) ldsm(a[p], a_at + p * L::PLANE + ks * 32);
#pragma unroll
        for (int np = 0; np < 2; ++np) {
            if (np > mt) break;
            uint32_t bb[NP][4];
#pragma unroll
            for (int p = 0; p < NP; ++p) ldsm(bb[p], b_at + p * L::PLANE + np * 16 * L::LD * 2 + ks * 32);
            mma_parts<NP>(c[2 * np], cl[2 * np], a, bb, 0);
            mma_parts<NP>(c[2 * np + 1], cl[2 * np + 1], a, bb, 1);
        }
    }
    if constexpr (NP > 1) join(c, cl);
    const int r = lane >> 2, t2 = (lane & 3) * 2;
    float* N = reinterpret_cast<float*>(sm + L::N);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const int i = mt * 16 + hf * 8 + r;
        const float gi = __shfl_sync(0xffffffffu, Gh, i), li = __shfl_sync(0xffffffffu, Gl, i), bi = __shfl_sync(0xffffffffu, beta, i);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float x[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = n * 8 + t2 + e;
                const float gj = __shfl_sync(0xffffffffu, Gh, j), lj = __shfl_sync(0xffffffffu, Gl, j),
                            bj = __shfl_sync(0xffffffffu, beta, j);
                const float w = expf((gi - gj) + (li - lj)) * (of_q ? scale : ROWS ? bi : bj);
                x[e] = (of_q ? j <= i : j < i) ? c[n][2 * hf + e] * w : 0.f;
            }
            if (n >= 2 * (mt + 1)) continue;
            if (of_q) {
                uint32_t w[PP];
                split<PP>(x[0], x[1], w);
#pragma unroll
                for (int p = 0; p < PP; ++p)
                    *reinterpret_cast<uint32_t*>(prep + L::P + p * L::PAIR + (i * PLD + n * 8 + t2) * 2) = w[p];
            } else {
                *reinterpret_cast<float2*>(N + i * NLD + n * 8 + t2) = make_float2(x[0], x[1]);
            }
        }
    }
    vla::named_bar(1, HELPERS);
    if (hw != 0) return;
    // the inverses of both blocks on the diagonal: lane (h, c) has column c of block h
    const int h = lane >> 4, col = lane & 15;
    float x[16];
    const float* Nd = N + h * (16 * NLD + 16);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s = i == col ? 1.f : 0.f, s2 = 0.f;
#pragma unroll
        for (int m = 0; m < i; m += 4) {
            const float4 w = *reinterpret_cast<const float4*>(Nd + i * NLD + m);
            s = fmaf(-w.x, x[m], s);
            if (m + 1 < i) s2 = fmaf(-w.y, x[m + 1], s2);
            if (m + 2 < i) s = fmaf(-w.z, x[m + 2], s);
            if (m + 3 < i) s2 = fmaf(-w.w, x[m + 3], s2);
        }
        x[i] = s + s2;
    }
    // the block below: -T22 (N21 T11), a lane's rows 8 h .. 8 h + 7 of its column
    float y[8] = {};
#pragma unroll
    for (int m = 0; m < 16; m += 4) {
        float t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = __shfl_sync(0xffffffffu, x[m + e], col);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(N + (16 + 8 * h + i) * NLD + m);
            y[i] = fmaf(w.x, t[0], fmaf(w.y, t[1], fmaf(w.z, t[2], fmaf(w.w, t[3], y[i]))));
        }
    }
    __syncwarp();
    if (h == 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) N[(16 + i) * NLD + 16 + col] = x[i];
    }
    __syncwarp();
    float z[8] = {};
#pragma unroll
    for (int m = 0; m < 16; m += 4) {
        float t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = __shfl_sync(0xffffffffu, y[(m + e) & 7], ((m + e) >> 3) * 16 + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(N + (16 + 8 * h + i) * NLD + 16 + m);
            z[i] = fmaf(-w.x, t[0], fmaf(-w.y, t[1], fmaf(-w.z, t[2], fmaf(-w.w, t[3], z[i]))));
        }
    }
    auto put = [&](int i, int j, float v) {
        uint32_t w[INV_PARTS];
        split<INV_PARTS>(v, 0.f, w);
#pragma unroll
        for (int p = 0; p < INV_PARTS; ++p)
            *reinterpret_cast<uint16_t*>(prep + L::INV + p * L::PAIR + (i * PLD + j) * 2) = (uint16_t)w[p];
    };
#pragma unroll
    for (int i = 0; i < 16; ++i) put(16 * h + i, 16 * h + col, x[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) put(16 + 8 * h + i, col, z[i]);
}

// Fragments (16 rows of S, eight columns a tile) from and to [d][d] float32 rows.
template <int D>
__device__ __forceinline__ void load_rows(float (&s)[D / 8][4], const float* m, int lane) {
    const int r = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
        const float2 a = m ? *reinterpret_cast<const float2*>(m + r * D + n * 8 + t2) : make_float2(0.f, 0.f);
        const float2 b = m ? *reinterpret_cast<const float2*>(m + (r + 8) * D + n * 8 + t2) : make_float2(0.f, 0.f);
        s[n][0] = a.x, s[n][1] = a.y, s[n][2] = b.x, s[n][3] = b.y;
    }
}
template <int D>
__device__ __forceinline__ void store_rows(const float (&s)[D / 8][4], float* m, int lane) {
    const int r = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
        *reinterpret_cast<float2*>(m + r * D + n * 8 + t2) = make_float2(s[n][0], s[n][1]);
        *reinterpret_cast<float2*>(m + (r + 8) * D + n * 8 + t2) = make_float2(s[n][2], s[n][3]);
    }
}

// A operand (16 rows x 16 tokens) of N parts from two tiles of fragments.
template <int N>
__device__ __forceinline__ void to_operand(uint32_t (&a)[N][4], const float (&x0)[4], const float (&x1)[4]) {
    uint32_t w[4][N];
    split<N>(x0[0], x0[1], w[0]);
    split<N>(x0[2], x0[3], w[1]);
    split<N>(x1[0], x1[1], w[2]);
    split<N>(x1[2], x1[3], w[3]);
#pragma unroll
    for (int p = 0; p < N; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) a[p][i] = w[i][p];
}

// X^T (16 rows x 32 tokens) = S A^T of a tile's 32 rows A, and of the first SP parts of S and a second tile Y^T =
// S A2^T (SP 0: none). `at`: the tiles with across_down.
template <int D, int LD, int NP, int SP, int PLANE>
__device__ __forceinline__ void times_rows(float (&x)[4][4], float (&y)[4][4], const float (&s)[D / 8][4], uint32_t at, uint32_t at2) {
    float xl[4][4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] = 0.f, y[i][e] = SP ? 0.f : y[i][e];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t a[3][4];
        to_operand<3>(a, s[2 * ks], s[2 * ks + 1]);
#pragma unroll
        for (int np = 0; np < 2; ++np) {
            uint32_t b[NP][4];
#pragma unroll
            for (int p = 0; p < NP; ++p) ldsm(b[p], at + p * PLANE + (np * 16 * LD + ks * 16) * 2);
            mma_parts<3>(x[2 * np], xl[2 * np], a, b, 0);
            mma_parts<3>(x[2 * np + 1], xl[2 * np + 1], a, b, 1);
            if constexpr (SP > 0) {
#pragma unroll
                for (int p = 0; p < NP; ++p) ldsm(b[p], at2 + p * PLANE + (np * 16 * LD + ks * 16) * 2);
                mma_parts<SP>(y[2 * np], a, b, 0);
                mma_parts<SP>(y[2 * np + 1], a, b, 1);
            }
        }
    }
    join(x, xl);
}

// X^T (16 rows x 32 tokens) += U^T W^T (`across`: W's rows, j <= i) or U^T W (else: W's columns), of a lower triangle
// W of WP parts at `at` with across_down, or down_across and ldsm_t.
template <int WP, int UP, int PAIR, bool ACROSS>
__device__ __forceinline__ void times_triangle(float (&x)[4][4], float (&xl)[4][4], const uint32_t (&a)[UP][4], int ks, uint32_t at) {
#pragma unroll
    for (int np = ACROSS ? ks : 0; np < (ACROSS ? 2 : ks + 1); ++np) {
        uint32_t w[WP][4];
#pragma unroll
        for (int q = 0; q < WP; ++q) {
            if constexpr (ACROSS)
                ldsm(w[q], at + q * PAIR + (np * 16 * PLD + ks * 16) * 2);
            else
                ldsm_t(w[q], at + q * PAIR + (ks * 16 * PLD + np * 16) * 2);
        }
        mma_parts<UP>(x[2 * np], xl[2 * np], a, w, 0);
        mma_parts<UP>(x[2 * np + 1], xl[2 * np + 1], a, w, 1);
    }
}

// The values of the 16 rows at two tiles of 8 tokens, as fragments, from a tile's 16 tokens (at: of the warp's
// columns), with ldsm_t; the parts of an fp32 value added up.
template <int NP, int PLANE>
__device__ __forceinline__ void columns_of(float (&x0)[4], float (&x1)[4], uint32_t at) {
#pragma unroll
    for (int p = NP - 1; p >= 0; --p) {
        uint32_t w[4];
        ldsm_t(w, at + p * PLANE);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float f[4] = {low_of(w[i]), high_of(w[i]), low_of(w[2 + i]), high_of(w[2 + i])};
            if (p == NP - 1) {
                x0[2 * i] = f[0], x0[2 * i + 1] = f[1], x1[2 * i] = f[2], x1[2 * i + 1] = f[3];
            } else {
                x0[2 * i] += f[0], x0[2 * i + 1] += f[1], x1[2 * i] += f[2], x1[2 * i + 1] += f[3];
            }
        }
    }
}

// S = whole S + U^T A, U^T (16 rows x 32 tokens) given as fragments, A a tile's 32 rows: `at` with down_across. The
// products have a sum of their own, which an fp32 addition rounds once into S.
template <int D, int LD, int NP, int PLANE>
__device__ __forceinline__ void add_outer(float (&s)[D / 8][4], float whole, const float (&u)[4][4], uint32_t at) {
    uint32_t a[2][3][4];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) to_operand<3>(a[ks], u[2 * ks], u[2 * ks + 1]);
#pragma unroll
    for (int np = 0; np < D / 16; ++np) {
        float t[2][4] = {}, low[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            uint32_t b[NP][4];
#pragma unroll
            for (int p = 0; p < NP; ++p) ldsm_t(b[p], at + p * PLANE + ks * 16 * LD * 2 + np * 32);
            mma_parts<3>(t[0], low[0], a[ks], b, 0);
            mma_parts<3>(t[1], low[1], a[ks], b, 1);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[2 * np + k][e] = fmaf(whole, s[2 * np + k][e], t[k][e] + low[k][e]);
    }
}

// A warp's fragments (16 columns of d, 32 tokens) to rows of a sequence: rows below n, zeros up to T.
template <typename T, int OUT_LD>
__device__ __forceinline__ void store_tokens(const float (&x)[4][4], char* stage, const Seq& s, int b, int h, long long t0, int col0,
                                             long long n, long long T_, int lane) {
    const int r = lane >> 2, t2 = (lane & 3) * 2;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const long long t = t0 + i * 8 + t2 + e;
                if (t >= T_) continue;
                T* row = row_of<T>(s, b, h, t) + col0 + r;
                row[0] = t < n ? x[i][e] : 0.f;
                row[8] = t < n ? x[i][2 + e] : 0.f;
            }
    } else {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i)  // 16 tokens: blocks (tokens, columns) as across_down
            stsm_t(vla::smem_u32(stage) + (i * 16 * OUT_LD + across_down<OUT_LD>(lane)) * 2, pack_bf16(x[2 * i][0], x[2 * i][1]),
                   pack_bf16(x[2 * i][2], x[2 * i][3]), pack_bf16(x[2 * i + 1][0], x[2 * i + 1][1]),
                   pack_bf16(x[2 * i + 1][2], x[2 * i + 1][3]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = i * 16 + (lane >> 1), c = (lane & 1) * 8;
            const long long t = t0 + row;
            if (t >= T_) continue;
            uint4 w = *reinterpret_cast<const uint4*>(stage + (row * OUT_LD + c) * 2);
            if (t >= n) w = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(row_of<T>(s, b, h, t) + col0 + c) = w;
        }
    }
}

// Zeros for rows [t0, T) of a block's columns.
template <typename T>
__device__ __forceinline__ void zero_tokens(const Seq& s, int b, int h, long long t0, long long T_, int col0, int cols) {
    const float zero[8] = {};
    const int per = cols / 8;
    for (long long i = threadIdx.x; i < (T_ - t0) * per; i += blockDim.x)
        store8(row_of<T>(s, b, h, t0 + i / per) + col0 + i % per * 8, zero);
}

// x summed over the eight lanes that hold the same tokens of a fragment
__device__ __forceinline__ float over_rows(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

}  // namespace vla_layer
