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
// The rows of S and R (coordinates of v) need nothing of each other. So a pair of
// warps keeps 16 of them in registers, a half of the columns each, as sums of
// warp-level products whose fragments are, cut into bf16 parts, the next product's
// operands: S to K S^T to E to S. Only K S^T, a sum over the columns, goes through
// shared memory between the two; what follows from it for all tokens both form (E),
// and a half of the tokens each what is written (O, dV). Three parts hold an fp32
// value's 24 bits and bf16 inputs are one part as they are, so states, E, dbeta
// and (but for strong decays) dlog_decay are fp32 results. Blocks of fewer rows use more SMs for few heads.
// Four helper warps work a chunk ahead: loads, N, P and the inverse, of which the
// two 16 x 16 blocks on the diagonal are solved a lane a column and joined by products.
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
    unsigned long long wait_ns;
    int stall;              // testing: the last chunk's loads are kept back
    // kept between the launches of a backward call
    float* E;               // [BH][T][d]
    float *before, *behind; // [BH][blocks + 1][d][d]: S before a block of tokens (the last one behind all), R behind it
    float *od, *vd, *bd;    // [BH][d / 16][T]: o . dO, v . dV and U' . E of 16 rows
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

// rows of S of a block at most: two warps for 16, with the helpers' 16 warps or 12
template <int D>
constexpr int MOST_ROWS = D == 128 ? 64 : D;
// (d = 32: registers for two blocks on an SM, 304 heads of 1,024 tokens, fp32 gradients: 429 us and 500)
template <int D>
constexpr int DELTA_THREADS = MOST_ROWS<D> * 4 + HELPERS;

// Shared memory of a block: stages of input tiles, two chunks' pairs and gates, and what pairs of warps exchange.
template <int D, typename T, int TILES, int PP>
struct DeltaLay {
    static constexpr int NP = PARTS<T>;
    static constexpr int LD = D + 8;                       // elements of a tile's row
    static constexpr int PLANE = DC * LD * 2, TILE = NP * PLANE;
    static constexpr int STAGES = NP == 1 ? 3 : 2;
    static constexpr int PAIR = DC * PLD * 2;              // bytes of a part of P or of the inverse
    static constexpr int INV = 0, P = INV_PARTS * PAIR, GATES = P + PP * PAIR, PREP = GATES + 5 * DC * 4;
    static constexpr int IN = 0, PREPS = STAGES * TILES * TILE, N = PREPS + 2 * PREP, SWAP = N + DC * NLD * 4;
    static constexpr int WARPS = MOST_ROWS<D> / 8;
    static constexpr int SWAPS = 24 * 32 * 4;              // of a warp: 16 values of K S^T a lane and 8 of o
    static constexpr int OUT = SWAP + WARPS * SWAPS;
    static constexpr int OUT_LD = 24;                      // elements of a row of a warp's staged outputs
    static constexpr int OUTS = NP == 1 ? 16 * OUT_LD * 2 : 0;
    static constexpr int BYTES = OUT + WARPS * OUTS;
};
// gates of a chunk: exp(G), exp(G_C - G), b of each token, then exp(G_C)
enum { GATE_NEAR = 0, GATE_FAR = DC, GATE_BETA = 2 * DC, GATE_WHOLE = 3 * DC };

// Rows [t0, t0 + DC) of a bf16 sequence to a tile, by a warp; those from `n` on are zero.
template <int LD, typename T>
__device__ __forceinline__ void load_tile(char* tile, const Seq& s, int b, int h, long long t0, int col0, int cols, long long n, int lane) {
    const int per = cols / 8, wide = per <= 2 ? 1 : per <= 4 ? 2 : per <= 8 ? 3 : 4;  // threads of a row, a power of two
    const int c = (lane & ((1 << wide) - 1)) * 8, first = lane >> wide, step = 32 >> wide;
    if (c >= cols) return;
    const int live = (int)min((long long)DC, n - t0);
    const T* src = row_of<T>(s, b, h, t0) + col0 + c;
    char* dst = tile + (first * LD + c) * 2;
#pragma unroll 4
    for (int r = first; r < DC; r += step, dst += step * LD * 2) cp_async16(vla::smem_u32(dst), r < live ? src + r * s.st : src, r < live ? 16 : 0);
}

// The same of an fp32 sequence by the helpers, in two steps: rows to registers, then their parts to the tile, so that the
// loads of several tiles are under way together. The chunk `ahead` tokens on is asked into the L2 cache.
template <int D>
struct Rows32 {
    static constexpr int MOST = D > 64 ? 4 : D / 32;  // rows of a thread at most
    Raw8F x[MOST];
    int c, first, step;

    __device__ __forceinline__ void load(const Seq& s, int b, int h, long long t0, int col0, int cols, long long n, int tid, int ahead) {
        const int per = cols / 8, wide = per <= 2 ? 1 : per <= 4 ? 2 : per <= 8 ? 3 : 4;
        c = (tid & ((1 << wide) - 1)) * 8, first = tid >> wide, step = HELPERS >> wide;
        if (c >= cols) first = DC;
        const int live = (int)min((long long)DC, n - t0);
        const float* src = row_of<float>(s, b, h, t0) + col0 + c;
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            const int r = first + i * step;
            x[i] = {};
            if (r < live) x[i] = raw8(src + r * s.st);
            const long long next = t0 + r + ahead;
            if (r < DC && next >= 0 && next < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + (r + ahead) * s.st));
        }
    }
    template <int LD>
    __device__ __forceinline__ void put(char* tile) const {
        char* dst = tile + (first * LD + c) * 2;
#pragma unroll
        for (int i = 0; i < MOST; ++i, dst += step * LD * 2) {
            if (first + i * step >= DC) break;
            float y[8];
            open8(x[i], y);
            uint32_t w[4][3];
#pragma unroll
            for (int j = 0; j < 4; ++j) split<3>(y[2 * j], y[2 * j + 1], w[j]);
#pragma unroll
            for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4*>(dst + p * DC * LD * 2) = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
        }
    }
};

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

// The sums of hi (+ lo) up to each lane, as two floats whose sum holds 48 bits: a difference of sums far from zero
// keeps its precision.
__device__ __forceinline__ void running_sums(float& hi, float& lo, int lane) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float a = __shfl_up_sync(0xffffffffu, hi, m), al = __shfl_up_sync(0xffffffffu, lo, m);
        if (lane >= m) {
            const float s = a + hi, d = s - a;
            lo += al + ((a - (s - d)) + (hi - d));
            hi = s;
        }
    }
}
// ... of g: exp(-256) is 0
__device__ __forceinline__ void sums_of(float g, int lane, float& hi, float& lo) {
    hi = g < -256.f ? -256.f : g;
    lo = 0.f;
    running_sums(hi, lo, lane);
}

// The helpers' part of a chunk: gates (warp 3), P and the inverse. Warps 0, 1, 2 have the 16 x 16 blocks (0, 0), (1, 0) and
// (1, 1) of both triangles; 0 and 2 invert theirs of 1 + N, a lane a column, 1 joins them: (1 + N)^-1 has -T22 N21 T11
// below. The inverse is kept transposed, [j][i]. ROWS: 1 + diag(b) N, else 1 + N diag(b).
template <typename L, int D, int NP, int PP, bool ROWS>
__device__ __forceinline__ void prepare_chunk(char* sm, const char* kt, const char* qt, char* prep, float g, float beta, float scale,
                                              Whole& whole, int hw, int lane) {
    float Gh, Gl;
    sums_of(g, lane, Gh, Gl);
    if (hw == 3) {
        const float all = __shfl_sync(0xffffffffu, Gh, 31), rest = __shfl_sync(0xffffffffu, Gl, 31);
        float* gates = reinterpret_cast<float*>(prep + L::GATES);
        gates[GATE_NEAR + lane] = expf(Gh + Gl);
        gates[GATE_FAR + lane] = expf((all - Gh) + (rest - Gl));
        gates[GATE_BETA + lane] = beta;
        const float w = whole.next(all + rest);
        if (lane == 0) gates[GATE_WHOLE] = w;
        return;
    }
    const int mt = hw ? 1 : 0, np = hw == 2 ? 1 : 0;
    float c[4][4] = {}, cl[4][4] = {};  // K K^T, Q K^T
    const uint32_t k_at = vla::smem_u32(kt) + (mt * 16 * L::LD + down_across<L::LD>(lane)) * 2;
    const uint32_t q_at = vla::smem_u32(qt) + (mt * 16 * L::LD + down_across<L::LD>(lane)) * 2;
    const uint32_t b_at = vla::smem_u32(kt) + (np * 16 * L::LD + across_down<L::LD>(lane)) * 2;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t a[NP][4], q[NP][4], bb[2][NP][2];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            ldsm(a[p], k_at + p * L::PLANE + ks * 32);
            ldsm(q[p], q_at + p * L::PLANE + ks * 32);
            ldsm_pair(bb, 0, p, b_at + p * L::PLANE + ks * 32);
        }
        mma_tiles<NP>(c, cl, a, bb);
        mma_tiles<NP>(c + 2, cl + 2, q, bb);
    }
    if constexpr (NP > 1) join(c, cl);
    const int r = lane >> 2, t2 = (lane & 3) * 2;
    float* N = reinterpret_cast<float*>(sm + L::N) + (hw >> 1) * 16 * NLD;
    float x[2][4];  // the block's N
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int j = np * 16 + n * 8 + t2;
        float gj[2], lj[2], bj[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            gj[e] = __shfl_sync(0xffffffffu, Gh, j + e), lj[e] = __shfl_sync(0xffffffffu, Gl, j + e);
            bj[e] = __shfl_sync(0xffffffffu, beta, j + e);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int i = mt * 16 + hf * 8 + r;
            const float gi = __shfl_sync(0xffffffffu, Gh, i), li = __shfl_sync(0xffffffffu, Gl, i), bi = __shfl_sync(0xffffffffu, beta, i);
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float w = expf((gi - gj[e]) + (li - lj[e]));
                x[n][2 * hf + e] = j + e < i ? c[n][2 * hf + e] * w * (ROWS ? bi : bj[e]) : 0.f;
                y[e] = j + e <= i ? c[2 + n][2 * hf + e] * w * scale : 0.f;
            }
            uint32_t w[PP];
            split<PP>(y[0], y[1], w);
#pragma unroll
            for (int p = 0; p < PP; ++p) *reinterpret_cast<uint32_t*>(prep + L::P + p * L::PAIR + (i * PLD + j) * 2) = w[p];
            if (hw != 1) *reinterpret_cast<float2*>(N + (hf * 8 + r) * NLD + n * 8 + t2) = make_float2(x[n][2 * hf], x[n][2 * hf + 1]);
        }
    }
    if (hw != 1) {
        __syncwarp();
        float t[16];
        const int col = lane & 15;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == col ? 1.f : 0.f, s2 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 w = *reinterpret_cast<const float4*>(N + i * NLD + m);
                s = fmaf(-w.x, t[m], s);
                if (m + 1 < i) s2 = fmaf(-w.y, t[m + 1], s2);
                if (m + 2 < i) s = fmaf(-w.z, t[m + 2], s);
                if (m + 3 < i) s2 = fmaf(-w.w, t[m + 3], s2);
            }
            t[i] = s + s2;
        }
        if (lane < 16) {
            uint32_t w[8][INV_PARTS];
#pragma unroll
            for (int i = 0; i < 8; ++i) split<INV_PARTS>(t[2 * i], t[2 * i + 1], w[i]);
#pragma unroll
            for (int p = 0; p < INV_PARTS; ++p) {
                uint4* to = reinterpret_cast<uint4*>(prep + L::INV + p * L::PAIR + ((mt * 16 + col) * PLD + mt * 16) * 2);
                to[0] = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
                to[1] = make_uint4(w[4][p], w[5][p], w[6][p], w[7][p]);
            }
        }
    }
    vla::named_bar(2, 96);
    if (hw != 1) return;
    // T21^T = -(T11^T N21^T) T22^T
    uint32_t a[INV_PARTS][4], w[2][INV_PARTS][2];
    const uint32_t inv = vla::smem_u32(prep + L::INV);
#pragma unroll
    for (int p = 0; p < INV_PARTS; ++p) ldsm(a[p], inv + p * L::PAIR + down_across<PLD>(lane) * 2);
#pragma unroll
    for (int n = 0; n < 2; ++n)  // eight rows of N21, their 16 values down
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t y[INV_PARTS];
            split<INV_PARTS>(x[k][2 * n], x[k][2 * n + 1], y);
#pragma unroll
            for (int p = 0; p < INV_PARTS; ++p) w[n][p][k] = y[p];
        }
    float y[2][4] = {}, yl[2][4] = {}, z[2][4] = {}, zl[2][4] = {};
    mma_tiles<INV_PARTS>(y, yl, a, w);
    join(y, yl);
    to_operand<INV_PARTS>(a, y[0], y[1]);
#pragma unroll
    for (int p = 0; p < INV_PARTS; ++p) ldsm_pair_t(w, 0, p, inv + p * L::PAIR + (16 * PLD + 16 + down_across<PLD>(lane)) * 2);
    mma_tiles<INV_PARTS>(z, zl, a, w);
    join(z, zl);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            uint32_t v[INV_PARTS];
            split<INV_PARTS>(-z[n][2 * hf], -z[n][2 * hf + 1], v);
#pragma unroll
            for (int p = 0; p < INV_PARTS; ++p)
                *reinterpret_cast<uint32_t*>(prep + L::INV + p * L::PAIR + ((hf * 8 + r) * PLD + 16 + n * 8 + t2) * 2) = v[p];
        }
}

// Fragments (16 rows of S, eight columns a tile, W in all) from and to [..][D] float32 rows.
template <int D, int W>
__device__ __forceinline__ void load_rows(float (&s)[W / 8][4], const float* m, int lane) {
    const int r = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
    for (int n = 0; n < W / 8; ++n) {
        const float2 a = m ? *reinterpret_cast<const float2*>(m + r * D + n * 8 + t2) : make_float2(0.f, 0.f);
        const float2 b = m ? *reinterpret_cast<const float2*>(m + (r + 8) * D + n * 8 + t2) : make_float2(0.f, 0.f);
        s[n][0] = a.x, s[n][1] = a.y, s[n][2] = b.x, s[n][3] = b.y;
    }
}
template <int D, int W>
__device__ __forceinline__ void store_rows(const float (&s)[W / 8][4], float* m, int lane) {
    const int r = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
    for (int n = 0; n < W / 8; ++n) {
        *reinterpret_cast<float2*>(m + r * D + n * 8 + t2) = make_float2(s[n][0], s[n][1]);
        *reinterpret_cast<float2*>(m + (r + 8) * D + n * 8 + t2) = make_float2(s[n][2], s[n][3]);
    }
}

// X^T (16 rows x 32 tokens) = S A^T over W columns of S and of a tile's 32 rows A, and of the first SP parts of S and a
// second tile Y^T = S A2^T (SP 0: none). `at`: the tiles with across_down.
template <int W, int LD, int NP, int SP, int PLANE>
__device__ __forceinline__ void times_rows(float (&x)[4][4], float (&y)[4][4], const float (&s)[W / 8][4], uint32_t at, uint32_t at2) {
    float xl[4][4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] = 0.f, y[i][e] = SP ? 0.f : y[i][e];
#pragma unroll
    for (int ks = 0; ks < W / 16; ++ks) {
        uint32_t a[3][4], b[4][NP][2];
        to_operand<3>(a, s[2 * ks], s[2 * ks + 1]);
#pragma unroll
        for (int np = 0; np < 2; ++np)
#pragma unroll
            for (int p = 0; p < NP; ++p) ldsm_pair(b, 2 * np, p, at + p * PLANE + (np * 16 * LD + ks * 16) * 2);
        mma_tiles<3>(x, xl, a, b);
        if constexpr (SP > 0) {
#pragma unroll
            for (int np = 0; np < 2; ++np)
#pragma unroll
                for (int p = 0; p < NP; ++p) ldsm_pair(b, 2 * np, p, at2 + p * PLANE + (np * 16 * LD + ks * 16) * 2);
            mma_tiles<SP>(y, y, a, b);
        }
    }
    join(x, xl);
}

// A tile pair of X^T (16 rows x 16 tokens) += U^T of 16 tokens times a 16 x 16 block of WP parts: from its rows (TRANS:
// `at` with down_across) or those of its transpose (with across_down).
template <int WP, int UP, int PAIR, bool TRANS>
__device__ __forceinline__ void times_block(float (*x)[4], float (*xl)[4], const uint32_t (&a)[UP][4], uint32_t at) {
    uint32_t w[2][WP][2];
#pragma unroll
    for (int q = 0; q < WP; ++q) {
        if constexpr (TRANS)
            ldsm_pair_t(w, 0, q, at + q * PAIR);
        else
            ldsm_pair(w, 0, q, at + q * PAIR);
    }
    mma_tiles<UP>(x, xl, a, w);
}

// X^T (16 rows x 32 tokens) += U^T W, W upper triangular (AFTER) or lower, in WP parts: as times_block. a[ks]: U^T of 16
// tokens. The four tiles of the whole block row go first, the two of the other after them.
template <int WP, int UP, int PAIR, bool AFTER, bool TRANS>
__device__ __forceinline__ void times_triangle(float (&x)[4][4], float (&xl)[4][4], const uint32_t (&a)[2][UP][4], uint32_t at) {
    constexpr int ks = AFTER ? 0 : 1, one = 1 - ks;
    auto place = [&](int ks, int np) { return at + (TRANS ? ks * 16 * PLD + np * 16 : np * 16 * PLD + ks * 16) * 2; };
    uint32_t w[4][WP][2], v[2][WP][2];
#pragma unroll
    for (int q = 0; q < WP; ++q) {
#pragma unroll
        for (int np = 0; np < 2; ++np) {
            if constexpr (TRANS)
                ldsm_pair_t(w, 2 * np, q, place(ks, np) + q * PAIR);
            else
                ldsm_pair(w, 2 * np, q, place(ks, np) + q * PAIR);
        }
        if constexpr (TRANS)
            ldsm_pair_t(v, 0, q, place(one, one) + q * PAIR);
        else
            ldsm_pair(v, 0, q, place(one, one) + q * PAIR);
    }
    mma_tiles<UP>(x, xl, a[ks], w);
    mma_tiles<UP>(x + 2 * one, xl + 2 * one, a[one], v);
}

// What a warp gives its pair's other warp: four values a lane at a time.
__device__ __forceinline__ void give(char* swap, int i, const float (&x)[4], int lane) {
    reinterpret_cast<float4*>(swap)[i * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void take(const char* swap, int i, float (&x)[4], int lane) {
    const float4 w = reinterpret_cast<const float4*>(swap)[i * 32 + lane];
    x[0] += w.x, x[1] += w.y, x[2] += w.z, x[3] += w.w;
}
// A warp's half of the tokens.
__device__ __forceinline__ void half_of(float (&y)[2][4], const float (&x)[4][4], int half) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = half ? x[2 + i][e] : x[i][e];
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

// S = whole S + U^T A, U^T (16 rows x 32 tokens) given as fragments, A W columns of a tile's 32 rows: `at` with
// down_across. The products have a sum of their own, which an fp32 addition rounds once into S.
template <int W, int LD, int NP, int PLANE>
__device__ __forceinline__ void add_outer(float (&s)[W / 8][4], float whole, const float (&u)[4][4], uint32_t at) {
    uint32_t a[2][3][4];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) to_operand<3>(a[ks], u[2 * ks], u[2 * ks + 1]);
    constexpr int NT = W % 32 == 0 ? 4 : 2;  // tiles at a time
#pragma unroll
    for (int n0 = 0; n0 < W / 8; n0 += NT) {
        float t[NT][4] = {}, low[NT][4] = {};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            uint32_t b[NT][NP][2];
#pragma unroll
            for (int n = 0; n < NT; n += 2)
#pragma unroll
                for (int p = 0; p < NP; ++p) ldsm_pair_t(b, n, p, at + p * PLANE + ks * 16 * LD * 2 + (n0 + n) * 16);
            mma_tiles<3>(t, low, a[ks], b);
        }
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n0 + k][e] = fmaf(whole, s[n0 + k][e], t[k][e] + low[k][e]);
    }
}

// A warp's fragments (16 columns of d, 16 tokens) to rows of a sequence from t0: rows below n, zeros up to T.
template <typename T, int OUT_LD>
__device__ __forceinline__ void store_tokens(const float (&x)[2][4], char* stage, const Seq& s, int b, int h, long long t0, int col0,
                                             long long n, long long T_, int lane) {
    const int r = lane >> 2, t2 = (lane & 3) * 2;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
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
        // blocks (tokens, columns) as across_down
        stsm_t(vla::smem_u32(stage) + across_down<OUT_LD>(lane) * 2, pack_bf16(x[0][0], x[0][1]), pack_bf16(x[0][2], x[0][3]),
               pack_bf16(x[1][0], x[1][1]), pack_bf16(x[1][2], x[1][3]));
        __syncwarp();
        const int row = lane >> 1, c = (lane & 1) * 8;
        const long long t = t0 + row;
        if (t >= T_) return;
        uint4 w = *reinterpret_cast<const uint4*>(stage + (row * OUT_LD + c) * 2);
        if (t >= n) w = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(row_of<T>(s, b, h, t) + col0 + c) = w;
    }
}

// Zeros for rows [t0, T) of a block's columns.
template <typename T>
__device__ __forceinline__ void zero_tokens(const Seq& s, int b, int h, long long t0, long long T_, int col0, int cols) {
    const float zero[8] = {};
    for (long long t = t0 + threadIdx.x; t < T_; t += blockDim.x) {
        T* row = row_of<T>(s, b, h, t) + col0;
        for (int c = 0; c < cols; c += 8) store8(row + c, zero);
    }
}

// x summed over the eight lanes that hold the same tokens of a fragment
__device__ __forceinline__ float over_rows(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

}  // namespace vla_layer
