// vla_delta_tc.cuh -- the gated delta rule over a sequence (vla_delta.cuh) on the
// tcgen05 tensor cores, bf16 inputs: outputs and final state, or (TAPE) what its
// gradients need of it. A block per head (R = 64 of d = 128: two) takes DC = 32
// tokens at a time, its R rows of S on the TMEM lanes:
//
//   [X | Y][x][i] = sum_y S[x][y] [k_i | q_i][y]     A: S in three bf16 parts (Y: its first two), TMEM
//   Z[x][j]  = v_j[x] - exp(G_j) X[x][j]
//   E[x][i]  = sum_j Z[x][j] Inv[i][j]               A: Z in three parts; Inv in three, six products
//   T[x][y]  = sum_j (b_j exp(G_C - G_j) E[x][j]) k_j[y]    A: in three parts
//   S        = exp(G_C) S + T                        fp32, in registers
//   o_i[x]   = scale exp(G_i) Y[x][i] + sum_j b_j E[x][j] P[i][j]   A: b E in two parts, P in two
//
// The workers' fragments of S, Z and E are what tcgen05.ld and st move (16x256b,
// 16x128b) and what ldmatrix gives of v, so that nothing but o and the helpers' small
// matrices passes through shared memory.
//
// What bounds it: the chain S, X, Z, E, T, S of a chunk, three products that
// wait for the workers and the workers for them. So S goes out and comes in by
// pieces of its columns, the products of the first beside the work on the next,
// and o is formed beside the next chunk's X.
//
// Warps: the workers (16 rows, a half of the columns and of the tokens each, 8 or
// 16 of them), one for the MMAs, one for loads, and behind them two groups of three
// with the helpers' part, two chunks ahead.
// Every wait on an mbarrier is bounded; one that runs out raises the block's abort flag. What has no limit of its own is the
// allocation of tensor memory, which waits for another block on the SM that holds some (another stream's call), and that
// block's waits are bounded.
//
// Measured: a chunk of 32 tokens takes 1.4 us at d = 64, 2.2 at d = 96 and 2.75 at d = 128 with a head to a block, 1.72
// at d = 128 with two blocks to a head, however many blocks run: 8 x 16 heads of 4,096 tokens 180, 286 and 353 us (60 us
// of memory traffic at d = 96), 32 heads of 32,768 tokens, d = 128, 1,757 us. The tensor cores are busy for 29 to 45% of
// it and the schedulers issue in 66% of the cycles of d = 96 (the workers' cutting into parts), 48% of 64 rows.
// Chunks of 32 tokens, as a group of helpers is longer at a chunk's pairs and inverse than the workers at the chunk, and
// that work grows with the square of its tokens. What came before, prompt d = 96 and long d = 128: the warp-level path with
// loads and matrices in the workers 623 and 4,200 us, in helper warps 407 and 2,668, two warps for 16 rows 421 and 1,936;
// this path with eight workers of plain loads 377 and 2,513, TMA, a second group of helpers and 16 workers 305 and 1,721,
// the outputs later (LATE) 275. Then for accuracy: two parts of S and P for o, 279 and 1,755; a sum of its own for X's
// small parts, 284 and 1,757.
#pragma once

#include "vla_delta.cuh"
#include "vla_tcgen.cuh"

namespace vla_layer {

struct DeltaMaps {
    CUtensorMap m[4];  // k, q, v, dO in boxes of 64 columns x 32 tokens, 128-byte swizzle
};

template <int D, int R, bool TAPE>
struct DeltaTc {
    static constexpr int NB = D > 64 ? 2 : 1, VB = R / 64;  // boxes of 64 columns x 32 tokens
    static constexpr int BOX = DC * 128;
    static constexpr int NST = 4;
    // a stage: for each box of d, K and Q; V (and dO) at the block's rows
    static constexpr int V = NB * 2 * BOX, O = V + VB * BOX, STAGE = O + (TAPE ? VB * BOX : 0);
    // parts of S, P and b E on their way to o, whose terms are then 2^-14 off at most (one part of S and of P would leave o
    // 2.4e-3 off, where its own rounding gives 1.65e-3)
    static constexpr int OP = TAPE ? 3 : 2;
    // a chunk's matrices, two of 64 columns: the inverse's parts 0 | 1, its 2 | P's 0, P's 1 | 2; gates
    static constexpr int MATS = 3 * BOX, PREP = MATS + 1024;
    // chunks' matrices: a chunk's are free once its outputs are formed, behind the next one's Z or (LATE) behind its E, and two
    // groups of helpers work on two at a time
    static constexpr int NPR = 4, GROUPS = 2, SCRATCH = (2 * 16 * NLD + 3 * 3 * DC) * 4;
    static constexpr int PREPS = NST * STAGE, N = PREPS + NPR * PREP, OUT = N + GROUPS * SCRATCH;
    static constexpr int OUT_LD = 24;                      // elements of a row of a warp's staged outputs
    static constexpr int NW = R / 8;                       // workers
    static constexpr int BAR = OUT + NW * 16 * OUT_LD * 2;
    static constexpr int NBAR = NST + 2 * NPR + 10, MISC = BAR + NBAR * 8, BYTES = MISC + 16;
    static_assert(BYTES <= 227 * 1024, "shared memory");
    static constexpr int W = D / 2;                        // a worker's columns
    static constexpr int PIECES = (W + 31) / 32;
    // TMEM columns; E takes X's place once Z is made of it, and what T is made of Z's. X's products with the small parts of S
    // have a sum of their own, as the tensor cores cut a sum off at every addition (S was up to 6e-7 off with one, a state and
    // keys of one sign, d = 128): where T's first 32 columns are, which are in registers before the next chunk's X begins.
    static constexpr int SB = 0, ZP = SB + 3 * (D / 2), UPC = ZP + 48, X = UPC + OP * 16, PO = X + 64, TC = PO + 32, XS = TC, COLS = 512;
    static_assert(TC + D <= COLS, "tensor memory");
    static constexpr int THREADS = (NW + 8) * 32;
    __host__ __device__ static constexpr int stage_of(int c) { return c % NST * STAGE; }  // the stage of a chunk
};

// Address of 16 bytes in a box: row `row`, group `j` of eight values
__device__ __forceinline__ uint32_t in_box(int row, int j) { return (uint32_t)(row * 128 + ((j ^ (row & 7)) << 4)); }

// prepare_chunk() for tiles in boxes, by a group of three warps; matrices in rows of i, or (BACK: of 1 + diag(b) N) of j.
template <typename L, int D, bool BACK>
__device__ __forceinline__ void prepare_boxes(char* scratch, uint32_t stage, char* prep, float g, float beta, float scale, Whole& whole,
                                              int group, int hw, int lane) {
    float Gh, Gl;
    sums_of(g, lane, Gh, Gl);
    const int mt = hw ? 1 : 0, np = hw == 2 ? 1 : 0;
    const int down = lane & 15, across = (lane & 7) + ((lane >> 4) << 3);  // rows of a 16 x 16 block for its four 8 x 8 ones
    float c[4][4] = {};  // K K^T, Q K^T
    // rolled: the roles' code of a scheduler is more than its instruction cache
#pragma unroll 1
    for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t box = stage + (ks >> 2) * 2 * L::BOX;
        uint32_t a[1][4], q[1][4], b[2][1][2];
        const uint32_t at = in_box(mt * 16 + down, (ks & 3) * 2 + (lane >> 4));
        ldsm(a[0], box + at);
        ldsm(q[0], box + L::BOX + at);
        ldsm_pair(b, 0, 0, box + in_box(np * 16 + across, (ks & 3) * 2 + ((lane >> 3) & 1)));
        mma_tiles<1>(c, c, a, b);
        mma_tiles<1>(c + 2, c + 2, q, b);
    }
    const int r = lane >> 2, t2 = (lane & 3) * 2;
    float* own = reinterpret_cast<float*>(scratch) + 2 * 16 * NLD + hw * 3 * DC;  // the sums of g and b of each token
    own[lane] = Gh, own[DC + lane] = Gl, own[2 * DC + lane] = beta;
    __syncwarp();
    float* N = reinterpret_cast<float*>(scratch) + (hw >> 1) * 16 * NLD;  // BACK, else transposed
    auto part_at = [&](int part, int row, int j8) {  // eight values of a part of the inverse
        return in_box(row, (part & 1) * 4 + j8) + (part >> 1) * L::BOX;
    };
    float x[2][4];
    uint32_t pw[4][L::OP];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int j = np * 16 + n * 8 + t2;
        const float2 gj = *reinterpret_cast<const float2*>(own + j), lj = *reinterpret_cast<const float2*>(own + DC + j),
                     bj = *reinterpret_cast<const float2*>(own + 2 * DC + j);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int i = mt * 16 + hf * 8 + r;
            const float gi = own[i], li = own[DC + i];
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float w = exp2f(((gi - (e ? gj.y : gj.x)) + (li - (e ? lj.y : lj.x))) * 1.4426950408889634f);
                x[n][2 * hf + e] = j + e < i ? c[n][2 * hf + e] * w * (BACK ? own[2 * DC + i] : e ? bj.y : bj.x) : 0.f;
                y[e] = j + e <= i ? c[2 + n][2 * hf + e] * w * scale : 0.f;
                if (hw != 1) N[BACK ? (hf * 8 + r) * NLD + n * 8 + t2 + e : (n * 8 + t2 + e) * NLD + hf * 8 + r] = x[n][2 * hf + e];
            }
            split<L::OP>(y[0], y[1], pw[2 * n + hf]);
            if constexpr (!BACK)
#pragma unroll
                for (int p = 0; p < L::OP; ++p)  // behind the inverse's three parts
                    *reinterpret_cast<uint32_t*>(prep + part_at(3 + p, i, np * 2 + n) + t2 * 2) = pw[2 * n + hf][p];
        }
    }
    if constexpr (BACK)
#pragma unroll
        for (int p = 0; p < L::OP; ++p)
            stsm_t(vla::smem_u32(prep) + part_at(3 + p, np * 16 + across, mt * 2 + ((lane >> 3) & 1)), pw[0][p], pw[1][p], pw[2][p], pw[3][p]);
    if (hw != 1) {
        __syncwarp();
        float t[16];
        const int row = lane & 15;
        if constexpr (BACK) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {  // (1 + N) T = 1, a lane a column
                float s = i == row ? 1.f : 0.f, s2 = 0.f;
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
        } else
#pragma unroll
        for (int j = 15; j >= 0; --j) {  // T (1 + N) = 1, a lane a row
            float s = j == row ? 1.f : 0.f, s2 = 0.f;
#pragma unroll
            for (int m = j / 4 * 4; m < 16; m += 4) {
                const float4 w = *reinterpret_cast<const float4*>(N + j * NLD + m);
                if (m > j) s2 = fmaf(-w.x, t[m], s2);
                if (m + 1 > j) s = fmaf(-w.y, t[m + 1], s);
                if (m + 2 > j) s2 = fmaf(-w.z, t[m + 2], s2);
                if (m + 3 > j) s = fmaf(-w.w, t[m + 3], s);
            }
            t[j] = s + s2;
        }
        if (lane < 16) {
            uint32_t w[8][INV_PARTS];
#pragma unroll
            for (int i = 0; i < 8; ++i) split<INV_PARTS>(t[2 * i], t[2 * i + 1], w[i]);
#pragma unroll
            for (int p = 0; p < INV_PARTS; ++p) {
                *reinterpret_cast<uint4*>(prep + part_at(p, mt * 16 + row, mt * 2)) = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
                *reinterpret_cast<uint4*>(prep + part_at(p, mt * 16 + row, mt * 2 + 1)) = make_uint4(w[4][p], w[5][p], w[6][p], w[7][p]);
            }
            if (mt == (BACK ? 1 : 0)) {  // nothing above the diagonal
#pragma unroll
                for (int p = 0; p < INV_PARTS + L::OP; ++p)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<uint4*>(prep + part_at(p, mt * 16 + row, (BACK ? 0 : 2) + k)) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
    vla::named_bar(2 + group, 96);
    if (hw == 0) {
        const float all = __shfl_sync(0xffffffffu, Gh, 31), rest = __shfl_sync(0xffffffffu, Gl, 31);
        float* gates = reinterpret_cast<float*>(prep + L::MATS);
        gates[GATE_NEAR + lane] = expf(Gh + Gl);
        gates[GATE_FAR + lane] = expf((all - Gh) + (rest - Gl));
        gates[GATE_BETA + lane] = beta;
        const float w = whole.next(all + rest);
        if (lane == 0) gates[GATE_WHOLE] = w;
    }
    if (hw != 1) return;
    // T21^T = -(T11^T N21^T) T22^T
    uint32_t a[INV_PARTS][4], w[2][INV_PARTS][2];
    const uint32_t inv = vla::smem_u32(prep);
#pragma unroll
    for (int p = 0; p < INV_PARTS; ++p) {
        if constexpr (BACK)
            ldsm(a[p], inv + part_at(p, down, lane >> 4));
        else
            ldsm_t(a[p], inv + part_at(p, across, (lane >> 3) & 1));
    }
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
    for (int p = 0; p < INV_PARTS; ++p) {
        if constexpr (BACK)
            ldsm_pair_t(w, 0, p, inv + part_at(p, 16 + down, 2 + (lane >> 4)));
        else
            ldsm_pair(w, 0, p, inv + part_at(p, 16 + across, 2 + ((lane >> 3) & 1)));
    }
    mma_tiles<INV_PARTS>(z, zl, a, w);
    join(z, zl);
    // its fragments are rows of j: blocks (j, i), (j + 8, i), (j, i + 8), (j + 8, i + 8)
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[p][e] = -z[p][e];
    uint32_t v[4][INV_PARTS];
#pragma unroll
    for (int i = 0; i < 4; ++i) split<INV_PARTS>(z[i >> 1][(i & 1) * 2], z[i >> 1][(i & 1) * 2 + 1], v[i]);
#pragma unroll
    for (int p = 0; p < INV_PARTS; ++p) {
        if constexpr (BACK)
            stmatrix4(inv + part_at(p, down, 2 + (lane >> 4)), v[0][p], v[1][p], v[2][p], v[3][p]);
        else
            stsm_t(inv + part_at(p, 16 + across, (lane >> 3) & 1), v[0][p], v[1][p], v[2][p], v[3][p]);
    }
}

// 16 lanes, NT tiles of eight 32-bit columns, as fragments
template <int NT>
__device__ __forceinline__ void ld_tiles(uint32_t at, float (*x)[4]) {
    if constexpr (NT == 4) {
        ld_frag32(at, *reinterpret_cast<float(*)[16]>(x));
    } else {
        ld_frag16(at, *reinterpret_cast<float(*)[8]>(x));
    }
}

template <int D, int R, bool TAPE>
__global__ void __launch_bounds__(DeltaTc<D, R, TAPE>::THREADS, 1) vla_delta_tc_kernel(const __grid_constant__ DeltaArgs p,
                                                                                           const __grid_constant__ DeltaMaps maps) {
    using T = __nv_bfloat16;
    using L = DeltaTc<D, R, TAPE>;
    constexpr int SPAN = BLOCK<T>, NW = L::NW, W = L::W, SPLITS = D > R ? D / R : 1;
    extern __shared__ __align__(1024) char delta_sm[];
    char* sm = delta_sm;
    const uint32_t sb = vla::smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
    uint64_t *full = bar, *prep_ready = full + L::NST, *done = prep_ready + L::NPR, *s_ready = done + L::NPR, *x_done = s_ready + 2,
             *z_ready = x_done + 1, *e_done = x_done + 2, *f_ready = x_done + 3, *t_done = x_done + 4, *u_ready = x_done + 5,
             *o_done = x_done + 6, *drained = x_done + 7;
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int bh = blockIdx.x / SPLITS, row0 = blockIdx.x % SPLITS * R, b = bh / p.H, h = bh % p.H;
    const int rows = min(R, D - row0);
    const long long n = delta_len(p, b);
    const int chunks = (int)((n + DC - 1) / DC);

    if (tid == 0) {
        for (int i = 0; i < L::NST; ++i) vla::mbar_init(full + i, 1);
        for (int i = 0; i < L::NPR; ++i) vla::mbar_init(prep_ready + i, 3), vla::mbar_init(done + i, NW);
        for (int i = 0; i < 2; ++i) vla::mbar_init(s_ready + i, NW);
        vla::mbar_init(x_done, 1);
        vla::mbar_init(z_ready, NW);
        vla::mbar_init(e_done, 1);
        vla::mbar_init(f_ready, NW);
        vla::mbar_init(u_ready, NW);
        vla::mbar_init(t_done, 1);
        vla::mbar_init(o_done, 1);
        vla::mbar_init(drained, 1);
        *abort_flag = 0;
        vla::fence_mbar_init();
    }
    if (warp == NW) vla::tc_alloc(tmem_ptr, L::COLS);
    vla::tc_fence_before();
    __syncthreads();
    vla::tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_ptr, 0);
    float bad = 0.f;

    auto wait_warp = [&](uint64_t* w, uint32_t parity) {
        if (__all_sync(0xffffffffu, vla::mbar_try_wait(w, parity & 1))) return true;
        const bool ok = wait_on(w, parity & 1, abort_flag, p.wait_ns, p.status, warp / 4, bh);
        return __all_sync(0xffffffffu, ok) != 0;
    };
    auto arrive_warp = [&](uint64_t* w) {  // one arrival a warp
        __syncwarp();
        if (lane == 0) vla::mbar_arrive(w);
    };

    if (warp == NW) {  // ---- MMAs, issued by one lane of a whole warp
        const bool one = elect_one();
        const uint32_t id64 = idesc_bf16(R, 64, 0, 0), id32 = idesc_bf16(R, 32, 0, 0), id_t = idesc_bf16(R, D, 0, 1);
        const uint64_t dk = desc_sw128(0, 16, 1024), dm = desc_sw128(0, L::NB == 2 ? 2 * L::BOX : 16, 1024);
        auto at = [](uint64_t d, uint32_t addr) { return d + (uint64_t)(addr >> 4); };
        for (int c = 0; c < chunks; ++c) {
            const uint32_t st = sb + L::stage_of(c), pr = sb + L::PREPS + c % L::NPR * L::PREP;
            const uint64_t keys = at(dk, st);
            if (!wait_warp(full + c % L::NST, c / L::NST)) break;
            bool ok = true;
#pragma unroll
            for (int q = 0; q < L::PIECES; ++q) {
                if (!(ok = wait_warp(s_ready + q, c))) break;
                vla::tc_fence_after();
                if (one) {
#pragma unroll
                    for (int part = 0; part < 3; ++part)
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            if (ks % (W / 16) / 2 != q) continue;
                            const uint32_t s = tm + L::SB + part * (D / 2) + ks * 8;
                            const uint64_t box = keys + (((ks >> 2) * 2 * L::BOX + (ks & 3) * 32) >> 4);
                            if (part == 0) {
                                mma_ts(tm + L::X, s, box, id64, q > 0 || ks > 0);
                            } else {
                                mma_ts(tm + L::XS, s, box, id32, q > 0 || part > 1 || ks > 0);
                                if (part < L::OP) mma_ts(tm + L::X + 32, s, box + (L::BOX >> 4), id32, 1);
                            }
                        }
                    if (q + 1 == L::PIECES) vla::tc_commit(x_done);
                }
                __syncwarp();
            }
            if (!ok || !wait_warp(prep_ready + c % L::NPR, c / L::NPR) || !wait_warp(z_ready, c)) break;
            vla::tc_fence_after();
            if (one) {
#pragma unroll
                for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                    for (int q = 0; q <= sum; ++q)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mma_ts(tm + L::X, tm + L::ZP + (sum - q) * 16 + k * 8, at(dk, pr + (q & 1) * 64 + (q >> 1) * L::BOX + k * 32), id32,
                                   !(sum == 2 && q == 0 && k == 0));
                vla::tc_commit(e_done);
            }
            __syncwarp();
            if (!wait_warp(f_ready, c)) break;
            vla::tc_fence_after();
            if (one) {
#pragma unroll
                for (int part = 2; part >= 0; --part)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        mma_ts(tm + L::TC, tm + L::ZP + part * 16 + k * 8, at(dm, st + k * 2048), id_t, !(part == 2 && k == 0));
                vla::tc_commit(t_done);
            }
            __syncwarp();
            if (!wait_warp(u_ready, c)) break;
            vla::tc_fence_after();
            if (one) {
#pragma unroll
                for (int part = L::OP - 1; part >= 0; --part)
#pragma unroll
                    for (int q = 0; q < L::OP; ++q) {
                        if (part + q >= L::OP) continue;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mma_ts(tm + L::PO, tm + L::UPC + part * 16 + k * 8,
                                   at(dk, pr + ((3 + q) & 1) * 64 + ((3 + q) >> 1) * L::BOX + k * 32), id32,
                                   !(part == L::OP - 1 && q == 0 && k == 0));
                    }
                vla::tc_commit(o_done);
            }
            __syncwarp();
        }
        if (one) vla::tc_commit(drained);  // what was issued has finished before the block frees its TMEM
        __syncwarp();
        if (!__all_sync(0xffffffffu, vla::mbar_try_wait(drained, 0))) vla::mbar_wait_slow(drained, 0, nullptr, p.wait_ns);
        __syncwarp();
    } else if (warp == NW + 1) {  // ---- loads
        // Whole chunks by TMA, three ahead; a last one of fewer tokens, whose other rows are zero whatever memory
        // holds there, by plain copies.
        const bool one = elect_one();
        constexpr int TILES = TAPE ? 4 : 3;
        auto load = [&](int c) {
            const long long t0 = (long long)c * DC;
            const int live = (int)min((long long)DC, n - t0);
            const uint32_t st = sb + L::stage_of(c);
            uint64_t* w = full + c % L::NST;
            if (live == DC) {
                if (one) {
                    vla::mbar_arrive_expect_tx(w, (2 * L::NB + (TILES - 2) * L::VB) * L::BOX);
#pragma unroll
                    for (int i = 0; i < L::NB; ++i) {
                        tma_load(st + i * 2 * L::BOX, &maps.m[0], i * 64, (int)t0, h, b, w);
                        tma_load(st + i * 2 * L::BOX + L::BOX, &maps.m[1], i * 64, (int)t0, h, b, w);
                    }
#pragma unroll
                    for (int i = 0; i < L::VB; ++i) {
                        tma_load(st + L::V + i * L::BOX, &maps.m[2], row0 + i * 64, (int)t0, h, b, w);
                        if constexpr (TAPE) tma_load(st + L::O + i * L::BOX, &maps.m[3], row0 + i * 64, (int)t0, h, b, w);
                    }
                }
                __syncwarp();
                return;
            }
#pragma unroll 1
            for (int m = 0; m < TILES; ++m) {
                const Seq& s = m == 0 ? p.k : m == 1 ? p.q : m == 2 ? p.v : p.dO;
                const int boxes = m < 2 ? L::NB : L::VB, cols = m < 2 ? D : rows;
                const uint32_t to = m == 0 ? 0 : m == 1 ? L::BOX : m == 2 ? L::V : L::O;
                for (int i = lane; i < boxes * DC * 8; i += 32) {
                    const int g8 = i % (boxes * 8), r = i / (boxes * 8);
                    const bool on = r < live && g8 * 8 < cols;
                    const T* src = row_of<T>(s, b, h, on ? t0 + r : t0) + (on ? (m < 2 ? 0 : row0) + g8 * 8 : 0);
                    cp_async16(st + to + (g8 >> 3) * (m < 2 ? 2 * L::BOX : L::BOX) + in_box(r, g8 & 7), src, on ? 16 : 0);
                }
            }
            cp_async_commit();
            cp_async_wait<0>();
            vla::fence_proxy_async_smem();
            arrive_warp(w);
        };
        int loaded = 0;
        for (; loaded < chunks; ++loaded) {
            const int before = loaded - L::NST;  // the stage's last chunk
            if (before >= 0 && !wait_warp(done + before % L::NPR, before / L::NPR)) break;
            if (!(p.stall && loaded + 1 == chunks)) load(loaded);
        }
        if (*abort_flag)  // leave only once the copies under way have landed
            for (int c = max(0, loaded - L::NST); c < loaded && !(p.stall && c + 1 == chunks); ++c) {
                if (!__all_sync(0xffffffffu, vla::mbar_try_wait(full + c % L::NST, (c / L::NST) & 1)))
                    vla::mbar_wait_slow(full + c % L::NST, (c / L::NST) & 1, nullptr, p.wait_ns);
                __syncwarp();
            }
    } else if (warp >= NW + 2) {  // ---- the helpers' part, two groups for every other chunk
        const int group = (warp - NW - 2) / 3, hw = (warp - NW - 2) % 3;
        Whole whole;
        float g = 0.f, beta = 0.f;
        auto gates = [&](int c) {
            const long long t = (long long)c * DC + lane;
            g = t < n && p.g.p ? *p.g.at(b, h, t) : 0.f;
            beta = t < n ? *p.beta.at(b, h, t) : 0.f;
        };
        gates(group);
        for (int c = group; c < chunks; c += L::GROUPS) {
            const float gc = g, bc = beta;
            gates(c + L::GROUPS);
            // the three warps that meet at a barrier leave together if a wait ran out
            const bool ok = wait_warp(full + c % L::NST, c / L::NST) && (c < L::NPR || wait_warp(done + c % L::NPR, c / L::NPR - 1));
            if (vla::bar_red_or(2 + group, 96, !ok)) break;
            prepare_boxes<L, D, false>(sm + L::N + group * L::SCRATCH, sb + L::stage_of(c), sm + L::PREPS + c % L::NPR * L::PREP, gc, bc, p.scale,
                                whole, group, hw, lane);
            vla::fence_proxy_async_smem();
            arrive_warp(prep_ready + c % L::NPR);
        }
    } else if (warp < NW) {  // ---- S
        const int quad = warp & 3, half = (warp >> 2) & 1, r = lane >> 2, t2 = (lane & 3) * 2;
        const int xb = quad * (R / 4) + (warp >> 3) * 16;   // first of the warp's 16 rows in the block
        const bool rows_in = xb < rows;                     // else zero throughout
        const uint32_t lanes = tm + ((uint32_t)(quad * 32 + (warp >> 3) * 16) << 16);
        float s[W / 8][4];
        load_rows<D, W>(s, p.S0 && rows_in ? p.S0 + ((size_t)bh * D + row0 + xb) * D + half * W : nullptr, lane);
        char* stage = sm + L::OUT + warp * 16 * L::OUT_LD * 2;
        // a piece of S in three parts
        auto publish = [&](int q) {
            constexpr int NT = W % 32 == 0 ? 4 : 2;
#pragma unroll
            for (int k0 = 0; k0 < 4; k0 += NT) {
                if (q * 4 + k0 >= W / 8) continue;
                uint32_t v[3][2 * NT];
#pragma unroll
                for (int k = 0; k < NT; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t y[3];
                        split<3>(s[q * 4 + k0 + k][2 * e], s[q * 4 + k0 + k][2 * e + 1], y);
#pragma unroll
                        for (int i = 0; i < 3; ++i) v[i][2 * k + e] = y[i];
                    }
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint32_t to = lanes + L::SB + i * (D / 2) + half * (W / 2) + (q * 4 + k0) * 4;
                    if constexpr (NT == 4)
                        st_frag8(to, *reinterpret_cast<const uint32_t(*)[8]>(v[i]));
                    else
                        st_frag4(to, v[i][0], v[i][1], v[i][2], v[i][3]);
                }
            }
        };
        auto ready = [&](uint64_t* w) {
            vla::tc_wait_st();
            vla::tc_fence_before();
            arrive_warp(w);
        };
        auto parts16 = [&](auto nc, uint32_t col, const float (&x)[2][4]) {  // 16 rows x 16 tokens
            constexpr int N = decltype(nc)::value;
            uint32_t y[4][N];
#pragma unroll
            for (int i = 0; i < 4; ++i) split<N>(x[i >> 1][(i & 1) * 2], x[i >> 1][(i & 1) * 2 + 1], y[i]);
#pragma unroll
            for (int i = 0; i < N; ++i) st_frag4(col + i * 16 + half * 8, y[0][i], y[1][i], y[2][i], y[3][i]);
        };
        if (chunks > 0) {
#pragma unroll
            for (int q = 0; q < L::PIECES; ++q) {
                __syncwarp();
                publish(q);
                ready(s_ready + q);
            }
        }
        // this warp's 16 columns of a chunk's tile at its 16 tokens
        auto columns = [&](int c, int tile, float (&x)[2][4]) {
            const int g16 = xb / 16;
            uint32_t w[4];
            ldsm_t(w, sb + L::stage_of(c) + tile + (g16 >> 2) * L::BOX +
                          in_box(half * 16 + (lane & 7) + ((lane >> 4) << 3), (g16 & 3) * 2 + ((lane >> 3) & 1)));
#pragma unroll
            for (int i = 0; i < 2; ++i)
                x[i][0] = low_of(w[2 * i]), x[i][1] = high_of(w[2 * i]), x[i][2] = low_of(w[2 * i + 1]), x[i][3] = high_of(w[2 * i + 1]);
        };
        float o[2][4];
        // Chunk c's outputs, from its share of the state in o and of the pairs: to the warp's buffer, or (TAPE) o . dO
        T* dst = TAPE ? nullptr : row_of<T>(p.out, b, h, half * 16 + lane / 2) + row0 + xb + lane % 2 * 8;
        float* od = TAPE ? p.od + ((size_t)bh * (D / 16) + (row0 + xb) / 16) * p.T + half * 16 : nullptr;
        // 16 workers with 48 columns each are longer at them than the products of E last, and not than those of T (8 x 16 heads of
        // 4,096 tokens, d = 96: 315 us, 287 late); others are not (d = 64: 182, 185; 32 heads, d = 128: 226, 232; 128 heads, d =
        // 128: 354, 360), nor are the gradients', which write nothing (d = 64 707, 713; d = 96 1,273, 1,285; d = 128 1,647, 1,649)
        constexpr bool LATE = D == 96 && !TAPE;
        auto add_pairs = [&](int c) {
            if (!wait_warp(o_done, c)) return false;
            vla::tc_fence_after();
            __syncwarp();
            float x[2][4];
            ld_tiles<2>(lanes + L::PO + half * 16, x);
            vla::tc_wait_ld();
            vla::tc_fence_before();
            join(o, x);
            return true;
        };
        auto output = [&](int c) {
            const int live = (int)min(16LL, n - (long long)c * DC - half * 16);
            if constexpr (TAPE) {
                float d[2][4];
                columns(c, L::O, d);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float y = over_rows(fmaf(o[i][e], d[i][e], o[i][2 + e] * d[i][2 + e]));
                        if (lane < 4 && rows_in && i * 8 + t2 + e < live) od[(size_t)c * DC + i * 8 + t2 + e] = y;
                    }
            } else {
                if (live < 16)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (i * 8 + t2 + (e & 1) >= live) o[i][e] = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) bad = fmaf(o[i][e], 0.f, bad);
                __syncwarp();
                stsm_t(vla::smem_u32(stage) + across_down<L::OUT_LD>(lane) * 2, pack_bf16(o[0][0], o[0][1]), pack_bf16(o[0][2], o[0][3]),
                       pack_bf16(o[1][0], o[1][1]), pack_bf16(o[1][2], o[1][3]));
                __syncwarp();
            }
            arrive_warp(done + c % L::NPR);
        };
        // ... and from there to their rows, up to T
        auto write_out = [&](int c) {
            if constexpr (!TAPE) {
                if (rows_in && (long long)c * DC + half * 16 + lane / 2 < p.T)
                    *reinterpret_cast<uint4*>(dst + (long long)c * DC * p.out.st) =
                        *reinterpret_cast<const uint4*>(stage + (lane / 2 * L::OUT_LD + lane % 2 * 8) * 2);
            }
        };
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const long long t0 = (long long)c * DC;
            if constexpr (TAPE) {
                if (t0 % SPAN == 0 && rows_in)
                    store_rows<D, W>(s, p.before + (((size_t)bh * (p.blocks + 1) + t0 / SPAN) * D + row0 + xb) * D + half * W, lane);
            }
            const float* gates = reinterpret_cast<const float*>(sm + L::PREPS + c % L::NPR * L::PREP + L::MATS) + half * 16;
            if (!(ok = wait_warp(prep_ready + c % L::NPR, c / L::NPR))) break;  // behind its loads
            float2 near[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) near[i] = *reinterpret_cast<const float2*>(gates + GATE_NEAR + i * 8 + t2);
            {
                float x[2][4], small[2][4], v[2][4];
                columns(c, L::V, v);
                if (c > 1) write_out(c - 2);
                if (!(ok = wait_warp(x_done, c))) break;
                vla::tc_fence_after();
                __syncwarp();
                uint32_t here = lanes + half * 16;  // formed here: held from chunk to chunk, the addresses leave no register for s
                asm volatile("" : "+r"(here));
                ld_tiles<2>(here + L::X, x);
                ld_tiles<2>(here + L::XS, small);
                vla::tc_wait_ld();
                join(x, small);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[i][e] = fmaf(-(e & 1 ? near[i].y : near[i].x), x[i][e], v[i][e]);
                parts16(std::integral_constant<int, 3>{}, lanes + L::ZP, x);
            }
            ready(z_ready);
            if (c > 0) {  // beside the products of E: the chunk before's pairs, and (see LATE) what becomes of its outputs
                if (!(ok = add_pairs(c - 1))) break;
                if (!LATE) output(c - 1);
            }
            if (!(ok = wait_warp(e_done, c))) break;
            vla::tc_fence_after();
            __syncwarp();
            {
                float u[2][4], f[2][4];
                ld_tiles<2>(lanes + L::X + half * 16, u);
                vla::tc_wait_ld();
                float2 beta[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 far = *reinterpret_cast<const float2*>(gates + GATE_FAR + i * 8 + t2);
                    beta[i] = *reinterpret_cast<const float2*>(gates + GATE_BETA + i * 8 + t2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[i][e] = u[i][e] * (e & 1 ? beta[i].y : beta[i].x) * (e & 1 ? far.y : far.x);
                }
                parts16(std::integral_constant<int, 3>{}, lanes + L::ZP, f);
                ready(f_ready);
                __syncwarp();
                if constexpr (TAPE) {
                    const long long h0 = t0 + half * 16;
                    if (rows_in) {
                        float* E = p.E + ((size_t)bh * p.T + h0) * D + row0 + xb + r;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = i * 8 + t2 + (e & 1);
                                if (h0 + j < n) E[(size_t)j * D + (e & 2) * 4] = u[i][e];
                            }
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[i][e] *= e & 1 ? beta[i].y : beta[i].x;
                parts16(std::integral_constant<int, L::OP>{}, lanes + L::UPC, u);
                ready(u_ready);
            }
            // beside the products of T: this chunk's share of the state in its outputs
            if (LATE && c > 0) output(c - 1);
            __syncwarp();
            ld_tiles<2>(lanes + L::X + 32 + half * 16, o);
            vla::tc_wait_ld();
            vla::tc_fence_before();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= p.scale * (e & 1 ? near[i].y : near[i].x);
            const float whole = gates[GATE_WHOLE - half * 16];
            if (!(ok = wait_warp(t_done, c))) break;
            vla::tc_fence_after();
#pragma unroll
            for (int q = 0; q < L::PIECES; ++q) {
                constexpr int NT = W % 32 == 0 ? 4 : 2;
                __syncwarp();
                float y[4][4];
#pragma unroll
                for (int k0 = 0; k0 < 4; k0 += NT)
                    if (q * 4 + k0 < W / 8) ld_tiles<NT>(lanes + L::TC + half * W + (q * 4 + k0) * 8, y + k0);
                vla::tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int e = 0; e < 4; e += 2)
                        if (q * 4 + k < W / 8) {
                            float* to = s[q * 4 + k] + e;
                            const float2 w = __ffma2_rn(make_float2(whole, whole), make_float2(to[0], to[1]), make_float2(y[k][e], y[k][e + 1]));
                            to[0] = w.x, to[1] = w.y;
                        }
                if (c + 1 < chunks) {
                    publish(q);
                    ready(s_ready + q);
                }
            }
        }
        if (ok && chunks > 1) write_out(chunks - 2);
        if (ok && chunks > 0 && (ok = add_pairs(chunks - 1))) {
            output(chunks - 1);
            write_out(chunks - 1);
        }
        if (ok && rows_in) {
            float* to = TAPE ? p.before + ((size_t)bh * (p.blocks + 1) + (n + SPAN - 1) / SPAN) * D * D : p.S + (size_t)bh * D * D;
            store_rows<D, W>(s, to + (size_t)(row0 + xb) * D + half * W, lane);
            if constexpr (!TAPE) {
#pragma unroll
                for (int m = 0; m < W / 8; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) bad = fmaf(s[m][e], 0.f, bad);
            }
        }
    }
    if constexpr (!TAPE) zero_tokens<T>(p.out, b, h, (long long)chunks * DC, p.T, row0, rows);
    if (bad != bad && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, 0);
    vla::tc_fence_before();
    __syncthreads();
    if (warp == NW) {
        vla::tc_fence_after();
        vla::tc_dealloc(tm, L::COLS);
    }
}

// The reverse recurrence (vla_delta_backward.cuh) in the same way, R rows of the states' gradient (R here, S in the code) on
// the lanes; X, D and Z with j against i:
//
//   X[x][j] = sum_y R[x][y] k_j[y],   D[x][j] = sum_i dO_i[x] P[i][j]     A of D: dO from shared memory
//   Z[x][j] = exp(G_C - G_j) X[x][j] + D[x][j],   U'[x][j] = sum_i Z[x][i] Inv[i][j]
//   T[x][y] = sum_i (scale exp(G_i) dO_i[x]) q_i[y] - sum_j (b_j exp(G_j) U'[x][j]) k_j[y]    A: both in three parts
//   R       = exp(G_C) R + T
template <int D>
struct ReverseTmem {
    static constexpr int SB = 0, ZP = SB + 3 * (D / 2), A2 = ZP + 48, X = A2 + 48, XS = X + 32, PD = XS + 32, TC = PD + 32;
    static_assert(TC + D <= 512, "tensor memory");
};

template <int D, int R>
__global__ void __launch_bounds__(DeltaTc<D, R, true>::THREADS, 1) vla_delta_tc_reverse_kernel(const __grid_constant__ DeltaArgs p,
                                                                                           const __grid_constant__ DeltaMaps maps) {
    using T = __nv_bfloat16;
    using L = DeltaTc<D, R, true>;
    using M = ReverseTmem<D>;
    constexpr int SPAN = BLOCK<T>, NW = L::NW, W = L::W, SPLITS = D > R ? D / R : 1;
    extern __shared__ __align__(1024) char delta_sm[];
    char* sm = delta_sm;
    const uint32_t sb = vla::smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
    uint64_t *full = bar, *prep_ready = full + L::NST, *done = prep_ready + L::NPR, *s_ready = done + L::NPR, *x_done = s_ready + 2,
             *z_ready = x_done + 1, *e_done = x_done + 2, *f_ready = x_done + 3, *t_done = x_done + 4,
             *drained = x_done + 5;
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int bh = blockIdx.x / SPLITS, row0 = blockIdx.x % SPLITS * R, b = bh / p.H, h = bh % p.H;
    const int rows = min(R, D - row0);
    const long long n = delta_len(p, b);
    const int chunks = (int)((n + DC - 1) / DC);

    if (tid == 0) {
        for (int i = 0; i < L::NST; ++i) vla::mbar_init(full + i, 1);
        for (int i = 0; i < L::NPR; ++i) vla::mbar_init(prep_ready + i, 3), vla::mbar_init(done + i, NW);
        for (int i = 0; i < 2; ++i) vla::mbar_init(s_ready + i, NW);
        vla::mbar_init(x_done, 1);
        vla::mbar_init(z_ready, NW);
        vla::mbar_init(e_done, 1);
        vla::mbar_init(f_ready, NW);
        vla::mbar_init(t_done, 1);
        vla::mbar_init(drained, 1);
        *abort_flag = 0;
        vla::fence_mbar_init();
    }
    if (warp == NW) vla::tc_alloc(tmem_ptr, L::COLS);
    vla::tc_fence_before();
    __syncthreads();
    vla::tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_ptr, 0);
    float bad = 0.f;

    auto wait_warp = [&](uint64_t* w, uint32_t parity) {
        if (__all_sync(0xffffffffu, vla::mbar_try_wait(w, parity & 1))) return true;
        const bool ok = wait_on(w, parity & 1, abort_flag, p.wait_ns, p.status, warp / 4, bh);
        return __all_sync(0xffffffffu, ok) != 0;
    };
    auto arrive_warp = [&](uint64_t* w) {  // one arrival a warp
        __syncwarp();
        if (lane == 0) vla::mbar_arrive(w);
    };

    if (warp == NW) {  // ---- MMAs, issued by one lane of a whole warp
        const bool one = elect_one();
        const uint32_t id32 = idesc_bf16(R, 32, 0, 0), id_o = idesc_bf16(R, 32, 1, 0), id_t = idesc_bf16(R, D, 0, 1);
        const uint64_t dk = desc_sw128(0, 16, 1024), dm = desc_sw128(0, L::NB == 2 ? 2 * L::BOX : 16, 1024),
                       dx = desc_sw128(0, L::VB == 2 ? L::BOX : 16, 1024);
        auto at = [](uint64_t d, uint32_t addr) { return d + (uint64_t)(addr >> 4); };
        auto part = [](int q) { return (uint32_t)((q & 1) * 64 + (q >> 1) * L::BOX); };
        for (int c = 0; c < chunks; ++c) {
            const uint32_t st = sb + L::stage_of(c), pr = sb + L::PREPS + c % L::NPR * L::PREP;
            if (!wait_warp(full + c % L::NST, c / L::NST) || !wait_warp(prep_ready + c % L::NPR, c / L::NPR)) break;
            vla::tc_fence_after();
            if (one) {  // P^T dO
#pragma unroll
                for (int q = 2; q >= 0; --q)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        mma_ss(tm + M::PD, at(dx, st + L::V + k * 2048), at(dk, pr + part(3 + q) + k * 32), id_o, !(q == 2 && k == 0));
            }
            __syncwarp();
            bool ok = true;
#pragma unroll
            for (int q = 0; q < L::PIECES; ++q) {
                if (!(ok = wait_warp(s_ready + q, c))) break;
                vla::tc_fence_after();
                if (one) {
#pragma unroll
                    for (int i = 0; i < 3; ++i)
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            if (ks % (W / 16) / 2 != q) continue;
                            mma_ts(tm + (i ? M::XS : M::X), tm + M::SB + i * (D / 2) + ks * 8,
                                   at(dk, st + (ks >> 2) * 2 * L::BOX + (ks & 3) * 32), id32, q > 0 || i > 1 || ks > 0);
                        }
                    if (q + 1 == L::PIECES) vla::tc_commit(x_done);
                }
                __syncwarp();
            }
            if (!ok || !wait_warp(z_ready, c)) break;
            vla::tc_fence_after();
            if (one) {
#pragma unroll
                for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                    for (int q = 0; q <= sum; ++q)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mma_ts(tm + M::X, tm + M::ZP + (sum - q) * 16 + k * 8, at(dk, pr + part(q) + k * 32), id32,
                                   !(sum == 2 && q == 0 && k == 0));
                vla::tc_commit(e_done);
#pragma unroll
                for (int i = 2; i >= 0; --i)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        mma_ts(tm + M::TC, tm + M::A2 + i * 16 + k * 8, at(dm, st + L::BOX + k * 2048), id_t, !(i == 2 && k == 0));
            }
            __syncwarp();
            if (!wait_warp(f_ready, c)) break;
            vla::tc_fence_after();
            if (one) {
#pragma unroll
                for (int i = 2; i >= 0; --i)
#pragma unroll
                    for (int k = 0; k < 2; ++k) mma_ts(tm + M::TC, tm + M::ZP + i * 16 + k * 8, at(dm, st + k * 2048), id_t, 1);
                vla::tc_commit(t_done);
            }
            __syncwarp();
        }
        if (one) vla::tc_commit(drained);  // what was issued has finished before the block frees its TMEM
        __syncwarp();
        if (!__all_sync(0xffffffffu, vla::mbar_try_wait(drained, 0))) vla::mbar_wait_slow(drained, 0, nullptr, p.wait_ns);
        __syncwarp();
    } else if (warp == NW + 1) {  // ---- loads
        // Whole chunks by TMA, three ahead; a last one of fewer tokens, whose other rows are zero whatever memory
        // holds there, by plain copies.
        const bool one = elect_one();
        constexpr int TILES = 4;
        auto load = [&](int c) {
            const long long t0 = (long long)(chunks - 1 - c) * DC;
            const int live = (int)min((long long)DC, n - t0);
            const uint32_t st = sb + L::stage_of(c);
            uint64_t* w = full + c % L::NST;
            if (live == DC) {
                if (one) {
                    vla::mbar_arrive_expect_tx(w, (2 * L::NB + (TILES - 2) * L::VB) * L::BOX);
#pragma unroll
                    for (int i = 0; i < L::NB; ++i) {
                        tma_load(st + i * 2 * L::BOX, &maps.m[0], i * 64, (int)t0, h, b, w);
                        tma_load(st + i * 2 * L::BOX + L::BOX, &maps.m[1], i * 64, (int)t0, h, b, w);
                    }
#pragma unroll
                    for (int i = 0; i < L::VB; ++i) {
                        tma_load(st + L::V + i * L::BOX, &maps.m[3], row0 + i * 64, (int)t0, h, b, w);
                        tma_load(st + L::O + i * L::BOX, &maps.m[2], row0 + i * 64, (int)t0, h, b, w);
                    }
                }
                __syncwarp();
                return;
            }
#pragma unroll 1
            for (int m = 0; m < TILES; ++m) {
                const Seq& s = m == 0 ? p.k : m == 1 ? p.q : m == 2 ? p.dO : p.v;
                const int boxes = m < 2 ? L::NB : L::VB, cols = m < 2 ? D : rows;
                const uint32_t to = m == 0 ? 0 : m == 1 ? L::BOX : m == 2 ? L::V : L::O;
                for (int i = lane; i < boxes * DC * 8; i += 32) {
                    const int g8 = i % (boxes * 8), r = i / (boxes * 8);
                    const bool on = r < live && g8 * 8 < cols;
                    const T* src = row_of<T>(s, b, h, on ? t0 + r : t0) + (on ? (m < 2 ? 0 : row0) + g8 * 8 : 0);
                    cp_async16(st + to + (g8 >> 3) * (m < 2 ? 2 * L::BOX : L::BOX) + in_box(r, g8 & 7), src, on ? 16 : 0);
                }
            }
            cp_async_commit();
            cp_async_wait<0>();
            vla::fence_proxy_async_smem();
            arrive_warp(w);
        };
        int loaded = 0;
        for (; loaded < chunks; ++loaded) {
            const int before = loaded - L::NST;  // the stage's last chunk
            if (before >= 0 && !wait_warp(done + before % L::NPR, before / L::NPR)) break;
            if (!(p.stall && loaded + 1 == chunks)) load(loaded);
        }
        if (*abort_flag)  // leave only once the copies under way have landed
            for (int c = max(0, loaded - L::NST); c < loaded && !(p.stall && c + 1 == chunks); ++c) {
                if (!__all_sync(0xffffffffu, vla::mbar_try_wait(full + c % L::NST, (c / L::NST) & 1)))
                    vla::mbar_wait_slow(full + c % L::NST, (c / L::NST) & 1, nullptr, p.wait_ns);
                __syncwarp();
            }
    } else if (warp >= NW + 2) {  // ---- the helpers' part, two groups for every other chunk
        const int group = (warp - NW - 2) / 3, hw = (warp - NW - 2) % 3;
        Whole whole;
        float g = 0.f, beta = 0.f;
        auto gates = [&](int c) {
            const long long t = (long long)(chunks - 1 - c) * DC + lane;
            g = t >= 0 && t < n && p.g.p ? *p.g.at(b, h, t) : 0.f;
            beta = t >= 0 && t < n ? *p.beta.at(b, h, t) : 0.f;
        };
        gates(group);
        for (int c = group; c < chunks; c += L::GROUPS) {
            const float gc = g, bc = beta;
            gates(c + L::GROUPS);
            // the three warps that meet at a barrier leave together if a wait ran out
            const bool ok = wait_warp(full + c % L::NST, c / L::NST) && (c < L::NPR || wait_warp(done + c % L::NPR, c / L::NPR - 1));
            if (vla::bar_red_or(2 + group, 96, !ok)) break;
            prepare_boxes<L, D, true>(sm + L::N + group * L::SCRATCH, sb + L::stage_of(c), sm + L::PREPS + c % L::NPR * L::PREP, gc, bc, p.scale,
                                whole, group, hw, lane);
            vla::fence_proxy_async_smem();
            arrive_warp(prep_ready + c % L::NPR);
        }
    } else if (warp < NW) {  // ---- S
        const int quad = warp & 3, half = (warp >> 2) & 1, r = lane >> 2, t2 = (lane & 3) * 2;
        const int xb = quad * (R / 4) + (warp >> 3) * 16;   // first of the warp's 16 rows in the block
        const bool rows_in = xb < rows;                     // else zero throughout
        const uint32_t lanes = tm + ((uint32_t)(quad * 32 + (warp >> 3) * 16) << 16);
        float s[W / 8][4];
        load_rows<D, W>(s, p.dS_T && rows_in ? p.dS_T + ((size_t)bh * D + row0 + xb) * D + half * W : nullptr, lane);
        char* stage = sm + L::OUT + warp * 16 * L::OUT_LD * 2;
        // a piece of S in three parts
        auto publish = [&](int q) {
            constexpr int NT = W % 32 == 0 ? 4 : 2;
#pragma unroll
            for (int k0 = 0; k0 < 4; k0 += NT) {
                if (q * 4 + k0 >= W / 8) continue;
                uint32_t v[3][2 * NT];
#pragma unroll
                for (int k = 0; k < NT; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t y[3];
                        split<3>(s[q * 4 + k0 + k][2 * e], s[q * 4 + k0 + k][2 * e + 1], y);
#pragma unroll
                        for (int i = 0; i < 3; ++i) v[i][2 * k + e] = y[i];
                    }
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint32_t to = lanes + M::SB + i * (D / 2) + half * (W / 2) + (q * 4 + k0) * 4;
                    if constexpr (NT == 4)
                        st_frag8(to, *reinterpret_cast<const uint32_t(*)[8]>(v[i]));
                    else
                        st_frag4(to, v[i][0], v[i][1], v[i][2], v[i][3]);
                }
            }
        };
        auto ready = [&](uint64_t* w) {
            vla::tc_wait_st();
            vla::tc_fence_before();
            arrive_warp(w);
        };
        auto parts16 = [&](auto nc, uint32_t col, const float (&x)[2][4]) {  // 16 rows x 16 tokens
            constexpr int N = decltype(nc)::value;
            uint32_t y[4][N];
#pragma unroll
            for (int i = 0; i < 4; ++i) split<N>(x[i >> 1][(i & 1) * 2], x[i >> 1][(i & 1) * 2 + 1], y[i]);
#pragma unroll
            for (int i = 0; i < N; ++i) st_frag4(col + i * 16 + half * 8, y[0][i], y[1][i], y[2][i], y[3][i]);
        };
        if (chunks > 0) {
#pragma unroll
            for (int q = 0; q < L::PIECES; ++q) {
                __syncwarp();
                publish(q);
                ready(s_ready + q);
            }
        }
        // this warp's 16 columns of a chunk's tile at its 16 tokens
        auto columns = [&](int c, int tile, float (&x)[2][4]) {
            const int g16 = xb / 16;
            uint32_t w[4];
            ldsm_t(w, sb + L::stage_of(c) + tile + (g16 >> 2) * L::BOX +
                          in_box(half * 16 + (lane & 7) + ((lane >> 4) << 3), (g16 & 3) * 2 + ((lane >> 3) & 1)));
#pragma unroll
            for (int i = 0; i < 2; ++i)
                x[i][0] = low_of(w[2 * i]), x[i][1] = high_of(w[2 * i]), x[i][2] = low_of(w[2 * i + 1]), x[i][3] = high_of(w[2 * i + 1]);
        };
        T* dst = row_of<T>(p.dv, b, h, half * 16 + lane / 2) + row0 + xb + lane % 2 * 8;
        const size_t shares = ((size_t)bh * (D / 16) + (row0 + xb) / 16) * p.T + half * 16;
        auto first_of = [&](int c) { return (long long)(chunks - 1 - c) * DC; };
        // chunk c's dV from the warp's buffer to its rows, up to T
        auto write_out = [&](int c) {
            const long long t0 = first_of(c);
            if (rows_in && t0 + half * 16 + lane / 2 < p.T)
                *reinterpret_cast<uint4*>(dst + t0 * p.dv.st) = *reinterpret_cast<const uint4*>(stage + (lane / 2 * L::OUT_LD + lane % 2 * 8) * 2);
        };
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const long long t0 = first_of(c);
            const int live = (int)min(16LL, n - t0 - half * 16);  // of the warp's tokens
            float e[2][4];
            {
                const float* E = p.E + ((size_t)bh * p.T + t0 + half * 16) * D + row0 + xb + r;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int j = i * 8 + t2 + (k & 1);
                        e[i][k] = rows_in && j < live ? E[(size_t)j * D + (k & 2) * 4] : 0.f;
                    }
            }
            const float* gates = reinterpret_cast<const float*>(sm + L::PREPS + c % L::NPR * L::PREP + L::MATS) + half * 16;
            if (!(ok = wait_warp(prep_ready + c % L::NPR, c / L::NPR))) break;  // behind its loads
            float2 near[2], beta[2];
            {  // scale exp(G) dO for the products with q
                float x[2][4];
                columns(c, L::V, x);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    near[i] = *reinterpret_cast<const float2*>(gates + GATE_NEAR + i * 8 + t2);
                    beta[i] = *reinterpret_cast<const float2*>(gates + GATE_BETA + i * 8 + t2);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[i][k] *= p.scale * (k & 1 ? near[i].y : near[i].x);
                }
                __syncwarp();
                parts16(std::integral_constant<int, 3>{}, lanes + M::A2, x);
            }
            if (c > 0) write_out(c - 1);
            if (!(ok = wait_warp(x_done, c))) break;
            vla::tc_fence_after();
            {
                float x[2][4], small[2][4], y[2][4];
                __syncwarp();
                ld_tiles<2>(lanes + M::X + half * 16, x);
                ld_tiles<2>(lanes + M::XS + half * 16, small);
                ld_tiles<2>(lanes + M::PD + half * 16, y);
                vla::tc_wait_ld();
                join(x, small);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 far = *reinterpret_cast<const float2*>(gates + GATE_FAR + i * 8 + t2);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[i][k] = fmaf(k & 1 ? far.y : far.x, x[i][k], y[i][k]);
                }
                parts16(std::integral_constant<int, 3>{}, lanes + M::ZP, x);
            }
            ready(z_ready);
            // beside the products of U'
            if (rows_in && (c == 0 || (t0 + DC) % SPAN == 0)) {
                const long long blk = t0 / SPAN;
                const size_t own = (((size_t)bh * (p.blocks + 1) + blk) * D + row0 + xb) * D + half * W;
                store_rows<D, W>(s, p.behind + own, lane);
            }
            float v[2][4], u[2][4];
            columns(c, L::O, v);
            if (!(ok = wait_warp(e_done, c))) break;
            vla::tc_fence_after();
            __syncwarp();
            ld_tiles<2>(lanes + M::X + half * 16, u);
            vla::tc_wait_ld();
            {
                float f[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) f[i][k] = u[i][k] * -((k & 1 ? near[i].y : near[i].x) * (k & 1 ? beta[i].y : beta[i].x));
                parts16(std::integral_constant<int, 3>{}, lanes + M::ZP, f);
            }
            ready(f_ready);
            // beside the products of T: dV, and the rows' shares of the gates' gradients
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float bt = k ? beta[i].y : beta[i].x;
                    const float bd = over_rows(fmaf(u[i][k], e[i][k], u[i][2 + k] * e[i][2 + k]));
                    u[i][k] *= bt, u[i][2 + k] *= bt;
                    const float vd = over_rows(fmaf(u[i][k], v[i][k], u[i][2 + k] * v[i][2 + k]));
                    const int j = i * 8 + t2 + k;
                    if (j >= live)
                        u[i][k] = u[i][2 + k] = 0.f;
                    else if (lane < 4 && rows_in)
                        p.bd[shares + t0 + j] = bd, p.vd[shares + t0 + j] = vd;
                    bad = fmaf(u[i][k], 0.f, fmaf(u[i][2 + k], 0.f, bad));
                }
            __syncwarp();
            stsm_t(vla::smem_u32(stage) + across_down<L::OUT_LD>(lane) * 2, pack_bf16(u[0][0], u[0][1]), pack_bf16(u[0][2], u[0][3]),
                   pack_bf16(u[1][0], u[1][1]), pack_bf16(u[1][2], u[1][3]));
            __syncwarp();
            const float whole = gates[GATE_WHOLE - half * 16];
            if (!(ok = wait_warp(t_done, c))) break;
            vla::tc_fence_after();
            arrive_warp(done + c % L::NPR);
#pragma unroll
            for (int q = 0; q < L::PIECES; ++q) {
                constexpr int NT = W % 32 == 0 ? 4 : 2;
                __syncwarp();
                float y[4][4];
#pragma unroll
                for (int k0 = 0; k0 < 4; k0 += NT)
                    if (q * 4 + k0 < W / 8) ld_tiles<NT>(lanes + M::TC + half * W + (q * 4 + k0) * 8, y + k0);
                vla::tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int i = 0; i < 4; i += 2)
                        if (q * 4 + k < W / 8) {
                            float* to = s[q * 4 + k] + i;
                            const float2 w = __ffma2_rn(make_float2(whole, whole), make_float2(to[0], to[1]), make_float2(y[k][i], y[k][i + 1]));
                            to[0] = w.x, to[1] = w.y;
                        }
                if (c + 1 < chunks) {
                    publish(q);
                    ready(s_ready + q);
                }
            }
        }
        if (ok && chunks > 0) write_out(chunks - 1);
        if (ok && rows_in && p.dS0) {
            store_rows<D, W>(s, p.dS0 + ((size_t)bh * D + row0 + xb) * D + half * W, lane);
#pragma unroll
            for (int m = 0; m < W / 8; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) bad = fmaf(s[m][i], 0.f, bad);
        }
    }
    zero_tokens<T>(p.dv, b, h, (long long)chunks * DC, p.T, row0, rows);
    if (bad != bad && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, 0);
    vla::tc_fence_before();
    __syncthreads();
    if (warp == NW) {
        vla::tc_fence_after();
        vla::tc_dealloc(tm, L::COLS);
    }
}

}  // namespace vla_layer
