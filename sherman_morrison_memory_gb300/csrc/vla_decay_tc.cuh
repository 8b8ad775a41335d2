// vla_decay_tc.cuh -- the operation of vla_decay.cuh on the tcgen05 tensor
// cores, bf16 inputs. A block per (role, head, segment) takes C = 64 tokens at
// a time. Per chunk, with i, j its tokens, n its length, w the decay's powers
// and x, y the coordinates of c and b:
//
//   SC[i][j] = a_i . b_j                               A, B from shared memory
//   P[i][j]  = w_in w^(i-j) SC[i][j] for j <= i, in bf16
//   OE[x][i] = sum_y Sb[x][y] a_i[y],  Sb = bf16(S)     A from TMEM
//   OI[x][i] = sum_j c_j[x] P[i][j]
//   out_i    = OI[.][i] + w_st w^(i+1) OE[.][i]
//   T[x][y]  = sum_j c_j[x] (k_st w^(n-1-j) b_j[y])
//   S[x][y]  = w^n S[x][y] + T[x][y]                    fp32, in registers
//
// All but SC have the state's rows x on the 128 TMEM lanes, so that S is added
// up and turned into the A operand Sb by the lane's own threads, and only P
// (64 x 64) and the decayed b go through shared memory. OI and OE are kept
// apart because their weights would otherwise be one more rounding. The
// decayed b is split in three bf16 parts, which hold its 24 bits: S is an fp32
// result (two parts left it 2e-6 off). P and Sb are rounded to bf16 once: o is
// rounded to bf16 afterwards anyway, and a term meets only one of the two.
//
// d is padded to DP = 64 or 128 columns by TMA's zero fill. Where DP is 64 the
// A operand repeats its 64 rows (stride 0 between its 64-row halves), so that
// lanes 64-127 hold a copy and the output's four warps take half of the tokens
// each. SC uses M = 128 with the upper 64 rows reading what follows the tile
// in shared memory; nothing reads those lanes.
//
// Warps: 0-3 output, 4-11 decayed b and S (half of the columns each), 12-13 P,
// 14 TMA loads, 15 MMA. Every wait is bounded; one that runs out raises the
// block's abort flag.
//
// STATE: only the segment's own state, from zero (b and c).
#pragma once

#include <cuda.h>

#include "vla_decay.cuh"

namespace vla_layer {

struct DecayMaps {
    // [B, H, T, d] in boxes of 64 columns x 64 tokens, 128-byte swizzle
    CUtensorMap m[4];           // the inputs
    CUtensorMap out[MAX_ROLES];  // the roles' outputs
};

template <int D>
struct TcLay {
    static constexpr int C = 64;
    static constexpr int DP = D <= 64 ? 64 : 128;
    static constexpr int NB = DP / 64;         // boxes of a tile
    static constexpr int BOX = C * 128;        // bytes
    static constexpr int TILE = NB * BOX;
    static constexpr int NST = 3;              // chunks in flight
    static constexpr int PARTS = 3;            // of the decayed b
    static constexpr int OCC = DP == 64 ? 2 : 1;
    // buffers of T, of SC with OI behind it, and of P: one each where two blocks share an SM
    static constexpr int NT = DP == 64 ? 1 : 2, NX = NT, NP = NT;
    static constexpr int THREADS = 512;
    // shared memory
    static constexpr int ST = 0;                           // [NST] a | b | c
    static constexpr int KW = ST + NST * 3 * TILE;         // [PARTS]
    static constexpr int P = KW + PARTS * TILE;
    static constexpr int OUT = P + NP * BOX;
    // weights of 64 each: the state to tokens, tokens to the state, pairs by
    // their lag. Tokens behind a chunk's end read into the next table and pairs
    // against the order of time into the one before; what they get is thrown away
    static constexpr int WO = OUT + TILE, WK = WO + 64 * 4, WP = WK + 64 * 4;
    static constexpr int BAR = WP + 64 * 4;
    static constexpr int NBAR = 2 * NST + 2 * NT + 11;
    static constexpr int MISC = BAR + NBAR * 8;
    static constexpr int SMEM = MISC + 16;
    static_assert((SMEM + 1024) * OCC <= 228 * 1024, "shared memory");
    // TMEM columns; OI takes SC's place once P is made of it
    static constexpr int T = 0, SB = T + NT * DP, OE = SB + DP / 2, X = OE + 64;
    static constexpr int COLS = DP == 64 ? 256 : 512;
    static_assert(X + NX * 64 <= COLS, "tensor memory");
};

__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16: fp32 accumulator, bf16 A and B; a_mn, b_mn: operand stored with M (N) contiguous
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, int a_mn, int b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int t, int h, int b,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(t), "r"(h), "r"(b), "r"(vla::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void st_cols8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int t, int h, int b, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(map),
                 "r"(x), "r"(t), "r"(h), "r"(b), "r"(src)
                 : "memory");
}

// true in one lane of a whole warp
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
template <int D, bool STATE>
__global__ void __launch_bounds__(TcLay<D>::THREADS, TcLay<D>::OCC)
    vla_decay_tc_kernel(const __grid_constant__ DecayArgs p, const __grid_constant__ DecayMaps maps, int roles) {
    using L = TcLay<D>;
    extern __shared__ __align__(1024) unsigned char tc_sm[];
    unsigned char* sm = tc_sm;
    const uint32_t sb = vla::smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
    uint64_t *full = bar, *empty = full + L::NST, *t_done = empty + L::NST, *t_free = t_done + L::NT;
    uint64_t *sc_done = t_free + L::NT, *o_done = sc_done + 2, *p_ready = sc_done + 4, *sb_ready = sc_done + 5,
             *oe_done = sc_done + 6, *oe_free = sc_done + 7, *o_free = sc_done + 8, *kw_full = sc_done + 9,
             *drained = sc_done + 10;
    float *WP = reinterpret_cast<float*>(sm + L::WP), *WK = reinterpret_cast<float*>(sm + L::WK),
          *WO = reinterpret_cast<float*>(sm + L::WO);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int ri = blockIdx.x % roles, rest = blockIdx.x / roles;
    const int seg = rest % p.nseg, bh = rest / p.nseg, b = bh / p.H, h = bh % p.H;
    const Role& r = p.role[ri];
    const float g = p.log_decay[h];
    const Span sp = span_of(p, b, seg);
    const bool rev = r.reverse != 0;
    const int chunks = (sp.n + L::C - 1) / L::C;

    // With time, a token's weight towards the state counts from the chunk's
    // end; against it, its weight from the state does: those tables hold the
    // powers 63, 62, .. and a chunk of n tokens begins 64 - n behind.
    if (tid < 64) {
        const int up = tid + 1, down = 63 - tid;
        WK[tid] = r.k_st * decay_pow(g, rev ? up : down);
        WO[tid] = r.w_st * decay_pow(g, rev ? down : up);
        WP[tid] = r.w_in * decay_pow(g, tid);
    }
    for (int i = tid; i < L::NP * L::BOX / 16; i += L::THREADS)  // the pairs that no chunk writes stay zero
        *reinterpret_cast<uint4*>(sm + L::P + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    vla::fence_proxy_async_smem();
    if (tid == 0) {
        for (int i = 0; i < L::NST; ++i) vla::mbar_init(full + i, 1), vla::mbar_init(empty + i, 1);
        for (int i = 0; i < L::NT; ++i) vla::mbar_init(t_done + i, 1), vla::mbar_init(t_free + i, 8);
        for (int i = 0; i < 2; ++i) vla::mbar_init(sc_done + i, 1), vla::mbar_init(o_done + i, 1);
        vla::mbar_init(p_ready, 2);
        vla::mbar_init(sb_ready, 8);
        vla::mbar_init(oe_done, 1);
        vla::mbar_init(oe_free, 4);
        vla::mbar_init(o_free, 4);
        vla::mbar_init(kw_full, 8);
        vla::mbar_init(drained, 1);
        *abort_flag = 0;
        vla::fence_mbar_init();
    }
    if (warp == 15) vla::tc_alloc(tmem_ptr, L::COLS);
    vla::tc_fence_before();
    __syncthreads();
    vla::tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_ptr, 0);
    float2 bad = make_float2(0.f, 0.f);  // NaN once an output or a final state is not finite
    const float2 zero2 = make_float2(0.f, 0.f);

    // bounded wait: false once this or another wait of the block has run out
    auto wait = [&](uint64_t* w, uint32_t parity) {
        if (vla::mbar_wait(w, parity & 1, (const volatile int*)abort_flag, p.wait_ns)) return true;
        if (*abort_flag == 0 && p.status) vla::record_failure(p.status, vla::BIT_TIMEOUT, warp / 4, bh, sp.t0);
        *abort_flag = 1;
        return false;
    };
    auto wait_warp = [&](uint64_t* w, uint32_t parity) { return __all_sync(0xffffffffu, wait(w, parity)) != 0; };
    auto arrive_warp = [&](uint64_t* w) {  // one arrival a warp
        __syncwarp();
        if (lane == 0) vla::mbar_arrive(w);
    };
    // first token (within the segment) of the m-th chunk in the role's order
    auto chunk0 = [&](int m) { return (rev ? chunks - 1 - m : m) * L::C; };

    if (warp == 14) {  // ---- TMA loads
        if (lane == 0) {
            int m = 0;
            for (; m < chunks; ++m) {
                const int st = m % L::NST;
                if (m >= L::NST && !wait(empty + st, m / L::NST - 1)) break;
                const int t = sp.t0 + chunk0(m);
                const uint32_t dst = sb + L::ST + st * 3 * L::TILE;
                vla::mbar_arrive_expect_tx(full + st, (STATE ? 2 : 3) * L::TILE);
                const int id[3] = {r.map_a, r.map_b, r.map_c};
#pragma unroll
                for (int q = STATE ? 1 : 0; q < 3; ++q)
#pragma unroll
                    for (int x = 0; x < L::NB; ++x)
                        tma_load(dst + q * L::TILE + x * L::BOX, &maps.m[id[q]], x * 64, t, h, b, full + st);
            }
            if (*abort_flag)  // leave only once the copies under way have landed
                for (int i = max(0, m - L::NST); i < m; ++i)
                    vla::mbar_wait(full + i % L::NST, (i / L::NST) & 1, nullptr, p.wait_ns);
        }
    } else if (warp == 15) {  // ---- MMA
        // The whole warp runs the loop, so that operands stay in uniform
        // registers, and one elected thread issues: issued under a test of the
        // lane, each MMA took 100 cycles.
        const bool one = elect_one();
        const uint32_t id_k = idesc_bf16(128, 64, 0, 0);    // SC, OE
        const uint32_t id_oi = idesc_bf16(128, 64, 1, 0);
        const uint32_t id_t = idesc_bf16(128, D, 1, 1);
        constexpr uint32_t HALF = L::NB == 2 ? L::BOX : 0;  // second 64 rows of an A operand: the next box, or again
        const uint64_t dk = desc_sw128(0, 16, 1024), dm = desc_sw128(0, HALF, 1024);
        auto at = [](uint64_t d, uint32_t addr) { return d + (uint64_t)(addr >> 4); };
        auto pairs = [&](int m) {  // SC of chunk m
            const uint32_t ta = sb + L::ST + (m % L::NST) * 3 * L::TILE;
            if (!wait_warp(full + m % L::NST, m / L::NST)) return false;
            if (m >= L::NX && !wait_warp(o_free, m - L::NX)) return false;
            vla::tc_fence_after();
            if (one) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k / 4) * L::BOX + (k % 4) * 32;
                    mma_ss(tm + L::X + (m % L::NX) * 64, at(dk, ta + off), at(dk, ta + L::TILE + off), id_k, k > 0);
                }
                vla::tc_commit(sc_done + m % 2);
            }
            __syncwarp();
            return true;
        };
        bool ok = STATE || L::NX == 1 || chunks == 0 || pairs(0);
        for (int m = 0; ok && m < chunks; ++m) {
            const int st = m % L::NST, tbuf = m % L::NT;
            const uint32_t ta = sb + L::ST + st * 3 * L::TILE, tc = ta + 2 * L::TILE;
            if (!wait_warp(kw_full, m)) break;
            if (m >= L::NT && !wait_warp(t_free + tbuf, m / L::NT - 1)) break;
            vla::tc_fence_after();
            if (one) {
#pragma unroll
                for (int part = 0; part < L::PARTS; ++part)
#pragma unroll
                    for (int k = 0; k < L::C / 16; ++k)
                        mma_ss(tm + L::T + tbuf * L::DP, at(dm, tc + k * 2048),
                               at(dm, sb + L::KW + part * L::TILE + k * 2048), id_t, part > 0 || k > 0);
                vla::tc_commit(t_done + tbuf);
            }
            __syncwarp();
            if (!STATE) {
                if (L::NX == 1 && !pairs(m)) break;
                if (!wait_warp(sb_ready, m)) break;
                if (m > 0 && !wait_warp(oe_free, m - 1)) break;
                vla::tc_fence_after();
                if (one) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ts(tm + L::OE, tm + L::SB + k * 8, at(dk, ta + (k / 4) * L::BOX + (k % 4) * 32), id_k, k > 0);
                    vla::tc_commit(oe_done);
                }
                __syncwarp();
                if (L::NX > 1 && m + 1 < chunks && !pairs(m + 1)) break;
                if (!wait_warp(p_ready, m)) break;
                vla::tc_fence_after();
                if (one) {
#pragma unroll
                    for (int k = 0; k < L::C / 16; ++k)
                        mma_ss(tm + L::X + (m % L::NX) * 64, at(dm, tc + k * 2048),
                               at(dk, sb + L::P + (m % L::NP) * L::BOX + k * 32), id_oi, k > 0);
                    vla::tc_commit(o_done + m % 2);
                }
                __syncwarp();
            }
            if (one) vla::tc_commit(empty + st);
            __syncwarp();
        }
        if (one) vla::tc_commit(drained);  // what was issued has finished before the block frees its TMEM
        __syncwarp();
        vla::mbar_wait(drained, 0, nullptr, p.wait_ns);
    } else if (warp >= 12) {  // ---- P
        // Of the four 32 x 32 blocks of pairs the two on the diagonal are cut
        // by it, one is whole and one empty; a warp has two of them in a row.
        if (!STATE) {
            const int rb = warp - 12, i = rb * 32 + lane;
            const uint32_t lanes = (uint32_t)(rb * 32) << 16;
            const bool whole = rb == (rev ? 0 : 1);
            const uint32_t tri = rev ? ~((1u << lane) - 1u) : (2u << lane) - 1u;
            for (int m = 0; m < chunks; ++m) {
                const int n = min(L::C, sp.n - chunk0(m));
                if (!wait_warp(sc_done + m % 2, m / 2)) break;
                const int was = m - L::NP;  // the chunk whose P was here: read by its OI
                if (was >= 0 && !wait_warp(o_done + was % 2, was / 2)) break;
                unsigned char* row = sm + L::P + (m % L::NP) * L::BOX + i * 128;
                vla::tc_fence_after();
#pragma unroll
                for (int blk = 0; blk < 2; ++blk) {
                    if (blk == 1 && !whole) break;
                    const int cb = blk == 0 ? rb : 1 - rb;
                    uint32_t mask = blk == 0 ? tri : 0xFFFFFFFFu;
                    if (n < cb * 32 + 32) mask &= n > cb * 32 ? (1u << (n - cb * 32)) - 1u : 0u;
                    const float* w = rev ? WP + (cb * 32 - i) : WP + (i - cb * 32);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float v[16];
                        __syncwarp();
                        vla::tc_ld16(tm + lanes + L::X + (m % L::NX) * 64 + cb * 32 + q * 16, v);
                        vla::tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int j = q * 16 + e;
                            v[e] = (mask >> j) & 1 ? v[e] * (rev ? w[j] : w[-j]) : 0.f;
                        }
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            *reinterpret_cast<uint4*>(row + (((cb * 4 + q * 2 + c) ^ (i & 7)) << 4)) =
                                make_uint4(pack_bf16(v[c * 8], v[c * 8 + 1]), pack_bf16(v[c * 8 + 2], v[c * 8 + 3]),
                                           pack_bf16(v[c * 8 + 4], v[c * 8 + 5]), pack_bf16(v[c * 8 + 6], v[c * 8 + 7]));
                    }
                }
                vla::tc_fence_before();
                vla::fence_proxy_async_smem();
                arrive_warp(p_ready);
            }
        }
    } else if (warp >= 4) {  // ---- the decayed b in parts, and S
        constexpr int HC = D / 2;  // columns of S a thread holds
        const int id = tid - 128, half = id / 128, quad = warp & 3;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const int x = (quad * 32 + lane) & (L::DP - 1);  // this lane's row
        const bool row_in = x < D;
        float2 S[HC / 2];
        {
            const float* init = r.init ? r.init + (size_t)bh * D * D : nullptr;
            int init_t = r.init_t;
            if (p.nseg > 1) {
                init = STATE ? nullptr : p.seg + (((size_t)p.seg_role[ri] * p.B * p.H + bh) * p.nseg + seg) * D * D;
                init_t = p.seg_t[ri];
            }
#pragma unroll
            for (int e = 0; e < HC / 2; ++e) {
                const int y = half * HC + 2 * e;
                S[e] = zero2;
                if (init && row_in)
                    S[e] = init_t ? make_float2(init[y * D + x], init[(y + 1) * D + x])
                                  : *reinterpret_cast<const float2*>(init + x * D + y);
            }
        }
        auto publish = [&] {  // Sb = bf16(S)
#pragma unroll
            for (int q = 0; q < HC / 16; ++q) {
                uint32_t u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = pack_bf16(S[q * 8 + e].x, S[q * 8 + e].y);
                __syncwarp();
                st_cols8(tm + lanes + L::SB + half * (HC / 2) + q * 8, u);
            }
            vla::tc_wait_st();
            vla::tc_fence_before();
            arrive_warp(sb_ready);
        };
        // Chunk m's b (rows behind its end cleared there and in c), 16 bytes a
        // thread at a time: whole boxes of 64 columns, then a half box where d
        // ends in one.
        auto decayed = [&](int m) {
            const int st = m % L::NST, n = min(L::C, sp.n - chunk0(m));
            if (!wait_warp(full + st, m / L::NST)) return false;
            unsigned char* tb = sm + L::ST + st * 3 * L::TILE + L::TILE;
            const float* w = WK + (rev ? 0 : L::C - n);
            auto part16 = [&](int o, int j) {
                const uint4 raw = *reinterpret_cast<const uint4*>(tb + o);
                const uint32_t y[4] = {raw.x, raw.y, raw.z, raw.w};
                const bool in = j < n;
                const float wj = in ? w[j] : 0.f;
                uint32_t u[3][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // the leading eight bits of what is left, cut off, three times: nothing remains
                    float2 z = fma2(make_float2(__uint_as_float(y[e] << 16), __uint_as_float(y[e] & 0xFFFF0000u)),
                                    make_float2(wj, wj), zero2);
                    if (n < L::C && !in) z = zero2;
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        u[k][e] = __byte_perm(__float_as_uint(z.x), __float_as_uint(z.y), 0x7632);
                        if (k < 2)
                            z = fma2(make_float2(__uint_as_float(__float_as_uint(z.x) & 0xFFFF0000u),
                                                 __uint_as_float(__float_as_uint(z.y) & 0xFFFF0000u)),
                                     make_float2(-1.f, -1.f), z);
                    }
                }
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    *reinterpret_cast<uint4*>(sm + L::KW + k * L::TILE + o) = make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
            };
#pragma unroll
            for (int it = 0; it < (D / 64) * 2; ++it) part16(it * 4096 + id * 16, (it & 1) * 32 + id / 8);
            if constexpr (D % 64 != 0) {
                const int j = id / 4;
                part16((D / 64) * L::BOX + j * 128 + (((id & 3) ^ (j & 7)) << 4), j);
            }
            if (n < L::C)
                for (int o = n * 128 + id * 16; o < L::BOX; o += 256 * 16)
#pragma unroll
                    for (int k = 0; k < L::NB; ++k)
                        *reinterpret_cast<uint4*>(tb + L::TILE + k * L::BOX + o) = make_uint4(0u, 0u, 0u, 0u);
            vla::fence_proxy_async_smem();
            arrive_warp(kw_full);
            return true;
        };
        bool ok = true;
        if (!STATE && chunks > 0) publish();
        if (chunks > 0) ok = decayed(0);
        int m = 0;
        for (; ok && m < chunks; ++m) {
            const int tbuf = m % L::NT;
            if (!(ok = wait_warp(t_done + tbuf, m / L::NT))) break;
            if (m + 1 < chunks && !(ok = decayed(m + 1))) break;
            vla::tc_fence_after();
            const float wn = decay_pow(g, min(L::C, sp.n - chunk0(m)));
            const float2 w2 = make_float2(wn, wn);
#pragma unroll
            for (int q = 0; q < HC / 16; ++q) {
                float v[16];
                __syncwarp();
                vla::tc_ld16(tm + lanes + L::T + tbuf * L::DP + half * HC + q * 16, v);
                vla::tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) S[q * 8 + e] = fma2(w2, S[q * 8 + e], make_float2(v[2 * e], v[2 * e + 1]));
            }
            vla::tc_fence_before();
            arrive_warp(t_free + tbuf);
            if (!STATE && m + 1 < chunks) {
                if (!(ok = wait_warp(oe_done, m))) break;  // Sb's last reader
                vla::tc_fence_after();
                publish();
            }
        }
        float* fin = STATE ? p.seg + (((size_t)ri * p.B * p.H + bh) * p.nseg + seg) * D * D
                           : (p.nseg > 1 || !r.fin ? nullptr : r.fin + (size_t)bh * D * D);
        if (ok && fin && quad * 32 + lane < D) {
#pragma unroll
            for (int e = 0; e < HC / 2; e += 2) {
                bad = fma2(S[e], zero2, bad);
                bad = fma2(S[e + 1], zero2, bad);
                *reinterpret_cast<float4*>(fin + x * D + half * HC + 2 * e) =
                    make_float4(S[e].x, S[e].y, S[e + 1].x, S[e + 1].y);
            }
        }
    } else if (!STATE) {  // ---- output
        const uint32_t lanes = (uint32_t)warp * 32 << 16;
        const int x = (warp * 32 + lane) & (L::DP - 1);
        // where the lanes hold the rows twice, each copy's warps take half of the tokens
        constexpr int NI = L::DP == 64 ? 32 : 64;
        const int i0 = L::DP == 64 ? (warp / 2) * 32 : 0;
        unsigned char* col = sm + L::OUT + (x / 64) * L::BOX + i0 * 128 + (x % 8) * 2;
        const int c16 = (x % 64) / 8;
        uint32_t at8[8];  // of tokens i, i + 8, ...: their 16 bytes of the swizzled row
#pragma unroll
        for (int i = 0; i < 8; ++i) at8[i] = (uint32_t)((c16 ^ i) << 4);
        for (int m = 0; m < chunks; ++m) {
            const int c0 = chunk0(m), n = min(L::C, sp.n - c0);
            float2 y[NI / 2];
            bool ok = wait_warp(oe_done, m);
            if (ok) {
                vla::tc_fence_after();
                const float* w = WO + i0 + (rev ? L::C - n : 0);
#pragma unroll
                for (int q = 0; q < NI / 16; ++q) {
                    float v[16];
                    __syncwarp();
                    vla::tc_ld16(tm + lanes + L::OE + i0 + q * 16, v);
                    vla::tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = q * 16 + 2 * e;
                        y[q * 8 + e] = fma2(make_float2(w[i], w[i + 1]), make_float2(v[2 * e], v[2 * e + 1]), zero2);
                    }
                }
                vla::tc_fence_before();
                arrive_warp(oe_free);
                ok = wait_warp(o_done + m % 2, m / 2);
            }
            if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            // the last chunk has left the buffer; the four warps leave together if a wait ran out
            if (vla::bar_red_or(1, 128, !ok)) break;
            vla::tc_fence_after();
#pragma unroll
            for (int q = 0; q < NI / 16; ++q) {
                float v[16];
                __syncwarp();
                vla::tc_ld16(tm + lanes + L::X + (m % L::NX) * 64 + i0 + q * 16, v);
                vla::tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[q * 8 + e] = fma2(make_float2(1.f, 1.f), y[q * 8 + e], make_float2(v[2 * e], v[2 * e + 1]));
            }
            vla::tc_fence_before();
            arrive_warp(o_free);
            if (n < L::C) {
#pragma unroll
                for (int e = 0; e < NI / 2; ++e) {
                    if (i0 + 2 * e >= n) y[e].x = 0.f;
                    if (i0 + 2 * e + 1 >= n) y[e].y = 0.f;
                }
            }
#pragma unroll
            for (int e = 0; e < NI / 2; ++e) {
                const int i = 2 * e;
                bad = fma2(y[e], zero2, bad);
                const uint32_t z = pack_bf16(y[e].x, y[e].y);
                *reinterpret_cast<uint16_t*>(col + i * 128 + at8[i & 7]) = (uint16_t)z;
                *reinterpret_cast<uint16_t*>(col + (i + 1) * 128 + at8[(i + 1) & 7]) = (uint16_t)(z >> 16);
            }
            vla::fence_proxy_async_smem();
            vla::named_bar(1, 128);
            if (tid == 0) {
#pragma unroll
                for (int k = 0; k < L::NB; ++k)
                    tma_store(&maps.out[ri], k * 64, sp.t0 + c0, h, b, sb + L::OUT + k * L::BOX);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        }
        if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    __syncwarp();
    // rows behind the sequence's last chunk (those within it were stored as zero)
    if (!STATE) {
        const int done = min(chunks * L::C, p.T - sp.t0);
        const int behind = min(p.seg_len, p.T - sp.t0) - done;
        const float zero[8] = {};
        for (int i = tid; i < behind * (D / 8); i += L::THREADS)
            store8(row_of<__nv_bfloat16>(r.out, b, h, sp.t0 + done + i / (D / 8)) + (i % (D / 8)) * 8, zero);
    }
    if ((bad.x != bad.x || bad.y != bad.y) && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, sp.t0);
    vla::tc_fence_before();
    __syncthreads();
    if (warp == 15) {
        vla::tc_fence_after();
        vla::tc_dealloc(tm, L::COLS);
    }
}

}  // namespace vla_layer
