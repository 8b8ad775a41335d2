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
//   T[x][y]  = sum_j (k_st w^(n-1-j) c_j[x]) b_j[y]     A from TMEM
//   S[x][y]  = w^n S[x][y] + T[x][y]                    fp32, in registers
//
// All but SC have the state's rows x on the 128 TMEM lanes, so that S is added
// up and turned into the A operand Sb by the lane's own threads. OI and OE are
// kept apart because their weights would otherwise be one more rounding. The
// decayed c is cut into three bf16 parts, which hold its 24 bits: S is an fp32
// result (two parts left it 2e-6 off). P and Sb are rounded to bf16 once: o is
// rounded to bf16 afterwards anyway, and a term meets only one of the two.
//
// What bounds it. At d = 128 on all SMs memory: 64 KB a chunk, 1.5 us of 1.55.
// Else the chain of one chunk's products through SC, P, OI and the read-out of
// its accumulator, 0.9 us at d = 64 and 1.25 us at d = 96 and 128, beside the
// chain through S (decayed c, T, S, Sb) of about the same length. The MMAs take a
// third to a half of it: at N = 64 they are fed at shared memory's 128 bytes a
// cycle. So the decayed c goes to TMEM, not to shared memory, from ldmatrix's
// transposed fragments; SC and the outputs are read in fragments (16x256b) that
// stmatrix writes in whole 16-byte rows; and the pairs' weights, which in
// fragments depend on the lane and the blocks' distance, stay in registers.
// (8 x 16 heads of 4,096 tokens, d = 96: 90 us, 4.5 TB/s of its sequences.)
//
// d is padded to DP = 64 or 128 columns by TMA's zero fill. DP is also the MMAs'
// M, so that at d <= 64 a warp's quarter of the TMEM lanes holds 16 rows of the
// state (lanes 0-15), at d > 64 32. SC has M = 128 with the upper 64 rows reading
// what follows the tile in shared memory; nothing reads those lanes.
//
// Warps: 0-3 output, 4-11 decayed c and S, 12-13 P, 14 TMA loads and the MMAs of
// the state (OE, T), 15 those of the pairs (SC, OI).
// Every wait is bounded; one that runs out raises the block's abort flag.
//
// P's zeros above the diagonal are multiplied too: where c holds an Inf or NaN, and
// for heads whose powers overflow, a block goes token by token (by_token()).
//
// STATE: only the segment's own state, from zero (b and c).
#pragma once

#include <cuda.h>

#include <type_traits>

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
    static constexpr int NST = DP == 64 ? 8 : 4;  // chunks in flight
    static constexpr int PARTS = 3;               // of the decayed c
    static constexpr int NCW = 2;                 // its buffers
    // buffers of SC with OI behind it, and of P (where TMEM has room: the pairs then run a chunk ahead)
    static constexpr int NX = DP == 64 ? 2 : 1;
    static constexpr int RW = DP / 4, NH = RW / 16;  // rows of the state in a warp's lanes; groups of 16
    static constexpr int THREADS = 512;
    // shared memory
    static constexpr int ST = 0;                           // [NST] a | b | c
    static constexpr int P = ST + NST * 3 * TILE;
    static constexpr int OUT = P + NX * BOX;
    // weights of 64 each: the state to tokens, tokens to the state, pairs by
    // their lag. Tokens behind a chunk's end read into the next table and pairs
    // against the order of time into the one before; what they get is thrown away
    static constexpr int WO = OUT + TILE, WK = WO + 64 * 4, WP = WK + 64 * 4;
    static constexpr int BAR = WP + 64 * 4;
    static constexpr int NBAR = 2 * NST + 16;
    static constexpr int MISC = BAR + NBAR * 8;
    static constexpr int SMEM = MISC + 16;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    // TMEM columns. OI takes SC's place once P is made of it.
    static constexpr int SB = 0, CW = SB + DP / 2, OE = CW + NCW * PARTS * 32, X = OE + 64, T = X + NX * 64;
    static constexpr int COLS = 512;
    static_assert(T + DP <= COLS, "tensor memory");
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
// Fragments: of 16 lanes, thread l holds rows l / 4 and l / 4 + 8. ld_frag:
// columns 8 k + 2 (l % 4) + {0, 1} of both rows in v[4 k ..]; st_frag: column
// 4 k + l % 4 of the two rows, the 2 k-th and the next value.
__device__ __forceinline__ void ld_frag64(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void ld_frag32(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void ld_frag16(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void st_frag8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void st_frag4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
// four 8 x 8 blocks of 16-bit values: lane l gives the address of row l % 8 of
// block l / 8; _t: rows and columns swapped on the way
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
__device__ __forceinline__ void stmatrix4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
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
// A wait that did not end at once, for at most p.wait_ns: false, recorded and
// the abort flag raised, if it or another of the block's ran out.
__device__ __noinline__ bool wait_on(uint64_t* w, uint32_t parity, volatile int* abort_flag, unsigned long long ns,
                                     vla::DeviceStatus* status, int role, int bh) {
    if (vla::mbar_wait_slow(w, parity, (const volatile int*)abort_flag, ns)) return true;
    if (*abort_flag == 0 && status) vla::record_failure(status, vla::BIT_TIMEOUT, role, bh, 0);
    *abort_flag = 1;
    return false;
}

template <int D, bool STATE>
__global__ void __launch_bounds__(TcLay<D>::THREADS, 1)
    vla_decay_tc_kernel(const __grid_constant__ DecayArgs p, const __grid_constant__ DecayMaps maps, int roles) {
    using L = TcLay<D>;
    extern __shared__ __align__(1024) unsigned char tc_sm[];
    unsigned char* sm = tc_sm;
    const uint32_t sb = vla::smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
    uint64_t *full = bar, *empty = full + L::NST, *cw_full = empty + L::NST, *p_ready = cw_full + 2,
             *sc_done = cw_full + 4, *o_done = cw_full + 6, *sb_ready = cw_full + 8, *oe_done = cw_full + 9,
             *oe_free = cw_full + 10, *o_free = cw_full + 11, *t_done = cw_full + 12, *cleared = cw_full + 13,
             *drained = cw_full + 14;
    float *WP = reinterpret_cast<float*>(sm + L::WP), *WK = reinterpret_cast<float*>(sm + L::WK),
          *WO = reinterpret_cast<float*>(sm + L::WO);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int ri = blockIdx.x % roles, rest = blockIdx.x / roles;
    const int seg = rest % p.nseg, bh = p.bh0 + rest / p.nseg, b = bh / p.H, h = bh % p.H;
    const Role& r = p.role[ri];
    const float g = p.log_decay[h];
    const Span sp = span_of(p, b, seg);
    const bool rev = r.reverse != 0;
    const int chunks = (sp.n + L::C - 1) / L::C;

    static_assert(L::SMEM >= (D * (D + 4) + 24 * D) * 4, "by_token's floats");
    if (outgrows(g, L::C)) {
        by_token<D, __nv_bfloat16, L::THREADS, STATE>(p, ri, bh, seg, reinterpret_cast<float*>(sm));
        return;
    }

    // With time, a token's weight towards the state counts from the chunk's
    // end; against it, its weight from the state does: those tables hold the
    // powers 63, 62, .. and a chunk of n tokens begins 64 - n behind.
    if (tid < 64) {
        const int up = tid + 1, down = 63 - tid;
        WK[tid] = r.k_st * decay_pow(g, rev ? up : down);
        WO[tid] = r.w_st * decay_pow(g, rev ? down : up);
        WP[tid] = r.w_in * decay_pow(g, tid);
    }
    for (int i = tid; i < L::NX * L::BOX / 16; i += L::THREADS)  // the pairs that no chunk writes stay zero
        *reinterpret_cast<uint4*>(sm + L::P + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    vla::fence_proxy_async_smem();
    if (tid == 0) {
        for (int i = 0; i < L::NST; ++i) vla::mbar_init(full + i, 1), vla::mbar_init(empty + i, STATE ? 1 : 2);
        // two, by the chunk's parity, where one side may be a chunk ahead of the other or of its own other warps
        for (int i = 0; i < 2; ++i) {
            vla::mbar_init(cw_full + i, 8);
            vla::mbar_init(p_ready + i, 2);
            vla::mbar_init(sc_done + i, 1);
            vla::mbar_init(o_done + i, 1);
        }
        vla::mbar_init(sb_ready, 8);
        vla::mbar_init(oe_done, 1);
        vla::mbar_init(oe_free, 4);
        vla::mbar_init(o_free, 4);
        vla::mbar_init(t_done, 1);
        vla::mbar_init(cleared, 8);
        for (int i = 0; i < 2; ++i) vla::mbar_init(drained + i, 1);
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

    // Bounded wait of a whole warp: false once this or another wait of the block
    // has run out. The lanes go into the slow path together: a call that only
    // some of them made would leave the others' uniform registers behind.
    auto wait_warp = [&](uint64_t* w, uint32_t parity) {
        if (__all_sync(0xffffffffu, vla::mbar_try_wait(w, parity & 1))) return true;
        const bool ok = wait_on(w, parity & 1, abort_flag, p.wait_ns, p.status, warp / 4, bh);
        return __all_sync(0xffffffffu, ok) != 0;
    };
    // The same for what has to end before the block does, also where a wait has run
    // out; the warp leaves it whole, as a barrier counts a split warp twice.
    auto drain_warp = [&](uint64_t* w, uint32_t parity) {
        if (!__all_sync(0xffffffffu, vla::mbar_try_wait(w, parity & 1)))
            vla::mbar_wait_slow(w, parity & 1, nullptr, p.wait_ns);
        __syncwarp();
    };
    auto arrive_warp = [&](uint64_t* w) {  // one arrival a warp
        __syncwarp();
        if (lane == 0) vla::mbar_arrive(w);
    };
    // first token (within the segment) of the m-th chunk in the role's order
    auto chunk0 = [&](int m) { return (rev ? chunks - 1 - m : m) * L::C; };

    // S, of warps 4-11. A warp has the rows [xb, xb + RW), xb = RW quad, and half of
    // the columns. Where the rows fill its 32 lanes, a lane has a row's: S[k] holds
    // columns 2 k + {0, 1} of the half. Where they are 16, in fragments: S[4 u + k]
    // holds columns 16 u + 8 (k / 2) + {0, 1} (from the lane's first) of row lane / 4
    // + 8 (k % 2).
    constexpr bool FRAG = L::NH == 1;
    constexpr int HC = D / 2, NU = HC / 16, NS = L::NH * NU * 4;
    const int id = tid - 128, half = id / 128, quad = warp & 3;
    auto row = [&](int k) { return quad * L::RW + (FRAG ? (lane >> 2) + 8 * (k % 2) : lane); };
    auto col = [&](int k) { return half * HC + (FRAG ? 2 * (lane & 3) + 16 * (k / 4) + 8 * ((k % 4) / 2) : 2 * k); };
    float2 S[NS];
    auto write_state = [&](float* to) {
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            bad = fma2(S[k], zero2, bad);
            if constexpr (FRAG)
                *reinterpret_cast<float2*>(to + row(k) * D + col(k)) = S[k];
            else if (k % 2 == 0)
                *reinterpret_cast<float4*>(to + row(k) * D + col(k)) = make_float4(S[k].x, S[k].y, S[k + 1].x, S[k + 1].y);
        }
    };
    float* in_place = nullptr;  // where the final state takes the initial one's place: written last

    // The whole warps run the MMA loops, so that operands stay in uniform
    // registers, and one elected thread issues: issued under a test of the lane,
    // each MMA took 100 cycles.
    constexpr uint32_t HALF = L::NB == 2 ? L::BOX : 16;  // from an MN-major operand's first 64 rows to the next
    const uint64_t dk = desc_sw128(0, 16, 1024), dm = desc_sw128(0, HALF, 1024);
    auto at = [](uint64_t d, uint32_t addr) { return d + (uint64_t)(addr >> 4); };

    if (warp == 14) {  // ---- TMA loads, MMAs of the state
        const bool one = elect_one();
        const uint32_t id_t = idesc_bf16(L::DP, D, 0, 1), id_oe = idesc_bf16(L::DP, 64, 0, 0);
        const int id[3] = {r.map_a, r.map_b, r.map_c};
        auto load = [&](int m) {
            const int i = m % L::NST, t = sp.t0 + chunk0(m);
            const uint32_t dst = sb + L::ST + i * 3 * L::TILE;
            if (one && !(p.stall && m + 1 == chunks)) {
                vla::mbar_arrive_expect_tx(full + i, (STATE ? 2 : 3) * L::TILE);
#pragma unroll
                for (int q = STATE ? 1 : 0; q < 3; ++q)
#pragma unroll
                    for (int x = 0; x < L::NB; ++x)
                        tma_load(dst + q * L::TILE + x * L::BOX, &maps.m[id[q]], x * 64, t, h, b, full + i);
            }
            __syncwarp();
        };
        int loaded = min(chunks, L::NST);
        for (int m = 0; m < loaded; ++m) load(m);
        for (int m = 0; m < chunks; ++m) {
            const int i = m % L::NST;
            const uint32_t ta = sb + L::ST + i * 3 * L::TILE, tb = ta + L::TILE;
            if (!wait_warp(full + i, m / L::NST)) break;
            if (!wait_warp(sb_ready, m)) break;  // T's last reader is done
            auto to_state = [&] {  // T
                if (!wait_warp(cw_full + m % 2, m / 2)) return false;
                const uint32_t cw = tm + L::CW + (m % L::NCW) * L::PARTS * 32;
                vla::tc_fence_after();
                if (one) {
#pragma unroll
                    for (int part = 0; part < L::PARTS; ++part)
#pragma unroll
                        for (int k = 0; k < L::C / 16; ++k)
                            mma_ts(tm + L::T, cw + part * 32 + k * 8, at(dm, tb + k * 2048), id_t, part > 0 || k > 0);
                    vla::tc_commit(t_done);
                }
                __syncwarp();
                return true;
            };
            auto from_state = [&] {  // OE
                if (m > 0 && !wait_warp(oe_free, m - 1)) return false;
                vla::tc_fence_after();
                if (one) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ts(tm + L::OE, tm + L::SB + k * 8, at(dk, ta + (k / 4) * L::BOX + (k % 4) * 32), id_oe, k > 0);
                    vla::tc_commit(oe_done);
                }
                __syncwarp();
                return true;
            };
            // the chain through S is the longer one where T is short, the outputs' where it is long
            if (STATE ? !to_state() : L::NH == 1 ? !to_state() || !from_state() : !from_state() || !to_state()) break;
            if (one) vla::tc_commit(empty + i);
            __syncwarp();
            if (m > 0 && loaded < chunks) {  // the stage of the chunk before takes a new one
                if (!wait_warp(empty + (m - 1) % L::NST, (m - 1) / L::NST)) break;
                load(loaded++);
            }
        }
        if (*abort_flag)  // leave only once the copies under way have landed
            for (int m = max(0, loaded - L::NST); m < loaded; ++m)
                drain_warp(full + m % L::NST, m / L::NST);
        if (one) vla::tc_commit(drained);  // what was issued has finished before the block frees its TMEM
        __syncwarp();
        drain_warp(drained, 0);
    } else if (warp == 15) {  // ---- MMAs of the pairs
        const bool one = elect_one();
        const uint32_t id_sc = idesc_bf16(128, 64, 0, 0), id_oi = idesc_bf16(L::DP, 64, 1, 0);
        auto pairs = [&](int m) {  // SC
            const int i = m % L::NST;
            const uint32_t ta = sb + L::ST + i * 3 * L::TILE, tb = ta + L::TILE, x = tm + L::X + (m % L::NX) * 64;
            if (!wait_warp(full + i, m / L::NST)) return false;
            if (m >= L::NX && !wait_warp(o_free, m - L::NX)) return false;
            vla::tc_fence_after();
            if (one) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k / 4) * L::BOX + (k % 4) * 32;
                    mma_ss(x, at(dk, ta + off), at(dk, tb + off), id_sc, k > 0);
                }
                vla::tc_commit(sc_done + m % 2);
            }
            __syncwarp();
            return true;
        };
        if (!STATE) {
            bool ok = L::NX == 1 || chunks == 0 || pairs(0);
            for (int m = 0; ok && m < chunks; ++m) {
                const int i = m % L::NST;
                const uint32_t tc = sb + L::ST + i * 3 * L::TILE + 2 * L::TILE, x = tm + L::X + (m % L::NX) * 64;
                const uint32_t pm = sb + L::P + (m % L::NX) * L::BOX;
                if (m + L::NX - 1 < chunks && !pairs(m + L::NX - 1)) break;
                if (!wait_warp(p_ready + m % 2, m / 2)) break;
                if (sp.n - chunk0(m) < L::C && !wait_warp(cleared, 0)) break;  // c's rows behind the end, once
                vla::tc_fence_after();
                if (one) {
#pragma unroll
                    for (int k = 0; k < L::C / 16; ++k)
                        mma_ss(x, at(dm, tc + k * 2048), at(dk, pm + k * 32), id_oi, k > 0);
                    vla::tc_commit(o_done + m % 2);
                    vla::tc_commit(empty + i);
                }
                __syncwarp();
            }
            if (one) vla::tc_commit(drained + 1);
            __syncwarp();
            drain_warp(drained + 1, 0);
        }
    } else if (warp >= 12) {  // ---- P
        // In blocks of 8 x 8 pairs: those of the later half of pairs are never
        // written and stay zero, those on the diagonal are cut by it. A warp
        // has 32 rows, 16 at a time; the weights depend on the blocks' distance.
        if (!STATE) {
            const int lr = lane >> 2, lc = 2 * (lane & 3);
            auto body = [&](auto rbc, auto revc) {
                constexpr int RB = decltype(rbc)::value;
                constexpr bool REV = decltype(revc)::value;
                float2 w[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int lag = 8 * q + (REV ? lc - lr : lr - lc);
                    w[q] = make_float2(WP[lag], WP[REV ? lag + 1 : lag - 1]);
                }
                const bool in0 = REV ? lc >= lr : lc <= lr, in1 = REV ? lc + 1 >= lr : lc + 1 <= lr;
                // rows of the blocks (r, k), (r + 1, k), (r, k + 1), (r + 1, k + 1)
                const int row8 = ((lane >> 3) & 1) * 8 + (lane & 7), kk = lane >> 4;
                for (int m = 0; m < chunks; ++m) {
                    const int n = min(L::C, sp.n - chunk0(m));
                    if (!wait_warp(sc_done + m % 2, m / 2)) return;
                    // P's last reader; with one buffer SC of this chunk was behind it
                    if (L::NX == 2 && m >= 2 && !wait_warp(o_done + m % 2, m / 2 - 1)) return;
                    vla::tc_fence_after();
                    float both[2][32];
                    __syncwarp();
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
                        ld_frag64(tm + ((uint32_t)(RB * 32 + hh * 16) << 16) + L::X + (m % L::NX) * 64, both[hh]);
                    vla::tc_wait_ld();
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int r = RB * 4 + hh * 2;  // first of two rows of blocks
                        const float* v = both[hh];
                        const uint32_t dst = sb + L::P + (m % L::NX) * L::BOX + (r * 8 + row8) * 128;
#pragma unroll
                        for (int k = 0; k < 8; k += 2) {
                            if (REV ? k < r : k > r) continue;
                            uint32_t u[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int kb = k + e / 2, dist = REV ? kb - (r + e % 2) : r + e % 2 - kb;
                                if (dist < 0) {
                                    u[e] = 0u;
                                    continue;
                                }
                                float2 z = fma2(make_float2(v[kb * 4 + (e % 2) * 2], v[kb * 4 + (e % 2) * 2 + 1]), w[dist], zero2);
                                if (dist == 0) {
                                    if (!in0) z.x = 0.f;
                                    if (!in1) z.y = 0.f;
                                }
                                if (REV && n < L::C) {
                                    if (kb * 8 + lc >= n) z.x = 0.f;
                                    if (kb * 8 + lc + 1 >= n) z.y = 0.f;
                                }
                                u[e] = pack_bf16(z.x, z.y);
                            }
                            stmatrix4(dst + (((k + kk) ^ (lane & 7)) << 4), u[0], u[1], u[2], u[3]);
                        }
                    }
                    vla::tc_fence_before();
                    vla::fence_proxy_async_smem();
                    arrive_warp(p_ready + m % 2);
                }
            };
            using std::integral_constant;
            if (warp == 12)
                rev ? body(integral_constant<int, 0>{}, integral_constant<bool, true>{})
                    : body(integral_constant<int, 0>{}, integral_constant<bool, false>{});
            else
                rev ? body(integral_constant<int, 1>{}, integral_constant<bool, true>{})
                    : body(integral_constant<int, 1>{}, integral_constant<bool, false>{});
        }
    } else if (warp >= 4) {  // ---- the decayed c in parts, and S
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const int xb = quad * L::RW;
        const bool rows_in = xb < D;  // else zero throughout
        int init_t;
        const float* init = start_of<D, STATE>(p, ri, bh, seg, init_t);
        {
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                const int x = row(k), y = col(k);
                if (FRAG || k % 2 == 0 || !init || init_t) S[k] = zero2;
                if (!init || !rows_in) continue;
                if (init_t) {
                    S[k] = make_float2(init[y * D + x], init[(y + 1) * D + x]);
                } else if constexpr (FRAG) {
                    S[k] = *reinterpret_cast<const float2*>(init + x * D + y);
                } else if (k % 2 == 0) {
                    const float4 v = *reinterpret_cast<const float4*>(init + x * D + y);
                    S[k] = make_float2(v.x, v.y), S[k + 1] = make_float2(v.z, v.w);
                }
            }
        }
        bool first = true;
        auto publish = [&] {  // Sb = bf16(S); T has been read
            if (!STATE && (rows_in || first)) {
                __syncwarp();
#pragma unroll
                for (int u = 0; u < NS / 8; ++u) {
                    uint32_t v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = pack_bf16(S[8 * u + k].x, S[8 * u + k].y);
                    const uint32_t dst = tm + lanes + L::SB + half * (HC / 2);
                    if constexpr (FRAG)
                        st_frag8(dst + u * 16, v);
                    else
                        st_cols8(dst + u * 8, v);
                }
                if constexpr (NS % 8 != 0)
                    st_frag4(tm + lanes + L::SB + half * (HC / 2) + NS / 8 * 16, pack_bf16(S[NS - 4].x, S[NS - 4].y),
                             pack_bf16(S[NS - 3].x, S[NS - 3].y), pack_bf16(S[NS - 2].x, S[NS - 2].y),
                             pack_bf16(S[NS - 1].x, S[NS - 1].y));
                vla::tc_wait_st();
            }
            first = false;
            vla::tc_fence_before();
            arrive_warp(sb_ready);
        };
        const int j0 = half * 32 + 2 * (lane & 3);  // this lane's tokens: j0 + 8 k + {0, 1}
        // the row of c that this lane addresses for ldmatrix: blocks (x, j), (x + 8, j), (x, j + 8), (x + 8, j + 8)
        const uint32_t src = (xb / 64) * L::BOX + (half * 32 + (lane >> 4) * 8 + (lane & 7)) * 128;
        const int chunk16 = (xb % 64) / 8 + ((lane >> 3) & 1);
        // Chunk m's c, decayed to the chunk's end, for this warp's rows and 32
        // tokens; rows behind the chunk's end cleared in b and c.
        auto decayed = [&](int m) {
            const int st = m % L::NST, n = min(L::C, sp.n - chunk0(m));
            if (!wait_warp(full + st, m / L::NST)) return false;
            const uint32_t tc = L::ST + st * 3 * L::TILE + 2 * L::TILE;
            const float* w = WK + j0 + (rev ? 0 : L::C - n);
            // rolled: the roles' code of a scheduler is more than its instruction cache
#pragma unroll 1
            for (int hh = 0; hh < L::NH && (D % 64 == 0 || rows_in); ++hh) {
                uint32_t y[8];
                float2 z[8];
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    ldmatrix4_t(sb + tc + src + k * 2048 + (((chunk16 + 2 * hh) ^ (lane & 7)) << 4), y[4 * k], y[4 * k + 1],
                                y[4 * k + 2], y[4 * k + 3]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = 8 * (e / 2);
                    z[e] = fma2(make_float2(__uint_as_float(y[e] << 16), __uint_as_float(y[e] & 0xFFFF0000u)),
                                make_float2(w[j], w[j + 1]), zero2);
                }
                if (n < L::C) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int j = j0 + 8 * (e / 2);
                        if (j >= n) z[e].x = 0.f;
                        if (j + 1 >= n) z[e].y = 0.f;
                    }
                }
                // the leading eight bits of what is left, cut off, three times: nothing remains
                uint32_t dst = tm + lanes + ((uint32_t)(hh * 16) << 16) + L::CW + (m % L::NCW) * L::PARTS * 32 + half * 16;
#pragma unroll
                for (int k = 0; k < L::PARTS; ++k, dst += 32) {
                    uint32_t u[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        u[e] = __byte_perm(__float_as_uint(z[e].x), __float_as_uint(z[e].y), 0x7632);
                        if (k + 1 == L::PARTS) continue;
                        z[e] = fma2(make_float2(__uint_as_float(__float_as_uint(z[e].x) & 0xFFFF0000u),
                                                __uint_as_float(__float_as_uint(z[e].y) & 0xFFFF0000u)),
                                    make_float2(-1.f, -1.f), z[e]);
                    }
                    st_frag8(dst, u);
                }
            }
            if (n < L::C) {
                for (int o = n * 128 + id * 16; o < L::BOX; o += 256 * 16)
#pragma unroll
                    for (int k = 0; k < L::NB; ++k) {
                        *reinterpret_cast<uint4*>(sm + tc + k * L::BOX + o) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4*>(sm + tc - L::TILE + k * L::BOX + o) = make_uint4(0u, 0u, 0u, 0u);
                    }
            }
            vla::tc_wait_st();
            vla::tc_fence_before();
            vla::fence_proxy_async_smem();
            arrive_warp(cw_full + m % 2);
            if (n < L::C) arrive_warp(cleared);
            return true;
        };
        bool ok = true;
        SlowDecay whole(g, L::C);
        if constexpr (D % 64 != 0) {  // lanes that no row of c fills
            const uint32_t none[8] = {};
            __syncwarp();
            for (int c = 0; c < L::NCW * L::PARTS * 32 && !rows_in; c += 8) st_cols8(tm + lanes + L::CW + c, none);
            vla::tc_wait_st();
        }
        if (chunks > 0) {
            publish();
            ok = decayed(0);
        }
        for (int m = 0; ok && m < chunks; ++m) {
            // the buffer's last reader, T of chunk m - 1, is done
            if (m + 1 < chunks && !(ok = decayed(m + 1))) break;
            if (!(ok = wait_warp(t_done, m))) break;
            vla::tc_fence_after();
            const int n = min(L::C, sp.n - chunk0(m));
            const float wn = n < L::C ? decay_pow(g, n) : whole.next();  // at most one chunk is shorter
            const float2 w2 = make_float2(wn, wn);
            if (rows_in) {
                const uint32_t src_t = tm + lanes + L::T + half * HC;
#pragma unroll
                for (int u = 0; u < NU; ++u) {  // 16 columns
                    float v[16];
                    __syncwarp();
                    if constexpr (FRAG)
                        ld_frag16(src_t + u * 16, *reinterpret_cast<float(*)[8]>(v));
                    else
                        vla::tc_ld16(src_t + u * 16, v);
                    vla::tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < NS / NU; ++k) {
                        float2& s = S[u * (NS / NU) + k];
                        s = fma2(w2, s, make_float2(v[2 * k], v[2 * k + 1]));
                    }
                }
            }
            if (m + 1 == chunks) break;
            if (!STATE) {
                if (!(ok = wait_warp(oe_done, m))) break;  // Sb's last reader
                vla::tc_fence_after();
            }
            publish();
        }
        float* fin = end_of<D, STATE>(p, ri, bh, seg);
        if (ok && fin && rows_in) {
            if (!STATE && fin == init)
                in_place = fin;
            else
                write_state(fin);
        }
    } else if (!STATE) {  // ---- output
        constexpr int NH = L::NH;
        const int lc = 2 * (lane & 3);
        const int xb = warp * L::RW;
        const bool rows_in = xb < D;  // else columns that no store takes
        // the row of the output that this lane addresses for stmatrix: blocks (x, i), (x + 8, i), (x, i + 8), (x + 8, i + 8)
        const uint32_t dst = sb + L::OUT + (xb / 64) * L::BOX + ((lane >> 4) * 8 + (lane & 7)) * 128;
        const int chunk16 = (xb % 64) / 8 + ((lane >> 3) & 1);
        auto load = [&](uint32_t col, int hh, int part, float* v) {  // 32 of the 64 tokens
            __syncwarp();
            ld_frag32(tm + ((uint32_t)(warp * 32 + hh * 16) << 16) + col + part * 32, *reinterpret_cast<float(*)[16]>(v));
        };
        for (int m = 0; m < chunks; ++m) {
            const int c0 = chunk0(m), n = min(L::C, sp.n - c0);
            float oe[NH][32];
            bool ok = wait_warp(oe_done, m);
            if (ok) {
                vla::tc_fence_after();
                if (rows_in) {
#pragma unroll
                    for (int k = 0; k < 2 * NH; ++k) load(L::OE, k / 2, k % 2, oe[k / 2] + (k % 2) * 16);
                    vla::tc_wait_ld();
                }
                vla::tc_fence_before();
                arrive_warp(oe_free);
                ok = wait_warp(o_done + m % 2, m / 2);
            }
            if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            // the last chunk has left the buffer; the four warps leave together if a wait ran out
            if (vla::bar_red_or(1, 128, !ok)) break;
            vla::tc_fence_after();
            const float* wo = WO + lc + (rev ? L::C - n : 0);
            if (rows_in) {
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    float v[32], *o = oe[hh];
                    load(L::X + (m % L::NX) * 64, hh, 0, v);
                    load(L::X + (m % L::NX) * 64, hh, 1, v + 16);
                    vla::tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float* w = wo + (e / 4) * 8;
                        const float2 y = fma2(make_float2(w[0], w[1]), make_float2(o[e], o[e + 1]), make_float2(v[e], v[e + 1]));
                        o[e] = y.x, o[e + 1] = y.y;
                    }
                }
            }
            vla::tc_fence_before();
            arrive_warp(o_free);
            if (n < L::C) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const int i = (e / 4) * 8 + lc;
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh) {
                        if (i >= n) oe[hh][e] = 0.f;
                        if (i + 1 >= n) oe[hh][e + 1] = 0.f;
                    }
                }
            }
            if (rows_in) {
#pragma unroll
                for (int hh = 0; hh < NH; ++hh)
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        uint32_t u[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float* y = oe[hh] + (k + e / 2) * 4 + (e % 2) * 2;
                            bad = fma2(make_float2(y[0], y[1]), zero2, bad);
                            u[e] = pack_bf16(y[0], y[1]);
                        }
                        stmatrix4_t(dst + k * 1024 + (((chunk16 + 2 * hh) ^ (lane & 7)) << 4), u[0], u[1], u[2], u[3]);
                    }
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
    bool again = false;
    if constexpr (!STATE) {
        // All copies and MMAs of the block are done.
        if (__syncthreads_or(bad.x != bad.x || bad.y != bad.y) && *abort_flag == 0)
            again = seen_too_early<D, __nv_bfloat16, L::THREADS, L::C>(p, r, b, h, sp, reinterpret_cast<int*>(sm));
        if (again) {
            by_token<D, __nv_bfloat16, L::THREADS, STATE>(p, ri, bh, seg, reinterpret_cast<float*>(sm));
            bad = zero2;  // recorded there
        }
        // rows behind the sequence's last chunk (those within it were stored as zero)
        const int done = min(chunks * L::C, p.T - sp.t0);
        const int behind = min(p.seg_len, p.T - sp.t0) - done;
        const float zero[8] = {};
        for (int i = tid; i < behind * (D / 8); i += L::THREADS)
            store8(row_of<__nv_bfloat16>(r.out, b, h, sp.t0 + done + i / (D / 8)) + (i % (D / 8)) * 8, zero);
    }
    if (in_place && !again) write_state(in_place);
    if ((bad.x != bad.x || bad.y != bad.y) && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, sp.t0);
    vla::tc_fence_before();
    __syncthreads();
    if (warp == 15) {
        vla::tc_fence_after();
        vla::tc_dealloc(tm, L::COLS);
    }
}

}  // namespace vla_layer
