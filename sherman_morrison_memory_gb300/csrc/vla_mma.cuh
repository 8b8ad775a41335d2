// vla_mma.cuh -- warp-level bf16 products of fp32 accuracy: an fp32 value as a
// sum of bf16 parts (three hold its 24 bits), products of parts with fp32 sums.
#pragma once

#include "vla_layer.cuh"

namespace vla_layer {

// x as the sum of N bf16 parts, two values at a time: the first is x rounded (it may stand for x alone), the others are
// of what is left, eight bits at a time; three parts hold the value's 24 bits. The last of two is rounded too.
template <int N>
__device__ __forceinline__ void split(float x0, float x1, uint32_t (&p)[N]) {
    float2 x = make_float2(x0, x1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool cut = N == 3 && i > 0;
        const uint32_t w0 = __float_as_uint(x.x), w1 = __float_as_uint(x.y);
        p[i] = cut ? __byte_perm(w0, w1, 0x7632) : pack_bf16(x.x, x.y);
        if (i + 1 < N)
            x = __ffma2_rn(cut ? make_float2(__uint_as_float(w0 & 0xFFFF0000u), __uint_as_float(w1 & 0xFFFF0000u))
                               : make_float2(__uint_as_float(p[i] << 16), __uint_as_float(p[i] & 0xFFFF0000u)),
                           make_float2(-1.f, -1.f), x);
    }
}
__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void stsm_t(uint32_t at, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(r0), "r"(r1),
                 "r"(r2), "r"(r3)
                 : "memory");
}

// Element offsets of a lane's row in a 16 x 16 block of rows of LD elements, for x4 loads of its four 8 x 8
// blocks: down then across (an A operand from rows of m, or with ldsm_t a B operand from rows of k), or across
// then down (a B operand from rows of n, or with ldsm_t an A operand from rows of k).
template <int LD>
__device__ __forceinline__ int down_across(int lane) {
    return (lane & 15) * LD + (lane >> 4) * 8;
}
template <int LD>
__device__ __forceinline__ int across_down(int lane) {
    return ((lane & 7) + ((lane >> 4) << 3)) * LD + ((lane >> 3) & 1) * 8;
}

// c + low += A B for N tiles of eight columns: over the first NA parts of A and the parts of B, the products whose size
// is at least that of the last part kept of either. b[n][part]: a tile's operand. The tensor cores cut the sum off at
// every addition, always towards zero, so the many small products have a sum of their own and only those of the first
// parts are added at full size (fp32 results were up to 4e-6 off with one sum, where a head's products add up 48 times).
// The tiles come innermost: a product waits for the one before it on the same sum, 21 cycles at 8 a product.
template <int NA, int NT, int M, int NB>
__device__ __forceinline__ void mma_tiles(float (*c)[4], float (*low)[4], const uint32_t (&a)[M][4], const uint32_t (&b)[NT][NB][2]) {
    constexpr int MOST = (NA > NB ? NA : NB) - 1;
#pragma unroll
    for (int sum = 0; sum <= MOST; ++sum)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int i = sum - j;
            if (i < 0 || i >= NA) continue;
#pragma unroll
            for (int n = 0; n < NT; ++n) mma(sum ? low[n] : c[n], a[i], b[n][j][0], b[n][j][1]);
        }
}
// The operands of two tiles from a 16 x 16 block.
template <int NT, int NB>
__device__ __forceinline__ void ldsm_pair(uint32_t (&b)[NT][NB][2], int n, int part, uint32_t at) {
    uint32_t r[4];
    ldsm(r, at);
    b[n][part][0] = r[0], b[n][part][1] = r[1], b[n + 1][part][0] = r[2], b[n + 1][part][1] = r[3];
}
template <int NT, int NB>
__device__ __forceinline__ void ldsm_pair_t(uint32_t (&b)[NT][NB][2], int n, int part, uint32_t at) {
    uint32_t r[4];
    ldsm_t(r, at);
    b[n][part][0] = r[0], b[n][part][1] = r[1], b[n + 1][part][0] = r[2], b[n + 1][part][1] = r[3];
}
// One tile, its operand a half of what ldsm gives.
template <int NA, int M, int NB>
__device__ __forceinline__ void mma_parts(float (&c)[4], float (&low)[4], const uint32_t (&a)[M][4], const uint32_t (&b)[NB][4],
                                          int half) {
    constexpr int MOST = (NA > NB ? NA : NB) - 1;
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j <= MOST) mma(i + j ? low : c, a[i], b[j][2 * half], b[j][2 * half + 1]);
}
template <int N>
__device__ __forceinline__ void join(float (&c)[N][4], const float (&low)[N][4]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[i][e] += low[i][e];
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace vla_layer
