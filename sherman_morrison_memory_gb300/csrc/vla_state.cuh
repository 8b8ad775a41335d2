// vla_state.cuh -- the quantised cache of states (include/vla_layer.h): groups
// of 32 values of a row with one fp32 scale, 8 or 4 bits a value, written to
// and read from the slots that an index names.
//
// Both kernels move each byte once and compute next to nothing, so they are
// bound by memory: 4 bytes a value on the fp32 side, 1.125 or 0.625 on the
// cache's. Eight lanes hold a group, four consecutive values each (16-byte
// accesses on the fp32 side, whole 128-byte lines a group).
#pragma once

#include "vla_layer.cuh"

namespace vla_layer {
namespace {

constexpr int STATE_THREADS = 256;
constexpr int UNROLL = 4;                          // float4 a thread has in flight
constexpr int BLOCK_VALUES = STATE_THREADS * UNROLL * 4;  // values a block handles

// 1.5 2^23: a float added to it is rounded to a whole number (ties to even),
// which the sum's low bits hold in two's complement.
constexpr float WHOLE = 12582912.f;

// WHOLE plus the code of value x for the scale s > 0 (inv its reciprocal,
// rounded): the whole number nearest to x / s, ties to the even one. x inv is
// rounded, so that its nearest whole number c may be the wrong neighbour where
// x / s is next to the middle between two. r = x - c s is exact there (a
// multiple of half of s's last place, at most about s / 2), so |r| against s / 2
// tells.
__device__ __forceinline__ float code_of(float x, float s, float inv) {
    float t = fmaf(x, inv, WHOLE);
    const float r = fmaf(-(t - WHOLE), s, x), half = 0.5f * s;
    if (fabsf(r) >= half && (fabsf(r) > half || (__float_as_int(t) & 1))) t += copysignf(1.f, r);
    return t;
}

template <int BITS>
__global__ void __launch_bounds__(STATE_THREADS) vla_state_store_kernel(const float* __restrict__ x, long long per,
                                                                  void* codes, float* scales, int N, const int* slots,
                                                                  vla::DeviceStatus* status) {
    constexpr int TOP = BITS == 8 ? 127 : 7;
    const int b = blockIdx.y;
    const long long first = (long long)blockIdx.x * BLOCK_VALUES + threadIdx.x * 4;
    const float* src = x + (long long)b * per;
    float4 v[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const long long e = first + (long long)i * STATE_THREADS * 4;
        v[i] = e < per ? __ldcs(reinterpret_cast<const float4*>(src + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int slot = slot_of(slots, b, N, true, status);
    if (slot < 0) return;
    const long long base = (long long)slot * per;
    // the groups' largest sizes, as bits: NaN and Inf lie above all others
    uint32_t top[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const uint32_t f[4] = {__float_as_uint(v[i].x), __float_as_uint(v[i].y), __float_as_uint(v[i].z),
                               __float_as_uint(v[i].w)};
        top[i] = max(max(f[0] & 0x7FFFFFFFu, f[1] & 0x7FFFFFFFu), max(f[2] & 0x7FFFFFFFu, f[3] & 0x7FFFFFFFu));
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], m));
    }
    // of a group's eight lanes, lane i divides for group i
    static_assert(UNROLL == 4, "lanes 0-3");
    const int lane8 = threadIdx.x & 7;
    const uint32_t mine = lane8 & 2 ? (lane8 & 1 ? top[3] : top[2]) : (lane8 & 1 ? top[1] : top[0]);
    float scale = __fdiv_rn(__uint_as_float(mine), (float)TOP);
    if (scale < 1.17549435e-38f) scale = 0.f;
    if (mine >= 0x7F800000u) scale = __uint_as_float(0x7FC00000u);
    const float recip = scale > 0.f ? __fdividef(1.f, scale) : 0.f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const long long e = first + (long long)i * STATE_THREADS * 4;
        const float s = __shfl_sync(0xffffffffu, scale, i, 8), inv = __shfl_sync(0xffffffffu, recip, i, 8);
        // a group stored as zero, and one that is not finite, has codes of 0
        const bool none = !(s > 0.f);
        const float f[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = none ? 0u : (uint32_t)__float_as_int(code_of(f[j], s, inv));
        if (e < per) {
            const long long at = base + e;
            if constexpr (BITS == 8) {
                const uint32_t w = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
                *reinterpret_cast<uint32_t*>(static_cast<char*>(codes) + at) = w;
            } else {
                const uint32_t w = (c[0] & 15) | (c[1] & 15) << 4 | (c[2] & 15) << 8 | (c[3] & 15) << 12;
                *reinterpret_cast<uint16_t*>(static_cast<char*>(codes) + at / 2) = (uint16_t)w;
            }
            if (lane8 == 0) scales[at / 32] = s;
            odd |= s != s;
        }
    }
    if (odd && status) vla::record_failure(status, vla::BIT_NONFINITE, kRoleSlot, b, slot);
}

template <int BITS>
__global__ void __launch_bounds__(STATE_THREADS) vla_state_load_kernel(const void* __restrict__ codes,
                                                                 const float* __restrict__ scales, int N,
                                                                 const int* slots, long long per, float* x,
                                                                 vla::DeviceStatus* status) {
    const int b = blockIdx.y;
    const long long first = (long long)blockIdx.x * BLOCK_VALUES + threadIdx.x * 4;
    float* dst = x + (long long)b * per;
    const int slot = slot_of(slots, b, N, false, blockIdx.x == 0 ? status : nullptr);
    const long long base = (long long)(slot < 0 ? 0 : slot) * per;
    uint32_t w[UNROLL];
    float s[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const long long e = first + (long long)i * STATE_THREADS * 4, at = base + e;
        const bool in = e < per && slot >= 0;
        if constexpr (BITS == 8)
            w[i] = in ? *reinterpret_cast<const uint32_t*>(static_cast<const char*>(codes) + at) : 0u;
        else
            w[i] = in ? *reinterpret_cast<const uint16_t*>(static_cast<const char*>(codes) + at / 2) : 0u;
        s[i] = in ? scales[at / 32] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const long long e = first + (long long)i * STATE_THREADS * 4;
        if (e >= per) continue;
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // the code's bits at the top of a word, shifted down with its sign
            const int c = BITS == 8 ? (int)(w[i] << (24 - 8 * j)) >> 24 : (int)(w[i] << (28 - 4 * j)) >> 28;
            f[j] = (float)c * s[i];
        }
        __stcs(reinterpret_cast<float4*>(dst + e), make_float4(f[0], f[1], f[2], f[3]));
    }
}

vla_status check_cache(const void* codes, const float* scales, int N, int B, long long rows, int d, int bits, const float* x,
                 const int* slots, const void* status) {
    if (B < 0 || N < 0 || rows < 0 || (bits != 8 && bits != 4)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if (B > 65535 || rows > (1LL << 36) / d) return VLA_ERR_INVALID_ARG;
    if (!slots && B > N) return VLA_ERR_INVALID_ARG;
    if (B == 0 || rows == 0) return VLA_OK;
    if ((N > 0 && (!codes || !scales)) || !x || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(x, 16) || !aligned(slots, 4) ||
        !aligned(status, 16))
        return VLA_ERR_INVALID_ARG;
    return VLA_OK;
}

}  // namespace
}  // namespace vla_layer

extern "C" {

vla_status vla_state_store(const float* x, int B, long long rows, int d, int bits, void* codes, float* scales, int N,
                           const int* slots, void* status, void* stream) {
    using namespace vla_layer;
    const vla_status st = check_cache(codes, scales, N, B, rows, d, bits, x, slots, status);
    if (st != VLA_OK || B == 0 || rows == 0) return st;
    const long long per = rows * d;
    const __int128 all = (__int128)N * per;
    const Region states = region(x, (__int128)B * per, 32), c = region(codes, all, bits), f = region(scales, all / 32, 32);
    if (!apart({c, f}, {states, region(slots, B, 32)})) return VLA_ERR_INVALID_ARG;
    const dim3 grid((unsigned)((per + BLOCK_VALUES - 1) / BLOCK_VALUES), (unsigned)B);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto* ds = static_cast<vla::DeviceStatus*>(status);
    if (bits == 8)
        vla_state_store_kernel<8><<<grid, STATE_THREADS, 0, s>>>(x, per, codes, scales, N, slots, ds);
    else
        vla_state_store_kernel<4><<<grid, STATE_THREADS, 0, s>>>(x, per, codes, scales, N, slots, ds);
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

vla_status vla_state_load(const void* codes, const float* scales, int N, const int* slots, int B, long long rows,
                          int d, int bits, float* x, void* status, void* stream) {
    using namespace vla_layer;
    const vla_status st = check_cache(codes, scales, N, B, rows, d, bits, x, slots, status);
    if (st != VLA_OK || B == 0 || rows == 0) return st;
    const long long per = rows * d;
    const __int128 all = (__int128)N * per;
    const Region states = region(x, (__int128)B * per, 32), c = region(codes, all, bits), f = region(scales, all / 32, 32);
    if (!apart({states}, {c, f, region(slots, B, 32)})) return VLA_ERR_INVALID_ARG;
    const dim3 grid((unsigned)((per + BLOCK_VALUES - 1) / BLOCK_VALUES), (unsigned)B);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto* ds = static_cast<vla::DeviceStatus*>(status);
    if (bits == 8)
        vla_state_load_kernel<8><<<grid, STATE_THREADS, 0, s>>>(codes, scales, N, slots, per, x, ds);
    else
        vla_state_load_kernel<4><<<grid, STATE_THREADS, 0, s>>>(codes, scales, N, slots, per, x, ds);
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

}  // extern "C"
