// vla_layer.cuh -- what the operators of include/vla_layer.h share: sequences
// with strides, eight values of a row at a time, status bits, argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "vla_device.cuh"
#include "vla_internal.h"
#include "vla_layer.h"
#include "vla_overlap.h"

namespace vla_layer {

constexpr int kRoleSlot = 4;

// element strides of a [B, H, T, d] sequence; a dimension of length 1 has stride 0
struct Seq {
    char* p;
    long long sb, sh, st;
};

template <typename T>
__device__ __forceinline__ T* row_of(const Seq& s, int b, int h, long long t) {
    return reinterpret_cast<T*>(s.p) + (b * s.sb + h * s.sh + t * s.st);
}

// Eight values of a row in two steps, so that several loads can be under way at once.
struct Raw8F {
    float4 a, b;
};
__device__ __forceinline__ Raw8F raw8(const float* p) {
    return Raw8F{*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4)};
}
__device__ __forceinline__ uint4 raw8(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void open8(const Raw8F& r, float (&x)[8]) {
    x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w, x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
}
__device__ __forceinline__ void open8(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    open8(raw8(p), x);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// exp(g n) for a whole number n >= 0: 1 for n = 0 also where g is -inf
__device__ __forceinline__ float decay_pow(float g, int n) { return n == 0 ? 1.f : expf(g * (float)n); }

// The decay over n tokens, exp(g n), for a state that is multiplied by it again
// and again: each factor is rounded, and what their roundings add up to is put
// right by the next ones, so that a slow decay stays the same over a long
// sequence (factors that are all rounded the same way can leave a state 1e-4
// off over 65,536 tokens). 1 + expm1(x) shows the rounding where it matters: near 1.
struct SlowDecay {
    float w, rest, inv;  // the rounded factor, how far (relative) it is below the true one, 1 / w
    float owed;          // ... and the product of all so far
    __device__ __forceinline__ SlowDecay(float g, int n) {  // n > 0
        const float m = expm1f(g * (float)n);
        w = 1.f + m;
        inv = w > 0.5f ? 1.f / w : 0.f;
        rest = (m - (w - 1.f)) * inv;
        owed = 0.f;
    }
    __device__ __forceinline__ float next() {
        owed += rest;
        const float v = fmaf(w, owed, w);
        owed = fmaf(w - v, inv, owed);
        return v;
    }
};

// The pool entry of sequence b, or -1 for none: a negative slot, or, recorded
// in the status, one out of range or (`unique`) one that an earlier sequence
// of the call has. Called by a whole block, which gets one answer.
__device__ __forceinline__ int slot_of(const int* slots, int b, int N, bool unique, vla::DeviceStatus* status) {
    if (!slots) return b;
    const int s = slots[b];
    if (s < 0) return -1;
    int bad = s >= N;
    if (unique) {
        for (int i = threadIdx.x; i < b; i += blockDim.x) bad |= slots[i] == s;
        bad = __syncthreads_or(bad);
    }
    if (!bad) return s;
    if (status && threadIdx.x == 0) vla::record_failure(status, vla_impl::kBitBadSlot, kRoleSlot, b, s);
    return -1;
}

// ---- host side -----------------------------------------------------------

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool good_d(int d) { return d == 32 || d == 64 || d == 96 || d == 128; }
inline bool good_dtype(vla_dtype t) { return t == VLA_F32 || t == VLA_BF16; }

// sizes that every index of the kernels can hold
inline bool good_sizes(int B, int H, int T) {
    if (B < 0 || H < 0 || T < 0) return false;
    const long long BH = (long long)B * H;
    return BH <= 2147483647LL && T <= 2147483647 - 256 && (unsigned long long)BH * (unsigned long long)T <= (1ull << 48);
}

inline bool good_seq(const void* data, long long sb, long long sh, long long st, int B, int H, int T, int es) {
    if (!data || !aligned(data, 16)) return false;
    const long long lim = 1LL << 40;  // bytes, of a tensor map's stride
    const long long s[3] = {sb, sh, st};
    const int n[3] = {B, H, T};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (s[i] <= 0 || s[i] >= lim / es || (s[i] * es) % 16 != 0)) return false;
    return true;
}
inline bool good_seq(const vla_seq* s, int B, int H, int T, int es) {
    return s && good_seq(s->data, s->stride_b, s->stride_h, s->stride_t, B, H, T, es);
}
inline bool good_seq(const vla_seq_out* s, int B, int H, int T, int es) {
    return s && good_seq(s->data, s->stride_b, s->stride_h, s->stride_t, B, H, T, es);
}
template <typename S>
inline Seq to_seq(const S* s, int B, int H, int T) {
    return Seq{(char*)s->data, B > 1 ? s->stride_b : 0, H > 1 ? s->stride_h : 0, T > 1 ? s->stride_t : 0};
}

// SMs of the current device, asked once per device (152 where none answers)
inline int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Dynamic shared memory of kernel K raised to `bytes`, once per device.
template <auto K>
inline bool allow_smem(int bytes) {
    static std::atomic<bool> done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (done[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done[dev].store(true, std::memory_order_release);
    return true;
}

}  // namespace vla_layer
