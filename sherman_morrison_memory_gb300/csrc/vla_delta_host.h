// vla_delta_host.h -- host side that the gated delta rule's translation units share.
#pragma once

#include <type_traits>

#include "vla_delta.cuh"
#include "vla_delta_forward.cuh"
#include "vla_delta_tc.cuh"
#include "vla_maps.h"

namespace vla_layer {

vla_status delta_backward_launch(DeltaArgs& p, vla_dtype dtype, int d, cudaStream_t s);

template <typename G>
inline bool good_gate(const G* g, int B, int H, int T, bool out) {
    if (!g || !g->data || !aligned(g->data, 4)) return false;
    const long long s[3] = {g->stride_b, g->stride_h, g->stride_t}, lim = 1LL << 40;
    const int n[3] = {B, H, T};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (s[i] < (out ? 1 : 0) || s[i] >= lim)) return false;
    return true;
}
template <typename G>
inline Gate to_gate(const G* g, int B, int H, int T) {
    if (!g) return Gate{};
    return Gate{const_cast<float*>(g->data), B > 1 ? g->stride_b : 0, H > 1 ? g->stride_h : 0, T > 1 ? g->stride_t : 0};
}
// a gate's memory: a dimension of stride 0 is the same values again
template <typename G>
inline Region gate_region(const G* g, int B, int H, int T) {
    if (!g) return Region{};
    auto len = [](int n, long long st) { return st == 0 ? 1 : n; };
    const int b = len(B, g->stride_b), h = len(H, g->stride_h), t = len(T, g->stride_t);
    return Region{reinterpret_cast<uintptr_t>(g->data), 4, {b > 1 ? g->stride_b * 4 : 0, h > 1 ? g->stride_h * 4 : 0, t > 1 ? g->stride_t * 4 : 0},
                  {b, h, t}};
}

template <typename F>
inline vla_status delta_pick(vla_dtype dtype, int d, F f) {
    auto with = [&](auto tag) {
        switch (d) {
            case 32: return f(tag, std::integral_constant<int, 32>{});
            case 64: return f(tag, std::integral_constant<int, 64>{});
            case 96: return f(tag, std::integral_constant<int, 96>{});
            default: return f(tag, std::integral_constant<int, 128>{});
        }
    };
    return dtype == VLA_BF16 ? with(__nv_bfloat16{}) : with(float{});
}

// Rows of S of a block on the warp-level path: as many as it can have, or a half, a quarter, ... while all blocks run at
// once, an SM each. Each block prepares its chunks for itself and one fills an SM's registers, so fewer rows shorten a
// chunk but not the work: fp32 outputs of 1,024 tokens, d = 128: 16 heads 183 us with 64 rows, 144 with 32, 139 with 16;
// 38 heads 184, 158, 299; 76 heads 189, 319, 598; 304 heads 750, 1,275, 2,290. d = 64: 16 heads 131, 103, 92; 76 heads
// 131, 119, 222; 100 heads 131, 213, 308.
inline int delta_rows(long long heads, int d, int rows) {
    while (rows % 32 == 0 && heads * (d / (rows / 2)) <= sm_count()) rows /= 2;
    return rows;
}

// One of the recurrences: two warps for 16 rows and the helpers.
template <auto K, int D, typename L>
inline vla_status delta_run(DeltaArgs& p, cudaStream_t s) {
    const long long heads = (long long)p.B * p.H;
    p.rows = delta_rows(heads, D, MOST_ROWS<D>);
    const long long grid = heads * (D / p.rows);
    if (grid > 2147483647LL) return VLA_ERR_INVALID_ARG;
    if (!allow_smem<K>(L::BYTES)) return VLA_ERR_CUDA;
    K<<<(unsigned)grid, p.rows * 4 + HELPERS, L::BYTES, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

// Whether a bf16 call's recurrences run on tcgen05, one block to an SM, or as warp-level products, which start sooner and
// can be cut finer. Outputs, us, warp-level against tcgen05, of 8 heads, 64 heads, 304 heads:
//   tokens  d = 32                                d = 64                               d = 128
//   64      8.2, 8.3;  8.3, 8.5;   10.4, 14.4     8.3, 8.5;   8.5, 10.3;  18.5, 16.5   10.3, 10.4; 12.4, 10.4; 40.0, 24.6
//   128     10.3, 10.4; 10.4, 10.4; 14.5, 18.6    10.6, 11.6; 12.3, 12.3; 26.7, 20.6   12.4, 13.7; 18.4, 14.4; 61.6, 34.9
//   256     16.4, 14.5; 16.5, 14.5; 22.7, 28.0    16.5, 16.6; 18.5, 16.5; 43.1, 32.8   18.6, 20.6; 28.9, 20.6; 110, 57.5
// and d = 96 between the last two; gradients of 304 heads of 64 tokens d = 32 28.7, 36.9, d = 64 53.4, 43.3, d = 128 135,
// 88.3, of 256 tokens 78.0, 88.1; 156, 121; 409, 269. Heads would decide better (many of d = 32 are sooner on the warp level at
// any of these lengths, many of d = 128 on tcgen05 already at 64 tokens), but then a head's bits would depend on the other
// heads of its call. By the tokens alone they do not, and the limit is where few heads of any d lose little.
inline bool delta_on_tc(const DeltaArgs& p) { return p.T > 64; }

template <int D, int R, bool TAPE, bool BACK = false>
inline vla_status delta_tc_run(DeltaArgs& p, cudaStream_t s) {
    using L = DeltaTc<D, R, TAPE>;
    const long long grid = (long long)p.B * p.H * (D > R ? D / R : 1);
    if (grid > 2147483647LL) return VLA_ERR_INVALID_ARG;
    DeltaMaps maps;
    const Seq* seq[4] = {&p.k, &p.q, &p.v, &p.dO};
    for (int i = 0; i < (TAPE ? 4 : 3); ++i) {
        const vla_seq x{seq[i]->p, seq[i]->sb, seq[i]->sh, seq[i]->st};
        if (!make_map(&maps.m[i], &x, p.B, p.H, p.T, D, DC)) return VLA_ERR_CUDA;
    }
    if constexpr (BACK) {
        if (!allow_smem<vla_delta_tc_reverse_kernel<D, R>>(L::BYTES)) return VLA_ERR_CUDA;
        vla_delta_tc_reverse_kernel<D, R><<<(unsigned)grid, L::THREADS, L::BYTES, s>>>(p, maps);
    } else {
        if (!allow_smem<vla_delta_tc_kernel<D, R, TAPE>>(L::BYTES)) return VLA_ERR_CUDA;
        vla_delta_tc_kernel<D, R, TAPE><<<(unsigned)grid, L::THREADS, L::BYTES, s>>>(p, maps);
    }
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

// A bf16 recurrence on tcgen05: heads of d = 128 take two blocks where that is sooner done, a block of 64 rows taking
// 5/8 to 2/3 of the time of one of 128 (4,096 tokens: 227 us and 353). Outputs of 76 heads, one block and two: 350 and
// 228 us; 100 heads 355, 447; 153 heads 680, 665; 304 heads 729, 897. Gradients, whose third launch is the same: 1,322, 1,016;
// 1,473, 1,678; 2,633, 2,518; 3,576, 4,020.
template <int D, bool TAPE, bool BACK = false>
inline vla_status delta_tc_pick(DeltaArgs& p, cudaStream_t s) {
    if constexpr (D == 128) {
        const long long heads = (long long)p.B * p.H, sms = sm_count();
        if ((2 * heads + sms - 1) / sms * 5 < (heads + sms - 1) / sms * 8) return delta_tc_run<D, 64, TAPE, BACK>(p, s);
    }
    return delta_tc_run<D, (D > 64 ? 128 : 64), TAPE, BACK>(p, s);
}

// The forward recurrence, or (TAPE) what its gradients need of it.
template <int D, typename T, bool TAPE>
inline vla_status delta_forward_run(DeltaArgs& p, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (delta_on_tc(p)) return delta_tc_pick<D, TAPE>(p, s);
    return delta_run<vla_delta_forward_kernel<D, T, TAPE>, D, typename DeltaForward<D, T, TAPE>::L>(p, s);
}

inline vla_status delta_copy_state(float* dst, const float* src, size_t n, cudaStream_t s) {
    if (!dst || dst == src || n == 0) return VLA_OK;
    const cudaError_t e = src ? cudaMemcpyAsync(dst, src, n * sizeof(float), cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(dst, 0, n * sizeof(float), s);
    return e == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

// What a backward call keeps between its launches, laid out from `base` (p null: its bytes alone).
inline size_t delta_scratch(DeltaArgs* p, void* base, vla_dtype dtype, int B, int H, int T, int d) {
    const int span = dtype == VLA_BF16 ? BLOCK<__nv_bfloat16> : BLOCK<float>;
    const int blocks = (T + span - 1) / span;
    const size_t heads = (size_t)B * H, states = heads * (blocks + 1) * d * d, per_warp = heads * (d / 16) * T;
    size_t at = 0;
    auto take = [&](float** to, size_t n) {
        if (p) *to = reinterpret_cast<float*>(static_cast<char*>(base) + at);
        at += (n * sizeof(float) + 255) / 256 * 256;
    };
    DeltaArgs none;
    DeltaArgs& a = p ? *p : none;
    take(&a.E, heads * T * d);
    take(&a.before, states);
    take(&a.behind, states);
    take(&a.od, per_warp);
    take(&a.vd, per_warp);
    take(&a.bd, per_warp);
    a.blocks = blocks;
    return at;
}

}  // namespace vla_layer
