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

// Rows of S of a block: as many as it can have, or a half, a quarter, ... while the blocks are fewer than the SMs.
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

// Tokens behind which a bf16 call's forward recurrence runs on tcgen05.
constexpr int DELTA_TC = 64;

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

// A bf16 recurrence on tcgen05: few heads of d = 128 take two blocks each.
template <int D, bool TAPE, bool BACK = false>
inline vla_status delta_tc_pick(DeltaArgs& p, cudaStream_t s) {
    if constexpr (D == 128) {
        if ((long long)p.B * p.H * 2 <= sm_count()) return delta_tc_run<D, 64, TAPE, BACK>(p, s);
    }
    return delta_tc_run<D, (D > 64 ? 128 : 64), TAPE, BACK>(p, s);
}

// The forward recurrence, or (TAPE) what its gradients need of it.
template <int D, typename T, bool TAPE>
inline vla_status delta_forward_run(DeltaArgs& p, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (p.T > DELTA_TC) return delta_tc_pick<D, TAPE>(p, s);
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
    take(&a.ends, heads * blocks * (d / 8));
    a.blocks = blocks;
    return at;
}

}  // namespace vla_layer
