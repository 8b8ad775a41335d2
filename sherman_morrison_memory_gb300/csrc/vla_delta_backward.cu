// vla_delta_backward.cu -- the launches of the gated delta rule's gradients.
#include "vla_delta_backward.cuh"
#include "vla_delta_host.h"

namespace vla_layer {
namespace {

template <int D, typename T>
vla_status backward(DeltaArgs& p, cudaStream_t s) {
    vla_status st = delta_forward_run<D, T, true>(p, s);
    if (st != VLA_OK) return st;
    bool on_tc = false;
    if constexpr (sizeof(T) == 2)
        if ((on_tc = delta_on_tc(p))) st = delta_tc_pick<D, true, true>(p, s);
    if (!on_tc) st = delta_run<vla_delta_reverse_kernel<D, T>, D, typename DeltaReverse<D, T>::L>(p, s);
    if (st != VLA_OK) return st;
    using L = DeltaGrads<D, T>;
    const long long grid = (long long)p.B * p.H * p.blocks;
    if (grid > 2147483647LL) return VLA_ERR_INVALID_ARG;
    if (!allow_smem<vla_delta_grads_kernel<D, T>>(L::BYTES)) return VLA_ERR_CUDA;
    vla_delta_grads_kernel<D, T><<<(unsigned)grid, L::THREADS, L::BYTES, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

}  // namespace

vla_status delta_backward_launch(DeltaArgs& p, vla_dtype dtype, int d, cudaStream_t s) {
    return delta_pick(dtype, d, [&](auto tag, auto dim) { return backward<decltype(dim)::value, decltype(tag)>(p, s); });
}

}  // namespace vla_layer
