// vla_norm.cuh -- layer norm of each head's readout and its gradients
// (include/vla_layer.h).
//
// A row is the d values of one (b, h, t). Both passes move each value once
// and are bound by memory. A lane holds groups of eight consecutive values of a
// row in fp32 (16 bytes of bf16) and a row's sums are butterflies over its
// lanes: 4 or 8 in the forward pass, with more groups a lane, d / 8 in the
// backward pass, which holds more of each; the mean is taken before the squares
// of the differences, both from registers. A thread has rows under way ahead. A block stays on one head, with that
// head's weight and bias in registers.
//
// Gradients, with g = dy weight and n = (x - mean) rstd:
//   dx = rstd (g - mean(g) - n mean(g n)),  dweight = sum dy n,  dbias = sum dy.
// The sums over the rows: each thread over its own rows, the block's threads
// through shared memory, the blocks of a head in a second launch, all in an
// order that the sizes fix.
#pragma once

#include "vla_layer.cuh"

namespace vla_layer {
namespace {

constexpr int NORM_THREADS = 256;
constexpr int ROWS = 256;  // rows a block handles

struct NormArgs {
    Seq x, dy, out;
    const float *weight, *bias;
    float *mean, *rstd;
    float* partial;  // [gridDim.x][2][d]
    int H, T, tb, shared;
    float eps;
};

template <int D>
struct Lanes {
    static constexpr int USED = D / 8;                    // lanes that hold a row
    static constexpr int W = D == 96 ? 16 : D / 8;        // lanes set aside for it (a power of two)
    static constexpr int PER = NORM_THREADS / W;               // rows of a block at a time
};

template <int W>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int m = 1; m < W; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// Lanes of a row in the forward pass: few, so that the two sums take few
// shuffles, each with V groups of eight values (W lanes apart).
template <int D>
struct ForwardLanes {
    static constexpr int W = D == 128 ? 8 : 4, V = D / 8 / W;
    static constexpr int PER = NORM_THREADS / W;
    static constexpr int U = V >= 2 ? 2 : 4;  // rows of a thread under way at once
    static_assert(ROWS % (U * PER) == 0, "whole passes");
};

template <int D, typename T>
__global__ void __launch_bounds__(NORM_THREADS, D == 96 || sizeof(T) == 4 ? 2 : 3)
    vla_head_norm_kernel(const NormArgs a) {
    using L = ForwardLanes<D>;
    constexpr int V = L::V;
    const int bh = blockIdx.x / a.tb, b = bh / a.H, h = bh % a.H;
    const int lane = threadIdx.x % L::W, r0 = threadIdx.x / L::W;
    const long long t0 = (long long)(blockIdx.x % a.tb) * ROWS;
    float w[V][8], bi[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[v][i] = 1.f, bi[v][i] = 0.f;
        const long long at = (a.shared ? 0LL : (long long)h * D) + (lane + v * L::W) * 8;
        if (a.weight) load8(a.weight + at, w[v]);
        if (a.bias) load8(a.bias + at, bi[v]);
    }
#pragma unroll 1
    for (int r = r0; r < ROWS; r += L::U * L::PER) {
        decltype(raw8((const T*)nullptr)) raw[L::U][V];
#pragma unroll
        for (int k = 0; k < L::U; ++k) {
            const long long t = t0 + r + k * L::PER;
            const T* x = row_of<T>(a.x, b, h, t) + lane * 8;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                raw[k][v] = {};
                if (t < a.T) raw[k][v] = raw8(x + v * L::W * 8);
            }
        }
#pragma unroll
        for (int k = 0; k < L::U; ++k) {
            const long long t = t0 + r + k * L::PER;
            float x[V][8], s = 0.f, q = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                open8(raw[k][v], x[v]);
#pragma unroll
                for (int i = 0; i < 8; ++i) s += x[v][i];
            }
            const float mean = row_sum<L::W>(s) * (1.f / D);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[v][i] -= mean;
                    q = fmaf(x[v][i], x[v][i], q);
                }
            const float rstd = rsqrtf(row_sum<L::W>(q) * (1.f / D) + a.eps);
            if (t < a.T) {
                T* y = row_of<T>(a.out, b, h, t) + lane * 8;
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[v][i] = fmaf(x[v][i] * rstd, w[v][i], bi[v][i]);
                    store8(y + v * L::W * 8, x[v]);
                }
                if (lane == 0) {
                    if (a.mean) a.mean[(long long)bh * a.T + t] = mean;
                    if (a.rstd) a.rstd[(long long)bh * a.T + t] = rstd;
                }
            }
        }
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(NORM_THREADS) vla_head_norm_backward_kernel(const NormArgs a) {
    using L = Lanes<D>;
    __shared__ float part[2][L::PER][D];
    const int bh = blockIdx.x / a.tb, b = bh / a.H, h = bh % a.H;
    const int lane = threadIdx.x % L::W, r0 = threadIdx.x / L::W;
    const bool on = lane < L::USED;
    const int col = lane * 8;
    const long long t0 = (long long)(blockIdx.x % a.tb) * ROWS;
    float w[8], dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f, dw[i] = 0.f, db[i] = 0.f;
    if (on && a.weight) load8(a.weight + (a.shared ? 0LL : (long long)h * D) + col, w);
    constexpr int U = sizeof(T) == 4 ? 2 : 4;  // rows under way at once
    static_assert(ROWS % (U * L::PER) == 0, "whole passes");
#pragma unroll 1
    for (int r = r0; r < ROWS; r += U * L::PER) {
        decltype(raw8((const T*)nullptr)) rx[U], rg[U];
        float mean[U], rstd[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const long long t = t0 + r + k * L::PER;
            rx[k] = {}, rg[k] = {}, mean[k] = rstd[k] = 0.f;
            if (on && t < a.T) {
                rx[k] = raw8(row_of<T>(a.x, b, h, t) + col);
                rg[k] = raw8(row_of<T>(a.dy, b, h, t) + col);
                mean[k] = a.mean[(long long)bh * a.T + t];
                rstd[k] = a.rstd[(long long)bh * a.T + t];
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const long long t = t0 + r + k * L::PER;
            float x[8], g[8], s = 0.f, p = 0.f;
            open8(rx[k], x);
            open8(rg[k], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = (x[i] - mean[k]) * rstd[k];
                dw[i] = fmaf(g[i], x[i], dw[i]);
                db[i] += g[i];
                g[i] *= w[i];
                s += g[i];
                p = fmaf(g[i], x[i], p);
            }
            s = row_sum<L::W>(s) * (1.f / D);
            p = row_sum<L::W>(p) * (1.f / D);
            if (on && t < a.T) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = (g[i] - s - x[i] * p) * rstd[k];
                store8(row_of<T>(a.out, b, h, t) + col, x);
            }
        }
    }
    if (!a.partial) return;
    if (on) {
        store8(&part[0][r0][col], dw);
        store8(&part[1][r0][col], db);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += NORM_THREADS) {
        float s = 0.f;
#pragma unroll 8
        for (int r = 0; r < L::PER; ++r) s += part[i / D][r][i % D];
        a.partial[(long long)blockIdx.x * 2 * D + i] = s;
    }
}

// dweight, dbias of head h (all heads where shared): the blocks' sums
// [B][H][tb][2][D], 32 threads a column, each over every 32nd block, and the
// threads' sums in order.
constexpr int SUMS_THREADS = 1024;

template <int D>
__global__ void __launch_bounds__(SUMS_THREADS) vla_head_norm_sums_kernel(const float* __restrict__ partial, int B, int H,
                                                                          int tb, int shared, float* dw, float* db) {
    __shared__ float sums[32][33];
    const int col = threadIdx.x % 32, k = threadIdx.x / 32;
    const int i = blockIdx.y * 32 + col;  // of the 2 D columns
    const int h = blockIdx.x;
    const long long n = (long long)B * tb * (shared ? H : 1);
    float s = 0.f;
#pragma unroll 8
    for (long long m = k; m < n; m += 32) {
        const long long blk = shared ? m : (m / tb * H + h) * tb + m % tb;
        s += partial[blk * 2 * D + i];
    }
    sums[k][col] = s;
    __syncthreads();
    if (k == 0) {
#pragma unroll
        for (int j = 1; j < 32; ++j) s += sums[j][col];
        (i < D ? dw : db)[(long long)h * D + i % D] = s;
    }
}

int blocks_per_head(int T) { return (T + ROWS - 1) / ROWS; }

template <int D>
void norm_launch(bool backward, vla_dtype dt, const NormArgs& a, unsigned grid, cudaStream_t s) {
    if (backward) {
        if (dt == VLA_BF16)
            vla_head_norm_backward_kernel<D, __nv_bfloat16><<<grid, NORM_THREADS, 0, s>>>(a);
        else
            vla_head_norm_backward_kernel<D, float><<<grid, NORM_THREADS, 0, s>>>(a);
    } else {
        if (dt == VLA_BF16)
            vla_head_norm_kernel<D, __nv_bfloat16><<<grid, NORM_THREADS, 0, s>>>(a);
        else
            vla_head_norm_kernel<D, float><<<grid, NORM_THREADS, 0, s>>>(a);
    }
}

vla_status norm_dispatch(bool backward, vla_dtype dt, int d, const NormArgs& a, long long grid, cudaStream_t s) {
    if (grid > 2147483647LL) return VLA_ERR_INVALID_ARG;
    switch (d) {
        case 32: norm_launch<32>(backward, dt, a, (unsigned)grid, s); break;
        case 64: norm_launch<64>(backward, dt, a, (unsigned)grid, s); break;
        case 96: norm_launch<96>(backward, dt, a, (unsigned)grid, s); break;
        default: norm_launch<128>(backward, dt, a, (unsigned)grid, s); break;
    }
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

}  // namespace
}  // namespace vla_layer

extern "C" {

size_t vla_head_norm_scratch_bytes(int B, int H, int T, int d) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_d(d)) return 0;
    return (size_t)B * H * blocks_per_head(T) * 2 * d * sizeof(float);
}

vla_status vla_head_norm(const vla_seq* x, vla_dtype dtype, int B, int H, int T, int d, const float* weight,
                         const float* bias, int shared, float eps, const vla_seq_out* y, float* mean, float* rstd,
                         void* stream) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_dtype(dtype)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || eps > 3.4e38f) return VLA_ERR_INVALID_ARG;
    if (B == 0 || H == 0 || T == 0) return VLA_OK;
    const int es = dtype == VLA_BF16 ? 2 : 4;
    if (!good_seq(x, B, H, T, es) || !good_seq(y, B, H, T, es) || !aligned(weight, 16) || !aligned(bias, 16) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return VLA_ERR_INVALID_ARG;
    const long long weights = (shared ? 1LL : (long long)H) * d, stats = (long long)B * H * T;
    if (!apart({region(y, B, H, T, d, es), region(mean, stats, 32), region(rstd, stats, 32)},
               {region(x, B, H, T, d, es), region(weight, weights, 32), region(bias, weights, 32)}, 1))
        return VLA_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = to_seq(x, B, H, T);
    a.out = to_seq(y, B, H, T);
    a.weight = weight;
    a.bias = bias;
    a.mean = mean;
    a.rstd = rstd;
    a.H = H;
    a.T = T;
    a.tb = blocks_per_head(T);
    a.shared = shared != 0;
    a.eps = eps;
    return norm_dispatch(false, dtype, d, a, (long long)B * H * a.tb, static_cast<cudaStream_t>(stream));
}

vla_status vla_head_norm_backward(const vla_seq* dy, const vla_seq* x, vla_dtype dtype, int B, int H, int T, int d,
                                  const float* weight, int shared, const float* mean, const float* rstd,
                                  const vla_seq_out* dx, float* dweight, float* dbias, void* scratch,
                                  size_t scratch_bytes, void* stream) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_dtype(dtype)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if ((dweight == nullptr) != (dbias == nullptr) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return VLA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0 || H == 0 || T == 0) {
        const size_t n = (size_t)(shared ? (d) : (size_t)H * d) * sizeof(float);
        if (!dweight || n == 0) return VLA_OK;
        const bool ok = cudaMemsetAsync(dweight, 0, n, s) == cudaSuccess && cudaMemsetAsync(dbias, 0, n, s) == cudaSuccess;
        return ok ? VLA_OK : VLA_ERR_CUDA;
    }
    const int es = dtype == VLA_BF16 ? 2 : 4;
    if (!good_seq(x, B, H, T, es) || !good_seq(dy, B, H, T, es) || !good_seq(dx, B, H, T, es) || !aligned(weight, 16) ||
        !mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4))
        return VLA_ERR_INVALID_ARG;
    if (dweight && (!scratch || !aligned(scratch, 16) || scratch_bytes < vla_head_norm_scratch_bytes(B, H, T, d)))
        return VLA_ERR_INVALID_ARG;
    const long long weights = (shared ? 1LL : (long long)H) * d, stats = (long long)B * H * T;
    const long long parts = dweight ? (long long)vla_head_norm_scratch_bytes(B, H, T, d) : 0;
    if (!apart({region(dx, B, H, T, d, es), region(dweight, weights, 32), region(dbias, weights, 32), region(scratch, parts, 8)},
               {region(x, B, H, T, d, es), region(dy, B, H, T, d, es), region(weight, weights, 32), region(mean, stats, 32),
                region(rstd, stats, 32)}, 2))
        return VLA_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = to_seq(x, B, H, T);
    a.dy = to_seq(dy, B, H, T);
    a.out = to_seq(dx, B, H, T);
    a.weight = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.partial = dweight ? static_cast<float*>(scratch) : nullptr;
    a.H = H;
    a.T = T;
    a.tb = blocks_per_head(T);
    a.shared = shared != 0;
    const vla_status st = norm_dispatch(true, dtype, d, a, (long long)B * H * a.tb, s);
    if (st != VLA_OK || !dweight) return st;
    const dim3 grid((unsigned)(shared ? 1 : H), (unsigned)(2 * d / 32));
    switch (d) {
        case 32: vla_head_norm_sums_kernel<32><<<grid, SUMS_THREADS, 0, s>>>(a.partial, B, H, a.tb, a.shared, dweight, dbias); break;
        case 64: vla_head_norm_sums_kernel<64><<<grid, SUMS_THREADS, 0, s>>>(a.partial, B, H, a.tb, a.shared, dweight, dbias); break;
        case 96: vla_head_norm_sums_kernel<96><<<grid, SUMS_THREADS, 0, s>>>(a.partial, B, H, a.tb, a.shared, dweight, dbias); break;
        default: vla_head_norm_sums_kernel<128><<<grid, SUMS_THREADS, 0, s>>>(a.partial, B, H, a.tb, a.shared, dweight, dbias); break;
    }
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

}  // extern "C"
