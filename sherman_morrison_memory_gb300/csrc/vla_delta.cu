// vla_delta.cu -- entry points of the gated delta rule (include/vla_layer.h), the
// forward launch and the single-token kernel.
#include <cmath>
#include <type_traits>

#include "vla_delta_host.h"

namespace vla_layer {
namespace {

// One token: S <- a S + b (v - a S k) k^T, o = scale S q. Bound by reading and writing S. Eight lanes hold a row,
// lane i the float4s i, i + 8, ... of it, so that a warp moves four rows in whole 128-byte lines; a warp has
// eight rows in flight. 256 sequences of 32 heads, d = 128: 156 us in a graph's replay, 6.9 TB/s; one sequence 4.4 us.
constexpr int STEP_THREADS = 128;
constexpr int STEP_ROWS = 32;  // rows of S a block handles

__device__ __forceinline__ float4 step4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 step4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(low_of(w.x), high_of(w.x), low_of(w.y), high_of(w.y));
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ float over_eight(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    return x + __shfl_xor_sync(0xffffffffu, x, 4);
}

template <int D, typename T>
__global__ void __launch_bounds__(STEP_THREADS) vla_delta_step_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                                      const T* __restrict__ v, int H,
                                                                      const float* __restrict__ log_decay,
                                                                      const float* __restrict__ beta, float scale,
                                                                      float* states, int N, const int* slots, T* o,
                                                                      vla::DeviceStatus* status) {
    constexpr int V = D / 32;  // float4s of a row in a lane
    const int blocks = D / STEP_ROWS;
    const int bh = blockIdx.x / blocks, row0 = (blockIdx.x % blocks) * STEP_ROWS, b = bh / H, h = bh % H;
    const int lane = threadIdx.x % 8, r0 = row0 + threadIdx.x / 8;
    const int slot = slot_of(slots, b, N, true, h == 0 && row0 == 0 ? status : nullptr);
    const size_t in = (size_t)bh * D;
    if (slot < 0) {
        if (lane == 0) o[in + r0] = o[in + r0 + 16] = (T)0.f;
        return;
    }
    float* S = states + ((size_t)slot * H + h) * D * D + lane * 4;
    float4 s[2][V];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < V; ++i) s[m][i] = step4(S + (size_t)(r0 + 16 * m) * D + 32 * i);
    const float a = log_decay ? expf(log_decay[bh]) : 1.f, bt = beta[bh];
    float4 kk[V], qq[V];
#pragma unroll
    for (int i = 0; i < V; ++i) kk[i] = step4(k + in + (lane + 8 * i) * 4), qq[i] = step4(q + in + (lane + 8 * i) * 4);
    float bad = 0.f;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        float at_k = 0.f, acc = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float4& x = s[m][i];
            x = make_float4(a * x.x, a * x.y, a * x.z, a * x.w);
            at_k = dot4(x, kk[i], at_k);
        }
        const float u = bt * ((float)v[in + r0 + 16 * m] - over_eight(at_k));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float4& x = s[m][i];
            x = make_float4(fmaf(u, kk[i].x, x.x), fmaf(u, kk[i].y, x.y), fmaf(u, kk[i].z, x.z), fmaf(u, kk[i].w, x.w));
            acc = dot4(x, qq[i], acc);
            bad = fmaf(x.x, 0.f, fmaf(x.y, 0.f, fmaf(x.z, 0.f, fmaf(x.w, 0.f, bad))));
            *reinterpret_cast<float4*>(S + (size_t)(r0 + 16 * m) * D + 32 * i) = x;
        }
        acc = over_eight(acc) * scale;
        bad = fmaf(acc, 0.f, bad);
        if (lane == 0) o[in + r0 + 16 * m] = (T)acc;
    }
    if (bad != bad && status) vla::record_failure(status, vla::BIT_NONFINITE, 3, bh, 0);
}

void take_options(DeltaArgs& p, const vla_options* opts) {
    p.wait_ns = 1000ull * (opts && opts->wait_limit_us ? opts->wait_limit_us : 2000000u);
    p.stall = opts && opts->test_stall_producer;
}

}  // namespace
}  // namespace vla_layer

extern "C" {

size_t vla_delta_scratch_bytes(vla_dtype dtype, int B, int H, int T, int d) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_dtype(dtype) || !good_d(d) || B == 0 || H == 0 || T == 0) return 0;
    return delta_scratch(nullptr, nullptr, dtype, B, H, T, d);
}

vla_status vla_delta_forward_ex(const vla_seq* q, const vla_seq* k, const vla_seq* v, vla_dtype dtype, int B, int H, int T,
                                int d, const vla_gate* log_decay, const vla_gate* beta, float scale, const int* lengths,
                                const float* S0, const vla_seq_out* o, float* S_out, void* status, void* stream,
                                const vla_options* opts) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_dtype(dtype) || !std::isfinite(scale)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if (B == 0 || H == 0) return VLA_OK;
    if (!S_out || !aligned(lengths, 4) || !aligned(S0, 16) || !aligned(S_out, 16) || !aligned(status, 16))
        return VLA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long states = (long long)B * H * d * d;
    const Region S_in = region(S0, states, 32), S_end = region(S_out, states, 32);
    if (!apart({S_end}, {S_in}, 1)) return VLA_ERR_INVALID_ARG;
    if (T == 0) return delta_copy_state(S_out, S0, (size_t)states, s);
    const int es = dtype == VLA_BF16 ? 2 : 4;
    if (!good_seq(q, B, H, T, es) || !good_seq(k, B, H, T, es) || !good_seq(v, B, H, T, es) || !good_seq(o, B, H, T, es) ||
        !good_gate(beta, B, H, T, false) || (log_decay && !good_gate(log_decay, B, H, T, false)))
        return VLA_ERR_INVALID_ARG;
    if (!apart({S_end, region(o, B, H, T, d, es)},
               {S_in, region(q, B, H, T, d, es), region(k, B, H, T, d, es), region(v, B, H, T, d, es),
                gate_region(log_decay, B, H, T), gate_region(beta, B, H, T), region(lengths, B, 32)}, 1))
        return VLA_ERR_INVALID_ARG;
    DeltaArgs p{};
    p.B = B, p.H = H, p.T = T;
    p.q = to_seq(q, B, H, T), p.k = to_seq(k, B, H, T), p.v = to_seq(v, B, H, T), p.out = to_seq(o, B, H, T);
    p.g = to_gate(log_decay, B, H, T), p.beta = to_gate(beta, B, H, T);
    p.scale = scale;
    p.lengths = lengths;
    p.S0 = S0, p.S = S_out;
    p.status = static_cast<vla::DeviceStatus*>(status);
    take_options(p, opts);
    return delta_pick(dtype, d, [&](auto tag, auto dim) { return delta_forward_run<decltype(dim)::value, decltype(tag), false>(p, s); });
}

vla_status vla_delta_backward_ex(const vla_seq* q, const vla_seq* k, const vla_seq* v, const vla_seq* dO, vla_dtype dtype,
                                 int B, int H, int T, int d, const vla_gate* log_decay, const vla_gate* beta, float scale,
                                 const int* lengths, const float* S0, const float* dS_T, const vla_seq_out* dq,
                                 const vla_seq_out* dk, const vla_seq_out* dv, const vla_gate_out* dlog_decay,
                                 const vla_gate_out* dbeta, float* dS0, void* scratch, size_t scratch_bytes, void* status,
                                 void* stream, const vla_options* opts) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_dtype(dtype) || !std::isfinite(scale)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if (B == 0 || H == 0) return VLA_OK;
    if (!aligned(lengths, 4) || !aligned(S0, 16) || !aligned(dS_T, 16) || !aligned(dS0, 16) || !aligned(status, 16))
        return VLA_ERR_INVALID_ARG;
    const long long states = (long long)B * H * d * d;
    const Region S_in = region(S0, states, 32), R_in = region(dS_T, states, 32), R_end = region(dS0, states, 32);
    if (!apart({R_end}, {S_in, R_in})) return VLA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return delta_copy_state(dS0, dS_T, (size_t)states, s);
    const int es = dtype == VLA_BF16 ? 2 : 4;
    if (!good_seq(q, B, H, T, es) || !good_seq(k, B, H, T, es) || !good_seq(v, B, H, T, es) || !good_seq(dO, B, H, T, es) ||
        !good_seq(dq, B, H, T, es) || !good_seq(dk, B, H, T, es) || !good_seq(dv, B, H, T, es) ||
        !good_gate(beta, B, H, T, false) || (log_decay && !good_gate(log_decay, B, H, T, false)) ||
        !good_gate(dbeta, B, H, T, true) || (dlog_decay && !good_gate(dlog_decay, B, H, T, true)))
        return VLA_ERR_INVALID_ARG;
    const size_t need = vla_delta_scratch_bytes(dtype, B, H, T, d);
    if (!scratch || !aligned(scratch, 256) || scratch_bytes < need) return VLA_ERR_INVALID_ARG;
    if (!apart({region(dq, B, H, T, d, es), region(dk, B, H, T, d, es), region(dv, B, H, T, d, es), R_end,
                gate_region(dlog_decay, B, H, T), gate_region(dbeta, B, H, T), region(scratch, need, 8)},
               {region(q, B, H, T, d, es), region(k, B, H, T, d, es), region(v, B, H, T, d, es), region(dO, B, H, T, d, es),
                S_in, R_in, gate_region(log_decay, B, H, T), gate_region(beta, B, H, T), region(lengths, B, 32)}))
        return VLA_ERR_INVALID_ARG;
    DeltaArgs p{};
    p.B = B, p.H = H, p.T = T;
    p.q = to_seq(q, B, H, T), p.k = to_seq(k, B, H, T), p.v = to_seq(v, B, H, T), p.dO = to_seq(dO, B, H, T);
    p.dq = to_seq(dq, B, H, T), p.dk = to_seq(dk, B, H, T), p.dv = to_seq(dv, B, H, T);
    p.g = to_gate(log_decay, B, H, T), p.beta = to_gate(beta, B, H, T);
    p.dg = to_gate(dlog_decay, B, H, T), p.dbeta = to_gate(dbeta, B, H, T);
    p.scale = scale;
    p.lengths = lengths;
    p.S0 = S0, p.dS_T = dS_T, p.dS0 = dS0;
    p.status = static_cast<vla::DeviceStatus*>(status);
    take_options(p, opts);
    delta_scratch(&p, scratch, dtype, B, H, T, d);
    return delta_backward_launch(p, dtype, d, s);
}

vla_status vla_delta_forward(const vla_seq* q, const vla_seq* k, const vla_seq* v, vla_dtype dtype, int B, int H, int T,
                             int d, const vla_gate* log_decay, const vla_gate* beta, float scale, const int* lengths,
                             const float* S0, const vla_seq_out* o, float* S_out, void* status, void* stream) {
    return vla_delta_forward_ex(q, k, v, dtype, B, H, T, d, log_decay, beta, scale, lengths, S0, o, S_out, status, stream,
                                nullptr);
}

vla_status vla_delta_backward(const vla_seq* q, const vla_seq* k, const vla_seq* v, const vla_seq* dO, vla_dtype dtype,
                              int B, int H, int T, int d, const vla_gate* log_decay, const vla_gate* beta, float scale,
                              const int* lengths, const float* S0, const float* dS_T, const vla_seq_out* dq,
                              const vla_seq_out* dk, const vla_seq_out* dv, const vla_gate_out* dlog_decay,
                              const vla_gate_out* dbeta, float* dS0, void* scratch, size_t scratch_bytes, void* status,
                              void* stream) {
    return vla_delta_backward_ex(q, k, v, dO, dtype, B, H, T, d, log_decay, beta, scale, lengths, S0, dS_T, dq, dk, dv,
                                 dlog_decay, dbeta, dS0, scratch, scratch_bytes, status, stream, nullptr);
}

vla_status vla_delta_step(const void* q, const void* k, const void* v, vla_dtype dtype, int B, int H, int d,
                          const float* log_decay, const float* beta, float scale, float* states, int N,
                          const int* slots, void* o, void* status, void* stream) {
    using namespace vla_layer;
    if (!good_sizes(B, H, 1) || N < 0 || !good_dtype(dtype) || !std::isfinite(scale)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if (!slots && B > N) return VLA_ERR_INVALID_ARG;
    if (B == 0 || H == 0) return VLA_OK;
    if (!q || !k || !v || !o || !beta || (!states && N > 0) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(o, 16) || !aligned(log_decay, 4) || !aligned(beta, 4) || !aligned(states, 16) || !aligned(slots, 4) ||
        !aligned(status, 16))
        return VLA_ERR_INVALID_ARG;
    const long long grid = (long long)B * H * (d / STEP_ROWS);
    if (grid > 2147483647LL) return VLA_ERR_INVALID_ARG;
    const long long heads = (long long)B * H, rows = heads * d;
    const int bits = dtype == VLA_BF16 ? 16 : 32;
    if (!apart({region(o, rows, bits), region(states, (__int128)N * H * d * d, 32)},
               {region(q, rows, bits), region(k, rows, bits), region(v, rows, bits), region(log_decay, heads, 32),
                region(beta, heads, 32), region(slots, B, 32)}))
        return VLA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto* ds = static_cast<vla::DeviceStatus*>(status);
    return delta_pick(dtype, d, [&](auto tag, auto dim) {
        using T = decltype(tag);
        vla_delta_step_kernel<decltype(dim)::value, T><<<(unsigned)grid, STEP_THREADS, 0, s>>>(
            static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), H, log_decay, beta, scale,
            states, N, slots, static_cast<T*>(o), ds);
        return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
    });
}

}  // extern "C"
