// vla_decay_host.cuh -- linear attention with a decay per head: entry points, the
// cut into segments, the single-token kernel (include/vla_layer.h).
#pragma once

#include <algorithm>
#include <cmath>

#include "vla_decay.cuh"
#include "vla_decay_fma.cuh"
#include "vla_decay_tc.cuh"
#include "vla_maps.h"

namespace vla_layer {
namespace {

// States of the segments (each its own, from zero) to the states they start
// from: the running sum over the segments in the role's order, with the whole
// decays between; the sum over all of them is the final state. A thread has
// four values of S, and up to eight segments' of them under way at once: it
// writes where it reads, so the compiler would wait for each.
struct ScanRole {
    const float* init;
    float* fin;
    int init_t;   // init holds the transposed state (of a role without fin)
    int reverse;
};
struct ScanArgs {
    ScanRole role[2];
};

constexpr int SCAN_THREADS = 128;

// exp(g n) s where the factor alone may overflow (g > 0), a part of the tokens at a time
__device__ __noinline__ float grown(float s, float g, int n) {
    while (n > 0 && s != 0.f && fabsf(s) < __int_as_float(0x7F800000)) {
        const int m = min(n, max(1, (int)(80.f / g)));
        s *= expf(g * (float)m);
        n -= m;
    }
    return s;
}

template <int D>
__global__ void __launch_bounds__(SCAN_THREADS) vla_decay_scan_kernel(const __grid_constant__ DecayArgs p,
                                                                      const __grid_constant__ ScanArgs q) {
    constexpr int BLOCKS = D * D / 4 / SCAN_THREADS, AHEAD = 8;
    const int bh = p.bh0 + blockIdx.x / BLOCKS, i = ((blockIdx.x % BLOCKS) * SCAN_THREADS + threadIdx.x) * 4;
    const int b = bh / p.H, h = bh % p.H;
    const ScanRole& r = q.role[blockIdx.y];
    const float g = p.log_decay[h];
    const int x = i / D, y = i % D;  // four columns of a row
    const size_t at = (size_t)bh * D * D;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r.init) {
        const float* m = r.init + at;
        s = r.init_t ? make_float4(m[y * D + x], m[(y + 1) * D + x], m[(y + 2) * D + x], m[(y + 3) * D + x])
                     : *reinterpret_cast<const float4*>(m + i);
    }
    float4* seg = reinterpret_cast<float4*>(seg_of(p, blockIdx.y, bh, 0, D) + i);
    auto place = [&](int k) { return r.reverse ? p.nseg - 1 - k : k; };
    auto join = [&](const float4& own, float4 w) {
        s = make_float4(fmaf(w.x, s.x, own.x), fmaf(w.y, s.y, own.y), fmaf(w.z, s.z, own.z), fmaf(w.w, s.w, own.w));
    };
    if (g * (float)p.seg_len > 80.f) {  // a segment's factor may overflow
        for (int k = 0; k < p.nseg; ++k) {
            const int n = span_of(p, b, place(k)).n;
            float4& at_k = seg[(size_t)place(k) * (D * D / 4)];
            const float4 own = at_k;
            at_k = s;
            s = make_float4(grown(s.x, g, n), grown(s.y, g, n), grown(s.z, g, n), grown(s.w, g, n));
            join(own, make_float4(1.f, 1.f, 1.f, 1.f));
        }
    } else {
        SlowDecay slow(g, p.seg_len);
        for (int k0 = 0; k0 < p.nseg; k0 += AHEAD) {
            float4 own[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (k0 + k < p.nseg) own[k] = seg[(size_t)place(k0 + k) * (D * D / 4)];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (k0 + k >= p.nseg) break;
                const int m = place(k0 + k);
                const int n = span_of(p, b, m).n;
                const float w = n < p.seg_len ? decay_pow(g, n) : slow.next();
                seg[(size_t)m * (D * D / 4)] = s;
                join(own[k], make_float4(w, w, w, w));
            }
        }
    }
    if (r.fin) {
        *reinterpret_cast<float4*>(r.fin + at + i) = s;
        const float bad = fmaf(s.x, 0.f, fmaf(s.y, 0.f, fmaf(s.z, 0.f, s.w * 0.f)));
        if (bad != bad && p.status) vla::record_failure(p.status, vla::BIT_NONFINITE, 3, bh, p.T);
    }
}

// One token: S <- l S + v k^T, o = scale S q. Bound by reading and writing S.
// Eight lanes hold a row, lane i the float4s i, i + 8, ... of it, so that a
// warp moves four rows in whole 128-byte lines; a warp has eight rows in
// flight.
constexpr int STEP_THREADS = 128;
constexpr int STEP_ROWS = 32;  // rows of S a block handles

template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float4*>(p);
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}

template <int D, typename T>
__global__ void __launch_bounds__(STEP_THREADS) vla_decay_step_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                                      const T* __restrict__ v, int H,
                                                                      const float* __restrict__ log_decay, float scale,
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
    float4* S = reinterpret_cast<float4*>(states + ((size_t)slot * H + h) * D * D);
    float4 s[2][V];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < V; ++i) s[m][i] = S[(size_t)(r0 + 16 * m) * (D / 4) + lane + 8 * i];
    const float l = expf(log_decay[h]);
    float4 kk[V], qq[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        kk[i] = load4(k + in + (lane + 8 * i) * 4);
        qq[i] = load4(q + in + (lane + 8 * i) * 4);
    }
    float bad = 0.f;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const float vv = (float)v[in + r0 + 16 * m];
        float acc = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float4& x = s[m][i];
            x.x = fmaf(l, x.x, vv * kk[i].x);
            x.y = fmaf(l, x.y, vv * kk[i].y);
            x.z = fmaf(l, x.z, vv * kk[i].z);
            x.w = fmaf(l, x.w, vv * kk[i].w);
            acc = fmaf(x.x, qq[i].x, fmaf(x.y, qq[i].y, fmaf(x.z, qq[i].z, fmaf(x.w, qq[i].w, acc))));
            bad = fmaf(x.x, 0.f, fmaf(x.y, 0.f, fmaf(x.z, 0.f, fmaf(x.w, 0.f, bad))));
            S[(size_t)(r0 + 16 * m) * (D / 4) + lane + 8 * i] = x;
        }
        acc += __shfl_xor_sync(0xffffffffu, acc, 1);
        acc += __shfl_xor_sync(0xffffffffu, acc, 2);
        acc += __shfl_xor_sync(0xffffffffu, acc, 4);
        acc *= scale;
        bad = fmaf(acc, 0.f, bad);
        if (lane == 0) o[in + r0 + 16 * m] = (T)acc;
    }
    if (bad != bad && status) vla::record_failure(status, vla::BIT_NONFINITE, 3, bh, 0);
}

void take_options(DecayArgs& p, const vla_options* opts) {
    p.wait_ns = 1000ull * (opts && opts->wait_limit_us ? opts->wait_limit_us : 2000000u);
    p.stall = opts && opts->test_stall_producer;
}

// A launch's heads and their cut into segments.
struct Cut {
    int bh0, bhs, nseg, seg_len;
};

// The time of so many blocks, in that of one with an SM to itself. The bf16
// kernel has an SM to itself; the fp32 kernel's blocks share one, but leave little
// idle to share. (us a 64 tokens for 1, 2, 3, .. of them an SM: d = 32 8.5, 9, 11
// and, for 7, 18.5; d = 64 10.8, 17, 25; d = 96 15.5, 27.5; d = 128 23.)
double waves(long long blocks, int d, vla_dtype dt) {
    int fit = 1;
    double more = 0;
    if (dt == VLA_F32 && d == 32) fit = FmaLay<32, float>::OCC, more = 0.2;
    if (dt == VLA_F32 && d == 64) fit = FmaLay<64, float>::OCC, more = 0.65;
    if (dt == VLA_F32 && d == 96) fit = FmaLay<96, float>::OCC, more = 0.77;
    const long long sms = sm_count(), full = blocks / (sms * fit), rest = (blocks - full * sms * fit + sms - 1) / sms;
    return (double)full * (1 + more * (fit - 1)) + (rest ? 1 + more * (double)(rest - 1) : 0);
}

// what a block's start and end take, in chunks of 64 tokens
double ends_of(vla_dtype dt) { return dt == VLA_BF16 ? 6 : 0.5; }

// The cut of `heads` heads, each `roles` runs of blocks for the outputs and
// `state_roles` for the segments' own states, into segments; returns its time.
// A cut costs the second pass, over two of the three sequences, which takes 0.7
// of the first (0.33 in fp32, where it leaves out most of the products); it pays
// where the runs leave SMs idle. Time is counted in chunks of 64 tokens: that of
// the blocks, each as long as a segment and its start and end, and of the scan.
// (At 32 heads of 65,536 tokens, d = 128: 1,394 us in one piece, 602 in 4, 571 in
// the 9 it takes, 590 in 19; gradients of 4 x 8 heads of 4,096 tokens, d = 64: 67
// us in the one piece it takes, 91 in 4; fp32, 40 heads of 1,021 tokens, d = 64:
// 178 in one, 85 in 6, 79 in the 8 it takes; their gradients 180 in the one piece
// it takes, 198 in 8. At most 64 segments: their states are the call's scratch, and
// the scan goes over them in turn; more were not measured.)
double plan(long long heads, int roles, int state_roles, int T, int d, vla_dtype dt, Cut* cut) {
    const int chunks = (T + 63) / 64;
    const bool bf16 = dt == VLA_BF16;
    const double ends = ends_of(dt), second = bf16 ? 0.7 : 0.33;
    double best = 0;
    int best_len = chunks;
    const int shortest = bf16 ? 4 : 1;  // chunks of a segment
    for (int n = 1; n <= 64 && n * shortest <= std::max(shortest, chunks); ++n) {
        const int len = (chunks + n - 1) / n, segs = (chunks + len - 1) / len;
        double t = waves(heads * roles * segs, d, dt) * (len + ends);
        if (segs > 1)
            t += second * waves(heads * state_roles * segs, d, dt) * (len + ends) +
                 (bf16 ? 5 + 0.1 * segs : 0.5 + 0.01 * segs);
        if (n == 1 || t < best) best = t, best_len = len;
    }
    cut->seg_len = std::max(1, best_len) * 64;
    cut->nseg = std::max(1, (chunks + best_len - 1) / std::max(1, best_len));
    return best;
}

// The launches of a call: all heads alike, or, where that is shorter, as many as
// fill whole waves in one piece and the rest cut into segments after them.
// (Gradients of 2 x 32 heads of 8,191 tokens, d = 128, 192 blocks on 152 SMs.)
int plan_call(int B, int H, int roles, int state_roles, int T, int d, vla_dtype dt, Cut (&cut)[2]) {
    const long long BH = (long long)B * H, wave = sm_count() / roles;
    cut[0] = Cut{0, (int)BH, 1, 0};
    const double all = plan(BH, roles, state_roles, T, d, dt, &cut[0]);
    const long long whole = wave > 0 ? BH / wave * wave : 0;
    if (whole == 0 || whole == BH) return 1;
    const int chunks = (T + 63) / 64;
    Cut rest{(int)whole, (int)(BH - whole), 1, 0};
    const double t = waves(whole / wave * sm_count(), d, dt) * (chunks + ends_of(dt)) +
                     plan(BH - whole, roles, state_roles, T, d, dt, &rest) + 2;
    if (rest.nseg == 1 || t >= all) return 1;
    cut[0] = Cut{0, (int)whole, 1, std::max(1, chunks) * 64};
    cut[1] = rest;
    return 2;
}

// A call's launches: with segments, their own states, the scan over them, and
// the outputs; else the outputs alone.
struct Call {
    DecayArgs main, states;  // states.role: the state roles
    int roles, state_roles;
    ScanArgs scan;
    DecayMaps maps;
    Cut cut[2];
    int cuts;
};

template <int D, bool TC, typename T>
vla_status launch(Call& c, cudaStream_t s) {
    for (int i = 0; i < c.cuts; ++i) {
        const Cut& cut = c.cut[i];
        for (DecayArgs* p : {&c.main, &c.states})
            p->bh0 = cut.bh0, p->bhs = cut.bhs, p->nseg = cut.nseg, p->seg_len = cut.seg_len;
        const long long grid = (long long)cut.bhs * cut.nseg * c.roles;
        const long long scan_blocks = (long long)cut.bhs * (D * D / 4 / SCAN_THREADS);
        if (grid > 2147483647LL || scan_blocks > 2147483647LL) return VLA_ERR_INVALID_ARG;
        const unsigned blocks = (unsigned)(cut.bhs * cut.nseg);
        auto scan = [&] {
            vla_decay_scan_kernel<D><<<dim3((unsigned)scan_blocks, c.state_roles), SCAN_THREADS, 0, s>>>(c.main, c.scan);
        };
        if constexpr (TC) {
            using L = TcLay<D>;
            constexpr auto main = vla_decay_tc_kernel<D, false>, own = vla_decay_tc_kernel<D, true>;
            if (!allow_smem<main>(L::SMEM) || !allow_smem<own>(L::SMEM)) return VLA_ERR_CUDA;
            if (cut.nseg > 1) {
                own<<<blocks * c.state_roles, L::THREADS, L::SMEM, s>>>(c.states, c.maps, c.state_roles);
                scan();
            }
            main<<<blocks * c.roles, L::THREADS, L::SMEM, s>>>(c.main, c.maps, c.roles);
        } else {
            using L = FmaLay<D, T>;
            constexpr auto main = vla_decay_fma_kernel<D, T, false>;
            if (!allow_smem<main>(L::SMEM)) return VLA_ERR_CUDA;
            if constexpr (sizeof(T) == 4) {  // the few tokens of a bf16 call are one segment
                constexpr auto own = vla_decay_fma_kernel<D, T, true>;
                if (!allow_smem<own>(L::SMEM)) return VLA_ERR_CUDA;
                if (cut.nseg > 1) {
                    own<<<dim3(blocks, c.state_roles), L::THREADS, L::SMEM, s>>>(c.states);
                    scan();
                }
            }
            main<<<dim3(blocks, c.roles), L::THREADS, L::SMEM, s>>>(c.main);
        }
    }
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

template <bool TC, typename T>
vla_status launch_d(Call& c, int d, cudaStream_t s) {
    switch (d) {
        case 32: return launch<32, TC, T>(c, s);
        case 64: return launch<64, TC, T>(c, s);
        case 96: return launch<96, TC, T>(c, s);
        default: return launch<128, TC, T>(c, s);
    }
}

bool on_tensor_cores(vla_dtype dt, int T) { return dt == VLA_BF16 && T > FMA_T; }

vla_status launch_call(Call& c, int d, vla_dtype dt, cudaStream_t s) {
    if (on_tensor_cores(dt, c.main.T)) return launch_d<true, __nv_bfloat16>(c, d, s);
    return dt == VLA_F32 ? launch_d<false, float>(c, d, s) : launch_d<false, __nv_bfloat16>(c, d, s);
}

// scratch of the larger of the two types' cuts, so that it need not be told the type
size_t scratch_bytes_of(int B, int H, int T, int d, bool backward) {
    if (!good_sizes(B, H, T) || !good_d(d) || B == 0 || H == 0 || T == 0) return 0;
    size_t most = 0;
    for (vla_dtype dt : {VLA_F32, VLA_BF16}) {
        Cut cut[2];
        const int n = plan_call(B, H, backward ? 3 : 1, backward ? 2 : 1, T, d, dt, cut);
        const Cut& last = cut[n - 1];
        if (last.nseg > 1)
            most = std::max(most, (size_t)last.bhs * last.nseg * (backward ? 2 : 1) * d * d * sizeof(float));
    }
    return most;
}

vla_status copy_state(float* dst, const float* src, size_t n, cudaStream_t s) {
    if (!dst || dst == src || n == 0) return VLA_OK;
    const cudaError_t e = src ? cudaMemcpyAsync(dst, src, n * sizeof(float), cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(dst, 0, n * sizeof(float), s);
    return e == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

}  // namespace
}  // namespace vla_layer

extern "C" {

size_t vla_decay_scratch_bytes(int B, int H, int T, int d, int backward) {
    return vla_layer::scratch_bytes_of(B, H, T, d, backward != 0);
}

vla_status vla_decay_forward_ex(const vla_seq* q, const vla_seq* k, const vla_seq* v, vla_dtype dtype, int B, int H,
                                int T, int d, const float* log_decay, float scale, const int* lengths,
                                const float* S0, const vla_seq_out* o, float* S_out, void* scratch,
                                size_t scratch_bytes, void* status, void* stream, const vla_options* opts) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_dtype(dtype) || !std::isfinite(scale)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if (B == 0 || H == 0) return VLA_OK;
    if (!log_decay || !S_out || !aligned(log_decay, 4) || !aligned(lengths, 4) || !aligned(S0, 16) ||
        !aligned(S_out, 16) || !aligned(status, 16))
        return VLA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long states = (long long)B * H * d * d;
    const Region S_in = region(S0, states, 32), S_end = region(S_out, states, 32);
    if (!apart({S_end}, {S_in}, 1)) return VLA_ERR_INVALID_ARG;
    if (T == 0) return copy_state(S_out, S0, (size_t)B * H * d * d, s);
    const int es = dtype == VLA_BF16 ? 2 : 4;
    if (!good_seq(q, B, H, T, es) || !good_seq(k, B, H, T, es) || !good_seq(v, B, H, T, es) ||
        !good_seq(o, B, H, T, es))
        return VLA_ERR_INVALID_ARG;
    const size_t need = scratch_bytes_of(B, H, T, d, false);
    if (need && (!scratch || !aligned(scratch, 256) || scratch_bytes < need)) return VLA_ERR_INVALID_ARG;
    if (!apart({S_end, region(o, B, H, T, d, es), region(scratch, need, 8)},
               {S_in, region(q, B, H, T, d, es), region(k, B, H, T, d, es), region(v, B, H, T, d, es),
                region(log_decay, H, 32), region(lengths, B, 32)}, 1))
        return VLA_ERR_INVALID_ARG;
    Call c{};
    DecayArgs& p = c.main;
    p.B = B, p.H = H, p.T = T;
    p.log_decay = log_decay;
    p.lengths = lengths;
    p.status = static_cast<vla::DeviceStatus*>(status);
    take_options(p, opts);
    c.cuts = plan_call(B, H, 1, 1, T, d, dtype, c.cut);
    p.seg = static_cast<float*>(scratch);
    p.role[0] = Role{to_seq(q, B, H, T), to_seq(k, B, H, T), to_seq(v, B, H, T), to_seq(o, B, H, T),
                     S0, S_out, 0, 0, scale, scale, 1.f, 0, 1, 2};
    c.states = p;
    c.roles = c.state_roles = 1;
    c.scan.role[0] = ScanRole{S0, S_out, 0, 0};
    if (on_tensor_cores(dtype, T) &&
        (!make_map(&c.maps.m[0], q, B, H, T, d) || !make_map(&c.maps.m[1], k, B, H, T, d) ||
         !make_map(&c.maps.m[2], v, B, H, T, d) || !make_map(&c.maps.out[0], o, B, H, T, d)))
        return VLA_ERR_CUDA;
    return launch_call(c, d, dtype, s);
}

vla_status vla_decay_backward_ex(const vla_seq* q, const vla_seq* k, const vla_seq* v, const vla_seq* dO,
                                 vla_dtype dtype, int B, int H, int T, int d, const float* log_decay, float scale,
                                 const int* lengths, const float* S0, const float* dS_T, const vla_seq_out* dq,
                                 const vla_seq_out* dk, const vla_seq_out* dv, float* dS0, void* scratch,
                                 size_t scratch_bytes, void* status, void* stream, const vla_options* opts) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_dtype(dtype) || !std::isfinite(scale)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if (B == 0 || H == 0) return VLA_OK;
    if (!log_decay || !aligned(log_decay, 4) || !aligned(lengths, 4) || !aligned(S0, 16) || !aligned(dS_T, 16) ||
        !aligned(dS0, 16) || !aligned(status, 16))
        return VLA_ERR_INVALID_ARG;
    // the blocks of dk read dS_T and those of dq S0, when those of dv write dS0
    const long long states = (long long)B * H * d * d;
    const Region S_in = region(S0, states, 32), G_in = region(dS_T, states, 32), G_end = region(dS0, states, 32);
    if (!apart({G_end}, {S_in, G_in})) return VLA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return copy_state(dS0, dS_T, (size_t)B * H * d * d, s);
    const int es = dtype == VLA_BF16 ? 2 : 4;
    if (!good_seq(q, B, H, T, es) || !good_seq(k, B, H, T, es) || !good_seq(v, B, H, T, es) ||
        !good_seq(dO, B, H, T, es) || !good_seq(dq, B, H, T, es) || !good_seq(dk, B, H, T, es) ||
        !good_seq(dv, B, H, T, es))
        return VLA_ERR_INVALID_ARG;
    const size_t need = scratch_bytes_of(B, H, T, d, true);
    if (need && (!scratch || !aligned(scratch, 256) || scratch_bytes < need)) return VLA_ERR_INVALID_ARG;
    if (!apart({region(dq, B, H, T, d, es), region(dk, B, H, T, d, es), region(dv, B, H, T, d, es), G_end,
                region(scratch, need, 8)},
               {region(q, B, H, T, d, es), region(k, B, H, T, d, es), region(v, B, H, T, d, es),
                region(dO, B, H, T, d, es), S_in, G_in, region(log_decay, H, 32), region(lengths, B, 32)}))
        return VLA_ERR_INVALID_ARG;
    const Seq Q = to_seq(q, B, H, T), K = to_seq(k, B, H, T), V = to_seq(v, B, H, T), G = to_seq(dO, B, H, T);
    Call c{};
    DecayArgs& p = c.main;
    p.B = B, p.H = H, p.T = T;
    p.log_decay = log_decay;
    p.lengths = lengths;
    p.status = static_cast<vla::DeviceStatus*>(status);
    take_options(p, opts);
    c.cuts = plan_call(B, H, 3, 2, T, d, dtype, c.cut);
    p.seg = static_cast<float*>(scratch);
    p.role[0] = Role{G, V, K, to_seq(dq, B, H, T), S0, nullptr, 1, 0, scale, scale, 1.f, 3, 2, 1};
    p.role[1] = Role{V, G, Q, to_seq(dk, B, H, T), dS_T, nullptr, 1, 1, scale, 1.f, scale, 2, 3, 0};
    p.role[2] = Role{K, Q, G, to_seq(dv, B, H, T), dS_T, dS0, 0, 1, scale, 1.f, scale, 1, 0, 3};
    // the segments' own states: those of dq's role and of dv's, which is dk's transposed
    c.states = p;
    c.states.role[1] = p.role[2];
    p.seg_role[0] = 0, p.seg_role[1] = 1, p.seg_role[2] = 1;
    p.seg_t[1] = 1;
    c.roles = 3;
    c.state_roles = 2;
    c.scan.role[0] = ScanRole{S0, nullptr, 1, 0};
    c.scan.role[1] = ScanRole{dS_T, dS0, 0, 1};
    if (on_tensor_cores(dtype, T) &&
        (!make_map(&c.maps.m[0], q, B, H, T, d) || !make_map(&c.maps.m[1], k, B, H, T, d) ||
         !make_map(&c.maps.m[2], v, B, H, T, d) || !make_map(&c.maps.m[3], dO, B, H, T, d) ||
         !make_map(&c.maps.out[0], dq, B, H, T, d) || !make_map(&c.maps.out[1], dk, B, H, T, d) ||
         !make_map(&c.maps.out[2], dv, B, H, T, d)))
        return VLA_ERR_CUDA;
    return launch_call(c, d, dtype, s);
}

vla_status vla_decay_forward(const vla_seq* q, const vla_seq* k, const vla_seq* v, vla_dtype dtype, int B, int H,
                             int T, int d, const float* log_decay, float scale, const int* lengths, const float* S0,
                             const vla_seq_out* o, float* S_out, void* scratch, size_t scratch_bytes, void* status,
                             void* stream) {
    return vla_decay_forward_ex(q, k, v, dtype, B, H, T, d, log_decay, scale, lengths, S0, o, S_out, scratch,
                                scratch_bytes, status, stream, nullptr);
}

vla_status vla_decay_backward(const vla_seq* q, const vla_seq* k, const vla_seq* v, const vla_seq* dO,
                              vla_dtype dtype, int B, int H, int T, int d, const float* log_decay, float scale,
                              const int* lengths, const float* S0, const float* dS_T, const vla_seq_out* dq,
                              const vla_seq_out* dk, const vla_seq_out* dv, float* dS0, void* scratch,
                              size_t scratch_bytes, void* status, void* stream) {
    return vla_decay_backward_ex(q, k, v, dO, dtype, B, H, T, d, log_decay, scale, lengths, S0, dS_T, dq, dk, dv, dS0,
                                 scratch, scratch_bytes, status, stream, nullptr);
}

vla_status vla_decay_step(const void* q, const void* k, const void* v, vla_dtype dtype, int B, int H, int d,
                          const float* log_decay, float scale, float* states, int N, const int* slots, void* o,
                          void* status, void* stream) {
    using namespace vla_layer;
    if (!good_sizes(B, H, 1) || N < 0 || !good_dtype(dtype) || !std::isfinite(scale)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if (!slots && B > N) return VLA_ERR_INVALID_ARG;
    if (B == 0 || H == 0) return VLA_OK;
    if (!q || !k || !v || !o || !log_decay || (!states && N > 0) || !aligned(q, 16) || !aligned(k, 16) ||
        !aligned(v, 16) || !aligned(o, 16) || !aligned(log_decay, 4) || !aligned(states, 16) || !aligned(slots, 4) ||
        !aligned(status, 16))
        return VLA_ERR_INVALID_ARG;
    const long long grid = (long long)B * H * (d / STEP_ROWS);
    if (grid > 2147483647LL) return VLA_ERR_INVALID_ARG;
    // each block reads all of q and k of its head, o is written by several
    const long long rows = (long long)B * H * d;
    const int bits = dtype == VLA_BF16 ? 16 : 32;
    if (!apart({region(o, rows, bits), region(states, (__int128)N * H * d * d, 32)},
               {region(q, rows, bits), region(k, rows, bits), region(v, rows, bits), region(log_decay, H, 32), region(slots, B, 32)}))
        return VLA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto* ds = static_cast<vla::DeviceStatus*>(status);
    auto go = [&](auto tag, auto dim) {
        using T = decltype(tag);
        vla_decay_step_kernel<decltype(dim)::value, T><<<(unsigned)grid, STEP_THREADS, 0, s>>>(
            static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), H, log_decay, scale, states,
            N, slots, static_cast<T*>(o), ds);
    };
    auto pick = [&](auto tag) {
        switch (d) {
            case 32: go(tag, std::integral_constant<int, 32>{}); break;
            case 64: go(tag, std::integral_constant<int, 64>{}); break;
            case 96: go(tag, std::integral_constant<int, 96>{}); break;
            default: go(tag, std::integral_constant<int, 128>{}); break;
        }
    };
    if (dtype == VLA_BF16)
        pick(__nv_bfloat16{});
    else
        pick(float{});
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

}  // extern "C"
