// vla_qk.cu -- norm and position rotation of queries and keys, and their
// gradients (include/vla_layer.h).
//
// With r = 1 / sqrt(c sum x^2 + eps), n = x r, z = n w and a token's angles a_i,
//   y_i = z_i cos a_i - z_(i+m) sin a_i,  y_(i+m) = z_(i+m) cos a_i + z_i sin a_i  for i < m = rot / 2, y = z behind;
// against it, with dz the gradient turned back and p = dz w:
//   dx = r (p - n c sum(p n)),  dw = sum over the rows of dz n.
//
// Both passes move each value once and are bound by memory. A block takes a tile of
// tokens of several heads, q and k, and forms the tile's cosines and sines once: an
// angle is a 64-bit fraction of a turn, the position times the frequency's fraction in
// whole numbers, so that a far position loses nothing and no product in 64-bit floating
// point is left but one a frequency and block. A warp takes a head's q or k rows, its
// weight in registers; a lane holds eight values of a row and the eight they are turned
// with, in fp32, and has the loads of several rows under way. (q and k of 32 heads of
// 32,768 tokens, d = 128, bf16: see the table of measured forms at launch_forward().)
#include <cmath>
#include <type_traits>

#include "vla_layer.cuh"

namespace vla_layer {
namespace {

constexpr int QK_THREADS = 256, QK_WARPS = QK_THREADS / 32;

struct QkRows {
    Seq x, dy, out;
    const float* w;
    float* rstd;
};
struct QkArgs {
    QkRows r[2];            // q and k
    const double* freqs;    // [rot / 2], radians a position
    const int* pos;         // [B][T], or null for t
    long long pos_sb;
    int H, T, rot;
    int heads, groups;      // heads of a block, and blocks that share a tile
    int tiles, spans;       // tiles of a block, and blocks along the sequence
    int shared;             // one weight for all heads
    float c, eps;
    float* partial;         // backward: [B][spans][2][H][d] sums dz n
};

template <int D>
struct QkLay {
    static constexpr int L = D / 16;          // lanes of a row
    static constexpr int ROWS = 32 / L;       // rows of a warp at a time (d = 96: five, of 30 lanes)
    static constexpr int DEEP = 4, TT = ROWS * DEEP;  // tokens of a tile
};

// The sum over a row's lanes, the same in each.
template <int L>
__device__ __forceinline__ float row_total(float v, int lane) {
    if constexpr (L == 6) {  // six lanes: three pairs, then the pairs in order
        const int base = lane / 6 * 6, i = lane - base;
        v += __shfl_sync(0xffffffffu, v, base + (i < 3 ? i + 3 : i - 3));
        const float a = __shfl_sync(0xffffffffu, v, base), b = __shfl_sync(0xffffffffu, v, base + 1),
                    c = __shfl_sync(0xffffffffu, v, base + 2);
        return a + b + c;
    } else {
#pragma unroll
        for (int m = 1; m < L; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        return v;
    }
}

// cos and sin of a fraction of a turn in 2^-64 of it: the nearest quarter aside, an eighth of a turn at most is left
__device__ __forceinline__ float2 turn_of(unsigned long long u) {
    const uint32_t top = (uint32_t)(u >> 32), quarter = (top + 0x20000000u) >> 30;
    float s, c;
    sincospif((float)(int)(top - (quarter << 30)) * 0x1p-31f, &s, &c);
    const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -x : x, quarter & 2 ? -y : y);
}

// The tile's (cos, sin): frequency 8 l + j of a token is at [token][j / 2][l], two frequencies to a float4, so that
// the lanes of a row read in order.
template <int D>
__device__ __forceinline__ void make_turns(const QkArgs& a, float2* turns, const unsigned long long* fraction, const bool* odd, int b,
                                           long long t0) {
    using Q = QkLay<D>;
    const int m = a.rot / 2, per = a.rot / 16;
    for (int i = threadIdx.x; i < Q::TT * m; i += QK_THREADS) {
        const int tok = i / m, f = i - tok * m;
        const long long t = t0 + tok;
        if (t >= a.T) break;
        const int pos = a.pos ? a.pos[b * a.pos_sb + t] : (int)t;
        const float nan = __int_as_float(0x7FC00000);
        turns[((tok * 4 + (f & 7) / 2) * per + f / 8) * 2 + (f & 1)] =
            odd[f] ? make_float2(nan, nan) : turn_of((unsigned long long)(long long)pos * fraction[f]);
    }
}

// The frequencies as fractions of a turn, and which are not finite (NaN at every position)
__device__ __forceinline__ void make_fractions(const QkArgs& a, unsigned long long* fraction, bool* odd) {
    for (int f = threadIdx.x; f < a.rot / 2; f += QK_THREADS) {
        const double turns = a.freqs[f] * 0.15915494309189533577;
        const double part = turns - floor(turns);
        odd[f] = !isfinite(turns);
        // in two halves, as a product of 2^64 and a part near 1 would not fit
        const double high = floor(part * 4294967296.0);
        fraction[f] = ((unsigned long long)(uint32_t)high << 32) + (unsigned long long)((part * 4294967296.0 - high) * 4294967296.0);
    }
    __syncthreads();
}

// a and b, a lane's values and those they are turned with, by +- the token's angles
template <int SIGN>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float2* turns, int tok, int per, int l) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 w = *reinterpret_cast<const float4*>(turns + ((tok * 4 + i) * per + l) * 2);
        const float c[2] = {w.x, w.z}, s[2] = {SIGN * w.y, SIGN * w.w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float x = a[2 * i + e], y = b[2 * i + e];
            a[2 * i + e] = fmaf(x, c[e], -y * s[e]);
            b[2 * i + e] = fmaf(y, c[e], x * s[e]);
        }
    }
}

template <int D, typename T, bool BACKWARD>
__global__ void __launch_bounds__(QK_THREADS) vla_qk_kernel(const __grid_constant__ QkArgs a) {
    using Q = QkLay<D>;
    constexpr int L = Q::L, AT_ONCE = sizeof(T) == 4 || BACKWARD ? 2 : 4;  // rows of a lane under way
    __shared__ __align__(16) float2 turns[Q::TT * D / 2];
    __shared__ unsigned long long fraction[D / 2];
    __shared__ bool odd[D / 2];
    const int span = blockIdx.x % a.spans, bg = blockIdx.x / a.spans, h0 = bg % a.groups * a.heads, b = bg / a.groups;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, l = lane % L, row = lane / L;
    const int P = a.rot ? a.rot / 16 : L;  // lanes whose two groups are turned with each other
    const bool turned = a.rot && l < P, on = row < Q::ROWS;
    const int c0 = (l < P ? l : P + l) * 8, c1 = (l < P ? l + P : L + l) * 8;
    if (a.rot) make_fractions(a, fraction, odd);
    float dw[2][8] = {};
    for (int k = 0; k < a.tiles; ++k) {
        const long long t0 = ((long long)span * a.tiles + k) * Q::TT;
        if (t0 >= a.T) break;
        if (a.rot) {
            if (k) __syncthreads();
            make_turns<D>(a, turns, fraction, odd, b, t0);
            __syncthreads();
        }
        for (int unit = warp; unit < 2 * a.heads; unit += QK_WARPS) {
            const int h = h0 + unit / 2;
            if (h >= a.H) break;
            const QkRows& r = a.r[unit & 1];
            float w[2][8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[0][i] = w[1][i] = 1.f;
            if (r.w) {
                const float* p = r.w + (a.shared ? 0 : (size_t)h * D);
                load8(p + c0, w[0]);
                load8(p + c1, w[1]);
            }
            const size_t stats = ((size_t)b * a.H + h) * a.T;
#pragma unroll 1
            for (int u = 0; u < Q::DEEP; u += AT_ONCE) {
                decltype(raw8((const T*)nullptr)) raw[AT_ONCE][2], rg[AT_ONCE][2];
                float rs[AT_ONCE];
#pragma unroll
                for (int e = 0; e < AT_ONCE; ++e) {
                    const long long t = t0 + (u + e) * Q::ROWS + row;
                    raw[e][0] = raw[e][1] = rg[e][0] = rg[e][1] = {};
                    rs[e] = 0.f;
                    if (!on || t >= a.T) continue;
                    const T* x = row_of<T>(r.x, b, h, t);
                    raw[e][0] = raw8(x + c0), raw[e][1] = raw8(x + c1);
                    if constexpr (BACKWARD) {
                        const T* g = row_of<T>(r.dy, b, h, t);
                        rg[e][0] = raw8(g + c0), rg[e][1] = raw8(g + c1);
                        rs[e] = r.rstd[stats + t];
                    }
                }
#pragma unroll
                for (int e = 0; e < AT_ONCE; ++e) {
                    const int tok = (u + e) * Q::ROWS + row;
                    const long long t = t0 + tok;
                    const bool live = on && t < a.T;
                    float x[2][8], sum = 0.f;
                    open8(raw[e][0], x[0]);
                    open8(raw[e][1], x[1]);
                    if constexpr (!BACKWARD) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) sum = fmaf(x[0][i], x[0][i], fmaf(x[1][i], x[1][i], sum));
                        const float rstd = rsqrtf(fmaf(a.c, row_total<L>(sum, lane), a.eps));
                        if (!live) continue;
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[0][i] *= rstd * w[0][i], x[1][i] *= rstd * w[1][i];
                        if (turned) turn<1>(x[0], x[1], turns, tok, P, l);
                        T* y = row_of<T>(r.out, b, h, t);
                        store8(y + c0, x[0]);
                        store8(y + c1, x[1]);
                        if (l == 0 && r.rstd) r.rstd[stats + t] = rstd;
                    } else {
                        float g[2][8];
                        open8(rg[e][0], g[0]);
                        open8(rg[e][1], g[1]);
                        if (turned && live) turn<-1>(g[0], g[1], turns, tok, P, l);
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                x[q][i] *= rs[e];
                                dw[q][i] = fmaf(g[q][i], x[q][i], dw[q][i]);
                                g[q][i] *= w[q][i];
                                sum = fmaf(g[q][i], x[q][i], sum);
                            }
                        sum = a.c * row_total<L>(sum, lane);
                        if (!live) continue;
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int i = 0; i < 8; ++i) g[q][i] = fmaf(-sum, x[q][i], g[q][i]) * rs[e];
                        T* y = row_of<T>(r.out, b, h, t);
                        store8(y + c0, g[0]);
                        store8(y + c1, g[1]);
                    }
                }
            }
        }
    }
    if constexpr (BACKWARD) {
        // one unit a warp: its rows' sums, in the order of the lanes
        const int h = h0 + warp / 2;
        if (!a.partial || h >= a.H || warp >= 2 * a.heads) return;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float s = on ? dw[q][i] : 0.f;
                if constexpr (L == 6) {
                    float all = 0.f;
#pragma unroll
                    for (int k = 0; k < Q::ROWS; ++k) all += __shfl_sync(0xffffffffu, s, k * L + l);
                    s = all;
                } else {
#pragma unroll
                    for (int m = L; m < 32; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                }
                dw[q][i] = s;
            }
        if (row == 0) {
            float* out = a.partial + ((((size_t)b * a.spans + span) * 2 + (warp & 1)) * a.H + h) * D;
            store8(out + c0, dw[0]);
            store8(out + c1, dw[1]);
        }
    }
}

// dw of q and k from the blocks' sums [n][2][H][d]: a block per 32 columns of (q or k, head), 32 threads a column, each
// over every 32nd of the sums, and the threads' sums in order.
constexpr int QK_SUMS = 1024;
__global__ void __launch_bounds__(QK_SUMS) vla_qk_sums_kernel(const float* __restrict__ partial, int n, int H, int d, int shared,
                                                              float* dwq, float* dwk) {
    __shared__ float sums[32][33];
    const int col = threadIdx.x % 32, k = threadIdx.x / 32, which = blockIdx.z;
    const int i = blockIdx.y * 32 + col;
    const long long all = (long long)n * (shared ? H : 1);
    float s = 0.f;
#pragma unroll 8
    for (long long m = k; m < all; m += 32) {
        const long long blk = shared ? m / H : m, h = shared ? m % H : blockIdx.x;
        s += partial[((blk * 2 + which) * H + h) * d + i];
    }
    sums[k][col] = s;
    __syncthreads();
    if (k == 0) {
#pragma unroll
        for (int j = 1; j < 32; ++j) s += sums[j][col];
        (which ? dwk : dwq)[(size_t)blockIdx.x * d + i] = s;
    }
}

int tile_of(int d) { return d == 128 ? QkLay<128>::TT : d == 96 ? QkLay<96>::TT : d == 64 ? QkLay<64>::TT : QkLay<32>::TT; }

// A block's heads and tiles. Forward: a tile of as many heads as leave every SM four blocks, for which its angles
// are formed once. Backward: a head of q and of k a warp, and tiles enough that the sums over the rows are few.
struct QkPlan {
    int heads, groups, tiles, spans;
    long long grid;
};
QkPlan qk_plan(bool backward, int B, int H, int T, int d) {
    const long long tiles = ((long long)T + tile_of(d) - 1) / tile_of(d), enough = 4LL * sm_count();
    QkPlan p;
    p.heads = QK_WARPS / 2;
    p.tiles = 1;
    if (backward) {
        const long long groups = (H + p.heads - 1) / p.heads;
        while (p.tiles < 16 && (long long)B * groups * ((tiles + 2 * p.tiles - 1) / (2 * p.tiles)) >= enough) p.tiles *= 2;
    } else {
        while (p.heads < H && (long long)B * tiles * ((H + 2 * p.heads - 1) / (2 * p.heads)) >= enough) p.heads *= 2;
    }
    p.groups = (H + p.heads - 1) / p.heads;
    p.spans = (int)((tiles + p.tiles - 1) / p.tiles);
    p.grid = (long long)B * p.groups * p.spans;
    return p;
}

template <bool BACKWARD>
vla_status qk_launch(QkArgs& a, const QkPlan& p, vla_dtype dt, int d, cudaStream_t s) {
    if (p.grid > 2147483647LL) return VLA_ERR_INVALID_ARG;
    a.heads = p.heads, a.groups = p.groups, a.tiles = p.tiles, a.spans = p.spans;
    auto go = [&](auto tag) {
        using T = decltype(tag);
        switch (d) {
            case 32: vla_qk_kernel<32, T, BACKWARD><<<(unsigned)p.grid, QK_THREADS, 0, s>>>(a); break;
            case 64: vla_qk_kernel<64, T, BACKWARD><<<(unsigned)p.grid, QK_THREADS, 0, s>>>(a); break;
            case 96: vla_qk_kernel<96, T, BACKWARD><<<(unsigned)p.grid, QK_THREADS, 0, s>>>(a); break;
            default: vla_qk_kernel<128, T, BACKWARD><<<(unsigned)p.grid, QK_THREADS, 0, s>>>(a); break;
        }
    };
    if (dt == VLA_BF16)
        go(__nv_bfloat16{});
    else
        go(float{});
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

bool good_rotation(const double* freqs, int rot, const int* positions, long long stride_b, int B) {
    if (rot == 0) return true;
    return freqs && aligned(freqs, 8) && aligned(positions, 4) && (!positions || B <= 1 || stride_b >= 0);
}
Region positions_region(const int* positions, long long stride_b, int B, int T) {
    const bool again = B <= 1 || stride_b == 0;
    return Region{reinterpret_cast<uintptr_t>(positions), 4LL * T, {again ? 0 : stride_b * 4, 0, 0}, {again ? 1 : B, 1, 1}};
}

}  // namespace
}  // namespace vla_layer

extern "C" {

vla_status vla_qk_norm(const vla_seq* q, const vla_seq* k, vla_dtype dtype, int B, int H, int T, int d,
                       const float* weight_q, const float* weight_k, int shared, int unit, float eps,
                       const double* freqs, int rot, const int* positions, long long positions_stride_b,
                       const vla_seq_out* yq, const vla_seq_out* yk, float* rstd_q, float* rstd_k, void* stream) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_dtype(dtype)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if (rot < 0 || rot > d || rot % 16 != 0 || !(eps >= 0.f) || eps > 3.4e38f) return VLA_ERR_INVALID_ARG;
    if (B == 0 || H == 0 || T == 0) return VLA_OK;
    const int es = dtype == VLA_BF16 ? 2 : 4;
    if (!good_seq(q, B, H, T, es) || !good_seq(k, B, H, T, es) || !good_seq(yq, B, H, T, es) || !good_seq(yk, B, H, T, es) ||
        !aligned(weight_q, 16) || !aligned(weight_k, 16) || !aligned(rstd_q, 4) || !aligned(rstd_k, 4) ||
        !good_rotation(freqs, rot, positions, positions_stride_b, B))
        return VLA_ERR_INVALID_ARG;
    const long long weights = (shared ? 1LL : (long long)H) * d, stats = (long long)B * H * T;
    const Region Q = region(q, B, H, T, d, es), K = region(k, B, H, T, d, es), YQ = region(yq, B, H, T, d, es),
                 YK = region(yk, B, H, T, d, es), RQ = region(rstd_q, stats, 32), RK = region(rstd_k, stats, 32);
    if (!apart({YQ, YK, RQ, RK},
               {region(weight_q, weights, 32), region(weight_k, weights, 32), region(rot ? freqs : nullptr, rot / 2, 64),
                positions_region(rot ? positions : nullptr, positions_stride_b, B, T)}) ||
        !apart({RQ, RK}, {Q, K}) || !apart({YQ}, {Q, K}, 1) || !apart({YK}, {K, Q}, 1))
        return VLA_ERR_INVALID_ARG;
    QkArgs a{};
    a.r[0] = QkRows{to_seq(q, B, H, T), Seq{}, to_seq(yq, B, H, T), weight_q, rstd_q};
    a.r[1] = QkRows{to_seq(k, B, H, T), Seq{}, to_seq(yk, B, H, T), weight_k, rstd_k};
    a.freqs = freqs, a.rot = rot;
    a.pos = positions, a.pos_sb = B > 1 ? positions_stride_b : 0;
    a.H = H, a.T = T, a.shared = shared != 0;
    a.c = unit ? 1.f : 1.f / (float)d, a.eps = eps;
    return qk_launch<false>(a, qk_plan(false, B, H, T, d), dtype, d, static_cast<cudaStream_t>(stream));
}

size_t vla_qk_norm_scratch_bytes(int B, int H, int T, int d) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_d(d) || B == 0 || H == 0 || T == 0) return 0;
    return (size_t)B * qk_plan(true, B, H, T, d).spans * 2 * H * d * sizeof(float);
}

vla_status vla_qk_norm_backward(const vla_seq* dyq, const vla_seq* dyk, const vla_seq* q, const vla_seq* k,
                                vla_dtype dtype, int B, int H, int T, int d, const float* weight_q,
                                const float* weight_k, int shared, int unit, const double* freqs, int rot,
                                const int* positions, long long positions_stride_b, const float* rstd_q,
                                const float* rstd_k, const vla_seq_out* dq, const vla_seq_out* dk, float* dweight_q,
                                float* dweight_k, void* scratch, size_t scratch_bytes, void* stream) {
    using namespace vla_layer;
    if (!good_sizes(B, H, T) || !good_dtype(dtype)) return VLA_ERR_INVALID_ARG;
    if (!good_d(d)) return VLA_ERR_UNSUPPORTED;
    if (rot < 0 || rot > d || rot % 16 != 0 || (dweight_q == nullptr) != (dweight_k == nullptr) || !aligned(dweight_q, 4) ||
        !aligned(dweight_k, 4))
        return VLA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long weights = (shared ? 1LL : (long long)H) * d, stats = (long long)B * H * T;
    if (B == 0 || H == 0 || T == 0) {
        if (!dweight_q || weights == 0) return VLA_OK;
        const bool ok = cudaMemsetAsync(dweight_q, 0, weights * 4, s) == cudaSuccess && cudaMemsetAsync(dweight_k, 0, weights * 4, s) == cudaSuccess;
        return ok ? VLA_OK : VLA_ERR_CUDA;
    }
    const int es = dtype == VLA_BF16 ? 2 : 4;
    if (!good_seq(q, B, H, T, es) || !good_seq(k, B, H, T, es) || !good_seq(dyq, B, H, T, es) || !good_seq(dyk, B, H, T, es) ||
        !good_seq(dq, B, H, T, es) || !good_seq(dk, B, H, T, es) || !aligned(weight_q, 16) || !aligned(weight_k, 16) ||
        !rstd_q || !rstd_k || !aligned(rstd_q, 4) || !aligned(rstd_k, 4) ||
        !good_rotation(freqs, rot, positions, positions_stride_b, B))
        return VLA_ERR_INVALID_ARG;
    const size_t need = dweight_q ? vla_qk_norm_scratch_bytes(B, H, T, d) : 0;
    if (need && (!scratch || !aligned(scratch, 16) || scratch_bytes < need)) return VLA_ERR_INVALID_ARG;
    const Region Q = region(q, B, H, T, d, es), K = region(k, B, H, T, d, es), GQ = region(dyq, B, H, T, d, es),
                 GK = region(dyk, B, H, T, d, es), DQ = region(dq, B, H, T, d, es), DK = region(dk, B, H, T, d, es),
                 WQ = region(dweight_q, weights, 32), WK = region(dweight_k, weights, 32), X = region(need ? scratch : nullptr, need, 8);
    if (!apart({DQ, DK, WQ, WK, X},
               {region(weight_q, weights, 32), region(weight_k, weights, 32), region(rstd_q, stats, 32), region(rstd_k, stats, 32),
                region(rot ? freqs : nullptr, rot / 2, 64), positions_region(rot ? positions : nullptr, positions_stride_b, B, T)}) ||
        !apart({WQ, WK, X}, {Q, K, GQ, GK}) || !apart({DQ}, {Q, GQ, K, GK}, 2) || !apart({DK}, {K, GK, Q, GQ}, 2))
        return VLA_ERR_INVALID_ARG;
    QkArgs a{};
    a.r[0] = QkRows{to_seq(q, B, H, T), to_seq(dyq, B, H, T), to_seq(dq, B, H, T), weight_q, const_cast<float*>(rstd_q)};
    a.r[1] = QkRows{to_seq(k, B, H, T), to_seq(dyk, B, H, T), to_seq(dk, B, H, T), weight_k, const_cast<float*>(rstd_k)};
    a.freqs = freqs, a.rot = rot;
    a.pos = positions, a.pos_sb = B > 1 ? positions_stride_b : 0;
    a.H = H, a.T = T, a.shared = shared != 0;
    a.c = unit ? 1.f : 1.f / (float)d;
    a.partial = dweight_q ? static_cast<float*>(scratch) : nullptr;
    const QkPlan p = qk_plan(true, B, H, T, d);
    const vla_status st = qk_launch<true>(a, p, dtype, d, s);
    if (st != VLA_OK || !dweight_q) return st;
    vla_qk_sums_kernel<<<dim3((unsigned)(shared ? 1 : H), (unsigned)(d / 32), 2), QK_SUMS, 0, s>>>(a.partial, B * p.spans, H, d, a.shared,
                                                                                                  dweight_q, dweight_k);
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

}  // extern "C"
