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
// with, in fp32, and has the loads of several rows under way.
//
// Measured: q and k of 32 heads of 32,768 tokens, d = 128, bf16: forward 183 us (1.07 GB, 5.85 TB/s), 164 without the
// rotation; gradients 412 us (1.61 GB, 3.9 TB/s), which are short of registers for loads under way: two blocks of 128
// registers a thread on an SM. Loads through a ring of shared memory instead were slower (244 and 529 us), as was
// fetching a row's successors while it is worked on (469 us: it spills). fp32 operations in pairs took the forward
// pass from 214 to 183 us, the gradients from 468 to 432.
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

template <int D, bool BACKWARD>
struct QkLay {
    static constexpr int L = D / 16;          // lanes of a row
    static constexpr int ROWS = 32 / L;       // rows of a warp at a time (d = 96: five, of 30 lanes)
    // rows of a lane in a tile (q and k of 32 heads of 32,768 tokens, d = 128: forward 182 us for 4, 190 for 8, gradients
    // 432 and 408)
    static constexpr int DEEP = BACKWARD ? 8 : 4, TT = ROWS * DEEP;
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

// The tile's cosines and sines: frequencies 8 l + j and j + 1 of a token are at [token][j / 2][l], two cosines and two
// sines to a float4, so that the lanes of a row read in order.
template <typename Q>
__device__ __forceinline__ void make_turns(const QkArgs& a, float* turns, const unsigned long long* fraction, const bool* odd, int b,
                                           long long t0) {
    const int m = a.rot / 2, per = a.rot / 16;
    for (int i = threadIdx.x; i < Q::TT * m; i += QK_THREADS) {
        const int tok = i / m, f = i - tok * m;
        const long long t = t0 + tok;
        if (t >= a.T) break;
        const int pos = a.pos ? a.pos[b * a.pos_sb + t] : (int)t;
        const float nan = __int_as_float(0x7FC00000);
        const float2 w = odd[f] ? make_float2(nan, nan) : turn_of((unsigned long long)(long long)pos * fraction[f]);
        float* at = turns + ((tok * 4 + (f & 7) / 2) * per + f / 8) * 4 + (f & 1);
        at[0] = w.x, at[2] = w.y;
    }
}

// The frequencies as fractions of a turn, and which are not finite (NaN at every position)
__device__ __forceinline__ void make_fractions(const QkArgs& a, unsigned long long* fraction, bool* odd) {
    for (int f = threadIdx.x; f < a.rot / 2; f += QK_THREADS) {
        // of its size, as what is left of a small negative number beside the whole turn below it is rounded, to 1 even
        const double turns = fabs(a.freqs[f]) * 0.15915494309189533577;
        const double part = turns - floor(turns);
        odd[f] = !isfinite(turns);
        // in two halves, as a product of 2^64 and a part near 1 would not fit
        const double high = floor(part * 4294967296.0);
        const unsigned long long u = ((unsigned long long)(uint32_t)high << 32) + (unsigned long long)((part * 4294967296.0 - high) * 4294967296.0);
        fraction[f] = a.freqs[f] < 0 ? 0ull - u : u;
    }
    __syncthreads();
}

// Eight values as pairs: two fp32 operations an instruction, which is what the passes are short of beside memory.
__device__ __forceinline__ void open_pairs(const Raw8F& r, float2 (&x)[4]) {
    x[0] = make_float2(r.a.x, r.a.y), x[1] = make_float2(r.a.z, r.a.w), x[2] = make_float2(r.b.x, r.b.y), x[3] = make_float2(r.b.z, r.b.w);
}
__device__ __forceinline__ void open_pairs(const uint4& r, float2 (&x)[4]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void store_pairs(float* p, const float2 (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}
__device__ __forceinline__ void store_pairs(__nv_bfloat16* p, const float2 (&x)[4]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y), pack_bf16(x[3].x, x[3].y));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// a and b, a lane's values and those they are turned with, by +- the token's angles
template <int SIGN>
__device__ __forceinline__ void turn(float2 (&a)[4], float2 (&b)[4], const float* turns, int tok, int per, int l) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 w = *reinterpret_cast<const float4*>(turns + ((tok * 4 + i) * per + l) * 4);  // two cosines, two sines
        const float2 c = make_float2(w.x, w.y), s = make_float2(SIGN * w.z, SIGN * w.w), x = a[i], y = b[i];
        a[i] = __ffma2_rn(x, c, __fmul2_rn(y, make_float2(-s.x, -s.y)));
        b[i] = __ffma2_rn(y, c, __fmul2_rn(x, s));
    }
}

template <int D, typename T, bool BACKWARD>
__global__ void __launch_bounds__(QK_THREADS, sizeof(T) == 4 && !BACKWARD ? 3 : 2) vla_qk_kernel(const __grid_constant__ QkArgs a) {
    using Q = QkLay<D, BACKWARD>;
    // rows of a lane under way, as the registers of two blocks on an SM (three: fp32 forward) allow: d = 96, 8 x 16 heads of
    // 4,096, bf16: gradients 232 us for 1, 209 for 2 (which spill 12 to 28 bytes), more for 4, which spill more; fp32, d = 64, 4 x 16 heads: forward
    // 56.9 us for 1, 61.8 for 2
    constexpr int L = Q::L, AT_ONCE = sizeof(T) == 4 ? 1 : BACKWARD ? 2 : 4;
    __shared__ __align__(16) float turns[2][Q::TT * D];                    // of a tile and of the next one
    __shared__ unsigned long long fraction[D / 2];
    __shared__ bool odd[D / 2];
    const int span = blockIdx.x % a.spans, bg = blockIdx.x / a.spans, h0 = bg % a.groups * a.heads, b = bg / a.groups;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, l = lane % L, row = lane / L;
    const int P = a.rot ? a.rot / 16 : L;  // lanes whose two groups are turned with each other
    const bool turned = a.rot && l < P, on = row < Q::ROWS;
    const int c0 = (l < P ? l : P + l) * 8, c1 = (l < P ? l + P : L + l) * 8;
    const long long first = (long long)span * a.tiles * Q::TT;
    const int tiles = (int)min((long long)a.tiles, (a.T - first + Q::TT - 1) / Q::TT);
    if (a.rot) {
        make_fractions(a, fraction, odd);
        make_turns<Q>(a, turns[0], fraction, odd, b, first);
        __syncthreads();
    }
    float2 dw[2][4] = {};
#pragma unroll 1
    for (int k = 0; k < tiles; ++k) {
        const long long t0 = first + (long long)k * Q::TT;
        if (a.rot && k + 1 < tiles) make_turns<Q>(a, turns[(k + 1) & 1], fraction, odd, b, t0 + Q::TT);
        const float* turn_at = turns[k & 1];
        for (int unit = warp; unit < 2 * a.heads; unit += QK_WARPS) {
            const int h = h0 + unit / 2;
            if (h >= a.H) break;
            const QkRows& r = a.r[unit & 1];
            float2 w[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[0][i] = w[1][i] = both(1.f);
            if (r.w) {
                const float* p = r.w + (a.shared ? 0 : (size_t)h * D);
                open_pairs(raw8(p + c0), w[0]);
                open_pairs(raw8(p + c1), w[1]);
            }
            float* stats = r.rstd + ((size_t)b * a.H + h) * a.T;
            const T *from = row_of<T>(r.x, b, h, t0 + row), *grad = BACKWARD ? row_of<T>(r.dy, b, h, t0 + row) : nullptr;
            T* to = row_of<T>(r.out, b, h, t0 + row);
            const int left = (int)min((long long)Q::TT, a.T - t0) - row;  // of the tile, from this lane's first row
            decltype(raw8((const T*)nullptr)) raw[AT_ONCE][2], rg[AT_ONCE][2];
            float rs[AT_ONCE];
            auto load = [&](int e, int m) {  // a row to slot e
                raw[e][0] = raw[e][1] = rg[e][0] = rg[e][1] = {};
                rs[e] = 0.f;
                if (!on || m >= left) return;
                const T* x = from + m * r.x.st;
                raw[e][0] = raw8(x + c0), raw[e][1] = raw8(x + c1);
                if constexpr (BACKWARD) {
                    const T* g = grad + m * r.dy.st;
                    rg[e][0] = raw8(g + c0), rg[e][1] = raw8(g + c1);
                    rs[e] = stats[t0 + row + m];
                }
            };
#pragma unroll 1
            for (int u = 0; u < Q::DEEP; u += AT_ONCE) {
#pragma unroll
                for (int e = 0; e < AT_ONCE; ++e) load(e, (u + e) * Q::ROWS);
#pragma unroll
                for (int e = 0; e < AT_ONCE; ++e) {
                    const int m = (u + e) * Q::ROWS, tok = m + row;
                    const bool live = on && m < left;
                    float2 x[2][4], sum = both(0.f);
                    open_pairs(raw[e][0], x[0]);
                    open_pairs(raw[e][1], x[1]);
                    T* y = to + m * r.out.st;
                    if constexpr (!BACKWARD) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum = __ffma2_rn(x[0][i], x[0][i], __ffma2_rn(x[1][i], x[1][i], sum));
                        const float rstd = rsqrtf(fmaf(a.c, row_total<L>(sum.x + sum.y, lane), a.eps));
                        if (!live) continue;
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[q][i] = __fmul2_rn(x[q][i], __fmul2_rn(both(rstd), w[q][i]));
                        if (turned) turn<1>(x[0], x[1], turn_at, tok, P, l);
                        store_pairs(y + c0, x[0]);
                        store_pairs(y + c1, x[1]);
                        if (l == 0 && r.rstd) stats[t0 + tok] = rstd;
                    } else {
                        float2 g[2][4];
                        open_pairs(rg[e][0], g[0]);
                        open_pairs(rg[e][1], g[1]);
                        const float rstd = rs[e];
                        if (turned && live) turn<-1>(g[0], g[1], turn_at, tok, P, l);
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                x[q][i] = __fmul2_rn(x[q][i], both(rstd));
                                dw[q][i] = __ffma2_rn(g[q][i], x[q][i], dw[q][i]);
                                g[q][i] = __fmul2_rn(g[q][i], w[q][i]);
                                sum = __ffma2_rn(g[q][i], x[q][i], sum);
                            }
                        const float share = a.c * row_total<L>(sum.x + sum.y, lane);
                        if (!live) continue;
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i) g[q][i] = __fmul2_rn(__ffma2_rn(both(-share), x[q][i], g[q][i]), both(rstd));
                        store_pairs(y + c0, g[0]);
                        store_pairs(y + c1, g[1]);
                    }
                }
            }
        }
        if (a.rot) __syncthreads();  // the next tile's angles are there, and this one's are read
    }
    if constexpr (BACKWARD) {
        // one unit a warp: its rows' sums, in the order of the lanes
        const int h = h0 + warp / 2;
        if (!a.partial || h >= a.H || warp >= 2 * a.heads) return;
        auto over_rows = [&](float s) {
            if (!on) s = 0.f;
            if constexpr (L == 6) {
                float all = 0.f;
#pragma unroll
                for (int k = 0; k < Q::ROWS; ++k) all += __shfl_sync(0xffffffffu, s, k * L + l);
                return all;
            } else {
#pragma unroll
                for (int m = L; m < 32; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                return s;
            }
        };
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) dw[q][i] = make_float2(over_rows(dw[q][i].x), over_rows(dw[q][i].y));
        if (row == 0) {
            float* out = a.partial + ((((size_t)b * a.spans + span) * 2 + (warp & 1)) * a.H + h) * D;
            store_pairs(out + c0, dw[0]);
            store_pairs(out + c1, dw[1]);
        }
    }
}

// dw of q and k from the blocks' sums [n][2][H][d]: a block per eight columns (a sector of memory) of (q or k, head, or all
// heads), 128 threads a column, each over every 128th of the rows, eight loads under way, and the threads' sums in a
// fixed order. The loads' latency is all there is to it: with 32 columns a block and a load at a time it took 62 us of 2.5
// MB (8 x 16 heads of 4,096 tokens, d = 96, one weight).
constexpr int QK_SUMS = 1024, QK_COLS = 8, QK_SLICES = QK_SUMS / QK_COLS;
__global__ void __launch_bounds__(QK_SUMS) vla_qk_sums_kernel(const float* __restrict__ partial, int n, int H, int d, int shared,
                                                              float* dwq, float* dwk) {
    __shared__ float sums[QK_SUMS / 32][QK_COLS];
    const int col = threadIdx.x % QK_COLS, slice = threadIdx.x / QK_COLS, which = blockIdx.z;
    const int i = blockIdx.y * QK_COLS + col, heads = shared ? H : 1;
    const float* from = partial + ((size_t)which * H + blockIdx.x) * d + i;
    const unsigned rows = (unsigned)n * heads;  // of 256 bytes and more: below 2^32 in any memory
    float s = 0.f;
    for (unsigned j = slice; j < rows; j += 8 * QK_SLICES) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const unsigned row = j + u * QK_SLICES, m = row / (unsigned)heads;
            v[u] = row < rows ? from[((size_t)m * 2 * H + (row - m * heads)) * d] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) s += v[u];
    }
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (threadIdx.x % 32 < QK_COLS) sums[threadIdx.x / 32][col] = s;
    __syncthreads();
    if (threadIdx.x >= QK_COLS) return;
    s = 0.f;
#pragma unroll
    for (int w = 0; w < QK_SUMS / 32; ++w) s += sums[w][col];
    (which ? dwk : dwq)[(size_t)blockIdx.x * d + i] = s;
}

template <bool BACKWARD>
int tile_of(int d) {
    return d == 128 ? QkLay<128, BACKWARD>::TT : d == 96 ? QkLay<96, BACKWARD>::TT : d == 64 ? QkLay<64, BACKWARD>::TT : QkLay<32, BACKWARD>::TT;
}

// A block's heads and tiles. Forward: a tile of as many heads as leave every SM four blocks, for which its angles
// are formed once (8 x 16 heads of 4,096 tokens, d = 96: 86 us, 112 with four heads a block; 32 heads of 32,768, d = 128:
// 180 and 259). Backward: a head of q and of k a warp, and tiles enough, eight at most, that the sums over the rows are few
// (the same: 209 us, 336 with one tile; 409 us, 451 with four, 790 with one; 16 tiles gain nothing).
struct QkPlan {
    int heads, groups, tiles, spans;
    long long grid;
};
QkPlan qk_plan(bool backward, int B, int H, int T, int d) {
    const int tile = backward ? tile_of<true>(d) : tile_of<false>(d);
    const long long tiles = ((long long)T + tile - 1) / tile, enough = 4LL * sm_count();
    QkPlan p;
    p.heads = QK_WARPS / 2;
    p.tiles = 1;
    if (backward) {
        const long long groups = (H + p.heads - 1) / p.heads;
        while (p.tiles < 8 && (long long)B * groups * ((tiles + 2 * p.tiles - 1) / (2 * p.tiles)) >= enough) p.tiles *= 2;
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
    vla_qk_sums_kernel<<<dim3((unsigned)(shared ? 1 : H), (unsigned)(d / QK_COLS), 2), QK_SUMS, 0, s>>>(a.partial, B * p.spans, H, d, a.shared,
                                                                                                  dweight_q, dweight_k);
    return cudaGetLastError() == cudaSuccess ? VLA_OK : VLA_ERR_CUDA;
}

}  // extern "C"
