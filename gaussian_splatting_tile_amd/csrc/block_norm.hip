// The norms around a block with gate, residual scale and residual between
// them, forward and backward (include/gs.h, gs_block_norm_*).
//
// Per row: yhat = (y - m) r, t = yhat w + b, c = act(z) t, x = res + s c,
// xhat = (x - m') r', norm = xhat w' + b'. Backwards, with d the gradient of
// x and <> the mean over the row,
//   d = grad_out + r' (g - [layer] <g> - xhat <g xhat>),  g = grad_norm w'
//   grad_residual = d;  grad_scale = sum d c;  grad_gate = d s t act'(z)
//   h = d s act(z);  grad_post_weight = sum h yhat;  grad_post_bias = sum h
//   grad_y = r (h w - [layer] <h w> - yhat <h w yhat>).
//
// Both directions are bound by memory: every row is read and written once, all
// of it in the registers of the threads that share it, so the backward
// recomputes the forward's values (a few operations each) instead of reading
// them. A row belongs to `lanes` threads (a power of two, chosen so that a
// thread holds at most NE elements) and a workgroup walks rows in strides of
// the grid. The sums over the rows are formed per workgroup and added over the
// workgroups by a second launch, in a fixed order.
//
// Measured (a copy of as many bytes moves 5.06 TB/s): forward with residual,
// sigmoid gate and both norms, 16384 x 2048 bf16, 335 MB: 64 us, 5.2 TB/s; its
// backward, 537 MB: 120 us, 4.5 TB/s; 8192 x 8192 f16 forward, 671 MB: 136 us,
// 4.9 TB/s; 262144 x 128 bf16 with a silu gate, both directions, 537 MB: 103 us.
// One of 64 x 2048 takes 4.2 us, a launch's latency.
#include <algorithm>
#include <type_traits>

#include "gs_internal.h"

namespace gs {
namespace {

struct Geometry {
    int lanes;    // threads of a row
    int block;    // threads of a workgroup
    int grid;
    int64_t rows;
    int per;      // elements of a thread, at most
};

typedef __bf16 bf16;
typedef _Float16 f16;
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Aligned to an element only: the hardware takes 16-byte accesses at any address.
template <typename T, int N>
struct Pack {
    typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};
template <typename T>
struct Pack<T, 1> {
    typedef T type;
};

// A thread's elements of a row: NV groups of V neighbours. The last group of a
// row whose width is no multiple of V is read where it ends with the row and
// moved to its place, and stored element by element; so rows of odd widths are
// read in 16-byte pieces as well (rows narrower than one have V = 1).
template <typename T, int V, int NV>
struct Rows {
    static constexpr int NE = V * NV, NVs = NV;
    typedef typename Pack<T, V>::type P;
    struct Raw {
        P r[NV];
        __device__ __forceinline__ float operator[](int i) const {
            if constexpr (V == 1)
                return (float)r[i];
            else
                return (float)r[i / V][i % V];
        }
    };
    int lane, lanes, width;

    __device__ __forceinline__ int at(int j) const { return (j * lanes + lane) * V; }
    __device__ __forceinline__ bool in(int i) const { return at(i / V) + i % V < width; }
    // the elements of a group move down by the ones it was read too early; what is behind them counts for nothing
    template <typename Q>
    static __device__ __forceinline__ Q moved(Q r, int by) {
        if constexpr (sizeof(Q) == 16 && V == 8) {
            typedef uint32_t U4 __attribute__((ext_vector_type(4)));
            U4 u = __builtin_bit_cast(U4, r);
            if (by & 4) u = U4{u[2], u[3], 0, 0};
            if (by & 2) u = U4{u[1], u[2], u[3], 0};
            if (by & 1)
                u = U4{__builtin_amdgcn_alignbit(u[1], u[0], 16), __builtin_amdgcn_alignbit(u[2], u[1], 16),
                       __builtin_amdgcn_alignbit(u[3], u[2], 16), u[3] >> 16};
            return __builtin_bit_cast(Q, u);
        } else if constexpr (V == 8) {
            if (by & 4) r = Q{r[4], r[5], r[6], r[7], 0, 0, 0, 0};
            if (by & 2) r = Q{r[2], r[3], r[4], r[5], r[6], r[7], 0, 0};
            if (by & 1) r = Q{r[1], r[2], r[3], r[4], r[5], r[6], r[7], 0};
        } else if constexpr (V == 4) {
            if (by & 2) r = Q{r[2], r[3], 0, 0};
            if (by & 1) r = Q{r[1], r[2], r[3], 0};
        }
        return r;
    }
    // group j of a row of W at p, 0 past the width
    template <typename W>
    __device__ __forceinline__ typename Pack<W, V>::type group(const W* p, int j) const {
        typedef typename Pack<W, V>::type Q;
        Q q{};
        const int from = V == 1 ? at(j) : min(at(j), width - V);
        if (at(j) < width) {
            q = *(const Q*)((const char*)p + (uint32_t)(from * (int)sizeof(W)));
            if constexpr (V > 1)
                if (from != at(j)) q = moved(q, at(j) - from);
        }
        return q;
    }
    // Loads first, all of them, and the moves behind them.
    __device__ __forceinline__ void load(const void* base, int64_t row, Raw& v) const {
        const T* const p = (const T*)base + row;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            v.r[j] = P{};
            const int from = V == 1 ? at(j) : min(at(j), width - V);
            if (at(j) < width) v.r[j] = *(const P*)((const char*)p + (uint32_t)(from * (int)sizeof(T)));
        }
    }
    __device__ __forceinline__ void settle(Raw& v) const {
        if (V > 1 && width % V)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (at(j) < width && at(j) + V > width) v.r[j] = moved(v.r[j], at(j) + V - width);
    }
    __device__ __forceinline__ void store(void* base, int64_t row, const float (&v)[NE]) const {
        T* const p = (T*)base + row;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            P r;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if constexpr (V == 1)
                    r = (T)v[j];
                else
                    r[i] = (T)v[j * V + i];
            }
            if (at(j) + V <= width) {
                *(P*)((char*)p + (uint32_t)(at(j) * (int)sizeof(T))) = r;
            } else if constexpr (V > 1) {
                for (int i = 0; i < V - 1; ++i)
                    if (at(j) + i < width) p[at(j) + i] = (T)v[j * V + i];
            }
        }
    }
    // A vector of weights, of type float32 or that of the rows; `fill` where there is none.
    __device__ __forceinline__ void weights(const void* w, int dtype, float fill, float (&v)[NE]) const {
#pragma unroll
        for (int e = 0; e < NE; ++e) v[e] = fill;
        if (!w) return;
        auto take = [&](auto* p) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const auto q = group(p, j);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if constexpr (V == 1)
                        v[j] = (float)q;
                    else
                        v[j * V + i] = (float)q[i];
                }
            }
        };
        if (sizeof(T) == 4 || dtype == GS_F32)
            take((const float*)w);
        else
            take((const T*)w);
    }
};

// x and that of another lane: the neighbour at a power of two, or its mirror
// image where all lanes up to that power hold the same sum already.
template <int CTRL>
__device__ __forceinline__ float with_lane(float x) {
    return x + __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
// The sum over `n` neighbouring lanes (a power of two, 1 to 64), in all of them;
// register moves only: shuffles through LDS waited for each other (8192 x 8192
// forward 167 us with them, 143 without).
__device__ __forceinline__ float over_lanes(float x, int n) {
    if (n > 1) x = with_lane<0xB1>(x);   // lane ^ 1
    if (n > 2) x = with_lane<0x4E>(x);   // lane ^ 2
    if (n > 4) x = with_lane<0x141>(x);  // 7 - lane of 8
    if (n > 8) x = with_lane<0x140>(x);  // 15 - lane of 16
    if (n > 16) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    if (n > 32) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    return x;
}

// Sums of one or two values over the threads of a row, the same in all of them.
// One barrier where a row is more than a wave; the two halves of `lds` alternate.
struct RowSum {
    float (*lds)[16][2];
    int lanes, turn;
    __device__ __forceinline__ void operator()(float& a, float& b) {
        sum<true>(a, b);
    }
    __device__ __forceinline__ void operator()(float& a) {
        float none = 0.0f;
        sum<false>(a, none);
    }
    template <bool BOTH>
    __device__ __forceinline__ void sum(float& a, float& b) {
        const int in_wave = min(lanes, 64);
        a = over_lanes(a, in_wave);
        if (BOTH) b = over_lanes(b, in_wave);
        if (lanes > 64) {
            const int wave = threadIdx.x >> 6, waves = lanes >> 6, first = wave & ~(waves - 1);
            float (*const to)[2] = lds[turn];
            if ((threadIdx.x & 63) == 0) {
                to[wave][0] = a;
                if (BOTH) to[wave][1] = b;
            }
            __syncthreads();
            const int from = first + (threadIdx.x & (waves - 1));
            a = over_lanes(to[from][0], waves);
            if (BOTH) b = over_lanes(to[from][1], waves);
            turn ^= 1;
        }
    }
};

// 1 / sqrt(v) within an ulp; the hardware's takes normal numbers only.
__device__ __forceinline__ float inverse_root(float v) {
    const bool small = v < 0x1p-96f;
    return __builtin_amdgcn_rsqf(small ? v * 0x1p64f : v) * (small ? 0x1p32f : 1.0f);
}

// x -> (x - m) r in place; returns r. Elements past the width are 0 and stay it. `inv`: 1 / width.
template <typename R>
__device__ __forceinline__ float normalise(const R& rows, RowSum& sum, int kind, float inv, float eps, float (&x)[R::NE]) {
    float s = 0.0f;
    if (kind == GS_BLOCK_NORM_LAYER) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < R::NE; ++i) m += x[i];
        sum(m);
        m *= inv;
#pragma unroll
        for (int i = 0; i < R::NE; ++i) x[i] = rows.in(i) ? x[i] - m : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < R::NE; ++i) s = fmaf(x[i], x[i], s);
    sum(s);
    const float r = inverse_root(fmaf(s, inv, eps));
#pragma unroll
    for (int i = 0; i < R::NE; ++i) x[i] *= r;
    return r;
}

// g -> r (g - [layer] <g> - xhat <g xhat>); 0 past the width where g and xhat are.
template <typename R>
__device__ __forceinline__ void normalise_back(const R& rows, RowSum& sum, int kind, float inv, float r,
                                               const float (&xhat)[R::NE], float (&g)[R::NE]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < R::NE; ++i) a = fmaf(g[i], xhat[i], a);
    if (kind == GS_BLOCK_NORM_LAYER) {
        float b = 0.0f;
#pragma unroll
        for (int i = 0; i < R::NE; ++i) b += g[i];
        sum(a, b);
        a *= -inv;
        b *= inv;
#pragma unroll
        for (int i = 0; i < R::NE; ++i) g[i] = rows.in(i) ? r * fmaf(xhat[i], a, g[i] - b) : 0.0f;
    } else {
        sum(a);
        a *= -inv;
#pragma unroll
        for (int i = 0; i < R::NE; ++i) g[i] = r * fmaf(xhat[i], a, g[i]);
    }
}

// q / (1 + q) with q = exp(-|z|): the smaller of sigmoid(z) and its rest to 1, from which both follow without a
// difference of close numbers. For float32 the exponential's argument |z| log2(e) is taken with what its rounding, and
// that of log2(e), leave out; without, that is |z| 2^-24 of the result, at most 2^-17 before it is 0, which 16-bit outputs
// do not show (8192 x 8192 f16 forward 136 us without, 149 with). |z| over 128 gives 0 as 128 does.
template <typename T>
__device__ __forceinline__ float smaller_side(float z) {
    float a = fabsf(z), q;
    if constexpr (sizeof(T) == 4) {
        a = a > 128.0f ? 128.0f : a;
        const float t = -1.44269502f * a, rest = fmaf(-1.92596303e-8f, a, fmaf(-1.44269502f, a, -t));
        q = __builtin_amdgcn_exp2f(t);
        q = fmaf(q, rest * 0.693147182f, q);
    } else {
        q = __builtin_amdgcn_exp2f(-1.44269502f * a);
    }
    return q * __builtin_amdgcn_rcpf(1.0f + q);
}
// sigmoid(z), of its smaller side
__device__ __forceinline__ float sigmoid(float z, float side) { return z > 0.0f ? 1.0f - side : side; }
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    if constexpr (sizeof(T) == 4) return sigmoid(z, smaller_side<T>(z));
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269502f * z));
}

// What differs between the gates act(z) = sigmoid(z) e, e being z (silu) or 1,
// chosen by bits: a select on a value that all threads share becomes a branch
// for every element (8192 x 8192 forward 143 us with, 139 without). act'(z) = sigmoid(z) [silu] + e sigmoid(z) (1 - sigmoid(z)).
struct Gate {
    uint32_t silu;
    __device__ __forceinline__ explicit Gate(int gating) : silu(gating == GS_BLOCK_GATE_SILU ? ~0u : 0u) {
        asm volatile("" : "+v"(silu));
    }
    __device__ __forceinline__ float factor(float z) const {
        return __uint_as_float((__float_as_uint(z) & silu) | (__float_as_uint(1.0f) & ~silu));
    }
    __device__ __forceinline__ float slope(float e, float sg, float side) const {
        return fmaf(e, side - side * side, __uint_as_float(__float_as_uint(sg) & silu));
    }
};

// Where a row lies: rows are fewer than 2^31, so their place is found in 32 bits, and without a division where they
// follow at one stride.
struct Place {
    uint32_t outer, inner;
    __device__ __forceinline__ Place(int64_t row, int n) : outer((uint32_t)row), inner(0) {
        if (n > 1) {
            outer = (uint32_t)row / (uint32_t)n;
            inner = (uint32_t)row - outer * (uint32_t)n;
        }
    }
    __device__ __forceinline__ int64_t at(int64_t so, int64_t si) const { return outer * so + inner * si; }
};

// Rows of up to 2048 elements: 256 threads that keep the weights in registers.
// Longer ones: 512 or 1024 threads, whose registers do not hold them; they are
// read again for every row, from the caches.
template <typename T, int V, int NV, int BLOCK, bool GATED>
__global__ __launch_bounds__(BLOCK) void k_block_norm_fwd(BlockNormArgs a, Geometry g) {
    typedef Rows<T, V, NV> R;
    constexpr int NE = R::NE;
    constexpr bool KEEP = BLOCK == 256;
    __shared__ float lds[2][16][2];
    const gs_block_norm& d = a.d;
    R rows;
    // a row of more than 2048 elements has the workgroup to itself
    const int lanes = KEEP ? g.lanes : BLOCK, sets = BLOCK / lanes;
    rows.lanes = lanes;
    rows.lane = threadIdx.x & (lanes - 1);
    rows.width = d.width;
    RowSum sum{lds, lanes, 0};
    float w[NE], b[NE], s[NE], w2[NE], b2[NE];
    auto weights = [&](bool first, bool second) {
        if (first) {
            rows.weights(a.post_weight, d.weight_dtype, 1.0f, w);
            rows.weights(a.post_bias, d.weight_dtype, 0.0f, b);
            rows.weights(a.scale, d.weight_dtype, 1.0f, s);
        }
        if (second) {
            rows.weights(a.pre_weight, d.weight_dtype, 1.0f, w2);
            rows.weights(a.pre_bias, d.weight_dtype, 0.0f, b2);
        }
    };
    if constexpr (KEEP) weights(true, true);
    const float inv = 1.0f / (float)d.width;
    const Gate gate(d.gating);
    for (int64_t base = (int64_t)blockIdx.x * sets; base < g.rows; base += (int64_t)gridDim.x * sets) {
        const int64_t row = KEEP ? base + threadIdx.x / lanes : base;
        const bool here = row < g.rows;
        rows.width = here ? d.width : 0;
        typename R::Raw y{}, z{}, res{};
        float x[NE];
        const Place place(row, d.inner);
        rows.load(a.y, place.at(d.y_outer, d.y_inner), y);
        if (GATED) rows.load(a.gate, place.at(d.gate_outer, d.gate_inner), z);
        if (a.residual) rows.load(a.residual, place.at(d.residual_outer, d.residual_inner), res);
        rows.width = d.width;
        rows.settle(y);
        rows.settle(z);
        rows.settle(res);
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = y[i];
        // rows behind the last one hold zeros, which no eps may turn into others
        const float eps = here ? d.eps : 1.0f;
        if (d.post != GS_BLOCK_NORM_NONE) normalise(rows, sum, d.post, inv, eps, x);
        if constexpr (!KEEP) weights(true, false);
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = fmaf(x[i], w[i], b[i]);
        if constexpr (GATED) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                x[i] *= sigmoid<T>(z[i]) * gate.factor(z[i]);
                if (NE > 8 && i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // 16 at once would not fit the registers
            }
        }
        if (a.residual) {
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = fmaf(s[i], x[i], res[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] *= s[i];
        }
        const int64_t at = row * d.width;
        if (!here) rows.width = 0;
        if (a.out) rows.store(a.out, at, x);
        if (d.pre != GS_BLOCK_NORM_NONE) {
            rows.width = d.width;
            if constexpr (!KEEP) weights(false, true);
            normalise(rows, sum, d.pre, inv, eps, x);
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = fmaf(x[i], w2[i], b2[i]);
            if (here) rows.store(a.norm, at, x);
        }
    }
}

// What a backward kernel is compiled for: a pre norm, a gate, and norms by RMS
// without biases or any. Branches that all threads take alike cost no time by
// themselves, but every value that lives across them costs registers: of bf16
// the kernel for any norm, a pre norm and a gate takes 251, that for a pre norm
// and a gate 202, for a gate alone 142 and for neither 110 (both directions of
// 16384 x 2048 222 -> 183 us, of 262144 x 128 125 -> 107 at that step). Two waves
// a SIMD at least, which the first of float32 would miss by two registers.
enum { kWithPre = 1, kWithGate = 2, kAnyNorm = 4 };

// The sums of a workgroup go to partial[workgroup][5][width].
template <typename T, int V, int NV, int BLOCK, int KIND>
__global__ __launch_bounds__(BLOCK, 2) void k_block_norm_bwd(BlockNormArgs a, Geometry g, float* partial) {
    typedef Rows<T, V, NV> R;
    constexpr int NE = R::NE;
    constexpr bool KEEP = BLOCK == 256, BIAS = (KIND & kAnyNorm) != 0;
    __shared__ float lds[2][16][2];
    const gs_block_norm& d = a.d;
    R rows;
    // a row of more than 2048 elements has the workgroup to itself
    const int lanes = KEEP ? g.lanes : BLOCK, sets = BLOCK / lanes;
    rows.lanes = lanes;
    rows.lane = threadIdx.x & (lanes - 1);
    rows.width = d.width;
    RowSum sum{lds, lanes, 0};
    float w[NE], b[NE], s[NE], w2[NE];
    auto weights = [&] {
        rows.weights(a.post_weight, d.weight_dtype, 1.0f, w);
        if constexpr (BIAS) rows.weights(a.post_bias, d.weight_dtype, 0.0f, b);
        rows.weights(a.scale, d.weight_dtype, 1.0f, s);
    };
    if constexpr (KEEP) {
        weights();
        rows.weights(a.pre_weight, d.weight_dtype, 1.0f, w2);
    }
    // The next rows are fetched in front of the work on these, where their registers allow it: two workgroups a CU that
    // do so (16384 x 2048: 183 us) are as good as three that do not (186), and leave half the partial sums.
    constexpr bool AHEAD = BLOCK < 1024;
    constexpr int NS = BIAS ? 5 : 3;
    // Sums over the rows: post_weight, scale, pre_weight, post_bias, pre_bias. 1024 threads have 128 registers each and
    // keep the first of them in LDS, where a thread's 4 neighbours of one sum lie together (4096 x 8192 bf16: 181 us; at
    // that step 182, from 248 with all in registers and 242 with 512 threads of 16 elements). Rows of more than 8192 spill all the same.
    constexpr int NL = BLOCK < 1024 ? 0 : NE == 8 ? std::min(NS, 4) : 2;
    __shared__ f32x4 held[NL ? NL * NE / 4 * BLOCK : 1];
    float acc[NS][NE];
    auto slot = [&](int k, int i) -> f32x4& { return held[(k * (NE / 4) + i / 4) * BLOCK + threadIdx.x]; };
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            if (k >= NL)
                acc[k][i] = 0.0f;
            else if (i % 4 == 0)
                slot(k, i) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    auto add = [&](int k, const float (&x)[NE], const float (&y)[NE]) {
        if (k >= NL) {
#pragma unroll
            for (int i = 0; i < NE; ++i) acc[k][i] = fmaf(x[i], y[i], acc[k][i]);
        } else {
#pragma unroll
            for (int i = 0; i < NE; i += 4) {
                f32x4 t = slot(k, i);
#pragma unroll
                for (int j = 0; j < 4; ++j) t[j] = fmaf(x[i + j], y[i + j], t[j]);
                slot(k, i) = t;
            }
        }
    };
    auto add_one = [&](int k, const float (&x)[NE]) {
        if (k >= NL) {
#pragma unroll
            for (int i = 0; i < NE; ++i) acc[k][i] += x[i];
        } else {
#pragma unroll
            for (int i = 0; i < NE; i += 4) slot(k, i) += f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]};
        }
    };
    constexpr bool gated = (KIND & kWithGate) != 0, pre = (KIND & kWithPre) != 0;
    const Gate gate(d.gating);
    const int post_kind = BIAS ? d.post : GS_BLOCK_NORM_RMS, pre_kind = BIAS ? d.pre : GS_BLOCK_NORM_RMS;
    const float inv = 1.0f / (float)d.width;
    struct In {
        typename R::Raw y, z, res, gn, go;
    };
    auto fetch = [&](int64_t base, In& in) {
        const int64_t row = KEEP ? base + threadIdx.x / lanes : base;
        R from = rows;
        from.width = row < g.rows ? d.width : 0;
        const Place place(row, d.inner);
        from.load(a.y, place.at(d.y_outer, d.y_inner), in.y);
        if (gated) from.load(a.gate, place.at(d.gate_outer, d.gate_inner), in.z);
        if (pre) {
            if (a.residual) from.load(a.residual, place.at(d.residual_outer, d.residual_inner), in.res);
            from.load(a.grad_norm, row * d.width, in.gn);
        }
        if (a.grad_out) from.load(a.grad_out, row * d.width, in.go);
    };
    In next{};
    const int64_t stride = (int64_t)gridDim.x * sets;
    if constexpr (AHEAD) fetch((int64_t)blockIdx.x * sets, next);
    for (int64_t base = (int64_t)blockIdx.x * sets; base < g.rows; base += stride) {
        const int64_t row = KEEP ? base + threadIdx.x / lanes : base;
        const bool here = row < g.rows;
        const int64_t at = row * d.width;
        float x[NE], u[NE], dn[NE];
        if constexpr (!AHEAD) fetch(base, next);
        In in = next;
        typename R::Raw &y = in.y, &z = in.z, &res = in.res, &gn = in.gn, &go = in.go;
        if constexpr (AHEAD)
            if (base + stride < g.rows) fetch(base + stride, next);
        rows.width = d.width;
        rows.settle(y);
        rows.settle(z);
        rows.settle(res);
        rows.settle(gn);
        rows.settle(go);
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = y[i];
        // rows behind the last one hold zeros, which no eps may turn into others
        const float eps = here ? d.eps : 1.0f;
        float r = 1.0f;
        if (d.post != GS_BLOCK_NORM_NONE) r = normalise(rows, sum, post_kind, inv, eps, x);
        if constexpr (!KEEP) weights();
        // the post norm's output
        auto normed = [&](int i) {
            if constexpr (BIAS) return fmaf(x[i], w[i], b[i]);
            return x[i] * w[i];
        };
        float side[NE];
        if (gated) {
#pragma unroll
            for (int i = 0; i < NE; ++i) side[i] = smaller_side<T>(z[i]);
        }
        if (pre) {
#pragma unroll
            for (int i = 0; i < NE; ++i) u[i] = normed(i);
            if (gated) {
#pragma unroll
                for (int i = 0; i < NE; ++i) u[i] *= sigmoid(z[i], side[i]) * gate.factor(z[i]);
            }
#pragma unroll
            for (int i = 0; i < NE; ++i) u[i] = fmaf(s[i], u[i], res[i]);  // no residual: zeros
            const float r2 = normalise(rows, sum, pre_kind, inv, eps, u);
            if constexpr (!KEEP) rows.weights(a.pre_weight, d.weight_dtype, 1.0f, w2);
#pragma unroll
            for (int i = 0; i < NE; ++i) dn[i] = gn[i];
            add(2, dn, u);
            if constexpr (BIAS) add_one(4, dn);
#pragma unroll
            for (int i = 0; i < NE; ++i) dn[i] *= w2[i];
            normalise_back(rows, sum, pre_kind, inv, r2, u, dn);
#pragma unroll
            for (int i = 0; i < NE; ++i) dn[i] += go[i];  // no grad_out: zeros
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) dn[i] = go[i];
        }
        if (!here) rows.width = 0;
        if (a.grad_residual) rows.store(a.grad_residual, at, dn);
        // dn: from the gradient of the sum to that of the post norm's output; u: the gate's
        if (gated) {
#pragma unroll
            for (int i = 0; i < NE; ++i) u[i] = sigmoid(z[i], side[i]) * gate.factor(z[i]) * normed(i);
            add(1, dn, u);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const float ds = dn[i] * s[i], e = gate.factor(z[i]), sg = sigmoid(z[i], side[i]);
                u[i] = ds * normed(i) * gate.slope(e, sg, side[i]);
                dn[i] = ds * (sg * e);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) u[i] = normed(i);
            add(1, dn, u);
#pragma unroll
            for (int i = 0; i < NE; ++i) dn[i] *= s[i];
        }
        add(0, dn, x);
        if constexpr (BIAS) add_one(3, dn);
#pragma unroll
        for (int i = 0; i < NE; ++i) dn[i] *= w[i];
        if (gated && a.grad_gate) rows.store(a.grad_gate, at, u);
        if (d.post != GS_BLOCK_NORM_NONE) {
            rows.width = d.width;
            normalise_back(rows, sum, post_kind, inv, r, x, dn);
            if (!here) rows.width = 0;
        }
        rows.store(a.grad_y, at, dn);
    }
    rows.width = d.width;
    __shared__ float join[KEEP ? 256 * 8 : 1];
    constexpr int kTo[5] = {0, 2, 3, 1, 4};
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        if (!a.sums[kTo[k]]) continue;
        float* const to = partial + ((int64_t)blockIdx.x * 5 + kTo[k]) * d.width;
        if (!KEEP || sets == 1) {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (rows.in(i)) to[rows.at(i / V) + i % V] = k < NL ? slot(k, i)[i % 4] : acc[k][i];
        } else if constexpr (KEEP) {  // the rows a workgroup holds at once, through LDS in their order
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NE; ++i) join[i * BLOCK + threadIdx.x] = acc[k][i];
            __syncthreads();
            for (int e = threadIdx.x; e < NE * lanes; e += BLOCK) {
                const int i = e / lanes, lane = e & (lanes - 1);
                float t = 0.0f;
                for (int q = 0; q < sets; ++q) t += join[i * BLOCK + q * lanes + lane];
                const int col = ((i / V) * lanes + lane) * V + i % V;
                if (col < d.width) to[col] = t;
            }
        }
    }
}

// Sums over the workgroups' partials: 64 columns a workgroup, 16 waves over the partials.
struct SumArgs {
    float* to[5];
};
__global__ __launch_bounds__(1024) void k_block_norm_sums(const float* partial, int n, int width, SumArgs s) {
    float* const to = s.to[blockIdx.y];
    if (!to) return;
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
    float t = 0.0f;
    if (col < width) {
        const float* const p = partial + (int64_t)blockIdx.y * width + col;
#pragma unroll 8
        for (int k = wave; k < n; k += 16) t += p[(int64_t)k * 5 * width];
    }
    lds[wave][lane] = t;
    __syncthreads();
    if (wave == 0 && col < width) {
        float r = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) r += lds[k][lane];
        to[col] = r;
    }
}

Geometry geometry(const gs_block_norm& d, bool backward) {
    Geometry g;
    g.rows = d.outer * d.inner;
    g.per = d.width > 8192 ? 16 : 8;
    int lanes = 8;
    while ((int64_t)lanes * g.per < d.width) lanes *= 2;
    g.lanes = lanes;
    g.block = std::max(lanes, 256);
    const int64_t sets = (g.rows + g.block / lanes - 1) / (g.block / lanes);
    // Workgroups: what the chip holds at once; more would wait for the first (and backward write more rows of sums).
    const bool heavy = d.post == GS_BLOCK_NORM_LAYER || d.pre == GS_BLOCK_NORM_LAYER ||
                       (d.pre != GS_BLOCK_NORM_NONE && d.gating != GS_BLOCK_GATE_NONE);
    const int64_t most = backward ? std::max((heavy ? 512 : 768) * 256 / g.block, 256) : 2048 * 256 / g.block;
    g.grid = (int)std::min(sets, most);
    return g;
}

template <typename T, int V, int NV, int BLOCK>
hipError_t go(const BlockNormArgs& a, const Geometry& g, float* scratch, bool back, hipStream_t stream) {
    const bool pre = a.d.pre != GS_BLOCK_NORM_NONE, gated = a.d.gating != GS_BLOCK_GATE_NONE;
    if (!back) {
        if (gated)
            k_block_norm_fwd<T, V, NV, BLOCK, true><<<g.grid, BLOCK, 0, stream>>>(a, g);
        else
            k_block_norm_fwd<T, V, NV, BLOCK, false><<<g.grid, BLOCK, 0, stream>>>(a, g);
        return hipGetLastError();
    }
    auto run = [&](auto kind) {
        k_block_norm_bwd<T, V, NV, BLOCK, decltype(kind)::value><<<g.grid, BLOCK, 0, stream>>>(a, g, scratch);
    };
    auto kinds = [&](auto any) {
        constexpr int K = decltype(any)::value;
        if (pre && gated)
            run(std::integral_constant<int, K | kWithPre | kWithGate>{});
        else if (pre)
            run(std::integral_constant<int, K | kWithPre>{});
        else if (gated)
            run(std::integral_constant<int, K | kWithGate>{});
        else
            run(std::integral_constant<int, K>{});
    };
    const bool any = a.post_bias || a.sums[1] || a.sums[4] || a.d.post == GS_BLOCK_NORM_LAYER || a.d.pre == GS_BLOCK_NORM_LAYER;
    if (V == 1 || any)
        kinds(std::integral_constant<int, kAnyNorm>{});
    else if constexpr (V > 1)
        kinds(std::integral_constant<int, 0>{});
    return hipGetLastError();
}

template <typename T>
hipError_t go(const BlockNormArgs& a, const Geometry& g, float* scratch, bool back, hipStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    if (a.d.width < V) return go<T, 1, 1, 256>(a, g, scratch, back, stream);
    if (g.block == 256) return go<T, V, 8 / V, 256>(a, g, scratch, back, stream);
    if (g.block == 512) return go<T, V, 8 / V, 512>(a, g, scratch, back, stream);
    if (g.per == 8) return go<T, V, 8 / V, 1024>(a, g, scratch, back, stream);
    return go<T, V, 16 / V, 1024>(a, g, scratch, back, stream);
}

hipError_t launch(const BlockNormArgs& a, const Geometry& g, float* scratch, bool back, hipStream_t stream) {
    switch (a.d.dtype) {
        case GS_F32: return go<float>(a, g, scratch, back, stream);
        case GS_BF16: return go<bf16>(a, g, scratch, back, stream);
        default: return go<f16>(a, g, scratch, back, stream);
    }
}

}  // namespace

size_t block_norm_scratch_bytes(const gs_block_norm& d) {
    if (d.outer == 0) return 0;
    return (size_t)geometry(d, true).grid * 5 * d.width * sizeof(float);
}

hipError_t launch_block_norm_fwd(const BlockNormArgs& a, hipStream_t stream) {
    return launch(a, geometry(a.d, false), nullptr, false, stream);
}

hipError_t launch_block_norm_bwd(const BlockNormArgs& a, float* scratch, hipStream_t stream) {
    Geometry g = geometry(a.d, true);
    hipError_t e = hipSuccess;
    if (a.d.outer == 0)
        g.grid = 0;  // the sums of no rows are 0
    else
        e = launch(a, g, scratch, true, stream);
    SumArgs s;
    bool any = false;
    for (int k = 0; k < 5; ++k) any |= (s.to[k] = a.sums[k]) != nullptr;
    if (e != hipSuccess || !any) return e;
    k_block_norm_sums<<<dim3((a.d.width + 63) / 64, 5), 1024, 0, stream>>>(scratch, g.grid, a.d.width, s);
    return hipGetLastError();
}

}  // namespace gs
