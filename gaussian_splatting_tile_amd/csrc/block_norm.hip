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
// thread holds at most NE elements), a workgroup walks rows in strides of the
// grid and keeps the weights in registers. The sums over the rows are formed
// per workgroup in registers and added over the workgroups by a second launch,
// in a fixed order.
#include <algorithm>

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

// Sums of two values over the threads of a row, the same in all of them. One
// barrier where a row is more than a wave; the two halves of `lds` alternate.
struct RowSum {
    float (*lds)[16][2];
    int lanes, turn;
    __device__ __forceinline__ void operator()(float& a, float& b) {
        const int in_wave = min(lanes, 64);
        for (int m = 1; m < in_wave; m <<= 1) {
            a += __shfl_xor(a, m);
            b += __shfl_xor(b, m);
        }
        if (lanes > 64) {
            const int wave = threadIdx.x >> 6, waves = lanes >> 6, first = wave & ~(waves - 1);
            if ((threadIdx.x & 63) == 0) {
                lds[turn][wave][0] = a;
                lds[turn][wave][1] = b;
            }
            __syncthreads();
            a = b = 0.0f;
            for (int w = 0; w < waves; ++w) {
                a += lds[turn][first + w][0];
                b += lds[turn][first + w][1];
            }
            turn ^= 1;
        }
    }
};

// x -> (x - m) r in place (0 past the width); returns r.
template <typename R>
__device__ __forceinline__ float normalise(const R& rows, RowSum& sum, int kind, float eps, float (&x)[R::NE]) {
    const float inv = 1.0f / (float)rows.width;
    float s = 0.0f, none = 0.0f;
    if (kind == GS_BLOCK_NORM_LAYER) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < R::NE; ++i) m += x[i];
        sum(m, none);
        m *= inv;
#pragma unroll
        for (int i = 0; i < R::NE; ++i) x[i] = rows.in(i) ? x[i] - m : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < R::NE; ++i) s = fmaf(x[i], x[i], s);
    sum(s, none);
    const float r = 1.0f / sqrtf(fmaf(s, inv, eps));
#pragma unroll
    for (int i = 0; i < R::NE; ++i) x[i] *= r;
    return r;
}

// g -> r (g - [layer] <g> - xhat <g xhat>).
template <typename R>
__device__ __forceinline__ void normalise_back(const R& rows, RowSum& sum, int kind, float r,
                                               const float (&xhat)[R::NE], float (&g)[R::NE]) {
    const float inv = 1.0f / (float)rows.width;
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int i = 0; i < R::NE; ++i) {
        a = fmaf(g[i], xhat[i], a);
        b += g[i];
    }
    sum(a, b);
    a *= inv;
    b = kind == GS_BLOCK_NORM_LAYER ? b * inv : 0.0f;
#pragma unroll
    for (int i = 0; i < R::NE; ++i) g[i] = r * (g[i] - b - xhat[i] * a);
}

// 1 / (1 + exp(-z)); the hardware's exponential and reciprocal are within an ulp, the product z log2(e) adds |z| 2^-24.
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

__device__ __forceinline__ int64_t row_at(int64_t row, int inner, int64_t so, int64_t si) {
    const int64_t o = row / inner;
    return o * so + (row - o * inner) * si;
}

// Rows of up to 2048 elements: 256 threads that keep the weights in registers.
// Longer ones: 512 or 1024 threads, whose registers do not hold them; they are
// read again for every row, from the caches.
template <typename T, int V, int NV, int BLOCK>
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
    for (int64_t base = (int64_t)blockIdx.x * sets; base < g.rows; base += (int64_t)gridDim.x * sets) {
        const int64_t row = KEEP ? base + threadIdx.x / lanes : base;
        const bool here = row < g.rows;
        rows.width = here ? d.width : 0;
        typename R::Raw y{}, z{}, res{};
        float x[NE];
        rows.load(a.y, row_at(row, d.inner, d.y_outer, d.y_inner), y);
        if (d.gating != GS_BLOCK_GATE_NONE) rows.load(a.gate, row_at(row, d.inner, d.gate_outer, d.gate_inner), z);
        if (a.residual) rows.load(a.residual, row_at(row, d.inner, d.residual_outer, d.residual_inner), res);
        rows.width = d.width;
        rows.settle(y);
        rows.settle(z);
        rows.settle(res);
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = y[i];
        if (d.post != GS_BLOCK_NORM_NONE) normalise(rows, sum, d.post, d.eps, x);
        if constexpr (!KEEP) weights(true, false);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            x[i] = fmaf(x[i], w[i], b[i]);
            if (d.gating != GS_BLOCK_GATE_NONE) x[i] *= sigmoid(z[i]) * (d.gating == GS_BLOCK_GATE_SILU ? z[i] : 1.0f);
            x[i] = a.residual ? fmaf(s[i], x[i], res[i]) : s[i] * x[i];
        }
        const int64_t at = row * d.width;
        if (!here) rows.width = 0;
        if (a.out) rows.store(a.out, at, x);
        if (d.pre != GS_BLOCK_NORM_NONE) {
            rows.width = d.width;
            if constexpr (!KEEP) weights(false, true);
            // what lies past the width holds the biases
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = rows.in(i) ? x[i] : 0.0f;
            normalise(rows, sum, d.pre, d.eps, x);
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = fmaf(x[i], w2[i], b2[i]);
            if (here) rows.store(a.norm, at, x);
        }
    }
}

// The sums of a workgroup go to partial[workgroup][5][width]. BIAS: with a bias
// of the post norm, or the gradient of one asked for.
template <typename T, int V, int NV, int BLOCK, bool BIAS>
__global__ __launch_bounds__(BLOCK) void k_block_norm_bwd(BlockNormArgs a, Geometry g, float* partial) {
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
    constexpr int NS = BIAS ? 5 : 3;
    float acc[NS][NE];  // post_weight, scale, pre_weight, post_bias, pre_bias
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int i = 0; i < NE; ++i) acc[k][i] = 0.0f;
    const bool gated = d.gating != GS_BLOCK_GATE_NONE, silu = d.gating == GS_BLOCK_GATE_SILU;
    const bool pre = d.pre != GS_BLOCK_NORM_NONE;
    for (int64_t base = (int64_t)blockIdx.x * sets; base < g.rows; base += (int64_t)gridDim.x * sets) {
        const int64_t row = KEEP ? base + threadIdx.x / lanes : base;
        const bool here = row < g.rows;
        const int64_t at = row * d.width;
        rows.width = here ? d.width : 0;
        typename R::Raw y{}, z{}, res{}, gn{}, go{};
        float x[NE], u[NE], dn[NE];
        rows.load(a.y, row_at(row, d.inner, d.y_outer, d.y_inner), y);
        if (gated) rows.load(a.gate, row_at(row, d.inner, d.gate_outer, d.gate_inner), z);
        if (pre) {
            if (a.residual) rows.load(a.residual, row_at(row, d.inner, d.residual_outer, d.residual_inner), res);
            rows.load(a.grad_norm, at, gn);
        }
        if (a.grad_out) rows.load(a.grad_out, at, go);
        rows.width = d.width;
        rows.settle(y);
        rows.settle(z);
        rows.settle(res);
        rows.settle(gn);
        rows.settle(go);
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = y[i];
        float r = 1.0f;
        if (d.post != GS_BLOCK_NORM_NONE) r = normalise(rows, sum, d.post, d.eps, x);
        if constexpr (!KEEP) weights();
        // the post norm's output, and that with the gate's factor
        auto normed = [&](int i) {
            float t = x[i] * w[i];
            if constexpr (BIAS) t += b[i];
            return t;
        };
        auto factor = [&](int i, float sg) { return silu ? z[i] * sg : sg; };
        if (pre) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                float v = normed(i);
                if (gated) v *= factor(i, sigmoid(z[i]));
                v = a.residual ? fmaf(s[i], v, res[i]) : s[i] * v;
                u[i] = here && rows.in(i) ? v : 0.0f;
            }
            const float r2 = normalise(rows, sum, d.pre, d.eps, u);
            if constexpr (!KEEP) rows.weights(a.pre_weight, d.weight_dtype, 1.0f, w2);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                acc[2][i] = fmaf(gn[i], u[i], acc[2][i]);
                if constexpr (BIAS) acc[4][i] += gn[i];
                dn[i] = gn[i] * w2[i];
            }
            normalise_back(rows, sum, d.pre, r2, u, dn);
#pragma unroll
            for (int i = 0; i < NE; ++i) dn[i] = a.grad_out ? dn[i] + go[i] : dn[i];
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) dn[i] = go[i];
        }
        // past the width (and past the rows) everything upstream is 0, but for a layer norm's mean
#pragma unroll
        for (int i = 0; i < NE; ++i) dn[i] = here && rows.in(i) ? dn[i] : 0.0f;
        if (!here) rows.width = 0;
        if (a.grad_residual) rows.store(a.grad_residual, at, dn);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            float t = normed(i), f = 1.0f;
            const float ds = dn[i] * s[i];
            if (gated) {
                const float sg = sigmoid(z[i]);
                f = factor(i, sg);
                u[i] = ds * t * (silu ? sg * fmaf(z[i], 1.0f - sg, 1.0f) : sg * (1.0f - sg));
            }
            acc[1][i] = fmaf(dn[i], f * t, acc[1][i]);
            dn[i] = ds * f;
            acc[0][i] = fmaf(dn[i], x[i], acc[0][i]);
            if constexpr (BIAS) acc[3][i] += dn[i];
            dn[i] *= w[i];
        }
        if (gated && a.grad_gate) rows.store(a.grad_gate, at, u);
        if (d.post != GS_BLOCK_NORM_NONE) {
            rows.width = d.width;
            normalise_back(rows, sum, d.post, r, x, dn);
            if (!here) rows.width = 0;
        }
        rows.store(a.grad_y, at, dn);
    }
    rows.width = d.width;
    __shared__ float join[256 * 8];
    constexpr int kTo[5] = {0, 2, 3, 1, 4};
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        if (!a.sums[kTo[k]]) continue;
        float* const to = partial + ((int64_t)blockIdx.x * 5 + kTo[k]) * d.width;
        if (sets == 1) {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (rows.in(i)) to[rows.at(i / V) + i % V] = acc[k][i];
        } else {  // the rows a workgroup holds at once, through LDS in their order
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
    // Workgroups: what the chip holds at once forward; backward every one writes a row of sums.
    const int64_t most = (backward ? (d.width > 1024 ? 512 : 1024) : 2048) * 256 / g.block;
    g.grid = (int)std::min(sets, most);
    return g;
}

template <typename T, int V, int NV, int BLOCK>
hipError_t go(const BlockNormArgs& a, const Geometry& g, float* scratch, bool back, hipStream_t stream) {
    if (!back)
        k_block_norm_fwd<T, V, NV, BLOCK><<<g.grid, BLOCK, 0, stream>>>(a, g);
    else if (a.post_bias || a.sums[1] || a.sums[4])
        k_block_norm_bwd<T, V, NV, BLOCK, true><<<g.grid, BLOCK, 0, stream>>>(a, g, scratch);
    else
        k_block_norm_bwd<T, V, NV, BLOCK, false><<<g.grid, BLOCK, 0, stream>>>(a, g, scratch);
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
