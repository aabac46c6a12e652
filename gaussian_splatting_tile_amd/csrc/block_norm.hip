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
    bool wide;    // 16-byte accesses
    int per;      // elements of a thread
};

typedef __bf16 bf16;
typedef _Float16 f16;

template <typename T, int N>
struct Pack {
    typedef T type __attribute__((ext_vector_type(N)));
};
template <typename T>
struct Pack<T, 1> {
    typedef T type;
};

// A thread's elements of a row: NV groups of V neighbours.
template <typename T, int V, int NV>
struct Rows {
    static constexpr int NE = V * NV;
    typedef typename Pack<T, V>::type P;
    int lane, lanes, width;

    __device__ __forceinline__ int at(int j) const { return (j * lanes + lane) * V; }
    __device__ __forceinline__ void load(const void* base, int64_t row, float fill, float (&v)[NE]) const {
        const T* const p = (const T*)base + row;
        P r[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at(j) < width) r[j] = *(const P*)(p + at(j));
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if constexpr (V == 1)
                    v[j] = at(j) < width ? (float)r[j] : fill;
                else
                    v[j * V + i] = at(j) < width ? (float)r[j][i] : fill;
            }
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
            if (at(j) < width) *(P*)(p + at(j)) = r;
        }
    }
    // A vector of weights of type `dtype`, `fill` where there is none.
    __device__ __forceinline__ void weights(const void* w, int dtype, float fill, float (&v)[NE]) const {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int k = at(j) + i;
                float x = fill;
                if (w && k < width)
                    x = dtype == GS_F32 ? ((const float*)w)[k]
                                        : dtype == GS_BF16 ? (float)((const bf16*)w)[k] : (float)((const f16*)w)[k];
                v[j * V + i] = x;
            }
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
        for (int i = 0; i < R::NE; ++i) x[i] = rows.at(i / (R::NE / R::NVs)) < rows.width ? x[i] - m : 0.0f;
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

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

template <typename T, int V, int NV>
struct RowsN : Rows<T, V, NV> {
    static constexpr int NVs = NV;
};

__device__ __forceinline__ int64_t row_at(int64_t row, int inner, int64_t so, int64_t si) {
    const int64_t o = row / inner;
    return o * so + (row - o * inner) * si;
}

template <typename T, int V, int NV>
__global__ __launch_bounds__(1024) void k_block_norm_fwd(BlockNormArgs a, Geometry g) {
    typedef RowsN<T, V, NV> R;
    constexpr int NE = R::NE;
    __shared__ float lds[2][16][2];
    const gs_block_norm& d = a.d;
    R rows;
    rows.lanes = g.lanes;
    rows.lane = threadIdx.x & (g.lanes - 1);
    rows.width = d.width;
    RowSum sum{lds, g.lanes, 0};
    const int sets = blockDim.x / g.lanes;
    float w[NE], b[NE], s[NE], w2[NE], b2[NE];
    rows.weights(a.post_weight, d.weight_dtype, 1.0f, w);
    rows.weights(a.post_bias, d.weight_dtype, 0.0f, b);
    rows.weights(a.scale, d.weight_dtype, 1.0f, s);
    rows.weights(a.pre_weight, d.weight_dtype, 1.0f, w2);
    rows.weights(a.pre_bias, d.weight_dtype, 0.0f, b2);
    for (int64_t base = (int64_t)blockIdx.x * sets; base < g.rows; base += (int64_t)gridDim.x * sets) {
        const int64_t row = base + threadIdx.x / g.lanes;
        const bool here = row < g.rows;
        rows.width = here ? d.width : 0;
        float x[NE], z[NE], res[NE];
        rows.load(a.y, row_at(row, d.inner, d.y_outer, d.y_inner), 0.0f, x);
        if (d.gating != GS_BLOCK_GATE_NONE)
            rows.load(a.gate, row_at(row, d.inner, d.gate_outer, d.gate_inner), 0.0f, z);
        if (a.residual) rows.load(a.residual, row_at(row, d.inner, d.residual_outer, d.residual_inner), 0.0f, res);
        if (d.post != GS_BLOCK_NORM_NONE) {
            rows.width = d.width;
            normalise(rows, sum, d.post, d.eps, x);
        }
        if (!here) rows.width = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            x[i] = fmaf(x[i], w[i], b[i]);
            if (d.gating != GS_BLOCK_GATE_NONE) x[i] *= sigmoid(z[i]) * (d.gating == GS_BLOCK_GATE_SILU ? z[i] : 1.0f);
            x[i] = a.residual ? fmaf(s[i], x[i], res[i]) : s[i] * x[i];
        }
        const int64_t at = row * d.width;
        if (a.out) rows.store(a.out, at, x);
        if (d.pre != GS_BLOCK_NORM_NONE) {
            rows.width = d.width;
            // what lies past the width holds the biases
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = rows.at(i / V) < d.width ? x[i] : 0.0f;
            normalise(rows, sum, d.pre, d.eps, x);
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = fmaf(x[i], w2[i], b2[i]);
            if (here) rows.store(a.norm, at, x);
        }
    }
}

// The sums of a workgroup go to partial[workgroup][5][width].
template <typename T, int V, int NV, bool BIAS>
__global__ __launch_bounds__(1024) void k_block_norm_bwd(BlockNormArgs a, Geometry g, float* partial) {
    typedef RowsN<T, V, NV> R;
    constexpr int NE = R::NE;
    __shared__ float lds[2][16][2];
    const gs_block_norm& d = a.d;
    R rows;
    rows.lanes = g.lanes;
    rows.lane = threadIdx.x & (g.lanes - 1);
    rows.width = d.width;
    RowSum sum{lds, g.lanes, 0};
    const int sets = blockDim.x / g.lanes;
    float w[NE], b[NE], s[NE], w2[NE];
    rows.weights(a.post_weight, d.weight_dtype, 1.0f, w);
    rows.weights(a.post_bias, d.weight_dtype, 0.0f, b);
    rows.weights(a.scale, d.weight_dtype, 1.0f, s);
    rows.weights(a.pre_weight, d.weight_dtype, 1.0f, w2);
    constexpr int NS = BIAS ? 5 : 3;
    float acc[NS][NE];  // post_weight, scale, pre_weight, post_bias, pre_bias
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int i = 0; i < NE; ++i) acc[k][i] = 0.0f;
    for (int64_t base = (int64_t)blockIdx.x * sets; base < g.rows; base += (int64_t)gridDim.x * sets) {
        const int64_t row = base + threadIdx.x / g.lanes;
        const bool here = row < g.rows;
        const int64_t at = row * d.width;
        rows.width = here ? d.width : 0;
        float x[NE], z[NE], c[NE], u[NE], dn[NE];
        rows.load(a.y, row_at(row, d.inner, d.y_outer, d.y_inner), 0.0f, x);
        const bool gated = d.gating != GS_BLOCK_GATE_NONE, pre = d.pre != GS_BLOCK_NORM_NONE;
        if (gated) rows.load(a.gate, row_at(row, d.inner, d.gate_outer, d.gate_inner), 0.0f, z);
        if (pre) {
            if (a.residual) rows.load(a.residual, row_at(row, d.inner, d.residual_outer, d.residual_inner), 0.0f, u);
            rows.load(a.grad_norm, at, 0.0f, dn);
        }
        float up[NE];
        if (a.grad_out) rows.load(a.grad_out, at, 0.0f, up);
        rows.width = d.width;
        float r = 1.0f;
        if (d.post != GS_BLOCK_NORM_NONE) r = normalise(rows, sum, d.post, d.eps, x);
        float act[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float t = fmaf(x[i], w[i], b[i]);
            act[i] = 1.0f;
            c[i] = t;
            if (gated) {
                const float sg = sigmoid(z[i]);
                const bool silu = d.gating == GS_BLOCK_GATE_SILU;
                act[i] = silu ? z[i] * sg : sg;
                c[i] = act[i] * t;
                // the derivative of the gate's factor, times what it multiplies
                z[i] = t * (silu ? sg * fmaf(z[i], 1.0f - sg, 1.0f) : sg * (1.0f - sg));
            }
        }
        if (pre) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const float v = a.residual ? fmaf(s[i], c[i], u[i]) : s[i] * c[i];
                u[i] = here && rows.at(i / V) < d.width ? v : 0.0f;
            }
            const float r2 = normalise(rows, sum, d.pre, d.eps, u);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                acc[2][i] = fmaf(dn[i], u[i], acc[2][i]);
                if constexpr (BIAS) acc[4][i] += dn[i];
                dn[i] *= w2[i];
            }
            normalise_back(rows, sum, d.pre, r2, u, dn);
#pragma unroll
            for (int i = 0; i < NE; ++i) dn[i] = a.grad_out ? dn[i] + up[i] : dn[i];
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) dn[i] = up[i];
        }
        // past the width (and past the rows) everything upstream is 0, but for a layer norm's mean
#pragma unroll
        for (int i = 0; i < NE; ++i) dn[i] = here && rows.at(i / V) < d.width ? dn[i] : 0.0f;
        if (!here) rows.width = 0;
        if (a.grad_residual) rows.store(a.grad_residual, at, dn);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            acc[1][i] = fmaf(dn[i], c[i], acc[1][i]);
            dn[i] *= s[i];
            if (gated) {
                z[i] *= dn[i];
                dn[i] *= act[i];
            }
        }
        if (gated && a.grad_gate) rows.store(a.grad_gate, at, z);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            acc[0][i] = fmaf(dn[i], x[i], acc[0][i]);
            if constexpr (BIAS) acc[3][i] += dn[i];
            dn[i] *= w[i];
        }
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
                if (rows.at(i / V) < d.width) to[rows.at(i / V) + i % V] = acc[k][i];
        } else {  // the rows a workgroup holds at once, through LDS in their order
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NE; ++i) join[i * blockDim.x + threadIdx.x] = acc[k][i];
            __syncthreads();
            for (int e = threadIdx.x; e < NE * g.lanes; e += blockDim.x) {
                const int i = e / g.lanes, lane = e & (g.lanes - 1);
                float t = 0.0f;
                for (int q = 0; q < sets; ++q) t += join[i * blockDim.x + q * g.lanes + lane];
                const int col = ((i / V) * g.lanes + lane) * V + i % V;
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

template <typename... P>
bool aligned16(P... p) {
    return !((0 | ... | (uintptr_t)p) & 15);
}

Geometry geometry(const gs_block_norm& d, bool wide, bool backward) {
    Geometry g;
    g.rows = d.outer * d.inner;
    g.wide = wide;
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

// Whether rows can be read and written in 16-byte pieces.
bool wide_rows(const BlockNormArgs& a) {
    const gs_block_norm& d = a.d;
    const int v = d.dtype == GS_F32 ? 4 : 8;
    int64_t all = d.width | d.y_outer | d.y_inner;
    if (d.gating != GS_BLOCK_GATE_NONE) all |= d.gate_outer | d.gate_inner;
    if (a.residual) all |= d.residual_outer | d.residual_inner;
    if (all & (v - 1)) return false;
    return aligned16(a.y, a.gate, a.residual, a.out, a.norm, a.grad_out, a.grad_norm, a.grad_y, a.grad_gate,
                     a.grad_residual);
}

template <typename T, int V>
hipError_t forward(const BlockNormArgs& a, const Geometry& g, hipStream_t stream) {
    if (g.per == 8)
        k_block_norm_fwd<T, V, 8 / V><<<g.grid, g.block, 0, stream>>>(a, g);
    else
        k_block_norm_fwd<T, V, 16 / V><<<g.grid, g.block, 0, stream>>>(a, g);
    return hipGetLastError();
}

template <typename T, int V, bool BIAS>
hipError_t backward(const BlockNormArgs& a, const Geometry& g, float* scratch, hipStream_t stream) {
    if (g.per == 8)
        k_block_norm_bwd<T, V, 8 / V, BIAS><<<g.grid, g.block, 0, stream>>>(a, g, scratch);
    else
        k_block_norm_bwd<T, V, 16 / V, BIAS><<<g.grid, g.block, 0, stream>>>(a, g, scratch);
    return hipGetLastError();
}

template <typename T>
hipError_t forward_of(const BlockNormArgs& a, const Geometry& g, hipStream_t stream) {
    return g.wide ? forward<T, 16 / sizeof(T)>(a, g, stream) : forward<T, 1>(a, g, stream);
}

template <typename T>
hipError_t backward_of(const BlockNormArgs& a, const Geometry& g, float* scratch, hipStream_t stream) {
    if (a.sums[1] || a.sums[4])
        return g.wide ? backward<T, 16 / sizeof(T), true>(a, g, scratch, stream) : backward<T, 1, true>(a, g, scratch, stream);
    return g.wide ? backward<T, 16 / sizeof(T), false>(a, g, scratch, stream) : backward<T, 1, false>(a, g, scratch, stream);
}

}  // namespace

size_t block_norm_scratch_bytes(const gs_block_norm& d) {
    if (d.outer == 0) return 0;
    return (size_t)geometry(d, false, true).grid * 5 * d.width * sizeof(float);
}

hipError_t launch_block_norm_fwd(const BlockNormArgs& a, hipStream_t stream) {
    const Geometry g = geometry(a.d, wide_rows(a), false);
    switch (a.d.dtype) {
        case GS_F32: return forward_of<float>(a, g, stream);
        case GS_BF16: return forward_of<bf16>(a, g, stream);
        default: return forward_of<f16>(a, g, stream);
    }
}

hipError_t launch_block_norm_bwd(const BlockNormArgs& a, float* scratch, hipStream_t stream) {
    Geometry g = geometry(a.d, wide_rows(a), true);
    hipError_t e = hipSuccess;
    if (a.d.outer == 0)
        g.grid = 0;  // the sums of no rows are 0
    else
    switch (a.d.dtype) {
        case GS_F32: e = backward_of<float>(a, g, scratch, stream); break;
        case GS_BF16: e = backward_of<bf16>(a, g, scratch, stream); break;
        default: e = backward_of<f16>(a, g, scratch, stream); break;
    }
    SumArgs s;
    bool any = false;
    for (int k = 0; k < 5; ++k) any |= (s.to[k] = a.sums[k]) != nullptr;
    if (e != hipSuccess || !any) return e;
    k_block_norm_sums<<<dim3((a.d.width + 63) / 64, 5), 1024, 0, stream>>>(scratch, g.grid, a.d.width, s);
    return hipGetLastError();
}

}  // namespace gs
