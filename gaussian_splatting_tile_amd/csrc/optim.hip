// Global gradient norm over a list of tensors, clipping by it, and the Adam
// update that clips on the way (include/gs.h, gs_grad_norm, gs_clip_grads,
// gs_adam_step).
//
// A list is worked through in tiles of kOptTile elements, a tile within one
// tensor. The descriptions travel as kernel arguments (kOptTensors of them
// in one launch, longer lists in several), so a call copies nothing to the
// device and can be recorded in a graph. A first pass leaves one partial sum
// per workgroup in the workspace; every workgroup of the second pass adds
// the partials again in the same order, so neither atomics nor a third
// launch is needed.
#include <algorithm>

#include "gs_internal.h"

namespace gs {
namespace {

constexpr int kOptThreads = 256;
constexpr int kOptTile = 4096;
constexpr int kOptTensors = 64;
constexpr int kOptSlots = 4096;  // partial sums of all launches of a call

struct OptScratch {
    double partial[kOptSlots];
    int64_t step;
    float inv_bc1, inv_bc2;
};

// The tensors of one launch; ends[i] is the tile behind tensor i's last.
template <typename D>
struct OptTable {
    D tensor[kOptTensors];
    uint32_t ends[kOptTensors];
    int n;
};

__device__ __forceinline__ float load_as(const void* p, int64_t i, int dtype) {
    if (dtype == GS_F32) return ((const float*)p)[i];
    if (dtype == GS_BF16) return (float)((const __bf16*)p)[i];
    return (float)((const _Float16*)p)[i];
}
__device__ __forceinline__ void store_as(void* p, int64_t i, int dtype, float v) {
    if (dtype == GS_F32)
        ((float*)p)[i] = v;
    else if (dtype == GS_BF16)
        ((__bf16*)p)[i] = (__bf16)v;
    else
        ((_Float16*)p)[i] = (_Float16)v;
}

// Partials of GS_NORM_MAX hold the bits of the largest |g| (as an integer,
// which orders NaN above infinity).
__device__ __forceinline__ double combine(double a, double b, int kind) {
    if (kind == GS_NORM_L2) return a + b;
    const uint64_t x = __double_as_longlong(a), y = __double_as_longlong(b);
    return __longlong_as_double((long long)(x > y ? x : y));
}

__device__ double block_combine(double v, int kind) {
    __shared__ double part[kOptThreads / 64];
#pragma unroll
    for (int d = 32; d; d >>= 1) v = combine(v, __shfl_xor(v, d), kind);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < kOptThreads / 64; ++w) v = combine(v, part[w], kind);
    return v;
}

// The norm in float64 from the partials: the same sum in every workgroup.
__device__ double total_norm(const OptScratch* s, int slots, int kind) {
    double v = 0.0;
    for (int i = threadIdx.x; i < slots; i += kOptThreads) v = combine(v, s->partial[i], kind);
    v = block_combine(v, kind);
    return kind == GS_NORM_L2 ? sqrt(v) : (double)__uint_as_float((uint32_t)__double_as_longlong(v));
}

__device__ __forceinline__ float clip_factor(double norm, float max_norm) {
    const double c = (double)max_norm / (norm + 1e-6);
    return c > 1.0 ? 1.0f : (float)c;  // a NaN norm gives NaN
}

__device__ double power(double b, int64_t n) {
    double r = 1.0;
    for (; n > 0; n >>= 1, b *= b)
        if (n & 1) r *= b;
    return r;
}

// Takes the step count into the workspace: t = *step + 1 and the bias
// corrections of t.
__device__ void adam_begin(OptScratch* s, const int64_t* step, double beta1, double beta2) {
    const int64_t t = *step + 1;
    s->step = t;
    s->inv_bc1 = (float)(1.0 / (1.0 - power(beta1, t)));
    s->inv_bc2 = (float)(1.0 / (1.0 - power(beta2, t)));
}

__global__ void k_adam_begin(OptScratch* s, const int64_t* step, double beta1, double beta2) {
    adam_begin(s, step, beta1, beta2);
}

struct NormTensor {
    const void* g;
    int64_t count;
    int32_t dtype;
};

__global__ __launch_bounds__(kOptThreads) void k_norm_partial(OptTable<NormTensor> t, OptScratch* s, int slot0,
                                                              int kind, const int64_t* step, double beta1,
                                                              double beta2) {
    if (step && blockIdx.x == 0 && threadIdx.x == 0) adam_begin(s, step, beta1, beta2);
    const uint32_t tiles = t.ends[t.n - 1];
    double v = 0.0;
    int k = 0;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        while (tile >= t.ends[k]) ++k;
        const int64_t e0 = (int64_t)(tile - (k ? t.ends[k - 1] : 0)) * kOptTile;
        const int64_t e1 = min(e0 + kOptTile, t.tensor[k].count);
        for (int64_t e = e0 + threadIdx.x; e < e1; e += kOptThreads) {
            const float g = load_as(t.tensor[k].g, e, t.tensor[k].dtype);
            if (kind == GS_NORM_L2)
                v = fma((double)g, (double)g, v);
            else
                v = combine(v, __longlong_as_double((long long)(__float_as_uint(g) & 0x7fffffffu)), kind);
        }
    }
    v = block_combine(v, kind);
    if (threadIdx.x == 0) s->partial[slot0 + blockIdx.x] = v;
}

__global__ __launch_bounds__(kOptThreads) void k_norm_total(const OptScratch* s, int slots, int kind, float* norm) {
    const double n = total_norm(s, slots, kind);
    if (threadIdx.x == 0) *norm = (float)n;
}

struct ClipTensor {
    const void* g;
    void* out;
    int64_t count;
    int32_t dtype;
};

__global__ __launch_bounds__(kOptThreads) void k_clip(OptTable<ClipTensor> t, const OptScratch* s, int slots, int kind,
                                                      float max_norm, float* norm) {
    const double n = total_norm(s, slots, kind);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    const float c = clip_factor(n, max_norm);
    const uint32_t tiles = t.ends[t.n - 1];
    int k = 0;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        while (tile >= t.ends[k]) ++k;
        const ClipTensor& d = t.tensor[k];
        const int64_t e0 = (int64_t)(tile - (k ? t.ends[k - 1] : 0)) * kOptTile;
        const int64_t e1 = min(e0 + kOptTile, d.count);
        for (int64_t e = e0 + threadIdx.x; e < e1; e += kOptThreads)
            store_as(d.out, e, d.dtype, load_as(d.g, e, d.dtype) * c);
    }
}

__global__ __launch_bounds__(kOptThreads) void k_adam(OptTable<gs_adam_tensor> t, const OptScratch* s, int slots,
                                                      gs_adam cfg, int64_t* step, float* norm, bool last) {
    float c = 1.0f;
    if (slots) {
        const double n = total_norm(s, slots, GS_NORM_L2);
        if (norm && last && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
        if ((cfg.flags & GS_ADAM_SKIP_NONFINITE) && !isfinite(n)) return;
        if (cfg.max_norm > 0.0f) c = clip_factor(n, cfg.max_norm);
    }
    if (last && blockIdx.x == 0 && threadIdx.x == 0) *step = s->step;
    const float b1 = (float)cfg.beta1, b2 = (float)cfg.beta2, r1 = (float)(1.0 - cfg.beta1),
                r2 = (float)(1.0 - cfg.beta2), eps = (float)cfg.eps;
    const float inv1 = s->inv_bc1, inv2 = s->inv_bc2;
    const uint32_t tiles = t.n ? t.ends[t.n - 1] : 0;
    int k = 0;
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        while (tile >= t.ends[k]) ++k;
        const gs_adam_tensor& d = t.tensor[k];
        const int64_t e0 = (int64_t)(tile - (k ? t.ends[k - 1] : 0)) * kOptTile;
        const int64_t e1 = min(e0 + kOptTile, d.count);
        const float keep = (float)(1.0 - (double)d.lr * (double)d.weight_decay);
        for (int64_t e = e0 + threadIdx.x; e < e1; e += kOptThreads) {
            const float g = load_as(d.grad, e, d.grad_dtype) * c;
            const float m = fmaf(b1, d.m[e], r1 * g), v = fmaf(b2, d.v[e], r2 * (g * g));
            const float q = (m * inv1) / (sqrtf(v * inv2) + eps);
            store_as(d.param, e, d.param_dtype, fmaf(keep, load_as(d.param, e, d.param_dtype), -(d.lr * q)));
            d.m[e] = m;
            d.v[e] = v;
        }
    }
}

// The tensors [first, first + kOptTensors) of a list that are not empty, as
// a launch's table; returns the number of tiles.
template <typename D, typename S, typename F>
uint32_t fill_table(OptTable<D>& t, const S* tensors, int first, int n, F make) {
    uint32_t tiles = 0;
    t.n = 0;
    for (int i = first; i < std::min(n, first + kOptTensors); ++i) {
        if (tensors[i].count == 0) continue;
        t.tensor[t.n] = make(tensors[i]);
        tiles += (uint32_t)((tensors[i].count + kOptTile - 1) / kOptTile);
        t.ends[t.n++] = tiles;
    }
    return tiles;
}

int blocks_of(uint32_t tiles, int n_tensors) {
    const int launches = std::max(1, (n_tensors + kOptTensors - 1) / kOptTensors);
    return (int)std::min<uint32_t>(tiles, (uint32_t)std::min(2048, kOptSlots / launches));
}

// First pass over the whole list; returns the number of partials.
template <typename S, typename F>
hipError_t launch_partials(const S* tensors, int n, OptScratch* s, int kind, const int64_t* step, double beta1,
                           double beta2, int* slots, F make, hipStream_t stream) {
    *slots = 0;
    for (int first = 0; first < n; first += kOptTensors) {
        OptTable<NormTensor> t;
        const uint32_t tiles = fill_table(t, tensors, first, n, make);
        if (!tiles) continue;
        const int blocks = blocks_of(tiles, n);
        k_norm_partial<<<blocks, kOptThreads, 0, stream>>>(t, s, *slots, kind, *slots ? nullptr : step, beta1, beta2);
        *slots += blocks;
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

NormTensor norm_of(const gs_grad_tensor& d) { return {d.grad, d.count, d.dtype}; }
NormTensor norm_of_adam(const gs_adam_tensor& d) { return {d.grad, d.count, d.grad_dtype}; }

}  // namespace

size_t optim_scratch_bytes() { return sizeof(OptScratch); }

hipError_t launch_grad_norm(const gs_grad_tensor* tensors, int n, int kind, float* norm, void* scratch,
                            hipStream_t stream) {
    OptScratch* s = (OptScratch*)scratch;
    int slots = 0;
    if (hipError_t e = launch_partials(tensors, n, s, kind, nullptr, 0.0, 0.0, &slots, norm_of, stream)) return e;
    k_norm_total<<<1, kOptThreads, 0, stream>>>(s, slots, kind, norm);
    return hipGetLastError();
}

hipError_t launch_clip_grads(const gs_grad_tensor* tensors, int n, int kind, float max_norm, float* norm,
                             void* scratch, hipStream_t stream) {
    OptScratch* s = (OptScratch*)scratch;
    int slots = 0;
    if (hipError_t e = launch_partials(tensors, n, s, kind, nullptr, 0.0, 0.0, &slots, norm_of, stream)) return e;
    if (!slots) {
        k_norm_total<<<1, kOptThreads, 0, stream>>>(s, 0, kind, norm);
        return hipGetLastError();
    }
    for (int first = 0; first < n; first += kOptTensors) {
        OptTable<ClipTensor> t;
        const uint32_t tiles = fill_table(t, tensors, first, n, [](const gs_grad_tensor& d) {
            return ClipTensor{d.grad, d.out, d.count, d.dtype};
        });
        if (!tiles) continue;
        k_clip<<<std::min<uint32_t>(tiles, 4096), kOptThreads, 0, stream>>>(t, s, slots, kind, max_norm, norm);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

hipError_t launch_adam_step(const gs_adam& cfg, const gs_adam_tensor* tensors, int n, int64_t* step, float* norm,
                            void* scratch, hipStream_t stream) {
    OptScratch* s = (OptScratch*)scratch;
    const bool want = norm || cfg.max_norm > 0.0f || (cfg.flags & GS_ADAM_SKIP_NONFINITE);
    int slots = 0;
    if (want) {
        if (hipError_t e = launch_partials(tensors, n, s, GS_NORM_L2, step, cfg.beta1, cfg.beta2, &slots,
                                           norm_of_adam, stream))
            return e;
    }
    if (!slots) {
        k_adam_begin<<<1, 1, 0, stream>>>(s, step, cfg.beta1, cfg.beta2);
        if (hipError_t e = hipGetLastError()) return e;
        if (norm) k_norm_total<<<1, kOptThreads, 0, stream>>>(s, 0, GS_NORM_L2, norm);
    }
    // the last launch takes the new step count; one with no tensor at all if the list is empty
    int lastfirst = 0;
    for (int first = 0; first < n; first += kOptTensors)
        for (int i = first; i < std::min(n, first + kOptTensors); ++i)
            if (tensors[i].count) lastfirst = first;
    for (int first = 0; first <= lastfirst; first += kOptTensors) {
        OptTable<gs_adam_tensor> t;
        const uint32_t tiles = fill_table(t, tensors, first, n, [](const gs_adam_tensor& d) { return d; });
        if (!tiles && first != lastfirst) continue;
        k_adam<<<std::max(1u, std::min<uint32_t>(tiles, 4096)), kOptThreads, 0, stream>>>(t, s, slots, cfg, step, norm,
                                                                                         first == lastfirst);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

}  // namespace gs
