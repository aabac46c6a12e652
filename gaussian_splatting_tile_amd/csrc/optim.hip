// Global gradient norm over a list of tensors, clipping by it, and the Adam
// update that clips on the way (include/gs.h, gs_grad_norm, gs_clip_grads,
// gs_adam_step).
//
// All three are bound by memory. A list is worked through in tiles, each
// within one tensor, in accesses of 16 bytes a lane (8 for the 16-bit side of
// an update). A tensor may start at any element: its tiles are laid out from
// the aligned address in front of it, so that only its first and last access
// go element by element. The descriptions travel as kernel arguments (as many
// as fit 4 KB a launch, longer lists in several launches), so a call copies
// nothing to the device and can be recorded in a graph.
//
// A first pass leaves one partial sum per workgroup in the workspace; every
// workgroup of the second pass adds the partials again in the same order, so
// neither atomics nor a third launch is needed. The second pass walks the
// tiles from the last to the first, as the end of the list is what the first
// pass read last; it makes little difference (against ascending: 300 tensors
// clipped in 67.5 and 67.8 us, a clipped update of 120 tensors in 100.8 and
// 101.9, of 59M float32 parameters in 288 and 284). Small lists take one launch
// of one workgroup instead.
#include <algorithm>
#include <type_traits>

#include "gs_internal.h"

namespace gs {
namespace {

constexpr int kOptThreads = 256;     // threads that share a tile
constexpr int kNormTile = 16384;     // bytes
constexpr int kClipTile = 16384;
constexpr int kAdamTile = 8192;      // bytes of the float32 moments
constexpr int kNormThreads = 1024;   // first pass: four tiles at once, one partial
constexpr int kNormBlocks = 512;     // of a launch: two to a compute unit
constexpr int kOptSlots = 2048;      // partial sums of all launches of a call
// Workgroups of a second-pass launch: one for each tile up to a bound that
// only keeps the grid within limits. Fewer that take several tiles each were
// slower (a clipped update of 59M float32 parameters: 320 us with 2048, 298
// without the bound at that step, 287 now).
constexpr int kOptBlocks = 1 << 22;
constexpr int kSmallThreads = 1024;  // small lists: a wave shares a tile
constexpr int kSmallTile = 2048;
constexpr int64_t kSmallClip = 32768;  // elements: 7.7 us against 9.5 with two launches; at 65536 12.1
constexpr int64_t kSmallAdam = 16384;  // 9.1 us against 9.5; at 32768 14.9

struct OptScratch {
    double partial[kOptSlots];
    int64_t step;
    float inv_bc1, inv_bc2;
};

// The tensors of one launch; ends[i] is the tile behind tensor i's last.
// A kernel's arguments are at most 4 KB: 240 bytes are left for the others.
template <typename D>
struct OptTable {
    static constexpr int kMost = (4096 - 240) / (int)(sizeof(D) + 4);
    D tensor[kMost];
    uint32_t ends[kMost];
    int n;
};

// Elements e .. e + U - 1 of a tensor of `count`, all of which are there if
// WHOLE; else (at its ends) the others read as 0 and are not written. p is
// aligned to its type only: an access is still one instruction. STREAM: what
// is not used again soon and should not push the gradients out of the caches
// between the two passes (a clipped update of 59M float32 parameters when
// it took 353 us in all: 373 without; on the gradients themselves it costs
// 13%).
template <typename T, int U>
struct Access {
    typedef T Vec __attribute__((ext_vector_type(U), aligned(sizeof(T))));
};
template <bool WHOLE, bool STREAM, typename T, int U>
__device__ __forceinline__ void load_n(const T* p, int64_t e, int64_t count, float (&v)[U]) {
    using Vec = typename Access<T, U>::Vec;
    Vec r = {};
    if (WHOLE || (e >= 0 && e + U <= count)) {
        const Vec* const at = (const Vec*)(p + e);
        r = STREAM ? __builtin_nontemporal_load(at) : *at;
    } else if (e + U > 0 && e < count) {  // one lane at either end of a tensor
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (e + j >= 0 && e + j < count) r[j] = p[e + j];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = (float)r[j];
}
template <bool WHOLE, typename T, int U>
__device__ __forceinline__ void store_n(T* p, int64_t e, int64_t count, const float (&v)[U]) {
    using Vec = typename Access<T, U>::Vec;
    if (WHOLE || (e >= 0 && e + U <= count)) {
        Vec r;
#pragma unroll
        for (int j = 0; j < U; ++j) r[j] = (T)v[j];
        __builtin_nontemporal_store(r, (Vec*)(p + e));
    } else if (e + U > 0 && e < count) {
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (e + j >= 0 && e + j < count) p[e + j] = (T)v[j];
    }
}

// Calls f(whole): whether `elements` from e0 on lie inside their tensor. The
// common case then has no branch between the loads of a thread.
template <typename F>
__device__ __forceinline__ void by_extent(int64_t e0, int elements, int64_t count, F f) {
    if (e0 >= 0 && e0 + elements <= count)
        f(std::true_type());
    else
        f(std::false_type());
}

// Calls f with a value of the element type.
template <typename F>
__device__ __forceinline__ void with_type(int dtype, F f) {
    if (dtype == GS_F32)
        f(float());
    else if (dtype == GS_BF16)
        f(__bf16());
    else
        f(_Float16());
}
// Elements of one access of 16 bytes.
template <typename T>
constexpr int kUnit = 16 / (int)sizeof(T);

// Elements between the aligned address in front of a tensor and its start.
__host__ __device__ inline int head_of(const void* p, int bytes, int unit) {
    return (int)((uintptr_t)p / bytes) & (unit - 1);
}

// Partials of GS_NORM_MAX hold the bits of the largest |g| (as an integer,
// which orders NaN above infinity).
__device__ __forceinline__ double combine(double a, double b, int kind) {
    if (kind == GS_NORM_L2) return a + b;
    const uint64_t x = __double_as_longlong(a), y = __double_as_longlong(b);
    return __longlong_as_double((long long)(x > y ? x : y));
}

// Squares in float64: no float32 overflows or underflows in them, and the
// sum of any list is good to a float32 rounding whatever its order. The
// vector units do one such multiply-add per element ten times faster than
// memory delivers elements.
__device__ __forceinline__ double take(double v, float g, int kind) {
    if (kind == GS_NORM_L2) return fma((double)g, (double)g, v);
    return combine(v, __longlong_as_double((long long)(__float_as_uint(g) & 0x7fffffffu)), kind);
}

// Of a whole workgroup of THREADS.
template <int THREADS>
__device__ double block_combine(double v, int kind) {
    __shared__ double part[THREADS / 64];
#pragma unroll
    for (int d = 32; d; d >>= 1) v = combine(v, __shfl_xor(v, d), kind);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v = combine(v, part[w], kind);
    return v;
}

__device__ __forceinline__ double norm_of_sum(double v, int kind) {
    return kind == GS_NORM_L2 ? sqrt(v) : (double)__uint_as_float((uint32_t)__double_as_longlong(v));
}

// The norm in float64 from the partials: the same sum in every workgroup.
__device__ double total_norm(const OptScratch* s, int slots, int kind) {
    double v = 0.0;
    for (int i = threadIdx.x; i < slots; i += kOptThreads) v = combine(v, s->partial[i], kind);
    return norm_of_sum(block_combine<kOptThreads>(v, kind), kind);
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

// Descriptions as the kernels take them: the types ride on the count.
struct NormTensor {
    const void* g;
    int64_t count_type;
};
struct ClipTensor {
    const void* g;
    void* out;
    int64_t count_type;
};
struct AdamTensor {
    void* param;
    const void* grad;
    float *m, *v;
    int64_t count_type;
    float lr, keep;  // keep: 1 - lr weight_decay
};
__host__ __device__ constexpr int64_t with_types(int64_t count, int type, int type2) {
    return count << 4 | type << 2 | type2;
}
template <typename D>
__device__ __forceinline__ int64_t count_of(const D& d) {
    return d.count_type >> 4;
}
template <typename D>
__device__ __forceinline__ int type_of(const D& d) {
    return (int)(d.count_type >> 2) & 3;
}
template <typename D>
__device__ __forceinline__ int type2_of(const D& d) {
    return (int)d.count_type & 3;
}

// One tile of a tensor: TILE bytes from element e0 on (e0 counts from the tensor's
// start and may be negative), by THREADS threads of which this is number i.
template <int THREADS, int TILE, typename T>
__device__ __forceinline__ double norm_tile(const T* g, int64_t e0, int64_t count, int kind, int i, double v) {
    constexpr int U = kUnit<T>, N = TILE / (THREADS * 16);
    by_extent(e0, TILE / (int)sizeof(T), count, [&](auto whole) {
        float x[N][U];
#pragma unroll
        for (int k = 0; k < N; ++k) load_n<whole.value, false>(g, e0 + (k * THREADS + i) * U, count, x[k]);
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int j = 0; j < U; ++j) v = take(v, x[k][j], kind);
    });
    return v;
}

template <int THREADS, int TILE, typename T>
__device__ __forceinline__ void clip_tile(const T* g, T* out, int64_t e0, int64_t count, float c, int i) {
    constexpr int U = kUnit<T>, N = TILE / (THREADS * 16);
    by_extent(e0, TILE / (int)sizeof(T), count, [&](auto whole) {
        float x[N][U];
#pragma unroll
        for (int k = 0; k < N; ++k) load_n<whole.value, false>(g, e0 + (k * THREADS + i) * U, count, x[k]);
#pragma unroll
        for (int k = 0; k < N; ++k) {
#pragma unroll
            for (int j = 0; j < U; ++j) x[k][j] *= c;
            store_n<whole.value>(out, e0 + (k * THREADS + i) * U, count, x[k]);
        }
    });
}

struct AdamConsts {
    float b1, b2, r1, r2, eps, inv1, inv2, c;
    __device__ __forceinline__ AdamConsts(const gs_adam& cfg, float inv_bc1, float inv_bc2, float factor)
        : b1((float)cfg.beta1), b2((float)cfg.beta2), r1((float)(1.0 - cfg.beta1)), r2((float)(1.0 - cfg.beta2)),
          eps((float)cfg.eps), inv1(inv_bc1), inv2(inv_bc2), c(factor) {}
};

// What an update holds of N accesses of four elements (for every type: the
// float32 moments set the pace).
constexpr int kAdamUnit = 4;
template <int N>
struct AdamRegs {
    float p[N][kAdamUnit], g[N][kAdamUnit], m[N][kAdamUnit], v[N][kAdamUnit];
};
template <bool WHOLE, int THREADS, int N>
__device__ __forceinline__ void adam_load_grad(float (&g)[N][kAdamUnit], const AdamTensor& d, int64_t e0, int i) {
    with_type(type2_of(d), [&](auto t) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            load_n<WHOLE, false>((const decltype(t)*)d.grad, e0 + (k * THREADS + i) * kAdamUnit, count_of(d), g[k]);
    });
}
template <bool WHOLE, int THREADS, int N>
__device__ __forceinline__ void adam_load(AdamRegs<N>& x, const AdamTensor& d, int64_t e0, int i) {
    constexpr int U = kAdamUnit;
    const int64_t count = count_of(d);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        load_n<WHOLE, true>((const float*)d.m, e0 + (k * THREADS + i) * U, count, x.m[k]);
        load_n<WHOLE, true>((const float*)d.v, e0 + (k * THREADS + i) * U, count, x.v[k]);
    }
    adam_load_grad<WHOLE, THREADS, N>(x.g, d, e0, i);
    with_type(type_of(d), [&](auto t) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            load_n<WHOLE, true>((const decltype(t)*)d.param, e0 + (k * THREADS + i) * U, count, x.p[k]);
    });
}
template <bool WHOLE, int THREADS, int N>
__device__ __forceinline__ void adam_update(AdamRegs<N>& x, const AdamTensor& d, int64_t e0, int i,
                                            const AdamConsts& c) {
    constexpr int U = kAdamUnit;
    const int64_t count = count_of(d);
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const float g = x.g[k][j] * c.c;
            const float m = fmaf(c.b1, x.m[k][j], c.r1 * g), v = fmaf(c.b2, x.v[k][j], c.r2 * (g * g));
            const float q = (m * c.inv1) / (sqrtf(v * c.inv2) + c.eps);
            x.m[k][j] = m;
            x.v[k][j] = v;
            x.p[k][j] = fmaf(d.keep, x.p[k][j], -(d.lr * q));
        }
        store_n<WHOLE>(d.m, e0 + (k * THREADS + i) * U, count, x.m[k]);
        store_n<WHOLE>(d.v, e0 + (k * THREADS + i) * U, count, x.v[k]);
    }
    with_type(type_of(d), [&](auto t) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            store_n<WHOLE>((decltype(t)*)d.param, e0 + (k * THREADS + i) * U, count, x.p[k]);
    });
}

template <int THREADS, int TILE>
__device__ __forceinline__ double norm_tile_of(const NormTensor& d, int64_t at, int kind, int i, double v) {
    with_type(type_of(d), [&](auto t) {
        using T = decltype(t);
        const int head = head_of(d.g, sizeof(T), kUnit<T>);
        v = norm_tile<THREADS, TILE>((const T*)d.g, at / (int)sizeof(T) - head, count_of(d), kind, i, v);
    });
    return v;
}
template <int THREADS, int TILE>
__device__ __forceinline__ void clip_tile_of(const ClipTensor& d, int64_t at, float c, int i) {
    if (c == 1.0f && d.g == d.out) return;
    with_type(type_of(d), [&](auto t) {
        using T = decltype(t);
        const int head = head_of(d.g, sizeof(T), kUnit<T>);
        clip_tile<THREADS, TILE>((const T*)d.g, (T*)d.out, at / (int)sizeof(T) - head, count_of(d), c, i);
    });
}
// An update's tiles are laid out by the moments.
__device__ __forceinline__ int64_t adam_first(const AdamTensor& d, int64_t at) {
    return at / (int)sizeof(float) - head_of(d.m, sizeof(float), kAdamUnit);
}

template <typename D>
__host__ __device__ inline uint32_t tiles_in(const OptTable<D>& t) {
    return t.n ? t.ends[t.n - 1] : 0;
}

// Calls f(tensor, first byte from its aligned front) for every `stride`th
// tile of a table from `begin` on, in ascending order or (BACK) descending.
// A wave holds the table's ends, one a lane, and finds a tile's tensor by
// counting those at or below the tile: walking the ends in scalar loads cost
// more than the tiles for lists of a hundred tensors.
template <int TILE, bool BACK, typename D, typename F>
__device__ __forceinline__ void for_tiles(const OptTable<D>& t, uint32_t begin, uint32_t stride, F f) {
    constexpr int kLoads = (OptTable<D>::kMost + 63) / 64;
    const int lane = threadIdx.x & 63;
    uint32_t ends[kLoads];
#pragma unroll
    for (int m = 0; m < kLoads; ++m) ends[m] = m * 64 + lane < t.n ? t.ends[m * 64 + lane] : ~0u;
    const uint32_t tiles = tiles_in(t);
    for (uint32_t i = begin; i < tiles; i += stride) {
        const uint32_t tile = BACK ? tiles - 1 - i : i;
        int k = 0;
#pragma unroll
        for (int m = 0; m < kLoads; ++m) k += __popcll(__ballot(ends[m] <= tile));
        f(t.tensor[k], (int64_t)(tile - (k ? t.ends[k - 1] : 0)) * TILE);
    }
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// sum g^2 (or max |g|) of a workgroup's share. Bound by memory, reads alone
// (medians here and below): 59M float32 in 45 us, 5.2 TB/s; 9.4M in 9.2 us (4.1
// TB/s), of which 3 are the launch and the first latency. Two workgroups of 1024 threads to a unit rather
// than one per tile: each leaves a partial that the whole second pass reads
// again, and 512 of them are two loads a thread there.
__global__ __launch_bounds__(kNormThreads) void k_norm_partial(OptTable<NormTensor> t, OptScratch* s, int slot0,
                                                               int kind, const int64_t* step, double beta1,
                                                               double beta2) {
    if (step && blockIdx.x == 0 && threadIdx.x == 0) adam_begin(s, step, beta1, beta2);
    constexpr int kTeams = kNormThreads / kOptThreads;
    const int team = wave_id() / (kOptThreads / 64), i = threadIdx.x % kOptThreads;
    double v = 0.0;
    for_tiles<kNormTile, false>(t, blockIdx.x * kTeams + team, gridDim.x * kTeams, [&](const NormTensor& d, int64_t at) {
        v = norm_tile_of<kOptThreads, kNormTile>(d, at, kind, i, v);
    });
    v = block_combine<kNormThreads>(v, kind);
    if (threadIdx.x == 0) s->partial[slot0 + blockIdx.x] = v;
}

__global__ __launch_bounds__(kOptThreads) void k_norm_total(const OptScratch* s, int slots, int kind, float* norm) {
    const double n = total_norm(s, slots, kind);
    if (threadIdx.x == 0) *norm = (float)n;
}

// out = c g, c = min(1, max_norm / (norm + 1e-6)). Bound by memory: 9.4M float32
// in 14.6 us, 5.2 TB/s read and written. Its first loads wait for the partials'
// reduction. With a factor of 1 gradients in place stay untouched (the whole
// call on 59M float32 138 -> 61 us).
__global__ __launch_bounds__(kOptThreads) void k_clip(OptTable<ClipTensor> t, const OptScratch* s, int slots, int kind,
                                                      float max_norm, float* norm) {
    const double n = total_norm(s, slots, kind);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    const float c = clip_factor(n, max_norm);
    for_tiles<kClipTile, true>(t, blockIdx.x, gridDim.x, [&](const ClipTensor& d, int64_t at) {
        clip_tile_of<kOptThreads, kClipTile>(d, at, c, threadIdx.x);
    });
}

// m = b1 m + (1 - b1) c g, v = b2 v + (1 - b2) (c g)^2, p = keep p - lr (m / bc1)
// / (sqrt(v / bc2) + eps), in float32 from one reading of each. Bound by memory:
// 59M float32 parameters (1.65 GB) in 245 us, 6.7 TB/s (above a copy's rate of
// 5.2: where its bytes come from was not measured); 40 bf16 tensors in 49 us. The
// division and the
// root are correctly rounded: their operations hide behind the rows.
__global__ __launch_bounds__(kOptThreads) void k_adam(OptTable<AdamTensor> t, const OptScratch* s, int slots,
                                                      gs_adam cfg, int64_t* step, float* norm, bool last) {
    float c = 1.0f;
    if (slots) {
        const double n = total_norm(s, slots, GS_NORM_L2);
        if (norm && last && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
        if ((cfg.flags & GS_ADAM_SKIP_NONFINITE) && !isfinite(n)) return;
        if (cfg.max_norm > 0.0f) c = clip_factor(n, cfg.max_norm);
    }
    if (last && blockIdx.x == 0 && threadIdx.x == 0) *step = s->step;
    const AdamConsts consts(cfg, s->inv_bc1, s->inv_bc2, c);
    for_tiles<kAdamTile, true>(t, blockIdx.x, gridDim.x, [&](const AdamTensor& d, int64_t at) {
        constexpr int kElements = kAdamTile / (int)sizeof(float), N = kElements / (kOptThreads * kAdamUnit);
        const int64_t e0 = adam_first(d, at);
        by_extent(e0, kElements, count_of(d), [&](auto whole) {
            AdamRegs<N> x;
            adam_load<whole.value, kOptThreads>(x, d, e0, threadIdx.x);
            adam_update<whole.value, kOptThreads>(x, d, e0, threadIdx.x, consts);
        });
    });
}

// Small lists: one workgroup, a tile per wave, does both passes; the second
// finds the gradients in its L2. Bound by latency: two loads from memory or L2
// behind each other, a barrier and the stores (4.3 us for 2307 elements).
__global__ __launch_bounds__(kSmallThreads) void k_clip_small(OptTable<ClipTensor> t, int kind, float max_norm,
                                                              float* norm) {
    const int wave = wave_id(), lane = threadIdx.x & 63, waves = kSmallThreads / 64;
    double v = 0.0;
    for_tiles<kSmallTile, false>(t, wave, waves, [&](const ClipTensor& d, int64_t at) {
        v = norm_tile_of<64, kSmallTile>(NormTensor{d.g, d.count_type}, at, kind, lane, v);
    });
    const double n = norm_of_sum(block_combine<kSmallThreads>(v, kind), kind);
    if (threadIdx.x == 0) *norm = (float)n;
    const float c = clip_factor(n, max_norm);
    for_tiles<kSmallTile, true>(t, wave, waves, [&](const ClipTensor& d, int64_t at) {
        clip_tile_of<64, kSmallTile>(d, at, c, lane);
    });
}

// The wave's first tile is loaded at the start and stays in registers: lists
// of up to kSmallThreads / 64 tiles wait for memory once (5.5 us for 483
// elements in four tensors). Most tiles here have an end of their tensor in them.
__global__ __launch_bounds__(kSmallThreads) void k_adam_small(OptTable<AdamTensor> t, gs_adam cfg, bool want,
                                                              int64_t* step, float* norm) {
    constexpr int kElements = kSmallTile / (int)sizeof(float), N = kElements / (64 * kAdamUnit);
    __shared__ OptScratch s;
    const int wave = wave_id(), lane = threadIdx.x & 63, waves = kSmallThreads / 64;
    AdamRegs<N> first = {};
    for_tiles<kSmallTile, false>(t, wave, tiles_in(t), [&](const AdamTensor& d, int64_t at) {
        adam_load<false, 64>(first, d, adam_first(d, at), lane);
    });
    if (threadIdx.x == 0) adam_begin(&s, step, cfg.beta1, cfg.beta2);
    float c = 1.0f;
    bool skip = false;
    if (want) {
        double v = 0.0;
        const auto add = [&](const float(&g)[N][kAdamUnit]) {
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int j = 0; j < kAdamUnit; ++j) v = take(v, g[k][j], GS_NORM_L2);
        };
        add(first.g);
        for_tiles<kSmallTile, false>(t, wave + waves, waves, [&](const AdamTensor& d, int64_t at) {
            float g[N][kAdamUnit];
            adam_load_grad<false, 64, N>(g, d, adam_first(d, at), lane);
            add(g);
        });
        const double n = sqrt(block_combine<kSmallThreads>(v, GS_NORM_L2));
        if (norm && threadIdx.x == 0) *norm = (float)n;
        skip = (cfg.flags & GS_ADAM_SKIP_NONFINITE) && !isfinite(n);
        if (cfg.max_norm > 0.0f) c = clip_factor(n, cfg.max_norm);
    } else {
        __syncthreads();
    }
    if (skip) return;
    if (threadIdx.x == 0) *step = s.step;
    const AdamConsts consts(cfg, s.inv_bc1, s.inv_bc2, c);
    for_tiles<kSmallTile, false>(t, wave, tiles_in(t), [&](const AdamTensor& d, int64_t at) {
        adam_update<false, 64>(first, d, adam_first(d, at), lane, consts);
    });
    for_tiles<kSmallTile, false>(t, wave + waves, waves, [&](const AdamTensor& d, int64_t at) {
        AdamRegs<N> x;
        adam_load<false, 64>(x, d, adam_first(d, at), lane);
        adam_update<false, 64>(x, d, adam_first(d, at), lane, consts);
    });
}

int bytes_of(int dtype) { return dtype == GS_F32 ? 4 : 2; }

// Tiles of a tensor of elements of `bytes` each, from its aligned front on.
uint32_t tiles_of(const void* p, int bytes, int64_t count, int tile) {
    return (uint32_t)(((count + head_of(p, bytes, 16 / bytes)) * bytes + tile - 1) / tile);
}
uint32_t tiles_of(const NormTensor& d, int tile) {
    const int bytes = bytes_of((int)(d.count_type >> 2) & 3);
    return tiles_of(d.g, bytes, d.count_type >> 4, tile);
}
uint32_t tiles_of(const ClipTensor& d, int tile) { return tiles_of(NormTensor{d.g, d.count_type}, tile); }
uint32_t tiles_of(const AdamTensor& d, int tile) {
    return tiles_of(d.m, sizeof(float), d.count_type >> 4, tile);
}

NormTensor norm_of(const gs_grad_tensor& d) { return {d.grad, with_types(d.count, d.dtype, 0)}; }
NormTensor norm_of_adam(const gs_adam_tensor& d) { return {d.grad, with_types(d.count, d.grad_dtype, 0)}; }
ClipTensor clip_of(const gs_grad_tensor& d) { return {d.grad, d.out, with_types(d.count, d.dtype, 0)}; }
AdamTensor adam_of(const gs_adam_tensor& d) {
    return {d.param, d.grad, d.m, d.v, with_types(d.count, d.param_dtype, d.grad_dtype), d.lr,
            (float)(1.0 - (double)d.lr * (double)d.weight_decay)};
}

// Fills a launch's table from tensors[from ..) with those that are not empty
// and returns the index behind the last one taken.
template <typename D, typename S, typename F>
int fill_table(OptTable<D>& t, const S* tensors, int from, int n, int tile, F make) {
    uint32_t tiles = 0;
    t.n = 0;
    int i = from;
    for (; i < n && t.n < OptTable<D>::kMost; ++i) {
        if (tensors[i].count == 0) continue;
        t.tensor[t.n] = make(tensors[i]);
        tiles += tiles_of(t.tensor[t.n], tile);
        t.ends[t.n++] = tiles;
    }
    return i;
}

// First pass over the whole list; gives the number of partials.
template <typename S, typename F>
hipError_t launch_partials(const S* tensors, int n, OptScratch* s, int kind, const int64_t* step, double beta1,
                           double beta2, int* slots, F make, hipStream_t stream) {
    *slots = 0;
    int taken = 0;
    for (int i = 0; i < n; ++i) taken += tensors[i].count > 0;
    const int launches = std::max(1, (taken + OptTable<NormTensor>::kMost - 1) / OptTable<NormTensor>::kMost);
    const uint64_t share = std::min(kNormBlocks, kOptSlots / launches);
    for (int i = 0; i < n;) {
        OptTable<NormTensor> t;
        i = fill_table(t, tensors, i, n, kNormTile, make);
        const uint64_t tiles = tiles_in(t);
        if (!tiles) continue;
        const uint64_t needed = (tiles * kOptThreads + kNormThreads - 1) / kNormThreads;
        const int blocks = (int)std::min(needed, share);
        k_norm_partial<<<blocks, kNormThreads, 0, stream>>>(t, s, *slots, kind, *slots ? nullptr : step, beta1, beta2);
        *slots += blocks;
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

template <typename S>
bool is_small(const S* tensors, int n, int most, int64_t most_elements) {
    int64_t elements = 0, taken = 0;
    for (int i = 0; i < n; ++i) {
        elements += tensors[i].count;
        taken += tensors[i].count > 0;
        if (elements > most_elements || taken > most) return false;
    }
    return taken > 0;
}

// Where the launches of a second pass begin in the list, first to last.
template <typename D, typename S>
int launch_starts(const S* tensors, int n, int* starts) {
    int launches = 0, taken = 0;
    for (int i = 0; i < n; ++i) {
        if (!tensors[i].count) continue;
        if (taken++ % OptTable<D>::kMost == 0) starts[launches++] = i;
    }
    return launches;
}
template <typename D>
constexpr int kMostLaunches = (GS_MAX_TENSORS + OptTable<D>::kMost - 1) / OptTable<D>::kMost;
// A launch's tiles, and one stride past them, are counted in 32 bits.
template <typename D>
constexpr bool tiles_fit(int tile) {
    return (GS_MAX_TENSOR_COUNT * 4 / tile + 1) * OptTable<D>::kMost + kOptBlocks < (int64_t)1 << 32;
}
static_assert(tiles_fit<NormTensor>(kNormTile) && tiles_fit<ClipTensor>(kClipTile) && tiles_fit<AdamTensor>(kAdamTile),
              "tile counts");
static_assert(kMostLaunches<NormTensor> < kOptSlots, "every launch of the first pass has a partial");

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
    OptTable<ClipTensor> t;
    if (is_small(tensors, n, OptTable<ClipTensor>::kMost, kSmallClip)) {
        fill_table(t, tensors, 0, n, kSmallTile, clip_of);
        k_clip_small<<<1, kSmallThreads, 0, stream>>>(t, kind, max_norm, norm);
        return hipGetLastError();
    }
    OptScratch* s = (OptScratch*)scratch;
    int slots = 0;
    if (hipError_t e = launch_partials(tensors, n, s, kind, nullptr, 0.0, 0.0, &slots, norm_of, stream)) return e;
    if (!slots) {
        k_norm_total<<<1, kOptThreads, 0, stream>>>(s, 0, kind, norm);
        return hipGetLastError();
    }
    int starts[kMostLaunches<ClipTensor>];
    for (int l = launch_starts<ClipTensor>(tensors, n, starts); l--;) {
        fill_table(t, tensors, starts[l], n, kClipTile, clip_of);
        k_clip<<<std::min<uint32_t>(tiles_in(t), kOptBlocks), kOptThreads, 0, stream>>>(t, s, slots, kind, max_norm,
                                                                                        norm);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

hipError_t launch_adam_step(const gs_adam& cfg, const gs_adam_tensor* tensors, int n, int64_t* step, float* norm,
                            void* scratch, hipStream_t stream) {
    const bool want = norm || cfg.max_norm > 0.0f || (cfg.flags & GS_ADAM_SKIP_NONFINITE);
    OptTable<AdamTensor> t;
    if (is_small(tensors, n, OptTable<AdamTensor>::kMost, kSmallAdam)) {
        fill_table(t, tensors, 0, n, kSmallTile, adam_of);
        k_adam_small<<<1, kSmallThreads, 0, stream>>>(t, cfg, want, step, norm);
        return hipGetLastError();
    }
    OptScratch* s = (OptScratch*)scratch;
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
    // the last launch takes the new step count; one without tensors if the list has none
    int starts[kMostLaunches<AdamTensor> + 1] = {};
    for (int l = std::max(1, launch_starts<AdamTensor>(tensors, n, starts)); l--;) {
        fill_table(t, tensors, starts[l], n, kAdamTile, adam_of);
        k_adam<<<std::max(1u, std::min<uint32_t>(tiles_in(t), kOptBlocks)), kOptThreads, 0, stream>>>(
            t, s, slots, cfg, step, norm, l == 0);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

}  // namespace gs
