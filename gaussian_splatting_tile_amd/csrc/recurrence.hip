// Gated linear recurrence h_t = a_t h_{t-1} + u_t along the steps of a
// sequence, forward and backward (include/gs.h, gs_recurrence_*).
//
// A run of steps is the affine map h -> A h + H (A the product of its gates,
// H its state from a zero start), and two runs in a row compose to another
// such map, so a sequence can be cut:
//  * A thread holds kSub = 16 steps of V neighbouring channels in registers
//    (V = 2 for 16-bit types where alignment allows: 4 bytes a lane), a wave
//    64 V channels, so every load and store is a contiguous 256-byte row.
//    Every input is read once, all loads of a thread are issued together.
//  * The waves of a workgroup cover up to kWaves * 16 = 128 steps of the
//    same channels and exchange (A, H) through LDS; a thread then walks its
//    16 steps from its true state. With few steps the waves lie side by side
//    over the channels instead.
//  * Longer sequences are chunks of 128 steps, one workgroup each, in one
//    pass: a chunk publishes (A, H) per channel as one 64-bit word and takes
//    the state in front of it from the words of the chunks before it in its
//    group of kGroup and the state behind the group before. All words of a
//    group are published without waiting for anything, so the chain that
//    has to be waited for has one link per group, and the formula does not
//    depend on which word came first: results are the same bits every time.
//    A word carries its own validity (all ones: not there yet; a NaN of that
//    pattern is stored as another one), so no fence is needed.
//  * Chunks are handed out per chain (a sequence's group of channels) by a
//    counter, in order: a workgroup waits only for chunks whose workgroups
//    have started and themselves wait only for earlier ones, so every wait
//    ends whatever the dispatch order. It is bounded all the same.
//  * The backward passes back c_t = a_t (g_t + c_{t+1}), the same kind of map
//    from the other end, C = sum over t of g_t times the gates up to t. The
//    states it needs are recomputed from the forward's checkpoints (one
//    float32 row per 128 steps), in LDS and registers as in the forward.
#include <algorithm>

#include "gs_internal.h"

namespace gs {
namespace {

constexpr int kRecChunk = GS_RECURRENCE_CHUNK;
constexpr int kSub = 16;
constexpr int kWaves = 8;
constexpr int kRecThreads = 64 * kWaves;
constexpr int kGroup = 2 * kWaves;  // chunks per group: each wave fetches two words
static_assert(kRecChunk == kSub * kWaves, "a chunk is one workgroup's steps");

constexpr uint32_t kDropped = 0x80000000u;  // A of a run in which the state is dropped (a restart)

// Geometry of a launch and its workspace.
struct RecShape {
    int chunks;     // K
    int groups;     // of kGroup chunks
    int columns;    // groups of 64 V channels
    int steps_log2; // waves of a workgroup along the steps (1 << steps_log2)
    uint32_t* ticket;  // [batch * columns], all ones: none taken
    uint64_t* word;    // [batch][K][channels] (A, H) or (A, C) of a chunk
    uint32_t* state;   // [batch][groups][channels] state behind a group
};

template <typename T, int V>
struct Lanes;
template <>
struct Lanes<float, 1> {
    static __device__ __forceinline__ uint32_t load(const void* p, uint32_t i) { return ((const uint32_t*)p)[i]; }
    static __device__ __forceinline__ float get(uint32_t r, int) { return __uint_as_float(r); }
    static __device__ __forceinline__ void store(void* p, uint32_t i, const float (&v)[1]) { ((float*)p)[i] = v[0]; }
};
template <typename T>
struct Lanes<T, 1> {
    static __device__ __forceinline__ uint32_t load(const void* p, uint32_t i) { return ((const uint16_t*)p)[i]; }
    static __device__ __forceinline__ float get(uint32_t r, int) { return (float)__builtin_bit_cast(T, (uint16_t)r); }
    static __device__ __forceinline__ void store(void* p, uint32_t i, const float (&v)[1]) { ((T*)p)[i] = (T)v[0]; }
};
template <typename T>
struct Lanes<T, 2> {
    static __device__ __forceinline__ uint32_t load(const void* p, uint32_t i) {
        return *(const uint32_t*)((const uint16_t*)p + i);
    }
    static __device__ __forceinline__ float get(uint32_t r, int j) {
        return (float)__builtin_bit_cast(T, (uint16_t)(j ? r >> 16 : r));
    }
    static __device__ __forceinline__ void store(void* p, uint32_t i, const float (&v)[2]) {
        typedef T Pair __attribute__((ext_vector_type(2)));
        *(Pair*)((T*)p + i) = Pair{(T)v[0], (T)v[1]};
    }
};

// sigmoid(z) and 1 - sigmoid(z), each without cancellation: with e = exp(-z)
// kept below the largest float they are 1 / (1 + e) and e / (1 + e). The
// hardware's exponential and reciprocal are within an ulp; the product
// z log2(e) adds a relative |z| 2^-24.
__device__ __forceinline__ void sigmoids(float z, float& a, float& rest) {
    const float e = fminf(__builtin_amdgcn_exp2f(z * -1.44269504f), 1e38f);
    a = __builtin_amdgcn_rcpf(1.0f + e);
    rest = e * a;
}

template <bool SIGMOID>
__device__ __forceinline__ void step_terms(float gate, float x, float& a, float& u, float& rest) {
    if (SIGMOID) {
        sigmoids(gate, a, rest);
        u = rest * x;
    } else {
        a = gate;
        u = x;
        rest = 1.0f;
    }
}

// The terms of row i; one that is not there leaves the state as it is.
template <typename T, int V, bool SIGMOID, bool FULL>
__device__ __forceinline__ void row_terms(const uint32_t (&gate)[kSub], const uint32_t (&x)[kSub], int i, int v,
                                          int rows, float& a, float& u, float& rest) {
    step_terms<SIGMOID>(Lanes<T, V>::get(gate[i], v), Lanes<T, V>::get(x[i], v), a, u, rest);
    if (!FULL && i >= rows) {
        a = 1.0f;
        u = 0.0f;
    }
}

template <typename T, int V, bool FULL>
__device__ __forceinline__ float row_grad(const uint32_t (&g)[kSub], int i, int v, int rows) {
    return FULL || i < rows ? Lanes<T, V>::get(g[i], v) : 0.0f;
}

// The map h -> A h + H of a run of steps. A state of exactly 0 gives H even
// where A overflowed, and a dropped state leaves no trace whatever it was.
struct Run {
    float A, H;
};
__device__ __forceinline__ float apply(const Run& f, float h) {
    return __float_as_uint(f.A) == kDropped || h == 0.0f ? f.H : fmaf(f.A, h, f.H);
}
// f and then g. A natural product of -0 becomes +0: that pattern is kDropped.
__device__ __forceinline__ Run then(const Run& f, const Run& g) {
    const bool dropped = __float_as_uint(f.A) == kDropped || __float_as_uint(g.A) == kDropped;
    return {dropped ? __uint_as_float(kDropped) : f.A * g.A + 0.0f, apply(g, f.H)};
}

constexpr uint32_t kNaN = 0x7fc00000u;
constexpr int kMostPolls = 1 << 22;  // seconds; see above: no wait is expected to reach it

__device__ __forceinline__ void publish(uint64_t* p, const Run& f) {
    uint64_t w = (uint64_t)__float_as_uint(f.H) << 32 | __float_as_uint(f.A);
    if (w == ~0ull) w = (uint64_t)kNaN << 32 | kNaN;
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Run await(const uint64_t* p) {
    uint64_t w = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int polls = 0; w == ~0ull && polls < kMostPolls; ++polls) {
        __builtin_amdgcn_s_sleep(1);
        w = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    return {__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}
__device__ __forceinline__ void publish(uint32_t* p, float h) {
    const uint32_t w = __float_as_uint(h);
    __hip_atomic_store(p, w == ~0u ? kNaN : w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float await(const uint32_t* p) {
    uint32_t w = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int polls = 0; w == ~0u && polls < kMostPolls; ++polls) {
        __builtin_amdgcn_s_sleep(1);
        w = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    return __uint_as_float(w);
}

// Where a wave works. All but `at` are the same in every lane.
template <int V>
struct Place {
    int wave, row;       // wave in the workgroup, wave along the steps
    int waves;           // along the steps
    int first;           // first wave of the same channels
    int b, pos;          // sequence; the chunk's place in its chain
    int len;
    int64_t c0;          // first channel of the wave
    uint32_t at;         // this lane's first channel behind c0 (the last ones again behind the end)
    bool mine;           // whether this lane has channels of its own (else it stores nothing)

    __device__ __forceinline__ Place(const RecurrenceArgs& r, const RecShape& s, int* shared_pos) {
        const int lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        waves = 1 << s.steps_log2;
        row = wave & (waves - 1);
        first = wave - row;
        int column;
        if (s.chunks > 1) {
            const unsigned chains = (unsigned)r.batch * s.columns, chain = blockIdx.x % chains;
            if (threadIdx.x == 0)
                *shared_pos = (int)(__hip_atomic_fetch_add(&s.ticket[chain], 1u, __ATOMIC_RELAXED,
                                                           __HIP_MEMORY_SCOPE_AGENT) + 1u);
            __syncthreads();
            pos = __builtin_amdgcn_readfirstlane(*shared_pos);
            b = chain / s.columns;
            column = chain % s.columns;
        } else {
            const int across = kWaves >> s.steps_log2, blocks = (s.columns + across - 1) / across;
            pos = 0;
            b = blockIdx.x / blocks;
            column = (blockIdx.x % blocks) * across + (wave >> s.steps_log2);
        }
        const bool there = column < s.columns;
        c0 = (int64_t)min(column, s.columns - 1) * (64 * V);
        const int left = (int)(r.channels - c0);  // channels from c0 on, >= 1 (a multiple of V)
        mine = there && lane * V < left;
        at = (uint32_t)min(lane * V, left - V);
        len = r.lengths ? min(max(r.lengths[b], 0), r.steps) : r.steps;
    }
};

// Bits of the steps row0 .. row0 + 15 below len that restart.
__device__ __forceinline__ uint32_t restarts(const RecurrenceArgs& r, int b, int row0, int len) {
    if (!r.restart) return 0u;
    const int i = threadIdx.x & 63;
    const bool set = i < kSub && row0 + i < len && r.restart[(int64_t)b * r.steps + row0 + i];
    return (uint32_t)__ballot(set);
}

// Lets the compiler believe that the packed rows changed, so that it computes
// their terms again where they are used rather than keep them in registers.
__device__ __forceinline__ void forget(uint32_t (&rows)[kSub]) {
#pragma unroll
    for (int i = 0; i < kSub; ++i) asm volatile("" : "+v"(rows[i]));
}

// v, or +0 if step i restarts (whatever v was); ... if any step up to i does.
__device__ __forceinline__ float unless_at(float v, uint32_t cut, int i) {
    return __uint_as_float(__float_as_uint(v) & ~(uint32_t)((int32_t)(cut << (31 - i)) >> 31));
}
__device__ __forceinline__ float unless_before(float v, uint32_t cut, int i) {
    return __uint_as_float(__float_as_uint(v) & (cut & ((2u << i) - 1) ? 0u : ~0u));
}

template <typename T>
__device__ __forceinline__ const void* step_ptr(const void* p, int64_t offset) {
    return (const T*)p + offset;
}
template <typename T>
__device__ __forceinline__ void* step_ptr(void* p, int64_t offset) {
    return (T*)p + offset;
}

// Loads the wave's rows of one tensor of a sequence whose first element is
// at `base`. Rows that are not there (unless FULL) repeat the last step that
// is, or step 0 of an empty sequence: no branch, and nothing out of bounds.
template <typename T, int V, bool FULL>
__device__ __forceinline__ void load_rows(uint32_t (&out)[kSub], const void* p, int64_t base, int64_t step, int row0,
                                          int len, uint32_t at) {
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
        const int t = FULL ? row0 + i : max(0, min(row0 + i, len - 1));
        out[i] = Lanes<T, V>::load(step_ptr<T>(p, base + t * step), at);
    }
}

// Zeroes rows [from, to) of a [T][channels] output of a sequence.
template <typename T, int V>
__device__ __forceinline__ void zero_rows(void* p, int64_t base, int64_t channels, int from, int to, uint32_t at) {
    const float zero[V] = {};
    for (int t = from; t < to; ++t) Lanes<T, V>::store(step_ptr<T>(p, base + t * channels), at, zero);
}

// LDS of a workgroup: one run per wave and channel, the runs of pairs of
// earlier chunks, and the state (or gradient) that enters the group.
template <int V>
struct RecLds {
    Run wave[kWaves][64 * V];
    Run pair[kWaves][64 * V];
    float enter[64 * V];
    int pos;
};

// Fetches what enters the chunk at p.pos: leaves the pairs of words before it
// in the group, and the state behind the group before, in LDS. Ends with a
// barrier; returns the number of pairs.
template <int V>
__device__ __forceinline__ int gather(RecLds<V>& lds, const RecurrenceArgs& r, const RecShape& s, const Place<V>& p) {
    const int lane = threadIdx.x & 63, g = p.pos / kGroup, j = p.pos % kGroup;
    const int64_t D = r.channels, c = p.c0 + p.at;
    const int k = 2 * p.wave;
    if (k < j) {
        const uint64_t* w = s.word + ((int64_t)p.b * s.chunks + (g * kGroup + k)) * D + c;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Run f = await(w + v);
            if (k + 1 < j) f = then(f, await(w + D + v));
            lds.pair[p.wave][lane * V + v] = f;
        }
    }
    if (p.wave == kWaves - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            lds.enter[lane * V + v] = g ? await(s.state + ((int64_t)p.b * s.groups + g - 1) * D + c + v) : 0.0f;
    }
    __syncthreads();
    return (j + 1) / 2;
}

// The state that enters the chunk.
template <int V>
__device__ __forceinline__ float entering(const RecLds<V>& lds, int pairs, int i) {
    float h = lds.enter[i];
    for (int w = 0; w < pairs; ++w) h = apply(lds.pair[w][i], h);
    return h;
}

// Wave 0 publishes the chunk's own run f as its word.
template <int V>
__device__ __forceinline__ void publish_chunk(const RecurrenceArgs& r, const RecShape& s, const Place<V>& p,
                                              const Run (&f)[V]) {
    uint64_t* w = s.word + ((int64_t)p.b * s.chunks + p.pos) * r.channels + p.c0 + p.at;
#pragma unroll
    for (int v = 0; v < V; ++v) publish(w + v, f[v]);
}
// ... and, for the last chunk of a group, the state behind it.
template <int V>
__device__ __forceinline__ void publish_group(const RecurrenceArgs& r, const RecShape& s, const Place<V>& p,
                                              const Run (&f)[V], const float (&h)[V]) {
    uint32_t* w = s.state + ((int64_t)p.b * s.groups + p.pos / kGroup) * r.channels + p.c0 + p.at;
#pragma unroll
    for (int v = 0; v < V; ++v) publish(w + v, apply(f[v], h[v]));
}

template <typename T, int V, bool SIGMOID, bool FULL>
__device__ __forceinline__ void forward(const RecurrenceArgs& r, const RecShape& s, RecLds<V>& lds, const Place<V>& p) {
    const int lane = threadIdx.x & 63;
    const int64_t D = r.channels;
    const int t0 = p.pos * kRecChunk, row0 = t0 + p.row * kSub;
    const int64_t out0 = (int64_t)p.b * r.steps * D + p.c0, state0 = (int64_t)p.b * D + p.c0 + p.at;
    const int rows = FULL ? kSub : max(0, min(p.len - row0, kSub));
    const bool starts = p.pos == 0 && p.row == 0;
    float a[kSub][V], u[kSub][V], h0[V];
    uint32_t cut;
    {
        uint32_t gate[kSub], x[kSub];
        load_rows<T, V, FULL>(gate, r.gate, p.b * r.gate_batch + p.c0, r.gate_step, row0, p.len, p.at);
        load_rows<T, V, FULL>(x, r.x, p.b * r.x_batch + p.c0, r.x_step, row0, p.len, p.at);
#pragma unroll
        for (int v = 0; v < V; ++v) h0[v] = starts && r.h0 ? r.h0[state0 + v] : 0.0f;
        cut = restarts(r, p.b, row0, p.len);
#pragma unroll
        for (int i = 0; i < kSub; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float rest;
                row_terms<T, V, SIGMOID, FULL>(gate, x, i, v, rows, a[i][v], u[i][v], rest);
                a[i][v] = unless_at(a[i][v], cut, i);
            }
    }
    Run own[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        own[v] = {1.0f, h0[v]};
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
            own[v].A *= a[i][v];
            own[v].H = fmaf(a[i][v], unless_at(own[v].H, cut, i), u[i][v]);
        }
        own[v].A = cut ? __uint_as_float(kDropped) : own[v].A + 0.0f;
        lds.wave[p.wave][lane * V + v] = own[v];
    }
    __syncthreads();
    Run chunk[V];
    const bool followed = t0 + kRecChunk < p.len;
    if (followed && p.wave == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            chunk[v] = own[v];
            for (int w = 1; w < kWaves; ++w) chunk[v] = then(chunk[v], lds.wave[w][lane * V + v]);
        }
        if (p.mine) publish_chunk<V>(r, s, p, chunk);
    }
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.0f;
    if (p.pos) {
        const int pairs = gather<V>(lds, r, s, p);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = entering<V>(lds, pairs, lane * V + v);
        if (p.wave == 0 && p.mine && r.ckpt) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                r.ckpt[((int64_t)p.b * (s.chunks - 1) + p.pos - 1) * D + p.c0 + p.at + v] = h[v];
        }
    }
    if (followed && p.wave == 0 && p.mine && p.pos % kGroup == kGroup - 1) publish_group<V>(r, s, p, chunk, h);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (starts) h[v] = h0[v];
        for (int w = p.first; w < p.wave; ++w) h[v] = apply(lds.wave[w][lane * V + v], h[v]);
    }
    if (!p.mine) return;
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(a[i][v], unless_at(h[v], cut, i), u[i][v]);
        if (FULL || i < rows) Lanes<T, V>::store(step_ptr<T>(r.h, out0 + (row0 + i) * D), p.at, h);
    }
    if (!FULL) zero_rows<T, V>(r.h, out0, D, row0 + rows, min(row0 + kSub, r.steps), p.at);
    // the wave with the last step, or the first one of an empty sequence
    if (r.h_last && (rows ? row0 + rows == p.len : starts && p.len == 0)) {
#pragma unroll
        for (int v = 0; v < V; ++v) r.h_last[state0 + v] = h[v];
    }
}

template <typename T, int V, bool SIGMOID>
__global__ __launch_bounds__(kRecThreads, 4) void k_recurrence_fwd(RecurrenceArgs r, RecShape s) {
    __shared__ RecLds<V> lds;
    const Place<V> p(r, s, &lds.pos);
    const int t0 = p.pos * kRecChunk, row0 = t0 + p.row * kSub;
    if (t0 + p.waves * kSub <= p.len)
        forward<T, V, SIGMOID, true>(r, s, lds, p);
    else if (t0 < p.len || p.pos == 0)
        forward<T, V, SIGMOID, false>(r, s, lds, p);
    else if (p.mine)  // padding
        zero_rows<T, V>(r.h, (int64_t)p.b * r.steps * r.channels + p.c0, r.channels, row0, min(row0 + kSub, r.steps),
                        p.at);
}

template <typename T, int V, bool SIGMOID, bool FULL>
__device__ __forceinline__ void backward(const RecurrenceArgs& r, const RecShape& s, RecLds<V>& lds,
                                         float (&wave_c)[kWaves][64 * V], const Place<V>& p, int k) {
    const int lane = threadIdx.x & 63;
    const int64_t D = r.channels;
    const int t0 = k * kRecChunk, row0 = t0 + p.row * kSub;
    const int64_t out0 = (int64_t)p.b * r.steps * D + p.c0, state0 = (int64_t)p.b * D + p.c0 + p.at;
    const bool starts = k == 0 && p.row == 0;
    const int rows = FULL ? kSub : max(0, min(p.len - row0, kSub));
    uint32_t gate[kSub], x[kSub], g[kSub];
    load_rows<T, V, FULL>(gate, r.gate, p.b * r.gate_batch + p.c0, r.gate_step, row0, p.len, p.at);
    load_rows<T, V, FULL>(x, r.x, p.b * r.x_batch + p.c0, r.x_step, row0, p.len, p.at);
    load_rows<T, V, FULL>(g, r.grad_h, out0, D, row0, p.len, p.at);
    const bool ends = rows ? row0 + rows == p.len : starts && p.len == 0;  // has the last step
    float h[V], last[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = k ? r.ckpt_in[((int64_t)p.b * (s.chunks - 1) + k - 1) * D + p.c0 + p.at + v]
                 : r.h0 ? r.h0[state0 + v] : 0.0f;
        last[v] = ends && r.grad_last ? r.grad_last[state0 + v] : 0.0f;
    }
    const uint32_t cut = restarts(r, p.b, row0, p.len);

    // the wave's run of the states, (A, H), and of what it passes back, (A, C)
    Run own[V];
    float C[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        own[v] = {1.0f, 0.0f};
        C[v] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a, u, rest;
            row_terms<T, V, SIGMOID, FULL>(gate, x, i, v, rows, a, u, rest);
            own[v].H = fmaf(unless_at(a, cut, i), unless_at(own[v].H, cut, i), u);
            // steps from a restart on pass nothing back in front of it
            own[v].A = unless_before(own[v].A * a, cut, i);
            C[v] = fmaf(own[v].A, unless_before(row_grad<T, V, FULL>(g, i, v, rows), cut, i), C[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (!cut) C[v] = fmaf(own[v].A, last[v], C[v]);
        own[v].A = cut ? __uint_as_float(kDropped) : own[v].A + 0.0f;
        lds.wave[p.wave][lane * V + v] = own[v];
        wave_c[p.wave][lane * V + v] = C[v];
    }
    __syncthreads();

    Run chunk[V];
    const bool followed = k > 0;
    if (followed && p.wave == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = lane * V + v;
            chunk[v] = {lds.wave[kWaves - 1][i].A, wave_c[kWaves - 1][i]};
            for (int w = kWaves - 2; w >= 0; --w) chunk[v] = then(chunk[v], Run{lds.wave[w][i].A, wave_c[w][i]});
        }
        if (p.mine) publish_chunk<V>(r, s, p, chunk);
    }
    // the states in front of the wave's steps
    forget(gate);
    forget(x);
    float prev[kSub][V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        for (int w = p.first; w < p.wave; ++w) h[v] = apply(lds.wave[w][lane * V + v], h[v]);
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a, u, rest;
            row_terms<T, V, SIGMOID, FULL>(gate, x, i, v, rows, a, u, rest);
            prev[i][v] = unless_at(h[v], cut, i);
            h[v] = fmaf(unless_at(a, cut, i), prev[i][v], u);
        }
    }
    forget(gate);
    forget(x);
    // what the steps behind the wave's pass back
    float c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = 0.0f;
    if (p.pos) {
        const int pairs = gather<V>(lds, r, s, p);
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = entering<V>(lds, pairs, lane * V + v);
    }
    if (followed && p.wave == 0 && p.mine && p.pos % kGroup == kGroup - 1) publish_group<V>(r, s, p, chunk, c);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = lane * V + v;
        for (int w = p.first + p.waves - 1; w > p.wave; --w) c[v] = apply(Run{lds.wave[w][i].A, wave_c[w][i]}, c[v]);
        c[v] += last[v];
    }
    if (!p.mine) return;
#pragma unroll
    for (int i = kSub - 1; i >= 0; --i) {
        float dg[V], dx[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a, u, rest;
            row_terms<T, V, SIGMOID, FULL>(gate, x, i, v, rows, a, u, rest);
            const float d = row_grad<T, V, FULL>(g, i, v, rows) + c[v], xi = Lanes<T, V>::get(x[i], v);
            dg[v] = SIGMOID ? d * (prev[i][v] - xi) * (a * rest) : d * prev[i][v];
            dx[v] = SIGMOID ? d * rest : d;
            c[v] = unless_at(a * d, cut, i);
        }
        if (FULL || i < rows) {
            Lanes<T, V>::store(step_ptr<T>(r.grad_gate, out0 + (row0 + i) * D), p.at, dg);
            Lanes<T, V>::store(step_ptr<T>(r.grad_x, out0 + (row0 + i) * D), p.at, dx);
        }
    }
    if (!FULL) {
        zero_rows<T, V>(r.grad_gate, out0, D, row0 + rows, min(row0 + kSub, r.steps), p.at);
        zero_rows<T, V>(r.grad_x, out0, D, row0 + rows, min(row0 + kSub, r.steps), p.at);
    }
    if (r.grad_h0 && starts) {
#pragma unroll
        for (int v = 0; v < V; ++v) r.grad_h0[state0 + v] = c[v];
    }
}

template <typename T, int V, bool SIGMOID>
__global__ __launch_bounds__(kRecThreads, 4) void k_recurrence_bwd(RecurrenceArgs r, RecShape s) {
    __shared__ RecLds<V> lds;
    __shared__ float wave_c[kWaves][64 * V];
    const Place<V> p(r, s, &lds.pos);
    const int used = (p.len + kRecChunk - 1) / kRecChunk;  // chunks with steps: taken from the last on
    const int k = p.pos < used ? used - 1 - p.pos : p.pos;
    const int t0 = k * kRecChunk, row0 = t0 + p.row * kSub;
    if (t0 + p.waves * kSub <= p.len) {
        backward<T, V, SIGMOID, true>(r, s, lds, wave_c, p, k);
    } else if (t0 < p.len || k == 0) {
        backward<T, V, SIGMOID, false>(r, s, lds, wave_c, p, k);
    } else if (p.mine) {  // padding
        const int64_t out0 = (int64_t)p.b * r.steps * r.channels + p.c0;
        zero_rows<T, V>(r.grad_gate, out0, r.channels, row0, min(row0 + kSub, r.steps), p.at);
        zero_rows<T, V>(r.grad_x, out0, r.channels, row0, min(row0 + kSub, r.steps), p.at);
    }
}

// No steps at all: the state, or its gradient, passes through.
__global__ void k_recurrence_pass(const float* from, float* to, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * kRecThreads + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : 0.0f;
}

int chunks_of(int steps) { return std::max(1, (int)(((int64_t)steps + kRecChunk - 1) / kRecChunk)); }

size_t layout(int batch, int steps, int channels, int columns, RecShape* s, void* base) {
    s->chunks = chunks_of(steps);
    s->groups = (s->chunks + kGroup - 1) / kGroup;
    s->columns = columns;
    s->steps_log2 = 0;
    while ((kSub << s->steps_log2) < std::min(steps, kRecChunk)) ++s->steps_log2;
    s->ticket = nullptr;
    s->word = nullptr;
    s->state = nullptr;
    if (s->chunks == 1) return 0;
    const size_t words = (size_t)batch * s->chunks * channels, states = (size_t)batch * s->groups * channels;
    s->word = (uint64_t*)base;
    s->state = (uint32_t*)(s->word + words);
    s->ticket = s->state + states;
    return words * 8 + (states + (size_t)batch * columns) * 4;
}

template <typename T, int V, bool SIGMOID>
hipError_t launch_of(const RecurrenceArgs& r, bool backward, void* scratch, hipStream_t stream) {
    RecShape s;
    const size_t bytes = layout(r.batch, r.steps, r.channels, (r.channels + 64 * V - 1) / (64 * V), &s, scratch);
    int64_t blocks = (int64_t)r.batch * s.columns * s.chunks;
    if (s.chunks == 1) {
        const int across = kWaves >> s.steps_log2;
        blocks = (int64_t)r.batch * ((s.columns + across - 1) / across);
    } else if (hipError_t e = launch_fill_u32((uint32_t*)scratch, bytes / 4, ~0u, stream)) {
        return e;
    }
    if (backward)
        k_recurrence_bwd<T, V, SIGMOID><<<(unsigned)blocks, kRecThreads, 0, stream>>>(r, s);
    else
        k_recurrence_fwd<T, V, SIGMOID><<<(unsigned)blocks, kRecThreads, 0, stream>>>(r, s);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t launch_of(const RecurrenceArgs& r, bool sigmoid, bool backward, void* scratch, hipStream_t stream) {
    return sigmoid ? launch_of<T, V, true>(r, backward, scratch, stream)
                   : launch_of<T, V, false>(r, backward, scratch, stream);
}

// Two 16-bit channels a lane need every row of every tensor on a 4-byte boundary.
bool pairs_fit(const RecurrenceArgs& r) {
    const uintptr_t p = (uintptr_t)r.gate | (uintptr_t)r.x | (uintptr_t)r.h | (uintptr_t)r.grad_h |
                        (uintptr_t)r.grad_gate | (uintptr_t)r.grad_x;
    const int64_t n = r.channels | r.gate_batch | r.gate_step | r.x_batch | r.x_step;
    return !(p & 3) && !(n & 1);
}

hipError_t launch(const RecurrenceArgs& r, int dtype, bool sigmoid, bool backward, void* scratch, hipStream_t stream) {
    if (r.steps == 0) {
        const float* from = backward ? r.grad_last : r.h0;
        float* to = backward ? r.grad_h0 : r.h_last;
        const int64_t n = (int64_t)r.batch * r.channels;
        if (!to || to == from) return hipSuccess;
        k_recurrence_pass<<<(unsigned)((n + kRecThreads - 1) / kRecThreads), kRecThreads, 0, stream>>>(from, to, n);
        return hipGetLastError();
    }
    if (dtype == GS_F32) return launch_of<float, 1>(r, sigmoid, backward, scratch, stream);
    if (dtype == GS_BF16)
        return pairs_fit(r) ? launch_of<__bf16, 2>(r, sigmoid, backward, scratch, stream)
                            : launch_of<__bf16, 1>(r, sigmoid, backward, scratch, stream);
    return pairs_fit(r) ? launch_of<_Float16, 2>(r, sigmoid, backward, scratch, stream)
                        : launch_of<_Float16, 1>(r, sigmoid, backward, scratch, stream);
}

}  // namespace

bool recurrence_fits(const gs_recurrence& r) {
    const int64_t most = INT32_MAX;
    const int64_t columns = ((int64_t)r.channels + 63) / 64, chains = columns * std::max(r.batch, 1);
    return chains <= most && chains * chunks_of(r.steps) <= most;
}

size_t recurrence_scratch_bytes(const gs_recurrence& r) {
    RecShape s;
    if (r.batch == 0 || r.channels == 0) return 0;
    return layout(r.batch, r.steps, r.channels, (r.channels + 63) / 64, &s, nullptr);
}

hipError_t launch_recurrence_fwd(const RecurrenceArgs& r, int dtype, bool sigmoid, void* scratch, hipStream_t stream) {
    return launch(r, dtype, sigmoid, false, scratch, stream);
}

hipError_t launch_recurrence_bwd(const RecurrenceArgs& r, int dtype, bool sigmoid, void* scratch, hipStream_t stream) {
    return launch(r, dtype, sigmoid, true, scratch, stream);
}

}  // namespace gs
