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
//    same channels and exchange (A, H) through LDS; one of them hands each
//    wave the state in front of its steps, and every thread walks its 16
//    steps from there. With few steps the waves lie side by side over the
//    channels instead.
//  * Longer sequences are chunks of 128 steps, one workgroup each, in one
//    pass: a chunk publishes (A, H) per channel as one 64-bit word, the last
//    of kGroup chunks the run of its group, and the last of kGroup groups the
//    state behind it. A chunk takes the state in front of it from the words
//    of the chunks before it in its group, of the groups before that in
//    theirs, and the state behind the super-group before: a sequence of 65536
//    steps has a chain of 8 links to wait for, where one that passes the
//    state from chunk to chunk would have 512. The formula does not depend on
//    which word came first, so results are the same bits every time. A word
//    carries its own validity (all ones: not there yet; a NaN of that pattern
//    is stored as another one), so no fence is needed.
//  * A product of gates is a float32 over at most 128 steps: a group's A, over
//    1024, can leave the range where no state does (gates that decay by 1e-28
//    and then grow by 1e42). A state that such an A would lose walks the words
//    of the group's chunks.
//  * No workgroup depends on another one's progress: one that has waited
//    kPatience polls for a word computes it from the inputs itself, by the
//    same formula (Alone, below). With workgroups started in order that never
//    happens; it makes every wait end whatever the order of dispatch, without
//    the counter that would otherwise have to hand chunks out in the order of
//    their start (8 of 110 us on 65536 x 1024 bf16, its latency in front of
//    every workgroup's loads).
//  * The backward passes back c_t = a_t (g_t + c_{t+1}), the same kind of map
//    from the other end, C = sum over t of g_t times the gates up to t. The
//    states it needs are recomputed from the forward's checkpoints (one
//    float32 row per 128 steps), in LDS and registers as in the forward.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "gs_internal.h"

namespace gs {
namespace {

constexpr int kRecChunk = GS_RECURRENCE_CHUNK;
constexpr int kSub = 16;
// Rows a thread holds where a sequence has no more (and 1 forward for T = 1):
// the rows up to kSub would be loads and steps for nothing.
constexpr int kFew = 4;
constexpr int kWaves = 8;
constexpr int kRecThreads = 64 * kWaves;
constexpr int kGroup = kWaves;  // a wave fetches one word of either level, the last one the state
static_assert(kRecChunk == kSub * kWaves, "a chunk is one workgroup's steps");

constexpr uint32_t kDropped = 0x80000000u;  // A of a run in which the state is dropped (a restart)

// Geometry of a launch and its workspace.
struct RecShape {
    int chunks;      // K
    int groups;      // of kGroup chunks
    int supers;      // of kGroup groups
    int columns;     // groups of 64 V channels
    int64_t row;     // columns * 64 V: words of a row of the workspace
    int steps_log2;  // waves of a workgroup along the steps (1 << steps_log2)
    bool lines;      // every row of every tensor is whole 128-byte lines
    uint64_t* word;    // [batch][chunks][row] (A, H) or (A, C) of a chunk
    uint64_t* group;   // [batch][groups][row] of a group
    uint32_t* state;   // [batch][supers][row] state behind a super-group; nothing is behind the
                       // last one, whose row holds a copy of h0 if h_last is to replace it
    int patience;      // polls; 0: waits for nothing and computes every word itself
};

// A lane's V channels of one row, packed in 32 bits. Rows can go past the
// caches (PAST): nothing is read twice, and the pure copy of a sequence's rows
// reaches 3.7 TB/s without it and 5.6 with it (65536 x 1024 bf16, two in, one
// out). That holds for rows that are whole 128-byte lines: others share lines
// with their neighbours, and are read the common way (8 x 2048 x 2047 float32
// forward 145 us past the caches, 92 through them). A wave's rows of single
// 16-bit channels are one line, read the common way always (16 x 2048 x 1024
// bf16 backward 74 us past the caches, 54 through them) and written past them
// if they are whole lines (54 and 66 us; 16 x 2049 x 1025: 115 and 98).
template <typename T, int V>
struct Lanes;
template <>
struct Lanes<float, 1> {
    template <bool PAST>
    static __device__ __forceinline__ uint32_t load(const float* p, uint32_t i) {
        const uint32_t* const q = (const uint32_t*)p + i;
        return PAST ? __builtin_nontemporal_load(q) : *q;
    }
    static __device__ __forceinline__ float get(uint32_t r, int) { return __uint_as_float(r); }
    template <bool PAST>
    static __device__ __forceinline__ void store(float* p, uint32_t i, const float (&v)[1]) {
        __builtin_nontemporal_store(v[0], p + i);
    }
};
template <typename T>
struct Lanes<T, 1> {
    template <bool PAST>
    static __device__ __forceinline__ uint32_t load(const T* p, uint32_t i) {
        return ((const uint16_t*)p)[i];
    }
    static __device__ __forceinline__ float get(uint32_t r, int) { return (float)__builtin_bit_cast(T, (uint16_t)r); }
    template <bool PAST>
    static __device__ __forceinline__ void store(T* p, uint32_t i, const float (&v)[1]) {
        if (PAST)
            __builtin_nontemporal_store((T)v[0], p + i);
        else
            p[i] = (T)v[0];
    }
};
template <typename T>
struct Lanes<T, 2> {
    template <bool PAST>
    static __device__ __forceinline__ uint32_t load(const T* p, uint32_t i) {
        const uint32_t* const q = (const uint32_t*)(p + i);
        return PAST ? __builtin_nontemporal_load(q) : *q;
    }
    static __device__ __forceinline__ float get(uint32_t r, int j) {
        return (float)__builtin_bit_cast(T, (uint16_t)(j ? r >> 16 : r));
    }
    template <bool PAST>
    static __device__ __forceinline__ void store(T* p, uint32_t i, const float (&v)[2]) {
        typedef T Pair __attribute__((ext_vector_type(2)));
        const Pair r = {(T)v[0], (T)v[1]};
        __builtin_nontemporal_store(r, (Pair*)(p + i));
    }
};

// sigmoid(z) and 1 - sigmoid(z), each without cancellation: with e = exp(-z)
// they are 1 / (1 + e) and e / (1 + e). The hardware's exponential and
// reciprocal are within an ulp; the product z log2(e) adds a relative |z| 2^-24.
// Results below 2^-126 are flushed to 0 by both. For z below -86.6 that (or an
// e of infinity) leaves e times the reciprocal far from 1, so its factors stop
// at 2^125 and 2^-125: the second value is then 1, and the first is on its way
// to 0 unhindered (z = -inf is a complete forget). The maximum passes a NaN; a
// plain one would drop it, and a diverged gate with it.
__device__ __forceinline__ float exp_minus(float z) { return __builtin_amdgcn_exp2f(z * -1.44269504f); }
__device__ __forceinline__ void of_exp_minus(float e, float& a, float& rest) {
    a = __builtin_amdgcn_rcpf(1.0f + e);
    rest = fminf(e, 0x1p125f) * __builtin_elementwise_maximum(a, 0x1p-125f);
}
__device__ __forceinline__ void sigmoids(float z, float& a, float& rest) { of_exp_minus(exp_minus(z), a, rest); }

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
template <typename T, int V, bool SIGMOID, bool FULL, int SUB>
__device__ __forceinline__ void row_terms(const uint32_t (&gate)[SUB], const uint32_t (&x)[SUB], int i, int v,
                                          int rows, float& a, float& u, float& rest) {
    step_terms<SIGMOID>(Lanes<T, V>::get(gate[i], v), Lanes<T, V>::get(x[i], v), a, u, rest);
    if (!FULL && i >= rows) {
        a = 1.0f;
        u = 0.0f;
    }
}

template <typename T, int V, bool FULL, int SUB>
__device__ __forceinline__ float row_grad(const uint32_t (&g)[SUB], int i, int v, int rows) {
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
// A group's run, from its chunks' in turn. Its A is a product over 1024 steps,
// eight floats: in float64 none of the products between leaves the range.
struct GroupRun {
    double A;
    float H;
    bool dropped;
    __device__ __forceinline__ GroupRun(const Run& f)
        : A(f.A), H(f.H), dropped(__float_as_uint(f.A) == kDropped) {}
    __device__ __forceinline__ void then(const Run& g) {
        A *= (double)g.A;
        H = apply(g, H);
        dropped |= __float_as_uint(g.A) == kDropped;
    }
    __device__ __forceinline__ Run run() const { return {dropped ? __uint_as_float(kDropped) : (float)A + 0.0f, H}; }
};
// Whether a group's A left float32's range and says too little about what is
// left of a state h in front: A is infinite (or NaN), or below the normal
// numbers and its error, up to 2^-150, times h reaches both 2^-126 and the last
// bit of H. The group's chunks are walked then. (Over 1024 steps A is 0 for most
// forgetting gates; walking always takes 65536 x 1024 bf16 from 101 to 240 us.)
constexpr float kLarge = 0x1p24f;
__device__ __forceinline__ bool too_long(const Run& f, float h) {
    const float a = fabsf(f.A), m = fabsf(h);
    return __float_as_uint(f.A) != kDropped && h != 0.0f &&
           (!(a < __builtin_inff()) || (a < 0x1p-126f && !(m < kLarge) && !(fabsf(f.H) >= m * 0x1p-125f)));
}

constexpr uint32_t kNaN = 0x7fc00000u;
constexpr int kPatience = 1 << 14;  // polls, some 20 ms

// A word of all ones is not there yet.
template <typename W>
__device__ __forceinline__ void publish_word(W* p, W w, W nan) {
    __hip_atomic_store(p, w == (W)~(W)0 ? nan : w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W>
__device__ __forceinline__ W word_at(const W* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// w, read from p (one word a lane), if all lanes' are there; else waits, and
// at the end of its patience takes help(). One lane watches its own word until
// it is there; then all read theirs, which were stored together, and only
// lanes that came too early go on. (All lanes watching took bandwidth from
// the rows.)
template <typename W, typename F>
__device__ __forceinline__ W settle_word(const W* p, W w, int patience, F help) {
    if (patience && !__any(w == (W)~(W)0)) return w;
    int polls = 0;
    if ((threadIdx.x & 63) == 0) {
        while (polls < patience && word_at(p) == (W)~(W)0) {
            ++polls;
            __builtin_amdgcn_s_sleep(4);
        }
    }
    polls = __builtin_amdgcn_readfirstlane(polls);
    if (patience) w = word_at(p);
    while (polls < patience && __any(w == (W)~(W)0)) {
        ++polls;
        __builtin_amdgcn_s_sleep(1);
        w = word_at(p);
    }
    if (__builtin_expect(polls >= patience, 0)) w = help();
    return w;
}
__device__ __forceinline__ uint64_t word_of(const Run& f) {
    return (uint64_t)__float_as_uint(f.H) << 32 | __float_as_uint(f.A);
}
__device__ __forceinline__ Run run_of(uint64_t w) {
    return {__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}
__device__ __forceinline__ void publish(uint64_t* p, const Run& f) {
    publish_word(p, word_of(f), (uint64_t)kNaN << 32 | kNaN);
}
__device__ __forceinline__ void publish(uint32_t* p, float h) { publish_word(p, __float_as_uint(h), kNaN); }
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

    __device__ __forceinline__ Place(const RecurrenceArgs& r, const RecShape& s) {
        const int lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        waves = 1 << s.steps_log2;
        row = wave & (waves - 1);
        first = wave - row;
        int column;
        if (s.chunks > 1) {
            const unsigned chains = (unsigned)r.batch * s.columns, chain = blockIdx.x % chains;
            pos = blockIdx.x / chains;
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

// Bits of the steps row0 .. row0 + SUB - 1 below len that restart.
template <int SUB>
__device__ __forceinline__ uint32_t restarts(const RecurrenceArgs& r, int b, int row0, int len) {
    const int i = threadIdx.x & 63;
    const bool set = i < SUB && row0 + i < len && r.restart[(int64_t)b * r.steps + row0 + i];
    return (uint32_t)__ballot(set);
}

// Lets the compiler believe that the packed rows changed, so that it computes
// their terms again where they are used rather than keep them in registers.
template <int SUB>
__device__ __forceinline__ void forget(uint32_t (&rows)[SUB]) {
#pragma unroll
    for (int i = 0; i < SUB; ++i) asm volatile("" : "+v"(rows[i]));
}

// v, or +0 if step i restarts (whatever v was); ... if any step up to i does.
// Without CUT none does.
template <bool CUT>
__device__ __forceinline__ float unless_at(float v, uint32_t cut, int i) {
    return CUT ? __uint_as_float(__float_as_uint(v) & ~(uint32_t)((int32_t)(cut << (31 - i)) >> 31)) : v;
}
template <bool CUT>
__device__ __forceinline__ float unless_before(float v, uint32_t cut, int i) {
    return CUT ? __uint_as_float(__float_as_uint(v) & (cut & ((2u << i) - 1) ? 0u : ~0u)) : v;
}
// Keeps the compiler from holding every row's distance: sixteen 64-bit values a
// tensor are more than there are scalar registers. From row to row it is one
// addition.
__device__ __forceinline__ void hide(int64_t& step) { asm volatile("" : "+s"(step)); }
// Keeps the compiler from moving work across every kBlock rows: taken all
// together, the rows' terms fill the registers.
constexpr int kBlock = 4;
__device__ __forceinline__ void end_of_row(int i) {
    if (i % kBlock == kBlock - 1) __builtin_amdgcn_sched_barrier(0);
}
// Loads the wave's rows of one tensor of a sequence whose first element is
// at `base`. Rows that are not there (unless FULL) repeat the last step that
// is, or step 0 of an empty sequence: no branch, and nothing out of bounds.
template <typename T, int V, bool FULL, bool PAST, int SUB>
__device__ __forceinline__ void load_rows(uint32_t (&out)[SUB], const void* p, int64_t base, int64_t step, int row0,
                                          int len, uint32_t at) {
    const T* q = (const T*)p + base + (FULL ? row0 : max(0, min(row0, len - 1))) * step;
    hide(step);
#pragma unroll
    for (int i = 0; i < SUB; ++i) {
        out[i] = Lanes<T, V>::template load<PAST>(q, at);
        if (FULL || row0 + i + 1 < len) q += step;
    }
}

// A row of a [T][channels] output of a sequence.
template <typename T, int V>
__device__ __forceinline__ T* row_of(void* p, int64_t base, int64_t channels, int row) {
    return (T*)p + base + row * channels;
}

// Calls f(PAST) by how rows of this kind are written (see Lanes).
template <typename T, int V, typename F>
__device__ __forceinline__ void by_lines(bool lines, F f) {
    if (sizeof(T) == 2 && V == 1 && !lines) {
        f(std::false_type());
    } else {
        asm volatile("");  // else the compiler makes one way of the two, through the caches
        f(std::true_type());
    }
}

// Zeroes rows [from, to) of a [T][channels] output of a sequence.
template <typename T, int V>
__device__ __forceinline__ void zero_rows(void* p, int64_t base, int64_t channels, int from, int to, uint32_t at,
                                          bool lines) {
    const float zero[V] = {};
    by_lines<T, V>(lines, [&](auto past) {
        T* q = row_of<T, V>(p, base, channels, from);
        for (int t = from; t < to; ++t, q += channels) Lanes<T, V>::template store<past.value>(q, at, zero);
    });
}

// LDS of a workgroup: one run per wave and channel, the runs of the groups
// and chunks in front, what enters the super-group, and what enters each
// wave's steps.
template <int V>
struct RecLds {
    Run wave[kWaves][64 * V];
    Run group[kGroup - 1][64 * V];
    Run chunk[kGroup - 1][64 * V];
    float enter[64 * V];
    float start[kWaves][64 * V];
};

// The words of one channel computed from the inputs, by the steps and in the
// order in which the chunks compute them: the same bits. No thread of a launch
// whose workgroups start in order gets here.
template <typename T, bool SIGMOID, bool CUT, bool BACK>
struct Alone {
    const RecurrenceArgs& r;
    int b, len;
    int64_t c;

    __device__ Run wave(int pos, int w) const {
        const int k = BACK ? (len + kRecChunk - 1) / kRecChunk - 1 - pos : pos;
        const int row0 = k * kRecChunk + w * kSub, rows = max(0, min(len - row0, kSub));
        Run f = {1.0f, 0.0f};
        bool dropped = false;
#pragma unroll 1
        for (int i = 0; i < kSub; ++i) {
            const int t = max(0, min(row0 + i, len - 1));
            float a, u, rest, g = 0.0f;
            step_terms<SIGMOID>((float)((const T*)r.gate)[b * r.gate_batch + t * r.gate_step + c],
                                (float)((const T*)r.x)[b * r.x_batch + t * r.x_step + c], a, u, rest);
            if (BACK) g = (float)((const T*)r.grad_h)[((int64_t)b * r.steps + t) * r.channels + c];
            if (i >= rows) {
                a = 1.0f;
                u = g = 0.0f;
            }
            const bool cut = CUT && i < rows && r.restart[(int64_t)b * r.steps + t];
            dropped |= cut;
            f.A *= a;
            if (BACK) {
                if (dropped) f.A = g = 0.0f;
                f.H = fmaf(f.A, g, f.H);
            } else {
                f.H = cut ? fmaf(0.0f, 0.0f, u) : fmaf(a, f.H, u);
            }
        }
        if (BACK && !dropped) {
            const bool ends = rows && row0 + rows == len;
            f.H = fmaf(f.A, ends && r.grad_last ? r.grad_last[(int64_t)b * r.channels + c] : 0.0f, f.H);
        }
        f.A = dropped ? __uint_as_float(kDropped) : f.A + 0.0f;
        return f;
    }
    // ... of the wave that is i-th in the direction of the walk
    __device__ Run in_turn(int pos, int i) const { return wave(pos, BACK ? kWaves - 1 - i : i); }
    __device__ Run chunk(int pos) const {
        Run f = in_turn(pos, 0);
#pragma unroll 1
        for (int i = 1; i < kWaves; ++i) f = then(f, in_turn(pos, i));
        if (!BACK && pos == 0) f.H = apply(f, r.h0 ? r.h0[b * r.h0_batch + c] : 0.0f);
        return f;
    }
    __device__ Run group(int g) const {
        GroupRun f = chunk(g * kGroup);
#pragma unroll 1
        for (int j = 1; j < kGroup; ++j) f.then(chunk(g * kGroup + j));
        return f.run();
    }
    __device__ float through_group(int g, float e) const {
        const Run f = group(g);
        if (!too_long(f, e)) return apply(f, e);
#pragma unroll 1
        for (int j = 0; j < kGroup; ++j) e = apply(chunk(g * kGroup + j), e);
        return e;
    }
    __device__ float state(int sg) const {
        float e = 0.0f;
#pragma unroll 1
        for (int s = 0; s <= sg; ++s) {
            const int last = s * kGroup + kGroup - 1;  // group
#pragma unroll 1
            for (int g = s * kGroup; g < last; ++g) e = through_group(g, e);
#pragma unroll 1
            for (int j = 0; j < kGroup - 1; ++j) e = apply(chunk(last * kGroup + j), e);
#pragma unroll 1
            for (int i = 0; i < kWaves; ++i) e = apply(in_turn(last * kGroup + kGroup - 1, i), e);
        }
        return e;
    }
};

// Hands the chunk's run f on to the chunks behind (wave 0; followed: there
// are some) and fetches what the chunk's place in the chain needs. With
// pos > 0 it ends with a barrier, after which entering() can be called.
template <typename T, int V, bool SIGMOID, bool CUT, bool BACK>
__device__ __forceinline__ void exchange(RecLds<V>& lds, const RecurrenceArgs& r, const RecShape& s, const Place<V>& p,
                                         bool followed, const Run (&f)[V]) {
    const int lane = threadIdx.x & 63;
    // words lie by channel group, one row of 64 for each of a lane's V channels
    const int64_t D = (int64_t)s.columns * (64 * V), c = p.c0 + lane;
    const int g = p.pos / kGroup, j = p.pos % kGroup, sg = g / kGroup, gj = g % kGroup;
    uint64_t* const word = s.word + ((int64_t)p.b * s.chunks + g * kGroup) * D + c;
    uint64_t* const group = s.group + ((int64_t)p.b * s.groups + sg * kGroup) * D + c;
    const bool tells = followed && p.wave == 0;
    if (tells) {
#pragma unroll
        for (int v = 0; v < V; ++v) publish(word + j * D + v * 64, f[v]);
    }
    if (!p.pos) return;
    // all words at once: as a rule they are there
    const uint32_t* const state = s.state + ((int64_t)p.b * s.supers + sg - 1) * D + c;
    uint64_t near[V], far[V];
    uint32_t before[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        near[v] = p.wave < j ? word_at(word + p.wave * D + v * 64) : 0u;
        far[v] = p.wave < gj ? word_at(group + p.wave * D + v * 64) : 0u;
        before[v] = p.wave == kWaves - 1 && sg ? word_at(state + v * 64) : 0u;
    }
    if (p.wave < j) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const auto help = [&] {
                return word_of(Alone<T, SIGMOID, CUT, BACK>{r, p.b, p.len, p.c0 + p.at + v}.chunk(g * kGroup + p.wave));
            };
            lds.chunk[p.wave][lane * V + v] =
                run_of(settle_word(word + p.wave * D + v * 64, near[v], s.patience, help));
        }
    }
    if (j == kGroup - 1) {  // the group's run, before anything of earlier groups is waited for
        __syncthreads();
        if (tells) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = lane * V + v;
                GroupRun all = lds.chunk[0][i];
                for (int w = 1; w < kGroup - 1; ++w) all.then(lds.chunk[w][i]);
                all.then(f[v]);
                publish(group + gj * D + v * 64, all.run());
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = lane * V + v;
        const Alone<T, SIGMOID, CUT, BACK> alone{r, p.b, p.len, p.c0 + p.at + v};
        if (p.wave < gj) {
            const auto help = [&] { return word_of(alone.group(sg * kGroup + p.wave)); };
            lds.group[p.wave][i] = run_of(settle_word(group + p.wave * D + v * 64, far[v], s.patience, help));
        }
        if (p.wave == kWaves - 1) {
            const auto help = [&] { return __float_as_uint(alone.state(sg - 1)); };
            lds.enter[i] = sg ? __uint_as_float(settle_word(state + v * 64, before[v], s.patience, help)) : 0.0f;
        }
    }
    __syncthreads();
}

// h through the groups in front of the chunk's, walking the chunks of those
// whose A is too long (all lanes of a wave).
template <typename T, int V, bool SIGMOID, bool CUT, bool BACK>
__device__ __forceinline__ float walk_groups(const RecLds<V>& lds, const RecurrenceArgs& r, const RecShape& s,
                                             const Place<V>& p, int v, float h) {
    const int lane = threadIdx.x & 63, i = lane * V + v, gj = p.pos / kGroup % kGroup;
    const Alone<T, SIGMOID, CUT, BACK> alone{r, p.b, p.len, p.c0 + p.at + v};
    const int first = (p.pos / kGroup - gj) * kGroup;
    const uint64_t* const words = s.word + ((int64_t)p.b * s.chunks + first) * s.row + p.c0 + v * 64 + lane;
#pragma unroll 1
    for (int w = 0; w < gj; ++w) {
        const Run f = lds.group[w][i];
        const bool walk = too_long(f, h);
        float through = apply(f, h);
        if (__any(walk)) {
            float e = h;
#pragma unroll 1
            for (int k = w * kGroup; k < (w + 1) * kGroup; ++k) {
                const uint64_t* const word = words + k * s.row;
                const auto help = [&] { return word_of(alone.chunk(first + k)); };
                e = apply(run_of(settle_word(word, word_at(word), s.patience, help)), e);
            }
            if (walk) through = e;
        }
        h = through;
    }
    return h;
}

// What enters the chunk at channel v of the lane (pos > 0; all lanes of a wave).
template <typename T, int V, bool SIGMOID, bool CUT, bool BACK>
__device__ __forceinline__ float entering(const RecLds<V>& lds, const RecurrenceArgs& r, const RecShape& s,
                                          const Place<V>& p, int v) {
    const int i = (threadIdx.x & 63) * V + v;
    const int j = p.pos % kGroup, gj = p.pos / kGroup % kGroup;
    const float e = lds.enter[i];
    float h = e;
    // no A is too long for a state below 2^24 that it leaves below 2^24
    bool large = !(fabsf(h) < kLarge);
    for (int w = 0; w < gj; ++w) {
        h = apply(lds.group[w][i], h);
        large |= !(fabsf(h) < kLarge);
    }
    if (__builtin_expect(__any(large), 0)) h = walk_groups<T, V, SIGMOID, CUT, BACK>(lds, r, s, p, v, e);
    for (int w = 0; w < j; ++w) h = apply(lds.chunk[w][i], h);
    return h;
}

// ... and, behind the last chunk of a super-group, what leaves it.
template <int V>
__device__ __forceinline__ void tell_state(const RecurrenceArgs& r, const RecShape& s, const Place<V>& p, bool followed,
                                           int v, float h) {
    if (followed && p.pos % (kGroup * kGroup) == kGroup * kGroup - 1)
        publish(s.state + ((int64_t)p.b * s.supers + p.pos / (kGroup * kGroup)) * s.columns * (64 * V) + p.c0 + v * 64 +
                    (threadIdx.x & 63),
                h);
}

template <typename T, int V, bool SIGMOID, bool CUT, bool FULL, int SUB>
__device__ __forceinline__ void forward(const RecurrenceArgs& r, const RecShape& s, RecLds<V>& lds, const Place<V>& p) {
    const int lane = threadIdx.x & 63;
    const int64_t D = r.channels;
    const int t0 = p.pos * kRecChunk, row0 = t0 + p.row * SUB;
    const int64_t out0 = (int64_t)p.b * r.steps * D + p.c0, state0 = (int64_t)p.b * D + p.c0 + p.at;
    const int rows = FULL ? SUB : max(0, min(p.len - row0, SUB));
    uint32_t gate[SUB], x[SUB];
    const int64_t gate0 = p.b * r.gate_batch + p.c0, x0 = p.b * r.x_batch + p.c0;
    if (s.lines) {
        load_rows<T, V, FULL, true>(gate, r.gate, gate0, r.gate_step, row0, p.len, p.at);
        load_rows<T, V, FULL, true>(x, r.x, x0, r.x_step, row0, p.len, p.at);
    } else {
        load_rows<T, V, FULL, false>(gate, r.gate, gate0, r.gate_step, row0, p.len, p.at);
        load_rows<T, V, FULL, false>(x, r.x, x0, r.x_step, row0, p.len, p.at);
    }
    float h[V];  // the state in front of the sequence, then of the wave's steps
#pragma unroll
    for (int v = 0; v < V; ++v)
        h[v] = p.pos == 0 && p.row == 0 && r.h0 ? r.h0[p.b * r.h0_batch + p.c0 + p.at + v] : 0.0f;
    const uint32_t cut = CUT ? restarts<SUB>(r, p.b, row0, p.len) : 0u;
    if (SUB == kSub && p.waves > 1) {  // fewer rows a thread: fewer steps than a wave holds
        Run own[V];
#pragma unroll
        for (int v = 0; v < V; ++v) own[v] = {1.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a, u, rest;
                row_terms<T, V, SIGMOID, FULL>(gate, x, i, v, rows, a, u, rest);
                own[v].A *= a;
                own[v].H = fmaf(unless_at<CUT>(a, cut, i), unless_at<CUT>(own[v].H, cut, i), u);
            }
            end_of_row(i);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            own[v].A = cut ? __uint_as_float(kDropped) : own[v].A + 0.0f;
            lds.wave[p.wave][lane * V + v] = own[v];
        }
        __syncthreads();
        const bool followed = t0 + kRecChunk < p.len;
        if (s.chunks > 1) {
            if (followed && p.wave == 0) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    for (int w = 1; w < kWaves; ++w) own[v] = then(own[v], lds.wave[w][lane * V + v]);
                    if (p.pos == 0) own[v].H = apply(own[v], h[v]);
                }
            }
            exchange<T, V, SIGMOID, CUT, false>(lds, r, s, p, followed, own);
        }
        if (p.row == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = lane * V + v;
                float e = p.pos ? entering<T, V, SIGMOID, CUT, false>(lds, r, s, p, v) : h[v];
                if (p.pos && p.mine && r.ckpt)
                    r.ckpt[((int64_t)p.b * (s.chunks - 1) + p.pos - 1) * D + p.c0 + p.at + v] = e;
                for (int w = p.first; w < p.first + p.waves; ++w) {
                    lds.start[w][i] = e;
                    e = apply(lds.wave[w][i], e);
                }
                tell_state<V>(r, s, p, followed, v, e);
            }
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = lds.start[p.wave][lane * V + v];
        forget(gate);
        forget(x);
    }
    if (!p.mine) return;
    T* out = row_of<T, V>(r.h, out0, D, row0);
    int64_t next = D;
    hide(next);
#pragma unroll
    for (int i = 0; i < SUB; ++i, out += next) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a, u, rest;
            row_terms<T, V, SIGMOID, FULL>(gate, x, i, v, rows, a, u, rest);
            h[v] = fmaf(unless_at<CUT>(a, cut, i), unless_at<CUT>(h[v], cut, i), u);
        }
        if (FULL || i < rows) Lanes<T, V>::template store<(V > 1 || sizeof(T) > 2)>(out, p.at, h);
        end_of_row(i);
    }
    if (!FULL) zero_rows<T, V>(r.h, out0, D, row0 + rows, min(row0 + SUB, r.steps), p.at, s.lines);
    // the wave with the last step, or the first one of an empty sequence
    if (r.h_last && (rows ? row0 + rows == p.len : p.row == 0 && p.len == 0)) {
#pragma unroll
        for (int v = 0; v < V; ++v) r.h_last[state0 + v] = h[v];
    }
}

// Forward. Rows of whole sequences in a wave are bound by memory: 16 steps of
// 1.28M float32 channels in 42.8 us, 5.7 TB/s; 8 x 2048 x 2048 bf16 (ragged,
// SIGMOID) in 32 us, of which some 1.5 are the second of the two instructions
// that bound the factors of 1 - a. 65536 x 1024 bf16 takes 100 us, 4.0 TB/s: the
// same rows copied take 72, the rest is the exchange between chunks. One step
// (64 x 2048 bf16) is one launch of 3.0 us: latency. (Medians.) Six waves a SIMD let three workgroups share a
// unit, so that one's loads fill another's exchange.
template <typename T, int V, bool SIGMOID, bool CUT, int SUB>
__global__ __launch_bounds__(kRecThreads, 6) void k_recurrence_fwd(RecurrenceArgs r, RecShape s) {
    __shared__ RecLds<V> lds;
    const Place<V> p(r, s);
    const int t0 = p.pos * kRecChunk, row0 = t0 + p.row * SUB;
    if (t0 + p.waves * SUB <= p.len)
        forward<T, V, SIGMOID, CUT, true, SUB>(r, s, lds, p);
    else if (t0 < p.len || p.pos == 0)
        forward<T, V, SIGMOID, CUT, false, SUB>(r, s, lds, p);
    else if (p.mine)  // padding
        zero_rows<T, V>(r.h, (int64_t)p.b * r.steps * r.channels + p.c0, r.channels, row0,
                        min(row0 + SUB, r.steps), p.at, s.lines);
}

template <typename T, int V, bool SIGMOID, bool CUT, bool FULL, int SUB>
__device__ __forceinline__ void backward(const RecurrenceArgs& r, const RecShape& s, RecLds<V>& lds,
                                         float (&wave_c)[kWaves][64 * V], float (&start_h)[kWaves][64 * V],
                                         const Place<V>& p, int k) {
    const int lane = threadIdx.x & 63;
    const int64_t D = r.channels;
    const int t0 = k * kRecChunk, row0 = t0 + p.row * SUB;
    const int64_t out0 = (int64_t)p.b * r.steps * D + p.c0, state0 = (int64_t)p.b * D + p.c0 + p.at;
    const bool starts = k == 0 && p.row == 0;
    const int rows = FULL ? SUB : max(0, min(p.len - row0, SUB));
    uint32_t gate[SUB], x[SUB], g[SUB];
    const int64_t gate0 = p.b * r.gate_batch + p.c0, x0 = p.b * r.x_batch + p.c0;
    if (s.lines) {
        load_rows<T, V, FULL, true>(gate, r.gate, gate0, r.gate_step, row0, p.len, p.at);
        load_rows<T, V, FULL, true>(x, r.x, x0, r.x_step, row0, p.len, p.at);
        load_rows<T, V, FULL, true>(g, r.grad_h, out0, D, row0, p.len, p.at);
    } else {
        load_rows<T, V, FULL, false>(gate, r.gate, gate0, r.gate_step, row0, p.len, p.at);
        load_rows<T, V, FULL, false>(x, r.x, x0, r.x_step, row0, p.len, p.at);
        load_rows<T, V, FULL, false>(g, r.grad_h, out0, D, row0, p.len, p.at);
    }
    const bool ends = rows ? row0 + rows == p.len : starts && p.len == 0;  // has the last step
    const bool leads = p.row == p.waves - 1;  // hands the waves of these channels their states
    float h[V], last[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = !leads ? 0.0f
               : k    ? r.ckpt_in[((int64_t)p.b * (s.chunks - 1) + k - 1) * D + p.c0 + p.at + v]
               : r.h0 ? r.h0[state0 + v]
                      : 0.0f;
        last[v] = ends && r.grad_last ? r.grad_last[state0 + v] : 0.0f;
    }
    const uint32_t cut = CUT ? restarts<SUB>(r, p.b, row0, p.len) : 0u;
    const bool followed = k > 0;
    if (SUB == kSub && p.waves > 1) {
        // the wave's run of the states, (A, H), and of what it passes back, (A, C)
        Run own[V];
        float C[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            own[v] = {1.0f, 0.0f};
            C[v] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a, u, rest;
                row_terms<T, V, SIGMOID, FULL>(gate, x, i, v, rows, a, u, rest);
                own[v].H = fmaf(unless_at<CUT>(a, cut, i), unless_at<CUT>(own[v].H, cut, i), u);
                // steps from a restart on pass nothing back in front of it
                own[v].A = unless_before<CUT>(own[v].A * a, cut, i);
                C[v] = fmaf(own[v].A,
                            unless_before<CUT>(row_grad<T, V, FULL>(g, i, v, rows), cut, i), C[v]);
            }
            end_of_row(i);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!cut) C[v] = fmaf(own[v].A, last[v], C[v]);
            own[v].A = cut ? __uint_as_float(kDropped) : own[v].A + 0.0f;
            lds.wave[p.wave][lane * V + v] = own[v];
            wave_c[p.wave][lane * V + v] = C[v];
        }
        __syncthreads();
        if (leads) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float e = h[v];
                for (int w = p.first; w <= p.wave; ++w) {
                    start_h[w][lane * V + v] = e;
                    e = apply(lds.wave[w][lane * V + v], e);
                }
            }
        }
        if (s.chunks > 1) {
            if (followed && p.wave == 0) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int i = lane * V + v;
                    own[v] = {lds.wave[kWaves - 1][i].A, wave_c[kWaves - 1][i]};
                    for (int w = kWaves - 2; w >= 0; --w) own[v] = then(own[v], Run{lds.wave[w][i].A, wave_c[w][i]});
                }
            }
            exchange<T, V, SIGMOID, CUT, true>(lds, r, s, p, followed, own);
        }
        if (p.row == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = lane * V + v;
                float e = p.pos ? entering<T, V, SIGMOID, CUT, true>(lds, r, s, p, v) : 0.0f;
                for (int w = p.first + p.waves - 1; w >= p.first; --w) {
                    lds.start[w][i] = e;
                    e = apply(Run{lds.wave[w][i].A, wave_c[w][i]}, e);
                }
                tell_state<V>(r, s, p, followed, v, e);
            }
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = start_h[p.wave][lane * V + v];
        forget(gate);
        forget(x);
        forget(g);
    }
    if (!p.mine) return;
    // Walk the states, keeping what step i's gradients take: weight, by which
    // d_i is grad_gate_i, and (SIGMOID) e = exp(-gate), of which a and 1 - a
    // are cheap; then walk back.
    float weight[SUB][V], e[SUB][V];
#pragma unroll
    for (int i = 0; i < SUB; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a = Lanes<T, V>::get(gate[i], v), u = Lanes<T, V>::get(x[i], v);
            const float prev = unless_at<CUT>(h[v], cut, i);
            weight[i][v] = prev;
            if (SIGMOID) {
                float rest;
                e[i][v] = exp_minus(a);
                of_exp_minus(e[i][v], a, rest);
                weight[i][v] = (prev - u) * (a * rest);
                u *= rest;
            }
            h[v] = FULL || i < rows ? fmaf(unless_at<CUT>(a, cut, i), prev, u) : h[v];
        }
        end_of_row(i);
    }
    float c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = (SUB == kSub && p.waves > 1 ? lds.start[p.wave][lane * V + v] : 0.0f) + last[v];
    by_lines<T, V>(s.lines, [&](auto past) {
        T* dg = row_of<T, V>(r.grad_gate, out0, D, row0 + SUB - 1);
        T* dx = row_of<T, V>(r.grad_x, out0, D, row0 + SUB - 1);
        int64_t next = D;
        hide(next);
#pragma unroll
        for (int i = SUB - 1; i >= 0; --i, dg -= next, dx -= next) {
            float vg[V], vx[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a, rest = 1.0f;
                if (SIGMOID)
                    of_exp_minus(e[i][v], a, rest);
                else
                    a = Lanes<T, V>::get(gate[i], v);
                const float d = row_grad<T, V, FULL>(g, i, v, rows) + c[v];
                vg[v] = d * weight[i][v];
                vx[v] = SIGMOID ? d * rest : d;
                if (FULL || i < rows) c[v] = unless_at<CUT>(a * d, cut, i);
            }
            if (FULL || i < rows) {
                Lanes<T, V>::template store<past.value>(dg, p.at, vg);
                Lanes<T, V>::template store<past.value>(dx, p.at, vx);
            }
            end_of_row(SUB - 1 - i);
        }
    });
    if (!FULL) {
        zero_rows<T, V>(r.grad_gate, out0, D, row0 + rows, min(row0 + SUB, r.steps), p.at, s.lines);
        zero_rows<T, V>(r.grad_x, out0, D, row0 + rows, min(row0 + SUB, r.steps), p.at, s.lines);
    }
    if (r.grad_h0 && starts) {
#pragma unroll
        for (int v = 0; v < V; ++v) r.grad_h0[state0 + v] = c[v];
    }
}

// Backward: three tensors in, two out. Bound by memory while rows move: 8 x 2048
// x 2048 bf16 (ragged) in 52 to 53 us, 4.5 TB/s; all rows there (LINEAR) 79 us,
// 4.2 TB/s. A thread's 16 rows of three inputs and what it keeps of the walk
// (weight, e) take 85 to 92 registers, so two workgroups share a unit; a third,
// with 80 registers, gains nothing (83 us), and two channels a lane spill (99
// against 85 us forward and backward). 3 x 1001 x 777 float32 takes 17 us: eight
// chunks in turn.
template <typename T, int V, bool SIGMOID, bool CUT, int SUB>
__global__ __launch_bounds__(kRecThreads, 4) void k_recurrence_bwd(RecurrenceArgs r, RecShape s) {
    __shared__ RecLds<V> lds;
    __shared__ float wave_c[kWaves][64 * V], start_h[kWaves][64 * V];
    const Place<V> p(r, s);
    const int used = (p.len + kRecChunk - 1) / kRecChunk;  // chunks with steps: taken from the last on
    const int k = p.pos < used ? used - 1 - p.pos : p.pos;
    const int t0 = k * kRecChunk, row0 = t0 + p.row * SUB;
    if (t0 + p.waves * SUB <= p.len) {
        backward<T, V, SIGMOID, CUT, true, SUB>(r, s, lds, wave_c, start_h, p, k);
    } else if (t0 < p.len || k == 0) {
        backward<T, V, SIGMOID, CUT, false, SUB>(r, s, lds, wave_c, start_h, p, k);
    } else if (p.mine) {  // padding
        const int64_t out0 = (int64_t)p.b * r.steps * r.channels + p.c0;
        zero_rows<T, V>(r.grad_gate, out0, r.channels, row0, min(row0 + SUB, r.steps), p.at, s.lines);
        zero_rows<T, V>(r.grad_x, out0, r.channels, row0, min(row0 + SUB, r.steps), p.at, s.lines);
    }
}

__global__ void k_recurrence_pass(const float* from, float* to, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * kRecThreads + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : 0.0f;
}

std::atomic<int> g_patience{kPatience};

int chunks_of(int steps) { return std::max(1, (int)(((int64_t)steps + kRecChunk - 1) / kRecChunk)); }

// columns of `column` channels each
size_t layout(int batch, int steps, int channels, int columns, int column, RecShape* s, void* base) {
    s->chunks = chunks_of(steps);
    s->groups = (s->chunks + kGroup - 1) / kGroup;
    s->supers = (s->groups + kGroup - 1) / kGroup;
    s->columns = columns;
    s->row = (int64_t)columns * column;
    s->steps_log2 = 0;
    while ((kSub << s->steps_log2) < std::min(steps, kRecChunk)) ++s->steps_log2;
    s->word = s->group = nullptr;
    s->state = nullptr;
    s->patience = g_patience.load(std::memory_order_relaxed);
    if (s->chunks == 1) return 0;
    const size_t row = (size_t)batch * (((size_t)channels + 127) / 128 * 128);
    const size_t words = row * (s->chunks + s->groups), states = row * s->supers;
    s->word = (uint64_t*)base;
    s->group = s->word + row * s->chunks;
    s->state = (uint32_t*)(s->word + words);
    return words * 8 + states * 4;
}

// Fills words of the workspace with ones, 16 bytes a thread.
__device__ __forceinline__ void fill_ones(uint32_t* p, size_t words, size_t i) {
    if (i + 4 <= words) {
        *(uint4*)(p + i) = make_uint4(~0u, ~0u, ~0u, ~0u);
    } else {
        for (size_t j = i; j < words; ++j) p[j] = ~0u;
    }
}
__device__ __forceinline__ size_t clear_at() { return ((size_t)blockIdx.x * kRecThreads + threadIdx.x) * 4; }
__global__ void k_recurrence_clear(uint32_t* p, size_t words) { fill_ones(p, words, clear_at()); }
// ... and the last super-group's row of each sequence with h0. Rows are a
// multiple of 64 words, so a thread's four words are in one row.
__global__ void k_recurrence_clear_keep(uint32_t* p, size_t words, RecShape s, const float* h0, int batch,
                                        int channels) {
    const size_t i = clear_at(), first = s.state - p;
    if (i >= first && i < words) {
        const size_t row = (i - first) / s.row, c = (i - first) % s.row, b = row / s.supers;
        if (row % s.supers == (size_t)s.supers - 1 && b < (size_t)batch) {
            for (int j = 0; j < 4; ++j)
                p[i + j] = c + j < (size_t)channels ? __float_as_uint(h0[b * channels + c + j]) : 0u;
            return;
        }
    }
    fill_ones(p, words, i);
}

// The low bits of where the rows of any tensor start: of the tensors' addresses
// and (in elements) of the distances between rows.
uint64_t starts_of(const RecurrenceArgs& r) {
    return (uint64_t)r.gate | (uint64_t)r.x | (uint64_t)r.h | (uint64_t)r.grad_h | (uint64_t)r.grad_gate |
           (uint64_t)r.grad_x;
}
uint64_t strides_of(const RecurrenceArgs& r) {
    return (uint64_t)r.channels | (uint64_t)(r.gate_batch | r.gate_step | r.x_batch | r.x_step);
}

// Lays out the launch (and clears its workspace); gives its workgroups. Where
// h_last takes h0's place, workgroups that run later than they are numbered, or
// compute for themselves what they wait for, would find the final state: from
// then on r.h0 is a copy in the workspace. (A single chunk reads it before
// anything is written.)
template <int V>
hipError_t prepare(RecurrenceArgs& r, int bytes_each, void* scratch, RecShape* s, unsigned* blocks,
                   hipStream_t stream) {
    const size_t bytes = layout(r.batch, r.steps, r.channels, (r.channels + 64 * V - 1) / (64 * V), 64 * V, s, scratch);
    s->lines = !((starts_of(r) | (strides_of(r) * bytes_each)) & 127);
    r.h0_batch = r.channels;
    if (s->chunks == 1) {
        const int across = kWaves >> s->steps_log2;
        *blocks = (unsigned)r.batch * ((s->columns + across - 1) / across);
        return hipSuccess;
    }
    *blocks = (unsigned)r.batch * s->columns * s->chunks;
    const size_t threads = (bytes + 15) / 16;
    const unsigned clears = (unsigned)((threads + kRecThreads - 1) / kRecThreads);
    if (r.h0 && r.h0 == r.h_last) {
        k_recurrence_clear_keep<<<clears, kRecThreads, 0, stream>>>((uint32_t*)scratch, bytes / 4, *s, r.h0, r.batch,
                                                                    r.channels);
        r.h0 = (const float*)(s->state + (s->supers - 1) * s->row);
        r.h0_batch = s->supers * s->row;
    } else {
        k_recurrence_clear<<<clears, kRecThreads, 0, stream>>>((uint32_t*)scratch, bytes / 4);
    }
    return hipGetLastError();
}

template <typename T, int V, bool SIGMOID, bool CUT>
struct Forward {
    static hipError_t launch(RecurrenceArgs r, void* scratch, hipStream_t stream) {
        RecShape s;
        unsigned blocks;
        if (hipError_t e = prepare<V>(r, sizeof(T), scratch, &s, &blocks, stream)) return e;
        if (r.steps == 1)  // serving: no row but the one
            k_recurrence_fwd<T, V, SIGMOID, CUT, 1><<<blocks, kRecThreads, 0, stream>>>(r, s);
        else if (r.steps <= kFew)
            k_recurrence_fwd<T, V, SIGMOID, CUT, kFew><<<blocks, kRecThreads, 0, stream>>>(r, s);
        else
            k_recurrence_fwd<T, V, SIGMOID, CUT, kSub><<<blocks, kRecThreads, 0, stream>>>(r, s);
        return hipGetLastError();
    }
};
template <typename T, int V, bool SIGMOID, bool CUT>
struct Backward {
    static hipError_t launch(RecurrenceArgs r, void* scratch, hipStream_t stream) {
        RecShape s;
        unsigned blocks;
        if (hipError_t e = prepare<V>(r, sizeof(T), scratch, &s, &blocks, stream)) return e;
        if (r.steps <= kFew)
            k_recurrence_bwd<T, V, SIGMOID, CUT, kFew><<<blocks, kRecThreads, 0, stream>>>(r, s);
        else
            k_recurrence_bwd<T, V, SIGMOID, CUT, kSub><<<blocks, kRecThreads, 0, stream>>>(r, s);
        return hipGetLastError();
    }
};

template <template <typename, int, bool, bool> class K, typename T, int V>
hipError_t launch_of(const RecurrenceArgs& r, bool sigmoid, void* scratch, hipStream_t stream) {
    if (sigmoid)
        return r.restart ? K<T, V, true, true>::launch(r, scratch, stream)
                         : K<T, V, true, false>::launch(r, scratch, stream);
    return r.restart ? K<T, V, false, true>::launch(r, scratch, stream)
                     : K<T, V, false, false>::launch(r, scratch, stream);
}

// Two 16-bit channels a lane need every row of every tensor on a 4-byte boundary.
bool pairs_fit(const RecurrenceArgs& r) { return !((starts_of(r) | (strides_of(r) * 2)) & 3); }

// No steps at all: the state, or its gradient, passes through.
hipError_t pass_through(const RecurrenceArgs& r, const float* from, float* to, hipStream_t stream) {
    const int64_t n = (int64_t)r.batch * r.channels;
    if (!to || to == from) return hipSuccess;
    k_recurrence_pass<<<(unsigned)((n + kRecThreads - 1) / kRecThreads), kRecThreads, 0, stream>>>(from, to, n);
    return hipGetLastError();
}

}  // namespace

int set_recurrence_patience(int polls) { return g_patience.exchange(polls < 0 ? kPatience : polls); }

bool recurrence_fits(const gs_recurrence& r) {
    const int64_t most = ((int64_t)1 << 32) / kRecThreads - 1;  // a grid has less than 2^32 threads
    const int64_t columns = ((int64_t)r.channels + 63) / 64, chains = columns * std::max(r.batch, 1);
    return chains <= most && chains * chunks_of(r.steps) <= most;
}

size_t recurrence_scratch_bytes(const gs_recurrence& r) {
    RecShape s;
    if (r.batch == 0 || r.channels == 0) return 0;
    return layout(r.batch, r.steps, r.channels, (r.channels + 63) / 64, 64, &s, nullptr);
}

hipError_t launch_recurrence_fwd(const RecurrenceArgs& r, int dtype, bool sigmoid, void* scratch, hipStream_t stream) {
    if (r.steps == 0) return pass_through(r, r.h0, r.h_last, stream);
    if (dtype == GS_F32) return launch_of<Forward, float, 1>(r, sigmoid, scratch, stream);
    // two channels a lane: 65536 x 1024 bf16 in 102 us, one: 112 us
    const bool pairs = pairs_fit(r);
    if (dtype == GS_BF16)
        return pairs ? launch_of<Forward, __bf16, 2>(r, sigmoid, scratch, stream)
                     : launch_of<Forward, __bf16, 1>(r, sigmoid, scratch, stream);
    return pairs ? launch_of<Forward, _Float16, 2>(r, sigmoid, scratch, stream)
                 : launch_of<Forward, _Float16, 1>(r, sigmoid, scratch, stream);
}

hipError_t launch_recurrence_bwd(const RecurrenceArgs& r, int dtype, bool sigmoid, void* scratch, hipStream_t stream) {
    if (r.steps == 0) return pass_through(r, r.grad_last, r.grad_h0, stream);
    if (dtype == GS_F32) return launch_of<Backward, float, 1>(r, sigmoid, scratch, stream);
    if (dtype == GS_BF16) return launch_of<Backward, __bf16, 1>(r, sigmoid, scratch, stream);
    return launch_of<Backward, _Float16, 1>(r, sigmoid, scratch, stream);
}

}  // namespace gs
