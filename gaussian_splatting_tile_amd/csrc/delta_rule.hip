// Gated delta rule, forward and backward (include/gs.h, gs_delta_rule_*).
//
// A sequence is cut into chunks of 64 steps. Inside a chunk, with S the state
// in front, gamma_i the product of the decays up to step i, D_ij that of the
// decays behind j up to i (0 across a restart), the steps' u solve
//   (I + A) U = R,  A_ij = beta_i D_ij k_i.k_j (j < i),  R = beta (V - gamma K S)
// and with M = (I + A)^-1, P_ij = scale D_ij q_i.k_j (j <= i), e_j = D_{63,j}:
//   U = M R;  O = scale gamma Q S + P U;  S' = gamma_63 S + K^T (e U).
// Backwards, with dS the gradient of S' and dO that of O:
//   dU = P^T dO + e K dS;  dR = M^T dU;  dV = beta dR
//   dS <- gamma_63 dS + Q^T (scale gamma dO) - K^T (beta gamma dR)
// and, D included in both, Pd = scale D (dO U^T), Ad = -beta D (dR U^T) (j < i):
//   dQ = scale gamma (dO S^T) + Pd K
//   dK = Pd^T Q + Ad K + Ad^T K - beta gamma (dR S^T) + e (U dS^T)
//   dbeta_i = dR_i.(v_i - gamma_i S^T k_i) + sum_j Ad_ij k_i.k_j / beta_i
// The decay of step t lies between all j < t <= i, so with
// X_ij = Pd_ij q_i.k_j + Ad_ij k_i.k_j
//   dlog_decay_t = sum_{j < t <= i} X_ij + sum_{i >= t} f_i + sum_{j < t} b_j + gamma_63 <S, dS>
//   f_i = q_i.(scale gamma dO S^T)_i - k_i.(beta gamma dR S^T)_i,  b_j = k_j.(e U dS^T)_j
// formed as these sums, without differences of larger ones.
#include <algorithm>
#include <type_traits>

#include "gs_internal.h"

namespace gs {
namespace {

constexpr int kC = GS_DELTA_CHUNK;
constexpr int kTiles = 10;               // lower 16 x 16 tiles of a chunk's 64 x 64 matrix
constexpr int kLower = kTiles * 256;     // their floats
constexpr int kPitch = kC + 4;           // of a 64 x 64 matrix in LDS

typedef __bf16 bf16;
typedef _Float16 f16;
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ constexpr int tri(int i, int j) { return i * (i + 1) / 2 + j; }

// Products of 16 x 16 tiles over 16: lane (i, g) of a wave holds A[i][4g + r] in a[r], B[4g + r][i] in b[r]
// and C[4g + r][i] in c[r], so one product's result is the next one's right operand as it stands.
__device__ __forceinline__ f32x4 mma(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
}

struct Chunk {
    double G[kC];       // log2 of the product of the decays up to each step
    float gamma[kC];    // that product, 0 behind a restart
    float end[kC];      // product of the decays behind each step, 0 in front of a restart
    float beta[kC];
    int seg[kC];        // restarts up to each step
    float whole;        // product of all decays, 0 with a restart
    float ends[2];      // steps in front of the first restart (64 without one), the last restart (or 0)
};

__device__ __forceinline__ int length_of(const gs_delta_rule& r, int b) {
    return r.lengths ? min(max(r.lengths[b], 0), r.steps) : r.steps;
}

// By one wave, a lane a step. A decay that is 0 in float32 acts as a restart, so every sum is finite.
__device__ __forceinline__ void load_gates(const DeltaArgs& a, int b, int h, int t0, int len, Chunk& s) {
    const int lane = threadIdx.x & 63, t = t0 + lane;
    const bool live = t < len;
    float g = live ? a.log_decay[b * a.r.decay_batch + t * a.r.decay_step + h] : 0.0f;
    const float beta = live ? a.beta[b * a.r.beta_batch + t * a.r.beta_step + h] : 0.0f;
    const bool cut = live && (g < -104.0f || (a.r.restart && a.r.restart[(int64_t)b * a.r.steps + t]));
    const uint64_t cuts = __ballot(cut);
    const int seg = __popcll(cuts & (~0ull >> (63 - lane))), segs = __popcll(cuts);
    double G = cut ? 0.0 : (double)g * 1.4426950408889634;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double p = __shfl_up(G, m);
        if (lane >= m) G += p;
    }
    const double last = __shfl(G, 63);
    s.G[lane] = G;
    s.seg[lane] = seg;
    s.beta[lane] = beta;
    s.gamma[lane] = seg == 0 ? __builtin_amdgcn_exp2f((float)G) : 0.0f;
    s.end[lane] = seg == segs ? __builtin_amdgcn_exp2f((float)(last - G)) : 0.0f;
    if (lane == 63) {
        s.whole = segs == 0 ? __builtin_amdgcn_exp2f((float)G) : 0.0f;
        s.ends[0] = cuts ? __ffsll((unsigned long long)cuts) - 1 : kC;
        s.ends[1] = cuts ? 63 - __clzll(cuts) : 0;
    }
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

__device__ __forceinline__ float decay(const Chunk& s, int i, int j) {
    return s.seg[i] == s.seg[j] ? __builtin_amdgcn_exp2f((float)(s.G[i] - s.G[j])) : 0.0f;
}

// 64 rows of a [B][T][heads][dim] tensor as float32 in LDS, 0 at padding and past dim.
template <int DK, typename T>
__device__ __forceinline__ void load_rows(const T* p, int64_t step, int rows, int dim, float* to, int threads) {
    for (int e = threadIdx.x; e < kC * DK; e += threads) {
        const int t = e / DK, d = e % DK;
        to[t * (DK + 4) + d] = t < rows && d < dim ? (float)p[t * step + d] : 0.0f;
    }
}

template <int DK>
__device__ __forceinline__ f32x4 row4(const float* m, int row, int col) {
    return *(const f32x4*)(m + row * (DK + 4) + col);
}
__device__ __forceinline__ f32x4 col4(const float* m, int pitch, int row, int col) {
    const float* const p = m + row * pitch + col;
    return f32x4{p[0], p[pitch], p[2 * pitch], p[3 * pitch]};
}

// For the gradients of float32 inputs: M = (I + A)^-1 of every chunk and head,
// its lower 16 x 16 tiles, row-major, in to[b][chunk][h][10][16][16]. The diagonal tiles by forward substitution, the
// others from them, M21 = -M22 A21 M11 for pairs of tiles and of pairs. 18 us for
// 195 of them (3 x 777 steps of 5 heads).
template <typename T, int DK>
__global__ __launch_bounds__(256) void k_delta_inverse(DeltaArgs a, int chunks, float* to) {
    __shared__ float K[kC * (DK + 4)];
    __shared__ float M[kC * kPitch];
    __shared__ Chunk s;
    const int h = blockIdx.x % a.r.heads, c = blockIdx.x / a.r.heads % chunks, b = blockIdx.x / a.r.heads / chunks;
    const int len = length_of(a.r, b), t0 = c * kC;
    if (t0 >= len) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
    const int kh = h / (a.r.heads / a.r.key_heads);
    const T* const k = (const T*)a.k + b * a.r.k_batch + t0 * a.r.k_step + kh * a.r.k_head;
    load_rows<DK>(k, a.r.k_step, len - t0, a.r.key_dim, K, 256);
    if (w == 0) load_gates(a, b, h, t0, len, s);
    __syncthreads();
    for (int cj = 0; cj <= w; ++cj) {
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt)
            acc = mma(row4<DK>(K, 16 * w + n, 16 * kt + 4 * g), row4<DK>(K, 16 * cj + n, 16 * kt + 4 * g), acc);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * w + 4 * g + r, j = 16 * cj + n;
            M[i * kPitch + j] = i > j ? s.beta[i] * decay(s, i, j) * acc[r] : 0.0f;
        }
    }
    __syncthreads();
    {
        float x[16];
        const float* const A = M + 16 * w * (kPitch + 1);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float t = i == n ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < i; ++j) t = fmaf(-A[i * kPitch + j], x[j], t);
            x[i] = t;
        }
        __syncthreads();
        if (lane < 16)
#pragma unroll
            for (int i = 0; i < 16; ++i) M[(16 * w + i) * kPitch + 16 * w + n] = x[i];
    }
    __syncthreads();
    auto tile = [&](int i, int j) { return *(const f32x4*)(M + (16 * i + n) * kPitch + 16 * j + 4 * g); };
    auto right = [&](int i, int j) { return col4(M, kPitch, 16 * i + 4 * g, 16 * j + n); };
    const f32x4 zero = {0, 0, 0, 0};
    auto put = [&](int i, int j, f32x4 v) {
#pragma unroll
        for (int r = 0; r < 4; ++r) M[(16 * i + 4 * g + r) * kPitch + 16 * j + n] = -v[r];
    };
    if (w < 2) {
        const f32x4 x = mma(tile(2 * w + 1, 2 * w), right(2 * w, 2 * w), zero);
        put(2 * w + 1, 2 * w, mma(tile(2 * w + 1, 2 * w + 1), x, zero));
    }
    __syncthreads();
    f32x4 y2 = zero, y3 = zero;
    if (w < 2) {
        f32x4 x2 = zero, x3 = zero;
        for (int q = w; q < 2; ++q) {
            const f32x4 m = right(q, w);
            x2 = mma(tile(2, q), m, x2);
            x3 = mma(tile(3, q), m, x3);
        }
        y2 = mma(tile(2, 2), x2, zero);
        y3 = mma(tile(3, 3), x3, mma(tile(3, 2), x2, zero));
    }
    __syncthreads();
    if (w < 2) {
        put(2, w, y2);
        put(3, w, y3);
    }
    __syncthreads();
    float* const out = to + (int64_t)blockIdx.x * kLower;
    for (int e = threadIdx.x; e < kLower; e += 256) {
        const int q = e >> 8, i = q >= 6 ? 3 : q >= 3 ? 2 : q >= 1 ? 1 : 0, j = q - tri(i, 0);
        out[e] = M[(16 * i + (e >> 4 & 15)) * kPitch + 16 * j + (e & 15)];
    }
}

// ---------------------------------------------------------------------------
// Float32 values on the 16-bit matrix instructions. Scaled by a power of two to
// at most 1, a value is the sum of two float16 ones (planes), the rounding of
// it and that of the rest: 22 bits, or 2^-25 of the largest value that shares
// the scale. Left operands are scaled by rows, right ones by columns, so the
// scales leave every sum as one factor. Inputs of 16 bits are one plane
// (bfloat16's 8 bits fit float16's 11), float32 ones two; a product of two
// planes leaves out the product of the rests. An instruction takes 1/16 of the
// float32 one's time for the same product, so float32 results cost 2/16
// (16-bit inputs) or 3/16.
//
// In lane (i, g) of a wave a tile's right operand is 8 values of column i, its
// left operand 8 of row i, for the same 8 terms of the sum; the result holds
// rows 4g + r of column i. Which 8 terms is free as long as both sides agree:
// with the terms 4g + r of two tiles in a row, two results are a right operand
// as they stand.
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int N>
struct Planes {
    f16x8 p[N];
};

// The place (i, g) of a lane. here(): the same, which the compiler does not
// know, so that the many addresses that follow from it are formed where they
// are used and not held in registers through a loop.
struct Lane {
    int n, g;
    __device__ __forceinline__ explicit Lane(int id = threadIdx.x) : n(id & 15), g(id >> 4 & 3) {}
    static __device__ __forceinline__ Lane here() {
        int id = threadIdx.x;
        asm volatile("" : "+v"(id));
        return Lane(id);
    }
};

template <int N>
__device__ __forceinline__ Planes<N> split(f32x4 a, f32x4 b, float scale) {
    Planes<N> out;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const f32x2 v = e < 4 ? f32x2{a[e], a[e + 1]} : f32x2{b[e - 4], b[e - 3]};
        const f16x2 h = __builtin_convertvector(f32x2{v[0] * scale, v[1] * scale}, f16x2);
        out.p[0][e] = h[0];
        out.p[0][e + 1] = h[1];
        if constexpr (N > 1) {
            const f32x2 rest = {fmaf(v[0], scale, -(float)h[0]), fmaf(v[1], scale, -(float)h[1])};
            const f16x2 l = __builtin_convertvector(rest, f16x2);
            out.p[1][e] = l[0];
            out.p[1][e + 1] = l[1];
        }
    }
    return out;
}

// A power of two that brings values of this largest size to [1/2, 1), and its inverse.
struct Scale {
    float by, back;
    __device__ __forceinline__ explicit Scale(float largest) {
        const int e = min(max(__builtin_amdgcn_frexp_expf(largest), -126), 127);
        by = __builtin_amdgcn_ldexpf(1.0f, -e);
        back = __builtin_amdgcn_ldexpf(1.0f, e);
    }
};

template <int N>
__device__ __forceinline__ float largest(const f32x4 (&v)[N]) {
    float m = 0.0f;
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(v[t][r]));
    return m;
}
// Over the four lanes that hold a column of a result.
__device__ __forceinline__ float over_column(float m) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    m = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    a = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
// Over N neighbouring lanes (N = 8 or 16).
template <int N>
__device__ __forceinline__ float over_lanes(float m) {
    auto with = [&](auto ctrl) {
        m = fmaxf(m, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(m), decltype(ctrl)::value, 0xf, 0xf, true)));
    };
    with(std::integral_constant<int, 0xB1>{});   // quad_perm 1 0 3 2
    with(std::integral_constant<int, 0x4E>{});   // quad_perm 2 3 0 1
    with(std::integral_constant<int, 0x141>{});  // row_half_mirror
    if constexpr (N == 16) with(std::integral_constant<int, 0x140>{});  // row_mirror
    return m;
}

// c[t] += A[t] B for COUNT left operands, the planes' products but that of the rests, smaller ones first.
template <int COUNT, int NA, int NB>
__device__ __forceinline__ void products(const Planes<NA> (&A)[COUNT], const Planes<NB>& B, f32x4* c) {
#pragma unroll
    for (int sum = 1; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i <= sum; ++i)
            if (i < NA && sum - i < NB)
#pragma unroll
                for (int t = 0; t < COUNT; ++t)
                    c[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(A[t].p[i], B.p[sum - i], c[t], 0, 0, 0);
}

// Planes of an input. What the kernels form themselves has two, whatever it is rounded to at the end.
template <typename T>
constexpr int kPlanes = sizeof(T) == 4 ? 2 : 1;

// 64 rows of an input, plane after plane, in 16-byte pieces; piece c of row t
// lies at c ^ t (within the row), so that the same piece of 16 rows covers all
// banks of LDS.
template <int NX, int DK>
struct Operand {
    static constexpr int N = NX, PIECES = DK / 8, PLANE = kC * DK, SIZE = N * PLANE;
    static __device__ __forceinline__ int at(int t, int c) { return t * DK + (c ^ (t & (PIECES - 1))) * 8; }
    // the rows 16 tile + i, terms 32 s + 8 g ..
    static __device__ __forceinline__ Planes<N> row(const f16* m, int tile, int s, Lane l = Lane()) {
        const int n = l.n, g = l.g;
        Planes<N> x;
#pragma unroll
        for (int k = 0; k < N; ++k) x.p[k] = *(const f16x8*)(m + k * PLANE + at(16 * tile + n, 4 * s + g));
        return x;
    }
    // the transposed rows: dimensions 32 s + 8 (i / 4) + 4 h + i % 4, terms the steps 4g + r of tiles 2p and 2p + 1
    static __device__ __forceinline__ Planes<N> column(const f16* m, int s, int h, int p, Lane l = Lane()) {
        const int n = l.n, g = l.g;
        typedef short i16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) i16x4* Lds;
        Planes<N> x;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int t = 32 * p + 4 * g + n / 4;
            const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(m + k * PLANE + at(t, 4 * s + (n & 3)) + 4 * h));
            const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(m + k * PLANE + at(t + 16, 4 * s + (n & 3)) + 4 * h));
            const f16x4 lo = __builtin_bit_cast(f16x4, a), hi = __builtin_bit_cast(f16x4, b);
            x.p[k] = f16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
        return x;
    }
};

// A uniform base and a 32-bit offset in bytes.
template <typename V, typename T>
__device__ __forceinline__ V& at_bytes(T* p, uint32_t off) {
    typedef std::conditional_t<std::is_const_v<T>, const char, char> Byte;
    return *(V*)((Byte*)p + off);
}

// A uniform base of `bytes` bytes (below 2^31) and 32-bit offsets: what lies at
// or behind the end is read as 0 and not written, without a branch.
constexpr uint32_t kNowhere = 0x80000000u;
struct Buffer {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ Buffer(const void* p, uint32_t bytes)
        : r(__builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00020000)) {}
    template <typename T>
    __device__ __forceinline__ T load(uint32_t off) const {
        if constexpr (sizeof(T) == 2)
            return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
        else
            return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
    }
    template <typename T>
    __device__ __forceinline__ void store(uint32_t off, T v) const {
        if constexpr (sizeof(T) == 2)
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), r, off, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, off, 0, 0);
    }
};

// What the chunks' kernels share, made once, in the form in which they take it.
// Of a chunk and key head: the planes of keys and queries, rows scaled.
template <int NX, int DK>
struct Keys {
    f16 K[NX * kC * DK], Q[NX * kC * DK];
};
// Of a chunk and head: left operands in the order in which lanes take them (the
// pairs of tiles (0,0) (1,0) (2,0) (2,1) (3,0) (3,1), or (0,0) (0,1) (1,0)
// (1,1) (2,1) (3,1) of transposed ones), and per step, with the scales of the
// keys' and queries' rows in them, gamma of K S, scale gamma of Q S, e of K^T U,
// and beta.
constexpr int kPairs = 6;
constexpr int kPair = 512;  // elements of a pair's plane
struct Forward {
    f16 M[kPairs * 2 * kPair], P[kPairs * 2 * kPair];
    float gamma[kC], query[kC], end[kC], beta[kC];
    float misc[kC];  // 0: gamma of the chunk, 1 and 2: the inverse scales of M and P, 3 and 4: Chunk's ends
};
// Of the backward's: M, and M and P transposed, and per step gamma, e, beta and
// the inverse scales of the keys' and queries' rows.
struct Backward {
    f16 M[kPairs * 2 * kPair], MT[kPairs * 2 * kPair], PT[kPairs * 2 * kPair];
    float gamma[kC], end[kC], beta[kC], k_back[kC], q_back[kC];
    float misc[kC];  // as Forward's
};

__device__ __forceinline__ constexpr int pair_row(int f) { return f < 2 ? f : f < 4 ? 2 : 3; }
__device__ __forceinline__ constexpr int pair_col(int f) { return f == 3 || f == 5; }
__device__ __forceinline__ constexpr int upper_row(int f) { return f < 2 ? 0 : f < 4 ? 1 : f - 2; }
__device__ __forceinline__ constexpr int upper_col(int f) { return f == 1 || f >= 3; }

constexpr int kPrepThreads = 256;

// Records of a chunk for all heads of a key head: the rows of keys and queries
// (0 at padding), K K^T and Q K^T, then per head the decays, and M by forward
// substitution in the diagonal tiles and M21 = -M22 A21 M11 for pairs of tiles
// and of pairs, in float32. Bound by the waits between its steps (two in three
// of its cycles), which three workgroups a compute unit (two with float32 inputs)
// share. All rows are fetched before the first is used, and as many heads' gates
// as there are waves are formed meanwhile (a call of 8192 steps of 16 key heads
// and 32 heads of 128, bf16: 329 us at that step, 344 with one after another).
// Of that call, now 340 us, 94 us for 242 MB, 2.6 TB/s.
template <typename T, int DK, typename Record>
__global__ __launch_bounds__(kPrepThreads, sizeof(T) == 4 ? 2 : 3) void k_delta_prepare(DeltaArgs a, int chunks, Keys<kPlanes<T>, DK>* keys,
                                                                Record* to) {
    constexpr bool BACK = std::is_same_v<Record, Backward>;
    constexpr int NX = kPlanes<T>;
    typedef Operand<NX, DK> O;
    // the rows until their products are in registers, then M and P
    __shared__ union Shared {
        Keys<NX, DK> kq;
        float mp[2][kC * kPitch];
    } sh;
    Keys<NX, DK>& kq = sh.kq;
    float* const M = sh.mp[0];
    float* const P = sh.mp[1];
    __shared__ float k_back[kC], q_back[kC], most[2][4];
    constexpr int WAVES = kPrepThreads / 64;
    __shared__ Chunk gates[WAVES];  // of as many heads, a wave each
    const gs_delta_rule& d = a.r;
    const int kh = blockIdx.x % d.key_heads, c = blockIdx.x / d.key_heads % chunks, b = blockIdx.x / d.key_heads / chunks;
    const int len = length_of(d, b), t0 = c * kC, rows = len - t0, group = d.heads / d.key_heads;
    if (rows <= 0) return;
    const int w = threadIdx.x >> 6;
    typedef T T8 __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    constexpr int PIECES = O::PIECES, BY = kPrepThreads / PIECES, JOBS = kC / BY;
    const int at = threadIdx.x % PIECES, dim = at * 8;
    auto fetch = [&](const T* p, int64_t step, T8 (&x)[JOBS]) {
#pragma unroll
        for (int j = 0; j < JOBS; ++j) {
            const int t = threadIdx.x / PIECES + j * BY;
            const T* const from = p + min(t, rows - 1) * step + dim;
            x[j] = T8{};
            if (dim + 8 <= d.key_dim) {
                x[j] = *(const T8*)from;
            } else if (dim < d.key_dim) {
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if (dim + i < d.key_dim) x[j][i] = from[i];
            }
        }
    };
    auto stage = [&](const T8 (&x)[JOBS], f16* m, f16* out, float* back) {
#pragma unroll
        for (int j = 0; j < JOBS; ++j) {
            const int t = threadIdx.x / PIECES + j * BY;
            f32x4 v[2];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i / 4][i % 4] = t < rows ? (float)x[j][i] : 0.0f;
            const Scale scale(over_lanes<PIECES>(largest(v)));
            const Planes<NX> y = split<NX>(v[0], v[1], scale.by);
#pragma unroll
            for (int k = 0; k < NX; ++k) {
                *(f16x8*)(m + k * O::PLANE + O::at(t, at)) = y.p[k];
                *(f16x8*)(out + k * O::PLANE + O::at(t, at)) = y.p[k];
            }
            if (at == 0) back[t] = scale.back;
        }
    };
    Keys<NX, DK>* const key = keys + ((int64_t)b * chunks + c) * d.key_heads + kh;
    {
        T8 k[JOBS], q[JOBS];
        fetch((const T*)a.k + b * d.k_batch + t0 * d.k_step + kh * d.k_head, d.k_step, k);
        fetch((const T*)a.q + b * d.q_batch + t0 * d.q_step + kh * d.q_head, d.q_step, q);
        if (w < group) load_gates(a, b, kh * group + w, t0, len, gates[w]);
        stage(k, kq.K, key->K, k_back);
        stage(q, kq.Q, key->Q, q_back);
    }
    __syncthreads();
    const f32x4 zero = {0, 0, 0, 0};
    f32x4 kk[4], qk[4];  // of row tile w
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = zero;
#pragma unroll
    for (int x = 0; x < DK / 32; ++x) {
        const Planes<NX> left[2] = {O::row(kq.K, w, x), O::row(kq.Q, w, x)};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= w) {
                f32x4 t[2] = {kk[j], qk[j]};
                products(left, O::row(kq.K, j, x), t);
                kk[j] = t[0];
                qk[j] = t[1];
            }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 512; e += kPrepThreads) {  // the tiles over the diagonal that pairs take along
        const int i = (e >> 4 & 15) + (e >> 8) * 32, j = (e & 15) + (e >> 8) * 32 + 16;
        M[i * kPitch + j] = P[i * kPitch + j] = 0.0f;
    }
    for (int hh = 0; hh < group; ++hh) {
        const Lane l = Lane::here();
        const int n = l.n, g = l.g, lane = 16 * g + n;
        const int h = kh * group + hh;
        Record* const out = to + ((int64_t)b * chunks + c) * d.heads + h;
        if (hh) __syncthreads();
        if (hh && hh % WAVES == 0) {
            if (hh + w < group) load_gates(a, b, h + w, t0, len, gates[w]);
            __syncthreads();
        }
        const Chunk& s = gates[hh % WAVES];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= w)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * w + 4 * g + r, col = 16 * j + n;
                    const float D = row >= col ? decay(s, row, col) * k_back[col] : 0.0f;
                    M[row * kPitch + col] = row > col ? s.beta[row] * k_back[row] * D * kk[j][r] : 0.0f;
                    P[row * kPitch + col] = d.scale * q_back[row] * D * qk[j][r];
                }
        __syncthreads();
        {
            float x[16];
            const float* const A = M + 16 * w * (kPitch + 1);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float t = i == n ? 1.0f : 0.0f;
#pragma unroll
                for (int j = 0; j < i; ++j) t = fmaf(-A[i * kPitch + j], x[j], t);
                x[i] = t;
            }
            __syncthreads();
            if (lane < 16)
#pragma unroll
                for (int i = 0; i < 16; ++i) M[(16 * w + i) * kPitch + 16 * w + n] = x[i];
        }
        __syncthreads();
        auto tile = [&](int i, int j) { return *(const f32x4*)(M + (16 * i + n) * kPitch + 16 * j + 4 * g); };
        auto right = [&](int i, int j) { return col4(M, kPitch, 16 * i + 4 * g, 16 * j + n); };
        auto put = [&](int i, int j, f32x4 v) {
#pragma unroll
            for (int r = 0; r < 4; ++r) M[(16 * i + 4 * g + r) * kPitch + 16 * j + n] = -v[r];
        };
        if (w < 2) {
            const f32x4 x = mma(tile(2 * w + 1, 2 * w), right(2 * w, 2 * w), zero);
            put(2 * w + 1, 2 * w, mma(tile(2 * w + 1, 2 * w + 1), x, zero));
        }
        __syncthreads();
        f32x4 y2 = zero, y3 = zero;
        if (w < 2) {
            f32x4 x2 = zero, x3 = zero;
            for (int q = w; q < 2; ++q) {
                const f32x4 m = right(q, w);
                x2 = mma(tile(2, q), m, x2);
                x3 = mma(tile(3, q), m, x3);
            }
            y2 = mma(tile(2, 2), x2, zero);
            y3 = mma(tile(3, 3), x3, mma(tile(3, 2), x2, zero));
        }
        __syncthreads();
        if (w < 2) {
            put(2, w, y2);
            put(3, w, y3);
        }
        __syncthreads();
        f32x4 m[4], p[4];  // this thread's operands: pair w of all, pair 4 + w of the first two waves
        auto take = [&](int f, f32x4* to, const float* from) {
            const int at = (16 * pair_row(f) + n) * kPitch + 32 * pair_col(f) + 4 * g;
            to[0] = *(const f32x4*)(from + at);
            to[1] = *(const f32x4*)(from + at + 16);
        };
        take(w, m, M);
        take(w, p, P);
        if (w < 2) {
            take(4 + w, m + 2, M);
            take(4 + w, p + 2, P);
        } else {
            m[2] = m[3] = p[2] = p[3] = zero;
        }
        const float mm = over_column(over_lanes<16>(largest(m))), pm = over_column(over_lanes<16>(largest(p)));
        if (lane == 0) {
            most[0][w] = mm;
            most[1][w] = pm;
        }
        __syncthreads();
        const Scale ms(fmaxf(fmaxf(most[0][0], most[0][1]), fmaxf(most[0][2], most[0][3])));
        const Scale ps(fmaxf(fmaxf(most[1][0], most[1][1]), fmaxf(most[1][2], most[1][3])));
#pragma unroll
        for (int f = 0; f < 2; ++f)
            if (f == 0 || w < 2) {
                const int pair = 4 * f + w;
                auto put_planes = [&](f16* to, const Planes<2>& x) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) *(f16x8*)(to + (pair * 2 + k) * kPair + lane * 8) = x.p[k];
                };
                put_planes(out->M, split<2>(m[2 * f], m[2 * f + 1], ms.by));
                if constexpr (BACK) {
                    auto transposed = [&](const float* from, float scale) {
                        const int row = 32 * upper_col(pair) + 4 * g, col = 16 * upper_row(pair) + n;
                        return split<2>(col4(from, kPitch, row, col), col4(from, kPitch, row + 16, col), scale);
                    };
                    put_planes(out->MT, transposed(M, ms.by));
                    put_planes(out->PT, transposed(P, ps.by));
                } else {
                    put_planes(out->P, split<2>(p[2 * f], p[2 * f + 1], ps.by));
                }
            }
        if (w == 2) {
            if constexpr (BACK) {
                out->gamma[lane] = s.gamma[lane];
                out->end[lane] = s.end[lane];
                out->k_back[lane] = k_back[lane];
                out->q_back[lane] = q_back[lane];
            } else {
                out->gamma[lane] = s.gamma[lane] * k_back[lane];
                out->query[lane] = d.scale * s.gamma[lane] * q_back[lane];
                out->end[lane] = s.end[lane] * k_back[lane];
            }
            out->beta[lane] = s.beta[lane];
            out->misc[lane] = lane == 0 ? s.whole : lane == 1 ? ms.back : lane == 2 ? ps.back : s.ends[lane == 4];
        }
    }
}

// 16-byte pieces on their way from memory to LDS; the threads that have none of the last ones copy the last one too.
template <int BYTES, int THREADS>
struct Copy {
    static_assert(BYTES % 16 == 0, "whole pieces");
    static constexpr int PIECES = BYTES / 16, JOBS = (PIECES + THREADS - 1) / THREADS;
    f32x4 x[JOBS];
    __device__ __forceinline__ void load(const void* p) {
#pragma unroll
        for (int j = 0; j < JOBS; ++j)
            x[j] = at_bytes<const f32x4>((const char*)p, (uint32_t)min((int)threadIdx.x + j * THREADS, PIECES - 1) * 16u);
    }
    __device__ __forceinline__ void store(void* p) const {
#pragma unroll
        for (int j = 0; j < JOBS; ++j) ((f32x4*)p)[min((int)threadIdx.x + j * THREADS, PIECES - 1)] = x[j];
    }
};

template <int N>
__device__ __forceinline__ Planes<N> operand(const f16* m, int f, Lane l = Lane()) {
    Planes<N> x;
#pragma unroll
    for (int k = 0; k < N; ++k) x.p[k] = *(const f16x8*)(m + (f * N + k) * kPair + (16 * l.g + l.n) * 8);
    return x;
}

// c += A B over the steps, A a lower triangular matrix of a record, B two columns' planes.
template <int NA, int NB>
__device__ __forceinline__ void lower(const f16* m, const Planes<NB> (&B)[2], f32x4 (&c)[4], Lane l = Lane()) {
    const Planes<NA> A[4] = {operand<NA>(m, 0, l), operand<NA>(m, 1, l), operand<NA>(m, 2, l), operand<NA>(m, 4, l)};
    products(A, B[0], c);
    const Planes<NA> C[2] = {operand<NA>(m, 3, l), operand<NA>(m, 5, l)};
    products(C, B[1], c + 2);
}

// The same of an upper triangular one.
template <int NA, int NB>
__device__ __forceinline__ void upper(const f16* m, const Planes<NB> (&B)[2], f32x4 (&c)[4], Lane l = Lane()) {
    const Planes<NA> A[2] = {operand<NA>(m, 0, l), operand<NA>(m, 2, l)};
    products(A, B[0], c);
    const Planes<NA> C[4] = {operand<NA>(m, 1, l), operand<NA>(m, 3, l), operand<NA>(m, 4, l), operand<NA>(m, 5, l)};
    products(C, B[1], c);
}

// The dimension of the keys that row 4g + r of tile t of a state's column stands for.
__device__ __forceinline__ int key_row(int t, int g, int r) { return 32 * (t / 2) + 8 * g + 4 * (t & 1) + r; }

// A column of a state in registers: rows in the order of key_row, zero past the dimensions.
template <int KT>
struct Column {
    f32x4 t[KT];
    // of a matrix with `rows` rows of `pitch`
    static __device__ __forceinline__ uint32_t offset(int col, int pitch, Lane l) {
        return (uint32_t)(8 * l.g * pitch + col) * 4u;
    }
    __device__ __forceinline__ void load(const float* p, bool on, int col, int rows, int pitch, Lane l = Lane()) {
        const Buffer m(p, p ? rows * pitch * 4 : 0);
        const uint32_t off = on ? offset(col, pitch, l) : kNowhere;
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) t[k][r] = m.load<float>(off + key_row(k, 0, r) * pitch * 4);
    }
    __device__ __forceinline__ void store(float* p, bool on, int col, int rows, int pitch, float scale, Lane l = Lane()) const {
        const Buffer m(p, rows * pitch * 4);
        uint32_t off = on ? offset(col, pitch, l) : kNowhere;
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                m.store(off, t[k][r] * scale);
                off += ((k & 1) && r == 3 ? 25 : 1) * pitch * 4;
            }
    }
};

// A restart drops a state (its gradient) whatever it holds, and a product with a factor of 0 would not. Zeros the columns
// that are not finite, which are the bits (by lanes) of what it returns.
template <int KT>
__device__ __forceinline__ uint64_t drop(Column<KT>& S) {
    float x = 0.0f;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) x = fmaf(S.t[t][r], 0.0f, x);  // 0 or NaN
    uint64_t lost = __ballot(x != x);
    lost |= lost >> 32;
    lost = (lost | lost >> 16) & 0xffff;
    lost |= lost << 16;
    lost |= lost << 32;
    if (lost >> (threadIdx.x & 63) & 1)
#pragma unroll
        for (int t = 0; t < KT; ++t) S.t[t] = f32x4{0, 0, 0, 0};
    return lost;
}

// The values of a chunk in a column, as results lie: rows 16 t + 4g + r; p at the chunk's first row, rows from `rows`
// on are 0. (Where rows overlap, step < dim, the rows behind the last one may hold something of it instead, which
// their beta of 0 keeps out.)
template <typename T>
struct Values {
    uint32_t x[16];  // a register each: packed, they would be waited for where they are fetched
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (sizeof(T) == 2)
            return (float)__builtin_bit_cast(T, (uint16_t)x[e]);
        else
            return __uint_as_float(x[e]);
    }
    __device__ __forceinline__ void load(const T* p, int64_t step, int rows, bool on, int col, int dim, Lane l = Lane()) {
        const int by = (int)step * (int)sizeof(T);
        const Buffer m(p, (min(rows, kC) - 1) * by + dim * (int)sizeof(T));
        uint32_t off = on ? 4 * l.g * by + col * (uint32_t)sizeof(T) : kNowhere;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if constexpr (sizeof(T) == 2)
                x[e] = m.load<uint16_t>(off);
            else
                x[e] = m.load<uint32_t>(off);
            off += e % 4 == 3 ? 13 * by : by;
        }
    }
    // rows from `rows` on are 0, those from `all` on are not there
    static __device__ __forceinline__ void store(T* p, int64_t step, int rows, int all, bool on, int col, int dim, f32x4 (&v)[4],
                                                 Lane l = Lane()) {
        const int g = l.g, by = (int)step * (int)sizeof(T);
        if (rows < kC)
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e / 4][e % 4] = 16 * (e / 4) + 4 * g + e % 4 < rows ? v[e / 4][e % 4] : 0.0f;
        const Buffer m(p, (min(all, kC) - 1) * by + dim * (int)sizeof(T));
        uint32_t off = on ? 4 * g * by + col * (uint32_t)sizeof(T) : kNowhere;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            m.store(off, (T)v[e / 4][e % 4]);
            off += e % 4 == 3 ? 13 * by : by;
        }
    }
};

// Where there are few sequences and heads, a sequence is cut into segments that
// run side by side. A segment takes a state S to Phi S + B, so a first pass
// without outputs (OUT false) gives B (from a state of 0) and Phi (as columns
// of a state that starts as the identity, without values), a short walk over
// the segments (k_delta_join) the state in front of each, and the pass with
// outputs starts from those.
struct Segments {
    int count, chunks;  // of a sequence (at most 32); of a segment
    float* front;       // [b][h][segment][key_dim][value_dim] B, then the state in front
    float* phi;         // [b][h][segment][key_dim][key_dim]
    uint32_t* cut;      // [b][h][segment] whether it holds a restart, so that Phi is 0
};

// The states, chunk after chunk, 16 columns of the values a wave: S and
// what follows from it (R, U) never leave its registers, each product's result
// is the next one's right operand. What the waves share is fetched a chunk
// ahead. The columns of S are held scaled to at most about 1, S = unit * S.t.
// Bound by the splitting of states into planes and by LDS, from which every wave
// reads all operands of a chunk for its 16 columns (32 columns a wave would read
// half as much and spill): 4.9 us a chunk where a compute unit holds 64 columns
// (8 x 2048 steps of 16 heads: 159 us) and 7.4 where it holds 128 (8192 steps of
// 32 heads in 8 segments: 118 us), of which the matrix instructions are 0.9 and
// 1.8. (One plane of S, U and P for a bfloat16 o, 11 bits, took 144 and 104 us.)
template <typename T, int DK, int WAVES, bool OUT>
__global__ __launch_bounds__(64 * WAVES) void k_delta_chain(DeltaArgs a, int chunks, const Keys<kPlanes<T>, DK>* keys,
                                                               const Forward* records, Segments seg) {
    constexpr int NX = kPlanes<T>, KT = DK / 16, KS = DK / 32, kThreads = 64 * WAVES;
    typedef Operand<NX, DK> O;
    constexpr int KEYS = OUT ? sizeof(Keys<NX, DK>) : sizeof(Keys<NX, DK>) / 2;  // without outputs no queries
    __shared__ alignas(16) char kq[KEYS];
    __shared__ Forward rec;
    const f16* const K = (const f16*)kq;
    const f16* const Q = K + O::SIZE;
    const gs_delta_rule& d = a.r;
    const int b = blockIdx.x / d.heads, h = blockIdx.x % d.heads, kh = h / (d.heads / d.key_heads);
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
    // behind the values' columns, in workgroups of their own, those of Phi
    const int blocks = (d.value_dim + 16 * WAVES - 1) / (16 * WAVES);
    const bool values = OUT || (int)blockIdx.y < blocks;
    const int col0 = ((values ? blockIdx.y : blockIdx.y - blocks) * WAVES + w) * 16, col = col0 + n;
    const bool on = col < (values ? d.value_dim : d.key_dim);
    const int len = length_of(d, b), z = blockIdx.z;
    const int c0 = z * seg.chunks, c1 = min((len + kC - 1) / kC, c0 + seg.chunks);
    const int64_t size = (int64_t)d.key_dim * d.value_dim, head = (int64_t)b * d.heads + h;
    const T* const v = (const T*)a.v + b * d.v_batch + h * d.v_head;
    const int64_t o_step = (int64_t)d.heads * d.value_dim;
    T* const o = (T*)a.o + ((int64_t)b * d.steps * d.heads + h) * d.value_dim;
    const Forward* const first = records + (int64_t)b * chunks * d.heads + h;
    const Keys<NX, DK>* const first_keys = keys + (int64_t)b * chunks * d.key_heads + kh;
    Column<KT> S;
    float unit = 1.0f;
    if constexpr (OUT) {
        const float* const from = seg.count > 1 ? seg.front + (head * seg.count + z) * size : a.h0 ? a.h0 + head * size : nullptr;
        S.load(from, on, col, d.key_dim, d.value_dim);
    } else {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) S.t[t][r] = !values && key_row(t, g, r) == col ? 1.0f : 0.0f;
    }
    Copy<KEYS, kThreads> fk;
    Copy<sizeof(Forward), kThreads> fr;
    Values<T> fv;
    auto fetch = [&](int c) {
        const int t0 = c * kC;
        fr.load(first + (int64_t)c * d.heads);
        fk.load(first_keys + (int64_t)c * d.key_heads);
        __builtin_amdgcn_sched_barrier(0);  // the values last: when they are there, so is the rest
        if (values) fv.load(v + t0 * d.v_step, d.v_step, len - t0, on, col, d.value_dim);
    };
    // The values are taken over before the chunk's stores: behind them they would be waited for together.
    f32x4 V[4];
    auto take = [&] {
#pragma unroll
        for (int e = 0; e < 16; ++e) V[e / 4][e % 4] = values ? fv[e] : 0.0f;
    };
    if (c0 < c1) {
        fetch(c0);
        take();
    }
    const f32x4 zero = {0, 0, 0, 0};
    [[maybe_unused]] bool cut = false;
    for (int c = c0; c < c1; ++c) {
        const Lane l = Lane::here();
        const int g = l.g, col = col0 + l.n;
        const int t0 = c * kC;
        __syncthreads();
        fr.store(&rec);
        fk.store(kq);
        __syncthreads();
        if (c + 1 < c1) fetch(c + 1);
        f32x4 R[4] = {zero, zero, zero, zero}, y[4] = {zero, zero, zero, zero};  // K S, then R; Q S, then O
        uint64_t lost = 0;  // columns that are not finite, in a chunk with a restart
        if (rec.misc[3] < (float)kC) {
            lost = drop(S);
            cut = true;
        }
        const float top = over_column(largest(S.t));
        const Scale big(top);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const Planes<2> sp = split<2>(S.t[2 * s], S.t[2 * s + 1], big.by);
            Planes<NX> A[4];
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) A[ti] = O::row(K, ti, s, l);
            products(A, sp, R);
            if constexpr (OUT) {
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) A[ti] = O::row(Q, ti, s, l);
                products(A, sp, y);
            }
        }
        const float from = unit * big.back;
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) {
            const f32x4 gamma = *(const f32x4*)(rec.gamma + 16 * ti + 4 * g), beta = *(const f32x4*)(rec.beta + 16 * ti + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                R[ti][r] = beta[r] * fmaf(-gamma[r] * from, R[ti][r], V[ti][r]);
            if constexpr (OUT) {
                const f32x4 query = *(const f32x4*)(rec.query + 16 * ti + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) y[ti][r] *= query[r] * from;
            }
        }
        f32x4 U[4] = {zero, zero, zero, zero};
        {
            const Scale rs(over_column(largest(R)));
            const Planes<2> B[2] = {split<2>(R[0], R[1], rs.by), split<2>(R[2], R[3], rs.by)};
            lower<2>(rec.M, B, U, l);
            const float back = rs.back * rec.misc[1];
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) U[ti] *= back;
        }
        if constexpr (OUT) {
            const Scale us(over_column(largest(U)));
            const Planes<2> B[2] = {split<2>(U[0], U[1], us.by), split<2>(U[2], U[3], us.by)};
            f32x4 x[4] = {zero, zero, zero, zero};
            lower<2>(rec.P, B, x, l);
            const float back = us.back * rec.misc[2];
#pragma unroll
            for (int ti = 0; ti < 4; ++ti)
#pragma unroll
                for (int r = 0; r < 4; ++r) y[ti][r] = fmaf(x[ti][r], back, y[ti][r]);
            take();
            if (lost >> lane & 1)  // they end with the step in front of the restart
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if ((float)(16 * (e / 4) + 4 * g + e % 4) < rec.misc[3]) y[e / 4][e % 4] = __builtin_nanf("");
            Values<T>::store(o + t0 * o_step, o_step, len - t0, d.steps - t0, on, col, d.value_dim, y, l);
        }
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) U[ti] *= *(const f32x4*)(rec.end + 16 * ti + 4 * g);
        if constexpr (!OUT) take();
        // one scale for what is kept of S and what is added; a column of zeros, which keeps nothing, has no part in it
        const float whole = top == 0.0f ? 0.0f : rec.misc[0] * unit;
        const Scale es(fmaxf(over_column(largest(U)), whole * big.back));
        const float keep = whole * es.by;
#pragma unroll
        for (int t = 0; t < KT; ++t) S.t[t] *= keep;
        unit = es.back;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const Planes<2> up = split<2>(U[2 * p], U[2 * p + 1], es.by);
#pragma unroll
            for (int s = 0; s < KS; s += 2) {
                const Planes<NX> A[4] = {O::column(K, s, 0, p, l), O::column(K, s, 1, p, l), O::column(K, s + 1, 0, p, l), O::column(K, s + 1, 1, p, l)};
                products(A, up, S.t + 2 * s);
            }
        }
        if (OUT && a.ckpt && t0 + kC < len)
            S.store(a.ckpt + (((int64_t)b * (chunks - 1) + c) * d.heads + h) * size, on, col, d.key_dim, d.value_dim, unit, l);
    }
    if constexpr (OUT) {
        // the steps of the segment that are padding behind its last chunk
        const int end = z + 1 < seg.count ? min((c0 + seg.chunks) * kC, d.steps) : d.steps;
        if (on)
            for (int t = max(c0, c1) * kC + g; t < end; t += 4) o[t * o_step + col] = (T)0.0f;
        if (a.h_last && z + 1 == seg.count) S.store(a.h_last + head * size, on, col, d.key_dim, d.value_dim, unit);
    } else {
        const int64_t at = head * seg.count + z;
        S.store(values ? seg.front + at * size : seg.phi + at * d.key_dim * d.key_dim, on, col, d.key_dim,
                values ? d.value_dim : d.key_dim, unit);
        if (blockIdx.y == 0 && threadIdx.x == 0) seg.cut[at] = cut;
    }
}

// The state in front of every segment, in place of its B: S <- Phi S + B from
// segment to segment (`back`: from the last to the first, the gradient behind), 16 columns a workgroup and 16 rows a wave, on the float32
// matrix instructions. Bound by the latency of a step (2.3 us; its products are
// 0.9): Phi is fetched three steps ahead. 4 heads of 32 segments: 72 us.
template <int DK>
__global__ __launch_bounds__(DK * 4) void k_delta_join(DeltaArgs a, Segments seg, const float* start, bool back) {
    constexpr int KT = DK / 16, PITCH = DK + 4, AHEAD = 4;
    __shared__ float L[2][16 * PITCH];  // S by columns
    const gs_delta_rule& d = a.r;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
    const int col = blockIdx.y * 16 + n, row = 16 * w + 4 * g, left = 16 * w + n;
    const int64_t head = blockIdx.x;
    const int size = d.key_dim * d.value_dim, square = d.key_dim * d.key_dim;
    float* const front = seg.front + head * seg.count * size;
    const float* const phi = seg.phi + head * seg.count * square;
    const uint32_t at = col < d.value_dim ? (uint32_t)(row * d.value_dim + col) * 4u : kNowhere;
    const uint32_t from = (uint32_t)(left * d.key_dim + 4 * g) * 4u;
    f32x4 A[AHEAD][KT], B[AHEAD], S;
    // What is read past a row's end meets rows of S that are 0.
    auto place = [&](int z) { return (int64_t)(back ? seg.count - 1 - z : z); };
    auto fetch = [&](int z, f32x4 (&x)[KT], f32x4& y) {
        const Buffer p(phi + place(z) * square, square * 4), f(front + place(z) * size, size * 4);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
            x[kt] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(p.r, from + 64 * kt, 0, 0));
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = f.load<float>(at + r * d.value_dim * 4);
    };
    // bit z: a restart in segment place(z) drops what S holds
    const uint64_t cuts = __ballot(lane < seg.count && seg.cut[head * seg.count + place(min(lane, seg.count - 1))]);
    {
        const Buffer h(start + head * size, start ? size * 4 : 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) S[r] = h.load<float>(at + r * d.value_dim * 4);
    }
#pragma unroll
    for (int x = 0; x + 1 < AHEAD; ++x)
        if (x < seg.count) fetch(x, A[x], B[x]);
    for (int z = 0; z < seg.count; z += AHEAD)
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) {
            if (z + x >= seg.count) break;
            if (z + x + AHEAD - 1 < seg.count) fetch(z + x + AHEAD - 1, A[(x + AHEAD - 1) % AHEAD], B[(x + AHEAD - 1) % AHEAD]);
            float* const s = L[x & 1];
            *(f32x4*)(s + n * PITCH + row) = S;
            __syncthreads();
            const Buffer f(front + place(z + x) * size, size * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) f.store(at + r * d.value_dim * 4, S[r]);
            if (cuts >> (z + x) & 1) {
                S = B[x];
                continue;
            }
            f32x4 acc[2] = {B[x], {0, 0, 0, 0}};
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) acc[kt & 1] = mma(A[x][kt], *(const f32x4*)(s + n * PITCH + 16 * kt + 4 * g), acc[kt & 1]);
            S = acc[0] + acc[1];
        }
}

// The gradients of the states, from the last chunk to the first, 16 columns a
// wave, held and scaled as the states of k_delta_chain; behind[b][chunk][h]
// receives the one behind each chunk. Bound as k_delta_chain: 5.2 us a chunk
// (8 x 2048 steps of 16 heads of 128: 167 us). In segments as it is: the
// gradient in front of a segment is Phi^T of that behind it and a B of its own.
template <typename T, int DK, int WAVES, bool OUT>
__global__ __launch_bounds__(64 * WAVES) void k_delta_back(DeltaArgs a, int chunks, const Keys<kPlanes<T>, DK>* keys,
                                                               const Backward* records, float* behind, Segments seg) {
    constexpr int NX = kPlanes<T>, KT = DK / 16, KS = DK / 32, kThreads = 64 * WAVES;
    typedef Operand<NX, DK> O;
    __shared__ Keys<NX, DK> kq;
    // of a record: all but M
    constexpr int SKIP = sizeof(Backward::M);
    __shared__ alignas(16) char part[sizeof(Backward) - SKIP];
    const Backward& rec = *(const Backward*)(part - SKIP);
    const gs_delta_rule& d = a.r;
    const int b = blockIdx.x / d.heads, h = blockIdx.x % d.heads, kh = h / (d.heads / d.key_heads);
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
    // behind the values' columns, in workgroups of their own, those of Phi^T
    const int blocks = (d.value_dim + 16 * WAVES - 1) / (16 * WAVES);
    const bool values = OUT || (int)blockIdx.y < blocks;
    const int col0 = ((values ? blockIdx.y : blockIdx.y - blocks) * WAVES + w) * 16, col = col0 + n;
    const bool on = col < (values ? d.value_dim : d.key_dim);
    const int len = length_of(d, b), z = blockIdx.z;
    const int c0 = z * seg.chunks, c1 = min((len + kC - 1) / kC, c0 + seg.chunks);
    const int64_t size = (int64_t)d.key_dim * d.value_dim, head = (int64_t)b * d.heads + h;
    const int64_t o_step = (int64_t)d.heads * d.value_dim, first_o = ((int64_t)b * d.steps * d.heads + h) * d.value_dim;
    const T* const go = (const T*)a.grad_o + first_o;
    T* const gv = (T*)a.grad_v + first_o;
    const Backward* const first = records + (int64_t)b * chunks * d.heads + h;
    const Keys<NX, DK>* const first_keys = keys + (int64_t)b * chunks * d.key_heads + kh;
    Column<KT> S;
    float unit = 1.0f;
    if constexpr (OUT) {
        const float* const from = seg.count > 1 ? seg.front + (head * seg.count + z) * size
                                  : a.grad_last ? a.grad_last + head * size : nullptr;
        S.load(from, on, col, d.key_dim, d.value_dim);
        // the steps of the segment that are padding behind its last chunk
        const int end = z + 1 < seg.count ? min((c0 + seg.chunks) * kC, d.steps) : d.steps;
        if (on)
            for (int t = max(c0, c1) * kC + g; t < end; t += 4) gv[t * o_step + col] = (T)0.0f;
    } else {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) S.t[t][r] = !values && key_row(t, g, r) == col ? 1.0f : 0.0f;
    }
    Copy<sizeof(Keys<NX, DK>), kThreads> fk;
    Copy<sizeof(Backward) - SKIP, kThreads> fr;
    Values<T> fo;
    auto fetch = [&](int c) {
        const int t0 = c * kC;
        fr.load((const char*)(first + (int64_t)c * d.heads) + SKIP);
        fk.load(first_keys + (int64_t)c * d.key_heads);
        __builtin_amdgcn_sched_barrier(0);  // the values last: when they are there, so is the rest
        if (values) fo.load(go + t0 * o_step, o_step, len - t0, on, col, d.value_dim);
    };
    // taken over before a chunk's stores, with which they would be waited for
    f32x4 next[4];
    auto take = [&] {
#pragma unroll
        for (int e = 0; e < 16; ++e) next[e / 4][e % 4] = values ? fo[e] : 0.0f;
    };
    if (c0 < c1) {
        fetch(c1 - 1);
        take();
    }
    const f32x4 zero = {0, 0, 0, 0};
    [[maybe_unused]] bool cut = false;
    for (int c = c1 - 1; c >= c0; --c) {
        const Lane l = Lane::here();
        const int g = l.g, col = col0 + l.n;
        const int t0 = c * kC;
        if constexpr (OUT)
            S.store(behind + (((int64_t)b * chunks + c) * d.heads + h) * size, on, col, d.key_dim, d.value_dim, unit, l);
        __syncthreads();
        fr.store(part);
        fk.store(&kq);
        f32x4 dO[4] = {next[0], next[1], next[2], next[3]};
        __syncthreads();
        if (c > c0) fetch(c - 1);
        const float top = over_column(largest(S.t));
        const Scale big(top);
        f32x4 dU[4] = {zero, zero, zero, zero}, x[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const Planes<2> sp = split<2>(S.t[2 * s], S.t[2 * s + 1], big.by);
            Planes<NX> A[4];
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) A[ti] = O::row(kq.K, ti, s, l);
            products(A, sp, dU);
        }
        // as in k_delta_chain; where an element is not finite, so are all sums of its column (one of its planes is NaN)
        const bool restart = rec.misc[3] < (float)kC;
        const uint64_t lost = __ballot(restart && !finite(dU[0][0]));
        cut |= restart;
        if (lost) {
            const bool mine = lost >> lane & 1;
#pragma unroll
            for (int ti = 0; ti < 4; ++ti)
                if (mine) dU[ti] = zero;
#pragma unroll
            for (int t = 0; t < KT; ++t)
                if (mine) S.t[t] = zero;
        }
        {
            const Scale os(over_column(largest(dO)));
            const Planes<NX> B[2] = {split<NX>(dO[0], dO[1], os.by), split<NX>(dO[2], dO[3], os.by)};
            upper<2>(rec.PT, B, x, l);
            const float back = os.back * rec.misc[2], from = unit * big.back;
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                const f32x4 end = *(const f32x4*)(rec.end + 16 * ti + 4 * g), kb = *(const f32x4*)(rec.k_back + 16 * ti + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) dU[ti][r] = fmaf(end[r] * kb[r] * from, dU[ti][r], back * x[ti][r]);
            }
        }
        f32x4 dR[4] = {zero, zero, zero, zero};
        {
            const Scale us(over_column(largest(dU)));
            const Planes<2> B[2] = {split<2>(dU[0], dU[1], us.by), split<2>(dU[2], dU[3], us.by)};
            upper<2>(rec.MT, B, dR, l);
            const float back = us.back * rec.misc[1];
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                const f32x4 beta = *(const f32x4*)(rec.beta + 16 * ti + 4 * g), gamma = *(const f32x4*)(rec.gamma + 16 * ti + 4 * g);
                const f32x4 kb = *(const f32x4*)(rec.k_back + 16 * ti + 4 * g), qb = *(const f32x4*)(rec.q_back + 16 * ti + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[ti][r] = beta[r] * back * dR[ti][r];  // dV
                    dR[ti][r] = -gamma[r] * kb[r] * x[ti][r];
                    dO[ti][r] *= d.scale * gamma[r] * qb[r];
                }
            }
        }
        take();
        if (OUT && (lost >> lane & 1))
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if ((float)(16 * (e / 4) + 4 * g + e % 4) >= rec.misc[4]) x[e / 4][e % 4] = __builtin_nanf("");
        if constexpr (OUT)
            Values<T>::store(gv + t0 * o_step, o_step, len - t0, d.steps - t0, on, col, d.value_dim, x, l);
        const float whole = top == 0.0f ? 0.0f : rec.misc[0] * unit;  // as in k_delta_chain
        const Scale es(fmaxf(over_column(fmaxf(largest(dO), largest(dR))), whole * big.back));
        const float keep = whole * es.by;
#pragma unroll
        for (int t = 0; t < KT; ++t) S.t[t] *= keep;
        unit = es.back;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const Planes<2> op = split<2>(dO[2 * p], dO[2 * p + 1], es.by), rp = split<2>(dR[2 * p], dR[2 * p + 1], es.by);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Planes<NX> A[2] = {O::column(kq.Q, s, 0, p, l), O::column(kq.Q, s, 1, p, l)};
                products(A, op, S.t + 2 * s);
                const Planes<NX> B[2] = {O::column(kq.K, s, 0, p, l), O::column(kq.K, s, 1, p, l)};
                products(B, rp, S.t + 2 * s);
            }
        }
    }
    if constexpr (OUT) {
        if (a.grad_h0 && z == 0) S.store(a.grad_h0 + head * size, on, col, d.key_dim, d.value_dim, unit);
    } else {
        const int64_t at = head * seg.count + z;
        S.store(values ? seg.front + at * size : seg.phi + at * d.key_dim * d.key_dim, on, col, d.key_dim,
                values ? d.value_dim : d.key_dim, unit);
        if (blockIdx.y == 0 && threadIdx.x == 0) seg.cut[at] = cut;
    }
}

constexpr int kGradWaves = 8;
constexpr int kV = GS_DELTA_MAX_DIM;

// The gradients of a chunk's queries, keys and gates from the states in front
// and the gradients behind, for all heads of a key head, one after another.
// First a wave takes 16 columns of the values (U and dR, to LDS), then 16 of
// the keys. Of float32 inputs, on the float32 matrix instructions: their two
// planes with those of U, dR and the states would not fit LDS. 3 x 777 steps of
// 5 heads of 96 x 80: 71 us.
template <typename T, int DK>
__global__ __launch_bounds__(64 * kGradWaves) void k_delta_grad(DeltaArgs a, int chunks, const float* inverse, const float* behind) {
    constexpr int KT = DK / 16, kThreads = 64 * kGradWaves;
    __shared__ float K[kC * (DK + 4)];
    __shared__ float U[kC * (kV + 4)];
    __shared__ float E[kC * (kV + 4)];   // dR
    __shared__ float P[kC * kPitch];     // P, then Pd
    __shared__ float A[kC * kPitch];     // Ad
    __shared__ float X[kC * (kC + 1)];
    __shared__ float betas[kGradWaves][kC], front[kGradWaves][kC], after[kGradWaves][kC], dots[kGradWaves];
    __shared__ float spoilt[2][kGradWaves];  // not finite where a restart drops such a state, or gradient, of a wave
    __shared__ Chunk s;
    const gs_delta_rule& d = a.r;
    const int kh = blockIdx.x % d.key_heads, c = blockIdx.x / d.key_heads % chunks, b = blockIdx.x / d.key_heads / chunks;
    const int w = threadIdx.x >> 6;
    const int len = length_of(d, b), t0 = c * kC, rows = len - t0, group = d.heads / d.key_heads;
    const int64_t first = (((int64_t)b * d.steps + t0) * d.key_heads + kh) * d.key_dim;
    T* const gq = (T*)a.grad_q + first;
    T* const gk = (T*)a.grad_k + first;
    const int64_t k_step = (int64_t)d.key_heads * d.key_dim, o_step = (int64_t)d.heads * d.value_dim;
    const int all = min(kC, d.steps - t0);  // steps of the chunk, padding included
    if (rows <= 0) {
        for (int e = threadIdx.x; e < all * d.key_dim; e += kThreads) {
            const int64_t at = e / d.key_dim * k_step + e % d.key_dim;
            gq[at] = gk[at] = (T)0.0f;
        }
        for (int e = threadIdx.x; e < all * group; e += kThreads) {
            const int64_t at = ((int64_t)b * d.steps + t0 + e / group) * d.heads + kh * group + e % group;
            a.grad_log_decay[at] = a.grad_beta[at] = 0.0f;
        }
        return;
    }
    const T* const q = (const T*)a.q + b * d.q_batch + t0 * d.q_step + kh * d.q_head;
    const T* const k = (const T*)a.k + b * d.k_batch + t0 * d.k_step + kh * d.k_head;
    const int qs = (int)d.q_step * (int)sizeof(T);
    const Buffer queries(q, (min(rows, kC) - 1) * qs + d.key_dim * (int)sizeof(T));
    auto four = [](const Buffer& m, uint32_t off, int left) {  // elements from `left` on are 0
        const f32x4 x = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(m.r, off, 0, 0));
        return f32x4{left > 0 ? x[0] : 0.0f, left > 1 ? x[1] : 0.0f, left > 2 ? x[2] : 0.0f, left > 3 ? x[3] : 0.0f};
    };
    auto q4 = [&](int row, int at) { return four(queries, row < rows ? row * qs + at * 4 : kNowhere, d.key_dim - at); };
    auto qcol = [&](int row, int at) {
        f32x4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = queries.load<float>(row + r < rows && at < d.key_dim ? (row + r) * qs + at * 4 : kNowhere);
        return x;
    };
    load_rows<DK>(k, d.k_step, rows, d.key_dim, K, kThreads);
    const f32x4 zero = {0, 0, 0, 0};
    f32x4 dq[4], dk[4];
#pragma unroll
    for (int ti = 0; ti < 4; ++ti) dq[ti] = dk[ti] = zero;
    for (int hh = 0; hh < group; ++hh) {
        const Lane l = Lane::here();
        const int n = l.n, g = l.g, lane = 16 * g + n;
        const int h = kh * group + hh;
        const int64_t size = (int64_t)d.key_dim * d.value_dim, head = (int64_t)b * d.heads + h;
        const float* const S0 = c == 0 ? (a.h0 ? a.h0 + head * size : nullptr)
                                       : a.ckpt_in + (((int64_t)b * (chunks - 1) + c - 1) * d.heads + h) * size;
        const float* const dS = behind + (((int64_t)b * chunks + c) * d.heads + h) * size;
        const float* const M = inverse + ((int64_t)(b * chunks + c) * d.heads + h) * kLower;
        const T* const v = (const T*)a.v + b * d.v_batch + t0 * d.v_step + h * d.v_head;
        const T* const go = (const T*)a.grad_o + (((int64_t)b * d.steps + t0) * d.heads + h) * d.value_dim;
        const Buffer front_state(S0, S0 ? (int)size * 4 : 0), behind_state(dS, (int)size * 4);
        const int os = (int)o_step * (int)sizeof(T);
        const Buffer upstream(go, (min(rows, kC) - 1) * os + d.value_dim * (int)sizeof(T));
        __syncthreads();
        if (w == 0) load_gates(a, b, h, t0, len, s);
        __syncthreads();
        for (int p = w; p < kTiles; p += kGradWaves) {
            const int ti = p >= 6 ? 3 : p >= 3 ? 2 : p >= 1 ? 1 : 0, tj = p - tri(ti, 0);
            f32x4 acc = zero;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
                acc = mma(q4(16 * ti + n, 16 * kt + 4 * g), row4<DK>(K, 16 * tj + n, 16 * kt + 4 * g), acc);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * ti + 4 * g + r, j = 16 * tj + n;
                P[i * kPitch + j] = i >= j ? d.scale * decay(s, i, j) * acc[r] : 0.0f;
            }
        }
        __syncthreads();
        {
            const int col = 16 * w + n;
            const bool on = col < d.value_dim;
            f32x4 S[KT], Z[KT];
            float dot = 0.0f;
            Values<T> vals, ups;
            vals.load(v, d.v_step, rows, on, col, d.value_dim, l);
            ups.load(go, o_step, rows, on, col, d.value_dim, l);
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t off = on ? ((16 * kt + 4 * g + r) * d.value_dim + col) * 4 : kNowhere;
                    S[kt][r] = front_state.load<float>(off);
                    Z[kt][r] = behind_state.load<float>(off);
                    dot = fmaf(S[kt][r], Z[kt][r], dot);
                }
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) dot += __shfl_xor(dot, m);
            if (lane == 0) dots[w] = dot;
            f32x4 R[4], e[4], dO[4], dU[4], dR[4], u[4];
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                f32x4 x = zero, y = zero;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const f32x4 kk = row4<DK>(K, 16 * ti + n, 16 * kt + 4 * g);
                    x = mma(kk, S[kt], x);
                    y = mma(kk, Z[kt], y);
                }
                // as in the chains
                const bool cut = s.seg[kC - 1] != 0, s_lost = cut && !finite(x[0]), z_lost = cut && !finite(y[0]);
                if (ti == 0) {
                    spoilt[0][w] = __ballot(s_lost) ? __builtin_nanf("") : 0.0f;
                    spoilt[1][w] = __ballot(z_lost) ? __builtin_nanf("") : 0.0f;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = 16 * ti + 4 * g + r;
                    e[ti][r] = vals[4 * ti + r] - (s_lost ? 0.0f : s.gamma[i] * x[r]);
                    R[ti][r] = s.beta[i] * e[ti][r];
                    dO[ti][r] = ups[4 * ti + r];
                    dU[ti][r] = z_lost ? 0.0f : s.end[i] * y[r];
                }
            }
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                u[ti] = zero;
#pragma unroll
                for (int tj = 0; tj <= ti; ++tj)
                    u[ti] = mma(*(const f32x4*)(M + tri(ti, tj) * 256 + n * 16 + 4 * g), R[tj], u[ti]);
#pragma unroll
                for (int tj = ti; tj < 4; ++tj) dU[ti] = mma(col4(P, kPitch, 16 * tj + 4 * g, 16 * ti + n), dO[tj], dU[ti]);
            }
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                dR[ti] = zero;
#pragma unroll
                for (int tj = ti; tj < 4; ++tj) dR[ti] = mma(col4(M + tri(tj, ti) * 256 + 64 * g + n, 16, 0, 0), dU[tj], dR[ti]);
            }
#pragma unroll
            for (int ti = 0; ti < 4; ++ti)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = 16 * ti + 4 * g + r;
                    U[i * (kV + 4) + col] = u[ti][r];
                    E[i * (kV + 4) + col] = dR[ti][r];
                    float t = dR[ti][r] * e[ti][r];
#pragma unroll
                    for (int m = 1; m < 16; m <<= 1) t += __shfl_xor(t, m);
                    if (n == 0) betas[w][i] = t;
                }
        }
        __syncthreads();
        auto o4 = [&](int row, int at) { return four(upstream, row < rows ? row * os + at * 4 : kNowhere, d.value_dim - at); };
        const int vt = (d.value_dim + 15) / 16;
        float part[2][4] = {};  // of the gradient of beta, from the tiles of this wave
        for (int p = w, turn = 0; p < kTiles; p += kGradWaves, ++turn) {
            const int ti = p >= 6 ? 3 : p >= 3 ? 2 : p >= 1 ? 1 : 0, tj = p - tri(ti, 0);
            f32x4 dp = zero, da = zero, qk = zero, kk = zero;
            for (int ct = 0; ct < vt; ++ct) {
                const f32x4 u = row4<kV>(U, 16 * tj + n, 16 * ct + 4 * g);
                dp = mma(o4(16 * ti + n, 16 * ct + 4 * g), u, dp);
                da = mma(row4<kV>(E, 16 * ti + n, 16 * ct + 4 * g), u, da);
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const f32x4 x = row4<DK>(K, 16 * tj + n, 16 * kt + 4 * g);
                qk = mma(q4(16 * ti + n, 16 * kt + 4 * g), x, qk);
                kk = mma(row4<DK>(K, 16 * ti + n, 16 * kt + 4 * g), x, kk);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * ti + 4 * g + r, j = 16 * tj + n;
                const float D = i >= j ? decay(s, i, j) : 0.0f;
                const float pd = d.scale * D * dp[r], ad = i > j ? -D * da[r] : 0.0f;
                P[i * kPitch + j] = pd;
                A[i * kPitch + j] = s.beta[i] * ad;
                X[i * (kC + 1) + j] = pd * qk[r] + s.beta[i] * ad * kk[r];
                float t = ad * kk[r];
#pragma unroll
                for (int m = 1; m < 16; m <<= 1) t += __shfl_xor(t, m);
                part[turn][r] = t;
            }
        }
        f32x4 aq[4], ar[4], au[4];
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) aq[ti] = ar[ti] = au[ti] = zero;
        const int row = 16 * w + n;  // of the keys
        if (w < KT) {
            for (int ct = 0; ct < vt; ++ct) {
                const int at = 16 * ct + 4 * g;
                const uint32_t off = row < d.key_dim ? (row * d.value_dim + at) * 4 : kNowhere;
                const f32x4 x = four(front_state, off, d.value_dim - at), y = four(behind_state, off, d.value_dim - at);
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                    aq[ti] = mma(o4(16 * ti + n, 16 * ct + 4 * g), x, aq[ti]);
                    ar[ti] = mma(row4<kV>(E, 16 * ti + n, 16 * ct + 4 * g), x, ar[ti]);
                    au[ti] = mma(row4<kV>(U, 16 * ti + n, 16 * ct + 4 * g), y, au[ti]);
                }
            }
        }
        __syncthreads();
        // what tile (ti, tj) adds to the gradient of beta: rows of ti, in the order of tj, behind the values' part
        for (int q = 0; q < kTiles; ++q) {
            if (q % kGradWaves == w && n == 0) {
                const int ti = q >= 6 ? 3 : q >= 3 ? 2 : q >= 1 ? 1 : 0;
#pragma unroll
                for (int r = 0; r < 4; ++r) betas[0][16 * ti + 4 * g + r] += part[q / kGradWaves][r];
            }
            __syncthreads();
        }
        if (w < KT) {
            if (s.seg[kC - 1]) {  // a restart drops the state and the gradient whatever they hold
                float s_spoilt = 0.0f, z_spoilt = 0.0f;
                for (int i = 0; i < kGradWaves; ++i) {
                    s_spoilt += spoilt[0][i];
                    z_spoilt += spoilt[1][i];
                }
#pragma unroll
                for (int ti = 0; ti < 4; ++ti)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int seg = s.seg[16 * ti + 4 * g + r];
                        aq[ti][r] = seg == 0 ? aq[ti][r] + s_spoilt : 0.0f;
                        ar[ti][r] = seg == 0 ? ar[ti][r] + s_spoilt : 0.0f;
                        au[ti][r] = seg == s.seg[kC - 1] ? au[ti][r] + z_spoilt : 0.0f;
                    }
            }
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                f32x4 x, y, fr, af;
                const f32x4 qq = qcol(16 * ti + 4 * g, row), kk = col4(K, DK + 4, 16 * ti + 4 * g, row);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = 16 * ti + 4 * g + r;
                    x[r] = d.scale * s.gamma[i] * aq[ti][r];
                    const float m = s.beta[i] * s.gamma[i] * ar[ti][r], z = s.end[i] * au[ti][r];
                    y[r] = z - m;
                    fr[r] = qq[r] * x[r] - kk[r] * m;
                    af[r] = kk[r] * z;
#pragma unroll
                    for (int t = 1; t < 16; t <<= 1) {
                        fr[r] += __shfl_xor(fr[r], t);
                        af[r] += __shfl_xor(af[r], t);
                    }
                    if (n == 0) {
                        front[w][i] = fr[r];
                        after[w][i] = af[r];
                    }
                }
#pragma unroll
                for (int tj = 0; tj < 4; ++tj) {
                    const f32x4 k4 = col4(K, DK + 4, 16 * tj + 4 * g, row);
                    if (tj <= ti) {
                        x = mma(*(const f32x4*)(P + (16 * ti + n) * kPitch + 16 * tj + 4 * g), k4, x);
                        y = mma(*(const f32x4*)(A + (16 * ti + n) * kPitch + 16 * tj + 4 * g), k4, y);
                    }
                    if (tj >= ti) {
                        y = mma(col4(P, kPitch, 16 * tj + 4 * g, 16 * ti + n), qcol(16 * tj + 4 * g, row), y);
                        y = mma(col4(A, kPitch, 16 * tj + 4 * g, 16 * ti + n), k4, y);
                    }
                }
                dq[ti] += x;
                dk[ti] += y;
            }
        }
        // X: sums over j < t of every row, in place
        if (w == kGradWaves - 1) {
            float t = 0.0f;
            for (int j = 0; j < lane; ++j) {
                const float x = X[lane * (kC + 1) + j];
                X[lane * (kC + 1) + j] = t;
                t += x;
            }
            X[lane * (kC + 1) + lane] = t;
        }
        __syncthreads();
        if (w == 0) {
            float f = 0.0f, af = 0.0f, be = 0.0f, dot = 0.0f;
            for (int x = 0; x < kGradWaves; ++x) {
                be += betas[x][lane];
                dot += dots[x];
            }
            for (int x = 0; x < KT; ++x) {
                f += front[x][lane];
                af += after[x][lane];
            }
            be += 0.0f * f + 0.0f * af;  // as in k_delta_grads
            float all_f = f, all_a = af;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const float p = __shfl_down(all_f, m), o = __shfl_up(all_a, m);
                if (lane + m < 64) all_f += p;
                if (lane >= m) all_a += o;
            }
            all_a = __shfl_up(all_a, 1);
            float t = 0.0f;
            for (int i = lane; i < kC; ++i) t += X[i * (kC + 1) + lane];
            t += all_f + (lane ? all_a : 0.0f) + (s.seg[kC - 1] ? 0.0f : s.whole * dot);
            if (lane < all) {
                const int64_t at = ((int64_t)b * d.steps + t0 + lane) * d.heads + h;
                const bool live = lane < rows;
                // the decay of a restart is not applied
                const bool cut = lane ? s.seg[lane] != s.seg[lane - 1] : s.seg[0] != 0;
                a.grad_log_decay[at] = live && !cut ? t : 0.0f;
                a.grad_beta[at] = live ? be : 0.0f;
            }
        }
    }
    const int n = threadIdx.x & 15, g = threadIdx.x >> 4 & 3, row = 16 * w + n;
    if (w < KT && row < d.key_dim)
#pragma unroll
        for (int ti = 0; ti < 4; ++ti)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * ti + 4 * g + r;
                if (i < all) {
                    gq[i * k_step + row] = (T)(i < rows ? dq[ti][r] : 0.0f);
                    gk[i * k_step + row] = (T)(i < rows ? dk[ti][r] : 0.0f);
                }
            }
}

// 16-bit matrices by columns: rows of 64 (steps), 16-byte pieces swizzled by the
// row, PLANE elements from plane to plane. Results of products are written in
// groups of four steps; read as operands with lanes along the steps (turned) or
// along the rows.
template <int ROWS>
struct Turned {
    static constexpr int PLANE = ROWS * kC;
    static __device__ __forceinline__ int at(int row, int piece) { return row * kC + (piece ^ (row & 7)) * 8; }
    // steps 16 tile + 4g .. of a row
    static __device__ __forceinline__ void write(f16* m, int row, int tile, f32x4 v, float scale, Lane l = Lane()) {
        const int g = l.g;
        f16* const to = m + at(row, 2 * tile + g / 2) + (g & 1) * 4;
        const f16x2 a = __builtin_convertvector(f32x2{v[0] * scale, v[1] * scale}, f16x2);
        const f16x2 b = __builtin_convertvector(f32x2{v[2] * scale, v[3] * scale}, f16x2);
        const f16x2 c = __builtin_convertvector(
            f32x2{fmaf(v[0], scale, -(float)a[0]), fmaf(v[1], scale, -(float)a[1])}, f16x2);
        const f16x2 e = __builtin_convertvector(
            f32x2{fmaf(v[2], scale, -(float)b[0]), fmaf(v[3], scale, -(float)b[1])}, f16x2);
        *(f16x4*)to = f16x4{a[0], a[1], b[0], b[1]};
        *(f16x4*)(to + PLANE) = f16x4{c[0], c[1], e[0], e[1]};
    }
    // lane i: step 16 tile + i, terms the rows 32 s + 8 g ..
    static __device__ __forceinline__ Planes<2> turned(const f16* m, int tile, int s, Lane l = Lane()) {
        const int n = l.n, g = l.g;
        typedef short i16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) i16x4* Lds;
        Planes<2> x;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int row = 32 * s + 8 * g + n / 4, piece = 2 * tile + (n & 3) / 2, in = (n & 1) * 4;
            const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(m + k * PLANE + at(row, piece) + in));
            const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(m + k * PLANE + at(row + 4, piece) + in));
            const f16x4 lo = __builtin_bit_cast(f16x4, a), hi = __builtin_bit_cast(f16x4, b);
            x.p[k] = f16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
        return x;
    }
    // lane i: row 16 tile + i, terms the steps 32 p + 8 g ..
    static __device__ __forceinline__ Planes<2> along(const f16* m, int tile, int p, Lane l = Lane()) {
        const int n = l.n, g = l.g;
        Planes<2> x;
#pragma unroll
        for (int k = 0; k < 2; ++k) x.p[k] = *(const f16x8*)(m + k * PLANE + at(16 * tile + n, 4 * p + g));
        return x;
    }
};

// Sums over 16 neighbouring lanes, and over the lanes in front of each.
__device__ __forceinline__ float sum_lanes(float x) {
    auto with = [&](auto ctrl) {
        x += __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    with(std::integral_constant<int, 0xB1>{});
    with(std::integral_constant<int, 0x4E>{});
    with(std::integral_constant<int, 0x141>{});
    with(std::integral_constant<int, 0x140>{});
    return x;
}
__device__ __forceinline__ float sum_before(float x) {
    auto from = [&](auto ctrl) {
        return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    auto with = [&](auto ctrl) { x += from(ctrl); };
    x = from(std::integral_constant<int, 0x111>{});  // row_shr
    with(std::integral_constant<int, 0x111>{});
    with(std::integral_constant<int, 0x112>{});
    with(std::integral_constant<int, 0x114>{});
    with(std::integral_constant<int, 0x118>{});
    return x;
}
__device__ __forceinline__ float sum_column(float m) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    m = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    a = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// k_delta_grad for 16-bit inputs, on float16 planes. A wave takes 16 columns of
// the values and leaves U and dR in LDS, then tiles of the 64 x 64 matrices and
// 16 columns of the keys, from rows of S and dS that it reads again. One
// workgroup fills a compute unit's LDS, so its waits show: 8 x 2048 steps of 8
// key heads and 16 heads of 128: 266 us, the chunk of a head reading 128 KB of
// states. (With addresses held in registers through the loop it spilled: 683 us.)
template <typename T, int DK>
__global__ __launch_bounds__(64 * kGradWaves) void k_delta_grads(DeltaArgs a, int chunks, const Keys<1, DK>* keys,
                                                                const Backward* records, const float* behind) {
    static_assert(sizeof(T) == 2, "one plane of the inputs");
    constexpr int KT = DK / 16, KS = DK / 32, kThreads = 64 * kGradWaves;
    typedef Operand<1, DK> O;
    typedef Operand<1, kV> OV;
    typedef Turned<kV> TV;
    typedef Turned<kC> TC;
    __shared__ Keys<1, DK> kq;
    __shared__ f16 dOs[OV::SIZE];
    __shared__ union Shared {
        f16 ue[2][2 * TV::PLANE];  // U and dR
        f16 pa[4][2 * TC::PLANE];  // Pd by the keys' scales, by the queries', Ad by the keys' of its columns, of its rows
    } m;
    __shared__ Backward rec;
    __shared__ float o_back[kC], betas[kGradWaves][kC], front[kGradWaves][kC], after[kGradWaves][kC], dots[kGradWaves];
    __shared__ float most[4][kGradWaves], spoilt[2][kGradWaves];
    __shared__ float inside[kTiles][16], across[kTiles][16], tile_beta[kTiles][16], total[kTiles];
    __shared__ Chunk gates;
    const gs_delta_rule& d = a.r;
    const int kh = blockIdx.x % d.key_heads, c = blockIdx.x / d.key_heads % chunks, b = blockIdx.x / d.key_heads / chunks;
    const int w = threadIdx.x >> 6;
    const int len = length_of(d, b), t0 = c * kC, rows = len - t0, group = d.heads / d.key_heads;
    const int all = min(kC, d.steps - t0);  // steps of the chunk, padding included
    const int64_t first = (((int64_t)b * d.steps + t0) * d.key_heads + kh) * d.key_dim;
    T* const gq = (T*)a.grad_q + first;
    T* const gk = (T*)a.grad_k + first;
    const int64_t k_step = (int64_t)d.key_heads * d.key_dim, o_step = (int64_t)d.heads * d.value_dim;
    if (rows <= 0) {
        for (int e = threadIdx.x; e < all * d.key_dim; e += kThreads) {
            const int64_t at = e / d.key_dim * k_step + e % d.key_dim;
            gq[at] = gk[at] = (T)0.0f;
        }
        for (int e = threadIdx.x; e < all * group; e += kThreads) {
            const int64_t at = ((int64_t)b * d.steps + t0 + e / group) * d.heads + kh * group + e % group;
            a.grad_log_decay[at] = a.grad_beta[at] = 0.0f;
        }
        return;
    }
    const f32x4 zero = {0, 0, 0, 0};
    f32x4 dq[4] = {zero, zero, zero, zero}, dk[4] = {zero, zero, zero, zero};
    {
        Copy<sizeof(kq), kThreads> f;
        f.load(keys + ((int64_t)b * chunks + c) * d.key_heads + kh);
        f.store(&kq);
    }
    const int vs = (d.value_dim + 31) / 32;  // terms of sums over the values, by 32
    for (int hh = 0; hh < group; ++hh) {
        const Lane l = Lane::here();
        const int n = l.n, g = l.g, lane = 16 * g + n, col = 16 * w + n;  // of the values, and the row of a state's transposed columns
        const int h = kh * group + hh;
        const int64_t size = (int64_t)d.key_dim * d.value_dim, head = (int64_t)b * d.heads + h;
        const float* const S0 = c == 0 ? (a.h0 ? a.h0 + head * size : nullptr)
                                       : a.ckpt_in + (((int64_t)b * (chunks - 1) + c - 1) * d.heads + h) * size;
        const float* const dS = behind + (((int64_t)b * chunks + c) * d.heads + h) * size;
        const T* const v = (const T*)a.v + b * d.v_batch + t0 * d.v_step + h * d.v_head;
        const T* const go = (const T*)a.grad_o + (((int64_t)b * d.steps + t0) * d.heads + h) * d.value_dim;
        Column<KT> S, Z;
        const bool on = col < d.value_dim;
        S.load(S0, on, col, d.key_dim, d.value_dim, l);
        Z.load(dS, on, col, d.key_dim, d.value_dim, l);
        Values<T> fv, fo;
        fv.load(v, d.v_step, rows, on, col, d.value_dim, l);
        fo.load(go, o_step, rows, on, col, d.value_dim, l);
        if (hh) __syncthreads();
        {
            Copy<sizeof(rec), kThreads> f;
            f.load(records + ((int64_t)b * chunks + c) * d.heads + h);
            f.store(&rec);
        }
        {  // the rows of dO, scaled
            typedef T T8 __attribute__((ext_vector_type(8), aligned(sizeof(T))));
            constexpr int PIECES = kV / 8, BY = kThreads / PIECES, JOBS = kC / BY;
            const int at = threadIdx.x % PIECES, dim = at * 8;
#pragma unroll
            for (int j = 0; j < JOBS; ++j) {
                const int t = threadIdx.x / PIECES + j * BY;
                T8 x{};
                if (t < rows) {
                    const T* const from = go + t * o_step + dim;
                    if (dim + 8 <= d.value_dim) {
                        x = *(const T8*)from;
                    } else {
#pragma unroll
                        for (int i = 0; i < 7; ++i)
                            if (dim + i < d.value_dim) x[i] = from[i];
                    }
                }
                f32x4 f[2];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i / 4][i % 4] = (float)x[i];
                const Scale scale(over_lanes<PIECES>(largest(f)));
                *(f16x8*)(dOs + OV::at(t, at)) = split<1>(f[0], f[1], scale.by).p[0];
                if (at == 0) o_back[t] = scale.back;
            }
        }
        if (w == 0) load_gates(a, b, h, t0, len, gates);
        __syncthreads();
        // Row `col` of S and of dS, terms 32 s + 8 g .., for the keys' columns below; what is read past a row's end is
        // the next rows' and has no part in a row's scale.
        f32x4 srow[8], zrow[8];
        auto take = [&](const float* p, f32x4 (&x)[8]) {
            const Buffer from(p, p ? (int)size * 4 : 0);
            const uint32_t off = col < d.key_dim ? (uint32_t)(col * d.value_dim + 8 * g) * 4u : kNowhere;
#pragma unroll
            for (int s = 0; s < 8; ++s) x[s] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(from.r, off + 128 * (s / 2) + 16 * (s & 1), 0, 0));
        };
        auto within = [&](f32x4 (&x)[8]) {
            if (d.value_dim < kV)
#pragma unroll
                for (int s = 0; s < 8; ++s)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (32 * (s / 2) + 8 * g + 4 * (s & 1) + r >= d.value_dim) x[s][r] = 0.0f;
        };
        // 16 columns of the values: U and dR
        f32x4 U[4] = {zero, zero, zero, zero}, E[4] = {zero, zero, zero, zero};
        {
            if (gates.seg[kC - 1]) {  // as in the chains
                spoilt[0][w] = drop(S) ? __builtin_nanf("") : 0.0f;
                spoilt[1][w] = drop(Z) ? __builtin_nanf("") : 0.0f;
            }
            float dot = 0.0f;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) dot = fmaf(S.t[t][r], Z.t[t][r], dot);
            dot = sum_column(sum_lanes(dot));
            if (lane == 0) dots[w] = dot;
            const Scale ss(over_column(largest(S.t))), zs(over_column(largest(Z.t)));
            f32x4 x[4] = {zero, zero, zero, zero}, y[4] = {zero, zero, zero, zero}, e[4];
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Planes<2> sp = split<2>(S.t[2 * s], S.t[2 * s + 1], ss.by), zp = split<2>(Z.t[2 * s], Z.t[2 * s + 1], zs.by);
                Planes<1> A[4];
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) A[ti] = O::row(kq.K, ti, s, l);
                products(A, sp, x);
                products(A, zp, y);
            }
            take(S0, srow);
            take(dS, zrow);
            f32x4 R[4], dO[4], dU[4] = {zero, zero, zero, zero};
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                const int i = 16 * ti + 4 * g;
                const f32x4 gamma = *(const f32x4*)(rec.gamma + i), beta = *(const f32x4*)(rec.beta + i), kb = *(const f32x4*)(rec.k_back + i);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    e[ti][r] = fmaf(-gamma[r] * kb[r] * ss.back, x[ti][r], fv[4 * ti + r]);
                    R[ti][r] = beta[r] * e[ti][r];
                    dO[ti][r] = fo[4 * ti + r];
                }
            }
            {
                const Scale rs(over_column(largest(R)));
                const Planes<2> B[2] = {split<2>(R[0], R[1], rs.by), split<2>(R[2], R[3], rs.by)};
                lower<2>(rec.M, B, U, l);
                const float back = rs.back * rec.misc[1];
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) U[ti] *= back;
            }
            {
                const Scale os(over_column(largest(dO)));
                const Planes<1> B[2] = {split<1>(dO[0], dO[1], os.by), split<1>(dO[2], dO[3], os.by)};
                upper<2>(rec.PT, B, dU, l);
                const float back = os.back * rec.misc[2];
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                    const int i = 16 * ti + 4 * g;
                    const f32x4 end = *(const f32x4*)(rec.end + i), kb = *(const f32x4*)(rec.k_back + i);
#pragma unroll
                    for (int r = 0; r < 4; ++r) dU[ti][r] = fmaf(end[r] * kb[r] * zs.back, y[ti][r], back * dU[ti][r]);
                }
            }
            {
                const Scale us(over_column(largest(dU)));
                const Planes<2> B[2] = {split<2>(dU[0], dU[1], us.by), split<2>(dU[2], dU[3], us.by)};
                upper<2>(rec.MT, B, E, l);
                const float back = us.back * rec.misc[1];
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                    E[ti] *= back;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float t = sum_lanes(E[ti][r] * e[ti][r]);
                        if (n == 0) betas[w][16 * ti + 4 * g + r] = t;
                    }
                }
            }
            const float um = over_column(over_lanes<16>(largest(U))), em = over_column(over_lanes<16>(largest(E)));
            if (lane == 0) {
                most[0][w] = um;
                most[1][w] = em;
            }
        }
        __syncthreads();
        auto over_waves = [&](const float* p) {
            float x = 0.0f;
#pragma unroll
            for (int i = 0; i < kGradWaves; ++i) x = fmaxf(x, p[i]);
            return x;
        };
        const Scale us(over_waves(most[0])), es(over_waves(most[1]));
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) {
            TV::write(m.ue[0], col, ti, U[ti], us.by, l);
            TV::write(m.ue[1], col, ti, E[ti], es.by, l);
        }
        __syncthreads();
        // 16 columns of the keys: dO S^T, dR S^T, U dS^T
        f32x4 aq[4] = {zero, zero, zero, zero}, ar[4] = {zero, zero, zero, zero}, au[4] = {zero, zero, zero, zero};
        float s_back = 0.0f, z_back = 0.0f;
        if (w < KT) {
            within(srow);
            within(zrow);
            Scale scale(over_column(largest(srow)));
            s_back = scale.back;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (s < vs) {
                    const Planes<2> B = split<2>(srow[2 * s], srow[2 * s + 1], scale.by);
                    Planes<1> A[4];
                    Planes<2> C[4];
#pragma unroll
                    for (int ti = 0; ti < 4; ++ti) {
                        A[ti] = OV::row(dOs, ti, s, l);
                        C[ti] = TV::turned(m.ue[1], ti, s, l);
                    }
                    products(A, B, aq);
                    products(C, B, ar);
                    }
            scale = Scale(over_column(largest(zrow)));
            z_back = scale.back;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (s < vs) {
                    const Planes<2> B = split<2>(zrow[2 * s], zrow[2 * s + 1], scale.by);
                    Planes<2> C[4];
#pragma unroll
                    for (int ti = 0; ti < 4; ++ti) C[ti] = TV::turned(m.ue[0], ti, s, l);
                    products(C, B, au);
                    }
            if (gates.seg[kC - 1])  // no gradient of a step that a dropped column belongs to is finite
                for (int i = 0; i < kGradWaves; ++i) {
                    s_back += spoilt[0][i];
                    z_back += spoilt[1][i];
                }
        }
        // tiles of Pd and Ad, and of what the gates' gradients need of them
        f32x4 pd[2] = {zero, zero}, ad[2] = {zero, zero};
        float pm = 0.0f, am = 0.0f;
#pragma unroll
        for (int turn = 0; turn < 2; ++turn) {
            const int q = w + turn * kGradWaves;
            if (q >= kTiles) continue;
            const int ti = q >= 6 ? 3 : q >= 3 ? 2 : q >= 1 ? 1 : 0, tj = q - tri(ti, 0);
            f32x4 dp = zero, da = zero, qk = zero, kk = zero;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (s < vs) {
                    const Planes<2> B = TV::turned(m.ue[0], tj, s, l);
                    const Planes<1> A[1] = {OV::row(dOs, ti, s, l)};
                    const Planes<2> C[1] = {TV::turned(m.ue[1], ti, s, l)};
                    products(A, B, &dp);
                    products(C, B, &da);
                    }
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Planes<1> B = O::row(kq.K, tj, s, l);
                const Planes<1> A[1] = {O::row(kq.Q, ti, s, l)}, C[1] = {O::row(kq.K, ti, s, l)};
                products(A, B, &qk);
                products(C, B, &kk);
            }
            const int j = 16 * tj + n;
            const float kj = rec.k_back[j];
            float column = 0.0f, whole = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * ti + 4 * g + r;
                const float D = i >= j ? decay(gates, i, j) : 0.0f;
                const float p = d.scale * D * us.back * o_back[i] * dp[r], t = i > j ? -D * us.back * es.back * da[r] : 0.0f;
                const float ki = rec.k_back[i], qi = rec.q_back[i], beta = rec.beta[i];
                const float tb = t * kk[r] * ki * kj;
                pd[turn][r] = p;
                ad[turn][r] = beta * t;
                pm = fmaxf(pm, fabsf(p) * fmaxf(kj, qi));
                am = fmaxf(am, fabsf(beta * t) * fmaxf(kj, ki));
                // sums over the columns in front of this one, behind which the decay of step j lies
                const float x = fmaf(p, qk[r] * qi * kj, beta * tb), before = sum_before(x);
                if (ti > tj || i >= j) column += before;
                if (n == 15) across[q][4 * g + r] = before + x;
                whole += before + x;
                const float sum = sum_lanes(tb);
                if (n == 0) tile_beta[q][4 * g + r] = sum;
            }
            column = sum_column(column);
            whole = sum_column(whole);
            if (g == 0) inside[q][n] = column;
            if (lane == 15) total[q] = whole;
        }
        pm = over_column(over_lanes<16>(pm));
        am = over_column(over_lanes<16>(am));
        if (lane == 0) {
            most[2][w] = pm;
            most[3][w] = am;
        }
        __syncthreads();
        const Scale ps(over_waves(most[2])), as(over_waves(most[3]));
#pragma unroll
        for (int turn = 0; turn < 2; ++turn) {
            const int q = w + turn * kGradWaves;
            if (q >= kTiles) continue;
            const int ti = q >= 6 ? 3 : q >= 3 ? 2 : q >= 1 ? 1 : 0, tj = q - tri(ti, 0), row = 16 * tj + n;
            const float kj = rec.k_back[row];
            const f32x4 ki = *(const f32x4*)(rec.k_back + 16 * ti + 4 * g), qi = *(const f32x4*)(rec.q_back + 16 * ti + 4 * g);
            TC::write(m.pa[0], row, ti, pd[turn] * kj, ps.by, l);
            TC::write(m.pa[1], row, ti, pd[turn] * qi, ps.by, l);
            TC::write(m.pa[2], row, ti, ad[turn] * kj, as.by, l);
            TC::write(m.pa[3], row, ti, ad[turn] * ki, as.by, l);
        }
        if (w >= 4)  // the tiles over the diagonal that pairs of tiles take along
#pragma unroll
            for (int p = 0; p < 2; ++p) TC::write(m.pa[w - 4], 32 * p + 16 + n, 2 * p, zero, 1.0f, l);
        __syncthreads();
        if (w < KT) {
            f32x4 xq[4] = {zero, zero, zero, zero}, xp[4] = {zero, zero, zero, zero}, xa[4] = {zero, zero, zero, zero};
            // a column of the keys' (queries') rows: terms the steps 32 p + 8 g ..
            auto columns = [&](const f16* from, int p) {
                typedef short i16x4 __attribute__((ext_vector_type(4)));
                typedef __attribute__((address_space(3))) i16x4* Lds;
                const int t = 32 * p + 8 * g + n / 4, piece = 2 * w + (n & 3) / 2, in = (n & 1) * 4;
                const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(from + O::at(t, piece) + in));
                const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(from + O::at(t + 4, piece) + in));
                const f16x4 lo = __builtin_bit_cast(f16x4, x), hi = __builtin_bit_cast(f16x4, y);
                return Planes<1>{{f16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}}};
            };
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const Planes<1> kc = columns(kq.K, p), qc = columns(kq.Q, p);
#pragma unroll
                for (int ti = 0; ti < 4; ++ti) {
                    if (p <= ti / 2) {
                        const Planes<2> A[1] = {TC::turned(m.pa[0], ti, p, l)}, C[1] = {TC::turned(m.pa[2], ti, p, l)};
                        products(A, kc, xq + ti);
                        products(C, kc, xa + ti);
                    }
                    if (p >= ti / 2) {
                        const Planes<2> A[1] = {TC::along(m.pa[1], ti, p, l)}, C[1] = {TC::along(m.pa[3], ti, p, l)};
                        products(A, qc, xp + ti);
                        products(C, kc, xa + ti);
                    }
                }
            }
            const int segs = __builtin_amdgcn_readfirstlane(gates.seg[kC - 1]);
#pragma unroll
            for (int ti = 0; ti < 4; ++ti) {
                const int i0 = 16 * ti + 4 * g;
                const f32x4 gamma = *(const f32x4*)(rec.gamma + i0), beta = *(const f32x4*)(rec.beta + i0), end = *(const f32x4*)(rec.end + i0);
                const f32x4 kb = *(const f32x4*)(rec.k_back + i0), qb = *(const f32x4*)(rec.q_back + i0), ob = *(const f32x4*)(o_back + i0);
                const int* const seg = gates.seg + i0;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = i0 + r, at = O::at(i, 2 * w + n / 8) + (n & 7);
                    const float kv = (float)kq.K[at] * kb[r], qv = (float)kq.Q[at] * qb[r];
                    // what a restart has dropped is 0 whatever it was
                    const float x = seg[r] == 0 ? d.scale * gamma[r] * ob[r] * s_back * aq[ti][r] : 0.0f;
                    const float y = seg[r] == 0 ? beta[r] * gamma[r] * es.back * s_back * ar[ti][r] : 0.0f;
                    const float z = seg[r] == segs ? end[r] * us.back * z_back * au[ti][r] : 0.0f;
                    const float f = sum_lanes(qv * x - kv * y), af = sum_lanes(kv * z);
                    if (n == 0) {
                        front[w][i] = f;
                        after[w][i] = af;
                    }
                    dq[ti][r] += fmaf(ps.back, xq[ti][r], x);
                    dk[ti][r] += fmaf(ps.back, xp[ti][r], fmaf(as.back, xa[ti][r], z - y));
                }
            }
        }
        __syncthreads();
        const int64_t at = ((int64_t)b * d.steps + t0 + lane) * d.heads + h;
        const int tt = lane >> 4;
        if (w == 0 && lane < all) {
            float be = 0.0f;
#pragma unroll
            for (int x = 0; x < kGradWaves; ++x) be += betas[x][lane];
#pragma unroll
            for (int tj = 0; tj < 4; ++tj)
                if (tj <= tt) be += tile_beta[tri(tt, tj)][n];
            // not finite where the state in front (the gradient behind) is not and no restart lies between
#pragma unroll
            for (int x = 0; x < KT; ++x) be += 0.0f * front[x][lane] + 0.0f * after[x][lane];
            a.grad_beta[at] = lane < rows ? be : 0.0f;
        }
        if (w == 1) {
            float f = 0.0f, af = 0.0f, dot = 0.0f, t = 0.0f, row = 0.0f;
#pragma unroll
            for (int x = 0; x < kGradWaves; ++x) dot += dots[x];
#pragma unroll
            for (int x = 0; x < KT; ++x) {
                f += front[x][lane];
                af += after[x][lane];
            }
            // between every j < t <= i: of the tiles of this step's columns, then of whole rows of the columns in front
#pragma unroll
            for (int ti = 0; ti < 4; ++ti)
                if (ti >= tt) t += inside[tri(ti, tt)][n];
#pragma unroll
            for (int tj = 0; tj < 3; ++tj)
                if (tj < tt) row += across[tri(tt, tj)][n];
#pragma unroll
            for (int ti = 2; ti < 4; ++ti)
#pragma unroll
                for (int tj = 0; tj < 3; ++tj)
                    if (ti > tt && tj < tt) t += total[tri(ti, tj)];
            float all_f = f, all_a = af;
#pragma unroll
            for (int x = 1; x < 64; x <<= 1) {
                const float p = __shfl_down(all_f, x), o = __shfl_up(all_a, x), q = __shfl_down(row, x);
                if (lane + x < 64) all_f += p;
                if (lane >= x) all_a += o;
                if (x < 16 && n + x < 16) row += q;  // rows from this one to the tile's last
            }
            all_a = __shfl_up(all_a, 1);
            t += row + all_f + (lane ? all_a : 0.0f) + gates.whole * dot;
            if (lane < all) {
                // the decay of a restart is not applied
                const bool cut = lane ? gates.seg[lane] != gates.seg[lane - 1] : gates.seg[0] != 0;
                a.grad_log_decay[at] = lane < rows && !cut ? t : 0.0f;
            }
        }
    }
    const int n = threadIdx.x & 15, g = threadIdx.x >> 4 & 3, col = 16 * w + n;
    if (w < KT && col < d.key_dim)
#pragma unroll
        for (int ti = 0; ti < 4; ++ti)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * ti + 4 * g + r;
                if (i < all) {
                    gq[i * k_step + col] = (T)(i < rows ? dq[ti][r] : 0.0f);
                    gk[i * k_step + col] = (T)(i < rows ? dk[ti][r] : 0.0f);
                }
            }
}

// A few steps (one new token, a few drafted ones): the state is read and
// written once, and that is the bound. A workgroup holds `slice` columns of one
// head's state in registers, V neighbouring columns a lane and the rows spread
// over lanes and waves. Both sums over the rows that a step needs, S^T k and
// S^T q, are formed of the state in front of it (o = a S^T q + (q.k) u), so a
// step has one exchange through LDS. Everything the steps read is fetched
// before the first one.
//
// Measured: one step of 64 sequences of 16 heads of 128 x 128, whose states are
// 134 MB: 29 us, 4.6 TB/s; of 1 sequence of 8 heads of 64: 5 us, a launch's
// latency. A call of 8 steps takes 61 us where the chunks' kernels take 81 to 89
// for 9 to 64 (64 sequences of 16 heads), or 19 and 20 (4 sequences).
constexpr int kFewSteps = GS_DELTA_FEW;

template <typename T, int V>
__global__ __launch_bounds__(256) void k_delta_steps(DeltaArgs a, int slice, int lanes) {
    constexpr int NR = 64 / V;
    typedef float Vec __attribute__((ext_vector_type(V)));
    const gs_delta_rule& d = a.r;
    __shared__ float ks[kFewSteps][kV], qs[kFewSteps][kV], vs[kFewSteps][kV], gates[kFewSteps][2], qk[kFewSteps];
    __shared__ float part[2][4][2][kV];
    const int b = blockIdx.x / d.heads, h = blockIdx.x % d.heads, kh = h / (d.heads / d.key_heads);
    const int len = length_of(d, b), c0 = blockIdx.y * slice, cols = min(slice, d.value_dim - c0);
    const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = 256 / lanes;
    const int wave = threadIdx.x >> 6, col = lane * V;
    const bool on = col < cols;  // and so are its V - 1 neighbours
    const int64_t state = ((int64_t)b * d.heads + h) * d.key_dim * d.value_dim + c0 + col;
    Vec S[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        if (j * groups >= d.key_dim) break;
        const int row = j * groups + group;
        S[j] = Vec{};
        if (a.h0 && on && row < d.key_dim) S[j] = *(const Vec*)(a.h0 + state + (int64_t)row * d.value_dim);
    }
    for (int e = threadIdx.x; e < len * d.key_dim; e += 256) {
        const int t = e / d.key_dim, i = e - t * d.key_dim;
        ks[t][i] = (float)((const T*)a.k)[b * d.k_batch + t * d.k_step + kh * d.k_head + i];
        qs[t][i] = (float)((const T*)a.q)[b * d.q_batch + t * d.q_step + kh * d.q_head + i];
    }
    for (int e = threadIdx.x; e < len * cols; e += 256) {
        const int t = e / cols, i = e - t * cols;
        vs[t][i] = (float)((const T*)a.v)[b * d.v_batch + t * d.v_step + h * d.v_head + c0 + i];
    }
    if ((int)threadIdx.x < len) {
        const int t = threadIdx.x;
        const bool cut = d.restart && d.restart[(int64_t)b * d.steps + t];
        const float g = a.log_decay[b * d.decay_batch + t * d.decay_step + h];
        gates[t][0] = cut || g < -104.0f ? 0.0f : expf(g);
        gates[t][1] = a.beta[b * d.beta_batch + t * d.beta_step + h];
    }
    __syncthreads();
    for (int t = wave; t < len; t += 4) {
        float x = 0.0f;
        for (int i = threadIdx.x & 63; i < d.key_dim; i += 64) x = fmaf(ks[t][i], qs[t][i], x);
        for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
        if ((threadIdx.x & 63) == 0) qk[t] = x;
    }
    T* const o = (T*)a.o + ((int64_t)b * d.steps * d.heads + h) * d.value_dim + c0 + col;
    const int64_t o_step = (int64_t)d.heads * d.value_dim;
    for (int t = 0; t < len; ++t) {
        Vec x{}, y{};
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            if (j * groups >= d.key_dim) break;
            const int row = min(j * groups + group, d.key_dim - 1);  // rows past the last one hold 0
            const float kk = ks[t][row], qq = qs[t][row];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[i] = fmaf(S[j][i], kk, x[i]);
                y[i] = fmaf(S[j][i], qq, y[i]);
            }
        }
        for (int m = lanes; m < 64; m <<= 1)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[i] += __shfl_xor(x[i], m);
                y[i] += __shfl_xor(y[i], m);
            }
        const int turn = t & 1;
        if ((int)(threadIdx.x & 63) < lanes && on) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                part[turn][wave][0][col + i] = x[i];
                part[turn][wave][1][col + i] = y[i];
            }
        }
        __syncthreads();
        const float decay = gates[t][0], beta = gates[t][1], dot = qk[t];
        Vec u{};
        if (on) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float sx = 0.0f, sy = 0.0f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    sx += part[turn][w][0][col + i];
                    sy += part[turn][w][1][col + i];
                }
                // a state that is dropped is dropped whatever it holds
                u[i] = beta * (vs[t][col + i] - (decay == 0.0f ? 0.0f : decay * sx));
                x[i] = d.scale * fmaf(dot, u[i], decay == 0.0f ? 0.0f : decay * sy);
            }
            if (group == 0)
#pragma unroll
                for (int i = 0; i < V; ++i) o[t * o_step + i] = (T)x[i];
        }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            if (j * groups >= d.key_dim) break;
            const int row = j * groups + group;
            const float kk = row < d.key_dim ? ks[t][row] : 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) S[j][i] = fmaf(kk, u[i], decay == 0.0f ? 0.0f : decay * S[j][i]);
        }
    }
    if (on && group == 0)
        for (int t = len; t < d.steps; ++t)
#pragma unroll
            for (int i = 0; i < V; ++i) o[t * o_step + i] = (T)0.0f;
    if (a.h_last && on)
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            if (j * groups >= d.key_dim) break;
            const int row = j * groups + group;
            if (row < d.key_dim) *(Vec*)(a.h_last + state + (int64_t)row * d.value_dim) = S[j];
        }
}

template <typename T>
hipError_t steps(const DeltaArgs& a, hipStream_t stream) {
    const gs_delta_rule& r = a.r;
    const bool wide = r.value_dim % 4 == 0 && !(((uintptr_t)a.h0 | (uintptr_t)a.h_last) & 15);
    // Columns of a workgroup: all, but fewer where that makes fewer than 512 of them. 16 heads of 128, one step: 8
    // sequences 7.4 us with 32 columns (512 workgroups), 7.8 with 64, 9.0 with 128, 11.3 with 16; 32 sequences 16 us
    // with 128 columns and 20 with 64; 1 sequence 5.4 us with 16 columns and 7.6 with 128.
    int slice = r.value_dim;
    const int most = wide ? 128 : 64;
    if (slice > most) slice = most;
    while (slice > 16 && (int64_t)r.batch * r.heads * ((r.value_dim + slice - 1) / slice) < 512) slice = (slice / 2 + 3) & ~3;
    const int v = wide ? 4 : 1;
    int lanes = 1;
    while (lanes * v < slice) lanes *= 2;
    const dim3 grid(r.batch * r.heads, (r.value_dim + slice - 1) / slice);
    if (wide)
        k_delta_steps<T, 4><<<grid, 256, 0, stream>>>(a, slice, lanes);
    else
        k_delta_steps<T, 1><<<grid, 256, 0, stream>>>(a, slice, lanes);
    return hipGetLastError();
}

int chunks_of(const gs_delta_rule& r) { return (r.steps + kC - 1) / kC; }
size_t inverse_floats(const gs_delta_rule& r) { return (size_t)r.batch * chunks_of(r) * r.heads * kLower; }

int padded(int dim) { return dim <= 64 ? 64 : 128; }
size_t key_bytes(const gs_delta_rule& r) {
    const size_t row = (size_t)2 * kC * padded(r.key_dim) * sizeof(f16) * (r.dtype == GS_F32 ? 2 : 1);
    return (size_t)r.batch * chunks_of(r) * r.key_heads * row;
}
size_t behind_floats(const gs_delta_rule& r) {
    return (size_t)r.batch * chunks_of(r) * r.heads * r.key_dim * r.value_dim;
}
size_t back_record_bytes(const gs_delta_rule& r) { return (size_t)r.batch * chunks_of(r) * r.heads * sizeof(Backward); }
size_t record_bytes(const gs_delta_rule& r) {
    return (size_t)r.batch * chunks_of(r) * r.heads * sizeof(Forward);
}

// Segments of a sequence: enough workgroups for the chip, each of them long
// enough for the walk over them and the first pass (more than the work of the
// second) to pay. Heads of 128 x 128, bf16, with segments and without: 4 heads
// of 65536 steps 460 and 4387 us; 32 heads of 2048 steps 121 and 162 us, of 8192
// 379 and 668; 64 heads of 2048 steps 214 and 187, of 8192 712 and 776; 85 heads
// of 8192 steps 1081 and 845. The backward of 4 heads of 8192 steps 206 and 639
// us, of 32 heads 1001 and 1269, of 64 heads 1918 and 1915.
constexpr int kUnits = 256;  // compute units
Segments segments_of(const gs_delta_rule& r) {
    Segments s{1, chunks_of(r), nullptr, nullptr, nullptr};
    const int64_t heads = (int64_t)r.batch * r.heads;
    if (heads > (s.chunks >= 128 ? kUnits / 4 : kUnits / 8) || s.chunks < 32) return s;
    const int most = (int)std::min<int64_t>((kUnits + heads - 1) / heads, 32);
    s.chunks = std::max((s.chunks + most - 1) / most, 8);
    s.count = (chunks_of(r) + s.chunks - 1) / s.chunks;
    return s;
}
size_t segment_bytes(const gs_delta_rule& r) {
    const Segments s = segments_of(r);
    if (s.count == 1) return 0;
    return (size_t)r.batch * r.heads * s.count * ((size_t)r.key_dim * (r.value_dim + r.key_dim) * sizeof(float) + sizeof(uint32_t));
}

// Waves (of 16 columns) of a chain's workgroup: 8, which read the operands from
// memory once for 128 columns, or 4 where their workgroups all run at once,
// each on a compute unit of its own (a call of 8 x 2048 steps of 16 heads of
// 128: 274 us with 4, 308 with 8; of 8192 steps of 32 heads in 8 segments, with
// 4 in both passes 427 and with 8 379).
bool narrow(int64_t groups, int columns) { return columns <= 64 || groups * ((columns + 63) / 64) <= kUnits; }

template <typename T, int DK, int WAVES, bool OUT>
void chain(const DeltaArgs& a, int chunks, const void* scratch, const Segments& seg, hipStream_t stream) {
    const gs_delta_rule& r = a.r;
    const auto* const keys = (const Keys<kPlanes<T>, DK>*)scratch;
    const auto* const records = (const Forward*)((const char*)scratch + key_bytes(r));
    constexpr int WIDE = 16 * WAVES;
    const int blocks = (r.value_dim + WIDE - 1) / WIDE + (OUT ? 0 : (r.key_dim + WIDE - 1) / WIDE);
    k_delta_chain<T, DK, WAVES, OUT><<<dim3(r.batch * r.heads, blocks, seg.count), 64 * WAVES, 0, stream>>>(
        a, chunks, keys, records, seg);
}

template <typename T, int DK>
hipError_t forward(const DeltaArgs& a, void* scratch, hipStream_t stream) {
    const gs_delta_rule& r = a.r;
    const int chunks = chunks_of(r), heads = r.batch * r.heads;
    k_delta_prepare<T, DK><<<r.batch * chunks * r.key_heads, kPrepThreads, 0, stream>>>(
        a, chunks, (Keys<kPlanes<T>, DK>*)scratch, (Forward*)((char*)scratch + key_bytes(r)));
    Segments seg = segments_of(r);
    const int64_t groups = (int64_t)heads * seg.count;
    if (seg.count > 1) {
        seg.front = (float*)((char*)scratch + key_bytes(r) + record_bytes(r));
        seg.phi = seg.front + (size_t)heads * seg.count * r.key_dim * r.value_dim;
        seg.cut = (uint32_t*)(seg.phi + (size_t)heads * seg.count * r.key_dim * r.key_dim);
        if (narrow(groups * 2, std::max(r.value_dim, r.key_dim)))
            chain<T, DK, 4, false>(a, chunks, scratch, seg, stream);
        else
            chain<T, DK, 8, false>(a, chunks, scratch, seg, stream);
        k_delta_join<DK><<<dim3(heads, (r.value_dim + 15) / 16), DK * 4, 0, stream>>>(a, seg, a.h0, false);
    }
    if (narrow(groups, r.value_dim))
        chain<T, DK, 4, true>(a, chunks, scratch, seg, stream);
    else
        chain<T, DK, 8, true>(a, chunks, scratch, seg, stream);
    return hipGetLastError();
}

template <typename T, int DK, int WAVES, bool OUT>
void chain_back(const DeltaArgs& a, int chunks, const void* scratch, float* behind, const Segments& seg, hipStream_t stream) {
    const gs_delta_rule& r = a.r;
    constexpr int WIDE = 16 * WAVES;
    const int blocks = (r.value_dim + WIDE - 1) / WIDE + (OUT ? 0 : (r.key_dim + WIDE - 1) / WIDE);
    k_delta_back<T, DK, WAVES, OUT><<<dim3(r.batch * r.heads, blocks, seg.count), 64 * WAVES, 0, stream>>>(
        a, chunks, (const Keys<kPlanes<T>, DK>*)scratch, (const Backward*)((const char*)scratch + key_bytes(r)), behind, seg);
}

template <typename T, int DK>
hipError_t backward(const DeltaArgs& a, void* scratch, hipStream_t stream) {
    const gs_delta_rule& r = a.r;
    const int chunks = chunks_of(r), heads = r.batch * r.heads;
    auto* const keys = (Keys<kPlanes<T>, DK>*)scratch;
    auto* const records = (Backward*)((char*)scratch + key_bytes(r));
    float* const behind = (float*)((char*)records + back_record_bytes(r));
    if (chunks)
        k_delta_prepare<T, DK><<<r.batch * chunks * r.key_heads, kPrepThreads, 0, stream>>>(a, chunks, keys, records);
    Segments seg = segments_of(r);
    const int64_t groups = (int64_t)heads * seg.count;
    float* const inverse = behind + behind_floats(r);
    if (seg.count > 1) {
        seg.front = inverse + (r.dtype == GS_F32 ? inverse_floats(r) : 0);
        seg.phi = seg.front + (size_t)heads * seg.count * r.key_dim * r.value_dim;
        seg.cut = (uint32_t*)(seg.phi + (size_t)heads * seg.count * r.key_dim * r.key_dim);
        if (narrow(groups * 2, std::max(r.value_dim, r.key_dim)))
            chain_back<T, DK, 4, false>(a, chunks, scratch, behind, seg, stream);
        else
            chain_back<T, DK, 8, false>(a, chunks, scratch, behind, seg, stream);
        k_delta_join<DK><<<dim3(heads, (r.value_dim + 15) / 16), DK * 4, 0, stream>>>(a, seg, a.grad_last, true);
    }
    if (narrow(groups, r.value_dim))
        chain_back<T, DK, 4, true>(a, chunks, scratch, behind, seg, stream);
    else
        chain_back<T, DK, 8, true>(a, chunks, scratch, behind, seg, stream);
    if (chunks) {
        const int grid = r.batch * chunks * r.key_heads;
        if constexpr (sizeof(T) == 2) {
            k_delta_grads<T, DK><<<grid, 64 * kGradWaves, 0, stream>>>(a, chunks, keys, records, behind);
        } else {
            k_delta_inverse<T, DK><<<r.batch * chunks * r.heads, 256, 0, stream>>>(a, chunks, inverse);
            k_delta_grad<T, DK><<<grid, 64 * kGradWaves, 0, stream>>>(a, chunks, inverse, behind);
        }
    }
    return hipGetLastError();
}

template <typename T>
hipError_t run(const DeltaArgs& a, void* scratch, bool back, hipStream_t stream) {
    if (a.r.key_dim <= 64)
        return back ? backward<T, 64>(a, scratch, stream) : forward<T, 64>(a, scratch, stream);
    return back ? backward<T, 128>(a, scratch, stream) : forward<T, 128>(a, scratch, stream);
}

hipError_t run(const DeltaArgs& a, void* scratch, bool back, hipStream_t stream) {
    switch (a.r.dtype) {
        case GS_F32: return run<float>(a, scratch, back, stream);
        case GS_BF16: return run<bf16>(a, scratch, back, stream);
        default: return run<f16>(a, scratch, back, stream);
    }
}

}  // namespace

size_t delta_rule_scratch_bytes(const gs_delta_rule& r, bool backward) {
    if (!backward && r.steps <= kFewSteps) return 0;
    if (!backward) return key_bytes(r) + record_bytes(r) + segment_bytes(r);
    return key_bytes(r) + back_record_bytes(r) + behind_floats(r) * sizeof(float) +
           (r.dtype == GS_F32 ? inverse_floats(r) * sizeof(float) : 0) + segment_bytes(r);
}

hipError_t launch_delta_rule_fwd(const DeltaArgs& a, void* scratch, hipStream_t stream) {
    if (a.r.steps <= kFewSteps) {
        switch (a.r.dtype) {
            case GS_F32: return steps<float>(a, stream);
            case GS_BF16: return steps<bf16>(a, stream);
            default: return steps<f16>(a, stream);
        }
    }
    return run(a, scratch, false, stream);
}

hipError_t launch_delta_rule_bwd(const DeltaArgs& a, void* scratch, hipStream_t stream) {
    return run(a, scratch, true, stream);
}

}  // namespace gs
