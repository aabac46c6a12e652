// Gated linear recurrence h_t = a_t h_{t-1} + u_t along the steps of a
// sequence, forward and backward (include/gs.h, gs_recurrence_*).
#include <algorithm>

#include "gs_internal.h"

namespace gs {
namespace {

constexpr int kRecChunk = GS_RECURRENCE_CHUNK;
constexpr int kRecSub = 16;  // steps whose states the backward holds at once

template <typename T>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    return (float)((const T*)p)[i];
}
template <typename T>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
    ((T*)p)[i] = (T)v;
}

// sigmoid(z) and 1 - sigmoid(z), each without cancellation.
__device__ __forceinline__ void sigmoids(float z, float& a, float& rest) {
    const float e = expf(-fabsf(z));
    const float big = 1.0f / (1.0f + e), small = e * big;
    a = z >= 0.0f ? big : small;
    rest = z >= 0.0f ? small : big;
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

template <typename T, bool SIGMOID>
__global__ void k_recurrence_fwd(RecurrenceArgs r) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (int64_t)r.batch * r.channels) return;
    const int b = (int)(i / r.channels), c = (int)(i % r.channels);
    const int len = r.lengths ? min(max(r.lengths[b], 0), r.steps) : r.steps;
    const int64_t g0 = b * r.gate_batch + c, x0 = b * r.x_batch + c;
    const int64_t o0 = (int64_t)b * r.steps * r.channels + c;
    const uint8_t* restart = r.restart ? r.restart + (int64_t)b * r.steps : nullptr;
    const int rows = (r.steps + kRecChunk - 1) / kRecChunk - 1;
    float h = r.h0 ? r.h0[i] : 0.0f;
    for (int t = 0; t < len; ++t) {
        if (r.ckpt && t && t % kRecChunk == 0)
            r.ckpt[((int64_t)b * rows + t / kRecChunk - 1) * r.channels + c] = h;
        float a, u, rest;
        step_terms<SIGMOID>(load1<T>(r.gate, g0 + t * r.gate_step), load1<T>(r.x, x0 + t * r.x_step), a, u, rest);
        h = restart && restart[t] ? u : fmaf(a, h, u);
        store1<T>(r.h, o0 + (int64_t)t * r.channels, h);
    }
    for (int t = len; t < r.steps; ++t) store1<T>(r.h, o0 + (int64_t)t * r.channels, 0.0f);
    if (r.h_last) r.h_last[i] = h;
}

template <typename T, bool SIGMOID>
__global__ void k_recurrence_bwd(RecurrenceArgs r) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (int64_t)r.batch * r.channels) return;
    const int b = (int)(i / r.channels), c = (int)(i % r.channels);
    const int len = r.lengths ? min(max(r.lengths[b], 0), r.steps) : r.steps;
    const int64_t g0 = b * r.gate_batch + c, x0 = b * r.x_batch + c;
    const int64_t o0 = (int64_t)b * r.steps * r.channels + c;
    const uint8_t* restart = r.restart ? r.restart + (int64_t)b * r.steps : nullptr;
    const int rows = (r.steps + kRecChunk - 1) / kRecChunk - 1;
    for (int t = len; t < r.steps; ++t) {
        store1<T>(r.grad_gate, o0 + (int64_t)t * r.channels, 0.0f);
        store1<T>(r.grad_x, o0 + (int64_t)t * r.channels, 0.0f);
    }
    float carry = r.grad_last ? r.grad_last[i] : 0.0f;  // dL/dh passed back by the steps behind
    for (int s0 = (len - 1) / kRecSub * kRecSub; s0 >= 0 && len; s0 -= kRecSub) {
        const int c0 = s0 / kRecChunk * kRecChunk;
        float h = c0 ? r.ckpt_in[((int64_t)b * rows + c0 / kRecChunk - 1) * r.channels + c] : r.h0 ? r.h0[i] : 0.0f;
        for (int t = c0; t < s0; ++t) {
            float a, u, rest;
            step_terms<SIGMOID>(load1<T>(r.gate, g0 + t * r.gate_step), load1<T>(r.x, x0 + t * r.x_step), a, u, rest);
            h = restart && restart[t] ? u : fmaf(a, h, u);
        }
        float prev[kRecSub];
#pragma unroll
        for (int k = 0; k < kRecSub; ++k) {
            const int t = s0 + k;
            prev[k] = 0.0f;
            if (t >= len) continue;
            float a, u, rest;
            step_terms<SIGMOID>(load1<T>(r.gate, g0 + t * r.gate_step), load1<T>(r.x, x0 + t * r.x_step), a, u, rest);
            const bool again = restart && restart[t];
            prev[k] = again ? 0.0f : h;
            h = again ? u : fmaf(a, h, u);
        }
#pragma unroll
        for (int k = kRecSub - 1; k >= 0; --k) {
            const int t = s0 + k;
            if (t >= len) continue;
            float a, u, rest;
            const float x = load1<T>(r.x, x0 + t * r.x_step);
            step_terms<SIGMOID>(load1<T>(r.gate, g0 + t * r.gate_step), x, a, u, rest);
            const float d = load1<T>(r.grad_h, o0 + (int64_t)t * r.channels) + carry;
            store1<T>(r.grad_gate, o0 + (int64_t)t * r.channels,
                      SIGMOID ? d * (prev[k] - x) * (a * rest) : d * prev[k]);
            store1<T>(r.grad_x, o0 + (int64_t)t * r.channels, d * rest);
            carry = restart && restart[t] ? 0.0f : a * d;
        }
    }
    if (r.grad_h0) r.grad_h0[i] = carry;
}

template <typename T>
hipError_t launch_fwd_of(const RecurrenceArgs& r, bool sigmoid, hipStream_t stream) {
    const unsigned grid = (unsigned)(((int64_t)r.batch * r.channels + 255) / 256);
    if (sigmoid)
        k_recurrence_fwd<T, true><<<grid, 256, 0, stream>>>(r);
    else
        k_recurrence_fwd<T, false><<<grid, 256, 0, stream>>>(r);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_bwd_of(const RecurrenceArgs& r, bool sigmoid, hipStream_t stream) {
    const unsigned grid = (unsigned)(((int64_t)r.batch * r.channels + 255) / 256);
    if (sigmoid)
        k_recurrence_bwd<T, true><<<grid, 256, 0, stream>>>(r);
    else
        k_recurrence_bwd<T, false><<<grid, 256, 0, stream>>>(r);
    return hipGetLastError();
}

}  // namespace

bool recurrence_fits(const gs_recurrence& r) {
    const int64_t most = INT32_MAX;
    const int64_t columns = ((int64_t)r.channels + 63) / 64, chunks = ((int64_t)r.steps + kRecChunk - 1) / kRecChunk;
    return columns * std::max(r.batch, 1) <= most && columns * std::max(r.batch, 1) * std::max<int64_t>(chunks, 1) <= most;
}

size_t recurrence_scratch_bytes(const gs_recurrence&) { return 0; }

hipError_t launch_recurrence_fwd(const RecurrenceArgs& r, int dtype, bool sigmoid, void*, hipStream_t stream) {
    if (dtype == GS_F32) return launch_fwd_of<float>(r, sigmoid, stream);
    if (dtype == GS_BF16) return launch_fwd_of<__bf16>(r, sigmoid, stream);
    return launch_fwd_of<_Float16>(r, sigmoid, stream);
}

hipError_t launch_recurrence_bwd(const RecurrenceArgs& r, int dtype, bool sigmoid, void*, hipStream_t stream) {
    if (dtype == GS_F32) return launch_bwd_of<float>(r, sigmoid, stream);
    if (dtype == GS_BF16) return launch_bwd_of<__bf16>(r, sigmoid, stream);
    return launch_bwd_of<_Float16>(r, sigmoid, stream);
}

}  // namespace gs
