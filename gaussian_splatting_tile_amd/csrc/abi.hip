// C ABI of libgs (include/gs.h): host-side argument validation, scratch
// layout, launch sequencing and error reporting. No C++ exception crosses
// this boundary; no device memory is allocated here.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

#include "gs_internal.h"

// The binning workspace of gs_bin_and_sort_async_noalloc: one fixed array
// per GPU, which each device holds from the library's load on it until the
// process ends. In host code this name is only a stand-in for the symbol;
// its device address on the current device comes from hipGetSymbolAddress
// (static_scratch below), and only that address is ever passed to kernels.
static __device__ __align__(256) unsigned char scratch[GS_NOALLOC_SCRATCH_BYTES];

namespace {

thread_local std::string g_last_error;

gs_status fail(gs_status code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return code;
}

gs_status hip_check(hipError_t e, const char* what) {
    if (e == hipSuccess) return GS_OK;
    return fail(GS_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

gs_status check_camera(const gs_camera* cam) {
    if (!cam) return fail(GS_ERR_INVALID, "camera is NULL");
    if (cam->width < 1 || cam->height < 1 || cam->width > GS_MAX_DIM || cam->height > GS_MAX_DIM)
        return fail(GS_ERR_INVALID, "image size %dx%d outside [1, %d]", cam->width, cam->height,
                    GS_MAX_DIM);
    if (!(cam->fx > 0.0f) || !(cam->fy > 0.0f) || !std::isfinite(cam->fx) || !std::isfinite(cam->fy))
        return fail(GS_ERR_INVALID, "focal lengths must be finite and positive");
    if (!std::isfinite(cam->cx) || !std::isfinite(cam->cy))
        return fail(GS_ERR_INVALID, "principal point must be finite");
    for (int i = 0; i < 9; ++i)
        if (!std::isfinite(cam->R[i])) return fail(GS_ERR_INVALID, "R must be finite");
    for (int i = 0; i < 3; ++i)
        if (!std::isfinite(cam->t[i]) || !std::isfinite(cam->campos[i]))
            return fail(GS_ERR_INVALID, "t and campos must be finite");
    return GS_OK;
}

// Bytes of an element type, 0 for an unknown one.
size_t type_bytes(int32_t dtype) {
    return dtype == GS_F32 ? 4 : dtype == GS_BF16 || dtype == GS_F16 ? 2 : 0;
}

gs_status check_recurrence(const gs_recurrence* r, const char* who) {
    constexpr int32_t kMost = 1 << 30;
    if (!r) return fail(GS_ERR_INVALID, "%s: the description is NULL", who);
    if (!type_bytes(r->dtype)) return fail(GS_ERR_INVALID, "%s: unknown dtype %d", who, r->dtype);
    if (r->gating != GS_GATE_LINEAR && r->gating != GS_GATE_SIGMOID)
        return fail(GS_ERR_INVALID, "%s: unknown gating %d", who, r->gating);
    if (r->batch < 0 || r->steps < 0 || r->channels < 0 || r->batch > kMost || r->steps > kMost || r->channels > kMost)
        return fail(GS_ERR_INVALID, "%s: batch %d, steps %d or channels %d outside [0, 2^30]", who, r->batch, r->steps,
                    r->channels);
    if (r->gate_batch < 0 || r->gate_step < 0 || r->x_batch < 0 || r->x_step < 0)
        return fail(GS_ERR_INVALID, "%s: a stride is negative", who);
    if (!gs::recurrence_fits(*r))
        return fail(GS_ERR_INVALID, "%s: %d sequences of %d steps and %d channels are too many for one call", who,
                    r->batch, r->steps, r->channels);
    if ((uintptr_t)r->lengths & 3) return fail(GS_ERR_INVALID, "%s: lengths is not 4-byte aligned", who);
    return GS_OK;
}

// Whether every pointer is aligned to `bytes` (a power of two).
template <typename... P>
bool aligned(size_t bytes, P... p) {
    return !((0 | ... | (uintptr_t)p) & (bytes - 1));
}

gs::RecurrenceArgs recurrence_args(const gs_recurrence& r) {
    gs::RecurrenceArgs a{};
    a.gate_batch = r.gate_batch;
    a.gate_step = r.gate_step;
    a.x_batch = r.x_batch;
    a.x_step = r.x_step;
    a.lengths = r.lengths;
    a.restart = r.restart;
    a.batch = r.batch;
    a.steps = r.steps;
    a.channels = r.channels;
    return a;
}

gs_status check_delta_rule(const gs_delta_rule* r, bool backward, const char* who) {
    if (!r) return fail(GS_ERR_INVALID, "%s: the description is NULL", who);
    if (!type_bytes(r->dtype)) return fail(GS_ERR_INVALID, "%s: unknown dtype %d", who, r->dtype);
    if (r->batch < 0 || r->steps < 0 || (int64_t)r->batch * r->steps > (1 << 30) || r->steps > (1 << 30))
        return fail(GS_ERR_INVALID, "%s: batch %d and steps %d negative, or more than 2^30 in all", who, r->batch,
                    r->steps);
    if (r->key_heads < 1 || r->heads < 1 || r->heads > 4096 || r->heads % r->key_heads)
        return fail(GS_ERR_INVALID, "%s: heads %d is not a multiple of key_heads %d in [1, 4096]", who, r->heads,
                    r->key_heads);
    if (r->key_dim < 1 || r->value_dim < 1 || r->key_dim > GS_DELTA_MAX_DIM || r->value_dim > GS_DELTA_MAX_DIM)
        return fail(GS_ERR_INVALID, "%s: key_dim %d or value_dim %d outside [1, %d]", who, r->key_dim, r->value_dim,
                    GS_DELTA_MAX_DIM);
    const int64_t chunks = ((int64_t)r->steps + GS_DELTA_CHUNK - 1) / GS_DELTA_CHUNK;
    const int64_t each = (int64_t)r->heads * (chunks > 0 ? chunks : 1);
    if (r->batch > 0 && each > (1 << 24) / r->batch)
        return fail(GS_ERR_INVALID, "%s: %d sequences of %d steps and %d heads are too many for one call", who, r->batch,
                    r->steps, r->heads);
    if (!std::isfinite(r->scale)) return fail(GS_ERR_INVALID, "%s: scale is not finite", who);
    for (int64_t s : {r->q_batch, r->q_step, r->q_head, r->k_batch, r->k_step, r->k_head, r->v_batch, r->v_step,
                      r->v_head, r->decay_batch, r->decay_step, r->beta_batch, r->beta_step})
        if (s < 0) return fail(GS_ERR_INVALID, "%s: a stride is negative", who);
    // a chunk's rows are addressed by 32-bit offsets in bytes; calls of a few steps know no chunks, and one step no stride
    if (r->steps > (backward ? 1 : GS_DELTA_FEW))
        for (int64_t s : {r->q_step, r->k_step, r->v_step})
            if (s > (1 << 22)) return fail(GS_ERR_INVALID, "%s: a step stride of %lld is over 2^22", who, (long long)s);
    if ((uintptr_t)r->lengths & 3) return fail(GS_ERR_INVALID, "%s: lengths is not 4-byte aligned", who);
    return GS_OK;
}

gs_status check_scratch(const void* scratch, size_t bytes, size_t need, size_t to, const char* who) {
    if (need && (!scratch || bytes < need))
        return fail(GS_ERR_INVALID, "%s: scratch of %zu bytes is smaller than the required %zu", who,
                    scratch ? bytes : (size_t)0, need);
    if (need && ((uintptr_t)scratch & (to - 1)))
        return fail(GS_ERR_INVALID, "%s: scratch is not %zu-byte aligned", who, to);
    return GS_OK;
}

gs_status check_block_norm(const gs_block_norm* d, const char* who) {
    if (!d) return fail(GS_ERR_INVALID, "%s: the description is NULL", who);
    if (!type_bytes(d->dtype) || !type_bytes(d->weight_dtype))
        return fail(GS_ERR_INVALID, "%s: unknown dtype %d or weight_dtype %d", who, d->dtype, d->weight_dtype);
    if (d->weight_dtype != GS_F32 && d->weight_dtype != d->dtype)
        return fail(GS_ERR_INVALID, "%s: weight_dtype %d is neither GS_F32 nor dtype %d", who, d->weight_dtype, d->dtype);
    for (int32_t k : {d->post, d->pre})
        if (k != GS_BLOCK_NORM_NONE && k != GS_BLOCK_NORM_RMS && k != GS_BLOCK_NORM_LAYER)
            return fail(GS_ERR_INVALID, "%s: unknown norm %d", who, k);
    if (d->gating != GS_BLOCK_GATE_NONE && d->gating != GS_BLOCK_GATE_SIGMOID && d->gating != GS_BLOCK_GATE_SILU)
        return fail(GS_ERR_INVALID, "%s: unknown gating %d", who, d->gating);
    if (d->outer < 0 || d->outer > (1 << 30) || d->inner < 1 || d->outer * d->inner > (1 << 30))
        return fail(GS_ERR_INVALID, "%s: outer %lld negative, inner %d below 1, or more than 2^30 rows in all", who,
                    (long long)d->outer, d->inner);
    if (d->width < 1 || d->width > GS_BLOCK_NORM_MAX_WIDTH)
        return fail(GS_ERR_INVALID, "%s: width %d outside [1, %d]", who, d->width, GS_BLOCK_NORM_MAX_WIDTH);
    if (!(d->eps >= 0.0f) || !std::isfinite(d->eps))
        return fail(GS_ERR_INVALID, "%s: eps %g is negative or not finite", who, d->eps);
    for (int64_t s : {d->y_outer, d->y_inner, d->gate_outer, d->gate_inner, d->residual_outer, d->residual_inner})
        if (s < 0) return fail(GS_ERR_INVALID, "%s: a stride is negative", who);
    return GS_OK;
}

// The inputs that both directions of the block norms take.
gs_status check_block_inputs(const gs_block_norm& d, const gs::BlockNormArgs& a, const char* who) {
    if (!a.y || (d.gating != GS_BLOCK_GATE_NONE && !a.gate))
        return fail(GS_ERR_INVALID, "%s: a required pointer is NULL", who);
    if (d.gating == GS_BLOCK_GATE_NONE && a.gate) return fail(GS_ERR_INVALID, "%s: gate is given without gating", who);
    if (d.post == GS_BLOCK_NORM_NONE && (a.post_weight || a.post_bias))
        return fail(GS_ERR_INVALID, "%s: post_weight or post_bias is given without the post norm", who);
    if (d.pre == GS_BLOCK_NORM_NONE && (a.pre_weight || a.pre_bias))
        return fail(GS_ERR_INVALID, "%s: pre_weight or pre_bias is given without the pre norm", who);
    if (!aligned(type_bytes(d.dtype), a.y, a.gate, a.residual, a.out, a.norm, a.grad_out, a.grad_norm, a.grad_y,
                 a.grad_gate, a.grad_residual) ||
        !aligned(type_bytes(d.weight_dtype), a.post_weight, a.post_bias, a.scale, a.pre_weight, a.pre_bias) ||
        !aligned(4, a.sums[0], a.sums[1], a.sums[2], a.sums[3], a.sums[4]))
        return fail(GS_ERR_INVALID, "%s: a buffer is not aligned to its type", who);
    return GS_OK;
}

// Checks that the lists of gs_grad_norm, gs_clip_grads and gs_adam_step share.
gs_status check_list(const void* tensors, int32_t n, const void* scratch, const char* who) {
    if (n < 0 || n > GS_MAX_TENSORS)
        return fail(GS_ERR_INVALID, "%s: n_tensors = %d outside [0, %d]", who, n, GS_MAX_TENSORS);
    if (n && !tensors) return fail(GS_ERR_INVALID, "%s: tensors is NULL", who);
    if (!scratch) return fail(GS_ERR_INVALID, "%s: scratch is NULL", who);
    if (!aligned(8, scratch)) return fail(GS_ERR_INVALID, "%s: scratch is not 8-byte aligned", who);
    return GS_OK;
}

gs_status check_count(int64_t count, int i, const char* who) {
    if (count < 0 || count > GS_MAX_TENSOR_COUNT)
        return fail(GS_ERR_INVALID, "%s: tensor %d has count %lld outside [0, 2^35]", who, i, (long long)count);
    return GS_OK;
}

gs_status check_grads(const gs_grad_tensor* tensors, int32_t n, int32_t kind, const float* norm, const void* scratch,
                      bool out, const char* who) {
    if (gs_status s = check_list(tensors, n, scratch, who)) return s;
    if (kind != GS_NORM_L2 && kind != GS_NORM_MAX) return fail(GS_ERR_INVALID, "%s: unknown kind %d", who, kind);
    if (!norm || !aligned(4, norm)) return fail(GS_ERR_INVALID, "%s: norm is NULL or misaligned", who);
    for (int i = 0; i < n; ++i) {
        const gs_grad_tensor& t = tensors[i];
        if (gs_status s = check_count(t.count, i, who)) return s;
        if (!t.count) continue;
        const size_t b = type_bytes(t.dtype);
        if (!b) return fail(GS_ERR_INVALID, "%s: tensor %d has unknown dtype %d", who, i, t.dtype);
        if (!t.grad || (out && !t.out)) return fail(GS_ERR_INVALID, "%s: tensor %d has a NULL pointer", who, i);
        if (!aligned(b, t.grad, out ? t.out : nullptr))
            return fail(GS_ERR_INVALID, "%s: tensor %d is not aligned to its type", who, i);
    }
    return GS_OK;
}

}  // namespace

extern "C" {

void gs_constants(float out[9]) {
    out[0] = (float)gs::kTile;
    out[1] = gs::kDilation;
    out[2] = gs::kZNear;
    out[3] = gs::kFrustumClamp;
    out[4] = gs::kDiscFloor;
    out[5] = gs::kSigma;
    out[6] = gs::kAlphaMin;
    out[7] = gs::kAlphaMax;
    out[8] = gs::kTStop;
}

const char* gs_last_error(void) { return g_last_error.c_str(); }

void gs_version(int32_t out[3]) {
    out[0] = 0;
    out[1] = 1;
    out[2] = 0;
}

gs_status gs_preprocess_ex(const gs_camera* cam, int32_t n, const float* means, const float* scales,
                           const float* quats, const float* opacity, const float* sh,
                           int32_t sh_degree, const float* rgb_in, float* xy_depth, float* conic_op,
                           float* rgb, uint32_t* tiles_touched, uint32_t flags, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_camera(cam)) return s;
    if (flags & ~(uint32_t)GS_TILES_ELLIPSE) return fail(GS_ERR_INVALID, "unknown flags 0x%x", flags);
    if (n < 0 || n > GS_MAX_GAUSSIANS) return fail(GS_ERR_INVALID, "n = %d outside [0, %d]", n, GS_MAX_GAUSSIANS);
    if (n == 0) return GS_OK;
    if (!means || !scales || !quats || !opacity || !xy_depth || !conic_op || !rgb || !tiles_touched)
        return fail(GS_ERR_INVALID, "gs_preprocess: a required pointer is NULL");
    if (sh) {
        if (sh_degree < 0 || sh_degree > 3) return fail(GS_ERR_INVALID, "sh_degree %d outside 0..3", sh_degree);
    } else if (!rgb_in) {
        return fail(GS_ERR_INVALID, "gs_preprocess: rgb_in is required when sh is NULL");
    }
    if (((uintptr_t)xy_depth | (uintptr_t)conic_op | (uintptr_t)rgb) & 15)
        return fail(GS_ERR_INVALID, "gs_preprocess: float4 outputs must be 16-byte aligned");
    return hip_check(gs::launch_preprocess(*cam, n, means, scales, quats, opacity, sh, sh_degree,
                                           rgb_in, (float4*)xy_depth, (float4*)conic_op,
                                           (float4*)rgb, tiles_touched, flags, (hipStream_t)stream),
                     "gs_preprocess launch");
}

gs_status gs_preprocess(const gs_camera* cam, int32_t n, const float* means, const float* scales,
                        const float* quats, const float* opacity, const float* sh,
                        int32_t sh_degree, const float* rgb_in, float* xy_depth, float* conic_op,
                        float* rgb, uint32_t* tiles_touched, void* stream) {
    return gs_preprocess_ex(cam, n, means, scales, quats, opacity, sh, sh_degree, rgb_in, xy_depth, conic_op,
                            rgb, tiles_touched, GS_TILES_SQUARE, stream);
}

gs_status gs_preprocess_views(const gs_camera* cams, int32_t n_views, int32_t n, const float* means,
                              const float* scales, const float* quats, const float* opacity, const float* sh,
                              int32_t sh_degree, const float* rgb_in, float* xy_depth, float* conic_op, float* rgb,
                              uint32_t* tiles_touched, uint32_t flags, void* stream) {
    g_last_error.clear();
    if (!cams) return fail(GS_ERR_INVALID, "gs_preprocess_views: cams is NULL");
    if (n_views < 1 || n_views > GS_MAX_VIEWS)
        return fail(GS_ERR_INVALID, "gs_preprocess_views: n_views = %d outside [1, %d]", n_views, GS_MAX_VIEWS);
    gs::CameraSet set{};
    set.n = n_views;
    for (int v = 0; v < n_views; ++v) {
        if (gs_status s = check_camera(&cams[v])) return s;
        if (cams[v].width != cams[0].width || cams[v].height != cams[0].height)
            return fail(GS_ERR_INVALID, "gs_preprocess_views: camera %d is not %dx%d like camera 0", v,
                        cams[0].width, cams[0].height);
        set.cam[v] = cams[v];
    }
    if (n < 0 || (int64_t)n * n_views > GS_MAX_GAUSSIANS)
        return fail(GS_ERR_INVALID, "n = %d (x %d views) outside [0, %d]", n, n_views, GS_MAX_GAUSSIANS);
    if (sh && (sh_degree < 0 || sh_degree > 3))
        return fail(GS_ERR_INVALID, "sh_degree %d outside [0, 3]", sh_degree);
    if (flags & ~(uint32_t)GS_TILES_ELLIPSE) return fail(GS_ERR_INVALID, "gs_preprocess_views: unknown flags");
    if (n == 0) return GS_OK;
    if (!means || !scales || !quats || !opacity || (!sh && !rgb_in) || !xy_depth || !conic_op || !rgb ||
        !tiles_touched)
        return fail(GS_ERR_INVALID, "gs_preprocess_views: a required pointer is NULL");
    if (((uintptr_t)xy_depth | (uintptr_t)conic_op | (uintptr_t)rgb) & 15)
        return fail(GS_ERR_INVALID, "gs_preprocess_views: float4 outputs must be 16-byte aligned");
    return hip_check(gs::launch_preprocess_views(set, n, means, scales, quats, opacity, sh, sh_degree, rgb_in,
                                                 (float4*)xy_depth, (float4*)conic_op, (float4*)rgb, tiles_touched,
                                                 flags, (hipStream_t)stream),
                     "gs_preprocess_views launch");
}

gs_status gs_preprocess_bwd(const gs_camera* cam, int32_t n, const float* means, const float* scales,
                            const float* quats, const float* sh, int32_t sh_degree,
                            const uint32_t* tiles_touched, const float* grad_mean2d,
                            const float* grad_conic_op, const float* grad_rgb, float* grad_means,
                            float* grad_scales, float* grad_quats, float* grad_opacity, float* grad_sh,
                            float* grad_rgb_in, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_camera(cam)) return s;
    if (n < 0 || n > GS_MAX_GAUSSIANS) return fail(GS_ERR_INVALID, "n = %d outside [0, %d]", n, GS_MAX_GAUSSIANS);
    if (n == 0) return GS_OK;
    if (!means || !scales || !quats || !tiles_touched || !grad_mean2d || !grad_conic_op || !grad_rgb ||
        !grad_means || !grad_scales || !grad_quats || !grad_opacity)
        return fail(GS_ERR_INVALID, "gs_preprocess_bwd: a required pointer is NULL");
    if (sh) {
        if (sh_degree < 0 || sh_degree > 3) return fail(GS_ERR_INVALID, "sh_degree %d outside 0..3", sh_degree);
        if (!grad_sh) return fail(GS_ERR_INVALID, "gs_preprocess_bwd: grad_sh is required when sh is given");
    } else if (!grad_rgb_in) {
        return fail(GS_ERR_INVALID, "gs_preprocess_bwd: grad_rgb_in is required when sh is NULL");
    }
    if (((uintptr_t)grad_conic_op | (uintptr_t)grad_rgb) & 15)
        return fail(GS_ERR_INVALID, "gs_preprocess_bwd: float4 gradients must be 16-byte aligned");
    if ((uintptr_t)grad_mean2d & 7)
        return fail(GS_ERR_INVALID, "gs_preprocess_bwd: grad_mean2d must be 8-byte aligned");
    return hip_check(gs::launch_preprocess_bwd(*cam, n, means, scales, quats, sh, sh_degree, tiles_touched,
                                               (const float2*)grad_mean2d, (const float4*)grad_conic_op,
                                               (const float4*)grad_rgb, grad_means, grad_scales, grad_quats,
                                               grad_opacity, sh ? grad_sh : nullptr, sh ? nullptr : grad_rgb_in,
                                               (hipStream_t)stream),
                     "gs_preprocess_bwd launch");
}

namespace {

// Checks shared by the blocking and the asynchronous binning entry points;
// on GS_OK with scratch != NULL, *s is laid out in scratch.
gs_status bin_args(const char* fn, const gs_camera* cam, int32_t n, const float* xy_depth,
                   const uint32_t* tiles_touched, const uint64_t* keys, const uint32_t* point_list,
                   int64_t capacity, void* scratch, size_t* scratch_bytes, bool* size_query, gs::BinScratch* s,
                   int32_t n_views = 1) {
    if (gs_status st = check_camera(cam)) return st;
    if (n_views < 1 || n_views > GS_MAX_VIEWS)
        return fail(GS_ERR_INVALID, "%s: n_views = %d outside [1, %d]", fn, n_views, GS_MAX_VIEWS);
    if (n < 0 || (int64_t)n * n_views > GS_MAX_GAUSSIANS)
        return fail(GS_ERR_INVALID, "n = %d (x %d views) outside [0, %d]", n, n_views, GS_MAX_GAUSSIANS);
    if ((int64_t)gs::tiles_x(*cam) * gs::tiles_y(*cam) * n_views > (1 << 24))
        return fail(GS_ERR_INVALID, "%s: more than 2^24 tiles", fn);
    n *= n_views;
    if (capacity < 0 || capacity > (int64_t)UINT32_MAX)
        return fail(GS_ERR_INVALID, "capacity %lld outside [0, 2^32 - 1]", (long long)capacity);
    if (!scratch_bytes) return fail(GS_ERR_INVALID, "%s: scratch_bytes is NULL", fn);
    const size_t need = gs::bin_scratch_layout(n, capacity, nullptr, nullptr);
    *size_query = scratch == nullptr;
    if (*size_query) {
        *scratch_bytes = need;
        return GS_OK;
    }
    if (*scratch_bytes < need)
        return fail(GS_ERR_INVALID, "%s: scratch of %zu bytes is smaller than the %zu required", fn,
                    *scratch_bytes, need);
    if ((uintptr_t)scratch & 255) return fail(GS_ERR_INVALID, "%s: scratch must be 256-byte aligned", fn);
    if (n > 0 && (!xy_depth || !tiles_touched || (capacity > 0 && (!keys || !point_list))))
        return fail(GS_ERR_INVALID, "%s: a required pointer is NULL", fn);
    if (n > 0 && ((uintptr_t)xy_depth & 15)) return fail(GS_ERR_INVALID, "%s: xy_depth must be 16-byte aligned", fn);
    gs::bin_scratch_layout(n, capacity, s, scratch);
    return GS_OK;
}

// The tile-test flags of the binning entry points: the ellipse test reads
// the conic of every splat.
gs_status tile_test_args(const char* fn, int32_t n, const float* conic_op, uint32_t flags) {
    if (flags & ~(uint32_t)GS_TILES_ELLIPSE) return fail(GS_ERR_INVALID, "%s: unknown flags 0x%x", fn, flags);
    if ((flags & GS_TILES_ELLIPSE) && n > 0 && (!conic_op || ((uintptr_t)conic_op & 15)))
        return fail(GS_ERR_INVALID, "%s: the ellipse test needs a 16-byte aligned conic_op", fn);
    return GS_OK;
}

}  // namespace

gs_status gs_bin_and_sort_ex(const gs_camera* cam, int32_t n, const float* xy_depth, const float* conic_op,
                             const uint32_t* tiles_touched, uint64_t* keys, uint32_t* point_list,
                             int64_t capacity, void* scratch, size_t* scratch_bytes, int64_t* n_entries,
                             uint32_t flags, void* stream) {
    g_last_error.clear();
    gs::BinScratch s{};
    bool query = false;
    if (gs_status e = bin_args("gs_bin_and_sort", cam, n, xy_depth, tiles_touched, keys, point_list, capacity,
                               scratch, scratch_bytes, &query, &s))
        return e;
    if (query) return GS_OK;
    if (gs_status e = tile_test_args("gs_bin_and_sort", n, conic_op, flags)) return e;
    if (!n_entries) return fail(GS_ERR_INVALID, "gs_bin_and_sort: n_entries is NULL");
    *n_entries = 0;
    if (n == 0) return GS_OK;
    hipStream_t st = (hipStream_t)stream;
    if (gs_status e = hip_check(gs::launch_bin_and_sort(*cam, 1, n, (const float4*)xy_depth, (const float4*)conic_op,
                                                        tiles_touched, keys, point_list, (uint32_t)capacity, s,
                                                        nullptr, flags, st),
                                "bin_and_sort launch"))
        return e;
    // the entry count, once everything is enqueued
    uint64_t total = 0;
    if (gs_status e = hip_check(hipMemcpyAsync(&total, s.total, sizeof(total), hipMemcpyDeviceToHost, st),
                                "entry count copy"))
        return e;
    if (gs_status e = hip_check(hipStreamSynchronize(st), "entry count sync")) return e;
    *n_entries = (int64_t)total;
    if (total > (uint64_t)UINT32_MAX)
        return fail(GS_ERR_OVERFLOW, "%llu entries do not fit in 32 bits", (unsigned long long)total);
    if ((int64_t)total > capacity)
        return fail(GS_ERR_CAPACITY, "%llu entries exceed the capacity %lld", (unsigned long long)total,
                    (long long)capacity);
    return GS_OK;
}

gs_status gs_bin_and_sort(const gs_camera* cam, int32_t n, const float* xy_depth,
                          const uint32_t* tiles_touched, uint64_t* keys, uint32_t* point_list,
                          int64_t capacity, void* scratch, size_t* scratch_bytes,
                          int64_t* n_entries, void* stream) {
    return gs_bin_and_sort_ex(cam, n, xy_depth, nullptr, tiles_touched, keys, point_list, capacity, scratch,
                              scratch_bytes, n_entries, GS_TILES_SQUARE, stream);
}

gs_status gs_bin_and_sort_views_async(const gs_camera* cam, int32_t n_views, int32_t n, const float* xy_depth,
                                      const float* conic_op, const uint32_t* tiles_touched, uint64_t* keys,
                                      uint32_t* point_list, int64_t capacity, void* scratch, size_t* scratch_bytes,
                                      uint64_t* n_entries_dev, uint32_t flags, void* stream) {
    g_last_error.clear();
    gs::BinScratch s{};
    bool query = false;
    if (gs_status e = bin_args("gs_bin_and_sort_async", cam, n, xy_depth, tiles_touched, keys, point_list,
                               capacity, scratch, scratch_bytes, &query, &s, n_views))
        return e;
    if (query) return GS_OK;
    const int32_t n_all = n * n_views;
    if (gs_status e = tile_test_args("gs_bin_and_sort_async", n_all, conic_op, flags)) return e;
    if (!n_entries_dev || ((uintptr_t)n_entries_dev & 7))
        return fail(GS_ERR_INVALID, "gs_bin_and_sort_async: n_entries_dev must be an 8-byte aligned device pointer");
    hipStream_t st = (hipStream_t)stream;
    if (n_all == 0)
        return hip_check(gs::launch_fill_u32((uint32_t*)n_entries_dev, 2, 0u, st), "entry count clear");
    return hip_check(gs::launch_bin_and_sort(*cam, n_views, n_all, (const float4*)xy_depth, (const float4*)conic_op,
                                             tiles_touched, keys, point_list, (uint32_t)capacity, s, n_entries_dev,
                                             flags, st),
                     "bin_and_sort launch");
}

gs_status gs_bin_and_sort_async_ex(const gs_camera* cam, int32_t n, const float* xy_depth, const float* conic_op,
                                   const uint32_t* tiles_touched, uint64_t* keys, uint32_t* point_list,
                                   int64_t capacity, void* scratch, size_t* scratch_bytes,
                                   uint64_t* n_entries_dev, uint32_t flags, void* stream) {
    return gs_bin_and_sort_views_async(cam, 1, n, xy_depth, conic_op, tiles_touched, keys, point_list, capacity,
                                       scratch, scratch_bytes, n_entries_dev, flags, stream);
}

gs_status gs_bin_and_sort_async(const gs_camera* cam, int32_t n, const float* xy_depth,
                                const uint32_t* tiles_touched, uint64_t* keys, uint32_t* point_list,
                                int64_t capacity, void* scratch, size_t* scratch_bytes,
                                uint64_t* n_entries_dev, void* stream) {
    return gs_bin_and_sort_async_ex(cam, n, xy_depth, nullptr, tiles_touched, keys, point_list, capacity,
                                    scratch, scratch_bytes, n_entries_dev, GS_TILES_SQUARE, stream);
}

}  // extern "C"

namespace {

// Device address of `scratch` on each device, looked up on the first
// no-allocation call made with that device current.
constexpr int kMaxDevices = 64;
std::mutex g_static_mu;
void* g_static_ptr[kMaxDevices] = {};

gs_status static_scratch(void** out) {
    int dev = -1;
    if (gs_status e = hip_check(hipGetDevice(&dev), "hipGetDevice")) return e;
    if (dev < 0 || dev >= kMaxDevices) return fail(GS_ERR_INVALID, "device %d outside [0, %d)", dev, kMaxDevices);
    std::lock_guard<std::mutex> lock(g_static_mu);
    if (!g_static_ptr[dev]) {
        void* p = nullptr;
        if (gs_status e = hip_check(hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)), "hipGetSymbolAddress(scratch)"))
            return e;
        if (!p || ((uintptr_t)p & 255)) return fail(GS_ERR_HIP, "static workspace has no 256-byte aligned address");
        g_static_ptr[dev] = p;
    }
    *out = g_static_ptr[dev];
    return GS_OK;
}

}  // namespace

extern "C" {

gs_status gs_bin_and_sort_async_noalloc(const gs_camera* cam, int32_t n, const float* xy_depth,
                                        const float* conic_op, const uint32_t* tiles_touched, uint64_t* keys,
                                        uint32_t* point_list, int64_t capacity, uint64_t* n_entries_dev,
                                        uint32_t flags, void* stream) {
    g_last_error.clear();
    const char* fn = "gs_bin_and_sort_async_noalloc";
    gs::BinScratch s{};
    bool query = false;
    size_t need = 0;
    // the size first (no device call): arguments and the workspace this call needs
    if (gs_status e = bin_args(fn, cam, n, xy_depth, tiles_touched, keys, point_list, capacity, nullptr, &need,
                               &query, &s))
        return e;
    if (need > (size_t)GS_NOALLOC_SCRATCH_BYTES)
        return fail(GS_ERR_INVALID,
                    "%s: n = %d and capacity = %lld need %zu bytes of workspace, more than the fixed %zu; "
                    "use gs_bin_and_sort_async_ex with a caller-owned workspace",
                    fn, n, (long long)capacity, need, (size_t)GS_NOALLOC_SCRATCH_BYTES);
    void* ws = nullptr;
    if (gs_status e = static_scratch(&ws)) return e;
    size_t have = GS_NOALLOC_SCRATCH_BYTES;
    if (gs_status e = bin_args(fn, cam, n, xy_depth, tiles_touched, keys, point_list, capacity, ws, &have, &query,
                               &s))
        return e;
    if (gs_status e = tile_test_args(fn, n, conic_op, flags)) return e;
    if (!n_entries_dev || ((uintptr_t)n_entries_dev & 7))
        return fail(GS_ERR_INVALID, "%s: n_entries_dev must be an 8-byte aligned device pointer", fn);
    hipStream_t st = (hipStream_t)stream;
    if (n == 0) return hip_check(gs::launch_fill_u32((uint32_t*)n_entries_dev, 2, 0u, st), "entry count clear");
    return hip_check(gs::launch_bin_and_sort(*cam, 1, n, (const float4*)xy_depth, (const float4*)conic_op,
                                             tiles_touched, keys, point_list, (uint32_t)capacity, s, n_entries_dev,
                                             flags, st),
                     "bin_and_sort launch");
}

namespace {

gs_status appearance_args(const char* fn, const gs_camera* cam, int32_t n, int32_t L, int32_t H) {
    if (gs_status s = check_camera(cam)) return s;
    if (n < 0 || n > GS_MAX_GAUSSIANS) return fail(GS_ERR_INVALID, "%s: n = %d outside [0, %d]", fn, n, GS_MAX_GAUSSIANS);
    if (L < 1 || L > GS_APP_MAX_LATENT) return fail(GS_ERR_INVALID, "%s: n_latent %d outside [1, %d]", fn, L, GS_APP_MAX_LATENT);
    if (H < 1 || H > GS_APP_MAX_HIDDEN) return fail(GS_ERR_INVALID, "%s: n_hidden %d outside [1, %d]", fn, H, GS_APP_MAX_HIDDEN);
    return GS_OK;
}

}  // namespace

gs_status gs_appearance_fwd(const gs_camera* cam, int32_t n, const float* means, const float* latent,
                            int32_t n_latent, int32_t n_hidden, const float* weights, float* rgb, void* stream) {
    g_last_error.clear();
    if (gs_status s = appearance_args("gs_appearance_fwd", cam, n, n_latent, n_hidden)) return s;
    if (n == 0) return GS_OK;
    if (!means || !latent || !weights || !rgb) return fail(GS_ERR_INVALID, "gs_appearance_fwd: a required pointer is NULL");
    return hip_check(gs::launch_appearance_fwd(*cam, n, means, latent, n_latent, n_hidden, weights, rgb,
                                               (hipStream_t)stream),
                     "gs_appearance_fwd launch");
}

gs_status gs_appearance_bwd(const gs_camera* cam, int32_t n, const float* means, const float* latent,
                            int32_t n_latent, int32_t n_hidden, const float* weights, const float* grad_rgb,
                            float* grad_latent, float* grad_weights, void* scratch, size_t* scratch_bytes,
                            void* stream) {
    g_last_error.clear();
    if (gs_status s = appearance_args("gs_appearance_bwd", cam, n, n_latent, n_hidden)) return s;
    if (!scratch_bytes) return fail(GS_ERR_INVALID, "gs_appearance_bwd: scratch_bytes is NULL");
    const size_t need = gs::appearance_bwd_scratch(n, n_latent, n_hidden);
    if (!scratch) {
        *scratch_bytes = need;
        return GS_OK;
    }
    if (*scratch_bytes < need)
        return fail(GS_ERR_INVALID, "gs_appearance_bwd: scratch of %zu bytes is smaller than the %zu required",
                    *scratch_bytes, need);
    if ((uintptr_t)scratch & 3) return fail(GS_ERR_INVALID, "gs_appearance_bwd: scratch must be 4-byte aligned");
    if (!grad_weights || (n > 0 && (!means || !latent || !weights || !grad_rgb || !grad_latent)))
        return fail(GS_ERR_INVALID, "gs_appearance_bwd: a required pointer is NULL");
    return hip_check(gs::launch_appearance_bwd(*cam, n, means, latent, n_latent, n_hidden, weights, grad_rgb,
                                               grad_latent, grad_weights, (float*)scratch, (hipStream_t)stream),
                     "gs_appearance_bwd launch");
}

gs_status gs_tile_ranges(const gs_camera* cam, const uint64_t* keys, int64_t n_entries,
                         uint32_t* ranges, uint32_t* tile_order, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_camera(cam)) return s;
    if (n_entries < 0 || n_entries > (int64_t)UINT32_MAX)
        return fail(GS_ERR_INVALID, "n_entries %lld outside [0, 2^32 - 1]", (long long)n_entries);
    if (!ranges || (n_entries > 0 && !keys)) return fail(GS_ERR_INVALID, "gs_tile_ranges: NULL pointer");
    const int n_tiles = gs::tiles_x(*cam) * gs::tiles_y(*cam);
    return hip_check(gs::launch_tile_ranges(keys, (uint32_t)n_entries, nullptr, 0u, n_tiles, ranges, tile_order,
                                            nullptr, (hipStream_t)stream),
                     "tile ranges launch");
}

gs_status gs_tile_ranges_async(const gs_camera* cam, const uint64_t* keys, const uint64_t* n_entries_dev,
                               int64_t capacity, uint32_t* ranges, uint32_t* tile_order, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_camera(cam)) return s;
    if (capacity < 0 || capacity > (int64_t)UINT32_MAX)
        return fail(GS_ERR_INVALID, "capacity %lld outside [0, 2^32 - 1]", (long long)capacity);
    if (!ranges || !n_entries_dev || ((uintptr_t)n_entries_dev & 7) || (capacity > 0 && !keys))
        return fail(GS_ERR_INVALID, "gs_tile_ranges_async: NULL or misaligned pointer");
    const int n_tiles = gs::tiles_x(*cam) * gs::tiles_y(*cam);
    return hip_check(gs::launch_tile_ranges(keys, 0u, n_entries_dev, (uint32_t)capacity, n_tiles, ranges,
                                            tile_order, nullptr, (hipStream_t)stream),
                     "tile ranges launch");
}

gs_status gs_tile_ranges_ex(const gs_camera* cam, int32_t n_views, const uint64_t* keys, int64_t n_entries,
                            const uint64_t* n_entries_dev, int64_t capacity, uint32_t* ranges,
                            uint32_t* tile_order, uint32_t* chunks, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_camera(cam)) return s;
    if (n_views < 1 || n_views > GS_MAX_VIEWS)
        return fail(GS_ERR_INVALID, "gs_tile_ranges_ex: n_views = %d outside [1, %d]", n_views, GS_MAX_VIEWS);
    if (capacity < 0 || capacity > (int64_t)UINT32_MAX)
        return fail(GS_ERR_INVALID, "capacity %lld outside [0, 2^32 - 1]", (long long)capacity);
    if (!n_entries_dev && (n_entries < 0 || n_entries > capacity))
        return fail(GS_ERR_INVALID, "n_entries %lld outside [0, capacity %lld]", (long long)n_entries,
                    (long long)capacity);
    if (!ranges || (capacity > 0 && !keys) || ((uintptr_t)n_entries_dev & 7) || ((uintptr_t)chunks & 15))
        return fail(GS_ERR_INVALID, "gs_tile_ranges_ex: NULL or misaligned pointer");
    const int n_tiles = gs::tiles_x(*cam) * gs::tiles_y(*cam) * n_views;
    return hip_check(gs::launch_tile_ranges(keys, n_entries_dev ? 0u : (uint32_t)n_entries, n_entries_dev,
                                            (uint32_t)capacity, n_tiles, ranges, tile_order, chunks,
                                            (hipStream_t)stream),
                     "tile ranges launch");
}

gs_status gs_composite_fwd(const gs_camera* cam, const uint32_t* ranges, const uint32_t* point_list,
                           const float* xy_depth, const float* conic_op, const float* rgb,
                           const float bg[3], float* image, float* final_T, uint32_t* n_contrib,
                           uint32_t* n_examined, const uint32_t* tile_order, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_camera(cam)) return s;
    if (!ranges || !bg || !image || !final_T || !n_contrib)
        return fail(GS_ERR_INVALID, "gs_composite_fwd: a required pointer is NULL");
    if (((uintptr_t)xy_depth | (uintptr_t)conic_op | (uintptr_t)rgb) & 15)
        return fail(GS_ERR_INVALID, "gs_composite_fwd: float4 inputs must be 16-byte aligned");
    const float3 b = make_float3(bg[0], bg[1], bg[2]);
    return hip_check(gs::launch_composite_fwd(*cam, 1, ranges, point_list, (const float4*)xy_depth,
                                              (const float4*)conic_op, (const float4*)rgb, b, image,
                                              final_T, n_contrib, n_examined, tile_order, nullptr, 0u,
                                              nullptr, nullptr, (hipStream_t)stream),
                     "composite fwd launch");
}

gs_status gs_composite_fwd_ex(const gs_camera* cam, int32_t n_views, const uint32_t* ranges,
                              const uint32_t* point_list, const float* xy_depth, const float* conic_op,
                              const float* rgb, const float bg[3], float* image, float* final_T, uint32_t* n_contrib,
                              uint32_t* n_examined, const uint32_t* tile_order, int64_t capacity,
                              float* ckpt, const uint32_t* chunks, void* part, void* stream) {
    g_last_error.clear();
    if (n_views < 1 || n_views > GS_MAX_VIEWS)
        return fail(GS_ERR_INVALID, "gs_composite_fwd_ex: n_views = %d outside [1, %d]", n_views, GS_MAX_VIEWS);
    if (!ckpt && !chunks && n_views == 1)
        return gs_composite_fwd(cam, ranges, point_list, xy_depth, conic_op, rgb, bg, image, final_T, n_contrib,
                                n_examined, tile_order, stream);
    if (gs_status s = check_camera(cam)) return s;
    if (capacity < 0 || capacity > (int64_t)UINT32_MAX)
        return fail(GS_ERR_INVALID, "gs_composite_fwd_ex: capacity %lld outside [0, 2^32 - 1]", (long long)capacity);
    if (!bg || !image || !final_T || !n_contrib || (!chunks && !ranges))
        return fail(GS_ERR_INVALID, "gs_composite_fwd_ex: a required pointer is NULL");
    if (chunks && !part) return fail(GS_ERR_INVALID, "gs_composite_fwd_ex: chunks without the part workspace");
    if (((uintptr_t)xy_depth | (uintptr_t)conic_op | (uintptr_t)rgb | (uintptr_t)ckpt | (uintptr_t)chunks |
         (uintptr_t)part) & 15)
        return fail(GS_ERR_INVALID, "gs_composite_fwd_ex: float4 buffers must be 16-byte aligned");
    const float3 b = make_float3(bg[0], bg[1], bg[2]);
    return hip_check(gs::launch_composite_fwd(*cam, n_views, ranges, point_list, (const float4*)xy_depth,
                                              (const float4*)conic_op, (const float4*)rgb, b, image,
                                              final_T, n_contrib, n_examined, tile_order, (float4*)ckpt,
                                              (uint32_t)capacity, chunks, part, (hipStream_t)stream),
                     "composite fwd launch");
}

size_t gs_composite_part_bytes(const gs_camera* cam, int32_t n_views, int64_t capacity) {
    if (!cam || check_camera(cam) != GS_OK || capacity < 0 || capacity > (int64_t)UINT32_MAX) return 0;
    if (n_views < 1 || n_views > GS_MAX_VIEWS) return 0;
    return gs::composite_part_bytes(*cam, n_views, (uint32_t)capacity);
}

gs_status gs_composite_bwd(const gs_camera* cam, int32_t n, const uint32_t* ranges,
                           const uint32_t* point_list, const float* xy_depth,
                           const float* conic_op, const float* rgb, const float bg[3],
                           const float* final_T, const uint32_t* n_contrib,
                           const float* dL_dimage, float* grad_mean2d, float* grad_conic_op,
                           float* grad_rgb, const uint32_t* tile_order, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_camera(cam)) return s;
    if (n < 0 || n > GS_MAX_GAUSSIANS) return fail(GS_ERR_INVALID, "n = %d outside [0, %d]", n, GS_MAX_GAUSSIANS);
    if (!ranges || !bg || !final_T || !n_contrib || !dL_dimage)
        return fail(GS_ERR_INVALID, "gs_composite_bwd: a required pointer is NULL");
    if (n > 0 && (!grad_mean2d || !grad_conic_op || !grad_rgb))
        return fail(GS_ERR_INVALID, "gs_composite_bwd: a gradient pointer is NULL");
    if (((uintptr_t)xy_depth | (uintptr_t)conic_op | (uintptr_t)rgb | (uintptr_t)grad_conic_op |
         (uintptr_t)grad_rgb) & 15 || ((uintptr_t)grad_mean2d & 7))
        return fail(GS_ERR_INVALID, "gs_composite_bwd: misaligned vector buffer");
    const float3 b = make_float3(bg[0], bg[1], bg[2]);
    return hip_check(gs::launch_composite_bwd(*cam, 1, n, ranges, point_list, (const float4*)xy_depth,
                                              (const float4*)conic_op, (const float4*)rgb, b, final_T,
                                              n_contrib, dL_dimage, (float2*)grad_mean2d,
                                              (float4*)grad_conic_op, (float4*)grad_rgb, tile_order,
                                              nullptr, 0u, nullptr, nullptr, (hipStream_t)stream),
                     "composite bwd launch");
}

gs_status gs_composite_bwd_ex(const gs_camera* cam, int32_t n_views, int32_t n, const uint32_t* ranges,
                              const uint32_t* point_list, const uint32_t* chunks, int64_t capacity,
                              const float* xy_depth, const float* conic_op, const float* rgb,
                              const float bg[3], const float* image, const float* final_T,
                              const uint32_t* n_contrib, const float* ckpt, const float* dL_dimage,
                              float* grad_mean2d, float* grad_conic_op, float* grad_rgb, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_camera(cam)) return s;
    if (n_views < 1 || n_views > GS_MAX_VIEWS)
        return fail(GS_ERR_INVALID, "gs_composite_bwd_ex: n_views = %d outside [1, %d]", n_views, GS_MAX_VIEWS);
    if (n < 0 || n > GS_MAX_GAUSSIANS) return fail(GS_ERR_INVALID, "n = %d outside [0, %d]", n, GS_MAX_GAUSSIANS);
    if (capacity < 0 || capacity > (int64_t)UINT32_MAX)
        return fail(GS_ERR_INVALID, "gs_composite_bwd_ex: capacity %lld outside [0, 2^32 - 1]", (long long)capacity);
    if (!ranges || !bg || !final_T || !n_contrib || !dL_dimage || !image || !chunks)
        return fail(GS_ERR_INVALID, "gs_composite_bwd_ex: a required pointer is NULL");
    if (capacity > 0 && !ckpt) return fail(GS_ERR_INVALID, "gs_composite_bwd_ex: ckpt is NULL");
    if (n > 0 && (!grad_mean2d || !grad_conic_op || !grad_rgb))
        return fail(GS_ERR_INVALID, "gs_composite_bwd_ex: a gradient pointer is NULL");
    if (((uintptr_t)xy_depth | (uintptr_t)conic_op | (uintptr_t)rgb | (uintptr_t)grad_conic_op |
         (uintptr_t)grad_rgb | (uintptr_t)ckpt | (uintptr_t)chunks) & 15 || ((uintptr_t)grad_mean2d & 7))
        return fail(GS_ERR_INVALID, "gs_composite_bwd_ex: misaligned vector buffer");
    const float3 b = make_float3(bg[0], bg[1], bg[2]);
    return hip_check(gs::launch_composite_bwd(*cam, n_views, n, ranges, point_list, (const float4*)xy_depth,
                                              (const float4*)conic_op, (const float4*)rgb, b, final_T,
                                              n_contrib, dL_dimage, (float2*)grad_mean2d,
                                              (float4*)grad_conic_op, (float4*)grad_rgb, nullptr, chunks,
                                              (uint32_t)capacity, (const float4*)ckpt, image, (hipStream_t)stream),
                     "composite bwd launch");
}

size_t gs_recurrence_scratch_bytes(const gs_recurrence* r) {
    g_last_error.clear();
    if (check_recurrence(r, "gs_recurrence_scratch_bytes")) return 0;
    return gs::recurrence_scratch_bytes(*r);
}

gs_status gs_recurrence_fwd(const gs_recurrence* r, const void* gate, const void* x, const float* h0, void* h,
                            float* h_last, float* ckpt, void* scratch, size_t scratch_bytes, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_recurrence(r, "gs_recurrence_fwd")) return s;
    if (r->batch == 0 || r->channels == 0) return GS_OK;
    if (r->steps > 0 && (!gate || !x || !h)) return fail(GS_ERR_INVALID, "gs_recurrence_fwd: a required pointer is NULL");
    if (!aligned(type_bytes(r->dtype), gate, x, h) || !aligned(4, h0, h_last, ckpt))
        return fail(GS_ERR_INVALID, "gs_recurrence_fwd: a buffer is not aligned to its type");
    const size_t need = gs::recurrence_scratch_bytes(*r);
    if (need && (!scratch || scratch_bytes < need))
        return fail(GS_ERR_INVALID, "gs_recurrence_fwd: scratch of %zu bytes is smaller than the required %zu",
                    scratch ? scratch_bytes : (size_t)0, need);
    if (need && !aligned(8, scratch)) return fail(GS_ERR_INVALID, "gs_recurrence_fwd: scratch is not 8-byte aligned");
    if (need && (h == gate || h == x))
        return fail(GS_ERR_INVALID, "gs_recurrence_fwd: h overlaps gate or x");
    gs::RecurrenceArgs a = recurrence_args(*r);
    a.gate = gate;
    a.x = x;
    a.h0 = h0;
    a.h = h;
    a.h_last = h_last;
    a.ckpt = ckpt;
    return hip_check(gs::launch_recurrence_fwd(a, r->dtype, r->gating == GS_GATE_SIGMOID, scratch, (hipStream_t)stream),
                     "gs_recurrence_fwd launch");
}

gs_status gs_recurrence_bwd(const gs_recurrence* r, const void* gate, const void* x, const float* h0,
                            const float* ckpt, const void* grad_h, const float* grad_last, void* grad_gate,
                            void* grad_x, float* grad_h0, void* scratch, size_t scratch_bytes, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_recurrence(r, "gs_recurrence_bwd")) return s;
    if (r->batch == 0 || r->channels == 0) return GS_OK;
    if (r->steps > 0 && (!gate || !x || !grad_h || !grad_gate || !grad_x))
        return fail(GS_ERR_INVALID, "gs_recurrence_bwd: a required pointer is NULL");
    if (r->steps > GS_RECURRENCE_CHUNK && !ckpt)
        return fail(GS_ERR_INVALID, "gs_recurrence_bwd: ckpt is NULL with more than %d steps", GS_RECURRENCE_CHUNK);
    if (!aligned(type_bytes(r->dtype), gate, x, grad_h, grad_gate, grad_x) ||
        !aligned(4, h0, ckpt, grad_last, grad_h0))
        return fail(GS_ERR_INVALID, "gs_recurrence_bwd: a buffer is not aligned to its type");
    const size_t need = gs::recurrence_scratch_bytes(*r);
    if (need && (!scratch || scratch_bytes < need))
        return fail(GS_ERR_INVALID, "gs_recurrence_bwd: scratch of %zu bytes is smaller than the required %zu",
                    scratch ? scratch_bytes : (size_t)0, need);
    if (need && !aligned(8, scratch)) return fail(GS_ERR_INVALID, "gs_recurrence_bwd: scratch is not 8-byte aligned");
    if (need) {
        for (const void* in : {gate, x, grad_h})
            if (grad_gate == in || grad_x == in)
                return fail(GS_ERR_INVALID, "gs_recurrence_bwd: a gradient overlaps an input");
    }
    gs::RecurrenceArgs a = recurrence_args(*r);
    a.gate = gate;
    a.x = x;
    a.h0 = h0;
    a.ckpt_in = ckpt;
    a.grad_h = grad_h;
    a.grad_last = grad_last;
    a.grad_gate = grad_gate;
    a.grad_x = grad_x;
    a.grad_h0 = grad_h0;
    return hip_check(gs::launch_recurrence_bwd(a, r->dtype, r->gating == GS_GATE_SIGMOID, scratch, (hipStream_t)stream),
                     "gs_recurrence_bwd launch");
}

// For tests of the way without waiting, which no timing reaches at will; not
// in gs.h. It changes no result.
int gs_test_recurrence_patience(int polls) { return gs::set_recurrence_patience(polls); }

size_t gs_grad_scratch_bytes(void) { return gs::optim_scratch_bytes(); }

gs_status gs_grad_norm(const gs_grad_tensor* tensors, int32_t n_tensors, int32_t kind, float* norm, void* scratch,
                       void* stream) {
    g_last_error.clear();
    if (gs_status s = check_grads(tensors, n_tensors, kind, norm, scratch, false, "gs_grad_norm")) return s;
    return hip_check(gs::launch_grad_norm(tensors, n_tensors, kind, norm, scratch, (hipStream_t)stream),
                     "gs_grad_norm launch");
}

gs_status gs_clip_grads(const gs_grad_tensor* tensors, int32_t n_tensors, int32_t kind, float max_norm, float* norm,
                        void* scratch, void* stream) {
    g_last_error.clear();
    if (gs_status s = check_grads(tensors, n_tensors, kind, norm, scratch, true, "gs_clip_grads")) return s;
    if (!(max_norm > 0.0f) || !std::isfinite(max_norm))
        return fail(GS_ERR_INVALID, "gs_clip_grads: max_norm %g is not positive and finite", max_norm);
    return hip_check(gs::launch_clip_grads(tensors, n_tensors, kind, max_norm, norm, scratch, (hipStream_t)stream),
                     "gs_clip_grads launch");
}

gs_status gs_adam_step(const gs_adam* cfg, const gs_adam_tensor* tensors, int32_t n_tensors, int64_t* step,
                       float* norm, void* scratch, void* stream) {
    g_last_error.clear();
    if (!cfg) return fail(GS_ERR_INVALID, "gs_adam_step: cfg is NULL");
    if (!(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0 && cfg->beta2 >= 0.0 && cfg->beta2 < 1.0))
        return fail(GS_ERR_INVALID, "gs_adam_step: beta1 %g or beta2 %g outside [0, 1)", cfg->beta1, cfg->beta2);
    if (!((float)cfg->eps > 0.0f) || !std::isfinite((float)cfg->eps))
        return fail(GS_ERR_INVALID, "gs_adam_step: eps %g is not positive and finite in float32", cfg->eps);
    if (!(cfg->max_norm >= 0.0f) || !std::isfinite(cfg->max_norm))
        return fail(GS_ERR_INVALID, "gs_adam_step: max_norm %g is negative or not finite", cfg->max_norm);
    if (cfg->flags & ~(uint32_t)GS_ADAM_SKIP_NONFINITE)
        return fail(GS_ERR_INVALID, "gs_adam_step: unknown flags 0x%x", cfg->flags);
    if (gs_status s = check_list(tensors, n_tensors, scratch, "gs_adam_step")) return s;
    if (!step || !aligned(8, step)) return fail(GS_ERR_INVALID, "gs_adam_step: step is NULL or misaligned");
    if (!aligned(4, norm)) return fail(GS_ERR_INVALID, "gs_adam_step: norm is misaligned");
    for (int i = 0; i < n_tensors; ++i) {
        const gs_adam_tensor& t = tensors[i];
        if (gs_status s = check_count(t.count, i, "gs_adam_step")) return s;
        if (!std::isfinite(t.lr) || !std::isfinite(t.weight_decay))
            return fail(GS_ERR_INVALID, "gs_adam_step: tensor %d has a rate or decay that is not finite", i);
        if (!t.count) continue;
        const size_t pb = type_bytes(t.param_dtype), gb = type_bytes(t.grad_dtype);
        if (!pb || !gb) return fail(GS_ERR_INVALID, "gs_adam_step: tensor %d has an unknown dtype", i);
        if (!t.param || !t.grad || !t.m || !t.v)
            return fail(GS_ERR_INVALID, "gs_adam_step: tensor %d has a NULL pointer", i);
        if (!aligned(pb, t.param) || !aligned(gb, t.grad) || !aligned(4, t.m, t.v))
            return fail(GS_ERR_INVALID, "gs_adam_step: tensor %d is not aligned to its type", i);
    }
    return hip_check(gs::launch_adam_step(*cfg, tensors, n_tensors, step, norm, scratch, (hipStream_t)stream),
                     "gs_adam_step launch");
}

size_t gs_delta_rule_scratch_bytes(const gs_delta_rule* r, int32_t backward) {
    g_last_error.clear();
    if (check_delta_rule(r, backward != 0, "gs_delta_rule_scratch_bytes")) return 0;
    return gs::delta_rule_scratch_bytes(*r, backward != 0);
}

gs_status gs_delta_rule_fwd(const gs_delta_rule* r, const void* q, const void* k, const void* v,
                            const float* log_decay, const float* beta, const float* h0, void* o, float* h_last,
                            float* ckpt, void* scratch, size_t scratch_bytes, void* stream) {
    const char* const who = "gs_delta_rule_fwd";
    g_last_error.clear();
    if (gs_status s = check_delta_rule(r, false, who)) return s;
    if (r->batch == 0) return GS_OK;
    if (r->steps > 0 && (!q || !k || !v || !log_decay || !beta || !o))
        return fail(GS_ERR_INVALID, "%s: a required pointer is NULL", who);
    if (!aligned(type_bytes(r->dtype), q, k, v, o) || !aligned(4, log_decay, beta, h0, h_last, ckpt))
        return fail(GS_ERR_INVALID, "%s: a buffer is not aligned to its type", who);
    if (gs_status s = check_scratch(scratch, scratch_bytes, gs::delta_rule_scratch_bytes(*r, false), 16, who)) return s;
    if (r->steps > 0) {
        for (const void* in : {q, k, v, (const void*)log_decay, (const void*)beta, (const void*)h0})
            for (const void* out : {(const void*)o, (const void*)ckpt, (const void*)(h_last == h0 ? nullptr : h_last)})
                if (in && in == out) return fail(GS_ERR_INVALID, "%s: o, ckpt or h_last overlaps an input", who);
        if (o == (void*)h_last || o == (void*)ckpt || (ckpt && ckpt == h_last))
            return fail(GS_ERR_INVALID, "%s: two outputs are one buffer", who);
    }
    gs::DeltaArgs a{};
    a.r = *r;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_decay = log_decay;
    a.beta = beta;
    a.h0 = h0;
    a.o = o;
    a.h_last = h_last;
    a.ckpt = ckpt;
    return hip_check(gs::launch_delta_rule_fwd(a, scratch, (hipStream_t)stream), "gs_delta_rule_fwd launch");
}

gs_status gs_delta_rule_bwd(const gs_delta_rule* r, const void* q, const void* k, const void* v,
                            const float* log_decay, const float* beta, const float* h0, const float* ckpt,
                            const void* grad_o, const float* grad_last, void* grad_q, void* grad_k, void* grad_v,
                            float* grad_log_decay, float* grad_beta, float* grad_h0, void* scratch,
                            size_t scratch_bytes, void* stream) {
    const char* const who = "gs_delta_rule_bwd";
    g_last_error.clear();
    if (gs_status s = check_delta_rule(r, true, who)) return s;
    if (r->batch == 0) return GS_OK;
    if (r->steps > 0 && (!q || !k || !v || !log_decay || !beta || !grad_o || !grad_q || !grad_k || !grad_v ||
                         !grad_log_decay || !grad_beta))
        return fail(GS_ERR_INVALID, "%s: a required pointer is NULL", who);
    if (r->steps > GS_DELTA_CHUNK && !ckpt)
        return fail(GS_ERR_INVALID, "%s: ckpt is NULL with more than %d steps", who, GS_DELTA_CHUNK);
    if (!aligned(type_bytes(r->dtype), q, k, v, grad_o, grad_q, grad_k, grad_v) ||
        !aligned(4, log_decay, beta, h0, ckpt, grad_last, grad_log_decay, grad_beta, grad_h0))
        return fail(GS_ERR_INVALID, "%s: a buffer is not aligned to its type", who);
    if (gs_status s = check_scratch(scratch, scratch_bytes, gs::delta_rule_scratch_bytes(*r, true), 16, who)) return s;
    for (const void* in : {q, k, v, grad_o, (const void*)log_decay, (const void*)beta, (const void*)h0})
        for (const void* out : {(const void*)grad_q, (const void*)grad_k, (const void*)grad_v,
                                (const void*)grad_log_decay, (const void*)grad_beta, (const void*)grad_h0})
            if (in && in == out) return fail(GS_ERR_INVALID, "%s: a gradient overlaps an input", who);
    const void* const outs[] = {grad_q, grad_k, grad_v, grad_log_decay, grad_beta, grad_h0};
    for (int i = 0; r->steps > 0 && i < 6; ++i)
        for (int j = 0; j < i; ++j)
            if (outs[i] && outs[i] == outs[j]) return fail(GS_ERR_INVALID, "%s: two gradients are one buffer", who);
    gs::DeltaArgs a{};
    a.r = *r;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_decay = log_decay;
    a.beta = beta;
    a.h0 = h0;
    a.ckpt_in = ckpt;
    if (r->steps == 1) a.r.q_step = a.r.k_step = a.r.v_step = 0;
    a.grad_o = grad_o;
    a.grad_last = grad_last;
    a.grad_q = grad_q;
    a.grad_k = grad_k;
    a.grad_v = grad_v;
    a.grad_log_decay = grad_log_decay;
    a.grad_beta = grad_beta;
    a.grad_h0 = grad_h0;
    return hip_check(gs::launch_delta_rule_bwd(a, scratch, (hipStream_t)stream), "gs_delta_rule_bwd launch");
}

gs_status gs_block_norm_fwd(const gs_block_norm* d, const void* y, const void* gate, const void* residual,
                            const void* post_weight, const void* post_bias, const void* scale, const void* pre_weight,
                            const void* pre_bias, void* out, void* norm, void* stream) {
    const char* const who = "gs_block_norm_fwd";
    g_last_error.clear();
    if (gs_status s = check_block_norm(d, who)) return s;
    if (d->outer == 0) return GS_OK;
    const bool pre = d->pre != GS_BLOCK_NORM_NONE;
    if (pre ? !norm : !out) return fail(GS_ERR_INVALID, "%s: a required pointer is NULL", who);
    gs::BlockNormArgs a{*d, y, gate, residual, post_weight, post_bias, scale, pre_weight, pre_bias};
    a.out = out;
    a.norm = pre ? norm : nullptr;
    if (gs_status s = check_block_inputs(*d, a, who)) return s;
    if (pre) {
        for (const void* p : {y, gate, residual, (const void*)out})
            if (p == norm) return fail(GS_ERR_INVALID, "%s: norm overlaps out or an input", who);
    }
    const int64_t w = d->width, o = w * d->inner;
    auto contiguous = [&](int64_t so, int64_t si) {
        return (d->outer == 1 || so == o) && (d->inner == 1 || si == w);
    };
    if ((out == y && !contiguous(d->y_outer, d->y_inner)) ||
        (out && out == gate && !contiguous(d->gate_outer, d->gate_inner)) ||
        (out && out == residual && !contiguous(d->residual_outer, d->residual_inner)))
        return fail(GS_ERR_INVALID, "%s: out replaces an input that is not contiguous", who);
    return hip_check(gs::launch_block_norm_fwd(a, (hipStream_t)stream), "gs_block_norm_fwd launch");
}

size_t gs_block_norm_scratch_bytes(const gs_block_norm* d) {
    g_last_error.clear();
    if (check_block_norm(d, "gs_block_norm_scratch_bytes")) return 0;
    return gs::block_norm_scratch_bytes(*d);
}

gs_status gs_block_norm_bwd(const gs_block_norm* d, const void* y, const void* gate, const void* residual,
                            const void* post_weight, const void* post_bias, const void* scale, const void* pre_weight,
                            const void* pre_bias, const void* grad_out, const void* grad_norm, void* grad_y,
                            void* grad_gate, void* grad_residual, float* grad_post_weight, float* grad_post_bias,
                            float* grad_scale, float* grad_pre_weight, float* grad_pre_bias, void* scratch,
                            size_t scratch_bytes, void* stream) {
    const char* const who = "gs_block_norm_bwd";
    g_last_error.clear();
    if (gs_status s = check_block_norm(d, who)) return s;
    gs::BlockNormArgs a{*d, y, gate, residual, post_weight, post_bias, scale, pre_weight, pre_bias};
    const bool pre = d->pre != GS_BLOCK_NORM_NONE;
    a.grad_out = grad_out;
    a.grad_norm = pre ? grad_norm : nullptr;
    a.grad_y = grad_y;
    a.grad_gate = d->gating != GS_BLOCK_GATE_NONE ? grad_gate : nullptr;
    a.grad_residual = grad_residual;
    const bool post = d->post != GS_BLOCK_NORM_NONE;
    if ((!post && (grad_post_weight || grad_post_bias)) || (!pre && (grad_pre_weight || grad_pre_bias)))
        return fail(GS_ERR_INVALID, "%s: the gradient of a weight is asked for without its norm", who);
    float* const sums[5] = {grad_post_weight, grad_post_bias, grad_scale, grad_pre_weight, grad_pre_bias};
    bool any = false;
    for (int i = 0; i < 5; ++i) any |= (a.sums[i] = sums[i]) != nullptr;
    if (d->outer == 0 && !any) return GS_OK;
    if (d->outer > 0) {
        if (!grad_y || (pre ? !grad_norm : !grad_out)) return fail(GS_ERR_INVALID, "%s: a required pointer is NULL", who);
        if (gs_status s = check_block_inputs(*d, a, who)) return s;
        for (const void* in : {y, gate, residual})
            for (const void* out : {(const void*)grad_y, (const void*)a.grad_gate, (const void*)grad_residual})
                if (in && in == out) return fail(GS_ERR_INVALID, "%s: a gradient overlaps an input", who);
        if (grad_y == a.grad_gate || grad_y == grad_residual || (grad_residual && grad_residual == a.grad_gate))
            return fail(GS_ERR_INVALID, "%s: two gradients are one buffer", who);
        if (any)
            if (gs_status s = check_scratch(scratch, scratch_bytes, gs::block_norm_scratch_bytes(*d), 4, who)) return s;
    } else if (!aligned(4, sums[0], sums[1], sums[2], sums[3], sums[4])) {
        return fail(GS_ERR_INVALID, "%s: a buffer is not aligned to its type", who);
    }
    return hip_check(gs::launch_block_norm_bwd(a, (float*)scratch, (hipStream_t)stream), "gs_block_norm_bwd launch");
}

}  // extern "C"
