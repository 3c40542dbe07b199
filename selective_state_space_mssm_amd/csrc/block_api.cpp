// block_api.cpp -- the C ABI declared in include/mssm_block.h.
//
// Host-only layer, as mssm_api.cpp: every argument is checked before anything
// is enqueued, and a validated argument block goes to the kernel launchers.
#include "block.h"

#include <cstdint>
#include <initializer_list>

namespace {

bool f32_or_bf16(int32_t t) { return t == MSSM_F32 || t == MSSM_BF16; }

mssm_status check_align(std::initializer_list<const void*> ptrs) {
    for (const void* q : ptrs)
        if (reinterpret_cast<uintptr_t>(q) & 15u) return MSSM_ERR_ALIGN;
    return MSSM_OK;
}

mssm_status from_hip(hipError_t e) { return e == hipSuccess ? MSSM_OK : MSSM_ERR_HIP; }

// Compute units of the current device; 256 if the query fails (only the schedule depends on it).
int64_t device_cus() {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1) {
        (void)hipGetLastError();
        return 256;
    }
    return n;
}

mssm_status check_norm(const mssm_norm_problem* p) {
    if (!p) return MSSM_ERR_NULL;
    if (!f32_or_bf16(p->dtype) || !f32_or_bf16(p->residual_dtype)) return MSSM_ERR_DTYPE;
    if (p->rows < 1 || p->rows >= (int64_t{1} << 31) || p->dim < 1 || p->dim >= (int64_t{1} << 24)) return MSSM_ERR_SHAPE;
    if (!(p->eps >= 0.0f)) return MSSM_ERR_SHAPE;
    return MSSM_OK;
}

mssm_status check_linear(const mssm_linear_problem* p) {
    if (!p) return MSSM_ERR_NULL;
    if (p->dtype != MSSM_F32 && p->dtype != MSSM_BF16 && p->dtype != MSSM_F8) return MSSM_ERR_DTYPE;
    if (!f32_or_bf16(p->out_dtype)) return MSSM_ERR_DTYPE;
    if (p->dtype == MSSM_F32 && p->out_dtype != MSSM_F32) return MSSM_ERR_DTYPE;
    if (p->rows < 1 || p->in_dim < 1 || p->out_dim < 1) return MSSM_ERR_SHAPE;
    // a 256-row tile's byte offsets stay below 2^31
    if (p->rows >= (int64_t{1} << 31) || p->out_dim >= (int64_t{1} << 31) || p->in_dim >= (int64_t{1} << 20))
        return MSSM_ERR_SHAPE;
    if (p->activation < MSSM_ACT_NONE || p->activation > MSSM_ACT_GELU) return MSSM_ERR_UNSUPPORTED;
    return MSSM_OK;
}

mssm_status check_beam(const mssm_beam_problem* p) {
    if (!p) return MSSM_ERR_NULL;
    if (!f32_or_bf16(p->dtype)) return MSSM_ERR_DTYPE;
    if (p->batch < 1 || p->beams < 1 || p->vocab < 1) return MSSM_ERR_SHAPE;
    if (p->beams > MSSM_MAX_BEAMS) return MSSM_ERR_UNSUPPORTED;
    if (p->vocab >= (int64_t{1} << 27)) return MSSM_ERR_SHAPE;  // k * vocab + v stays below 2^31
    if (p->batch >= (int64_t{1} << 31) / p->beams) return MSSM_ERR_SHAPE;
    if (p->end_token < -1 || p->end_token >= p->vocab) return MSSM_ERR_SHAPE;
    return MSSM_OK;
}

mssm_status norm_common(const mssm_norm_problem* p, const void* x, const void* residual, const float* weight, void* y,
                        float* scale, bool q8, void* residual_out, void* hip_stream) {
    mssm_status st = check_norm(p);
    if (st != MSSM_OK) return st;
    if (!x || !weight || !y || (q8 && !scale)) return MSSM_ERR_NULL;
    st = check_align({x, residual, weight, y, scale, residual_out});
    if (st != MSSM_OK) return st;
    const mssm::NormArgs a{p->rows, p->dim, p->dtype, p->residual_dtype, p->eps, x, residual, weight, y, scale,
                           residual_out};
    return from_hip(mssm::launch_norm(a, static_cast<hipStream_t>(hip_stream)));
}

}  // namespace

extern "C" {

mssm_status mssm_add_rmsnorm(const mssm_norm_problem* p, const void* x, const void* residual, const float* weight,
                             void* y, void* residual_out, void* hip_stream) {
    return norm_common(p, x, residual, weight, y, nullptr, false, residual_out, hip_stream);
}

mssm_status mssm_add_rmsnorm_q8(const mssm_norm_problem* p, const void* x, const void* residual,
                                const float* weight, void* q, float* scale, void* residual_out, void* hip_stream) {
    return norm_common(p, x, residual, weight, q, scale, true, residual_out, hip_stream);
}

size_t mssm_linear_workspace_bytes(const mssm_linear_problem* p) {
    if (check_linear(p) != MSSM_OK) return 0;
    return mssm::plan_linear(p->rows, p->in_dim, p->out_dim, p->dtype, p->out_dtype, device_cus()).ws_bytes;
}

mssm_status mssm_linear(const mssm_linear_problem* p, const void* x, const float* x_scale, const void* w,
                        const float* w_scale, const float* bias, const void* residual, void* y,
                        void* workspace, size_t workspace_bytes, void* hip_stream) {
    mssm_status st = check_linear(p);
    if (st != MSSM_OK) return st;
    if (!x || !w || !y) return MSSM_ERR_NULL;
    if (p->dtype == MSSM_F8 ? (!x_scale || !w_scale) : (x_scale || w_scale)) return MSSM_ERR_NULL;
    st = check_align({x, x_scale, w, w_scale, bias, residual, y, workspace});
    if (st != MSSM_OK) return st;
    const mssm::LinearPlan plan = mssm::plan_linear(p->rows, p->in_dim, p->out_dim, p->dtype, p->out_dtype, device_cus());
    if (plan.ws_bytes > 0 && (!workspace || workspace_bytes < plan.ws_bytes)) return MSSM_ERR_WORKSPACE;
    const mssm::LinearArgs a{p->rows, p->in_dim, p->out_dim, p->dtype, p->out_dtype, p->activation, x, x_scale, w,
                             w_scale, bias, residual, y, plan.splits > 1 ? static_cast<float*>(workspace) : nullptr};
    return from_hip(mssm::launch_linear(a, plan, static_cast<hipStream_t>(hip_stream)));
}

size_t mssm_beam_select_workspace_bytes(const mssm_beam_problem* p) {
    if (check_beam(p) != MSSM_OK) return 0;
    return mssm::beam_ws_bytes(p->batch, p->beams, p->vocab);
}

mssm_status mssm_beam_select(const mssm_beam_problem* p, const void* logits, const float* scores,
                             const uint8_t* finished, float* scores_out, int32_t* parent, int32_t* token,
                             uint8_t* finished_out, void* workspace, size_t workspace_bytes, void* hip_stream) {
    mssm_status st = check_beam(p);
    if (st != MSSM_OK) return st;
    if (!logits || !scores || !scores_out || !parent || !token) return MSSM_ERR_NULL;
    if (finished && p->end_token < 0) return MSSM_ERR_SHAPE;  // a finished beam continues with end_token
    st = check_align({logits, scores, finished, scores_out, parent, token, finished_out, workspace});
    if (st != MSSM_OK) return st;
    if (!workspace || workspace_bytes < mssm::beam_ws_bytes(p->batch, p->beams, p->vocab)) return MSSM_ERR_WORKSPACE;
    const mssm::BeamArgs a{p->batch, p->beams, p->vocab, p->dtype, p->end_token, logits, scores, finished,
                           scores_out, parent, token, finished_out, workspace};
    return from_hip(mssm::launch_beam_select(a, static_cast<hipStream_t>(hip_stream)));
}

mssm_status mssm_beam_reorder(int64_t batch, int64_t beams, const int32_t* parent, int32_t count,
                              const mssm_beam_state* states, void* hip_stream) {
    if (batch < 1 || beams < 1 || count < 1) return MSSM_ERR_SHAPE;
    if (beams > MSSM_MAX_BEAMS || count > MSSM_MAX_BEAM_STATES) return MSSM_ERR_UNSUPPORTED;
    if (batch >= (int64_t{1} << 31) / beams) return MSSM_ERR_SHAPE;
    if (!parent || !states) return MSSM_ERR_NULL;
    mssm_status st = check_align({parent});
    if (st != MSSM_OK) return st;
    for (int32_t i = 0; i < count; ++i) {
        if (!states[i].data) return MSSM_ERR_NULL;
        if (states[i].layers < 1 || states[i].bytes < 1 || states[i].bytes >= (int64_t{1} << 31)) return MSSM_ERR_SHAPE;
        if (states[i].layers >= (int64_t{1} << 31) / batch) return MSSM_ERR_SHAPE;
        st = check_align({states[i].data});
        if (st != MSSM_OK) return st;
    }
    return from_hip(mssm::launch_beam_reorder(batch, beams, parent, count, states, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
