// block.h -- host-side interface between the C ABI of the operators around the
// scan (block_api.cpp) and their kernel launchers (norm.hip, linear.hip,
// beam.hip).  Internal.  Element types are numbered as in the headers:
// 0 = float32, 1 = bfloat16, 2 = e4m3.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "linear_plan.h"
#include "mssm_block.h"

namespace mssm {

struct NormArgs {
    int64_t rows, dim;
    int dtype, residual_dtype;
    float eps;
    const void* x;
    const void* residual;  // nullable
    const float* weight;
    void* y;               // p->dtype, or e4m3 bytes when scale is set
    float* scale;          // nullable
    void* residual_out;    // nullable
};
hipError_t launch_norm(const NormArgs& a, hipStream_t s);

struct LinearArgs {
    int64_t M, K, N;
    int dtype, out_dtype, act;
    const void* x;
    const float* x_scale;
    const void* w;
    const float* w_scale;
    const float* bias;     // nullable
    const void* residual;  // nullable
    void* y;
    float* partial;        // split sums (splits, M, N), null: none
};
hipError_t launch_linear(const LinearArgs& a, const LinearPlan& plan, hipStream_t s);

struct BeamArgs {
    int64_t B, K, V;
    int dtype;
    int32_t end_token;
    const void* logits;
    const float* scores;
    const uint8_t* finished;  // nullable
    float* scores_out;
    int32_t* parent;
    int32_t* token;
    uint8_t* finished_out;    // nullable
    void* workspace;
};
size_t beam_ws_bytes(int64_t B, int64_t K, int64_t V);
hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s);
hipError_t launch_beam_reorder(int64_t B, int64_t K, const int32_t* parent, int count, const mssm_beam_state* st,
                               hipStream_t s);

}  // namespace mssm
