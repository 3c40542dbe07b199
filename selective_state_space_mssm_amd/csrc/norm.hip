// norm.hip -- residual addition + root-mean-square norm, output in the input's
// type or in 8 bits with a scale a row (mssm_add_rmsnorm, mssm_add_rmsnorm_q8).
#include "block.h"
#include "device_common.h"

namespace mssm {
namespace {

constexpr float kF8Max = 448.0f;        // largest e4m3 value
constexpr float kScaleFloor = 1e-30f;   // rows of smaller magnitude are scaled as if it were this

__device__ __forceinline__ float wave_sum(float v) {
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    for (int m = 32; m; m >>= 1) {
        const uint32_t o = __shfl_xor(v, m);
        v = o > v ? o : v;
    }
    return v;
}

__device__ __forceinline__ uint8_t to_f8(float v) {
    return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xff);
}

struct NormKernelArgs {
    const void* x;
    const void* res;
    const float* weight;
    void* y;
    float* scale;
    void* res_out;
    int64_t rows, dim;
    float eps;
};

// One wave a row.
template <typename T, typename R, bool Q8>
__global__ __launch_bounds__(256) void norm_kernel(NormKernelArgs a) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + wave_id();
    if (row >= a.rows) return;
    const int lane = threadIdx.x & 63;
    const int64_t e0 = row * a.dim;
    const T* x = static_cast<const T*>(a.x) + e0;
    const R* res = a.res ? static_cast<const R*>(a.res) + e0 : nullptr;
    auto h_at = [&](int64_t i) { return load_act(x, i) + (res ? load_act(res, i) : 0.0f); };
    float ss = 0.0f;
    for (int64_t i = lane; i < a.dim; i += 64) {
        const float h = h_at(i);
        ss = __builtin_fmaf(h, h, ss);
    }
    const float r = 1.0f / __builtin_sqrtf(wave_sum(ss) / static_cast<float>(a.dim) + a.eps);
    float inv = 0.0f;
    if constexpr (Q8) {
        // magnitudes compared as their bits: NaN above infinity above every number
        uint32_t m = 0;
        for (int64_t i = lane; i < a.dim; i += 64) {
            const uint32_t b = __float_as_uint(h_at(i) * r * a.weight[i]) & 0x7fffffffu;
            m = b > m ? b : m;
        }
        const float top = __uint_as_float(wave_max_u32(m));
        const float scale = (top < kScaleFloor ? kScaleFloor : top) / kF8Max;
        inv = 1.0f / scale;
        if (lane == 0) a.scale[row] = scale;
    }
    for (int64_t i = lane; i < a.dim; i += 64) {
        const float h = h_at(i);
        const float v = h * r * a.weight[i];
        if (a.res_out) store_act(static_cast<R*>(a.res_out) + e0, i, h);
        if constexpr (Q8)
            static_cast<uint8_t*>(a.y)[e0 + i] = to_f8(v * inv);
        else
            store_act(static_cast<T*>(a.y) + e0, i, v);
    }
}

template <typename T, typename R>
void launch_t(const NormArgs& a, hipStream_t s) {
    const NormKernelArgs k{a.x, a.residual, a.weight, a.y, a.scale, a.residual_out, a.rows, a.dim, a.eps};
    const dim3 grid(static_cast<uint32_t>((a.rows + 3) / 4));
    if (a.scale)
        norm_kernel<T, R, true><<<grid, 256, 0, s>>>(k);
    else
        norm_kernel<T, R, false><<<grid, 256, 0, s>>>(k);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    if (a.dtype == MSSM_F32)
        a.residual_dtype == MSSM_F32 ? launch_t<float, float>(a, s) : launch_t<float, uint16_t>(a, s);
    else
        a.residual_dtype == MSSM_F32 ? launch_t<uint16_t, float>(a, s) : launch_t<uint16_t, uint16_t>(a, s);
    return hipGetLastError();
}

}  // namespace mssm
