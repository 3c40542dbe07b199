// linear.hip -- projections with their epilogue (mssm_linear):
// y = act(x wᵀ * scales + bias) + residual on the matrix cores.
#include "block.h"
#include "device_common.h"

namespace mssm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Element types, by the header's numbers.
template <int DT> struct Elem;
template <> struct Elem<MSSM_F32> { static constexpr int kBytes = 4; };
template <> struct Elem<MSSM_BF16> { static constexpr int kBytes = 2; };
template <> struct Elem<MSSM_F8> { static constexpr int kBytes = 1; };

// One 16x16 block of products over the 64 bytes of k that the four 16-lane
// groups hold, 16 bytes a lane (row lane % 16 of either operand).  Both
// operands hold the same k at the same place, so the order of k inside the 64
// bytes is free.  acc[i] belongs to row 4 (lane / 16) + i of a and row
// lane % 16 of b.
template <int DT>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 acc) {
    if constexpr (DT == MSSM_BF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc,
                                                       0, 0, 0);
    } else if constexpr (DT == MSSM_F8) {
        typedef int64_t i64x2 __attribute__((ext_vector_type(2)));
        const i64x2 p = __builtin_bit_cast(i64x2, a), q = __builtin_bit_cast(i64x2, b);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(p[0], q[0], acc, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(p[1], q[1], acc, 0, 0, 0);
    } else {
        const f32x4 p = __builtin_bit_cast(f32x4, a), q = __builtin_bit_cast(f32x4, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(p[j], q[j], acc, 0, 0, 0);
        return acc;
    }
}

struct LinearKernelArgs {
    const uint8_t* x;
    const uint8_t* w;
    const float* xs;
    const float* ws;
    const float* bias;
    const void* res;
    void* y;
    int64_t M, K, N;
    int act;
};

__device__ __forceinline__ float activate(float v, int act) {
    if (act == MSSM_ACT_RELU) return v > 0.0f ? v : 0.0f;
    if (act == MSSM_ACT_SILU) return v / (1.0f + expf(-v));
    if (act == MSSM_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    return v;
}

// 64 x 64 outputs a workgroup of 4 waves, k in steps of 64 bytes through LDS,
// loaded byte group by byte group with bounds checks (zeros outside).
template <int DT, typename O>
__global__ __launch_bounds__(256) void linear_kernel(LinearKernelArgs a) {
    constexpr int E = Elem<DT>::kBytes, KB = 64, PITCH = KB + 16;
    __shared__ __align__(16) uint8_t sx[64 * PITCH], sw[64 * PITCH];
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 64, n0 = static_cast<int64_t>(blockIdx.x) * 64;
    const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, g = lane >> 4;
    const int64_t kbytes = a.K * E;
    f32x4 acc[4] = {};
    for (int64_t k0 = 0; k0 < kbytes; k0 += KB) {
        for (int i = threadIdx.x; i < 64 * KB / E; i += 256) {
            const int row = i / (KB / E), kb = i % (KB / E) * E;
            const bool in_k = k0 + kb < kbytes;
            const bool in_x = in_k && m0 + row < a.M, in_w = in_k && n0 + row < a.N;
            const int64_t ox = (m0 + row) * kbytes + k0 + kb, ow = (n0 + row) * kbytes + k0 + kb;
            if constexpr (E == 4) {
                *reinterpret_cast<uint32_t*>(sx + row * PITCH + kb) = in_x ? *reinterpret_cast<const uint32_t*>(a.x + ox) : 0;
                *reinterpret_cast<uint32_t*>(sw + row * PITCH + kb) = in_w ? *reinterpret_cast<const uint32_t*>(a.w + ow) : 0;
            } else if constexpr (E == 2) {
                *reinterpret_cast<uint16_t*>(sx + row * PITCH + kb) = in_x ? *reinterpret_cast<const uint16_t*>(a.x + ox) : 0;
                *reinterpret_cast<uint16_t*>(sw + row * PITCH + kb) = in_w ? *reinterpret_cast<const uint16_t*>(a.w + ow) : 0;
            } else {
                sx[row * PITCH + kb] = in_x ? a.x[ox] : 0;
                sw[row * PITCH + kb] = in_w ? a.w[ow] : 0;
            }
        }
        __syncthreads();
        const u32x4 wf = *reinterpret_cast<const u32x4*>(sw + (wave * 16 + r) * PITCH + g * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = mma<DT>(wf, *reinterpret_cast<const u32x4*>(sx + (j * 16 + r) * PITCH + g * 16), acc[j]);
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + j * 16 + r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = n0 + wave * 16 + g * 4 + i;
            if (m < a.M && n < a.N) {
                float v = acc[j][i];
                if constexpr (DT == MSSM_F8) v *= a.xs[m] * a.ws[n];
                if (a.bias) v += a.bias[n];
                v = activate(v, a.act);
                if (a.res) v += load_act(static_cast<const O*>(a.res), m * a.N + n);
                store_act(static_cast<O*>(a.y), m * a.N + n, v);
            }
        }
    }
}

template <int DT, typename O>
void launch_t(const LinearArgs& a, hipStream_t s) {
    const LinearKernelArgs k{static_cast<const uint8_t*>(a.x), static_cast<const uint8_t*>(a.w), a.x_scale, a.w_scale,
                             a.bias, a.residual, a.y, a.M, a.K, a.N, a.act};
    const dim3 grid(static_cast<uint32_t>((a.N + 63) / 64), static_cast<uint32_t>((a.M + 63) / 64));
    linear_kernel<DT, O><<<grid, 256, 0, s>>>(k);
}

}  // namespace

LinearPlan plan_linear(int64_t, int64_t, int64_t, int, int64_t) { return {1, 0}; }

hipError_t launch_linear(const LinearArgs& a, const LinearPlan&, hipStream_t s) {
    if (a.dtype == MSSM_F32)
        launch_t<MSSM_F32, float>(a, s);
    else if (a.dtype == MSSM_BF16)
        a.out_dtype == MSSM_F32 ? launch_t<MSSM_BF16, float>(a, s) : launch_t<MSSM_BF16, uint16_t>(a, s);
    else
        a.out_dtype == MSSM_F32 ? launch_t<MSSM_F8, float>(a, s) : launch_t<MSSM_F8, uint16_t>(a, s);
    return hipGetLastError();
}

}  // namespace mssm
