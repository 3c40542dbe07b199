// planes.h -- float32 products on the bfloat16 matrix cores.
//
// Matrix instruction 16x16x32 bfloat16 (wave64; lane l, c = l % 16, group g = l / 16):
//   operands: lane holds 8 values of row (column) c, its slots (g, 0..7) of the
//   32 summed over; any order of these will do if both operands have it.
//   accumulator item r: row 4 g + r, column c.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.h"

namespace mssm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ---- products ---------------------------------------------------------------

// A float32 is the sum of three bfloat16 values, the 8 upper bits of what the
// ones before leave: exact (24 bits), by masks and subtractions.  A product of
// two such operands is the sum of its planes' products, of which those below
// 2^-24 of the largest are left out: 6 of 9, or 3 where one operand is bfloat16
// already.  That is 16 / 6 times the rate of the float32 matrix instructions,
// and no less exact: every one of these products is exact, sums are float32.
template <int N>
struct Planes {
    u32x4 p[N];
};

__device__ __forceinline__ uint32_t upper_halves(float a, float b) {  // a's in the lower half
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float upper_part(float a) { return __uint_as_float(__float_as_uint(a) & 0xffff0000u); }

template <int N>
__device__ __forceinline__ Planes<N> split(float (&x)[8]) {
    Planes<N> out;
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out.p[n][i] = upper_halves(x[2 * i], x[2 * i + 1]);
        if (n + 1 < N) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] -= upper_part(x[i]);
        }
    }
    return out;
}
template <int N>
__device__ __forceinline__ Planes<N> split(f32x4 lo, f32x4 hi) {  // the rows of two accumulators
    float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return split<N>(x);
}

__device__ __forceinline__ f32x4 mma1(u32x4 a, u32x4 b, f32x4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}
template <int PA, int PB>
__device__ __forceinline__ f32x4 mma(const Planes<PA>& a, const Planes<PB>& b, f32x4 acc) {
    constexpr int M = PA > PB ? PA : PB;
#pragma unroll
    for (int s = M - 1; s >= 0; --s)  // the small ones first
#pragma unroll
        for (int i = 0; i < PA; ++i)
            if (s - i >= 0 && s - i < PB) acc = mma1(a.p[i], b.p[s - i], acc);
    return acc;
}

// Planes of the inputs' type: bfloat16 is one.
template <typename T> constexpr int kPlanes = sizeof(T) == 2 ? 1 : 3;

}  // namespace mssm
