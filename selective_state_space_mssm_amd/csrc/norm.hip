// norm.hip -- residual addition + root-mean-square norm, output in the input's
// type or in 8 bits with a scale a row (mssm_add_rmsnorm, mssm_add_rmsnorm_q8).
//
// One pass over memory: a row's h = x + residual stays in registers between
// the sum of its squares and the products with the weight (and, in 8 bits,
// between these and the division by their maximum's scale).
#include "block.h"
#include "device_common.h"

#include <type_traits>

namespace mssm {
namespace {

constexpr float kF8Max = 448.0f;       // largest e4m3 value
constexpr float kScaleFloor = 1e-30f;  // rows of smaller magnitude are scaled as if it were this
constexpr int VEC = 8;                 // elements of a vector: 16 bytes of bfloat16, 32 of float32

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

// Sums (maxima) over the wave by within-row DPP moves and the four row totals.
__device__ __forceinline__ float wave_sum(float v) {
    v = group_sum<16>(v);
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i * 16));
    return (r[0] + r[1]) + (r[2] + r[3]);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    auto step = [&](float moved) {
        const uint32_t o = __float_as_uint(moved);
        v = o > v ? o : v;
    };
    step(dpp_move<0xB1>(__uint_as_float(v)));
    step(dpp_move<0x4E>(__uint_as_float(v)));
    step(dpp_move<0x141>(__uint_as_float(v)));
    step(dpp_move<0x140>(__uint_as_float(v)));
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t o = __builtin_amdgcn_readlane(static_cast<int>(v), i * 16);
        top = o > top ? o : top;
    }
    return top;
}

// Eight neighbouring elements of a row from column c on.  WHOLE rows are whole
// vectors long and start on vector boundaries; in others a vector counts from
// the row's start rounded down to a vector (c may be negative), the elements
// outside the row are 0, and a vector that is partly outside goes by elements.
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void load8(const float* p, float (&v)[VEC]) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[VEC]) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(a[i]), v[2 * i + 1] = bf16_hi(a[i]);
}
// Stores go past the caches: 16,384 x 2,560 bfloat16 rows with a bfloat16
// residual take 63 us so and 74 us without (float32 residual, 8-bit output, before
// its remainders were carried: 87 and 89 us).
__device__ __forceinline__ void store8(float* p, const float (&v)[VEC]) {
    __builtin_nontemporal_store((f32x4{v[0], v[1], v[2], v[3]}), reinterpret_cast<f32x4*>(p));
    __builtin_nontemporal_store((f32x4{v[4], v[5], v[6], v[7]}), reinterpret_cast<f32x4*>(p + 4));
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[VEC]) {
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    bf16x8 b;
#pragma unroll
    for (int i = 0; i < VEC; ++i) b[i] = static_cast<__bf16>(v[i]);
    __builtin_nontemporal_store(b, reinterpret_cast<bf16x8*>(p));
}
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[VEC]) {  // e4m3, two at a time
    u32x2 q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
        q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], w, true);
    }
    __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(p));
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { store_act(p, 0, v); }
__device__ __forceinline__ void store1(uint8_t* p, float v) {
    *p = static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false));
}

template <bool WHOLE, typename T>
__device__ __forceinline__ void load_part(const T* row, int64_t c, int64_t dim, float (&v)[VEC]) {
    if (WHOLE ? c < dim : (c >= 0 && c + VEC <= dim)) {
        load8(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = 0.0f;
        if (!WHOLE && c + VEC > 0 && c < dim) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (c + i >= 0 && c + i < dim) v[i] = load_act(row, c + i);
        }
    }
}
template <bool WHOLE, typename T>
__device__ __forceinline__ void store_part(T* row, int64_t c, int64_t dim, const float (&v)[VEC]) {
    if (WHOLE ? c < dim : (c >= 0 && c + VEC <= dim)) {
        store8(row + c, v);
    } else if (!WHOLE && c + VEC > 0 && c < dim) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i >= 0 && c + i < dim) store1(row + c + i, v[i]);
    }
}
// The weight, from the same columns: its own vectors lie elsewhere (4-byte aligned).
template <bool WHOLE>
__device__ __forceinline__ void load_weight(const float* w, int64_t c, int64_t dim, float (&v)[VEC]) {
    if constexpr (WHOLE) {
        load_part<true>(w, c, dim, v);
    } else if (c >= 0 && c + VEC <= dim) {
        struct __attribute__((packed, aligned(4))) Quad { f32x4 v; };
        const f32x4 a = reinterpret_cast<const Quad*>(w + c)->v, b = reinterpret_cast<const Quad*>(w + c + 4)->v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = c + i >= 0 && c + i < dim ? w[c + i] : 0.0f;
    }
}

// ---- the 8-bit division ----------------------------------------------------------
//
// q = e4m3(y / scale) with y = h r w and scale = max |y| / 448: r cancels, and
// what is rounded to 4 bits is h w (448 / max |h w|).  One rounding of its
// float32 factors moves about one value in a million across a rounding
// boundary, by a step of 6 %, so products and quotient are carried as a float32
// and its remainder (exact sum, fused products) and rounded once, to e4m3: 2 us
// of 89 at 16,384 x 2,560, where the vector instructions hide behind memory, and up to 2 us of 8 for a thousand rows.

// a + b = s + the returned remainder, exactly
__device__ __forceinline__ float sum_rest(float a, float b, float s) {
#pragma clang fp contract(off)
    const float t = s - a;
    return (a - (s - t)) + (b - t);
}
// (h + rest) w as a float32 and its remainder, in the places of h and rest
__device__ __forceinline__ void times_weight(float& h, float& rest, float w) {
#pragma clang fp contract(off)  // what is rounded where is the point here
    const float p = h * w;
    rest = __builtin_fmaf(rest, w, __builtin_fmaf(h, w, -p));
    h = p;
}
// The row's largest magnitude so far, as the bits of a float32 (NaN above
// infinity above every number) and its remainder.
struct Largest {
    uint32_t bits = 0;
    float rest = 0.0f;
    __device__ __forceinline__ void take(float p, float e) {
        const uint32_t b = __float_as_uint(p) & 0x7fffffffu;
        if (b > bits) bits = b, rest = p < 0.0f ? -e : e;
    }
    __device__ __forceinline__ void wave() {
        const uint32_t top = wave_max(bits);
        // of the lanes that hold it (mostly one) the largest remainder; remainders compare as ordered bits
        uint32_t o = __float_as_uint(rest);
        o ^= o >> 31 ? 0xffffffffu : 0x80000000u;
        o = wave_max(bits == top ? o : 0u);
        bits = top;
        rest = __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu));
    }
};
// The scale and the factor of the row's h w, in float32 and remainder.
struct RowScale {
    float scale, hi, lo;
    __device__ __forceinline__ RowScale(uint32_t bits, float rest, float r) {
#pragma clang fp contract(off)
        const float top = __uint_as_float(bits), y = top * r;
        if (bits == 0 || y < kScaleFloor) {
            scale = kScaleFloor / kF8Max;
            hi = bits ? r / scale : 0.0f;  // a row of zeros: r is infinite with eps = 0
            lo = 0.0f;
        } else {  // 448 / (top + rest), with what hi leaves of it
            scale = y / kF8Max;
            hi = kF8Max / top;
            lo = __builtin_fmaf(-hi, rest, __builtin_fmaf(-hi, top, kF8Max)) * (hi / kF8Max);
        }
    }
    // (p + e) times the factor, as a float32 that e4m3 rounds as it would the
    // exact value: where a remainder is left and the last bit is 0 (as it is on
    // every rounding boundary), one unit towards it.
    __device__ __forceinline__ float apply(float p, float e) const {
#pragma clang fp contract(off)
        const float a = p * hi;
        const float rest = __builtin_fmaf(p, hi, -a) + __builtin_fmaf(p, lo, e * hi);
        const float v = a + rest, left = rest - (v - a);
        const uint32_t b = __float_as_uint(v);
        const bool away = (__float_as_uint(left) ^ b) >> 31 == 0;
        return left != 0.0f && (b & 1u) == 0 && b << 1 != 0 ? __uint_as_float(away ? b + 1 : b - 1) : v;
    }
};

// W waves a row (4 / W rows a workgroup), NV vectors a lane held in registers,
// every load of a row under way at once.  Bound by memory: 16,384 x 2,560
// bfloat16 with a float32 residual into 8 bits moves 461 MB in 89 us, 5.2 TB/s
// (a device copy: 5.0 to 5.4 TB/s); into bfloat16 with a bfloat16 residual 336 MB
// in 63 us.
template <typename T, typename R, typename Q, int W, int NV, bool WHOLE>
__global__ __launch_bounds__(256) void norm_kernel(NormKernelArgs a) {
    constexpr bool Q8 = sizeof(Q) == 1;
    __shared__ float part[3][4];
    const int lane = threadIdx.x & 63, wave = wave_id(), in_row = wave % W;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (4 / W) + wave / W;
    if (W < 4 && row >= a.rows) return;  // a whole wave, and no barrier below
    const int64_t e0 = row * a.dim;
    const int64_t head = WHOLE ? 0 : e0 & (VEC - 1);
    const T* x = static_cast<const T*>(a.x) + e0;
    const R* res = static_cast<const R*>(a.res) + e0;
    float h[NV][VEC], rest[Q8 ? NV : 1][VEC];
    auto column = [&](int i) { return static_cast<int64_t>((i * W + in_row) * 64 + lane) * VEC - head; };
#pragma unroll
    for (int i = 0; i < NV; ++i) load_part<WHOLE>(x, column(i), a.dim, h[i]);
    if constexpr (Q8) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) rest[i][j] = 0.0f;
    }
    if (a.res) {
        float r[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) load_part<WHOLE>(res, column(i), a.dim, r[i]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float s = h[i][j] + r[i][j];
                if constexpr (Q8) rest[i][j] = sum_rest(h[i][j], r[i][j], s);
                h[i][j] = s;
            }
    }
    // The 8-bit form holds two registers an element: its weight comes late, from L1
    // (16,384 x 2,560: 89 us, with the weight held from the start 102 us).
    float w[Q8 ? 1 : NV][VEC];
    if constexpr (!Q8) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load_weight<WHOLE>(a.weight, column(i), a.dim, w[i]);
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < VEC; ++j) s = __builtin_fmaf(h[i][j], h[i][j], s);
        ss += s;
    }
    ss = wave_sum(ss);
    if constexpr (W == 4) {
        if (lane == 0) part[0][wave] = ss;
        __syncthreads();
        ss = (part[0][0] + part[0][1]) + (part[0][2] + part[0][3]);
    }
    const float r = 1.0f / __builtin_sqrtf(ss / static_cast<float>(a.dim) + a.eps);
    if (a.res_out) {
#pragma unroll
        for (int i = 0; i < NV; ++i) store_part<WHOLE>(static_cast<R*>(a.res_out) + e0, column(i), a.dim, h[i]);
    }
    if constexpr (Q8) {
        Largest top;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            asm volatile("" ::: "memory");  // not before this vector's turn
            load_weight<WHOLE>(a.weight, column(i), a.dim, w[0]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                times_weight(h[i][j], rest[i][j], w[0][j]);
                top.take(h[i][j], rest[i][j]);
            }
        }
        top.wave();
        if constexpr (W == 4) {
            if (lane == 0) part[1][wave] = __uint_as_float(top.bits), part[2][wave] = top.rest;
            __syncthreads();
            top = Largest{};
#pragma unroll
            for (int i = 0; i < 4; ++i) top.take(part[1][i], part[2][i]);
        }
        const RowScale q(top.bits, top.rest, r);
        if (lane == 0 && in_row == 0) a.scale[row] = q.scale;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) h[i][j] = q.apply(h[i][j], rest[i][j]);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) h[i][j] = h[i][j] * r * w[i][j];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) store_part<WHOLE>(static_cast<Q*>(a.y) + e0, column(i), a.dim, h[i]);
}

// Rows of more than 16,384 elements: a workgroup a row, which it reads once for
// the sum and again (from the caches, mostly) for each later pass.
template <typename T, typename R, typename Q>
__global__ __launch_bounds__(256) void norm_long_kernel(NormKernelArgs a) {
    constexpr bool Q8 = sizeof(Q) == 1;
    __shared__ float part[3][4];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t row = blockIdx.x, e0 = row * a.dim;
    const T* x = static_cast<const T*>(a.x) + e0;
    const R* res = a.res ? static_cast<const R*>(a.res) + e0 : nullptr;
    const int64_t head = e0 & (VEC - 1);
    auto each = [&](auto f) {  // f(column, h, the remainders of its sums)
        for (int64_t c = static_cast<int64_t>(threadIdx.x) * VEC - head; c < a.dim; c += 256 * VEC) {
            float h[VEC], rest[VEC] = {};
            load_part<false>(x, c, a.dim, h);
            if (res) {
                float r[VEC];
                load_part<false>(res, c, a.dim, r);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float s = h[j] + r[j];
                    rest[j] = sum_rest(h[j], r[j], s);
                    h[j] = s;
                }
            }
            f(c, h, rest);
        }
    };
    float ss = 0.0f;
    each([&](int64_t, float (&h)[VEC], float (&)[VEC]) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < VEC; ++j) s = __builtin_fmaf(h[j], h[j], s);
        ss += s;
    });
    ss = wave_sum(ss);
    if (lane == 0) part[0][wave] = ss;
    __syncthreads();
    ss = (part[0][0] + part[0][1]) + (part[0][2] + part[0][3]);
    const float r = 1.0f / __builtin_sqrtf(ss / static_cast<float>(a.dim) + a.eps);
    Largest top;
    if constexpr (Q8) {
        each([&](int64_t c, float (&h)[VEC], float (&rest)[VEC]) {
            float w[VEC];
            load_weight<false>(a.weight, c, a.dim, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                times_weight(h[j], rest[j], w[j]);
                top.take(h[j], rest[j]);
            }
        });
        top.wave();
        if (lane == 0) part[1][wave] = __uint_as_float(top.bits), part[2][wave] = top.rest;
        __syncthreads();
        top = Largest{};
#pragma unroll
        for (int i = 0; i < 4; ++i) top.take(part[1][i], part[2][i]);
    }
    const RowScale q(top.bits, top.rest, r);
    if (Q8 && threadIdx.x == 0) a.scale[row] = q.scale;
    // each thread writes the places it has read, after its last read of them
    each([&](int64_t c, float (&h)[VEC], float (&rest)[VEC]) {
        float w[VEC];
        load_weight<false>(a.weight, c, a.dim, w);
        if (a.res_out) store_part<false>(static_cast<R*>(a.res_out) + e0, c, a.dim, h);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if constexpr (Q8) {
                times_weight(h[j], rest[j], w[j]);
                h[j] = q.apply(h[j], rest[j]);
            } else {
                h[j] = h[j] * r * w[j];
            }
        }
        store_part<false>(static_cast<Q*>(a.y) + e0, c, a.dim, h);
    });
}

template <typename T, typename R, typename Q>
void launch_q(const NormArgs& a, hipStream_t s) {
    NormKernelArgs k{a.x, a.residual, a.weight, a.y, a.scale, a.residual_out, a.rows, a.dim, a.eps};
    const bool whole = a.dim % VEC == 0;
    // vectors a row covers (others than whole rows: up to VEC - 1 elements earlier)
    const int64_t vectors = (a.dim + (whole ? 0 : VEC - 1) + VEC - 1) / VEC;
    auto run = [&](auto w, auto nv) {
        constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
        const dim3 grid(static_cast<uint32_t>((k.rows + 4 / W - 1) / (4 / W)));
        if (whole)
            norm_kernel<T, R, Q, W, NV, true><<<grid, 256, 0, s>>>(k);
        else
            norm_kernel<T, R, Q, W, NV, false><<<grid, 256, 0, s>>>(k);
    };
    typedef std::integral_constant<int, 1> C1;
    typedef std::integral_constant<int, 2> C2;
    typedef std::integral_constant<int, 3> C3;
    typedef std::integral_constant<int, 4> C4;
    typedef std::integral_constant<int, 5> C5;
    typedef std::integral_constant<int, 8> C8;
    // Four waves a row where rows are few: 4 x 2,560 takes 3.4 us (one wave: 4.1),
    // 2,047 x 1,537 14.4 us (15.5); from 4,096 rows on both take the same.
    const bool few = a.rows < 4096;
    auto launch = [&] {
        if (vectors <= 64) run(C1{}, C1{});
        else if (vectors <= 128 && !few) run(C1{}, C2{});
        else if (vectors <= 192 && !few) run(C1{}, C3{});
        else if (vectors <= 256 && !few) run(C1{}, C4{});
        else if (vectors <= 320 && !few) run(C1{}, C5{});
        else if (vectors <= 256) run(C4{}, C1{});
        else if (vectors <= 512) run(C4{}, C2{});
        else if (vectors <= 768) run(C4{}, C3{});
        else if (vectors <= 1024) run(C4{}, C4{});
        else if (vectors <= 2048) run(C4{}, C8{});
        else norm_long_kernel<T, R, Q><<<dim3(static_cast<uint32_t>(k.rows)), 256, 0, s>>>(k);
    };
    // a launch has fewer than 2^32 threads: 2^22 rows at a time (whole vectors apart)
    constexpr int64_t kRows = int64_t{1} << 22;
    for (int64_t r0 = 0; r0 < a.rows; r0 += kRows) {
        const int64_t e0 = r0 * a.dim;
        k.rows = imin64(kRows, a.rows - r0);
        k.x = static_cast<const T*>(a.x) + e0;
        k.res = a.residual ? static_cast<const R*>(a.residual) + e0 : nullptr;
        k.res_out = a.residual_out ? static_cast<R*>(a.residual_out) + e0 : nullptr;
        k.y = static_cast<Q*>(a.y) + e0;
        k.scale = a.scale ? a.scale + r0 : nullptr;
        launch();
    }
}

template <typename T, typename R>
void launch_t(const NormArgs& a, hipStream_t s) {
    a.scale ? launch_q<T, R, uint8_t>(a, s) : launch_q<T, R, T>(a, s);
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
