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

// Four neighbouring outputs of row m from column n on.
template <int DT, typename O>
__device__ __forceinline__ void store_outputs(const LinearKernelArgs& a, int64_t m, int64_t n, f32x4 v, float xs) {
    const int64_t o = m * a.N + n;
    if ((a.N & 3) == 0) {  // whole vectors, aligned
        if (n >= a.N) return;
        if constexpr (DT == MSSM_F8) v *= xs * *reinterpret_cast<const f32x4*>(a.ws + n);
        if (a.bias) v += *reinterpret_cast<const f32x4*>(a.bias + n);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = activate(v[i], a.act);
        if constexpr (sizeof(O) == 4) {
            if (a.res) v += *reinterpret_cast<const f32x4*>(static_cast<const O*>(a.res) + o);
            *reinterpret_cast<f32x4*>(static_cast<O*>(a.y) + o) = v;
        } else {
            if (a.res) {
                const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const O*>(a.res) + o);
                v += f32x4{bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
            }
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<bf16x4*>(static_cast<O*>(a.y) + o) = __builtin_convertvector(v, bf16x4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (n + i >= a.N) return;
            float u = v[i];
            if constexpr (DT == MSSM_F8) u *= xs * a.ws[n + i];
            if (a.bias) u += a.bias[n + i];
            u = activate(u, a.act);
            if (a.res) u += load_act(static_cast<const O*>(a.res), o + i);
            store_act(static_cast<O*>(a.y), o + i, u);
        }
    }
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

// ---- the tile kernel ---------------------------------------------------------

// Four words of a raw buffer descriptor over [base, base + bytes) in scalar registers.
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4 buffer_words(const uint8_t* base, uint32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(uniform_ptr(base));
    return i32x4{static_cast<int32_t>(p), static_cast<int32_t>((p >> 32) & 0xffff),
                 static_cast<int32_t>(__builtin_amdgcn_readfirstlane(bytes)), static_cast<int32_t>(kBufferWord3)};
}

// 16 bytes a lane straight from memory into LDS: lane l's go to lds + 16 l, an
// offset outside the descriptor's range gives zeros.  Written as one statement
// without outputs because the compiler orders every LDS read behind every such
// load it knows of, which would undo the double buffering; the counter wait is
// in tile_barrier().  (m0 needs one wait state before the load; nothing else in
// these kernels uses m0, which the compiler keeps reserved.)
__device__ __forceinline__ void load_to_lds(uint32_t lds, i32x4 rsrc, uint32_t voff, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory");
}

// The tile that was being loaded is in LDS and nobody reads the other one any more.
__device__ __forceinline__ void tile_barrier() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Workgroup -> tile: the hardware deals workgroups to the 8 XCDs in turn, so
// each XCD gets one contiguous range of tiles, walked in bands of 4 tile rows:
// its 32 CUs then share 4 + 8 operand slabs in their L2.
struct TileAt { int64_t m, n; };
__device__ __forceinline__ TileAt tile_of(uint32_t id, int64_t tm, int64_t tn) {
    const int64_t T = tm * tn, xcd = id & 7, i = id >> 3, q = T >> 3, rem = T & 7;
    const int64_t t = xcd * q + (xcd < rem ? xcd : rem) + i;
    const int64_t band = t / (4 * tn), m0 = band * 4, rows = tm - m0 < 4 ? tm - m0 : 4, in = t - band * 4 * tn;
    return {m0 + in % rows, in / rows};
}

constexpr int kTileBytes = 128;             // k bytes of a tile row: eight 16-byte chunks
constexpr uint32_t kOutside = 0x7fff0000u;  // beyond any tile's range (below 2^30 bytes)

// Products over a tile row's two 64-byte halves.
template <int DT>
__device__ __forceinline__ f32x4 mma2(const u32x4 (&a)[2], const u32x4 (&b)[2], f32x4 acc) {
    if constexpr (DT == MSSM_F8) {
        typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
        const i32x8 p = __builtin_bit_cast(i32x8, __builtin_shufflevector(a[0], a[1], 0, 1, 2, 3, 4, 5, 6, 7));
        const i32x8 q = __builtin_bit_cast(i32x8, __builtin_shufflevector(b[0], b[1], 0, 1, 2, 3, 4, 5, 6, 7));
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, acc, 0, 0, 0, 0, 0, 0);
    } else {
        return mma<DT>(a[1], b[1], mma<DT>(a[0], b[0], acc));
    }
}

template <int DT, typename O, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void linear_tile_kernel(LinearKernelArgs a) {
    constexpr int E = Elem<DT>::kBytes, WAVES = WM * WN;
    constexpr int XB = BM * kTileBytes, WB = BN * kTileBytes, STAGE = XB + WB;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // 16-row fragments of a wave
    constexpr int LX = BM / (8 * WAVES), LW = BN / (8 * WAVES);
    __shared__ __align__(1024) uint8_t lds[2 * STAGE];
    const TileAt at = tile_of(blockIdx.x, (a.M + BM - 1) / BM, (a.N + BN - 1) / BN);
    const int64_t m0 = at.m * BM, n0 = at.n * BN, kbytes = a.K * E;
    const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const i32x4 rx = buffer_words(a.x + m0 * kbytes, static_cast<uint32_t>(imin64(BM, a.M - m0) * kbytes));
    const i32x4 rw = buffer_words(a.w + n0 * kbytes, static_cast<uint32_t>(imin64(BN, a.N - n0) * kbytes));

    // Row `row` of a tile keeps its chunk c at place c ^ (row / 2 % 8): the 16
    // rows that a fragment read touches lie in 16 different bank groups.  The
    // loads write LDS linearly, so the lane fetches the chunk of its place.
    const int lrow = wave * 8 + (lane >> 3), lchunk = (lane & 7) ^ ((lrow >> 1) & 7);
    const uint32_t base = lrow * static_cast<uint32_t>(kbytes) + lchunk * 16;
    const int64_t tiles = (kbytes + kTileBytes - 1) / kTileBytes;
    const bool tail_out = (tiles - 1) * kTileBytes + lchunk * 16 >= kbytes;
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
    auto load = [&](int64_t t) {
        const uint32_t soff = static_cast<uint32_t>(t * kTileBytes);
        const bool out = t == tiles - 1 && tail_out;
        const uint32_t to = lds0 + static_cast<uint32_t>(t & 1) * STAGE + wave * 1024;
#pragma unroll
        for (int i = 0; i < LX; ++i)
            load_to_lds(to + i * WAVES * 1024, rx, out ? kOutside : base + i * WAVES * 8 * static_cast<uint32_t>(kbytes), soff);
#pragma unroll
        for (int i = 0; i < LW; ++i)
            load_to_lds(to + XB + i * WAVES * 1024, rw, out ? kOutside : base + i * WAVES * 8 * static_cast<uint32_t>(kbytes), soff);
    };

    f32x4 acc[FM][FN] = {};
    const int place = ((g ^ (r >> 1)) & 7) * 16;
    const int xo = (wm * (BM / WM) + r) * kTileBytes + place, wo = XB + (wn * (BN / WN) + r) * kTileBytes + place;
    load(0);
    for (int64_t t = 0; t < tiles; ++t) {
        tile_barrier();
        if (t + 1 < tiles) load(t + 1);
        const uint8_t* st = lds + (t & 1) * STAGE;
        u32x4 wf[FN][2], xf[2];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            wf[j][0] = *reinterpret_cast<const u32x4*>(st + wo + j * 16 * kTileBytes);
            wf[j][1] = *reinterpret_cast<const u32x4*>(st + (wo ^ 64) + j * 16 * kTileBytes);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            xf[0] = *reinterpret_cast<const u32x4*>(st + xo + i * 16 * kTileBytes);
            xf[1] = *reinterpret_cast<const u32x4*>(st + (xo ^ 64) + i * 16 * kTileBytes);
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = mma2<DT>(wf[j], xf, acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t m = m0 + wm * (BM / WM) + i * 16 + r;
        if (m >= a.M) continue;
        float xs = 1.0f;
        if constexpr (DT == MSSM_F8) xs = a.xs[m];
#pragma unroll
        for (int j = 0; j < FN; ++j)
            store_outputs<DT, O>(a, m, n0 + wn * (BN / WN) + j * 16 + g * 4, acc[i][j], xs);
    }
}

template <int DT, typename O>
void launch_t(const LinearArgs& a, hipStream_t s) {
    const LinearKernelArgs k{static_cast<const uint8_t*>(a.x), static_cast<const uint8_t*>(a.w), a.x_scale, a.w_scale,
                             a.bias, a.residual, a.y, a.M, a.K, a.N, a.act};
    if (a.K * Elem<DT>::kBytes % 16 == 0) {
        if (((a.M + 255) / 256) * ((a.N + 255) / 256) >= 256) {
            linear_tile_kernel<DT, O, 256, 256, 2, 4><<<dim3(static_cast<uint32_t>(((a.M + 255) / 256) * ((a.N + 255) / 256))), 512, 0, s>>>(k);
        } else {
            linear_tile_kernel<DT, O, 128, 128, 2, 2><<<dim3(static_cast<uint32_t>(((a.M + 127) / 128) * ((a.N + 127) / 128))), 256, 0, s>>>(k);
        }
        return;
    }
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
