// linear.hip -- projections with their epilogue (mssm_linear):
// y = act(x wᵀ * scales + bias) + residual on the matrix cores.
//
// Four ways, chosen by plan_linear (linear_plan.h) from the sizes:
//  * tiles of 256 x 256 or 128 x 128 outputs, k in 128-byte steps that go from
//    memory straight into a double buffer of LDS.  Bound by the matrix cores at
//    the clock that their power leaves (2.1 GHz): 16,384 x 2,560 x 10,240 in 8
//    bits 350 to 365 us (2,350 to 2,450 TFLOP/s; a library product 2,260), in
//    bfloat16 650 us (1,320; 1,250); 16,384 x 5,120 x 2,560 bfloat16 with a
//    float32 residual 400 us (1,070; without it 350 us, 1,220; 990).
//    Scheduling of the loop's reads and loads, wave priorities and products of
//    32 x 32 make no difference within 3 %, or cost up to 10 %.
//  * few tiles, cut along k as well, their partial sums joined in a second pass;
//  * few columns (at most 128) and many rows: all columns in one workgroup;
//  * few outputs: both operands straight into registers, k over 8 waves.
#include "block.h"
#include "device_common.h"

#include <type_traits>

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
    // tiles [0, full) are one workgroup each; each of the `rest` others is
    // `splits` workgroups that leave their sums of a part of k in `partial`
    int64_t full, rest;
    int splits;
    float* partial;
};

// A sum of 8-bit products with its row's and its column's scale, one after the
// other: the scales' own product may be out of range.
__device__ __forceinline__ float scaled(float sum, float xs, float ws) { return sum * xs * ws; }

// v / (1 + exp(-v)) to float32's accuracy: exp2 of the rounded -|v| log2 e alone
// is off by up to |v| 2^-24, so the remainder of that product is carried.  exp of
// the negative magnitude does not overflow, and is 0 from -104 on (an infinite
// remainder otherwise).
__device__ __forceinline__ float silu_whole(float v) {
    constexpr float kLog2eRest = 1.925963033500012e-08f;  // log2 e = kLog2e + this
    const float a = __builtin_fmaxf(-__builtin_fabsf(v), -104.0f), t = a * kLog2e;
    const float e0 = fast_exp2(t), e = __builtin_fmaf(e0, kLn2 * __builtin_fmaf(a, kLog2eRest, __builtin_fmaf(a, kLog2e, -t)), e0);
    return (v < 0.0f ? v * e : v) * fast_rcp(1.0f + e);
}

// A bfloat16 output (2^-8) does not show the short form's error.
template <int ACT, typename O>
__device__ __forceinline__ float activate(float v) {
    if constexpr (ACT == MSSM_ACT_RELU) return v > 0.0f || v != v ? v : 0.0f;  // NaN stays
    if constexpr (ACT == MSSM_ACT_SILU) return sizeof(O) == 4 ? silu_whole(v) : silu(v);
    if constexpr (ACT == MSSM_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    return v;
}

// f(std::integral_constant<int, activation>): the epilogue's loops are compiled
// once for each activation, a test in each element would multiply their code.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f) {
    if (act == MSSM_ACT_NONE) f(std::integral_constant<int, MSSM_ACT_NONE>{});
    else if (act == MSSM_ACT_RELU) f(std::integral_constant<int, MSSM_ACT_RELU>{});
    else if (act == MSSM_ACT_SILU) f(std::integral_constant<int, MSSM_ACT_SILU>{});
    else f(std::integral_constant<int, MSSM_ACT_GELU>{});
}

// `C` neighbouring values of a float32 row (C a multiple of 4, 16-byte aligned).
template <int C>
__device__ __forceinline__ void load_columns(const float* p, float (&v)[C]) {
#pragma unroll
    for (int c = 0; c < C; c += 4) {
        const f32x4 q = *reinterpret_cast<const f32x4*>(p + c);
        v[c] = q[0]; v[c + 1] = q[1]; v[c + 2] = q[2]; v[c + 3] = q[3];
    }
}

template <typename O> struct OutVec;  // 16 bytes of outputs
template <> struct OutVec<float> {
    typedef f32x4 Raw;
    static constexpr int kCols = 4;
    __device__ static float get(const Raw& r, int c) { return r[c]; }
    __device__ static void set(Raw& r, int c, float v) { r[c] = v; }
};
template <> struct OutVec<uint16_t> {
    typedef bf16x8 Raw;
    static constexpr int kCols = 8;
    __device__ static float get(const Raw& r, int c) { return static_cast<float>(r[c]); }
    __device__ static void set(Raw& r, int c, float v) { r[c] = static_cast<__bf16>(v); }
};

// A wave's 64 x 64 float32 block, staged in 16 KB of LDS, as finished outputs.
// The accumulators hold four columns of a row in each lane; stored from there
// a row's 128 bytes would leave in 32-byte pieces.  Through LDS (16-byte
// chunk c of row i at place c ^ i % 16: no bank is hit twice) every store is
// 16 bytes a lane and whole rows, past the caches: an 8-bit in-projection of
// 16,384 x 2,560 x 10,240 takes 396 us with it, 430 us without the streaming
// stores and 456 us storing from the accumulators.  The residual is read
// ahead of the stores, behind which it would have to wait.
template <int DT, typename O>
struct BlockOut {
    static constexpr int CPL = OutVec<O>::kCols, LPR = 64 / CPL, RPI = 64 / LPR, STEPS = 64 / RPI;
    typedef typename OutVec<O>::Raw Raw;
    Raw res[STEPS];

    __device__ __forceinline__ static bool whole(const LinearKernelArgs& a) { return a.N % CPL == 0; }

    __device__ __forceinline__ void load_residual(const LinearKernelArgs& a, int64_t m0, int64_t n0, int lane) {
        const int64_t n = n0 + lane % LPR * CPL;
        if (!a.res || !whole(a)) return;
#pragma unroll
        for (int q = 0; q < STEPS; ++q) {
            const int64_t m = m0 + q * RPI + lane / LPR;
            if (m < a.M && n < a.N) res[q] = *reinterpret_cast<const Raw*>(static_cast<const O*>(a.res) + m * a.N + n);
        }
    }

    __device__ __forceinline__ void stage(uint8_t* lds, int row, int col4, f32x4 v) const {
        *reinterpret_cast<f32x4*>(lds + row * 256 + ((col4 ^ (row & 15)) * 16)) = v;
    }

    template <int ACT>
    __device__ __forceinline__ void store_rows(const LinearKernelArgs& a, const uint8_t* lds, int64_t m0, int64_t n0, int lane) const {
        const int64_t n = n0 + lane % LPR * CPL;
        if (n >= a.N) return;
        float ws[CPL], bias[CPL] = {}, xs[STEPS];
        if constexpr (DT == MSSM_F8) load_columns<CPL>(a.ws + n, ws);
        if (a.bias) load_columns<CPL>(a.bias + n, bias);
        if constexpr (DT == MSSM_F8) {
#pragma unroll
            for (int q = 0; q < STEPS; ++q) xs[q] = a.xs[imin64(m0 + q * RPI + lane / LPR, a.M - 1)];
        }
#pragma unroll
        for (int q = 0; q < STEPS; ++q) {
            const int row = q * RPI + lane / LPR;
            const int64_t m = m0 + row;
            Raw out;
#pragma unroll
            for (int c4 = 0; c4 < CPL / 4; ++c4) {
                const f32x4 v =
                    *reinterpret_cast<const f32x4*>(lds + row * 256 + (((lane % LPR * (CPL / 4) + c4) ^ (row & 15)) * 16));
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float u = v[c];
                    if constexpr (DT == MSSM_F8) u = scaled(u, xs[q], ws[c4 * 4 + c]);
                    u = activate<ACT, O>(u + bias[c4 * 4 + c]);
                    if (a.res) u += OutVec<O>::get(res[q], c4 * 4 + c);
                    OutVec<O>::set(out, c4 * 4 + c, u);
                }
            }
            if (m < a.M) __builtin_nontemporal_store(out, reinterpret_cast<Raw*>(static_cast<O*>(a.y) + m * a.N + n));
        }
    }

    // Rows that start off a 16-byte boundary: a column a lane.
    template <int ACT>
    __device__ __forceinline__ void store_columns(const LinearKernelArgs& a, const uint8_t* lds, int64_t m0, int64_t n0, int lane) const {
        const int64_t n = n0 + lane;
        if (n >= a.N) return;
        const float ws = DT == MSSM_F8 ? a.ws[n] : 1.0f, bias = a.bias ? a.bias[n] : 0.0f;
        constexpr int BATCH = 8;
        for (int r0 = 0; r0 < 64 && m0 + r0 < a.M; r0 += BATCH) {
            float xs[BATCH], add[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int64_t m = imin64(m0 + r0 + i, a.M - 1);
                xs[i] = DT == MSSM_F8 ? a.xs[m] : 1.0f;
                add[i] = a.res ? load_act(static_cast<const O*>(a.res), m * a.N + n) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int row = r0 + i;
                float u = *reinterpret_cast<const float*>(lds + row * 256 + (((lane >> 2) ^ (row & 15)) * 16) + (lane & 3) * 4);
                if constexpr (DT == MSSM_F8) u = scaled(u, xs[i], ws);
                u = activate<ACT, O>(u + bias) + add[i];
                if (m0 + row < a.M) store_act(static_cast<O*>(a.y), (m0 + row) * a.N + n, u);
            }
        }
    }

    __device__ __forceinline__ static void store_sums(const uint8_t* lds, float* to, int pitch, int64_t rows, int lane) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int row = q * 4 + (lane >> 4);
            if (row < rows)
                *reinterpret_cast<f32x4*>(to + row * pitch + (lane & 15) * 4) =
                    *reinterpret_cast<const f32x4*>(lds + row * 256 + (((lane & 15) ^ (row & 15)) * 16));
        }
    }

    __device__ __forceinline__ void store(const LinearKernelArgs& a, const uint8_t* lds, int64_t m0, int64_t n0, int lane) const {
        with_activation(a.act, [&](auto act) {
            if (whole(a)) store_rows<act>(a, lds, m0, n0, lane);
            else store_columns<act>(a, lds, m0, n0, lane);
        });
    }
};

// ---- operand rows ------------------------------------------------------------

constexpr int kTileBytes = kLinearStepBytes;  // k bytes of a step's row: eight 16-byte chunks
constexpr uint32_t kOutside = 0x7fff0000u;  // beyond any slab's range (below 2^30 bytes)

// Some rows of an operand: reads outside them give zeros.
struct Slab {
    const uint8_t* base;
    uint32_t bytes;
    __amdgpu_buffer_rsrc_t rsrc;
    __device__ __forceinline__ Slab(const uint8_t* p, int64_t row, int64_t rows, int64_t end, int64_t kbytes)
        : base(uniform_ptr(p + row * kbytes)), bytes(static_cast<uint32_t>(imin64(rows, end - row) * kbytes)),
          rsrc(make_rsrc(base, __builtin_amdgcn_readfirstlane(bytes))) {}
};

// The 16 bytes at k byte `k` of slab row `row`, zeros beyond the row's kbytes,
// of rows that are multiples of 16 bytes long.
__device__ __forceinline__ u32x4 load_even(const Slab& s, uint32_t row, uint32_t k, uint32_t kbytes) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(s.rsrc, k < kbytes ? row * kbytes + k : kOutside, 0, 0));
}

// The same of rows of any length, whose chunks start anywhere: five aligned
// words around the chunk, shifted into place.  Only for k + 20 <= kbytes: the
// fifth word then lies in the row as well (rows outside the slab hold anything,
// as do the outputs that they go to).
__device__ __forceinline__ u32x4 load_inside(const Slab& s, uint32_t row, uint32_t k, uint32_t kbytes) {
    const uint32_t off = row * kbytes + k, at = off & ~3u, shift = off & 3u;
    const u32x4 q = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(s.rsrc, at, 0, 0));
    const uint32_t e = __builtin_amdgcn_raw_buffer_load_b32(s.rsrc, at + 16, 0, 0);
    return u32x4{__builtin_amdgcn_alignbyte(q[1], q[0], shift), __builtin_amdgcn_alignbyte(q[2], q[1], shift),
                 __builtin_amdgcn_alignbyte(q[3], q[2], shift), __builtin_amdgcn_alignbyte(e, q[3], shift)};
}

// The same near the end of a row: words that end inside the slab, the bytes of
// the slab's last word if that is cut off, zeros for what is not in the row.
__device__ __forceinline__ u32x4 load_end(const Slab& s, uint32_t row, uint32_t k, uint32_t kbytes) {
    const uint32_t off = row * kbytes + k, at = off & ~3u, shift = off & 3u, cut = s.bytes & ~3u;
    const uint32_t left = k < kbytes && off < s.bytes ? kbytes - k : 0;  // bytes of the row from here on
    uint32_t w[5], last = 0;
#pragma unroll
    for (uint32_t d = 0; d < 5; ++d)
        w[d] = __builtin_amdgcn_raw_buffer_load_b32(s.rsrc, left && at + 4 * d < cut ? at + 4 * d : kOutside, 0, 0);
#pragma unroll
    for (uint32_t i = 0; i < 3; ++i)
        last |= static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b8(s.rsrc, left && cut + i < s.bytes ? cut + i : kOutside, 0, 0)) << (8 * i);
#pragma unroll
    for (uint32_t d = 0; d < 5; ++d) w[d] = at + 4 * d == cut ? last : w[d];
    u32x4 v;
#pragma unroll
    for (uint32_t d = 0; d < 4; ++d) {
        v[d] = __builtin_amdgcn_alignbyte(w[d + 1], w[d], shift);
        v[d] = left >= 4 * d + 4 ? v[d] : left <= 4 * d ? 0 : v[d] & ((1u << (8 * (left - 4 * d))) - 1);
    }
    return v;
}

// ---- the tile kernel ---------------------------------------------------------

// Tile number -> place: tiles are walked in bands of 4 tile rows, so that
// neighbours in number share 4 + 8 operand slabs of 32 tiles.
struct TileAt { int64_t m, n; };
__device__ __forceinline__ TileAt tile_at(int64_t t, int64_t tm, int64_t tn) {
    const int64_t band = t / (4 * tn), m0 = band * 4, rows = tm - m0 < 4 ? tm - m0 : 4, in = t - band * 4 * tn;
    return {m0 + in % rows, in / rows};
}

// A fragment as the matrix instructions take it: two 16-byte chunks of a row,
// 64 bytes of k apart.  The 8-bit instructions cut each product towards zero at
// 2^-13 of the power of two of the largest of its eight (of 448 x 448 - 448 x 448
// + v, v = 8 is left and v = 7 is not): the sum of 2,560 normal ones is 1.5e-5
// off, relative, of positive ones with wide channels in both operands 1.2e-4, and
// any sum within 7 x 2^-13 of the sum of magnitudes.  With the operands widened to
// bfloat16, which is exact, 5e-8, at half the rate (few rows: 1 x 2,560 x 10,240
// 8.7 us instead of 7.7).  A bfloat16 output (2^-8) does not show it unless the
// sum cancels, a float32 one would: WIDE is that.
template <int DT, bool WIDE>
struct Frag {
    u32x4 h[2];
    __device__ __forceinline__ void set(u32x4 a, u32x4 b) { h[0] = a, h[1] = b; }
    __device__ __forceinline__ static f32x4 mma(const Frag& p, const Frag& q, f32x4 acc) {
        if constexpr (DT == MSSM_F8) {
            typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
            const i32x8 u = __builtin_bit_cast(i32x8, __builtin_shufflevector(p.h[0], p.h[1], 0, 1, 2, 3, 4, 5, 6, 7));
            const i32x8 v = __builtin_bit_cast(i32x8, __builtin_shufflevector(q.h[0], q.h[1], 0, 1, 2, 3, 4, 5, 6, 7));
            return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(u, v, acc, 0, 0, 0, 0, 0, 0);
        } else {
            return mssm::mma<DT>(p.h[1], q.h[1], mssm::mma<DT>(p.h[0], q.h[0], acc));
        }
    }
};
template <>
struct Frag<MSSM_F8, true> {
    bf16x8 v[4];
    __device__ __forceinline__ void set(u32x4 a, u32x4 b) {
        widen(a, v[0], v[1]);
        widen(b, v[2], v[3]);
    }
    __device__ __forceinline__ static void widen(u32x4 c, bf16x8& lo, bf16x8& hi) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        bf16x2 p[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, false);
            p[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, true);
        }
        lo = bf16x8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
        hi = bf16x8{p[4][0], p[4][1], p[5][0], p[5][1], p[6][0], p[6][1], p[7][0], p[7][1]};
    }
    __device__ __forceinline__ static f32x4 mma(const Frag& p, const Frag& q, f32x4 acc) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p.v[i], q.v[i], acc, 0, 0, 0);
        return acc;
    }
};

template <int DT, typename O, int BM, int BN, int WM, int WN, bool EVEN>
__global__ __launch_bounds__(64 * WM * WN, 2) void linear_tile_kernel(LinearKernelArgs a) {
    constexpr int E = Elem<DT>::kBytes, WAVES = WM * WN;
    constexpr int XB = BM * kTileBytes, WB = BN * kTileBytes, STAGE = XB + WB;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // 16-row fragments of a wave
    constexpr int LX = BM / (8 * WAVES), LW = BN / (8 * WAVES);
    __shared__ __align__(1024) uint8_t lds[2 * STAGE];
    // The hardware deals workgroups to the 8 XCDs in turn: each XCD gets one
    // contiguous range of the whole tiles (full is a multiple of 8, or all).
    const int64_t id = blockIdx.x + static_cast<int64_t>(blockIdx.y) * gridDim.x, whole = a.full;
    if (id >= whole + a.rest * a.splits) return;  // the grid's last row
    const bool split = id >= whole;
    const int64_t t_id = split ? whole + (id - whole) % a.rest
                               : (id & 7) * (whole >> 3) + ((id & 7) < (whole & 7) ? (id & 7) : (whole & 7)) + (id >> 3);
    const int part = split ? static_cast<int>((id - whole) / a.rest) : 0;
    const TileAt at = tile_at(t_id, (a.M + BM - 1) / BM, (a.N + BN - 1) / BN);
    const int64_t m0 = at.m * BM, n0 = at.n * BN, kbytes = a.K * E;
    const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    // Row `row` of a tile keeps its chunk c at place c ^ (row / 2 % 8): the 16
    // rows that a fragment read touches lie in 16 different bank groups.  The
    // loads write LDS linearly, so the lane fetches the chunk of its place.
    const int lrow = wave * 8 + (lane >> 3), lchunk = (lane & 7) ^ ((lrow >> 1) & 7);
    const int64_t tiles = (kbytes + kTileBytes - 1) / kTileBytes;
    const int64_t first = split ? tiles * part / a.splits : 0, last = split ? tiles * (part + 1) / a.splits : tiles;
    const Slab sx(a.x, m0, BM, a.M, kbytes), sw(a.w, n0, BN, a.N, kbytes);
    // EVEN rows go from memory to LDS by themselves; others through registers,
    // loaded a step ahead and written when their buffer is free.
    const i32x4 rx = buffer_words(sx.base, sx.bytes), rw = buffer_words(sw.base, sw.bytes);
    const uint32_t base = lrow * static_cast<uint32_t>(kbytes) + lchunk * 16;
    const bool tail_out = (tiles - 1) * kTileBytes + lchunk * 16 >= kbytes;
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
    u32x4 held[EVEN ? 1 : LX + LW];
    auto load = [&](int64_t t) {
        if constexpr (EVEN) {
            const uint32_t soff = static_cast<uint32_t>(t * kTileBytes);
            const bool out = t == tiles - 1 && tail_out;
            const uint32_t to = lds0 + static_cast<uint32_t>(t & 1) * STAGE + wave * 1024;
#pragma unroll
            for (int i = 0; i < LX; ++i)
                load_to_lds(to + i * WAVES * 1024, rx, out ? kOutside : base + i * WAVES * 8 * static_cast<uint32_t>(kbytes), soff);
#pragma unroll
            for (int i = 0; i < LW; ++i)
                load_to_lds(to + XB + i * WAVES * 1024, rw, out ? kOutside : base + i * WAVES * 8 * static_cast<uint32_t>(kbytes), soff);
        } else {
            const uint32_t k = static_cast<uint32_t>(t * kTileBytes) + lchunk * 16, kb = static_cast<uint32_t>(kbytes);
            if ((t + 1) * kTileBytes + 4 <= kbytes) {
#pragma unroll
                for (int i = 0; i < LX + LW; ++i)
                    held[i] = load_inside(i < LX ? sx : sw, lrow + (i < LX ? i : i - LX) * WAVES * 8, k, kb);
            } else {
#pragma unroll
                for (int i = 0; i < LX + LW; ++i)
                    held[i] = load_end(i < LX ? sx : sw, lrow + (i < LX ? i : i - LX) * WAVES * 8, k, kb);
            }
        }
    };
    auto keep = [&](int64_t t) {
        if constexpr (!EVEN) {
            uint8_t* to = lds + (t & 1) * STAGE + wave * 1024 + lane * 16;
#pragma unroll
            for (int i = 0; i < LX + LW; ++i)
                *reinterpret_cast<u32x4*>(to + (i < LX ? i * WAVES * 1024 : XB + (i - LX) * WAVES * 1024)) = held[i];
        }
    };

    f32x4 acc[FM][FN] = {};
    const int place = ((g ^ (r >> 1)) & 7) * 16;
    const int xo = (wm * (BM / WM) + r) * kTileBytes + place, wo = XB + (wn * (BN / WN) + r) * kTileBytes + place;
    load(first);
    keep(first);
    for (int64_t t = first; t < last; ++t) {
        tile_barrier();
        if (t + 1 < last) load(t + 1);
        const uint8_t* st = lds + (t & 1) * STAGE;
        auto at_lds = [&](int o) { return *reinterpret_cast<const u32x4*>(st + o); };
        typedef Frag<DT, sizeof(O) == 4> F;
        F wf[FN], xf;
#pragma unroll
        for (int j = 0; j < FN; ++j) wf[j].set(at_lds(wo + j * 16 * kTileBytes), at_lds((wo ^ 64) + j * 16 * kTileBytes));
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            xf.set(at_lds(xo + i * 16 * kTileBytes), at_lds((xo ^ 64) + i * 16 * kTileBytes));
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = F::mma(wf[j], xf, acc[i][j]);
        }
        if (t + 1 < last) keep(t + 1);
    }
    static_assert(BN / WN == 64 && FM % 4 == 0 && WAVES * 16384 <= 2 * STAGE, "64-column waves, 16 KB of LDS each");
    BlockOut<DT, O> out;
    uint8_t* mine = lds + wave * 16384;
    const int64_t mw = m0 + wm * (BM / WM), nw = n0 + wn * 64;
    auto stage = [&](int h) {
        wave_handoff();  // the block before has been read
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) out.stage(mine, i * 16 + r, j * 4 + g, acc[h * 4 + i][j]);
        wave_handoff();
    };
    if (split) {
        float* sums = a.partial + ((part * a.rest + t_id - whole) * BM + wm * (BM / WM)) * BN + wn * 64;
        tile_barrier();  // the last step's reads are done
#pragma unroll
        for (int h = 0; h < FM / 4; ++h) {
            stage(h);
            out.store_sums(mine, sums + h * 64 * BN, BN, a.M - mw - h * 64, lane);
        }
        return;
    }
    out.load_residual(a, mw, nw, lane);
    tile_barrier();
#pragma unroll
    for (int h = 0; h < FM / 4; ++h) {
        stage(h);
        out.store(a, mine, mw + h * 64, nw, lane);
        if (h + 1 < FM / 4) out.load_residual(a, mw + (h + 1) * 64, nw, lane);
    }
}

// ---- few rows ------------------------------------------------------------------

// Four neighbouring outputs of one row from the accumulators.
template <int DT, typename O, int ACT>
__device__ __forceinline__ void store_four(const LinearKernelArgs& a, int64_t m, int64_t n, f32x4 v) {
    if (m >= a.M || n >= a.N) return;
    const int64_t o = m * a.N + n;
    O* y = static_cast<O*>(a.y) + o;
    const O* res = a.res ? static_cast<const O*>(a.res) + o : nullptr;
    const float xs = DT == MSSM_F8 ? a.xs[m] : 1.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int64_t nc = imin64(n + c, a.N - 1);
        if constexpr (DT == MSSM_F8) v[c] = scaled(v[c], xs, a.ws[nc]);
        v[c] = activate<ACT, O>(v[c] + (a.bias ? a.bias[nc] : 0.0f));
    }
    if (a.N % 4 == 0) {
        if constexpr (sizeof(O) == 4) {
            if (res) v += *reinterpret_cast<const f32x4*>(res);
            *reinterpret_cast<f32x4*>(y) = v;
        } else {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            if (res) v += __builtin_convertvector(*reinterpret_cast<const bf16x4*>(res), f32x4);
            *reinterpret_cast<bf16x4*>(y) = __builtin_convertvector(v, bf16x4);
        }
    } else {
        float add[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) add[c] = res && n + c < a.N ? load_act(res, c) : 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (n + c < a.N) store_act(y, c, v[c] + add[c]);
    }
}

constexpr int kRowWaves = 8;

// Few outputs: 16 MF rows by 16 columns a workgroup, both operands straight from
// memory into registers as matrix operands.  The 8 waves take the 128-byte
// steps of k in turn, U of them in flight each, and add their sums through LDS
// in the order of the waves: one launch, and every wave of a decode step's
// product has its part of the weight under way at once.  1 x 2,560 x 10,240
// bfloat16 takes 12 us (4.4 TB/s), by split tiles and a second pass 20 us.
template <int DT, typename O, int MF, bool EVEN, int U>
__global__ __launch_bounds__(512) void linear_rows_kernel(LinearKernelArgs a) {
    constexpr int WAVES = kRowWaves;
    __shared__ __align__(16) f32x4 part[WAVES][MF][64];
    const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, g = lane >> 4;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
    const uint32_t kbytes = static_cast<uint32_t>(a.K * Elem<DT>::kBytes);
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (16 * MF);
    const Slab sw(a.w, n0, 16, a.N, kbytes), sx(a.x, m0, 16 * MF, a.M, kbytes);
    typedef Frag<DT, sizeof(O) == 4> F;
    f32x4 acc[MF] = {};
    auto steps = [&](auto count, uint32_t k0, auto chunk) {
        constexpr int C = decltype(count)::value;
        u32x4 wf[C][2], xf[C][MF][2];
#pragma unroll
        for (int u = 0; u < C; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t k = k0 + u * WAVES * kTileBytes + h * 64 + g * 16;
                wf[u][h] = chunk(sw, r, k, kbytes);
#pragma unroll
                for (int i = 0; i < MF; ++i) xf[u][i][h] = chunk(sx, i * 16 + r, k, kbytes);
            }
#pragma unroll
        for (int u = 0; u < C; ++u)
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                F p, q;
                p.set(wf[u][0], wf[u][1]);
                q.set(xf[u][i][0], xf[u][i][1]);
                acc[i] = F::mma(p, q, acc[i]);
            }
    };
    constexpr std::integral_constant<int, U> all;
    constexpr std::integral_constant<int, 1> one;
    for (uint32_t k0 = wave * kTileBytes; k0 < kbytes; k0 += WAVES * U * kTileBytes) {
        if constexpr (EVEN)
            steps(all, k0, load_even);
        else if (k0 + ((U - 1) * WAVES + 1) * kTileBytes + 4 <= kbytes)
            steps(all, k0, load_inside);
        else
            for (uint32_t k = k0; k < kbytes && k < k0 + WAVES * U * kTileBytes; k += WAVES * kTileBytes)
                k + kTileBytes + 4 <= kbytes ? steps(one, k, load_inside) : steps(one, k, load_end);
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave >= MF) return;
    f32x4 v = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += part[w][wave][lane];
    with_activation(a.act, [&](auto act) { store_four<DT, O, act>(a, m0 + wave * 16 + r, n0 + g * 4, v); });
}

// ---- few columns ---------------------------------------------------------------

// At most 16 FN columns: a workgroup computes all of them for 16 RG rows, so
// that x is read once.  The first RG waves take 16 rows each and the first 64
// bytes of every k step, the others the second 64 bytes (two waves a SIMD, one
// fetches while the other multiplies); their sums are added through LDS.  Steps
// arrive in four LDS stages, three of them in flight.  16,384 x 1,536 x 80 takes
// 39 us in float32 (its matrix instructions alone 26 us; 0.72 us a step, of them
// 0.53, and neither fewer barriers, nor fragments read a step ahead, nor more
// stages shorten it) and 12 us in bfloat16 (4.3 TB/s).
template <int DT, typename O, int FN, int RG>
__global__ __launch_bounds__(128 * RG, 2) void linear_columns_kernel(LinearKernelArgs a) {
    constexpr int STAGES = 4, WL = (FN + RG - 1) / RG, LOADS = 1 + WL;  // 16 RG rows a load of all the waves: x, then w
    constexpr int ROUND = 16 * RG * kTileBytes, STAGE = LOADS * ROUND;
    __shared__ __align__(1024) uint8_t lds[STAGES * STAGE];
    const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, g = lane >> 4;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * (16 * RG), kbytes = a.K * Elem<DT>::kBytes;
    const Slab sx(a.x, m0, 16 * RG, a.M, kbytes), sw(a.w, 0, 16 * FN, a.N, kbytes);
    const i32x4 rx = buffer_words(sx.base, sx.bytes), rw = buffer_words(sw.base, sw.bytes);
    const int lrow = wave * 8 + (lane >> 3), lchunk = (lane & 7) ^ ((lrow >> 1) & 7);
    const int tiles = static_cast<int>((kbytes + kTileBytes - 1) / kTileBytes);
    const uint32_t base = lrow * static_cast<uint32_t>(kbytes) + lchunk * 16;
    const bool tail_out = static_cast<int64_t>(tiles - 1) * kTileBytes + lchunk * 16 >= kbytes;
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
    auto load = [&](int t) {
        const uint32_t soff = static_cast<uint32_t>(t) * kTileBytes, to = lds0 + (t % STAGES) * STAGE + wave * 1024;
        const bool out = t == tiles - 1 && tail_out;
        load_to_lds(to, rx, out ? kOutside : base, soff);
#pragma unroll
        for (int i = 0; i < WL; ++i)
            load_to_lds(to + (i + 1) * ROUND, rw, out ? kOutside : base + i * 16 * RG * static_cast<uint32_t>(kbytes), soff);
    };
    const int half = wave / RG, xrow = wave % RG * 16 + r;
    const int place = ((half * 4 + g) ^ (r >> 1)) * 16;
    f32x4 acc[FN] = {};
    for (int t = 0; t < STAGES - 1 && t < tiles; ++t) load(t);
    for (int t = 0; t < tiles; ++t) {
        // step t is here when at most the two later steps are under way
        if (t + STAGES - 2 < tiles)
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(2 * LOADS) : "memory");
        else
            tile_barrier();
        if (t + STAGES - 1 < tiles) load(t + STAGES - 1);
        const uint8_t* st = lds + (t % STAGES) * STAGE;
        const u32x4 xf = *reinterpret_cast<const u32x4*>(st + xrow * kTileBytes + place);
        if constexpr (DT == MSSM_F8) {  // few columns never wait for the matrix cores: widened for both outputs
            typedef Frag<MSSM_F8, true> F;
            bf16x8 x0, x1, w0, w1;
            F::widen(xf, x0, x1);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                F::widen(*reinterpret_cast<const u32x4*>(st + (16 * RG + j * 16 + r) * kTileBytes + place), w0, w1);
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, x0, acc[j], 0, 0, 0);
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, x1, acc[j], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[j] = mma<DT>(*reinterpret_cast<const u32x4*>(st + (16 * RG + j * 16 + r) * kTileBytes + place), xf, acc[j]);
        }
    }
    tile_barrier();
    f32x4* part = reinterpret_cast<f32x4*>(lds) + wave % RG * FN * 64 + lane;
    if (half) {
#pragma unroll
        for (int j = 0; j < FN; ++j) part[j * 64] = acc[j];
    }
    __syncthreads();
    if (half) return;
    with_activation(a.act, [&](auto act) {
#pragma unroll
        for (int j = 0; j < FN; ++j) store_four<DT, O, act>(a, m0 + xrow, j * 16 + g * 4, acc[j] + part[j * 64]);
    });
}

// The split tiles' parts added in order, and the epilogue: 16 rows of a tile a
// workgroup, four columns a lane.  128 tiles of 256 x 256 in two parts with a
// float32 residual (134 MB) take 22 us.
template <int DT, typename O, int BM, int BN>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearKernelArgs a) {
    constexpr int LPR = BN / 4, ROWS = 256 / LPR;  // lanes a row, rows at a time
    const int64_t q = blockIdx.x / (BM / 16), r0 = blockIdx.x % (BM / 16) * 16;
    const TileAt at = tile_at(a.full + q, (a.M + BM - 1) / BM, (a.N + BN - 1) / BN);
    const int64_t n = at.n * BN + threadIdx.x % LPR * 4;
    if (n >= a.N) return;
    const bool whole = a.N % 4 == 0;
    f32x4 ws = {1, 1, 1, 1}, bias = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int64_t nc = imin64(n + c, a.N - 1);
        if constexpr (DT == MSSM_F8) ws[c] = a.ws[nc];
        if (a.bias) bias[c] = a.bias[nc];
    }
    with_activation(a.act, [&](auto act) {
        for (int i = threadIdx.x / LPR; i < 16; i += ROWS) {
            const int64_t m = at.m * BM + r0 + i;
            if (m >= a.M) break;
            const float* p = a.partial + (q * BM + r0 + i) * BN + threadIdx.x % LPR * 4;
            f32x4 v = *reinterpret_cast<const f32x4*>(p);
            for (int s = 1; s < a.splits; ++s) v += *reinterpret_cast<const f32x4*>(p + s * a.rest * (BM * BN));
            float xs = 1.0f;
            if constexpr (DT == MSSM_F8) xs = a.xs[m];
            const int64_t o = m * a.N + n;
            O* y = static_cast<O*>(a.y) + o;
            const O* res = a.res ? static_cast<const O*>(a.res) + o : nullptr;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if constexpr (DT == MSSM_F8) v[c] = scaled(v[c], xs, ws[c]);
                v[c] = activate<act, O>(v[c] + bias[c]);
            }
            if (whole) {
                if constexpr (sizeof(O) == 4) {
                    if (res) v += *reinterpret_cast<const f32x4*>(res);
                    *reinterpret_cast<f32x4*>(y) = v;
                } else {
                    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                    if (res) v += __builtin_convertvector(*reinterpret_cast<const bf16x4*>(res), f32x4);
                    *reinterpret_cast<bf16x4*>(y) = __builtin_convertvector(v, bf16x4);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (n + c < a.N) store_act(y, c, v[c] + (res ? load_act(res, c) : 0.0f));
            }
        }
    });
}

// ---- schedule ----------------------------------------------------------------

template <int DT, typename O, int B, int WM, int WN, bool EVEN>
void launch_tiles(const LinearKernelArgs& k, const LinearPlan& p, hipStream_t s) {
    const LinearGrid g = linear_grid(p.full + p.rest * p.splits);
    linear_tile_kernel<DT, O, B, B, WM, WN, EVEN><<<dim3(g.x, g.y), 64 * WM * WN, 0, s>>>(k);
    if (p.splits > 1) linear_join_kernel<DT, O, B, B><<<dim3(static_cast<uint32_t>(p.rest * (B / 16))), 256, 0, s>>>(k);
}

template <int DT, typename O, int MF>
void launch_rows(const LinearKernelArgs& k, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>((k.N + 15) / 16), static_cast<uint32_t>((k.M + 16 * MF - 1) / (16 * MF)));
    const int64_t kbytes = k.K * Elem<DT>::kBytes;
    if (kbytes % 16 != 0) {
        linear_rows_kernel<DT, O, MF, false, MF == 1 ? 4 : 2><<<grid, 512, 0, s>>>(k);
    } else if constexpr (MF > 1) {  // more steps in flight: no gain, or up to a third slower by their registers
        linear_rows_kernel<DT, O, MF, true, 2><<<grid, 512, 0, s>>>(k);
    } else {
        // A wave's steps in the fewest turns of at most 5, evenly: 5 steps in one
        // turn of 5 take 12.0 us where turns of 4 take 13.9; 3 steps in one of 3
        // 7.3 us, of 4 8.0 us, of 5 8.7 us.
        const int64_t steps = (kbytes + kTileBytes * kRowWaves - 1) / (kTileBytes * kRowWaves), turns = (steps + 4) / 5;
        switch ((steps + turns - 1) / turns) {
            case 1: linear_rows_kernel<DT, O, MF, true, 1><<<grid, 512, 0, s>>>(k); break;
            case 2: linear_rows_kernel<DT, O, MF, true, 2><<<grid, 512, 0, s>>>(k); break;
            case 3: linear_rows_kernel<DT, O, MF, true, 3><<<grid, 512, 0, s>>>(k); break;
            case 4: linear_rows_kernel<DT, O, MF, true, 4><<<grid, 512, 0, s>>>(k); break;
            default: linear_rows_kernel<DT, O, MF, true, 5><<<grid, 512, 0, s>>>(k); break;
        }
    }
}

template <int DT, typename O, int FN>
void launch_columns(const LinearKernelArgs& k, hipStream_t s) {
    constexpr int RG = 4;  // 16 or 32 rows take 1.8 and 1.04 times as long at 16,384 x 1,536 x 80
    linear_columns_kernel<DT, O, FN, RG><<<dim3(static_cast<uint32_t>((k.M + 16 * RG - 1) / (16 * RG))), 128 * RG, 0, s>>>(k);
}

template <int DT, typename O>
void launch_t(const LinearArgs& a, const LinearPlan& p, hipStream_t s) {
    const LinearKernelArgs k{static_cast<const uint8_t*>(a.x), static_cast<const uint8_t*>(a.w), a.x_scale, a.w_scale,
                             a.bias, a.residual, a.y, a.M, a.K, a.N, a.act, p.full, p.rest, p.splits, a.partial};
    const bool even = a.K * Elem<DT>::kBytes % 16 == 0;
    switch (p.path) {
        case LinearPath::kTile256:
            if constexpr (DT != MSSM_F8 || sizeof(O) == 2) launch_tiles<DT, O, 256, 2, 4, true>(k, p, s);
            break;
        case LinearPath::kTile128:
            even ? launch_tiles<DT, O, 128, 2, 2, true>(k, p, s) : launch_tiles<DT, O, 128, 2, 2, false>(k, p, s);
            break;
        case LinearPath::kRows:
            switch ((a.M + 15) / 16) {
                case 1: launch_rows<DT, O, 1>(k, s); break;
                case 2: launch_rows<DT, O, 2>(k, s); break;
                default: launch_rows<DT, O, 4>(k, s); break;
            }
            break;
        case LinearPath::kColumns:
            switch ((a.N + 15) / 16) {
                case 1: launch_columns<DT, O, 1>(k, s); break;
                case 2: launch_columns<DT, O, 2>(k, s); break;
                case 3: launch_columns<DT, O, 3>(k, s); break;
                case 4: launch_columns<DT, O, 4>(k, s); break;
                case 5: launch_columns<DT, O, 5>(k, s); break;
                case 6: launch_columns<DT, O, 6>(k, s); break;
                default: launch_columns<DT, O, 8>(k, s); break;
            }
            break;
    }
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, const LinearPlan& p, hipStream_t s) {
    if (a.dtype == MSSM_F32)
        launch_t<MSSM_F32, float>(a, p, s);
    else if (a.dtype == MSSM_BF16)
        a.out_dtype == MSSM_F32 ? launch_t<MSSM_BF16, float>(a, p, s) : launch_t<MSSM_BF16, uint16_t>(a, p, s);
    else
        a.out_dtype == MSSM_F32 ? launch_t<MSSM_F8, float>(a, p, s) : launch_t<MSSM_F8, uint16_t>(a, p, s);
    return hipGetLastError();
}

}  // namespace mssm
