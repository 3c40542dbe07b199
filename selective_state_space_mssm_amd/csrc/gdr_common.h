// gdr_common.h -- device helpers shared by the gated delta rule's kernels:
// float32 products on the bfloat16 matrix cores, where a sequence's chunks lie,
// and a chunk's q and k in LDS.
//
// Matrix instruction 16x16x32 bfloat16 (wave64; lane l, c = l % 16, group g = l / 16):
//   operands: lane holds 8 values of row (column) c, its slots (g, 0..7) of the
//   32 summed over; any order of these will do if both operands have it.
//   accumulator item r: row 4 g + r, column c.
// The order used throughout is slot (g, j) <-> 4 g + j for j < 4 and 16 + 4 g +
// (j - 4) otherwise ("folded"): two accumulators of 16 rows each, one above the
// other, are then an operand that is summed over these rows without any lane
// having to exchange a value.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.h"
#include "gdr.h"

namespace mssm {
namespace gdrk {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kC = kGdrChunk;

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

// Which of the 16 x 32 blocks of a 64 x 64 matrix are stored: those of a lower
// triangle (`LOWER`) or of an upper one; -1: the block is zero.
template <bool LOWER>
constexpr int block_of(int rt, int ks) {
    if (LOWER) return rt < 2 ? (ks == 0 ? rt : -1) : 2 + (rt - 2) * 2 + ks;
    return rt < 2 ? rt * 2 + ks : (ks == 1 ? 2 + rt : -1);
}

template <int N>
__device__ __forceinline__ Planes<N> load_block(const uint8_t* mat, int block, int lane) {
    Planes<N> out;
#pragma unroll
    for (int n = 0; n < N; ++n)
        out.p[n] = *reinterpret_cast<const u32x4*>(mat + (n * kGdrBlocks + block) * kGdrBlockBytes + lane * 16);
    return out;
}

// ---- sequences --------------------------------------------------------------

struct Span {
    int64_t start, len;
};
__device__ __forceinline__ Span span_of(const int32_t* offsets, int64_t n, int64_t T, int64_t N) {
    if (!offsets) {
        const int64_t len = T / N;
        return {n * len, len};
    }
    int64_t s = offsets[n], e = offsets[n + 1];
    s = s < 0 ? 0 : s > T ? T : s;
    e = e < s ? s : e > T ? T : e;
    return {s, e - s};
}
__device__ __forceinline__ int64_t first_slot(const Span& s, int64_t n) { return s.start / kC + n; }

// The sequence and chunk of a slot; len = 0: the slot is no chunk.
struct Chunk {
    int64_t seq, start;  // its first token
    int len;             // tokens, up to 64
};
__device__ __forceinline__ Chunk chunk_of(const int32_t* offsets, int64_t slot, int64_t T, int64_t N) {
    int64_t lo = 0, hi = N;  // the last sequence whose first slot is not behind this one
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (first_slot(span_of(offsets, mid, T, N), mid) <= slot) lo = mid;
        else hi = mid;
    }
    const Span s = span_of(offsets, lo, T, N);
    const int64_t t = (slot - first_slot(s, lo)) * kC;
    if (t < 0 || t >= s.len) return {lo, 0, 0};
    return {lo, s.start + t, static_cast<int>(imin64(kC, s.len - t))};
}

// ---- elements of rows ---------------------------------------------------------

// Eight neighbouring elements as planes, or zeros.
__device__ __forceinline__ Planes<1> load_planes(const uint16_t* p, bool in) {
    Planes<1> out;
    out.p[0] = in ? *reinterpret_cast<const u32x4*>(p) : u32x4{0, 0, 0, 0};
    return out;
}
__device__ __forceinline__ Planes<3> load_planes(const float* p, bool in) {
    const f32x4 zero = {0, 0, 0, 0};
    return split<3>(in ? *reinterpret_cast<const f32x4*>(p) : zero, in ? *reinterpret_cast<const f32x4*>(p + 4) : zero);
}
template <int N>
__device__ __forceinline__ float sum_squares(const Planes<N>& x) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int n = N - 1; n >= 0; --n) lo += bf16_lo(x.p[n][i]), hi += bf16_hi(x.p[n][i]);
        s = __builtin_fmaf(lo, lo, __builtin_fmaf(hi, hi, s));
    }
    return s;
}

// Neighbouring values of a row in float32: two (one column of each of two tiles) or one.
__device__ __forceinline__ void load_values(const float* p, float (&v)[2]) {
    const f32x2 a = *reinterpret_cast<const f32x2*>(p);
    v[0] = a[0]; v[1] = a[1];
}
__device__ __forceinline__ void load_values(const uint16_t* p, float (&v)[2]) {
    const uint32_t a = *reinterpret_cast<const uint32_t*>(p);
    v[0] = bf16_lo(a); v[1] = bf16_hi(a);
}
__device__ __forceinline__ void load_values(const float* p, float (&v)[1]) { v[0] = *p; }
__device__ __forceinline__ void load_values(const uint16_t* p, float (&v)[1]) { v[0] = load_act(p, 0); }
__device__ __forceinline__ void store_values(float* p, const float (&v)[2]) { *reinterpret_cast<f32x2*>(p) = f32x2{v[0], v[1]}; }
__device__ __forceinline__ void store_values(uint16_t* p, const float (&v)[2]) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    *reinterpret_cast<bf16x2*>(p) = bf16x2{static_cast<__bf16>(v[0]), static_cast<__bf16>(v[1])};
}
__device__ __forceinline__ void store_values(float* p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void store_values(uint16_t* p, const float (&v)[1]) { store_act(p, 0, v[0]); }

// N (a multiple of 4) neighbouring values to a row.
template <int N>
__device__ __forceinline__ void store_row(float* p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
}
template <int N>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[N]) {
    typedef __bf16 bf16xn __attribute__((ext_vector_type(N)));
    bf16xn b;
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = static_cast<__bf16>(v[i]);
    *reinterpret_cast<bf16xn*>(p) = b;
}

// ---- decays -------------------------------------------------------------------

// exp of a float64, to float32's accuracy also where its argument is large.
__device__ __forceinline__ float whole_exp(double x) {
    const float f = static_cast<float>(x), e = expf(f);
    return __builtin_fmaf(e, static_cast<float>(x - f), e);
}
// One wave, a token a lane: the sum of the chunk's log decays up to the lane's token.
__device__ __forceinline__ double decays_since_start(const float* g, int64_t stride, int len, int lane) {
    const float gl = lane < len ? g[lane * stride] : 0.0f;
    double b = gl < kGdrLeast ? kGdrLeast : gl;
#pragma unroll
    for (int d = 1; d < kC; d *= 2) {
        const double o = __shfl_up(b, d);
        if (lane >= d) b += o;
    }
    return b;
}
// exp(b_i - b_j) of sums kept as float32 and remainder
__device__ __forceinline__ float decay_between(float hi_i, float lo_i, float hi_j, float lo_j) {
    return expf((hi_i - hi_j) + (lo_i - lo_j));
}

// ---- a chunk's q and k in LDS ---------------------------------------------------

// 64 rows of a tensor (tokens) of up to KP columns, as planes in LDS, by rows (for
// products summed over the columns) or by columns (summed over the tokens), in
// the folded order of what is summed over.  A lane's operand is one 16-byte piece
// of a row; piece c of row r lies at place c ^ (r, or r / 2 where a row is 128
// bytes), so that the 16 rows that a read takes at once spread over the banks.
template <int KP>
struct RowTile {
    static constexpr int kRow = KP * 2, kBytes = kC * kRow;
    static constexpr int kMask = KP / 8 - 1;
    __device__ static __forceinline__ int at(int row, int piece) {
        return row * kRow + ((piece ^ ((KP == 64 ? row >> 1 : row) & kMask)) * 16);
    }
};
template <int KP>
struct ColumnTile {
    static constexpr int kRow = kC * 2, kBytes = KP * kRow;
    __device__ static __forceinline__ int at(int column, int piece) { return column * kRow + ((piece ^ ((column >> 1) & 7)) * 16); }
};
template <typename Tile, int N>
__device__ __forceinline__ Planes<N> read_tile(const uint8_t* lds, int row, int piece) {
    Planes<N> out;
#pragma unroll
    for (int n = 0; n < N; ++n) out.p[n] = *reinterpret_cast<const u32x4*>(lds + n * Tile::kBytes + Tile::at(row, piece));
    return out;
}

// One thread's share of a tile on its way from memory: 4 tokens of 8 columns.
// Held as loaded from the loads' issue (load) to the stores to LDS (store).
template <typename T, int KP>
struct Patch {
    static constexpr int kItems = (kC / 4) * (KP / 8);  // 128 or 256 threads have one
    static constexpr int kWords = sizeof(T) == 2 ? 4 : 8;
    uint32_t raw[4][kWords];

    __device__ static __forceinline__ int quad(int item) { return item % 16; }   // tokens 4 quad ..
    __device__ static __forceinline__ int octet(int item) { return item / 16; }  // columns 8 octet ..

    // rows: the chunk's first token's row; stride: elements from a token to the next
    __device__ __forceinline__ void load(const T* rows, int64_t stride, int len, int K, int item) {
        const int t0 = quad(item) * 4, k0 = octet(item) * 8;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const bool in = item < kItems && t0 + t < len && k0 < K;
            const u32x4* p = reinterpret_cast<const u32x4*>(rows + (t0 + t) * stride + k0);
#pragma unroll
            for (int w = 0; w < kWords; w += 4) {
                const u32x4 v = in ? p[w / 4] : u32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) raw[t][w + i] = v[i];
            }
        }
    }
    // plane n of token t: 4 words of column pairs
    __device__ __forceinline__ void plane(int n, uint32_t (&out)[4][4]) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) {
                    out[t][i] = raw[t][i];
                } else {
                    float a = __uint_as_float(raw[t][2 * i]), b = __uint_as_float(raw[t][2 * i + 1]);
                    out[t][i] = upper_halves(a, b);
                    raw[t][2 * i] = __float_as_uint(a - upper_part(a));
                    raw[t][2 * i + 1] = __float_as_uint(b - upper_part(b));
                }
            }
    }
    // to the tile by rows and / or by columns (null: not); leaves nothing to store again
    __device__ __forceinline__ void store(uint8_t* by_row, uint8_t* by_column, int item) {
        if (item >= kItems) return;
        const int t0 = quad(item) * 4, o = octet(item);
#pragma unroll
        for (int n = 0; n < kPlanes<T>; ++n) {
            uint32_t x[4][4];
            plane(n, x);
            if (by_row) {
                uint8_t* lds = by_row + n * RowTile<KP>::kBytes;
                // columns 8 o .. 8 o + 7 of 32 are two quads: slots of groups g and g + 1, lower or upper half
                const int piece = (o / 4) * 4 + (o % 2) * 2, half = (o % 4) / 2 * 8;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    *reinterpret_cast<u32x2*>(lds + RowTile<KP>::at(t0 + t, piece) + half) = u32x2{x[t][0], x[t][1]};
                    *reinterpret_cast<u32x2*>(lds + RowTile<KP>::at(t0 + t, piece + 1) + half) = u32x2{x[t][2], x[t][3]};
                }
            }
            if (by_column) {
                uint8_t* lds = by_column + n * ColumnTile<KP>::kBytes;
                const int q = quad(item), piece = (q / 8) * 4 + q % 4, half = (q % 8) / 4 * 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo01 = __builtin_amdgcn_perm(x[1][i], x[0][i], 0x05040100u),
                                   lo23 = __builtin_amdgcn_perm(x[3][i], x[2][i], 0x05040100u),
                                   hi01 = __builtin_amdgcn_perm(x[1][i], x[0][i], 0x07060302u),
                                   hi23 = __builtin_amdgcn_perm(x[3][i], x[2][i], 0x07060302u);
                    *reinterpret_cast<u32x2*>(lds + ColumnTile<KP>::at(o * 8 + 2 * i, piece) + half) = u32x2{lo01, lo23};
                    *reinterpret_cast<u32x2*>(lds + ColumnTile<KP>::at(o * 8 + 2 * i + 1, piece) + half) = u32x2{hi01, hi23};
                }
            }
        }
    }
};

}  // namespace gdrk
}  // namespace mssm
