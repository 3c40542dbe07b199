// gdr_common.h -- device helpers shared by the gated delta rule's kernels: where a
// sequence's chunks lie, their decays, and a chunk's rows in LDS.
//
// Products as in planes.h.  The order of the slots used throughout is slot (g, j)
// <-> 4 g + j for j < 4 and 16 + 4 g + (j - 4) otherwise ("folded"): two
// accumulators of 16 rows each, one above the other, are then an operand that is
// summed over these rows without any lane having to exchange a value.
#pragma once

#include <hip/hip_runtime.h>

#include "gdr.h"
#include "planes.h"

namespace mssm {
namespace gdrk {

constexpr int kC = kGdrChunk;

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

template <int N>
__device__ __forceinline__ void store_block(uint8_t* mat, int block, int lane, const Planes<N>& x) {
#pragma unroll
    for (int n = 0; n < N; ++n) *reinterpret_cast<u32x4*>(mat + (n * kGdrBlocks + block) * kGdrBlockBytes + lane * 16) = x.p[n];
}
// A block kept in float32, as the rows of two accumulators (as planes it is cut by split).
__device__ __forceinline__ Planes<2> words_of(f32x4 lo, f32x4 hi) {
    return Planes<2>{{__builtin_bit_cast(u32x4, lo), __builtin_bit_cast(u32x4, hi)}};
}
__device__ __forceinline__ Planes<3> split_words(const Planes<2>& w) {
    return split<3>(__builtin_bit_cast(f32x4, w.p[0]), __builtin_bit_cast(f32x4, w.p[1]));
}

// ---- sequences --------------------------------------------------------------

struct Span {
    int64_t start, len;
};
// Tokens are fewer than 2^31; of equal lengths, without a division, `each` is T / N.
__device__ __forceinline__ Span span_of(const int32_t* offsets, int64_t n, int64_t T, int64_t each) {
    if (!offsets) return {n * each, each};
    int64_t s = offsets[n], e = offsets[n + 1];
    s = s < 0 ? 0 : s > T ? T : s;
    e = e < s ? s : e > T ? T : e;
    return {s, e - s};
}
__device__ __forceinline__ int64_t first_slot(const Span& s, int64_t n) { return (s.start >> 6) + n; }
static_assert(kC == 64, "first_slot divides by 64");

// Of pieces of 2^shift tokens, numbered as the chunks are, the sequence of number
// `slot` (if it is one of its pieces).  By a whole wave, 64 sequences at a time: few
// loads behind one another.
__device__ __forceinline__ int64_t sequence_of(const int32_t* offsets, int64_t slot, int64_t T, int64_t N, int64_t each, int shift) {
    const int64_t lane = threadIdx.x & 63;
    int64_t lo = 0, count = N;  // the last of `count` sequences whose first slot is not behind this one
    while (count > 1) {
        const int64_t step = (count + 63) >> 6, n = lo + lane * step;
        int64_t s = 0;
        if (lane * step < count) s = offsets ? imin64(T, offsets[n] < 0 ? 0 : offsets[n]) : n * each;
        const int before = __builtin_popcountll(__ballot(lane * step < count && (s >> shift) + n <= slot));
        const int64_t at = (before > 1 ? before - 1 : 0) * step;
        lo += at;
        count = imin64(step, count - at);
    }
    return lo;
}

// The sequence and chunk of a slot; len = 0: the slot is no chunk.
struct Chunk {
    int64_t seq, start;  // its first token
    int len;             // tokens, up to 64
};
__device__ __forceinline__ Chunk chunk_of(const int32_t* offsets, int64_t slot, int64_t T, int64_t N, int64_t each) {
    const int64_t n = sequence_of(offsets, slot, T, N, each, 6);
    const Span s = span_of(offsets, n, T, each);
    const int64_t t = (slot - first_slot(s, n)) * kC;
    if (t < 0 || t >= s.len) return {n, 0, 0};
    return {n, s.start + t, static_cast<int>(imin64(kC, s.len - t))};
}

// What a chain goes through: a whole sequence, or one of its pieces of 2^shift tokens.
struct Piece {
    int64_t seq, start, len, slot0;  // slot0: of its first chunk
    bool first, last, none;          // none: not a piece (a sequence of no tokens has an empty one)
};
__device__ __forceinline__ Piece whole_of(const int32_t* offsets, int64_t n, int64_t T, int64_t each) {
    const Span s = span_of(offsets, n, T, each);
    return {n, s.start, s.len, first_slot(s, n), true, true, false};
}
__device__ __forceinline__ Piece piece_of(const int32_t* offsets, int64_t i, int64_t T, int64_t N, int64_t each, int shift) {
    const int64_t n = sequence_of(offsets, i, T, N, each, shift);
    const Span s = span_of(offsets, n, T, each);
    const int64_t t = (i - ((s.start >> shift) + n)) << shift;
    if (t < 0 || (t > 0 && t >= s.len)) return {n, 0, 0, 0, false, false, true};
    const int64_t len = imin64(int64_t{1} << shift, s.len - t);
    return {n, s.start + t, len, first_slot(s, n) + (t >> 6), t == 0, t + len == s.len, false};
}

// The parts of a head's value elements read the same rows and matrices: on the same
// XCD, which has its own L2.  Workgroups go to the 8 XCDs in turn, so of every 8 P
// of them the x-th of each eight is a part of the x-th head; grids are whole eights
// of heads.  (Heads next to each other stay on different XCDs: they are as long as
// their sequence.)
constexpr uint32_t kXcds = 8;
__host__ __device__ __forceinline__ uint32_t xcd_grid(int64_t heads, int64_t parts) {
    return static_cast<uint32_t>((heads + kXcds - 1) / kXcds * kXcds * parts);
}
struct HeadPart {
    uint32_t head, part;
};
__device__ __forceinline__ HeadPart head_part(uint32_t parts) {
    const uint32_t eight = blockIdx.x / kXcds, group = eight / parts;
    return {group * kXcds + blockIdx.x % kXcds, eight - group * parts};
}

// ---- elements of rows ---------------------------------------------------------

// Memory from `base` on (the same for all lanes), read by element number; what is
// not `in` reads as zeros.  By an offset outside of the buffer's range, not by a
// branch: behind a branch around a load the compiler waits for it.
template <typename T>
struct View {
    static constexpr uint32_t kOut = 0x7fffffffu, kBytes = 0x7ffffff0u;
    __amdgpu_buffer_rsrc_t rsrc;
    __device__ __forceinline__ explicit View(const T* base) : rsrc(make_rsrc(uniform_ptr(base), kBytes)) {}
    __device__ __forceinline__ static uint32_t offset(uint32_t at, bool in) { return in ? at * static_cast<uint32_t>(sizeof(T)) : kOut - 15; }
    __device__ __forceinline__ u32x4 words4(uint32_t at, bool in) const {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, offset(at, in), 0, 0));
    }
    __device__ __forceinline__ u32x2 words2(uint32_t at, bool in) const {
        return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rsrc, offset(at, in), 0, 0));
    }
    __device__ __forceinline__ float one(uint32_t at, bool in) const {
        if constexpr (sizeof(T) == 2) return __uint_as_float(static_cast<uint32_t>(static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rsrc, offset(at, in), 0, 0))) << 16);
        else return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsrc, offset(at, in), 0, 0));
    }
    __device__ __forceinline__ f32x4 four(uint32_t at, bool in) const {
        if constexpr (sizeof(T) == 2) {
            const u32x2 a = words2(at, in);
            return f32x4{bf16_lo(a[0]), bf16_hi(a[0]), bf16_lo(a[1]), bf16_hi(a[1])};
        } else {
            return __builtin_bit_cast(f32x4, words4(at, in));
        }
    }
    // eight neighbours as an operand
    __device__ __forceinline__ Planes<kPlanes<T>> planes(uint32_t at, bool in) const {
        if constexpr (sizeof(T) == 2) return Planes<1>{{words4(at, in)}};
        else return split<3>(four(at, in), four(at + 4, in));
    }
};

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

// Sixteen tokens of sixteen value elements: from four tokens (4 g + r) of element c a
// lane, as the accumulators have them, to four elements (4 (c / 4) + r) of token
// 4 g + c % 4, as they lie in memory: one 16-byte store instead of four of 4 bytes.
__device__ __forceinline__ f32x4 quad_transpose(f32x4 x, int c) {
    const bool odd = c & 1, upper = c & 2;
    auto swap = [](auto move, bool second, float& a, float& b) {
        const float other = move(second ? a : b);
        a = second ? other : a;
        b = second ? b : other;
    };
    auto by1 = [](float v) { return dpp_move<0xB1>(v); };
    auto by2 = [](float v) { return dpp_move<0x4E>(v); };
    float v[4] = {x[0], x[1], x[2], x[3]};
    swap(by1, odd, v[0], v[1]);
    swap(by1, odd, v[2], v[3]);
    swap(by2, upper, v[0], v[2]);
    swap(by2, upper, v[1], v[3]);
    return f32x4{v[0], v[1], v[2], v[3]};
}

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
// Lane `from`'s value (of the 64, modulo 64).
__device__ __forceinline__ double of_lane(double v, int from) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_ds_bpermute(from * 4, static_cast<int>(b)), hi = __builtin_amdgcn_ds_bpermute(from * 4, static_cast<int>(b >> 32));
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// One wave, a token a lane: the sum of the chunk's log decays up to the lane's token.
__device__ __forceinline__ double decays_since_start(float gl, int lane) {
    double b = gl < kGdrLeast ? kGdrLeast : gl;
#pragma unroll
    for (int d = 1; d < kC; d *= 2) {
        const double o = of_lane(b, lane - d);
        if (lane >= d) b += o;
    }
    return b;
}
// ---- a chunk's rows in LDS --------------------------------------------------------

// R rows (tokens, or value elements) of W columns, as bfloat16 planes.  A row's 16-byte pieces are
// exchanged among themselves by the row's number, so that the 16 rows that a read
// takes at once spread over the banks.  Read as operands by rows (summed over the
// columns) in one 16-byte read, or by columns (summed over the tokens) in two
// transposing reads: sixteen lanes read four rows of 16 values, 8 bytes a lane,
// and each gets a column's four.
template <int W, int R = kC>
struct Tile {
    static constexpr int kRow = W * 2, kBytes = R * kRow, kPieces = W / 8;
    static_assert(kPieces == 8 || kPieces == 16, "rows of 128 or 256 bytes");
    __device__ static __forceinline__ int turn(int row) { return kPieces == 16 ? row & 15 : (row >> 1) & 7; }
    __device__ static __forceinline__ int at(int row, int piece) { return row * kRow + ((piece ^ turn(row)) * 16); }

    // columns 32 s .. of row 16 rt + c, slots in their own order (state_column below has the accumulators' rows for it)
    template <int N>
    __device__ static __forceinline__ Planes<N> rows(const uint8_t* lds, int rt, int s, int c, int g) {
        Planes<N> out;
#pragma unroll
        for (int n = 0; n < N; ++n) out.p[n] = *reinterpret_cast<const u32x4*>(lds + n * kBytes + at(16 * rt + c, 4 * s + g));
        return out;
    }
    // four rows 16 rt + 4 g .. of the column at a byte offset that this lane helps to read
    __device__ static __forceinline__ u32x2 four(const uint8_t* lds, int rt, int piece, int byte, int c, int g) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        const uint8_t* p = lds + at(16 * rt + 4 * g + (c >> 2), piece) + byte;
        return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            reinterpret_cast<__attribute__((address_space(3))) s16x4*>(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)))));
    }
    // ... of column 16 m + c
    __device__ static __forceinline__ u32x2 four(const uint8_t* lds, int rt, int m, int c, int g) {
        return four(lds, rt, 2 * m + ((c >> 1) & 1), (c & 1) * 8, c, g);
    }
    // rows 32 s .. of column state_column(m, c), folded
    template <int N>
    __device__ static __forceinline__ Planes<N> columns(const uint8_t* lds, int m, int s, int c, int g) {
        Planes<N> out;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint8_t* p = lds + n * kBytes;
            const u32x2 a = four(p, 2 * s, 4 * (m >> 1) + (c & 3), (m & 1) * 8, c, g),
                        b = four(p, 2 * s + 1, 4 * (m >> 1) + (c & 3), (m & 1) * 8, c, g);
            out.p[n] = u32x4{a[0], a[1], b[0], b[1]};
        }
        return out;
    }
};

// The key element of row i of tile m of a state's accumulators: tiles 2 s and 2 s + 1
// together are an operand whose slot (g, j) is element 32 s + 8 g + j, which is how
// 16 bytes of a row of q or k lie.
__device__ __forceinline__ constexpr int state_column(int m, int i) { return 32 * (m >> 1) + 8 * (i >> 2) + 4 * (m & 1) + (i & 3); }

// The lower half of a pointer to LDS is its offset there.
__device__ __forceinline__ uint32_t lds_offset(const uint8_t* p) {
    return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)));
}

// bfloat16 rows from memory straight to a tile, by NW waves; rows from a chunk's
// length on and columns from `width` on become zeros.  What does not change from
// chunk to chunk is computed once: a chunk's loads cost a few instructions each.
template <int W, int NW>
struct RowsToLds {
    static constexpr int kPieces = Tile<W>::kPieces, kRows = 64 / kPieces, kLoads = kC / kRows / NW;  // rows of a load
    uint32_t at[kLoads];  // byte offsets of the lane's pieces
    int row[kLoads];
    __device__ __forceinline__ RowsToLds(uint32_t stride, int width, int w, int lane) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            row[i] = (i * NW + w) * kRows + lane / kPieces;
            const int piece = lane % kPieces ^ Tile<W>::turn(row[i]);
            at[i] = piece * 8 < width ? (row[i] * stride + piece * 8) * 2 : 0x7ffffffeu;
        }
    }
    __device__ __forceinline__ void load(uint32_t lds, const uint16_t* rows, int len, int w) const {
        const i32x4 rsrc = buffer_words(rows, 0x7ffffff0u);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_to_lds(lds + (i * NW + w) * kRows * Tile<W>::kRow, rsrc, row[i] < len ? at[i] : 0x7ffffffeu, 0);
    }
};
// `bytes` (a multiple of 16) from memory straight to LDS, by NW waves.
template <int NW, int bytes>
__device__ __forceinline__ void bytes_to_lds(uint32_t lds, const uint8_t* from, int w, int lane) {
    const i32x4 rsrc = buffer_words(from, bytes);  // each load ends within
#pragma unroll
    for (int i = 0; i < (bytes + 1024 * NW - 1) / (1024 * NW); ++i) {
        const int at = (i * NW + w) * 1024;
        if (at + 1024 <= bytes) load_to_lds(lds + at, rsrc, lane * 16, at);
        else if (at + lane * 16 < bytes) load_to_lds(lds + at, rsrc, lane * 16, at);  // the lanes of the last piece
    }
}
// Waits until at most N of the wave's loads and stores, the last ones, are under way.
template <int N>
__device__ __forceinline__ void wait_memory() { asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory"); }

// float32 rows on their way to a tile's planes: a thread's pieces, held from the loads' issue to the stores.
template <int W, int THREADS>
struct FloatRows {
    static constexpr int kItems = kC * (W / 8) / THREADS;
    f32x4 lo[kItems], hi[kItems];
    __device__ __forceinline__ void load(const float* rows, uint32_t stride, int len, int width, int tid) {
        const View<float> view(rows);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int item = i * THREADS + tid, row = item / (W / 8), piece = item % (W / 8);
            const bool in = row < len && piece * 8 < width;
            lo[i] = view.four(row * stride + piece * 8, in);
            hi[i] = view.four(row * stride + piece * 8 + 4, in);
        }
    }
    __device__ __forceinline__ void store(uint8_t* lds, int tid) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int item = i * THREADS + tid, row = item / (W / 8), piece = item % (W / 8);
            const Planes<3> p = split<3>(lo[i], hi[i]);
#pragma unroll
            for (int n = 0; n < 3; ++n) *reinterpret_cast<u32x4*>(lds + n * Tile<W>::kBytes + Tile<W>::at(row, piece)) = p.p[n];
        }
    }
};

}  // namespace gdrk
}  // namespace mssm
