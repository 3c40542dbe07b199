// gdr_fwd.hip -- the chain of the gated delta rule over a sequence's chunks
// (mssm_gdr_fwd, mssm_gdr_fwd_train; the equations are in gdr_prep.hip).
//
// The columns of the state's transpose (K x V), one for each value element, do
// not depend on one another, so each wave takes 16 of them through the whole
// sequence by itself: the state stays in its accumulators, and every
// product of the chain takes its float32 operand straight from the accumulators
// of the one before.  The other operands, q, k and the chunk's matrices, are
// shared by the waves of a workgroup.
//
// Measured, key and value dim 128, bfloat16: 4 sequences of 4,096 tokens, 40 heads,
// 390 us, 6.1 us a chunk (matrix instructions busy for 50 % of the time on the
// compute units in use, vector instructions for 51 %); 16 columns a workgroup, 1.8 us
// a chunk.  For the backward the states and e are written too, 96 KB a chunk and
// head: 8,192 packed tokens of 32 heads 378 us, 681 MB at 1.8 TB/s, the longest
// sequences alone at the end.  float32, 64 and 64: 6.8 us a chunk, 4 waves a compute unit.
#include "gdr_common.h"

namespace mssm {
namespace {

using namespace gdrk;

struct FwdArgs {
    const void *q, *k, *v;
    const int32_t* offsets;
    const uint8_t* mats;
    const float* h0;
    void* y;
    float* h_final;
    float* states;
    float* misses;
    int64_t T, N, each, G, H, K, V, parts;
    int64_t mat_bytes, at_n, at_p, at_f;
    int64_t pieces;
    int shift;
    float* starts;
    float* moves;
};

enum Form { kForward, kTrain, kEnds };

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// NW waves with a tile of 16 columns each.  While a chunk is worked on, the next
// one's rows and matrices come in: bfloat16 straight into the other half of LDS,
// float32 through registers, where it is cut into planes.  So is P, once by the whole
// workgroup, and lies in LDS once: it is written behind the barrier that ends the chunk
// before, and is there behind the next one.
// kEnds: only the state behind a piece, and what the piece makes of any row of a state:
// a second tile of each wave starts with unit rows (one for each key element) and sees
// values of zero.
// Whole sequences are a form of their own: with both in one, 8,192 packed tokens of 32
// heads with what the backward needs took a tenth longer.
template <typename T, int KP, int NW, int FORM, bool PIECES>
__global__ __launch_bounds__(NW * 64, NW / 4) void gdr_fwd_kernel(FwdArgs a) {
    constexpr bool B16 = sizeof(T) == 2, TRAIN = FORM == kTrain, ENDS = FORM == kEnds;
    constexpr int PL = kPlanes<T>, KS = KP / 32, KM = KP / 16, VC = NW * 16, CT = ENDS ? 2 : 1;
    typedef Tile<KP> Keys;
    typedef Tile<VC> Values;
    constexpr int kN = 3 * kGdrBlocks * kGdrBlockBytes, kF = kGdrFactors * kC * 4, kMats = kN + kF;
    constexpr int kOwn = (kGdrBlocks + NW - 1) / NW;  // blocks of P that a wave cuts
    constexpr int kKeys = (ENDS ? 1 : 2) * PL * Keys::kBytes;
    constexpr int kPart = B16 ? kKeys + Values::kBytes + kMats : kMats;  // of what LDS holds twice
    __shared__ __align__(16) uint8_t lds[2 * kPart + (B16 ? 0 : kKeys) + (ENDS ? 0 : kN)];
    static_assert(sizeof(lds) <= 160 * 1024, "LDS of a compute unit");
    uint8_t* lds_p = lds + 2 * kPart + (B16 ? 0 : kKeys);
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const HeadPart at = head_part(static_cast<uint32_t>(a.parts));
    if (at.head >= a.pieces * a.H) return;
    const int64_t part = at.part, piece = at.head / static_cast<uint32_t>(a.H), h = at.head - piece * a.H;
    const int64_t hg = h / (a.H / a.G);
    const int64_t vw = part * VC, v0 = vw + w * 16;  // the workgroup's first value element, and the wave's
    const Piece sp = PIECES ? piece_of(a.offsets, piece, a.T, a.N, a.each, a.shift) : whole_of(a.offsets, piece, a.T, a.each);
    if (sp.none || (ENDS && sp.last)) return;
    const int64_t n = sp.seq, slot0 = sp.slot0, chunks = (sp.len + kC - 1) / kC;
    const int K = static_cast<int>(a.K);
    const bool of_v = v0 < a.V, in_v = of_v || (ENDS && v0 < K);  // V and K are multiples of 16

    f32x4 S[CT][KM];
    const bool initial = !PIECES || gdr_reads_h0(ENDS, sp.first, sp.last);
    const float* start = initial ? a.h0 : ENDS ? nullptr : a.starts;
#pragma unroll
    for (int m = 0; m < KM; ++m) {
        const int col = state_column(m, 4 * g);
        S[0][m] = f32x4{0, 0, 0, 0};
        if (start && of_v && col < K)
            S[0][m] = *reinterpret_cast<const f32x4*>(start + (((initial ? n : piece) * a.H + h) * a.V + v0 + c) * a.K + col);
        if constexpr (ENDS) {
            if (initial && of_v && col < K)  // for the launch that may write h_final there
                *reinterpret_cast<f32x4*>(a.starts + ((piece * a.H + h) * a.V + v0 + c) * a.K + col) = S[0][m];
#pragma unroll
            for (int r = 0; r < 4; ++r) S[1][m][r] = col + r == v0 + c ? 1.0f : 0.0f;
        }
    }

    const int64_t qk_stride = a.G * a.K, v_stride = a.H * a.V;
    const T* kp = static_cast<const T*>(a.k) + sp.start * qk_stride + hg * a.K;
    const T* qp = static_cast<const T*>(a.q) + sp.start * qk_stride + hg * a.K;
    const T* vp = static_cast<const T*>(a.v) + sp.start * v_stride + h * a.V;
    T* yp = static_cast<T*>(a.y) + sp.start * v_stride + h * a.V + v0 + 4 * g;
    auto length = [&](int64_t chunk) { return static_cast<int>(imin64(kC, sp.len - chunk * kC)); };
    auto mats_of = [&](int64_t chunk) { return a.mats + ((slot0 + chunk) * a.H + h) * a.mat_bytes; };
    const RowsToLds<KP, NW> key_loads(static_cast<uint32_t>(qk_stride), K, w, lane);
    const RowsToLds<VC, NW> value_loads(static_cast<uint32_t>(v_stride), static_cast<int>(a.V - vw), w, lane);
    FloatRows<KP, NW * 64> fk, fq;
    Planes<2> pw[kOwn];
    // In four parts: a compute unit takes 1 KB into LDS in about 30 cycles, the 67 KB
    // of a bfloat16 chunk in 2,000, for which its waves would otherwise wait at once.
    constexpr int kParts = 4;
    auto fetch = [&](int64_t chunk, int half, int part) {
        const int len = length(chunk);
        uint8_t* to = lds + half * kPart;
        if (part == 0 && !ENDS) {
            const View<float> words(reinterpret_cast<const float*>(mats_of(chunk) + a.at_p));
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    pw[i].p[p] = words.words4((p * kGdrBlocks + i * NW + w) * 256 + lane * 4, i * NW + w < kGdrBlocks);
        }
        if constexpr (B16) {
            if (part == 0) bytes_to_lds<NW, kMats>(lds_offset(to) + kKeys + Values::kBytes, mats_of(chunk) + a.at_n, w, lane);
            if (part == 1) key_loads.load(lds_offset(to), kp + chunk * kC * qk_stride, len, w);
            if (part == 2 && !ENDS) key_loads.load(lds_offset(to) + Keys::kBytes, qp + chunk * kC * qk_stride, len, w);
            if (part == 3) value_loads.load(lds_offset(to) + kKeys, vp + vw + chunk * kC * v_stride, len, w);
        } else {
            if (part == 0) bytes_to_lds<NW, kMats>(lds_offset(to), mats_of(chunk) + a.at_n, w, lane);
            if (part == 1) fk.load(kp + chunk * kC * qk_stride, static_cast<uint32_t>(qk_stride), len, K, tid);
            if (part == 2 && !ENDS) fq.load(qp + chunk * kC * qk_stride, static_cast<uint32_t>(qk_stride), len, K, tid);
        }
    };
    f32x4 O[4];
    auto put_y = [&](int64_t chunk) {  // row 4 g + r: value elements; column c of tile rt: token 16 rt + c
        if (ENDS || !a.y || !in_v) return;
        const int len = length(chunk);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const float out[4] = {O[rt][0], O[rt][1], O[rt][2], O[rt][3]};
            if (16 * rt + c < len) store_row(yp + (chunk * kC + 16 * rt + c) * v_stride, out);
        }
    };
    if (chunks) {
#pragma unroll
        for (int q = 0; q < kParts; ++q) fetch(0, 0, q);
    }
    for (int64_t chunk = 0; chunk < chunks; ++chunk) {
        const int half = static_cast<int>(chunk & 1), len = length(chunk);
        const uint8_t* in = lds + half * kPart;
        const uint8_t *lds_k = B16 ? in : lds + 2 * kPart, *lds_q = lds_k + PL * Keys::kBytes, *lds_v = in + kKeys;
        const uint8_t* lds_n = B16 ? in + kKeys + Values::kBytes : in;
        const float* f = reinterpret_cast<const float*>(lds_n + kN);
        tile_barrier();  // this half is whole, nobody reads the other one, nor P
        if constexpr (!ENDS) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
                if (i * NW + w < kGdrBlocks) store_block(lds_p, i * NW + w, lane, split_words(pw[i]));
        }
        if constexpr (!B16) {
            fk.store(lds + 2 * kPart, tid);
            if constexpr (!ENDS) fq.store(lds + 2 * kPart + PL * Keys::kBytes, tid);
            __syncthreads();
        }
        if (chunk) put_y(chunk - 1);  // here, not when it was ready: the barrier waits for stores too
        const bool more = chunk + 1 < chunks;
        if (!in_v) {
            if constexpr (B16 && !ENDS) lds_barrier();  // as below
#pragma unroll
            for (int q = 0; q < kParts; ++q)
                if (more) fetch(chunk + 1, half ^ 1, q);
            continue;
        }

        int c = lane & 15, g = lane >> 4;
        if constexpr (ENDS) asm volatile("" : "+v"(c), "+v"(g));  // addresses are computed here, not kept (and spilled)
        f32x4 val[4];  // item r of tile rt: token 16 rt + 4 g + r of this lane's column
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            if constexpr (B16) {
                const u32x2 x = Values::four(lds_v, rt, w, c, g);
                val[rt] = f32x4{bf16_lo(x[0]), bf16_hi(x[0]), bf16_lo(x[1]), bf16_hi(x[1])};
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * rt + 4 * g + r;
                    val[rt][r] = View<T>(vp + chunk * kC * v_stride).one(t * static_cast<uint32_t>(v_stride) + static_cast<uint32_t>(v0) + c, t < len && of_v);
                }
            }
        }
        if constexpr (TRAIN) {
            float* to = a.states + (((slot0 + chunk) * a.H + h) * a.V + v0 + c) * a.K;
#pragma unroll
            for (int m = 0; m < KM; ++m)
                if (state_column(m, 4 * g) < K) *reinterpret_cast<f32x4*>(to + state_column(m, 4 * g)) = S[0][m];
        }
        // S k (tokens in the rows) and S q (tokens in the columns)
        f32x4 X[CT][4] = {};
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) O[rt] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            Planes<3> st[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) st[j] = split<3>(S[j][2 * s], S[j][2 * s + 1]);
            Planes<PL> kf[4], qf[4];
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                kf[rt] = Keys::template rows<PL>(lds_k, rt, s, c, g);
                if constexpr (!ENDS) qf[rt] = Keys::template rows<PL>(lds_q, rt, s, c, g);
            }
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
#pragma unroll
                for (int j = 0; j < CT; ++j) X[j][rt] = mma(kf[rt], st[j], X[j][rt]);
#pragma unroll
            for (int rt = 0; rt < 4 && !ENDS; ++rt) O[rt] = mma(st[0], qf[rt], O[rt]);
            if (more) {
#pragma unroll
                for (int q = s * kParts / KS; q < (s + 1) * kParts / KS; ++q) fetch(chunk + 1, half ^ 1, q);
            }
        }
        if constexpr (B16 && !ENDS) lds_barrier();  // P is there
        // e = r + N (beta r) with r = v - exp(b) S k
        f32x4 beta[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 ek = *reinterpret_cast<const f32x4*>(f + 16 * rt + 4 * g);
            beta[rt] = *reinterpret_cast<const f32x4*>(f + kC + 16 * rt + 4 * g);
            X[0][rt] = val[rt] - ek * X[0][rt];
            if constexpr (ENDS) X[1][rt] = -ek * X[1][rt];
        }
        Planes<3> mx[CT][2];
        auto cut = [&](int s) {
#pragma unroll
            for (int j = 0; j < CT; ++j) mx[j][s] = split<3>(beta[2 * s] * X[j][2 * s], beta[2 * s + 1] * X[j][2 * s + 1]);
        };
        if constexpr (!ENDS) cut(0), cut(1);  // two tiles' operands at once would not fit the registers
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int s = ENDS ? 1 - i : i;   // the later rows first: that leaves the earlier ones as they are
            if constexpr (ENDS) {
                __builtin_amdgcn_sched_barrier(0);
                cut(s);
            }
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
                if (block_of<true>(rt, s) >= 0) {
                    const Planes<3> nb = load_block<3>(lds_n, block_of<true>(rt, s), lane);
#pragma unroll
                    for (int j = 0; j < CT; ++j) X[j][rt] = mma(nb, mx[j][s], X[j][rt]);
                }
        }
        if constexpr (TRAIN) {
            float* e = a.misses + ((slot0 + chunk) * a.H + h) * kC * a.V + (4 * g + (c & 3)) * a.V + v0 + (c & ~3);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) *reinterpret_cast<f32x4*>(e + 16 * rt * a.V) = quad_transpose(X[0][rt], c);
        }
        // u; y = scale exp(b) S q + P u, and the state's update
        const float last = f[4 * kC];
        Planes<3> ud[CT][2];
        auto cut_u = [&](int s) {
            const f32x4 d0 = *reinterpret_cast<const f32x4*>(f + 2 * kC + 32 * s + 4 * g),
                        d1 = *reinterpret_cast<const f32x4*>(f + 2 * kC + 32 * s + 16 + 4 * g);
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                X[j][2 * s] *= beta[2 * s];
                X[j][2 * s + 1] *= beta[2 * s + 1];
                ud[j][s] = split<3>(d0 * X[j][2 * s], d1 * X[j][2 * s + 1]);
            }
        };
        if constexpr (!ENDS) cut_u(0), cut_u(1);
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int i = 0; i < KM; ++i) S[j][i] *= last;
#pragma unroll
        for (int rt = 0; rt < 4 && !ENDS; ++rt) O[rt] *= f[3 * kC + 16 * rt + c];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if constexpr (ENDS) {
                __builtin_amdgcn_sched_barrier(0);
                cut_u(s);
            }
#pragma unroll
            for (int m = 0; m < KM; ++m) {
                const Planes<PL> kt = Keys::template columns<PL>(lds_k, m, s, c, g);
#pragma unroll
                for (int j = 0; j < CT; ++j) S[j][m] = mma(kt, ud[j][s], S[j][m]);
            }
        }
#pragma unroll
        for (int s = 0; s < 2 && !ENDS; ++s) {
            const Planes<3> u = split<3>(X[0][2 * s], X[0][2 * s + 1]);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
                if (block_of<true>(rt, s) >= 0)
                    O[rt] = mma(u, load_block<3>(lds_p, block_of<true>(rt, s), lane), O[rt]);
        }
    }
    if constexpr (ENDS) {
        float* end = a.starts + (((piece + 1) * a.H + h) * a.V + v0 + c) * a.K;
        float* move = a.moves + (piece * a.H + h) * a.K * a.K + v0 + c;
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            const int col = state_column(m, 4 * g);
            if (col < K && of_v) *reinterpret_cast<f32x4*>(end + col) = S[0][m];
            if (col < K && v0 < K && !sp.first) {
#pragma unroll
                for (int r = 0; r < 4; ++r) move[(col + r) * a.K] = S[1][m][r];
            }
        }
        return;
    }
    if (chunks) put_y(chunks - 1);
    if (a.h_final && in_v && gdr_writes_h_final(ENDS, sp.last)) {
#pragma unroll
        for (int m = 0; m < KM; ++m)
            if (state_column(m, 4 * g) < K)
                *reinterpret_cast<f32x4*>(a.h_final + ((n * a.H + h) * a.V + v0 + c) * a.K + state_column(m, 4 * g)) = S[0][m];
    }
}

// The states before a sequence's pieces, one behind the other, from the states behind
// them (each from zeros, in the next one's place) and their moves:
//     start' = end + start move,   rows of 16 value elements a workgroup.
// Wave w has a quarter of the key elements, and the rows go round through LDS.
template <int KP>
__global__ __launch_bounds__(256) void gdr_join_kernel(FwdArgs a) {
    constexpr int KS = KP / 32, MT = KP / 64, ROW = KP + 4;
    __shared__ __align__(16) float rows[16 * ROW];
    const int lane = threadIdx.x & 63, w = wave_id(), c = lane & 15, g = lane >> 4, K = static_cast<int>(a.K);
    const HeadPart at = head_part(static_cast<uint32_t>(a.parts));  // a head's moves are read by all its workgroups
    if (at.head >= a.N * a.H) return;
    const int64_t v0 = at.part * 16, n = at.head / static_cast<uint32_t>(a.H), h = at.head - n * a.H;
    const Span s = span_of(a.offsets, n, a.T, a.each);
    const int64_t first = (s.start >> a.shift) + n, count = (s.len + (int64_t{1} << a.shift) - 1) >> a.shift;
    auto state = [&](int64_t piece, int m) { return a.starts + ((piece * a.H + h) * a.V + v0 + c) * a.K + 16 * m + 4 * g; };
    f32x4 move[2][MT][KS][2], end[2][MT];
    auto fetch = [&](int64_t piece, f32x4(&mv)[MT][KS][2], f32x4(&to)[MT]) {  // a piece's move, and the end that it adds to
        const View<float> from(a.moves + (piece * a.H + h) * a.K * a.K);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int m = MT * w + i;
            to[i] = 16 * m < K ? *reinterpret_cast<const f32x4*>(state(piece + 1, m)) : f32x4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < KS; ++q)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const int j = 32 * q + 8 * g + 4 * p;
                    mv[i][q][p] = from.four((16 * m + c) * K + j, 16 * m < K && j < K);
                }
        }
    };
    auto keep = [&](const f32x4(&x)[MT]) {
#pragma unroll
        for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(rows + c * ROW + 16 * (MT * w + i) + 4 * g) = x[i];
    };
    auto step = [&](int64_t piece, const f32x4(&mv)[MT][KS][2], f32x4(&to)[MT]) {
        Planes<3> in[KS];
#pragma unroll
        for (int q = 0; q < KS; ++q) {
            const float* p = rows + c * ROW + 32 * q + 8 * g;
            in[q] = split<3>(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4));
        }
        __syncthreads();  // the rows are read
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int q = 0; q < KS; ++q) to[i] = mma(split<3>(mv[i][q][0], mv[i][q][1]), in[q], to[i]);
        // the compiler leaves a wait state too few before the result is stored
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_nop 7" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MT; ++i)
            if (16 * (MT * w + i) < K) *reinterpret_cast<f32x4*>(state(piece + 1, MT * w + i)) = to[i];
        keep(to);
        __syncthreads();
    };
    if (count < 3) return;  // the second piece starts with the first one's end
    f32x4 x[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = MT * w + i;
        x[i] = 16 * m < K ? *reinterpret_cast<const f32x4*>(state(first + 1, m)) : f32x4{0, 0, 0, 0};
    }
    fetch(first + 1, move[0], end[0]);
    keep(x);
    __syncthreads();
    for (int64_t p = 1; p + 1 < count; p += 2) {
        if (p + 2 < count) fetch(first + p + 1, move[1], end[1]);
        step(first + p, move[0], end[0]);
        if (p + 2 >= count) break;
        if (p + 3 < count) fetch(first + p + 2, move[0], end[0]);
        step(first + p + 1, move[1], end[1]);
    }
}

// The rows of tile rt as half of an operand summed over the tokens, in planes.
template <int N>
__device__ __forceinline__ void put_half(uint8_t* area, int rt, f32x4 x, int lane) {
    uint8_t* to = area + (rt >> 1) * N * 1024 + lane * 16 + (rt & 1) * 8;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        *reinterpret_cast<u32x2*>(to + n * 1024) = u32x2{upper_halves(x[0], x[1]), upper_halves(x[2], x[3])};
        if (n + 1 < N) {
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] -= upper_part(x[r]);
        }
    }
}

// ---- few columns: the waves of a workgroup share a tile of 16 ------------------------

// One tile of 16 columns a workgroup, bfloat16.  What the next chunk waits for is
// cut over KS waves: each has 32 key elements of the state, multiplies its part of
// S k, and after an exchange through LDS has a part of the rows of e and u.  Four
// other waves fetch the chunks and compute y.  A compute unit takes 1 KB into LDS
// in about 30 cycles, 65 KB a chunk in 2,000, which would hold up every other
// access to memory and each barrier behind it: a fourth of a chunk's loads is
// issued between each two barriers, in the order in which they are needed.
template <int KP, bool TRAIN>
__global__ __launch_bounds__(64 * (KP / 32 + 4)) void gdr_fwd_narrow_kernel(FwdArgs a) {
    constexpr int KS = KP / 32, RPW = 4 / KS;  // RPW: row tiles of a chain wave
    typedef Tile<KP> Keys;
    constexpr int kPm = 2 * kGdrBlocks * kGdrBlockBytes, kN = 3 * kGdrBlocks * kGdrBlockBytes, kF = kGdrFactors * kC * 4;
    constexpr int kV = kC * 32, kPart = 2 * Keys::kBytes + kN + kF + kV;
    constexpr int kX = KS * (4 - RPW) * 1024, kS = KS * 3 * 1024, kM = 2 * 3 * 1024;
    constexpr int kU = 2 * (3 + 3) * 1024, kXU = kX > kU ? kX : kU;  // u lies where the sums were
    __shared__ __align__(16) uint8_t lds[2 * kPart + kXU + kS + kM + kPm];
    static_assert(sizeof(lds) <= 160 * 1024, "LDS of a compute unit");
    uint8_t *s_x = lds + 2 * kPart, *s_ud = s_x, *s_u = s_ud + 2 * 3 * 1024, *s_s = s_x + kXU, *s_m = s_s + kS, *lds_p = s_m + kM;
    const int lane = threadIdx.x & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const HeadPart at = head_part(static_cast<uint32_t>(a.parts));
    if (at.head >= a.N * a.H) return;
    const int64_t part = at.part, n = at.head / static_cast<uint32_t>(a.H), h = at.head - n * a.H;
    const int64_t hg = h / (a.H / a.G), v0 = part * 16;
    const Span sp = span_of(a.offsets, n, a.T, a.each);
    const int64_t slot0 = first_slot(sp, n), chunks = (sp.len + kC - 1) / kC;
    const int K = static_cast<int>(a.K);
    const int64_t qk_stride = a.G * a.K, v_stride = a.H * a.V;
    auto length = [&](int64_t chunk) { return static_cast<int>(imin64(kC, sp.len - chunk * kC)); };
    auto piece = [&](uint8_t* area, int i) { return reinterpret_cast<u32x4*>(area + i * 1024 + lane * 16); };

    if (w < KS) {
        __builtin_amdgcn_s_setprio(2);
        f32x4 S[2];
        const int64_t state = ((n * a.H + h) * a.V + v0 + c) * a.K;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int col = state_column(2 * w + m, 4 * g);
            S[m] = f32x4{0, 0, 0, 0};
            if (a.h0 && col < K) S[m] = *reinterpret_cast<const f32x4*>(a.h0 + state + col);
        }
        for (int64_t chunk = 0; chunk < chunks; ++chunk) {
            const uint8_t* in = lds + (chunk & 1) * kPart;
            const uint8_t* lds_n = in + 2 * Keys::kBytes;
            const float* f = reinterpret_cast<const float*>(lds_n + kN);
            const uint8_t* lds_v = lds_n + kN + kF;
            const Planes<3> st = split<3>(S[0], S[1]);
            if constexpr (TRAIN) {
                float* to = a.states + (((slot0 + chunk) * a.H + h) * a.V + v0 + c) * a.K;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int col = state_column(2 * w + m, 4 * g);
                    if (col < K) *reinterpret_cast<f32x4*>(to + col) = S[m];
                }
            }
            lds_barrier();  // the chunk is there, and what LDS holds of the one before is read
            f32x4 X[4] = {};
            {
                Planes<1> kf[4];
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) kf[rt] = Keys::template rows<1>(in, rt, w, c, g);
#pragma unroll
                for (int i = 0; i < 3; ++i) *piece(s_s, 3 * w + i) = st.p[i];
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) X[rt] = mma(kf[rt], st, X[rt]);
            }
            // the other waves' rows; a wave's own stay with it
            auto from = [&](int q, int rt) { return piece(s_x, q * (4 - RPW) + (rt < q * RPW ? rt : rt - RPW)); };
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
                if (rt / RPW != w) *reinterpret_cast<f32x4*>(from(w, rt)) = X[rt];
            lds_barrier();
            f32x4 own[RPW], part_x[RPW][KS];
#pragma unroll
            for (int i = 0; i < RPW; ++i) {
                own[i] = w == 0 ? X[i] : w == 1 ? X[RPW + i] : w == 2 ? X[2 * RPW + i & 3] : X[3 * RPW + i & 3];
#pragma unroll
                for (int q = 0; q < KS; ++q) part_x[i][q] = *reinterpret_cast<const f32x4*>(from(q == w ? (q + 1) % KS : q, w * RPW + i));
            }
            __builtin_amdgcn_sched_barrier(0);
            f32x4 ek[RPW], beta[RPW], ed[RPW];
            u32x2 val[RPW];
#pragma unroll
            for (int i = 0; i < RPW; ++i) {
                const int rt = w * RPW + i;
                const float* p = f + 16 * rt + 4 * g;
                ek[i] = *reinterpret_cast<const f32x4*>(p);
                beta[i] = *reinterpret_cast<const f32x4*>(p + kC);
                ed[i] = *reinterpret_cast<const f32x4*>(p + 2 * kC);
                // values: four of the wave's rows, 32 bytes each
                typedef short s16x4 __attribute__((ext_vector_type(4)));
                val[i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    reinterpret_cast<__attribute__((address_space(3))) s16x4*>(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
                        lds_v + (16 * rt + 4 * g + (c >> 2)) * 32 + (c & 3) * 8)))));
            }
            // what the steps behind the exchanges need, on its way during them
            const float last = f[4 * kC];
            Planes<3> nb[RPW][2];
#pragma unroll
            for (int i = 0; i < RPW; ++i)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int rt = w * RPW + i;
                    nb[i][s] = load_block<3>(lds_n, rt < 2 ? rt : 2 * rt - 2 + s, lane);  // s = 1: for the lower rows only
                }
            Planes<1> kt[2][2];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int m = 0; m < 2; ++m) kt[s][m] = Keys::template columns<1>(in, 2 * w + m, s, c, g);
            __builtin_amdgcn_sched_barrier(0);
            f32x4 e[RPW];
#pragma unroll
            for (int i = 0; i < RPW; ++i) {
                const int rt = w * RPW + i;
                f32x4 x = own[i];
#pragma unroll
                for (int q = 0; q < KS; ++q) x += q == w ? f32x4{0, 0, 0, 0} : part_x[i][q];
                e[i] = f32x4{bf16_lo(val[i][0]), bf16_hi(val[i][0]), bf16_lo(val[i][1]), bf16_hi(val[i][1])} - ek[i] * x;
                const f32x4 b = beta[i] * e[i];
                put_half<3>(s_m, rt, b, lane);
            }
            lds_barrier();
            {
                Planes<3> m[2];
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < 3; ++i) m[s].p[i] = *piece(s_m, s * 3 + i);
#pragma unroll
                for (int i = 0; i < RPW; ++i) {
                    const int rt = w * RPW + i;
                    f32x4 more = {0, 0, 0, 0};
                    e[i] = mma(nb[i][0], m[0], e[i]);
                    if (rt >= 2) more = mma(nb[i][1], m[1], more);
                    e[i] += more;
                }
            }
#pragma unroll
            for (int i = 0; i < RPW; ++i) {
                const f32x4 u = beta[i] * e[i];
                put_half<3>(s_ud, w * RPW + i, ed[i] * u, lane);
                put_half<3>(s_u, w * RPW + i, u, lane);
            }
            if constexpr (TRAIN) {
                float* to = a.misses + ((slot0 + chunk) * a.H + h) * kC * a.V + (4 * g + (c & 3)) * a.V + v0 + (c & ~3);
#pragma unroll
                for (int i = 0; i < RPW; ++i) *reinterpret_cast<f32x4*>(to + 16 * (w * RPW + i) * a.V) = quad_transpose(e[i], c);
            }
            lds_barrier();
            Planes<3> ud[2];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 3; ++i) ud[s].p[i] = *piece(s_ud, s * 3 + i);
            f32x4 more[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                more[m] = mma(kt[1][m], ud[1], f32x4{0, 0, 0, 0});
                S[m] = mma(kt[0][m], ud[0], last * S[m]);
            }
            S[0] += more[0];
            S[1] += more[1];
        }
        if (a.h_final) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int col = state_column(2 * w + m, 4 * g);
                if (col < K) *reinterpret_cast<f32x4*>(a.h_final + state + col) = S[m];
            }
        }
    } else {
        const int rt = w - KS;
        const uint16_t* kp = static_cast<const uint16_t*>(a.k) + sp.start * qk_stride + hg * a.K;
        const uint16_t* qp = static_cast<const uint16_t*>(a.q) + sp.start * qk_stride + hg * a.K;
        uint16_t* yp = static_cast<uint16_t*>(a.y) + sp.start * v_stride + h * a.V + v0 + 4 * g;
        const uint16_t* vp = static_cast<const uint16_t*>(a.v) + sp.start * v_stride + h * a.V + v0;
        const RowsToLds<KP, 4> loads(static_cast<uint32_t>(qk_stride), K, rt, lane);
        // Of a chunk the keys come first; the wave's kOthers loads behind them nobody
        // needs before the second barrier.
        constexpr int kKeyLoads = RowsToLds<KP, 4>::kLoads, kOthers = kKeyLoads + (kN + kF + 4095) / 4096 + kPm / 4096;
        auto to_half = [&](int64_t chunk) { return lds_offset(lds + (chunk & 1) * kPart); };
        auto mats = [&](int64_t chunk) { return a.mats + ((slot0 + chunk) * a.H + h) * a.mat_bytes + a.at_p; };
        auto fetch_k = [&](int64_t chunk) { loads.load(to_half(chunk), kp + chunk * kC * qk_stride, length(chunk), rt); };
        auto fetch_n = [&](int64_t chunk) {
            const uint32_t to = to_half(chunk) + 2 * Keys::kBytes;
            if (rt < 2) {  // two lanes a row
                const int row = 32 * rt + lane / 2;
                load_to_lds(to + kN + kF + rt * 1024, buffer_words(vp + chunk * kC * v_stride, 0x7ffffff0u),
                            row < length(chunk) ? (row * static_cast<uint32_t>(v_stride) + lane % 2 * 8) * 2 : 0x7ffffffeu, 0);
            }
            bytes_to_lds<4, kN + kF>(to, mats(chunk) + kPm, rt, lane);
        };
        auto fetch_q = [&](int64_t chunk) { loads.load(to_half(chunk) + Keys::kBytes, qp + chunk * kC * qk_stride, length(chunk), rt); };
        // it lies there once, and is read before the barrier that this comes behind
        auto fetch_p = [&](int64_t chunk) { bytes_to_lds<4, kPm>(lds_offset(lds_p), mats(chunk), rt, lane); };
        auto planes = [&](uint8_t* area, int i) { return Planes<3>{{*piece(area, 3 * i), *piece(area, 3 * i + 1), *piece(area, 3 * i + 2)}}; };
        f32x4 O;
        auto put_y = [&](int64_t chunk) {
            const int t = 16 * rt + c;
            const float out[4] = {O[0], O[1], O[2], O[3]};
            if (a.y && t < length(chunk)) store_row(yp + (chunk * kC + t) * v_stride, out);
        };
        if (chunks) {
            fetch_k(0);
            fetch_q(0);
            fetch_n(0);
            fetch_p(0);
        }
        for (int64_t chunk = 0; chunk < chunks; ++chunk) {
            const uint8_t* in = lds + (chunk & 1) * kPart;
            const uint8_t* lds_q = in + Keys::kBytes;
            const float* f = reinterpret_cast<const float*>(lds_q + Keys::kBytes + kN);
            const bool more = chunk + 1 < chunks;
            wait_memory<kOthers>();
            lds_barrier();
            if (more) {
                fetch_k(chunk + 1);
                wait_memory<kKeyLoads>();
            } else {
                wait_memory<0>();
            }
            lds_barrier();
            if (chunk) put_y(chunk - 1);  // not earlier: the waits above would be for it too
            if (more) fetch_q(chunk + 1);
            Planes<1> qf[KS];
            Planes<2> pb[2];
#pragma unroll
            for (int s = 0; s < KS; ++s) qf[s] = Keys::template rows<1>(lds_q, rt, s, c, g);
#pragma unroll
            for (int s = 0; s < 2; ++s) pb[s] = load_block<2>(lds_p, rt < 2 ? rt : 2 * rt - 2 + s, lane);
            const float eq = f[3 * kC + 16 * rt + c];
            O = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < KS; ++s) O = mma(planes(s_s, s), qf[s], O);
            O *= eq;
            lds_barrier();
            if (more) fetch_n(chunk + 1);
            lds_barrier();
            if (more) fetch_p(chunk + 1);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s && rt < 2) break;
                O = mma(planes(s_u, s), split_words(pb[s]), O);
            }
        }
        if (chunks) put_y(chunks - 1);
    }
}

FwdArgs arguments(const GdrArgs& a, const GdrPieces& p, int64_t parts) {
    const GdrLayout l(a.train);
    return {a.q, a.k, a.v, a.offsets, a.mats, a.h0, a.y, a.h_final, a.states, a.misses,
            a.T, a.N, a.T / a.N, a.G, a.H, a.K, a.V, parts, l.bytes, l.n, l.pm, l.factors, p.count, p.shift, a.starts, a.moves};
}
template <typename T, int KP, int NW, int FORM, bool PIECES>
hipError_t launch_v(const GdrArgs& a, const GdrPieces& p, hipStream_t s) {
    const int64_t parts = ((FORM == kEnds && a.K > a.V ? a.K : a.V) + 16 * NW - 1) / (16 * NW);
    gdr_fwd_kernel<T, KP, NW, FORM, PIECES><<<xcd_grid(p.count * a.H, parts), NW * 64, 0, s>>>(arguments(a, p, parts));
    return hipGetLastError();
}
template <typename T, int KP, int NW>
hipError_t launch_c(const GdrArgs& a, const GdrPieces& p, hipStream_t s) {
    if (p.shift) {
        hipError_t e = launch_v<T, KP, NW, kEnds, true>(a, p, s);
        if (e != hipSuccess) return e;
        gdr_join_kernel<KP><<<xcd_grid(a.N * a.H, a.V / 16), 256, 0, s>>>(arguments(a, p, a.V / 16));
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        return a.train ? launch_v<T, KP, NW, kTrain, true>(a, p, s) : launch_v<T, KP, NW, kForward, true>(a, p, s);
    }
    return a.train ? launch_v<T, KP, NW, kTrain, false>(a, p, s) : launch_v<T, KP, NW, kForward, false>(a, p, s);
}
template <int KP>
hipError_t launch_narrow(const GdrArgs& a, const GdrPieces& p, hipStream_t s) {
    const FwdArgs k = arguments(a, p, a.V / 16);
    const uint32_t blocks = xcd_grid(a.N * a.H, a.V / 16);
    if (a.train) gdr_fwd_narrow_kernel<KP, true><<<blocks, 64 * (KP / 32 + 4), 0, s>>>(k);
    else gdr_fwd_narrow_kernel<KP, false><<<blocks, 64 * (KP / 32 + 4), 0, s>>>(k);
    return hipGetLastError();
}
template <typename T, int KP>
hipError_t launch_k(const GdrArgs& a, hipStream_t s) {
    // A tile of 16 columns a workgroup while there are at most 512 (of key dim up to 64:
    // 256) of them.  1,024 tokens, with the chunks' own pass, us of this form / of the
    // wide one: key and value dim 128, 64 heads (512 tiles) 92 / 100, 96 heads 131 / 107;
    // 128 and 64, 128 heads (512) 102 / 110, 192 heads 149 / 128; dim 64, 64 heads (256)
    // 47 / 75, 96 heads 80 / 82; 64 and 128, 32 heads (256) 47 / 74, 64 heads 76 / 76.
    const GdrPieces p(a.T, a.N, a.H, a.K, a.V, a.dtype);
    if constexpr (sizeof(T) == 2) {
        if (!p.shift && a.N * a.H * (a.V / 16) <= (KP == 128 ? 512 : 256)) return launch_narrow<KP>(a, p, s);
    }
    // Workgroups of 128 columns once those of 64 are more than the 256 compute units; as
    // above, us with 64 / 128 columns: 128 and 128, 128 heads 114 / 130, 160 heads 195 /
    // 142; 128 and 256, 48 heads 97 / 115, 72 heads 178 / 125; float32, 64 and 128, 128
    // heads 123 / 138, 160 heads 230 / 162.  Their eight waves have 256 registers each,
    // too few for the float32 planes of a key dim of 128.
    if constexpr (sizeof(T) == 2 || KP == 64) {
        if (a.V > 64 && p.count * a.H * ((a.V + 63) / 64) > 256) return launch_c<T, KP, 8>(a, p, s);
    }
    return launch_c<T, KP, 4>(a, p, s);
}
template <typename T>
hipError_t launch_t(const GdrArgs& a, hipStream_t s) {
    return a.K <= 64 ? launch_k<T, 64>(a, s) : launch_k<T, 128>(a, s);
}

}  // namespace

// Pieces of 512 tokens or more, so long that their workgroups are at most the 256
// compute units, if a sequence of the mean length (their own are known on the device
// only) then has at least 8 of them (float32: 4).  What they cost is the pass over all
// but the last for their ends and moves, with twice the columns, and the join, 3 us a
// piece.  us in pieces / through whole sequences (bfloat16 by the form for few columns),
// key and value dim 128: bfloat16, 16 heads, 32,768 tokens (16 pieces) 650 / 1,085,
// 8,192 (16) 210 / 285, 32 heads, 16,384 (8) 620 / 618, 4 heads, 4,096 (8) 123 / 140,
// 1 head, 65,536 (128) 479 / 1,917; float32, 16 heads, 2,048 tokens (4) 171 / 269,
// 8,192 (8) 366 / 1,010.
GdrPieces::GdrPieces(int64_t T, int64_t N, int64_t H, int64_t K, int64_t V, int dtype) : count(N) {
    const int64_t columns = V > 64 && (dtype == MSSM_BF16 || K <= 64) ? 128 : 64, least = dtype == MSSM_BF16 ? 8 : 4;
    const int64_t units = N * H * (((K > V ? K : V) + columns - 1) / columns), each = (T + N - 1) / N;
    if (units * least > 256) return;
    int by = 9;
    while ((each + (int64_t{1} << by) - 1) >> by > 256 / units) ++by;
    if ((each + (int64_t{1} << by) - 1) >> by < least) return;
    shift = by;
    count = (T >> shift) + N;
}

hipError_t launch_gdr_fwd(const GdrArgs& a, hipStream_t s) {
    return a.dtype == MSSM_F32 ? launch_t<float>(a, s) : launch_t<uint16_t>(a, s);
}

}  // namespace mssm
