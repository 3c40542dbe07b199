// gdr_bwd.hip -- the gradients of the gated delta rule (mssm_gdr_bwd_saved,
// mssm_gdr_bwd), from what the forward keeps (S before every chunk, e, and the
// matrices N and P with their transposes; gdr_prep.hip has the equations).
//
// With L the adjoint of the state behind a chunk, b_C its whole log decay and
// k, q scaled, D = exp(b_C - b):
//
//     du = Pᵀ dy + D (L k)          Z = du + Nᵀ (beta du)        dr = beta Z = dv
//     L' = exp(b_C) L + sum_t scale exp(b_t) dy_t q_tᵀ - exp(b_t) dr_t k_tᵀ
//
// is the chain, backwards over the chunks and, as the forward's, for every value
// element by itself.  Given L and Z every chunk has its gradients by itself:
//
//     dbeta = e . Z                 dP_ij = dy_i . u_j     M_ij = -G_ij dr_i . u_j  (j < i)
//     dq    = scale exp(b) dy S + (G dP) k
//     dk    = -exp(b) dr S + M k    where a key is read with (its "row" part, decays exp(b))
//           + D u L + (G dP)ᵀ q + Mᵀ k    where it is written with (exp(-b))
//
// and of the decay of token i what passes it: the state to a token from i on or to the
// chunk's end, a token before i to that end, and a token before i to one from i on,
//
//     dg_i  = sum_{t >= i} s_t + exp(b_C) <L, S> + sum_{j < i} w_j + sum_{j < i <= t} c_tj
//     s_t   = q_t . scale exp(b_t) dy_t S - k_t . exp(b_t) dr_t S        w_j = k_j . D_j u_j L
//
// Of the pairs of different tokens, c_tj, row t has r_t = q . dq + k . dk_row - s_t and
// column j l_j = k . dk_column - w_j, and those of (j < i <= t) are sum_{m < i} l_m - r_m:
//
//     dg_i  = sum_{t >= i} s_t + exp(b_C) <L, S> + sum_{m < i} (s - q . dq - k . dk_row + k . dk_column)_m
//
// Nothing is added here and taken away there but what is part of some token's dg (a
// token with itself, dP_ii, comes to dq and dk behind that): strong decays, which make
// all of it small, cost no accuracy, and where no state goes in (S = 0) the first
// token's is 0.
//
// Measured: 8,192 packed tokens, 32 heads of 128 x 128, bfloat16: the chain 370 us,
// the chunks' gradients 503 us (628 MB, 1.2 TB/s; vector instructions busy for 45 %,
// matrix instructions for 21 %); 16,384 tokens, 24 heads of 64 x 64, float32: 342 and
// 464 us.
#include "gdr_common.h"

namespace mssm {
namespace {

using namespace gdrk;

struct AdjointArgs {
    const void *q, *k, *dy;
    const int32_t* offsets;
    const uint8_t* mats;
    const float* dh_final;
    void* dv;
    float* dh0;
    float* adjoints;
    float* pulls;
    int64_t T, N, each, G, H, K, V, parts;
    int64_t mat_bytes, at_f, at_nt, at_pt;
};

// The chain: as gdr_fwd_kernel, which see for its waves, LDS and lanes.  Pᵀ is in LDS
// once (bfloat16), from the barrier behind its use on the next chunk's, or comes from
// memory.
template <typename T, int KP, int NW>
__global__ __launch_bounds__(NW * 64) void gdr_adjoint_kernel(AdjointArgs a) {
    constexpr bool B16 = sizeof(T) == 2;
    constexpr int PL = kPlanes<T>, KS = KP / 32, KM = KP / 16, VC = NW * 16;
    typedef Tile<KP> Keys;
    typedef Tile<VC> Values;
    constexpr int kN = 3 * kGdrBlocks * kGdrBlockBytes, kF = kGdrFactors * kC * 4, kMats = kF + kN;
    constexpr int kKeys = 2 * PL * Keys::kBytes;
    constexpr int kPart = B16 ? kKeys + Values::kBytes + kMats : kMats;
    __shared__ __align__(16) uint8_t lds[2 * kPart + (B16 ? kN : kKeys)];
    static_assert(sizeof(lds) <= 160 * 1024, "LDS of a compute unit");
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const HeadPart at = head_part(static_cast<uint32_t>(a.parts));
    if (at.head >= a.N * a.H) return;
    const int64_t part = at.part, n = at.head / static_cast<uint32_t>(a.H), h = at.head - n * a.H;
    const int64_t hg = h / (a.H / a.G);
    const int64_t vw = part * VC, v0 = vw + w * 16;
    const bool in_v = v0 < a.V;
    const Span sp = span_of(a.offsets, n, a.T, a.each);
    const int64_t slot0 = first_slot(sp, n), chunks = (sp.len + kC - 1) / kC;
    const int K = static_cast<int>(a.K);

    f32x4 L[KM];
#pragma unroll
    for (int m = 0; m < KM; ++m) {
        L[m] = f32x4{0, 0, 0, 0};
        if (a.dh_final && in_v && state_column(m, 4 * g) < K)
            L[m] = *reinterpret_cast<const f32x4*>(a.dh_final + ((n * a.H + h) * a.V + v0 + c) * a.K + state_column(m, 4 * g));
    }

    const int64_t qk_stride = a.G * a.K, v_stride = a.H * a.V;
    const T* kp = static_cast<const T*>(a.k) + sp.start * qk_stride + hg * a.K;
    const T* qp = static_cast<const T*>(a.q) + sp.start * qk_stride + hg * a.K;
    const T* dyp = static_cast<const T*>(a.dy) + sp.start * v_stride + h * a.V;
    T* dvp = static_cast<T*>(a.dv) + sp.start * v_stride + h * a.V + v0 + (c & ~3);
    auto length = [&](int64_t chunk) { return static_cast<int>(imin64(kC, sp.len - chunk * kC)); };
    auto mats_of = [&](int64_t chunk) { return a.mats + ((slot0 + chunk) * a.H + h) * a.mat_bytes; };
    const RowsToLds<KP, NW> key_loads(static_cast<uint32_t>(qk_stride), K, w, lane);
    const RowsToLds<VC, NW> value_loads(static_cast<uint32_t>(v_stride), static_cast<int>(a.V - vw), w, lane);
    FloatRows<KP, NW * 64> fk, fq;
    constexpr int kParts = 4;  // as in gdr_fwd_kernel
    auto fetch = [&](int64_t chunk, int half, int part) {
        const int len = length(chunk);
        uint8_t* to = lds + half * kPart;
        if constexpr (B16) {
            if (part == 0) key_loads.load(lds_offset(to), kp + chunk * kC * qk_stride, len, w);
            if (part == 1) key_loads.load(lds_offset(to) + Keys::kBytes, qp + chunk * kC * qk_stride, len, w);
            if (part == 2) value_loads.load(lds_offset(to) + kKeys, dyp + vw + chunk * kC * v_stride, len, w);
            if (part == 3) bytes_to_lds<NW, kMats>(lds_offset(to) + kKeys + Values::kBytes, mats_of(chunk) + a.at_f, w, lane);
        } else {
            if (part == 0) bytes_to_lds<NW, kMats>(lds_offset(to), mats_of(chunk) + a.at_f, w, lane);
            if (part == 1) fk.load(kp + chunk * kC * qk_stride, static_cast<uint32_t>(qk_stride), len, K, tid);
            if (part == 2) fq.load(qp + chunk * kC * qk_stride, static_cast<uint32_t>(qk_stride), len, K, tid);
        }
    };
    auto fetch_pt = [&](int64_t chunk) {
        if constexpr (B16) bytes_to_lds<NW, kN>(lds_offset(lds) + 2 * kPart, mats_of(chunk) + a.at_pt, w, lane);
    };
    if (chunks) {
        fetch_pt(chunks - 1);
#pragma unroll
        for (int q = 0; q < kParts; ++q) fetch(chunks - 1, (chunks - 1) & 1, q);
    }
    for (int64_t chunk = chunks - 1; chunk >= 0; --chunk) {
        const int half = static_cast<int>(chunk & 1), len = length(chunk);
        const uint8_t* in = lds + half * kPart;
        const uint8_t *lds_k = B16 ? in : lds + 2 * kPart, *lds_q = lds_k + PL * Keys::kBytes, *lds_dy = in + kKeys;
        const uint8_t* lds_f = B16 ? lds_dy + Values::kBytes : in;
        const uint8_t* lds_n = lds_f + kF;
        const float* f = reinterpret_cast<const float*>(lds_f);
        tile_barrier();  // this half is whole, nobody reads the other one
        if constexpr (!B16) {
            fk.store(lds + 2 * kPart, tid);
            fq.store(lds + 2 * kPart + PL * Keys::kBytes, tid);
            __syncthreads();
        }
        f32x4 dy[4];  // item r of tile rt: token 16 rt + 4 g + r of this lane's column
        f32x4 X[4] = {};
        if (in_v) {
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                if constexpr (B16) {
                    const u32x2 x = Values::four(lds_dy, rt, w, c, g);
                    dy[rt] = f32x4{bf16_lo(x[0]), bf16_hi(x[0]), bf16_lo(x[1]), bf16_hi(x[1])};
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = 16 * rt + 4 * g + r;
                        dy[rt][r] = View<T>(dyp + chunk * kC * v_stride).one(t * static_cast<uint32_t>(v_stride) + static_cast<uint32_t>(v0) + c, t < len);
                    }
                }
            }
            // Pᵀ dy first: it waits for memory, and for nothing that the chunk before leaves
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Planes<PL> d = split<PL>(dy[2 * s], dy[2 * s + 1]);
#pragma unroll
                for (int rt = 0; rt < 4; ++rt)
                    if (block_of<false>(rt, s) >= 0) {
                        if constexpr (B16) X[rt] = mma(load_block<3>(lds + 2 * kPart, block_of<false>(rt, s), lane), d, X[rt]);
                        else X[rt] = mma(load_block<3>(mats_of(chunk) + a.at_pt, block_of<false>(rt, s), lane), d, X[rt]);
                    }
            }
        }
        if constexpr (B16) {
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // Pᵀ is read
        }
        const bool more = chunk > 0;
        if (more) fetch_pt(chunk - 1);
        if (!in_v) {
#pragma unroll
            for (int q = 0; q < kParts; ++q)
                if (more) fetch(chunk - 1, half ^ 1, q);
            continue;
        }

        {
            float* to = a.adjoints + (((slot0 + chunk) * a.H + h) * a.V + v0 + c) * a.K;
#pragma unroll
            for (int m = 0; m < KM; ++m)
                if (state_column(m, 4 * g) < K) *reinterpret_cast<f32x4*>(to + state_column(m, 4 * g)) = L[m];
        }
        // du = D (L k) + Pᵀ dy
        f32x4 Y[4] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const Planes<3> lt = split<3>(L[2 * s], L[2 * s + 1]);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) Y[rt] = mma(Keys::template rows<PL>(lds_k, rt, s, c, g), lt, Y[rt]);
            if (more) {
#pragma unroll
                for (int q = s * kParts / KS; q < (s + 1) * kParts / KS; ++q) fetch(chunk - 1, half ^ 1, q);
            }
        }
        f32x4 beta[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            beta[rt] = *reinterpret_cast<const f32x4*>(f + kC + 16 * rt + 4 * g);
            X[rt] += *reinterpret_cast<const f32x4*>(f + 2 * kC + 16 * rt + 4 * g) * Y[rt];
        }
        // Z = du + Nᵀ (beta du)
        const Planes<3> mx[2] = {split<3>(beta[0] * X[0], beta[1] * X[1]), split<3>(beta[2] * X[2], beta[3] * X[3])};
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (block_of<false>(rt, s) >= 0) X[rt] = mma(load_block<3>(lds_n, block_of<false>(rt, s), lane), mx[s], X[rt]);
        {   // four value elements of a token a lane
            float* z = a.pulls + ((slot0 + chunk) * a.H + h) * kC * a.V + (4 * g + (c & 3)) * a.V + v0 + (c & ~3);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                *reinterpret_cast<f32x4*>(z + 16 * rt * a.V) = quad_transpose(X[rt], c);
                X[rt] *= beta[rt];  // dr
                const f32x4 dr = quad_transpose(X[rt], c);
                const float out[4] = {dr[0], dr[1], dr[2], dr[3]};
                const int t = 16 * rt + 4 * g + (c & 3);
                if (t < len) store_row(dvp + (chunk * kC + t) * v_stride, out);
            }
        }
        // the adjoint of the state before the chunk
        const float last = f[4 * kC];
#pragma unroll
        for (int i = 0; i < KM; ++i) L[i] *= last;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            f32x4 ek[2], eq[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ek[i] = -*reinterpret_cast<const f32x4*>(f + 32 * s + 16 * i + 4 * g);
                eq[i] = *reinterpret_cast<const f32x4*>(f + 3 * kC + 32 * s + 16 * i + 4 * g);
            }
            const Planes<3> dr = split<3>(ek[0] * X[2 * s], ek[1] * X[2 * s + 1]);
            const Planes<3> dq = split<3>(eq[0] * dy[2 * s], eq[1] * dy[2 * s + 1]);
#pragma unroll
            for (int i = 0; i < KM; ++i) L[i] = mma(Keys::template columns<PL>(lds_q, i, s, c, g), dq, L[i]);
#pragma unroll
            for (int i = 0; i < KM; ++i) L[i] = mma(Keys::template columns<PL>(lds_k, i, s, c, g), dr, L[i]);
        }
    }
    if (a.dh0 && in_v) {
#pragma unroll
        for (int m = 0; m < KM; ++m)
            if (state_column(m, 4 * g) < K)
                *reinterpret_cast<f32x4*>(a.dh0 + ((n * a.H + h) * a.V + v0 + c) * a.K + state_column(m, 4 * g)) = L[m];
    }
}

// ---- the chunks' gradients --------------------------------------------------------

struct GradArgs {
    const void *q, *k, *dy;
    const float *g, *beta;
    const int32_t* offsets;
    const float *states, *misses, *adjoints, *pulls;
    void *dq, *dk;
    float *dg, *dbeta;
    int64_t T, N, each, G, H, K, V;
    float scale;
    int norm;
};

// Half of an operand's slots, in planes.
template <int N>
__device__ __forceinline__ void put_four(uint8_t* to, int plane_bytes, f32x4 x) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        *reinterpret_cast<u32x2*>(to + n * plane_bytes) = u32x2{upper_halves(x[0], x[1]), upper_halves(x[2], x[3])};
        if (n + 1 < N) {
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] -= upper_part(x[r]);
        }
    }
}

// 32 value elements of 64 tokens as planes in LDS, an operand row (64 bytes) for each
// token, in folded order.
struct TokenTile {
    static constexpr int kBytes = kC * 64;
    __device__ static __forceinline__ int at(int token, int piece) { return token * 64 + ((piece ^ ((token >> 1) & 3)) * 16); }
    // elements 4 q ..
    template <int N>
    __device__ static __forceinline__ void put(uint8_t* lds, int token, int q, f32x4 x) {
        put_four<N>(lds + at(token, q & 3) + (q >> 2) * 8, kBytes, x);
    }
    template <int N>
    __device__ static __forceinline__ Planes<N> read(const uint8_t* lds, int token, int piece) {
        Planes<N> out;
#pragma unroll
        for (int n = 0; n < N; ++n) out.p[n] = *reinterpret_cast<const u32x4*>(lds + n * kBytes + at(token, piece));
        return out;
    }
};

__device__ __forceinline__ float dot4(f32x4 a, f32x4 b, float s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __builtin_fmaf(a[i], b[i], s);
    return s;
}
__device__ __forceinline__ float group4_sum(float v) {  // over the lanes l, l ^ 16, l ^ 32, l ^ 48
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// A workgroup: one chunk and one head of q and k, with all value heads that share
// it, whose dq and dk are summed in registers.  Wave w of half kh has the tokens 16 w
// .. 16 w + 15 in the columns of its accumulators and half of the key elements in
// their rows, so that a lane's factors are one token's and it stores four neighbours.
// 32 value elements at a time are cut into planes in LDS, with the next ones' loads
// under way; a state's columns are read by transposing reads.  Of the two 64 x 64
// matrices the waves of one half have dy uᵀ, the others Z uᵀ, each the blocks of its
// rows, transposed, and of its columns: as they lie in the accumulators, and are
// exchanged through LDS, these are the operands that follow.
template <typename T, int KP>
__global__ __launch_bounds__(512, 2) void gdr_grad_kernel(GradArgs a) {
    constexpr int PL = kPlanes<T>, KH = KP / 32;  // row tiles of key elements of a wave
    constexpr int THREADS = 512, WAVES = 8;
    typedef Tile<KP> Keys;
    typedef Tile<KP, 32> State;
    typedef TokenTile Tokens;
    constexpr int kKeys = 2 * PL * Keys::kBytes, kStaged = 6 * State::kBytes + (6 + PL) * Tokens::kBytes;
    constexpr int kExchange = WAVES * 5 * 1024;
    constexpr bool kShare = kKeys + kStaged > 150 * 1024;  // q and k come after the sums, in the same place
    __shared__ __align__(16) uint8_t lds[kKeys + (kShare ? kExchange : kStaged)];
    __shared__ __align__(16) float s_hi[kC], s_lo[kC], s_beta[kC], s_rk[kC], s_rq[kC], s_db[2][kC], s_states[2][kC], s_diag[kC], s_dots[4][kC], s_end[8];
    static_assert(sizeof(lds) + 4300 <= 160 * 1024 && kStaged >= kExchange && (!kShare || kKeys >= kStaged), "LDS of a compute unit, and its parts");
    uint8_t *lds_k = lds, *lds_q = lds_k + PL * Keys::kBytes;
    uint8_t *lds_s = lds + (kShare ? 0 : kKeys), *lds_l = lds_s + 3 * State::kBytes, *lds_z = lds_l + 3 * State::kBytes,
            *lds_u = lds_z + 3 * Tokens::kBytes, *lds_dy = lds_u + 3 * Tokens::kBytes;
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), w = wave & 3, kh = wave >> 2, c = lane & 15, g = lane >> 4;
    const int64_t hg = blockIdx.x % static_cast<uint32_t>(a.G), slot = blockIdx.x / static_cast<uint32_t>(a.G);
    const Chunk ch = chunk_of(a.offsets, slot, a.T, a.N, a.each);
    if (ch.len == 0) return;
    const int K = static_cast<int>(a.K), V = static_cast<int>(a.V);
    const int64_t qk_stride = a.G * a.K, v_stride = a.H * a.V;
    const T* kp = static_cast<const T*>(a.k) + ch.start * qk_stride + hg * a.K;
    const T* qp = static_cast<const T*>(a.q) + ch.start * qk_stride + hg * a.K;
    const View<T> k_rows(kp), q_rows(qp);
    const int row = 16 * w + c;  // this lane's token
    const bool in_t = row < ch.len;
    // Everything that a chunk needs at first is asked for at once, and waited for behind the last of it.
    FloatRows<KP, THREADS> k_float, q_float;
    auto ask_keys = [&] {
        if constexpr (sizeof(T) == 2) {
            const RowsToLds<KP, WAVES> loads(static_cast<uint32_t>(qk_stride), K, wave, lane);
            loads.load(lds_offset(lds_k), kp, ch.len, wave);
            loads.load(lds_offset(lds_q), qp, ch.len, wave);
        } else {
            k_float.load(kp, static_cast<uint32_t>(qk_stride), ch.len, K, tid);
            q_float.load(qp, static_cast<uint32_t>(qk_stride), ch.len, K, tid);
        }
    };
    auto keep_keys = [&] {
        if constexpr (sizeof(T) == 4) {
            k_float.store(lds_k, tid);
            q_float.store(lds_q, tid);
        }
        wait_memory<0>();
    };
    if constexpr (!kShare) ask_keys();
    auto column = [&](int m) { return state_column(kh * KH + m, 4 * g); };  // of the wave's tile m, of this lane's rows

    // four key elements of a token out of a tile
    auto from_tile = [&](const uint8_t* tile, int token, int col) {
        f32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int n = PL - 1; n >= 0; --n) {
            const u32x2 x = *reinterpret_cast<const u32x2*>(tile + n * Keys::kBytes + Keys::at(token, col >> 3) + (col & 4) * 2);
            v += f32x4{bf16_lo(x[0]), bf16_hi(x[0]), bf16_lo(x[1]), bf16_hi(x[1])};
        }
        return v;
    };
    f32x4 dq_sum[KH] = {}, dk_sum[KH] = {};
    const int per = static_cast<int>(a.H / a.G);
    constexpr int kItems = KP * 8 / THREADS;    // four columns of an element each
    const int to_t = tid >> 3, to_q = tid & 7;  // eight lanes a token, four elements each
    float to_beta, dbeta;
    f32x4 st_s[kItems], st_l[kItems], to_z, to_e, to_dy;
    auto fetch = [&](int64_t h, int vb) {
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));  // addresses are computed here, not kept (and spilled) from before the loops
        const int to_t = tid >> 3, to_q = tid & 7;
        const int64_t cell = slot * a.H + h;
        const View<float> S(a.states + cell * a.V * a.K), L(a.adjoints + cell * a.V * a.K);
        const View<float> e(a.misses + cell * kC * a.V), z(a.pulls + cell * kC * a.V);
        const View<T> dy(static_cast<const T*>(a.dy) + ch.start * v_stride + h * a.V);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int item = tid + THREADS * i, v = vb + item / (KP / 4), k = item % (KP / 4) * 4;
            st_s[i] = S.four(v * K + k, v < V && k < K);
            st_l[i] = L.four(v * K + k, v < V && k < K);
        }
        const int v = vb + 4 * to_q;
        to_z = z.four(to_t * V + v, v < V);
        to_e = e.four(to_t * V + v, v < V);
        to_dy = dy.four(to_t * static_cast<uint32_t>(v_stride) + v, v < V && to_t < ch.len);
        if (vb == 0) to_beta = View<float>(a.beta + ch.start * a.H + h).one(to_t * static_cast<uint32_t>(a.H), to_t < ch.len);
    };
    fetch(hg * per, 0);
    float g_log = View<float>(a.g + ch.start * a.H + hg * per).one(lane * static_cast<uint32_t>(a.H), lane < ch.len);
    {   // the lengths of q and k
        float k2 = 0.0f, q2 = 0.0f;
#pragma unroll
        for (int p = 0; p < KP / 64; ++p) {
            const uint32_t col = 64 * p + 8 * to_q, at = to_t * static_cast<uint32_t>(qk_stride) + col;
            const bool in = to_t < ch.len && col < a.K;
            k2 += sum_squares(k_rows.planes(at, in));
            q2 += sum_squares(q_rows.planes(at, in));
        }
        k2 = group_sum<8>(k2);
        q2 = group_sum<8>(q2);
        if (to_q == 0) {
            s_rk[to_t] = a.norm ? 1.0f / __builtin_sqrtf(k2 + kGdrNormEps) : 1.0f;
            s_rq[to_t] = a.norm ? 1.0f / __builtin_sqrtf(q2 + kGdrNormEps) : 1.0f;
        }
    }
    if constexpr (!kShare) keep_keys();
    float rk = 1.0f, rq = 1.0f;
    for (int hh = 0; hh < per; ++hh) {
        const int64_t h = hg * per + hh;
        __syncthreads();  // the head before is done with LDS
        if (wave == 0) {
            int token = lane;
            asm volatile("" : "+v"(token));  // what the sum needs of it is computed here, not kept (and spilled)
            const double b = decays_since_start(g_log, token);
            const float hi = static_cast<float>(b);
            s_hi[token] = hi;
            s_lo[token] = static_cast<float>(b - hi);
        }
        // sums over the value elements; X: dy . u, or in the waves of the second half M: Z . u, of block b the rows
        // (tokens i) of column block w for b > w, transposed (rows: tokens j) for b <= w, and of the diagonal both
        f32x4 yS[KH] = {}, zS[KH] = {}, uL[KH] = {}, half[5] = {};
        float both = 0.0f;
        dbeta = 0.0f;
        if (to_q == 0) s_beta[to_t] = to_beta;
#pragma unroll 1
        for (int vb = 0; vb < V; vb += 32) {
            __syncthreads();  // what is staged has been read
            int tid = threadIdx.x;
            asm volatile("" : "+v"(tid));  // as above
            const int to_t = tid >> 3, to_q = tid & 7;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int item = tid + THREADS * i, v = item / (KP / 4), k = item % (KP / 4) * 4;
                const int at = State::at(v, k >> 3) + (k & 4) * 2;
                both = dot4(st_s[i], st_l[i], both);
                put_four<3>(lds_s + at, State::kBytes, st_s[i]);
                put_four<3>(lds_l + at, State::kBytes, st_l[i]);
            }
            dbeta = dot4(to_z, to_e, dbeta);
            Tokens::put<3>(lds_z, to_t, to_q, to_z);
            Tokens::put<3>(lds_u, to_t, to_q, to_beta * to_e);
            Tokens::put<PL>(lds_dy, to_t, to_q, to_dy);
            __syncthreads();
            if (vb + 32 < V) fetch(h, vb + 32);
            int c = lane & 15, g = lane >> 4;
            asm volatile("" : "+v"(c), "+v"(g));  // as above
            const int row = 16 * w + c;
            const Planes<3> zf = Tokens::read<3>(lds_z, row, g), uf = Tokens::read<3>(lds_u, row, g);
            const Planes<PL> dyf = Tokens::read<PL>(lds_dy, row, g);
#pragma unroll
            for (int m = 0; m < KH; ++m) {
                const Planes<3> sf = State::template columns<3>(lds_s, kh * KH + m, 0, c, g);
                yS[m] = mma(sf, dyf, yS[m]);
                zS[m] = mma(sf, zf, zS[m]);
                uL[m] = mma(State::template columns<3>(lds_l, kh * KH + m, 0, c, g), uf, uL[m]);
                if (m % 2) __builtin_amdgcn_sched_barrier(0);  // all operands at once would not fit the registers
            }
            // of Z or dy with u; the operands are chosen, not the instructions: behind a branch each read of LDS waits
            auto blocks = [&](const uint8_t* lds_x, auto& xf) {
                constexpr int PX = sizeof(xf) / 16;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const bool below = b <= w;
                    Planes<3> rows, columns;
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        const uint8_t* from = below ? lds_u + p * Tokens::kBytes : lds_x + p % PX * Tokens::kBytes;
                        rows.p[p] = Tokens::template read<1>(from, 16 * b + c, g).p[0];
                        columns.p[p] = below ? xf.p[p % PX] : uf.p[p];
                    }
                    if constexpr (PX == 3) {
                        half[b] = mma(rows, columns, half[b]);
                    } else {
#pragma unroll
                        for (int p = 2; p >= 0; --p) half[b] = mma(Planes<1>{{rows.p[p]}}, Planes<1>{{columns.p[p]}}, half[b]);
                    }
                    if (b % 2) __builtin_amdgcn_sched_barrier(0);
                }
                half[4] = mma(xf, uf, half[4]);
            };
            if (kh == 0) blocks(lds_dy, dyf);
            else blocks(lds_z, zf);
        }
        __syncthreads();  // what was staged has been read
        f32x4* exchange = reinterpret_cast<f32x4*>(lds + kKeys) + wave * 5 * 64 + lane;  // read from there: they would not fit the registers
        {   // with their decays: X_ij = scale G_ij dP_ij, M_ij = -G_ij beta_i Z_i . u_j (j < i); X_ii apart
            float diagonal = 0.0f;
            const float row_hi = s_hi[row], row_lo = s_lo[row], row_beta = s_beta[row];
#pragma unroll
            for (int n = 0; n < 5; ++n) {
                const int b = n < 4 ? n : w;
                const bool columns = n == 4 || b > w;  // rows are tokens i, the lane's is j
                const f32x4 hi = *reinterpret_cast<const f32x4*>(s_hi + 16 * b + 4 * g), lo = *reinterpret_cast<const f32x4*>(s_lo + 16 * b + 4 * g),
                            beta = *reinterpret_cast<const f32x4*>(s_beta + 16 * b + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int other = 16 * b + 4 * g + r, ahead = columns ? other - row : row - other;  // i - j
                    const float sum = (hi[r] - row_hi) + (lo[r] - row_lo);
                    const float d = fast_exp2(ahead > 0 ? (columns ? sum : -sum) * kLog2e : -1000.0f);  // 0 there
                    if (n < 4) diagonal = ahead == 0 ? half[n][r] : diagonal;
                    half[n][r] *= kh == 0 ? a.scale * d : -d * (columns ? beta[r] : row_beta);
                }
                exchange[n * 64] = half[n];
            }
            if (kh == 0 && g == c >> 2) s_diag[row] = a.scale * diagonal;
        }
        __syncthreads();
        if constexpr (kShare) {
            ask_keys();
            __syncthreads();
            keep_keys();
            __syncthreads();
        }
        rk = s_rk[row];
        rq = s_rq[row];
        if (hh + 1 < per) {  // the next head's, on their way meanwhile
            fetch(h + 1, 0);
            g_log = View<float>(a.g + ch.start * a.H + h + 1).one(lane * static_cast<uint32_t>(a.H), lane < ch.len);
        }
        const float row_hi = s_hi[row], row_lo = s_lo[row], row_beta = s_beta[row];
        const f32x4 zero = {0, 0, 0, 0};
        auto four = [&](const float* p, int b) { return *reinterpret_cast<const f32x4*>(p + 16 * b + 4 * g); };
        dbeta = group_sum<8>(dbeta);
        if (to_q == 0 && to_t < ch.len) a.dbeta[(ch.start + to_t) * a.H + h] = dbeta;
        both = group4_sum(group_sum<16>(both));
        if (lane == 0) s_end[wave] = both;

        int c = lane & 15, g = lane >> 4;
        asm volatile("" : "+v"(c), "+v"(g));  // as above
        const float in_chunk = whole_exp(static_cast<double>(row_hi) + row_lo);
        const double end = static_cast<double>(s_hi[kC - 1]) + s_lo[kC - 1];
        const float to_end = whole_exp(end - (static_cast<double>(row_hi) + row_lo));
        const float fy = a.scale * in_chunk, fz = -in_chunk * row_beta;
        float read = 0.0f, db = 0.0f;
        const int token = 16 * w + c;
#pragma unroll
        for (int m = 0; m < KH; ++m) {
            const int col = state_column(kh * KH + m, 4 * g);
            const f32x4 k4 = rk * from_tile(lds_k, token, col), q4 = rq * from_tile(lds_q, token, col);
            yS[m] *= fy;
            zS[m] *= fz;
            uL[m] *= to_end;
            read = dot4(q4, yS[m], read);
            read = dot4(k4, zS[m], read);
        }
        read = group4_sum(read);
        if (g == 0) s_states[kh][token] = read;
        // summed over the tokens of blocks 2 s and 2 s + 1: the lane's row of X and M, and its column
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            __builtin_amdgcn_sched_barrier(0);  // one after the other: both at once would not fit the registers
            auto operand = [&](int of, bool columns, const float* factor) {
                f32x4 part[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int b = 2 * s + i;
                    const f32x4 v = reinterpret_cast<const f32x4*>(lds + kKeys)[((4 * of + w) * 5 + (columns && b == w ? 4 : b)) * 64 + 16 * g + c];
                    part[i] = (columns ? b >= w : b <= w) ? v * four(factor, b) : zero;
                }
                return split<3>(part[0], part[1]);
            };
            const Planes<3> xr = operand(0, false, s_rk), mr = operand(1, false, s_rk), xc = operand(0, true, s_rq), mc = operand(1, true, s_rk);
#pragma unroll
            for (int m = 0; m < KH; ++m) {
                const Planes<PL> kt = Keys::template columns<PL>(lds_k, kh * KH + m, s, c, g);
                const Planes<PL> qt = Keys::template columns<PL>(lds_q, kh * KH + m, s, c, g);
                yS[m] = mma(kt, xr, yS[m]);
                zS[m] = mma(kt, mr, zS[m]);
                uL[m] = mma(kt, mc, uL[m]);
                uL[m] = mma(qt, xc, uL[m]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        const float diagonal = s_diag[token];
#pragma unroll
        for (int m = 0; m < KH; ++m) {
            const int col = state_column(kh * KH + m, 4 * g);
            const f32x4 k4 = rk * from_tile(lds_k, token, col), q4 = rq * from_tile(lds_q, token, col);
            db = dot4(q4, yS[m], db);
            db = dot4(k4, zS[m] - uL[m], db);
            dq_sum[m] += yS[m] + diagonal * k4;
            dk_sum[m] += zS[m] + uL[m] + diagonal * q4;
        }
        __builtin_amdgcn_sched_barrier(0);
        db = group4_sum(db);
        if (g == 0) s_db[kh][row] = db;
        __syncthreads();
        if (wave == 0) {
            int token = lane;
            asm volatile("" : "+v"(token));  // as above
            const double read = static_cast<double>(s_states[0][token]) + s_states[1][token];
            double from_here = read, up_to_here = read - s_db[0][token] - s_db[1][token];
#pragma unroll
            for (int d = 1; d < kC; d *= 2) {
                const double after = of_lane(from_here, token + d), before = of_lane(up_to_here, token - d);
                if (token + d < kC) from_here += after;
                if (token >= d) up_to_here += before;
            }
            const double before = of_lane(up_to_here, token - 1);
            double v = from_here + (token ? before : 0.0);
            double states = 0.0;
#pragma unroll
            for (int i = 0; i < WAVES; ++i) states += s_end[i];
            v += static_cast<double>(whole_exp(end)) * states;
            if (token < ch.len) a.dg[(ch.start + token) * a.H + h] = static_cast<float>(v);
        }
    }
    // through the division by their lengths
    float qd = 0.0f, kd = 0.0f;
    f32x4 k4[KH], q4[KH];
#pragma unroll
    for (int m = 0; m < KH; ++m) {
        k4[m] = (a.norm ? rk : 0.0f) * from_tile(lds_k, row, column(m));
        q4[m] = (a.norm ? rq : 0.0f) * from_tile(lds_q, row, column(m));
        qd = dot4(q4[m], dq_sum[m], qd);
        kd = dot4(k4[m], dk_sum[m], kd);
    }
    qd = group4_sum(qd);
    kd = group4_sum(kd);
    if (g == 0) s_dots[kh][row] = qd, s_dots[2 + kh][row] = kd;
    __syncthreads();
    qd = s_dots[0][row] + s_dots[1][row];
    kd = s_dots[2][row] + s_dots[3][row];
    T* dqp = static_cast<T*>(a.dq) + (ch.start + row) * qk_stride + hg * a.K;
    T* dkp = static_cast<T*>(a.dk) + (ch.start + row) * qk_stride + hg * a.K;
#pragma unroll
    for (int m = 0; m < KH; ++m) {
        if (!in_t || column(m) >= K) continue;
        const f32x4 x = rq * (dq_sum[m] - qd * q4[m]), y = rk * (dk_sum[m] - kd * k4[m]);
        const float xs[4] = {x[0], x[1], x[2], x[3]}, ys[4] = {y[0], y[1], y[2], y[3]};
        store_row(dqp + column(m), xs);
        store_row(dkp + column(m), ys);
    }
}

template <typename T, int KP, int NW>
hipError_t launch_c(const GdrArgs& a, hipStream_t s) {
    const GdrLayout l(true);
    const int64_t parts = (a.V + 16 * NW - 1) / (16 * NW);
    const AdjointArgs k{a.q, a.k, a.dy, a.offsets, a.mats, a.dh_final, a.dv, a.dh0, a.adjoints, a.pulls,
                        a.T, a.N, a.T / a.N, a.G, a.H, a.K, a.V, parts, l.bytes, l.factors, l.nt, l.pt};
    gdr_adjoint_kernel<T, KP, NW><<<xcd_grid(a.N * a.H, parts), NW * 64, 0, s>>>(k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const GradArgs d{a.q, a.k, a.dy, a.g, a.beta, a.offsets, a.states, a.misses, a.adjoints, a.pulls, a.dq, a.dk, a.dg, a.dbeta,
                     a.T, a.N, a.T / a.N, a.G, a.H, a.K, a.V, a.scale, a.norm};
    gdr_grad_kernel<T, KP><<<static_cast<uint32_t>(gdr_slots(a.T, a.N) * a.G), 512, 0, s>>>(d);
    return hipGetLastError();
}
template <typename T, int KP>
hipError_t launch_k(const GdrArgs& a, hipStream_t s) {
    // As the forward: chains of 128 columns once those of 64 are more than the compute
    // units.  1,024 tokens, the whole backward in us with 64 / 128 columns: key and value
    // dim 128, 128 heads 375 / 407; 128 and 256, 72 heads 440 / 395; float32, 64 and 128,
    // 128 heads 365 / 420, 64 and 256, 72 heads 480 / 393.  Eight waves have too few
    // registers for the float32 planes of a key dim of 128.
    if constexpr (sizeof(T) == 2 || KP == 64) {
        if (a.V > 64 && a.N * a.H * ((a.V + 63) / 64) > 256) return launch_c<T, KP, 8>(a, s);
    }
    return launch_c<T, KP, 4>(a, s);
}
template <typename T>
hipError_t launch_t(const GdrArgs& a, hipStream_t s) {
    return a.K <= 64 ? launch_k<T, 64>(a, s) : launch_k<T, 128>(a, s);
}

}  // namespace

hipError_t launch_gdr_bwd(const GdrArgs& a, hipStream_t s) {
    return a.dtype == MSSM_F32 ? launch_t<float>(a, s) : launch_t<uint16_t>(a, s);
}

}  // namespace mssm
