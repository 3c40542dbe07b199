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
//     db    = q . dq + k . dk_row - k . dk_column, and for the chunk's last token
//             exp(b_C) <L, S> + sum_t D_t k_t . (L u_t) more;   dg_i = sum_{t >= i} db_t
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
    int64_t T, N, each, G, H, K, V, slot0;
    float scale;
    int norm;
};

constexpr int kPitch = kC + 4;  // floats of a row of a 64 x 64 matrix in LDS

// 32 value elements of a state as planes in LDS, an operand row (64 bytes) for
// each of KP columns; slot (g, j) is element 8 g + j.
template <int KP>
struct StateTile {
    static constexpr int kBytes = KP * 64;
    __device__ static __forceinline__ int at(int column, int piece) { return column * 64 + ((piece ^ ((column >> 1) & 3)) * 16); }
    __device__ static __forceinline__ Planes<3> read(const uint8_t* lds, int column, int piece) {
        Planes<3> out;
#pragma unroll
        for (int n = 0; n < 3; ++n) out.p[n] = *reinterpret_cast<const u32x4*>(lds + n * kBytes + at(column, piece));
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

// A workgroup: one chunk and one head of q and k, with all value heads that
// share it, whose dq and dk are summed in registers.  Wave w has the tokens 16 w
// .. 16 w + 15 in the columns of its accumulators and the key elements in their
// rows, so that a lane's factors are one token's and it stores four neighbours.
template <typename T, int KP>
__global__ __launch_bounds__(256) void gdr_grad_kernel(GradArgs a) {
    constexpr int PL = kPlanes<T>, KM = KP / 16;
    typedef Tile<KP> Keys;
    typedef StateTile<KP> State;
    constexpr int kMatrix = kC * kPitch * 4, kKeys = 2 * PL * Keys::kBytes, kStates = 6 * State::kBytes;
    __shared__ __align__(16) uint8_t lds[kKeys + (2 * kMatrix > kStates ? 2 * kMatrix : kStates)];
    __shared__ float s_hi[kC], s_lo[kC], s_beta[kC], s_rk[kC], s_rq[kC], s_db[kC], s_end[8];
    uint8_t *lds_k = lds, *lds_q = lds + PL * Keys::kBytes;
    uint8_t *lds_s = lds + kKeys, *lds_l = lds_s + 3 * State::kBytes;             // while summing over value elements
    float *sX = reinterpret_cast<float*>(lds + kKeys), *sM = sX + kC * kPitch;  // then
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const int64_t hg = blockIdx.x % a.G, slot = a.slot0 + blockIdx.x / a.G;
    const Chunk ch = chunk_of(a.offsets, slot, a.T, a.N, a.each);
    if (ch.len == 0) return;
    const int K = static_cast<int>(a.K), V = static_cast<int>(a.V);
    const int64_t qk_stride = a.G * a.K, v_stride = a.H * a.V;
    const T* kp = static_cast<const T*>(a.k) + ch.start * qk_stride + hg * a.K;
    const T* qp = static_cast<const T*>(a.q) + ch.start * qk_stride + hg * a.K;
    const View<T> k_rows(kp), q_rows(qp);
    const int row = 16 * w + c;  // this lane's token
    const bool in_t = row < ch.len;
    const uint32_t row_at = row * static_cast<uint32_t>(qk_stride);
    float rk = 1.0f, rq = 1.0f;
    if (a.norm) {
        float k2 = 0.0f, q2 = 0.0f;
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            const f32x4 k4 = k_rows.four(row_at + 16 * m + 4 * g, in_t && 16 * m < K);
            const f32x4 q4 = q_rows.four(row_at + 16 * m + 4 * g, in_t && 16 * m < K);
            k2 = dot4(k4, k4, k2);
            q2 = dot4(q4, q4, q2);
        }
        rk = 1.0f / __builtin_sqrtf(group4_sum(k2) + kGdrNormEps);
        rq = 1.0f / __builtin_sqrtf(group4_sum(q2) + kGdrNormEps);
    }
    if (g == 0) s_rk[row] = rk, s_rq[row] = rq;

    if constexpr (sizeof(T) == 2) {
        const RowsToLds<KP, 4> loads(static_cast<uint32_t>(qk_stride), K, w, lane);
        loads.load(lds_offset(lds_k), kp, ch.len, w);
        loads.load(lds_offset(lds_q), qp, ch.len, w);
        tile_barrier();
    } else {
        FloatRows<KP, 256> rows;
        rows.load(kp, static_cast<uint32_t>(qk_stride), ch.len, K, tid);
        rows.store(lds_k, tid);
        rows.load(qp, static_cast<uint32_t>(qk_stride), ch.len, K, tid);
        rows.store(lds_q, tid);
    }
    f32x4 dq_sum[KM] = {}, dk_sum[KM] = {};
    const int per = static_cast<int>(a.H / a.G);
    for (int hh = 0; hh < per; ++hh) {
        const int64_t h = hg * per + hh, cell = slot * a.H + h;
        __syncthreads();  // the head before is done with LDS
        if (w == 0) {
            const double b = decays_since_start(a.g + ch.start * a.H + h, a.H, ch.len, lane);
            const float hi = static_cast<float>(b);
            s_hi[lane] = hi;
            s_lo[lane] = static_cast<float>(b - hi);
            s_beta[lane] = lane < ch.len ? a.beta[(ch.start + lane) * a.H + h] : 0.0f;
        }
        const View<float> S(a.states + cell * a.V * a.K), L(a.adjoints + cell * a.V * a.K);
        const View<float> e(a.misses + cell * kC * a.V), z(a.pulls + cell * kC * a.V);
        const View<T> dy(static_cast<const T*>(a.dy) + ch.start * v_stride + h * a.V);

        // sums over the value elements
        f32x4 yS[KM] = {}, zS[KM] = {}, uL[KM] = {}, dP[4] = {}, dA[4] = {};
        float dbeta = 0.0f, both = 0.0f;
        for (int vb = 0; vb < V; vb += 32) {
            __syncthreads();
            {   // 8 value elements of 2 columns a thread
                const int o = tid / (KP / 2), kc = tid % (KP / 2) * 2;
                if (o < 4) {
                    float s0[8], s1[8], l0[8], l1[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bool in = vb + 8 * o < V && kc < K;
                        const f32x2 s2 = S.two((vb + 8 * o + j) * K + kc, in), l2 = L.two((vb + 8 * o + j) * K + kc, in);
                        s0[j] = s2[0]; s1[j] = s2[1]; l0[j] = l2[0]; l1[j] = l2[1];
                        both = __builtin_fmaf(s2[0], l2[0], __builtin_fmaf(s2[1], l2[1], both));
                    }
                    auto put = [&](uint8_t* to, int column, const Planes<3>& p) {
#pragma unroll
                        for (int n = 0; n < 3; ++n) *reinterpret_cast<u32x4*>(to + n * State::kBytes + State::at(column, o)) = p.p[n];
                    };
                    put(lds_s, kc, split<3>(s0));
                    put(lds_s, kc + 1, split<3>(s1));
                    put(lds_l, kc, split<3>(l0));
                    put(lds_l, kc + 1, split<3>(l1));
                }
            }
            __syncthreads();
            const int v = vb + 8 * g;
            const bool in = v < V;
            auto eight = [&](const View<float>& p, int t, float (&x)[8]) {
                const f32x4 lo = p.four(t * V + v, in), hi = p.four(t * V + v + 4, in);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = lo[i], x[4 + i] = hi[i];
            };
            float x[8], zz[8];
            eight(z, row, zz);
            eight(e, row, x);
            const float beta = s_beta[row];
#pragma unroll
            for (int i = 0; i < 8; ++i) dbeta = __builtin_fmaf(x[i], zz[i], dbeta), x[i] *= beta;
            const Planes<PL> dyf = dy.planes(row * static_cast<uint32_t>(v_stride) + v, in && in_t);
            const Planes<3> zf = split<3>(zz), uf = split<3>(x);
#pragma unroll
            for (int m = 0; m < KM; ++m) {
                const Planes<3> sf = State::read(lds_s, state_column(m, c), g), lf = State::read(lds_l, state_column(m, c), g);
                yS[m] = mma(sf, dyf, yS[m]);
                zS[m] = mma(sf, zf, zS[m]);
                uL[m] = mma(lf, uf, uL[m]);
            }
#pragma unroll
            for (int jb = 0; jb < 4; ++jb) {  // rows (of the accumulator): token i of this wave; columns: token j
                if (jb > w) continue;
                float xj[8];
                eight(e, 16 * jb + c, xj);
                const float bj = s_beta[16 * jb + c];
#pragma unroll
                for (int i = 0; i < 8; ++i) xj[i] *= bj;
                const Planes<3> uj = split<3>(xj);
                dP[jb] = mma(dyf, uj, dP[jb]);
                dA[jb] = mma(zf, uj, dA[jb]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
            const int j = 16 * jb + c;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * w + 4 * g + r;
                float x = 0.0f, mm = 0.0f;
                if (j <= i) {
                    const float d = decay_between(s_hi[i], s_lo[i], s_hi[j], s_lo[j]);
                    x = a.scale * d * dP[jb][r];
                    mm = j < i ? -d * s_beta[i] * dA[jb][r] : 0.0f;
                }
                sX[i * kPitch + j] = x;
                sM[i * kPitch + j] = mm;
            }
        }
        dbeta = group4_sum(dbeta);
        if (g == 0 && in_t) a.dbeta[(ch.start + row) * a.H + h] = dbeta;
        both = group_sum<16>(both);
        both = group4_sum(both);
        if (lane == 0) s_end[w] = both;
        __syncthreads();

        const float in_chunk = whole_exp(static_cast<double>(s_hi[row]) + s_lo[row]);
        const double end = static_cast<double>(s_hi[kC - 1]) + s_lo[kC - 1];
        const float to_end = whole_exp(end - (static_cast<double>(s_hi[row]) + s_lo[row]));
        const float fy = a.scale * in_chunk, fz = -in_chunk * s_beta[row];
        f32x4 dq[KM], dkr[KM], dkc[KM], k4[KM], q4[KM];
        float wrote = 0.0f;
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            const bool in = in_t && state_column(m, 4 * g) < K;
            k4[m] = rk * k_rows.four(row_at + state_column(m, 4 * g), in);
            q4[m] = rq * q_rows.four(row_at + state_column(m, 4 * g), in);
            dq[m] = fy * yS[m];
            dkr[m] = fz * zS[m];
            dkc[m] = to_end * uL[m];
            wrote = dot4(k4[m], dkc[m], wrote);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            // the tokens summed over: 32 s + slot; this lane's row of X and M, and its column
            float xr[8], mr[8], xc[8], mc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = 32 * s + 4 * g + (i & 3) + (i >> 2) * 16;
                const float rkt = s_rk[t];
                xr[i] = sX[row * kPitch + t] * rkt;
                mr[i] = sM[row * kPitch + t] * rkt;
                xc[i] = sX[t * kPitch + row] * s_rq[t];
                mc[i] = sM[t * kPitch + row] * rkt;
            }
            const Planes<3> xrf = split<3>(xr), mrf = split<3>(mr), xcf = split<3>(xc), mcf = split<3>(mc);
#pragma unroll
            for (int m = 0; m < KM; ++m) {
                const Planes<PL> kt = Keys::template columns<PL>(lds_k, m, s, c, g);
                const Planes<PL> qt = Keys::template columns<PL>(lds_q, m, s, c, g);
                dq[m] = mma(kt, xrf, dq[m]);
                dkr[m] = mma(kt, mrf, dkr[m]);
                dkc[m] = mma(kt, mcf, dkc[m]);
                dkc[m] = mma(qt, xcf, dkc[m]);
            }
        }
        float db = 0.0f;
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            db = dot4(q4[m], dq[m], db);
            db = dot4(k4[m], dkr[m] - dkc[m], db);
            dq_sum[m] += dq[m];
            dk_sum[m] += dkr[m] + dkc[m];
        }
        db = group4_sum(db);
        if (g == 0) s_db[row] = db;
        wrote = group4_sum(wrote);
        wrote = group_sum<16>(wrote);
        if (lane == 0) s_end[4 + w] = wrote;
        __syncthreads();
        if (w == 0) {
            double v = s_db[lane];
            if (lane == kC - 1)
                v += static_cast<double>(whole_exp(end)) * ((static_cast<double>(s_end[0]) + s_end[1]) + (static_cast<double>(s_end[2]) + s_end[3])) +
                     ((static_cast<double>(s_end[4]) + s_end[5]) + (static_cast<double>(s_end[6]) + s_end[7]));
#pragma unroll
            for (int d = 1; d < kC; d *= 2) {  // from the last token on
                const double o = __shfl_down(v, d);
                if (lane + d < kC) v += o;
            }
            if (lane < ch.len) a.dg[(ch.start + lane) * a.H + h] = static_cast<float>(v);
        }
    }
    // through the division by their lengths
    float qd = 0.0f, kd = 0.0f;
    f32x4 k4[KM], q4[KM];
#pragma unroll
    for (int m = 0; m < KM; ++m) {
        const bool in = in_t && a.norm && state_column(m, 4 * g) < K;
        k4[m] = rk * k_rows.four(row_at + state_column(m, 4 * g), in);
        q4[m] = rq * q_rows.four(row_at + state_column(m, 4 * g), in);
        qd = dot4(q4[m], dq_sum[m], qd);
        kd = dot4(k4[m], dk_sum[m], kd);
    }
    qd = group4_sum(qd);
    kd = group4_sum(kd);
    T* dqp = static_cast<T*>(a.dq) + (ch.start + row) * qk_stride + hg * a.K;
    T* dkp = static_cast<T*>(a.dk) + (ch.start + row) * qk_stride + hg * a.K;
#pragma unroll
    for (int m = 0; m < KM; ++m) {
        if (!in_t || state_column(m, 4 * g) >= K) continue;
        const f32x4 x = rq * (dq_sum[m] - qd * q4[m]), y = rk * (dk_sum[m] - kd * k4[m]);
        const float xs[4] = {x[0], x[1], x[2], x[3]}, ys[4] = {y[0], y[1], y[2], y[3]};
        store_row(dqp + state_column(m, 4 * g), xs);
        store_row(dkp + state_column(m, 4 * g), ys);
    }
}

template <typename T, int KP, int NW>
hipError_t launch_c(const GdrArgs& a, hipStream_t s) {
    const GdrLayout l(a.dtype, true);
    const int64_t parts = (a.V + 16 * NW - 1) / (16 * NW);
    const AdjointArgs k{a.q, a.k, a.dy, a.offsets, a.mats, a.dh_final, a.dv, a.dh0, a.adjoints, a.pulls,
                        a.T, a.N, a.T / a.N, a.G, a.H, a.K, a.V, parts, l.bytes, l.factors, l.nt, l.pt};
    gdr_adjoint_kernel<T, KP, NW><<<xcd_grid(a.N * a.H, parts), NW * 64, 0, s>>>(k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const GradArgs d{a.q, a.k, a.dy, a.g, a.beta, a.offsets, a.states, a.misses, a.adjoints, a.pulls, a.dq, a.dk, a.dg, a.dbeta,
                     a.T, a.N, a.T / a.N, a.G, a.H, a.K, a.V, 0, a.scale, a.norm};
    gdr_grad_kernel<T, KP><<<static_cast<uint32_t>(gdr_slots(a.T, a.N) * a.G), 256, 0, s>>>(d);
    return hipGetLastError();
}
template <typename T, int KP>
hipError_t launch_k(const GdrArgs& a, hipStream_t s) {
    if constexpr (sizeof(T) == 2 || KP == 64) {  // eight waves have 256 registers each, too few for float32 planes of 128
        if (a.V > 64 && a.N * a.H >= 128) return launch_c<T, KP, 8>(a, s);
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
