// gdr_fwd.hip -- the chain of the gated delta rule over a sequence's chunks
// (mssm_gdr_fwd, mssm_gdr_fwd_train; the equations are in gdr_prep.hip).
//
// The columns of the state's transpose (K x V), one for each value element, do
// not depend on one another, so each wave takes 16 or 32 of them through the
// whole sequence by itself: the state stays in its accumulators, and every
// product of the chain takes its float32 operand straight from the accumulators
// of the one before.  The other operands, q, k and the chunk's matrices, are
// shared by the waves of a workgroup.
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
    int64_t T, N, G, H, K, V, parts;
    int64_t mat_bytes, at_n, at_p, at_f;
};

// CT: tiles of 16 columns a wave.  Column l % 16 of tile t is value element CT (l % 16) + t of
// the wave's 16 CT, so that a lane's columns (and its rows of the transposed y) are neighbours.
template <typename T, int KP, int CT, bool TRAIN>
__global__ __launch_bounds__(256) void gdr_fwd_kernel(FwdArgs a) {
    constexpr int PL = kPlanes<T>, PP = sizeof(T) == 2 ? 2 : 3, KS = KP / 32;
    typedef RowTile<KP> Rows;
    typedef ColumnTile<KP> Columns;
    __shared__ __align__(16) uint8_t lds[PL * (2 * Rows::kBytes + Columns::kBytes)];
    uint8_t *lds_k = lds, *lds_q = lds_k + PL * Rows::kBytes, *lds_kt = lds_q + PL * Rows::kBytes;
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const int64_t part = blockIdx.x % a.parts, head = blockIdx.x / a.parts, h = head % a.H, n = head / a.H;
    const int64_t hg = h / (a.H / a.G);
    const int64_t v0 = (part * 4 + w) * 16 * CT;  // the wave's first value element
    const bool in_v = v0 + c * CT < a.V;          // this lane's columns
    const Span sp = span_of(a.offsets, n, a.T, a.N);
    const int64_t slot0 = first_slot(sp, n), chunks = (sp.len + kC - 1) / kC;

    f32x4 S[CT][KP / 16];
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int m = 0; m < KP / 16; ++m) {
            S[t][m] = f32x4{0, 0, 0, 0};
            if (a.h0 && in_v && 16 * m < a.K)
                S[t][m] = *reinterpret_cast<const f32x4*>(a.h0 + ((n * a.H + h) * a.V + v0 + c * CT + t) * a.K + 16 * m + 4 * g);
        }

    const int64_t qk_stride = a.G * a.K, v_stride = a.H * a.V;
    const T* kp = static_cast<const T*>(a.k) + sp.start * qk_stride + hg * a.K;
    const T* qp = static_cast<const T*>(a.q) + sp.start * qk_stride + hg * a.K;
    const T* vp = static_cast<const T*>(a.v) + sp.start * v_stride + h * a.V + v0;
    T* yp = static_cast<T*>(a.y) + sp.start * v_stride + h * a.V + v0;
    Patch<T, KP> pk, pq;
    auto fetch = [&](int64_t chunk) {
        const int len = static_cast<int>(imin64(kC, sp.len - chunk * kC));
        pk.load(kp + chunk * kC * qk_stride, qk_stride, len, static_cast<int>(a.K), tid);
        pq.load(qp + chunk * kC * qk_stride, qk_stride, len, static_cast<int>(a.K), tid);
    };
    if (chunks) fetch(0);
    for (int64_t chunk = 0; chunk < chunks; ++chunk) {
        const int len = static_cast<int>(imin64(kC, sp.len - chunk * kC));
        const uint8_t* mat = a.mats + ((slot0 + chunk) * a.H + h) * a.mat_bytes;
        const float* f = reinterpret_cast<const float*>(mat + a.at_f);
        const int64_t t0 = chunk * kC;
        __syncthreads();  // the chunk before is done with
        pk.store(lds_k, lds_kt, tid);
        pq.store(lds_q, nullptr, tid);
        __syncthreads();
        if (chunk + 1 < chunks) fetch(chunk + 1);
        if (v0 >= a.V) continue;  // only helps with the loads

        float val[16][CT];  // item 4 rt + r: token 16 rt + 4 g + r
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int t = (i >> 2) * 16 + 4 * g + (i & 3);
#pragma unroll
            for (int j = 0; j < CT; ++j) val[i][j] = 0.0f;
            if (t < len && in_v) load_values(vp + (t0 + t) * v_stride + c * CT, val[i]);
        }
        if constexpr (TRAIN) {
            if (in_v) {
#pragma unroll
                for (int t = 0; t < CT; ++t)
#pragma unroll
                    for (int m = 0; m < KP / 16; ++m)
                        if (16 * m < a.K)
                            *reinterpret_cast<f32x4*>(a.states + (((slot0 + chunk) * a.H + h) * a.V + v0 + c * CT + t) * a.K + 16 * m + 4 * g) = S[t][m];
            }
        }

        // S k (tokens in the rows) and S q (tokens in the columns)
        f32x4 X[CT][4] = {}, O[CT][4] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            Planes<3> st[CT];
#pragma unroll
            for (int t = 0; t < CT; ++t) st[t] = split<3>(S[t][2 * s], S[t][2 * s + 1]);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                const Planes<PL> kf = read_tile<Rows, PL>(lds_k, 16 * rt + c, 4 * s + g);
                const Planes<PL> qf = read_tile<Rows, PL>(lds_q, 16 * rt + c, 4 * s + g);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    X[t][rt] = mma(kf, st[t], X[t][rt]);
                    Planes<PP> so;
#pragma unroll
                    for (int i = 0; i < PP; ++i) so.p[i] = st[t].p[i];
                    O[t][rt] = mma(so, qf, O[t][rt]);
                }
            }
        }
        // e = r + N (beta r)
        f32x4 beta[4];
        Planes<3> m[CT][2];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 ek = *reinterpret_cast<const f32x4*>(f + 16 * rt + 4 * g);
            beta[rt] = *reinterpret_cast<const f32x4*>(f + kC + 16 * rt + 4 * g);
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) X[t][rt][r] = __builtin_fmaf(-ek[r], X[t][rt][r], val[4 * rt + r][t]);
        }
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int s = 0; s < 2; ++s) m[t][s] = split<3>(beta[2 * s] * X[t][2 * s], beta[2 * s + 1] * X[t][2 * s + 1]);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (block_of<true>(rt, s) < 0) continue;
                const Planes<3> nb = load_block<3>(mat + a.at_n, block_of<true>(rt, s), lane);
#pragma unroll
                for (int t = 0; t < CT; ++t) X[t][rt] = mma(nb, m[t][s], X[t][rt]);
            }
        if constexpr (TRAIN) {
            float* e = a.misses + ((slot0 + chunk) * a.H + h) * kC * a.V + v0 + c * CT;
            if (in_v) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x[CT];
#pragma unroll
                    for (int t = 0; t < CT; ++t) x[t] = X[t][i >> 2][i & 3];
                    store_values(e + ((i >> 2) * 16 + 4 * g + (i & 3)) * a.V, x);
                }
            }
        }
        // y = scale exp(b) S q + P u, and the state's update
        const float last = f[4 * kC];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const float eq = f[3 * kC + 16 * rt + c];
#pragma unroll
            for (int t = 0; t < CT; ++t) O[t][rt] *= eq, X[t][rt] *= beta[rt];  // X: u
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            Planes<PP> u[CT];
#pragma unroll
            for (int t = 0; t < CT; ++t) u[t] = split<PP>(X[t][2 * s], X[t][2 * s + 1]);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                if (block_of<true>(rt, s) < 0) continue;
                const Planes<PP> pb = load_block<PP>(mat + a.at_p, block_of<true>(rt, s), lane);
#pragma unroll
                for (int t = 0; t < CT; ++t) O[t][rt] = mma(u[t], pb, O[t][rt]);
            }
        }
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int i = 0; i < KP / 16; ++i) S[t][i] *= last;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const f32x4 d0 = *reinterpret_cast<const f32x4*>(f + 2 * kC + 32 * s + 4 * g),
                        d1 = *reinterpret_cast<const f32x4*>(f + 2 * kC + 32 * s + 16 + 4 * g);
            Planes<3> u[CT];
#pragma unroll
            for (int t = 0; t < CT; ++t) u[t] = split<3>(d0 * X[t][2 * s], d1 * X[t][2 * s + 1]);
#pragma unroll
            for (int i = 0; i < KP / 16; ++i) {
                const Planes<PL> kt = read_tile<Columns, PL>(lds_kt, 16 * i + c, 4 * s + g);
#pragma unroll
                for (int t = 0; t < CT; ++t) S[t][i] = mma(kt, u[t], S[t][i]);
            }
        }
        // row 4 g + r of tile t, column (token) 16 rt + c: value elements v0 + CT (4 g + r) + t
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            float out[4 * CT];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int t = 0; t < CT; ++t) out[r * CT + t] = O[t][rt][r];
            if (a.y && 16 * rt + c < len && v0 + 4 * CT * g < a.V) store_row(yp + (t0 + 16 * rt + c) * v_stride + 4 * CT * g, out);
        }
    }
    if (a.h_final && in_v) {
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int m = 0; m < KP / 16; ++m)
                if (16 * m < a.K)
                    *reinterpret_cast<f32x4*>(a.h_final + ((n * a.H + h) * a.V + v0 + c * CT + t) * a.K + 16 * m + 4 * g) = S[t][m];
    }
}

template <typename T, int KP, int CT, bool TRAIN>
hipError_t launch_v(const GdrArgs& a, hipStream_t s) {
    const GdrLayout l(a.dtype, a.train);
    const int64_t parts = (a.V + 64 * CT - 1) / (64 * CT);
    const FwdArgs k{a.q, a.k, a.v, a.offsets, a.mats, a.h0, a.y, a.h_final, a.states, a.misses,
                    a.T, a.N, a.G, a.H, a.K, a.V, parts, l.bytes, l.n, l.pm, l.factors};
    gdr_fwd_kernel<T, KP, CT, TRAIN><<<static_cast<uint32_t>(a.N * a.H * parts), 256, 0, s>>>(k);
    return hipGetLastError();
}
template <typename T, int KP, int CT>
hipError_t launch_c(const GdrArgs& a, hipStream_t s) {
    return a.train ? launch_v<T, KP, CT, true>(a, s) : launch_v<T, KP, CT, false>(a, s);
}
template <typename T, int KP>
hipError_t launch_k(const GdrArgs& a, hipStream_t s) {
    if constexpr (sizeof(T) == 2 || KP == 64) {  // float32 planes of 128 columns leave no registers for a second tile
        if (a.N * a.H >= 128 && a.V > 64) return launch_c<T, KP, 2>(a, s);
    }
    return launch_c<T, KP, 1>(a, s);
}
template <typename T>
hipError_t launch_t(const GdrArgs& a, hipStream_t s) {
    return a.K <= 64 ? launch_k<T, 64>(a, s) : launch_k<T, 128>(a, s);
}

}  // namespace

hipError_t launch_gdr_fwd(const GdrArgs& a, hipStream_t s) {
    return a.dtype == MSSM_F32 ? launch_t<float>(a, s) : launch_t<uint16_t>(a, s);
}

}  // namespace mssm
