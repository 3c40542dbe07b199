// gdr_prep.hip -- what the gated delta rule's chunks can compute by themselves,
// before the chain over them.
//
// With b_i the sum of the chunk's log decays up to token i, G_ij = exp(b_i - b_j),
// q and k already scaled, u_j = beta_j e_j, S the state before the chunk:
//
//     e_i = v_i - exp(b_i) S k_i - sum_{j<i} A_ij u_j        A_ij = G_ij k_i . k_j
//     y_i = scale (exp(b_i) S q_i + sum_{j<=i} G_ij (q_i . k_j) u_j)
//
// so e = (1 + A beta)^-1 r with r = v - exp(b) S k.  The inverse is 1 + N beta
// with N strictly lower triangular and no division by beta: N = -A (1 + beta A)^-1,
// from (1 + A beta) N = -A by substitution, 16 x 16 blocks on the diagonal by
// lanes, the others as products of blocks with the float32 matrix instructions
// (substitution, and not a product of powers of A: those grow to 10^18 where
// keys repeat, and what is left of their sum then has no correct digit).
#include "gdr_common.h"

namespace mssm {
namespace {

using namespace gdrk;

constexpr int kPitch = kC + 4;  // floats of a row of a 64 x 64 matrix in LDS: 16-byte pieces, rows on different banks

struct PrepArgs {
    const void *q, *k;
    const float *g, *beta;
    const int32_t* offsets;
    uint8_t* mats;
    int64_t T, N, G, H, K, slot0;
    float scale;
    int norm;
    int64_t mat_bytes, at_n, at_p, at_f, at_nt, at_pt;
};

__device__ __forceinline__ f32x4 read4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// acc += (16 x 16 block of a at lds, rows of kPitch) * b, b's rows 4 g + r in the items r
__device__ __forceinline__ f32x4 block_product(const float* a, f32x4 b, f32x4 acc, int c, int g) {
    const f32x4 x = read4(a + c * kPitch + 4 * g);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], b[r], acc, 0, 0, 0);
    return acc;
}

// A workgroup: one chunk and one head of q and k, with all value heads that share it.
template <typename T, int KS, bool TRAIN, int P_PLANES>
__global__ __launch_bounds__(256) void gdr_prep_kernel(PrepArgs a) {
    __shared__ float sA[kC * kPitch], sN[kC * kPitch], sP[kC * kPitch];
    __shared__ float s_hi[kC], s_lo[kC], s_beta[kC], s_rk[kC], s_rq[kC];
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const int64_t head_g = blockIdx.x % a.G, slot = a.slot0 + blockIdx.x / a.G;
    const Chunk ch = chunk_of(a.offsets, slot, a.T, a.N);
    if (ch.len == 0) return;

    // K Kᵀ and Q Kᵀ: wave w has the rows 16 w .., its blocks of columns up to the diagonal
    const int64_t stride = a.G * a.K;
    const T* k0 = static_cast<const T*>(a.k) + ch.start * stride + head_g * a.K;
    const T* q0 = static_cast<const T*>(a.q) + ch.start * stride + head_g * a.K;
    f32x4 kk[4] = {}, qk[4] = {};
    {
        constexpr int PL = kPlanes<T>;
        const int row = 16 * w + c;
        Planes<PL> kw[KS], qw[KS];
        float k2 = 0.0f, q2 = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int64_t at = row * stride + s * 32 + 8 * g;
            const bool in = row < ch.len && s * 32 + 8 * g < a.K;
            kw[s] = load_planes(k0 + at, in);
            qw[s] = load_planes(q0 + at, in);
            k2 += sum_squares(kw[s]);
            q2 += sum_squares(qw[s]);
        }
        k2 += __shfl_xor(k2, 16); k2 += __shfl_xor(k2, 32);
        q2 += __shfl_xor(q2, 16); q2 += __shfl_xor(q2, 32);
        if (g == 0) {
            s_rk[row] = a.norm ? 1.0f / __builtin_sqrtf(k2 + kGdrNormEps) : 1.0f;
            s_rq[row] = a.norm ? 1.0f / __builtin_sqrtf(q2 + kGdrNormEps) : 1.0f;
        }
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
            if (jb > w) continue;
            const int col = 16 * jb + c;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const bool in = col < ch.len && s * 32 + 8 * g < a.K;
                const Planes<PL> kj = load_planes(k0 + col * stride + s * 32 + 8 * g, in);
                kk[jb] = mma(kw[s], kj, kk[jb]);
                qk[jb] = mma(qw[s], kj, qk[jb]);
            }
        }
    }
    // blocks above the diagonal stay zero
    for (int i = tid; i < kC * kPitch; i += 256) sA[i] = 0.0f, sN[i] = 0.0f, sP[i] = 0.0f;

    const int per = static_cast<int>(a.H / a.G);
    for (int hh = 0; hh < per; ++hh) {
        const int64_t h = head_g * per + hh;
        uint8_t* out = a.mats + (slot * a.H + h) * a.mat_bytes;
        __syncthreads();
        if (w == 0) {
            const bool in = lane < ch.len;
            const int64_t at = (ch.start + lane) * a.H + h;
            const float beta = in ? a.beta[at] : 0.0f;
            const double b = decays_since_start(a.g + ch.start * a.H + h, a.H, ch.len, lane);
            const double end = __shfl(b, kC - 1);
            const float hi = static_cast<float>(b), lo = static_cast<float>(b - hi);
            s_hi[lane] = hi; s_lo[lane] = lo; s_beta[lane] = beta;
            const float in_chunk = whole_exp(b);
            float* f = reinterpret_cast<float*>(out + a.at_f);
            f[lane] = in_chunk * s_rk[lane];                    // of S k
            f[kC + lane] = beta;
            f[2 * kC + lane] = whole_exp(end - b) * s_rk[lane];  // of k in the state's update
            f[3 * kC + lane] = a.scale * in_chunk * s_rq[lane];  // of S q
            f[4 * kC + lane] = whole_exp(end);                   // of S in the update
        }
        __syncthreads();
        // A and P; wave w's rows, item r: row 4 g + r
        float hi[4], lo[4], rk[4], rq[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * w + 4 * g + r;
            hi[r] = s_hi[i]; lo[r] = s_lo[i]; rk[r] = s_rk[i]; rq[r] = s_rq[i] * a.scale;
        }
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
            if (jb > w) continue;
            const int j = 16 * jb + c;
            const float hj = s_hi[j], lj = s_lo[j], rj = s_rk[j];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * w + 4 * g + r;
                const float d = decay_between(hi[r], lo[r], hj, lj) * rj;
                sA[i * kPitch + j] = i > j ? d * rk[r] * kk[jb][r] : 0.0f;
                sP[i * kPitch + j] = i >= j ? d * rq[r] * qk[jb][r] : 0.0f;
            }
        }
        __syncthreads();
        {  // diagonal block w of N, a column a lane: N_ic = -(A_ic + sum_{j<i} A_ij beta_j N_jc)
            const float* A = sA + 16 * w * kPitch + 16 * w;
            float m[16], n[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = A[i * kPitch + c];
#pragma unroll
                for (int j = 0; j < i; ++j) s = __builtin_fmaf(A[i * kPitch + j], m[j], s);
                n[i] = -s;
                m[i] = n[i] * s_beta[16 * w + i];
            }
            float* out_n = sN + 16 * w * kPitch + 16 * w;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i >> 2 == g) out_n[i * kPitch + c] = n[i];
        }
        __syncthreads();
        if (w < 3) {  // the blocks below: wave w's column of blocks
            const int j = w;
            f32x4 m[4];  // beta N of the rows so far
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i < j) continue;
                f32x4 beta;
#pragma unroll
                for (int r = 0; r < 4; ++r) beta[r] = s_beta[16 * i + 4 * g + r];
                f32x4 n;
                if (i == j) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) n[r] = sN[(16 * i + 4 * g + r) * kPitch + 16 * j + c];
                } else {
                    f32x4 x;
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[r] = sA[(16 * i + 4 * g + r) * kPitch + 16 * j + c];
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        if (k >= j && k < i) x = block_product(sA + 16 * i * kPitch + 16 * k, m[k], x, c, g);
                    n = -block_product(sN + 16 * i * kPitch + 16 * i, beta * x, x, c, g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) sN[(16 * i + 4 * g + r) * kPitch + 16 * j + c] = n[r];
                }
                m[i] = beta * n;
            }
        }
        __syncthreads();
        // out as operands
        auto put = [&](uint8_t* to, int block, auto planes) {
#pragma unroll
            for (int n = 0; n < static_cast<int>(sizeof(planes.p) / sizeof(planes.p[0])); ++n)
                *reinterpret_cast<u32x4*>(to + (n * kGdrBlocks + block) * kGdrBlockBytes + lane * 16) = planes.p[n];
        };
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int blk = w + 4 * b;  // 0 .. 5
            if (blk < kGdrBlocks) {
                const int rt = blk < 2 ? blk : blk / 2 + 1, ks = blk < 2 ? 0 : blk & 1;
                const int at = (16 * rt + c) * kPitch + 32 * ks + 4 * g;
                put(out + a.at_n, blk, split<3>(read4(sN + at), read4(sN + at + 16)));
                put(out + a.at_p, blk, split<P_PLANES>(read4(sP + at), read4(sP + at + 16)));
                if constexpr (TRAIN) {
                    const int rt2 = blk < 4 ? blk / 2 : blk - 2, ks2 = blk < 4 ? blk & 1 : 1;
                    float x[8], y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int t = (32 * ks2 + 4 * g + (i & 3) + (i >> 2) * 16) * kPitch + 16 * rt2 + c;
                        x[i] = sN[t];
                        y[i] = sP[t];
                    }
                    put(out + a.at_nt, blk, split<3>(x));
                    put(out + a.at_pt, blk, split<3>(y));
                }
            }
        }
    }
}

template <typename T, int KS>
void launch_t(const PrepArgs& k, bool train, uint32_t blocks, hipStream_t s) {
    constexpr int PP = sizeof(T) == 2 ? 2 : 3;
    if (train) gdr_prep_kernel<T, KS, true, PP><<<blocks, 256, 0, s>>>(k);
    else gdr_prep_kernel<T, KS, false, PP><<<blocks, 256, 0, s>>>(k);
}

}  // namespace

hipError_t launch_gdr_prep(const GdrArgs& a, hipStream_t s) {
    const GdrLayout l(a.dtype, a.train);
    const PrepArgs k{a.q, a.k, a.g, a.beta, a.offsets, a.mats, a.T, a.N, a.G, a.H, a.K, 0, a.scale, a.norm,
                     l.bytes, l.n, l.pm, l.factors, l.nt, l.pt};
    const uint32_t blocks = static_cast<uint32_t>(gdr_slots(a.T, a.N) * a.G);
    if (a.dtype == MSSM_F32) a.K <= 64 ? launch_t<float, 2>(k, a.train, blocks, s) : launch_t<float, 4>(k, a.train, blocks, s);
    else a.K <= 64 ? launch_t<uint16_t, 2>(k, a.train, blocks, s) : launch_t<uint16_t, 4>(k, a.train, blocks, s);
    return hipGetLastError();
}

}  // namespace mssm
