// gdr_prep.hip -- what the gated delta rule's chunks can compute by themselves,
// before the chain over them.
//
// With b_i the sum of the chunk's log decays up to token i, G_ij = exp(b_i - b_j),
// q and k already scaled, u_j = beta_j e_j, S the state before the chunk:
//
//     e_i = v_i - exp(b_i) S k_i - sum_{j<i} A_ij u_j        A_ij = G_ij k_i . k_j
//     y_i = scale exp(b_i) S q_i + sum_{j<=i} P_ij u_j       P_ij = scale G_ij q_i . k_j
//
// so e = (1 + A beta)^-1 r with r = v - exp(b) S k.  The inverse is 1 + N beta
// with N strictly lower triangular and no division by beta: N = -A (1 + beta A)^-1,
// from (1 + A beta) N = -A by substitution (and not as a product of powers of A:
// those grow to 10^18 where keys repeat, and what is left of their sum then has
// no correct digit).
//
// A wave has a chunk and head by itself, without LDS or barriers but for the
// tokens' factors.  Every 16 x 16 block is held in the accumulators' layout
// both as it is and transposed: the layout of a block (row 4 g + r, column c) is
// that of the transposed block as a matrix operand, so products need no exchange,
// and swapping the operands gives the transposed product.  The blocks on the
// diagonal are solved by lanes, all four at a time, a column a lane, with the
// matrix's elements broadcast within 16 lanes by DPP.
//
// Measured: 16,384 tokens, 40 heads, key dim 128, bfloat16, 124 us: 431 MB at 3.5
// TB/s, 76 % of them written (N and P, 30 KB a chunk and head); vector instructions
// are busy for half of it, matrix instructions for a fifth.  8,192 tokens of 32
// heads take 57 us, 82 us with the transposes for the backward.
#include "gdr_common.h"

namespace mssm {
namespace {

using namespace gdrk;

struct PrepArgs {
    const void *q, *k;
    const float *g, *beta;
    const int32_t* offsets;
    uint8_t* mats;
    int64_t T, N, each, cells;  // cells: (slot, head) pairs
    uint32_t G, H, K;
    float scale;
    int norm;
    int64_t mat_bytes, at_n, at_p, at_f, at_nt, at_pt;
};

// acc += a b of 16 x 16 float32 blocks: a transposed and b in the accumulators' layout
__device__ __forceinline__ f32x4 block_product(f32x4 a, f32x4 b, f32x4 acc) {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], acc, 0, 0, 0);
    return acc;
}

// x[i] of lane group g and x[g] of lane group i change places, i and g = 0 .. 3
__device__ __forceinline__ void swap_groups(f32x4 (&x)[4]) {
    auto swap = [](auto op, f32x4& a, f32x4& b) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const auto v = op(__float_as_uint(a[r]), __float_as_uint(b[r]));
            a[r] = __uint_as_float(v[0]);
            b[r] = __uint_as_float(v[1]);
        }
    };
    auto halves = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_permlane32_swap(a, b, false, false); };
    auto rows = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_permlane16_swap(a, b, false, false); };
    swap(halves, x[0], x[2]);
    swap(halves, x[1], x[3]);
    swap(rows, x[0], x[1]);
    swap(rows, x[2], x[3]);
}

// acc[i] += (lane J of the row's c[i]) * h for i = FROM .. TO - 1.  A DPP instruction
// may read no register that either of the two instructions before it wrote: each
// statement waits at its start, and its own accumulators are read once.
template <int J, int FROM, int TO>
__device__ __forceinline__ void fmac_row_lane(float (&acc)[16], const float (&c)[16], float h) {
    if constexpr (TO - FROM >= 4) {
        asm("s_nop 1\n\t"
            "v_fmac_f32_dpp %0, %4, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"
            "v_fmac_f32_dpp %1, %5, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"
            "v_fmac_f32_dpp %2, %6, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"
            "v_fmac_f32_dpp %3, %7, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf bound_ctrl:1"
            : "+&v"(acc[FROM]), "+&v"(acc[FROM + 1]), "+&v"(acc[FROM + 2]), "+&v"(acc[FROM + 3])
            : "v"(c[FROM]), "v"(c[FROM + 1]), "v"(c[FROM + 2]), "v"(c[FROM + 3]), "v"(h), "i"(J));
        fmac_row_lane<J, FROM + 4, TO>(acc, c, h);
    } else if constexpr (FROM < TO) {
        acc[FROM] = fmac_row_bcast<J>(acc[FROM], c[FROM], h);
        fmac_row_lane<J, FROM + 1, TO>(acc, c, h);
    }
}

// (1 + A beta) N = -A of 16 x 16, A strictly lower triangular: on entry x[i] is A's
// row i, a column a lane, on return N's.  `beta`: of the lane's own token.
template <int J>
__device__ __forceinline__ void solve_down(const float (&a)[16], float (&s)[16], float beta) {
    if constexpr (J < 15) {
        const float m = -s[J] * row_bcast<J>(beta);
        fmac_row_lane<J, J + 1, 16>(s, a, m);
        solve_down<J + 1>(a, s, beta);
    }
}
// The same transposed, (1 + Aᵀ beta) Nᵀ = -Aᵀ, Aᵀ strictly upper triangular.
template <int J>
__device__ __forceinline__ void solve_up(const float (&a)[16], float (&s)[16], float beta) {
    if constexpr (J > 0) {
        const float m = -s[J] * row_bcast<J>(beta);
        fmac_row_lane<J, 0, J>(s, a, m);
        solve_up<J - 1>(a, s, beta);
    }
}
template <bool DOWN>
__device__ __forceinline__ void solve(f32x4 (&x)[4], float beta) {
    swap_groups(x);  // the block on the diagonal of the lane's group, all of its column
    float a[16], s[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i] = s[i] = x[i >> 2][i & 3];
    if constexpr (DOWN) solve_down<0>(a, s, beta);
    else solve_up<15>(a, s, beta);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i >> 2][i & 3] = -s[i];
    swap_groups(x);
}

constexpr int kWaves = 4;

template <typename T, int KS, bool TRAIN>
__global__ __launch_bounds__(64 * kWaves, sizeof(T) == 4 && TRAIN ? 1 : 2) void gdr_prep_kernel(PrepArgs a) {
    constexpr int PL = kPlanes<T>;
    __shared__ __align__(16) float shared[kWaves][8][kC];
    const int lane = threadIdx.x & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const int64_t cell = static_cast<int64_t>(blockIdx.x) * kWaves + w;
    if (cell >= a.cells) return;
    const uint32_t slot = static_cast<uint32_t>(cell) / a.H, h = static_cast<uint32_t>(cell) - slot * a.H, hg = h / (a.H / a.G);
    const Chunk ch = chunk_of(a.offsets, slot, a.T, a.N, a.each);
    if (ch.len == 0) return;
    uint8_t* out = a.mats + cell * a.mat_bytes;
    float* f = reinterpret_cast<float*>(out + a.at_f);

    // the tokens' decays, a token a lane, under way with the first rows
    const float g_log = View<float>(a.g + ch.start * a.H + h).one(lane * a.H, lane < ch.len);
    const float beta = View<float>(a.beta + ch.start * a.H + h).one(lane * a.H, lane < ch.len);

    // K Kᵀ, block rows above columns (kk[i][j], i >= j) and transposed (kt[j][i]); K Qᵀ (kq[j][i]), Q Kᵀ (qk[i][j])
    f32x4 kk[4][4] = {}, kt[4][4] = {}, kq[4][4] = {}, qk[4][4] = {};
    float k2[4] = {}, q2[4] = {};
    {
        const uint32_t stride = a.G * a.K;
        const View<T> k0(static_cast<const T*>(a.k) + ch.start * stride + hg * a.K);
        const View<T> q0(static_cast<const T*>(a.q) + ch.start * stride + hg * a.K);
#pragma unroll 1
        for (int s = 0; s < KS; ++s) {
            if (s * 32u >= a.K) break;
            Planes<PL> kf[4], qf[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t row = 16 * t + c, col = s * 32 + 8 * g;
                const bool in = static_cast<int>(row) < ch.len && col < a.K;
                kf[t] = k0.planes(row * stride + col, in);
                qf[t] = q0.planes(row * stride + col, in);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                k2[t] += sum_squares(kf[t]);
                q2[t] += sum_squares(qf[t]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j) {
                    kk[i][j] = mma(kf[i], kf[j], kk[i][j]);
                    if (j < i) kt[j][i] = mma(kf[j], kf[i], kt[j][i]);
                    kq[j][i] = mma(kf[j], qf[i], kq[j][i]);
                    if constexpr (TRAIN) qk[i][j] = mma(qf[i], kf[j], qk[i][j]);
                }
        }
    }
    // 1 / length, of row 16 t + c in every group
    float rk = 1.0f, rq = 1.0f;
    if (a.norm) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            k2[t] += __shfl_xor(k2[t], 16); k2[t] += __shfl_xor(k2[t], 32);
            q2[t] += __shfl_xor(q2[t], 16); q2[t] += __shfl_xor(q2[t], 32);
        }
        const float kl = g == 0 ? k2[0] : g == 1 ? k2[1] : g == 2 ? k2[2] : k2[3];  // of the lane's own token
        const float ql = g == 0 ? q2[0] : g == 1 ? q2[1] : g == 2 ? q2[2] : q2[3];
        rk = 1.0f / __builtin_sqrtf(kl + kGdrNormEps);
        rq = 1.0f / __builtin_sqrtf(ql + kGdrNormEps);
    }
    const double b = decays_since_start(g_log, lane);
    // Between blocks a decay is the product of three, none above 1: from the row's
    // block's start, over the blocks between, to the column's block's end.
    const double end = __shfl(b, kC - 1), block_end = __shfl(b, lane | 15);
    const double last_before = __shfl(b, (lane & 48) - 1 & 63);  // by all lanes: the lanes asked have to be there
    const double before = lane < 16 ? 0.0 : last_before;
    const float in_chunk = whole_exp(b), from_start = whole_exp(b - before), to_block_end = whole_exp(block_end - b);
    const float hi = static_cast<float>(b), lo = static_cast<float>(b - hi);
    float(&sh)[8][kC] = shared[w];
    sh[0][lane] = hi; sh[1][lane] = lo; sh[2][lane] = rk; sh[3][lane] = rq * a.scale;
    sh[4][lane] = from_start; sh[5][lane] = to_block_end; sh[6][lane] = beta;
    f[lane] = in_chunk * rk;                        // of S k
    f[kC + lane] = beta;
    f[2 * kC + lane] = whole_exp(end - b) * rk;     // of k in the state's update
    f[3 * kC + lane] = a.scale * in_chunk * rq;     // of S q
    f[4 * kC + lane] = whole_exp(end);              // of S in the update
    const double e0 = __shfl(b, 15), e1 = __shfl(b, 31), e2 = __shfl(b, 47);
    const float over1 = whole_exp(e1 - e0), over2 = whole_exp(e2 - e1), over12 = whole_exp(e2 - e0);
    wave_handoff();

    auto row4 = [&](int n, int t) { return *reinterpret_cast<const f32x4*>(&sh[n][16 * t + 4 * g]); };
    f32x4 beta4[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) beta4[t] = row4(6, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // below the diagonal: rows i, columns j, and transposed
        const f32x4 row_k = row4(4, i) * row4(2, i), row_q = row4(4, i) * row4(3, i);
        const float col_k = sh[4][16 * i + c] * sh[2][16 * i + c], col_q = sh[4][16 * i + c] * sh[3][16 * i + c];
#pragma unroll
        for (int j = 0; j < i; ++j) {
            const float over = i - j == 1 ? 1.0f : i == 2 ? over1 : j == 1 ? over2 : over12;
            const float col = sh[5][16 * j + c] * sh[2][16 * j + c] * over;
            const f32x4 row = row4(5, j) * row4(2, j) * over;
            kk[i][j] *= row_k * col;
            kt[j][i] *= row * col_k;
            kq[j][i] *= row * col_q;
            if constexpr (TRAIN) qk[i][j] *= row_q * col;
        }
        // on it
        const f32x4 hr = row4(0, i), lr = row4(1, i), kr = row4(2, i), qr = row4(3, i);
        const float hc = sh[0][16 * i + c], lc = sh[1][16 * i + c], kc = sh[2][16 * i + c], qc = sh[3][16 * i + c];
        f32x4 x = kk[i][i];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 4 * g + r;
            const float d = (hr[r] - hc) + (lr[r] - lc);  // row over column
            const float down = fast_exp2(row >= c ? d * kLog2e : 0.0f), up = fast_exp2(row <= c ? -d * kLog2e : 0.0f);
            kk[i][i][r] = row > c ? x[r] * down * kr[r] * kc : 0.0f;
            kt[i][i][r] = row < c ? x[r] * up * kr[r] * kc : 0.0f;
            kq[i][i][r] = row <= c ? kq[i][i][r] * up * kr[r] * qc : 0.0f;
            if constexpr (TRAIN) qk[i][i][r] = row >= c ? qk[i][i][r] * down * qr[r] * kc : 0.0f;
        }
    }
    auto put = [&](int64_t to, int block, auto planes) { store_block(out + to, block, lane, planes); };
    const f32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (block_of<true>(i, s) >= 0) put(a.at_p, block_of<true>(i, s), words_of(kq[2 * s][i], 2 * s + 1 <= i ? kq[2 * s + 1][i] : zero));
            if constexpr (TRAIN)
                if (block_of<false>(i, s) >= 0) put(a.at_pt, block_of<false>(i, s), split<3>(2 * s >= i ? qk[2 * s][i] : zero, qk[2 * s + 1][i]));
        }
    // N, in place of A's blocks on the diagonal first; kk: N, kt: Nᵀ
    f32x4 dn[4], dt[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dn[i] = kk[i][i], dt[i] = kt[i][i];
    solve<true>(dn, beta);
    solve<false>(dt, beta);
    f32x4 n[4][4], nt[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        n[j][j] = dn[j];
        nt[j][j] = dt[j];
        f32x4 m[4];  // beta N of this column of blocks
        m[j] = beta4[j] * dn[j];
#pragma unroll
        for (int i = j + 1; i < 4; ++i) {
            f32x4 x = kk[i][j], xt = kt[j][i];
#pragma unroll
            for (int k = j; k < i; ++k) {
                x = block_product(kt[k][i], m[k], x);
                xt = block_product(m[k], kt[k][i], xt);
            }
            const f32x4 xb = beta4[i] * x;
            n[i][j] = -block_product(dt[i], xb, x);
            nt[j][i] = -block_product(xb, dt[i], xt);
            m[i] = beta4[i] * n[i][j];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (block_of<true>(i, s) >= 0) put(a.at_n, block_of<true>(i, s), split<3>(nt[2 * s][i], 2 * s + 1 <= i ? nt[2 * s + 1][i] : zero));
            if constexpr (TRAIN)
                if (block_of<false>(i, s) >= 0) put(a.at_nt, block_of<false>(i, s), split<3>(2 * s >= i ? n[2 * s][i] : zero, n[2 * s + 1][i]));
        }
}

template <typename T, int KS>
void launch_t(const PrepArgs& k, bool train, uint32_t blocks, hipStream_t s) {
    if (train) gdr_prep_kernel<T, KS, true><<<blocks, 64 * kWaves, 0, s>>>(k);
    else gdr_prep_kernel<T, KS, false><<<blocks, 64 * kWaves, 0, s>>>(k);
}

}  // namespace

hipError_t launch_gdr_prep(const GdrArgs& a, hipStream_t s) {
    const GdrLayout l(a.train);
    const int64_t cells = gdr_slots(a.T, a.N) * a.H;
    const PrepArgs k{a.q, a.k, a.g, a.beta, a.offsets, a.mats, a.T, a.N, a.T / a.N, cells, static_cast<uint32_t>(a.G), static_cast<uint32_t>(a.H),
                     static_cast<uint32_t>(a.K), a.scale, a.norm, l.bytes, l.n, l.pm, l.factors, l.nt, l.pt};
    const uint32_t blocks = static_cast<uint32_t>((cells + kWaves - 1) / kWaves);
    if (a.dtype == MSSM_F32) a.K <= 64 ? launch_t<float, 2>(k, a.train, blocks, s) : launch_t<float, 4>(k, a.train, blocks, s);
    else a.K <= 64 ? launch_t<uint16_t, 2>(k, a.train, blocks, s) : launch_t<uint16_t, 4>(k, a.train, blocks, s);
    return hipGetLastError();
}

}  // namespace mssm
