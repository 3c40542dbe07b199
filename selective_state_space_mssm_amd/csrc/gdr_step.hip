// gdr_step.hip -- one token of the gated delta rule a row, states in place
// (mssm_gdr_step).
//
// The rows of a state (V, K) are independent: with S k and S q of the old row,
//     e = v - a S k,   u = beta e,   y = scale (a S q + u (k . q)),   S' = a S + u k,
// so a row is read once, needs two sums at the same time, and is written once.
// Sixteen lanes have a row, 16 bytes a lane and load; sums by DPP.  Bound by memory:
// 256 rows of 40 heads of 128 x 128 take 255 us, 5.3 TB/s; 4 rows 4 us, a launch.
#include "device_common.h"
#include "gdr.h"

namespace mssm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct StepArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    const int32_t* slots;
    float* state;
    void* y;
    int64_t row0, rows, pool, G, H, K, V, parts;
    float scale;
    int norm;
};

__device__ __forceinline__ f32x4 load_quad(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load_quad(const uint16_t* p) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    return f32x4{bf16_lo(a.x), bf16_hi(a.x), bf16_lo(a.y), bf16_hi(a.y)};
}
__device__ __forceinline__ float dot(f32x4 a, f32x4 b, float s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __builtin_fmaf(a[i], b[i], s);
    return s;
}

// The next row behind `row` with this slot (rows if none); all lanes get it.
__device__ __forceinline__ int64_t next_row(const int32_t* slots, int64_t rows, int64_t row, int32_t slot, int lane) {
    for (int64_t r = row + 1; r < rows; r += 64) {
        const uint64_t hit = __ballot(r + lane < rows && slots[r + lane] == slot);
        if (hit) return r + __builtin_ctzll(hit);
    }
    return rows;
}

// QN: quads of a row that a lane has (K up to 64 QN); RI: rows of the state that
// a 16-lane group has, all loaded before the first is used.
template <typename T, int QN, int RI>
__global__ __launch_bounds__(256) void gdr_step_kernel(StepArgs a) {
    const int lane = threadIdx.x & 63, c = lane & 15;
    const int64_t part = blockIdx.x % a.parts, head = blockIdx.x / a.parts, h = head % a.H, hg = h / (a.H / a.G);
    int64_t row = a.row0 + head / a.H;
    const int64_t v0 = (part * 16 + (threadIdx.x >> 4)) * RI;
    const T *q = static_cast<const T*>(a.q), *k = static_cast<const T*>(a.k), *v = static_cast<const T*>(a.v);
    T* y = static_cast<T*>(a.y);
    int32_t slot = static_cast<int32_t>(row);
    if (a.slots) {
        slot = a.slots[row];
        if (slot < 0 || slot >= a.pool) {
#pragma unroll
            for (int i = 0; i < RI; ++i)
                if (c == 0 && v0 + i < a.V) store_act(y, (row * a.H + h) * a.V + v0 + i, 0.0f);
            return;
        }
    }
    float* s0 = a.state + ((slot * a.H + h) * a.V + v0) * a.K;
    f32x4 S[RI][QN];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int n = 0; n < QN; ++n) {
            const int col = 64 * n + 4 * c;
            S[i][n] = v0 + i < a.V && col < a.K ? load_quad(s0 + i * a.K + col) : f32x4{0, 0, 0, 0};
        }
    if (a.slots && next_row(a.slots, row, -1, slot, lane) < row) return;  // an earlier row takes this one along
    for (;;) {
        const T *qr = q + (row * a.G + hg) * a.K, *kr = k + (row * a.G + hg) * a.K;
        f32x4 kq[QN], qq[QN];
        float k2 = 0.0f, q2 = 0.0f, both = 0.0f;
#pragma unroll
        for (int n = 0; n < QN; ++n) {
            const int col = 64 * n + 4 * c;
            kq[n] = col < a.K ? load_quad(kr + col) : f32x4{0, 0, 0, 0};
            qq[n] = col < a.K ? load_quad(qr + col) : f32x4{0, 0, 0, 0};
            k2 = dot(kq[n], kq[n], k2);
            q2 = dot(qq[n], qq[n], q2);
        }
        if (a.norm) {
            const float rk = 1.0f / __builtin_sqrtf(group_sum<16>(k2) + kGdrNormEps);
            const float rq = 1.0f / __builtin_sqrtf(group_sum<16>(q2) + kGdrNormEps);
#pragma unroll
            for (int n = 0; n < QN; ++n) kq[n] *= rk, qq[n] *= rq;
        }
#pragma unroll
        for (int n = 0; n < QN; ++n) both = dot(kq[n], qq[n], both);
        both = group_sum<16>(both);
        const float gl = a.g[row * a.H + h], beta = a.beta[row * a.H + h];
        const float decay = expf(gl < kGdrLeast ? kGdrLeast : gl);
        float val[RI], sk[RI], sq[RI];
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            val[i] = v0 + i < a.V ? load_act(v, (row * a.H + h) * a.V + v0 + i) : 0.0f;
            sk[i] = sq[i] = 0.0f;
#pragma unroll
            for (int n = 0; n < QN; ++n) sk[i] = dot(S[i][n], kq[n], sk[i]), sq[i] = dot(S[i][n], qq[n], sq[i]);
        }
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            sk[i] = group_sum<16>(sk[i]);
            sq[i] = group_sum<16>(sq[i]);
            const float u = beta * __builtin_fmaf(-decay, sk[i], val[i]);
            const float out = a.scale * __builtin_fmaf(decay, sq[i], u * both);
#pragma unroll
            for (int n = 0; n < QN; ++n) S[i][n] = decay * S[i][n] + u * kq[n];
            if (c == 0 && v0 + i < a.V) store_act(y, (row * a.H + h) * a.V + v0 + i, out);
        }
        if (!a.slots) break;
        row = next_row(a.slots, a.rows, row, slot, lane);
        if (row >= a.rows) break;
    }
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int n = 0; n < QN; ++n) {
            const int col = 64 * n + 4 * c;
            if (v0 + i < a.V && col < a.K) *reinterpret_cast<f32x4*>(s0 + i * a.K + col) = S[i][n];
        }
}

template <typename T, int QN, int RI>
void launch_r(const GdrStepArgs& a, hipStream_t s) {
    StepArgs k{a.q, a.k, a.v, a.g, a.beta, a.slots, a.state, a.y, 0, a.rows, a.pool, a.G, a.H, a.K, a.V,
               (a.V + 16 * RI - 1) / (16 * RI), a.scale, a.norm};
    // a launch has fewer than 2^32 threads: as many rows at a time as fit
    const int64_t most = (int64_t{1} << 23) / (a.H * k.parts);  // heads are at most 2^20, parts 8
    for (k.row0 = 0; k.row0 < a.rows; k.row0 += most)
        gdr_step_kernel<T, QN, RI><<<static_cast<uint32_t>(imin64(most, a.rows - k.row0) * a.H * k.parts), 256, 0, s>>>(k);
}
template <typename T>
void launch_t(const GdrStepArgs& a, hipStream_t s) {
    a.K <= 64 ? launch_r<T, 1, 4>(a, s) : launch_r<T, 2, 4>(a, s);
}

}  // namespace

hipError_t launch_gdr_step(const GdrStepArgs& a, hipStream_t s) {
    a.dtype == MSSM_F32 ? launch_t<float>(a, s) : launch_t<uint16_t>(a, s);
    return hipGetLastError();
}

}  // namespace mssm
