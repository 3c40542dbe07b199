// lora.hip -- low-rank adapters of many requests beside a shared projection
// (mssm_lora): y[m] += scale[i] (x[m] A_iᵀ) B_iᵀ with i = index[m].
//
// Two launches, down to the rank and up again; what lies between is float32 in
// the workspace.  Many rows: tiles of 16 or 64 rows on the matrix cores, each
// tile once for every adapter that its rows name (packed requests: one or two),
// the other rows' results unused.  Few rows: a row for itself, by dot products,
// since each mostly has an adapter of its own and its weights are read once.
// y is read and written once, rounded once.
#include "block.h"
#include "planes.h"

namespace mssm {
namespace {

struct LoraKernelArgs {
    const void* x;
    const float* x_scale;
    const void *a, *b;
    const float* scale;
    const int32_t* index;
    void* y;
    float* inner;  // (splits, M, RP)
    int64_t M, K, N, R, RP, S;
    int splits;
    int64_t step;  // of K, for each split
};

// ---- eight neighbouring elements of a row, wherever it starts ----------------------

template <typename V> struct __attribute__((packed, aligned(1))) Loose { V v; };

template <int N>
__device__ __forceinline__ Planes<N> widen(const float (&x)[8]) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i];
    return split<N>(v);
}
__device__ __forceinline__ void to_floats(u32x4 q, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(q[i]), v[2 * i + 1] = bf16_hi(q[i]);
}
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const uint16_t* p) { return load_act(p, 0); }
__device__ __forceinline__ float load_one(const uint8_t* p) { return __builtin_amdgcn_cvt_f32_fp8(*p, 0); }
__device__ __forceinline__ void load_eight(const float* p, float (&v)[8]) {
    const f32x4 a = reinterpret_cast<const Loose<f32x4>*>(p)->v, b = reinterpret_cast<const Loose<f32x4>*>(p + 4)->v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
__device__ __forceinline__ void load_eight(const uint16_t* p, float (&v)[8]) { to_floats(reinterpret_cast<const Loose<u32x4>*>(p)->v, v); }
__device__ __forceinline__ void load_eight(const uint8_t* p, float (&v)[8]) {
    const u32x2 q = reinterpret_cast<const Loose<u32x2>*>(p)->v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q[i]), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q[i]), true);
        v[4 * i] = lo[0]; v[4 * i + 1] = lo[1]; v[4 * i + 2] = hi[0]; v[4 * i + 3] = hi[1];
    }
}
// Elements k .. k + 7 of a row of `end`; zeros behind its end.
template <typename T>
__device__ __forceinline__ void load_part(const T* row, int64_t k, int64_t end, float (&v)[8]) {
    if (k + 8 <= end) {
        load_eight(row + k, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k + i < end ? load_one(row + k + i) : 0.0f;
    }
}
// Planes of the type: bfloat16 and e4m3 (widened, which is exact) are one.
template <typename T> constexpr int kInner = sizeof(T) == 4 ? 3 : 1;
template <typename T>
__device__ __forceinline__ Planes<kInner<T>> load_operand(const T* row, int64_t k, int64_t end) {
    if constexpr (sizeof(T) == 2) {
        if (k + 8 <= end) {
            Planes<1> out;
            out.p[0] = reinterpret_cast<const Loose<u32x4>*>(row + k)->v;
            return out;
        }
    }
    float v[8];
    load_part(row, k, end, v);
    return split<kInner<T>>(v);
}

// ---- few rows ---------------------------------------------------------------------

__device__ __forceinline__ float wave_sum(float v) {
    v = group_sum<16>(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// A wave: one row and one of its adapter's rank.
template <typename X, typename W>
__global__ __launch_bounds__(256) void lora_row_down_kernel(LoraKernelArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t m = blockIdx.x, r = blockIdx.y * 4 + wave_id();
    const int32_t i = a.index[m];
    if (i < 0 || i >= a.S || r >= a.R) return;
    const X* x = static_cast<const X*>(a.x) + m * a.K;
    const W* w = static_cast<const W*>(a.a) + (i * a.R + r) * a.K;
    float s = 0.0f;
    for (int64_t k = lane * 8; k < a.K; k += 512) {
        float p[8], q[8];
        load_part(x, k, a.K, p);
        load_part(w, k, a.K, q);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(p[j], q[j], s);
    }
    s = wave_sum(s);
    if (sizeof(X) == 1) s *= a.x_scale[m];
    if (a.scale) s *= a.scale[i];
    if (lane == 0) a.inner[m * a.RP + r] = s;
}

// A thread: one output.
template <typename W, typename Y>
__global__ __launch_bounds__(256) void lora_row_up_kernel(LoraKernelArgs a) {
    const int64_t m = blockIdx.x, n = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x;
    const int32_t i = a.index[m];
    if (i < 0 || i >= a.S || n >= a.N) return;
    Y* y = static_cast<Y*>(a.y) + m * a.N + n;
    const W* w = static_cast<const W*>(a.b) + (i * a.N + n) * a.R;
    const float* t = a.inner + m * a.RP;
    float s = 0.0f;
    for (int64_t r = 0; r < a.R; r += 8) {
        float q[8];
        load_part(w, r, a.R, q);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(r + j < a.R ? t[r + j] : 0.0f, q[j], s);
    }
    store_act(y, 0, load_act(y, 0) + s);
}

// ---- tiles ------------------------------------------------------------------------

// The adapters that the rows of a tile name, one after the other: f(adapter, mask of its rows).
template <int ROWS, typename F>
__device__ __forceinline__ void each_adapter(const LoraKernelArgs& a, int64_t m0, int lane, F f) {
    const int32_t mine = lane < ROWS && m0 + lane < a.M ? a.index[m0 + lane] : -1;
    uint64_t todo = __ballot(mine >= 0 && mine < a.S);
    while (todo) {
        const int32_t i = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
        const uint64_t same = __ballot(mine == i);
        f(static_cast<int64_t>(i), same);
        todo &= ~same;
    }
}

// 16 MT rows and the whole rank; the four waves take every fourth 32 of K (of this split's part).
template <typename X, typename W, int RT, int MT>
__global__ __launch_bounds__(256) void lora_down_kernel(LoraKernelArgs a) {
    __shared__ f32x4 part[4][RT * MT][64];
    const int lane = threadIdx.x & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16 * MT, k0 = blockIdx.y * a.step, k1 = imin64(a.K, k0 + a.step);
    each_adapter<16 * MT>(a, m0, lane, [&](int64_t i, uint64_t same) {
        f32x4 acc[RT][MT] = {};
        const X* x = static_cast<const X*>(a.x);
        const W* wa = static_cast<const W*>(a.a) + i * a.R * a.K;
        for (int64_t k = k0 + w * 32 + g * 8; k - g * 8 < k1; k += 128) {
            Planes<kInner<X>> xf[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t m = m0 + 16 * t + c;
                xf[t] = load_operand(x + (m < a.M ? m : a.M - 1) * a.K, k, k1);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int64_t row = 16 * r + c;
                const auto wf = load_operand(wa + (row < a.R ? row : a.R - 1) * a.K, k, k1);
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[r][t] = mma(wf, xf[t], acc[r][t]);
            }
        }
        __syncthreads();  // the sums of the adapter before are read
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t) part[w][r * MT + t][lane] = acc[r][t];
        __syncthreads();
        const float s = a.scale ? a.scale[i] : 1.0f;
        for (int q = w; q < RT * MT; q += 4) {
            f32x4 v = (part[0][q][lane] + part[1][q][lane]) + (part[2][q][lane] + part[3][q][lane]);
            const int row = 16 * (q % MT) + c;
            if (!(same >> row & 1)) continue;
            if (sizeof(X) == 1) v *= a.x_scale[m0 + row];
            *reinterpret_cast<f32x4*>(a.inner + (blockIdx.y * a.M + m0 + row) * a.RP + 16 * (q / MT) + 4 * g) = v * s;
        }
    });
}

// A wave: 16 MT rows and 64 columns; row 4 g + r of tile j is column 16 g + 4 j + r,
// so that a lane has 16 neighbours of a row of y.
template <typename W, typename Y, int RS, int MT>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraKernelArgs a) {
    constexpr int PT = sizeof(Y) == 2 && sizeof(W) == 2 ? 2 : 3;  // planes of the inner values
    const int lane = threadIdx.x & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16 * MT, n0 = (static_cast<int64_t>(blockIdx.y) * 4 + w) * 64;
    if (n0 >= a.N) return;
    f32x4 acc[MT][4];
    uint64_t used = 0;
    Y* y = static_cast<Y*>(a.y);
    const int64_t n = n0 + 16 * g;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t m = m0 + 16 * t + c;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[t][j][r] = m < a.M && n + 4 * j + r < a.N ? load_act(y, m * a.N + n + 4 * j + r) : 0.0f;
    }
    each_adapter<16 * MT>(a, m0, lane, [&](int64_t i, uint64_t same) {
        used |= same;
        const W* wb = static_cast<const W*>(a.b) + i * a.N * a.R;
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            Planes<kInner<W>> bf[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t row = n0 + 16 * (c >> 2) + 4 * j + (c & 3);
                bf[j] = load_operand(wb + (row < a.N ? row : a.N - 1) * a.R, 32 * s + 8 * g, a.R);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int row = 16 * t + c;
                float v[8] = {};
                if (same >> row & 1) {
                    for (int p = 0; p < a.splits; ++p) {
                        float q[8];
                        load_part(a.inner + (p * a.M + m0 + row) * a.RP, 32 * s + 8 * g, a.R, q);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] += q[e];
                    }
                }
                const Planes<PT> tf = split<PT>(v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 sum = mma(bf[j], tf, acc[t][j]);
                    acc[t][j] = same >> row & 1 ? sum : acc[t][j];  // also where this adapter's weights are no numbers
                }
            }
        }
    });
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int row = 16 * t + c;
        if (!(used >> row & 1)) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + 4 * j + r < a.N) store_act(y, (m0 + row) * a.N + n + 4 * j + r, acc[t][j][r]);
    }
}

// ---- schedule -----------------------------------------------------------------------

template <typename X, typename W, typename Y, int MT>
void launch_tiles(const LoraKernelArgs& k, hipStream_t s) {
    const dim3 down(static_cast<uint32_t>((k.M + 16 * MT - 1) / (16 * MT)), static_cast<uint32_t>(k.splits));
    const dim3 up(down.x, static_cast<uint32_t>((k.N + 255) / 256));
    switch ((k.R + 15) / 16) {
        case 1: lora_down_kernel<X, W, 1, MT><<<down, 256, 0, s>>>(k); break;
        case 2: lora_down_kernel<X, W, 2, MT><<<down, 256, 0, s>>>(k); break;
        case 3: case 4: lora_down_kernel<X, W, 4, MT><<<down, 256, 0, s>>>(k); break;
        default: lora_down_kernel<X, W, 8, MT><<<down, 256, 0, s>>>(k); break;
    }
    switch ((k.R + 31) / 32) {
        case 1: lora_up_kernel<W, Y, 1, MT><<<up, 256, 0, s>>>(k); break;
        case 2: lora_up_kernel<W, Y, 2, MT><<<up, 256, 0, s>>>(k); break;
        default: lora_up_kernel<W, Y, 4, MT><<<up, 256, 0, s>>>(k); break;
    }
}

template <typename X, typename W, typename Y>
void launch_t(const LoraArgs& a, const LoraPlan& p, hipStream_t s) {
    const LoraKernelArgs k{a.x, a.x_scale, a.a, a.b, a.scale, a.index, a.y, a.inner, a.M, a.K, a.N, a.R, p.rank, a.S, p.splits, p.step};
    switch (p.rows) {
        case 1: {
            const uint32_t m = static_cast<uint32_t>(a.M);
            lora_row_down_kernel<X, W><<<dim3(m, static_cast<uint32_t>((a.R + 3) / 4)), 256, 0, s>>>(k);
            lora_row_up_kernel<W, Y><<<dim3(m, static_cast<uint32_t>((a.N + 255) / 256)), 256, 0, s>>>(k);
            break;
        }
        case 16: launch_tiles<X, W, Y, 1>(k, s); break;
        default: launch_tiles<X, W, Y, 4>(k, s); break;
    }
}

}  // namespace

LoraPlan plan_lora(int64_t M, int64_t K, int64_t R) {
    LoraPlan p;
    p.rank = (R + 15) / 16 * 16;
    if (p.rank == 48) p.rank = 64;
    if (p.rank > 64) p.rank = 128;
    p.rows = M <= 64 ? 1 : M <= 2048 ? 16 : 64;
    const int64_t tiles = (M + p.rows - 1) / p.rows;
    int64_t splits = 1;
    if (p.rows > 1)
        while (splits < 8 && tiles * splits < 256 && K / (splits * 2) >= 256) splits *= 2;
    p.step = ((K + splits - 1) / splits + 127) / 128 * 128;
    p.splits = static_cast<int>((K + p.step - 1) / p.step);
    p.ws_bytes = static_cast<size_t>(p.splits * M * p.rank) * 4;
    return p;
}

hipError_t launch_lora(const LoraArgs& a, const LoraPlan& p, hipStream_t s) {
    if (a.dtype == MSSM_F32)
        launch_t<float, float, float>(a, p, s);
    else if (a.dtype == MSSM_BF16)
        a.out_dtype == MSSM_F32 ? launch_t<uint16_t, uint16_t, float>(a, p, s) : launch_t<uint16_t, uint16_t, uint16_t>(a, p, s);
    else
        a.out_dtype == MSSM_F32 ? launch_t<uint8_t, uint16_t, float>(a, p, s) : launch_t<uint8_t, uint16_t, uint16_t>(a, p, s);
    return hipGetLastError();
}

}  // namespace mssm
