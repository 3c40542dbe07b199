// lora.hip -- low-rank adapters of many requests beside a shared projection
// (mssm_lora): y[m] += scale[i] (x[m] A_iᵀ) B_iᵀ with i = index[m].
//
// Two launches, down to the rank and up again; what lies between is float32 in
// the workspace.  Many rows: tiles of 16, 32 or 64 rows on the matrix cores, each
// tile once for every adapter that its rows name (packed requests: one or two),
// the other rows' results unused.  Few rows: a row for itself, by dot products,
// since each mostly has an adapter of its own and its weights are read once.
// y is read and written once, rounded once.
//
// Measured: 16,384 8-bit rows, 2560 -> 10240, rank 64, 16 adapters in runs: down 47 us,
// up 206 us (y, 671 MB, at 3.3 TB/s; bound by memory and its latency); 32 rows of an
// adapter each, rank 16: 3.8 and 3.9 us, launches.
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
// Stores past the caches, at any address.
template <typename V>
__device__ __forceinline__ void stream(void* p, V v) {
    typedef V Anywhere __attribute__((aligned(1)));
    __builtin_nontemporal_store(v, static_cast<Anywhere*>(p));
}

__device__ __forceinline__ void to_floats(u32x4 q, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(q[i]), v[2 * i + 1] = bf16_hi(q[i]);
}
__device__ __forceinline__ void store_eight(float* p, const float (&v)[8]) {
    stream(p, f32x4{v[0], v[1], v[2], v[3]});
    stream(p + 4, f32x4{v[4], v[5], v[6], v[7]});
}
__device__ __forceinline__ void store_eight(uint16_t* p, const float (&v)[8]) {
    bf16x8 b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = static_cast<__bf16>(v[i]);
    stream(p, b);
}
template <typename T>
__device__ __forceinline__ void store_part(T* row, int64_t n, int64_t end, const float (&v)[8]) {
    if (n + 8 <= end) {
        store_eight(row + n, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n + i < end) store_act(row, n + i, v[i]);
    }
}
// Planes of the type: bfloat16 and e4m3 (widened, which is exact) are one.
template <typename T> constexpr int kInner = sizeof(T) == 4 ? 3 : 1;

// Eight elements as loaded, to be made operands when they are needed.
template <typename T> struct Eight;
template <> struct Eight<float> {
    f32x4 lo, hi;
    __device__ __forceinline__ void load(const float* p) {
        lo = reinterpret_cast<const Loose<f32x4>*>(p)->v;
        hi = reinterpret_cast<const Loose<f32x4>*>(p + 4)->v;
    }
    __device__ __forceinline__ void load_part(const float* row, int64_t k, int64_t end) {
#pragma unroll
        for (int i = 0; i < 4; ++i) lo[i] = k + i < end ? row[k + i] : 0.0f, hi[i] = k + 4 + i < end ? row[k + 4 + i] : 0.0f;
    }
    __device__ __forceinline__ Planes<3> planes() const { return split<3>(lo, hi); }
    __device__ __forceinline__ void floats(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = lo[i], x[4 + i] = hi[i];
    }
};
template <> struct Eight<uint16_t> {
    u32x4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = reinterpret_cast<const Loose<u32x4>*>(p)->v; }
    __device__ __forceinline__ void load_part(const uint16_t* row, int64_t k, int64_t end) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = k + 2 * i < end ? row[k + 2 * i] : 0u, hi = k + 2 * i + 1 < end ? row[k + 2 * i + 1] : 0u;
            v[i] = hi << 16 | lo;
        }
    }
    __device__ __forceinline__ Planes<1> planes() const { return Planes<1>{{v}}; }
    __device__ __forceinline__ void floats(float (&x)[8]) const { to_floats(v, x); }
};
template <> struct Eight<uint8_t> {
    u32x2 v;
    __device__ __forceinline__ void load(const uint8_t* p) { v = reinterpret_cast<const Loose<u32x2>*>(p)->v; }
    __device__ __forceinline__ void load_part(const uint8_t* row, int64_t k, int64_t end) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i] |= k + 4 * i + j < end ? static_cast<uint32_t>(row[k + 4 * i + j]) << (8 * j) : 0u;
        }
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(v[i]), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(v[i]), true);
            x[4 * i] = lo[0]; x[4 * i + 1] = lo[1]; x[4 * i + 2] = hi[0]; x[4 * i + 3] = hi[1];
        }
    }
    __device__ __forceinline__ Planes<1> planes() const {  // widened, which is exact
        float x[8];
        floats(x);
        return split<1>(x);
    }
};
// Elements k .. k + 7 of a row of `end`; zeros behind its end.
template <typename T>
__device__ __forceinline__ void floats_of(const T* row, int64_t k, int64_t end, float (&v)[8]) {
    Eight<T> e;
    if (k + 8 <= end) e.load(row + k);
    else e.load_part(row, k, end);
    e.floats(v);
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
        floats_of(x, k, a.K, p);
        floats_of(w, k, a.K, q);
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
        floats_of(w, r, a.R, q);
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
__global__ __launch_bounds__(256, 2) void lora_down_kernel(LoraKernelArgs a) {
    __shared__ f32x4 part[4][RT * MT][64];
    const int lane = threadIdx.x & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16 * MT, k0 = blockIdx.y * a.step, k1 = imin64(a.K, k0 + a.step);
    each_adapter<16 * MT>(a, m0, lane, [&](int64_t i, uint64_t same) {
        f32x4 acc[RT][MT] = {};
        const X* x = static_cast<const X*>(a.x);
        const W* wa = static_cast<const W*>(a.a) + i * a.R * a.K;
        const X* xr[MT];
        const W* wr[RT];
#pragma unroll
        for (int t = 0; t < MT; ++t) xr[t] = x + imin64(m0 + 16 * t + c, a.M - 1) * a.K;
#pragma unroll
        for (int r = 0; r < RT; ++r) wr[r] = wa + imin64(16 * r + c, a.R - 1) * a.K;
        auto step = [&](const Eight<X>(&xe)[MT], const Eight<W>(&we)[RT]) {
            Planes<kInner<X>> xf[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) xf[t] = xe[t].planes();
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const Planes<kInner<W>> wf = we[r].planes();
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[r][t] = mma(wf, xf[t], acc[r][t]);
            }
        };
        auto fetch = [&](int64_t k, Eight<X>(&xe)[MT], Eight<W>(&we)[RT]) {
#pragma unroll
            for (int t = 0; t < MT; ++t) xe[t].load(xr[t] + k + 8 * g);
#pragma unroll
            for (int r = 0; r < RT; ++r) we[r].load(wr[r] + k + 8 * g);
        };
        // whole steps, the next one's loads under way if there are registers for them; then what is left of K
        constexpr bool AHEAD = RT * (sizeof(W) / 2) + MT <= 8;
        Eight<X> xe[AHEAD ? 2 : 1][MT];
        Eight<W> we[AHEAD ? 2 : 1][RT];
        int64_t k = k0 + w * 32;
        if constexpr (!AHEAD) {
            for (; k + 32 <= k1; k += 128) {
                fetch(k, xe[0], we[0]);
                step(xe[0], we[0]);
            }
        } else {
            if (k + 32 <= k1) fetch(k, xe[0], we[0]);
            for (; k + 32 <= k1; k += 256) {
                if (k + 160 <= k1) fetch(k + 128, xe[1], we[1]);
                step(xe[0], we[0]);
                if (k + 160 > k1) {
                    k += 128;
                    break;
                }
                if (k + 288 <= k1) fetch(k + 256, xe[0], we[0]);
                step(xe[1], we[1]);
            }
        }
        if (k < k1) {
#pragma unroll
            for (int t = 0; t < MT; ++t) xe[0][t].load_part(xr[t], k + 8 * g, k1);
#pragma unroll
            for (int r = 0; r < RT; ++r) we[0][r].load_part(wr[r], k + 8 * g, k1);
            step(xe[0], we[0]);
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

// A wave: 16 MT rows and 64 columns; row 4 g + r of tile j is column 32 (j / 2) + 8 g
// + 4 (j % 2) + r, so that a lane has eight neighbours of a row of y twice, and the
// four lanes of a row 64 bytes at a time.
// The rows' inner values are cut into planes once for the workgroup's 256 columns.
template <typename W, typename Y, int RS, int MT>
__global__ __launch_bounds__(256, 2) void lora_up_kernel(LoraKernelArgs a) {
    constexpr int PT = 3;  // planes of the inner values, which are float32 whatever y is
    constexpr int ROW = RS * 64 + 16, PLANE = 16 * MT * ROW;      // 16 bytes apart: the 16 rows of a read on different banks
    __shared__ __align__(16) uint8_t lds[PT * PLANE];
    const int lane = threadIdx.x & 63, w = wave_id(), c = lane & 15, g = lane >> 4;
    const uint32_t blocks = static_cast<uint32_t>((a.N + 255) / 256), rows = blockIdx.x / blocks;  // neighbours share rows
    const int64_t m0 = static_cast<int64_t>(rows) * 16 * MT, n0 = (static_cast<int64_t>(blockIdx.x - rows * blocks) * 4 + w) * 64;
    const bool whole = n0 + 64 <= a.N;  // the same for all lanes: no branch around a load
    Y* y = static_cast<Y*>(a.y);
    const int64_t n = n0 + 8 * g;
    Eight<Y> old[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const Y* row = y + imin64(m0 + 16 * t + c, a.M - 1) * a.N;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (whole) old[t][half].load(row + n + 32 * half);
            else old[t][half].load_part(row, n + 32 * half, a.N);
        }
    }
    const int32_t mine = lane < 16 * MT && m0 + lane < a.M ? a.index[m0 + lane] : -1;
    const uint64_t used = __ballot(mine >= 0 && mine < a.S);
    if (!used) return;
    for (int item = threadIdx.x; item < 16 * MT * RS * 4; item += 256) {
        const int row = item / (RS * 4), k = item % (RS * 4) * 8;
        f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
        if (used >> row & 1 && k < a.RP) {  // others' were never written
            const float* p = a.inner + (m0 + row) * a.RP + k;
            for (int q = 0; q < a.splits; ++q, p += a.M * a.RP) {
                lo += *reinterpret_cast<const f32x4*>(p);
                hi += *reinterpret_cast<const f32x4*>(p + 4);
            }
        }
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + e < a.R ? (e < 4 ? lo[e] : hi[e - 4]) : 0.0f;
        const Planes<PT> t = split<PT>(v);
#pragma unroll
        for (int i = 0; i < PT; ++i) *reinterpret_cast<u32x4*>(lds + i * PLANE + row * ROW + k * 2) = t.p[i];
    }
    __syncthreads();
    if (n0 >= a.N) return;
    f32x4 acc[MT][4] = {};
    each_adapter<16 * MT>(a, m0, lane, [&](int64_t i, uint64_t same) {
        const W* wb = static_cast<const W*>(a.b) + i * a.N * a.R;
        const W* row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) row[j] = wb + imin64(n0 + 32 * (j >> 1) + 8 * (c >> 2) + 4 * (j & 1) + (c & 3), a.N - 1) * a.R;
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            const int64_t k = 32 * s + 8 * g;
            Eight<W> be[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (s < RS / 2 || 32 * s + 32 <= a.R) {  // the rank is more than 16 RS, if RS is not 1
                    be[j].load(row[j] + k);
                } else if (RS < 4 && a.R % 8 == 0) {  // whole pieces of eight: no branch for each element
                    // (1,000 rows of rank 16: 16 us against 28); above 64 there are no registers for both ways
                    be[j].load(row[j] + (k < a.R ? k : 0));
                    if (k >= a.R) be[j] = Eight<W>{};
                } else {
                    be[j].load_part(row[j], k, a.R);
                }
            }
            Planes<kInner<W>> bf[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) bf[j] = be[j].planes();
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                Planes<PT> tf;
#pragma unroll
                for (int q = 0; q < PT; ++q) tf.p[q] = *reinterpret_cast<const u32x4*>(lds + q * PLANE + (16 * t + c) * ROW + k * 2);
                const bool this_one = same >> (16 * t + c) & 1;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 sum = mma(bf[j], tf, acc[t][j]);
                    acc[t][j] = this_one ? sum : acc[t][j];  // also where this adapter's weights are no numbers
                }
            }
            // The compiler leaves one wait state too few between the last of these and
            // what overwrites or reads their results behind the branch that follows.
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_nop 7" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        }
    });
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int row = 16 * t + c;
        if (!(used >> row & 1)) continue;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float v[8];
            old[t][half].floats(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += acc[t][2 * half + (i >> 2)][i & 3];
            store_part(y + (m0 + row) * a.N, n + 32 * half, a.N, v);
        }
    }
}

// ---- schedule -----------------------------------------------------------------------

template <typename X, typename W, typename Y, int ROWS>
void launch_tiles(const LoraKernelArgs& k, hipStream_t s) {
    const dim3 down(static_cast<uint32_t>((k.M + ROWS - 1) / ROWS), static_cast<uint32_t>(k.splits));
    constexpr int MT = ROWS / 16;
    switch ((k.R + 15) / 16) {
        case 1: lora_down_kernel<X, W, 1, MT><<<down, 256, 0, s>>>(k); break;
        case 2: lora_down_kernel<X, W, 2, MT><<<down, 256, 0, s>>>(k); break;
        case 3: case 4: lora_down_kernel<X, W, 4, MT><<<down, 256, 0, s>>>(k); break;
        default:
            if constexpr (MT < (sizeof(W) == 2 ? 4 : 2)) lora_down_kernel<X, W, 8, MT><<<down, 256, 0, s>>>(k);
            break;
    }
    constexpr int UT = MT < 2 ? 1 : sizeof(Y) == 4 ? 2 : 4;  // rows / 16; y and the sums in registers
    const dim3 up(static_cast<uint32_t>((k.M + 16 * UT - 1) / (16 * UT) * ((k.N + 255) / 256)));
    switch ((k.R + 31) / 32) {
        case 1: lora_up_kernel<W, Y, 1, UT><<<up, 256, 0, s>>>(k); break;
        case 2: lora_up_kernel<W, Y, 2, UT><<<up, 256, 0, s>>>(k); break;
        default: lora_up_kernel<W, Y, 4, UT><<<up, 256, 0, s>>>(k); break;
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
        case 16: launch_tiles<X, W, Y, 16>(k, s); break;
        case 32: launch_tiles<X, W, Y, 32>(k, s); break;
        default:
            if constexpr (sizeof(W) == 2) launch_tiles<X, W, Y, 64>(k, s);
            break;
    }
}

}  // namespace

LoraPlan plan_lora(int64_t M, int64_t K, int64_t R, bool f32) {
    LoraPlan p;
    p.rank = (R + 15) / 16 * 16;
    if (p.rank == 48) p.rank = 64;
    if (p.rank > 64) p.rank = 128;
    // Rows for themselves up to 64: the index is on the device, and where each row has an adapter of its own a tile
    // computes 16 rows for every one.  us by rows / by tiles of 16, bfloat16, 2560 -> 10240, rank 16: 32 rows of 32
    // adapters 14 / 35, 64 of 64 13 / 35, 64 of 2 in runs 13 / 11; rank 64: 64 rows of 64 67 / 58, of 2 in runs 27 / 11,
    // 128 of 2 in runs 48 / 12.
    // Tiles of 16 up to 2,048, then larger ones, whose weights are read less often.  us by 16 / 64, bfloat16, in runs of
    // 8 adapters: rank 64, 2,048 rows 46 / 48, 4,096 75 / 68; by 16 / 32: rank 128, 2,048 rows 67 / 60, 4,096 118 / 91;
    // float32, 1536 -> 1536, rank 16, 2,048 rows 16 / 17, 4,096 25 / 23.  Rows of many adapters in any order lose by
    // larger tiles (4,096 of 64, rank 16: 243 / 449).
    // The rank's and the rows' accumulators of a tile have to fit the registers, and float32 has three planes of each operand.
    p.rows = M <= 64 ? 1 : M <= 2048 || (f32 && R > 64) ? 16 : f32 || R > 64 ? 32 : 64;
    const int64_t tiles = (M + p.rows - 1) / p.rows;
    // Parts of K of at least 256, while there are fewer workgroups than compute units.  us in one part / in several:
    // 300 rows (19 tiles) of rank 16 18 / 12 (8 parts), 1,000 26 / 21 (4); 2,000 of rank 64 60 / 51 (2).
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
