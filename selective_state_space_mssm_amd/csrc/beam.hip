// beam.hip -- one beam-search selection (mssm_beam_select) and the reordering
// of the beams' states (mssm_beam_reorder).
#include "block.h"
#include "device_common.h"

namespace mssm {
namespace {

// A float32 as an unsigned number of the same order (no NaN).
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v);
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xffffffffu));
}
// (value, index) as one number: larger values first, then lower indexes.  0 is below every candidate.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t index) {
    return (static_cast<uint64_t>(ordered(v)) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return 0xffffffffu - static_cast<uint32_t>(key); }

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    for (int m = 32; m; m >>= 1) {
        const uint64_t o = __shfl_xor(static_cast<unsigned long long>(v), m);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
    for (int m = 32; m; m >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, m));
    return v;
}

constexpr float kInf = __builtin_inff();
constexpr float kBiggest = 3.402823466e+38f;

// A logit as the selection takes it: NaN is banned, +infinity the largest number.
__device__ __forceinline__ float clean(float v) { return v == v ? __builtin_fminf(v, kBiggest) : -kInf; }
// A score: what is no number, or +infinity, is a beam that is not in use.
__device__ __forceinline__ float clean_score(float v) { return v < kInf ? v : -kInf; }

struct RowStat { float max, sum; };

// The best K of one beam's row by (logit, lower index), and its softmax statistics.
template <typename T>
__global__ __launch_bounds__(256) void beam_row_kernel(const void* logits, const float* scores, const uint8_t* finished,
                                                       int32_t end, int64_t V, int K, uint64_t* best, RowStat* stat) {
    __shared__ float sf[4];
    __shared__ uint64_t su[4];
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const T* x = static_cast<const T*>(logits) + row * V;
    const bool dead = clean_score(scores[row]) == -kInf;
    const bool done = !dead && finished && finished[row];
    auto at = [&](int64_t v) { return dead ? -kInf : done ? (v == end ? 0.0f : -kInf) : clean(load_act(x, v)); };
    float m = -kInf;
    for (int64_t v = threadIdx.x; v < V; v += 256) m = __builtin_fmaxf(m, at(v));
    m = wave_max(m);
    if (lane == 0) sf[wave] = m;
    __syncthreads();
    m = __builtin_fmaxf(__builtin_fmaxf(sf[0], sf[1]), __builtin_fmaxf(sf[2], sf[3]));
    __syncthreads();
    const float base = m == -kInf ? 0.0f : m;
    float s = 0.0f;
    for (int64_t v = threadIdx.x; v < V; v += 256) s += expf(at(v) - base);
    s = wave_sum(s);
    if (lane == 0) sf[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) stat[row] = {base, (sf[0] + sf[1]) + (sf[2] + sf[3])};
    uint64_t last = ~uint64_t{0};
    for (int k = 0; k < K; ++k) {
        uint64_t top = 0;
        for (int64_t v = threadIdx.x; v < V; v += 256) {
            const uint64_t key = key_of(at(v), static_cast<uint32_t>(v));
            if (key < last && key > top) top = key;
        }
        top = wave_max(top);
        __syncthreads();
        if (lane == 0) su[wave] = top;
        __syncthreads();
        for (int i = 0; i < 4; ++i) top = su[i] > top ? su[i] : top;
        if (threadIdx.x == 0) best[row * K + k] = top;
        last = top;
    }
}

// The best K of a batch row's K lists: one wave a batch row.
__global__ __launch_bounds__(64) void beam_merge_kernel(const float* scores, const uint8_t* finished, int32_t end,
                                                        int64_t V, int K, const uint64_t* best, const RowStat* stat,
                                                        float* scores_out, int32_t* parent, int32_t* token,
                                                        uint8_t* finished_out) {
    const int64_t b = blockIdx.x;
    const int lane = threadIdx.x;
    __shared__ uint64_t keys[MSSM_MAX_BEAMS * MSSM_MAX_BEAMS];
    __shared__ uint8_t done[MSSM_MAX_BEAMS];
    if (lane < K) done[lane] = finished ? finished[b * K + lane] : 0;
    __syncthreads();
    for (int i = lane; i < K * K; i += 64) {
        const int k = i / K;
        const uint64_t e = best[b * K * K + i];
        uint64_t key = 0;
        if (e) {
            const float score = clean_score(scores[b * K + k]);
            const float x = from_ordered(static_cast<uint32_t>(e >> 32));
            const RowStat st = stat[b * K + k];
            float value = -kInf;
            if (x != -kInf) value = done[k] ? score : score + ((x - st.max) - logf(st.sum));
            key = key_of(value, static_cast<uint32_t>(k * V + index_of(e)));
        }
        keys[i] = key;
    }
    __syncthreads();
    uint64_t last = ~uint64_t{0};
    for (int k = 0; k < K; ++k) {
        uint64_t top = 0;
        for (int i = lane; i < K * K; i += 64)
            if (keys[i] < last && keys[i] > top) top = keys[i];
        top = wave_max(top);
        last = top;
        if (lane == 0) {
            const uint32_t idx = index_of(top);
            const int p = static_cast<int>(idx / V), t = static_cast<int>(idx % V);
            scores_out[b * K + k] = from_ordered(static_cast<uint32_t>(top >> 32));
            parent[b * K + k] = p;
            token[b * K + k] = t;
            if (finished_out) finished_out[b * K + k] = done[p] || t == end;
        }
    }
}

struct ReorderArgs {
    mssm_beam_state st[MSSM_MAX_BEAM_STATES];
};

// One thread holds one byte column of all beams of (layer, batch row): it reads every parent before it writes.
__global__ __launch_bounds__(256) void beam_reorder_kernel(ReorderArgs a, int64_t B, int K, const int32_t* parent) {
    const mssm_beam_state st = a.st[blockIdx.z];
    for (int64_t lb = blockIdx.y; lb < st.layers * B; lb += gridDim.y) {
        const int32_t* par = parent + lb % B * K;
        uint8_t* base = static_cast<uint8_t*>(st.data) + lb * K * st.bytes;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < st.bytes; i += static_cast<int64_t>(gridDim.x) * 256) {
            uint8_t v[MSSM_MAX_BEAMS];
            for (int k = 0; k < K; ++k) v[k] = base[k * st.bytes + i];
            for (int k = 0; k < K; ++k) {
                const int p = par[k];
                if (p >= 0 && p < K && p != k) base[k * st.bytes + i] = v[p];
            }
        }
    }
}

}  // namespace

size_t beam_ws_bytes(int64_t B, int64_t K, int64_t) {
    return static_cast<size_t>(B) * K * (K * sizeof(uint64_t) + sizeof(RowStat));
}

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s) {
    uint64_t* best = static_cast<uint64_t*>(a.workspace);
    RowStat* stat = reinterpret_cast<RowStat*>(best + a.B * a.K * a.K);
    const int K = static_cast<int>(a.K);
    const dim3 grid(static_cast<uint32_t>(a.B * a.K));
    if (a.dtype == MSSM_F32)
        beam_row_kernel<float><<<grid, 256, 0, s>>>(a.logits, a.scores, a.finished, a.end_token, a.V, K, best, stat);
    else
        beam_row_kernel<uint16_t><<<grid, 256, 0, s>>>(a.logits, a.scores, a.finished, a.end_token, a.V, K, best, stat);
    beam_merge_kernel<<<dim3(static_cast<uint32_t>(a.B)), 64, 0, s>>>(a.scores, a.finished, a.end_token, a.V, K, best,
                                                                     stat, a.scores_out, a.parent, a.token,
                                                                     a.finished_out);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(int64_t B, int64_t K, const int32_t* parent, int count, const mssm_beam_state* st,
                               hipStream_t s) {
    ReorderArgs a{};
    int64_t cols = 1, lb = 1;
    for (int i = 0; i < count; ++i) {
        a.st[i] = st[i];
        cols = st[i].bytes > cols ? st[i].bytes : cols;
        lb = st[i].layers * B > lb ? st[i].layers * B : lb;
    }
    const dim3 grid(static_cast<uint32_t>(imin64((cols + 255) / 256, 256)), static_cast<uint32_t>(imin64(lb, 65535)), count);
    beam_reorder_kernel<<<grid, 256, 0, s>>>(a, B, static_cast<int>(K), parent);
    return hipGetLastError();
}

}  // namespace mssm
