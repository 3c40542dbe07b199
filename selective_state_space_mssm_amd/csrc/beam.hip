// beam.hip -- one beam-search selection (mssm_beam_select) and the reordering
// of the beams' states (mssm_beam_reorder).
#include "block.h"
#include "device_common.h"

#include <type_traits>

namespace mssm {
namespace {

// A float32 as an unsigned number of the same order (no NaN; -0 is +0: the two are equal).
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
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

// The maximum (or sum) over the wave, the same in every lane.  Within-row
// DPP moves, then the row totals handed up to lane 63: no LDS round trip, of
// which a selection of K candidates would pay several per candidate.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {  // lanes of other rows keep their own
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(v), static_cast<int>(v), CTRL, ROWS, 0xF, false));
}
template <typename V, typename Op>
__device__ __forceinline__ V wave_reduce(V v, Op op) {
    auto step = [&](auto ctrl, auto rows) {
        v = op(v, __builtin_bit_cast(V, dpp_u32<decltype(ctrl)::value, decltype(rows)::value>(__builtin_bit_cast(uint32_t, v))));
    };
    typedef std::integral_constant<int, 0xF> All;
    step(std::integral_constant<int, 0xB1>{}, All{});   // quad_perm [1, 0, 3, 2]
    step(std::integral_constant<int, 0x4E>{}, All{});   // quad_perm [2, 3, 0, 1]
    step(std::integral_constant<int, 0x141>{}, All{});  // row_half_mirror
    step(std::integral_constant<int, 0x140>{}, All{});  // row_mirror
    V rows[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        rows[i] = __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), i * 16));
    return op(op(rows[0], rows[1]), op(rows[2], rows[3]));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_reduce(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
    return wave_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    const uint32_t hi = wave_max(static_cast<uint32_t>(v >> 32));
    const uint32_t lo = wave_max(static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}
constexpr float kInf = __builtin_inff();
constexpr float kBiggest = 3.402823466e+38f;

// A logit as the selection takes it: NaN is banned, +infinity the largest number.
__device__ __forceinline__ float clean(float v) { return __builtin_fminf(__builtin_fmaxf(v, -kInf), kBiggest); }
// A score: what is no number, or +infinity, is a beam that is not in use.
__device__ __forceinline__ float clean_score(float v) { return v < kInf ? v : -kInf; }

// ---- the selection: a part of a beam's logits a workgroup --------------------------
//
// The values of one beam are its logits shifted by one number, so its best
// tokens are known before the softmax sum is, and one pass over the logits
// gives both: each workgroup leaves its part's K best (logit, token) and its
// part's maximum and sum.  Every float32 sum is formed in a fixed order.
// 512 x 50,280 bfloat16 take 24.4 us (2.1 TB/s), bound by neither memory nor the
// vector units: their 407 instructions a wave and span are busy for 24,800 of
// the some 55,000 cycles (by counter), and the two waves of a SIMD wait half of
// their time, at the barrier, the lane reads and the ballots of each span.
// 512 x 131,072 float32 with the second launch 56 us (4.8 TB/s).

constexpr int kThreads = 256;
constexpr int kMaxParts = 32;              // of a row; more logits: several spans a part
constexpr int kHits = MSSM_MAX_BEAMS * 8;  // candidates a wave keeps of a span

struct PartStat { float max, sum; };

// Where a thread's PT logits of a span lie: 16 bytes a load where rows start on
// 16-byte boundaries, single elements otherwise.
template <typename T, int PT, bool EVEN>
struct Span {
    static constexpr int VEC = EVEN ? 16 / static_cast<int>(sizeof(T)) : 1, LEN = PT * kThreads, COUNT = PT;
    uint32_t raw[PT / VEC][EVEN ? 4 : 1];
    __device__ __forceinline__ static uint32_t index(int e) { return ((e / VEC) * kThreads + threadIdx.x) * VEC + e % VEC; }
    // the logits from x on, of which `left` are in the part
    __device__ __forceinline__ void load(const T* x, int64_t left) {
        if (left >= LEN) {
#pragma unroll
            for (int q = 0; q < PT / VEC; ++q) load_lane_row<T, VEC>(x + index(q * VEC), raw[q]);
        } else {
#pragma unroll
            for (int q = 0; q < PT / VEC; ++q)
                if (index(q * VEC) < left) load_lane_row<T, VEC>(x + index(q * VEC), raw[q]);
        }
    }
    __device__ __forceinline__ void values(int64_t left, float (&f)[PT]) const {
#pragma unroll
        for (int q = 0; q < PT / VEC; ++q) {
            float u[VEC];
            unpack_lane_row<T, VEC>(raw[q], u);
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[q * VEC + i] = clean(u[i]);
        }
        if (left < LEN) {
#pragma unroll
            for (int e = 0; e < PT; ++e) f[e] = index(e) < left ? f[e] : -kInf;
        }
    }
};

// The K best of n keys (0: none), key i in lane i % 64 of held[i / 64]: the k-th
// best in lane k, 0 where there are fewer.  Up to 64 different keys are ranked
// by counting the larger ones, more are taken in K rounds of a maximum.
template <int S>
__device__ __forceinline__ uint64_t best_of(uint64_t (&held)[S], int n, int K, int lane, uint64_t* sorted) {
    if (n <= 64) {
        int rank = 0;
        for (int j = 0; j < n; ++j) {
            const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(held[0] >> 32), j);
            const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(held[0]), j);
            rank += ((static_cast<uint64_t>(hi) << 32) | lo) > held[0] ? 1 : 0;
        }
        wave_handoff();  // sorted may be where held came from
        if (lane < K) sorted[lane] = 0;
        wave_handoff();
        if (held[0] && rank < K) sorted[rank] = held[0];
        wave_handoff();
        return lane < K ? sorted[lane] : 0;
    }
    uint64_t mine = 0;
    for (int k = 0; k < K; ++k) {
        uint64_t top = held[0];
#pragma unroll
        for (int i = 1; i < S; ++i) top = held[i] > top ? held[i] : top;
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < S; ++i) held[i] = held[i] == top ? 0 : held[i];
        if (lane == k) mine = top;
    }
    return mine;
}

// The K best of a wave's logits of a span, in K passes over memory: for spans
// of many equal logits, or of hardly any, which the bound does not thin out.
template <typename T, typename At>
__device__ __forceinline__ int pick_in_passes(const T* x, int64_t v0, int64_t hi, int K, uint64_t* hits, int lane) {
    uint64_t last = ~uint64_t{0};
    for (int k = 0; k < K; ++k) {
        uint64_t top = 0;
        for (int e = 0; e < At::COUNT; ++e) {
            const int64_t v = v0 + At::index(e);
            if (v >= hi) continue;
            const uint64_t key = key_of(clean(load_act(x, v)), static_cast<uint32_t>(v));
            if (key < last && key > top) top = key;
        }
        last = wave_max(top);
        if (lane == 0) hits[k] = last;
        if (last == 0) last = 1;  // none left: only zeros follow
    }
    wave_handoff();
    return K;
}

template <typename T, int PT, bool EVEN>
__global__ __launch_bounds__(kThreads) void beam_part_kernel(const void* logits, const float* scores,
                                                             const uint8_t* finished, int32_t end_token, int64_t V, int K,
                                                             int64_t part_len, uint64_t* best, PartStat* stat) {
    typedef Span<T, PT, EVEN> At;
    constexpr int GROUPS = kThreads / 16;
    static_assert(GROUPS >= MSSM_MAX_BEAMS, "a bound needs K groups");
    __shared__ float maxima[2][GROUPS], sums[4];
    __shared__ uint64_t list[4][kHits], sorted[4][MSSM_MAX_BEAMS];
    __shared__ int count[4];
    const int64_t row = blockIdx.y, part = blockIdx.x, parts = gridDim.x;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t lo = part * part_len, hi = imin64(lo + part_len, V);
    uint64_t* mine = best + (row * parts + part) * K;
    const T* x = static_cast<const T*>(logits) + row * V;
    At next;
    next.load(x + lo, hi - lo);
    const bool dead = clean_score(scores[row]) == -kInf;
    if (dead || (finished && finished[row])) {
        // No softmax: a beam out of use has the value -infinity everywhere, a
        // finished one everywhere but at its end token.
        if (threadIdx.x == 0) {
            stat[row * parts + part] = {0.0f, 1.0f};
            int n = 0;
            const bool here = !dead && end_token >= lo && end_token < hi;
            if (here) mine[n++] = key_of(0.0f, static_cast<uint32_t>(end_token));
            for (int64_t v = lo; v < hi && n < K; ++v)
                if (!here || v != end_token) mine[n++] = key_of(-kInf, static_cast<uint32_t>(v));
            while (n < K) mine[n++] = 0;
        }
        return;
    }
    uint64_t* hits = list[wave];
    float m = -kInf, s = 0.0f, floor = -kInf;
    int n = 0;  // the wave's candidates
    for (int64_t v0 = lo, turn = 0; v0 < hi; v0 += At::LEN, turn ^= 1) {
        float f[PT];
        next.values(hi - v0, f);
        if (v0 + At::LEN < hi) next.load(x + v0 + At::LEN, hi - v0 - At::LEN);  // under way during this span
        float tm = f[0];
#pragma unroll
        for (int e = 1; e < PT; ++e) tm = __builtin_fmaxf(tm, f[e]);
        tm = __builtin_fmaxf(tm, dpp_move<0xB1>(tm));
        tm = __builtin_fmaxf(tm, dpp_move<0x4E>(tm));
        tm = __builtin_fmaxf(tm, dpp_move<0x141>(tm));
        tm = __builtin_fmaxf(tm, dpp_move<0x140>(tm));
        if ((lane & 15) == 0) maxima[turn][threadIdx.x / 16] = tm;
        __syncthreads();
        // The K-th largest of the 16 groups' maxima: K logits reach it, so what is
        // below it is not among the K best, in this span and in the later ones.
        // About 11 of the first 8,192 are left for 8 beams.
        const float gm = maxima[turn][lane & 15];
        int rank = 0;
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) {
            const float o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gm), j));
            rank += o > gm || (o == gm && j < (lane & 15)) ? 1 : 0;
        }
        auto ranked = [&](int k) {
            return __int_as_float(__builtin_amdgcn_readlane(
                __float_as_int(gm), __ffsll(static_cast<unsigned long long>(__ballot(rank == k))) - 1));
        };
        floor = __builtin_fmaxf(floor, ranked(K - 1));
        const float top = __builtin_fmaxf(ranked(0), m);
        const int before = n;
        if (floor > -kInf) {
#pragma unroll
            for (int e = 0; e < PT; ++e) {
                const uint64_t at = __ballot(f[e] >= floor);
                if (at) {
                    const int place = n + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(at >> 32),
                                                                    __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(at), 0));
                    if (f[e] >= floor && place < kHits) hits[place] = key_of(f[e], static_cast<uint32_t>(v0) + At::index(e));
                    n += __builtin_popcountll(at);
                }
            }
        }
        wave_handoff();
        if (n > kHits || !(floor > -kInf)) n = before + pick_in_passes<T, At>(x, v0, hi, K, hits + before, lane);
        if (n > 64) {  // make room for the next span's
            uint64_t held[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) held[i] = i * 64 + lane < n ? hits[i * 64 + lane] : 0;
            const uint64_t kept = best_of(held, n, K, lane, sorted[wave]);
            wave_handoff();
            if (lane < K) hits[lane] = kept;
            n = K;
        }
        // this thread's share of the running sum; before the first span 0
        const float base = top == -kInf ? 0.0f : top;
        float span_sum = 0.0f;
#pragma unroll
        for (int e = 0; e < PT; ++e) span_sum += fast_exp2((f[e] - base) * kLog2e);
        s = s * fast_exp2((m - base) * kLog2e) + span_sum;
        m = top;
    }
    s = wave_sum(s);
    if (lane == 0) {
        sums[wave] = s;
        count[wave] = n;
    }
    __syncthreads();
    if (wave) return;
    if (lane == 0) stat[row * parts + part] = {m, (sums[0] + sums[1]) + (sums[2] + sums[3])};
    // the four waves' candidates, moved together (always downwards), and their best
    uint64_t* all = list[0];
    int total = 0;
    for (int w = 0; w < 4; ++w) {
        const int c = count[w];  // at most 64
        const uint64_t key = lane < c ? list[w][lane] : 0;
        if (lane < c) all[total + lane] = key;
        total += c;
    }
    wave_handoff();
    uint64_t held[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) held[i] = i * 64 + lane < total ? all[i * 64 + lane] : 0;
    const uint64_t kept = best_of(held, total, K, lane, sorted[0]);
    if (lane < K) mine[lane] = kept;
}

// A batch row: a wave joins a beam's parts, then the first one the beams: 4 us
// for a row, 5 us for 64 rows of 8 beams, the length of its chain of steps.
__global__ __launch_bounds__(512) void beam_merge_kernel(const float* scores, const uint8_t* finished, int32_t end_token,
                                                         int64_t V, int K, int parts, const uint64_t* best,
                                                         const PartStat* stat, float* scores_out, int32_t* parent,
                                                         int32_t* token, uint8_t* finished_out) {
    constexpr int WAVES = 8, HELD = kMaxParts * MSSM_MAX_BEAMS / 64;
    __shared__ uint64_t keys[MSSM_MAX_BEAMS * MSSM_MAX_BEAMS];
    __shared__ uint8_t done[MSSM_MAX_BEAMS];
    const int64_t b = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = wave_id();
    for (int k = wave; k < K; k += WAVES) {
        const int64_t row = b * K + k;
        const int n = parts * K;
        uint64_t held[HELD];
#pragma unroll
        for (int i = 0; i < HELD; ++i) held[i] = i * 64 + lane < n ? best[row * n + i * 64 + lane] : 0;
        const PartStat st = lane < parts ? stat[row * parts + lane] : PartStat{-kInf, 0.0f};
        const float score = clean_score(scores[row]);
        const bool fin = finished && finished[row];
        const float m = wave_max(st.max), base = m == -kInf ? 0.0f : m;
        const float log_sum = logf(wave_sum(st.sum * fast_exp2((st.max - base) * kLog2e)));
        if (lane == 0) done[k] = fin;
        const uint64_t mine = best_of(held, n, K, lane, keys + k * K);
        if (lane < K) {
            uint64_t key = 0;
            if (mine) {
                const float x = from_ordered(static_cast<uint32_t>(mine >> 32));
                const float value = x == -kInf ? -kInf : fin ? score : score + ((x - base) - log_sum);
                key = key_of(value, static_cast<uint32_t>(k * V + index_of(mine)));
            }
            keys[k * K + lane] = key;
        }
    }
    __syncthreads();
    if (wave) return;
    uint64_t held[MSSM_MAX_BEAMS * MSSM_MAX_BEAMS / 64];
#pragma unroll
    for (int i = 0; i < MSSM_MAX_BEAMS * MSSM_MAX_BEAMS / 64; ++i) held[i] = i * 64 + lane < K * K ? keys[i * 64 + lane] : 0;
    const uint64_t mine = best_of(held, K * K, K, lane, keys);
    if (lane < K) {
        const uint32_t index = index_of(mine);
        const int p = static_cast<int>(index / static_cast<uint32_t>(V)), t = static_cast<int>(index % static_cast<uint32_t>(V));
        scores_out[b * K + lane] = from_ordered(static_cast<uint32_t>(mine >> 32));
        parent[b * K + lane] = p;
        token[b * K + lane] = t;
        if (finished_out) finished_out[b * K + lane] = done[p] || t == end_token;
    }
}

// ---- reordering ------------------------------------------------------------------------

struct ReorderArgs {
    mssm_beam_state st[MSSM_MAX_BEAM_STATES];
    int64_t first[MSSM_MAX_BEAM_STATES + 1];  // workgroups of the tensors before
    int64_t B;
    int K, count;
    const int32_t* parent;
};

constexpr int kColumns = 256;  // 16-byte columns of a workgroup

// The beams that move (p[k] != k) get their parents' columns, 16 bytes or one
// at `at`.  One thread holds its column of all the beams: it reads every parent
// before it writes, so that the states are reordered in place whatever the
// parents are.  Up to four beams the choice is a few register selects: 8 x 4
// beams, 734 MB of states, of which they read and write 1.0 GB, 169 us (6.0
// TB/s).  More go through the thread's own slots of LDS, which can be indexed, and
// are slower by it: the same states as 4 x 8 beams 474 us (2.2 TB/s, at 257
// registers one wave a SIMD), as 2 x 16 beams 289 us (3.7 TB/s); bytes that are no
// multiple of 16 move at 1.8 to 2.0 TB/s there, at 5.0 with up to four beams.
template <int MAXK, bool STREAM, typename C>
__device__ __forceinline__ void move_column(uint8_t* base, int64_t bytes, const int (&p)[MAXK], uint32_t need, int64_t at,
                                            uint8_t* slots) {
    C v[MAXK];
#pragma unroll
    for (int k = 0; k < MAXK; ++k)
        if (need >> k & 1) {
            if constexpr (STREAM) v[k] = __builtin_nontemporal_load(reinterpret_cast<const C*>(base + k * bytes + at));
            else v[k] = *reinterpret_cast<const C*>(base + k * bytes + at);
        }
    if constexpr (MAXK > 4) {
#pragma unroll
        for (int k = 0; k < MAXK; ++k)
            if (need >> k & 1) *reinterpret_cast<C*>(slots + k * kColumns * 16) = v[k];
    }
#pragma unroll
    for (int k = 0; k < MAXK; ++k) {
        if (p[k] == k) continue;
        C u;
        if constexpr (MAXK > 4) {
            u = *reinterpret_cast<const C*>(slots + p[k] * kColumns * 16);
        } else {
            u = v[0];
#pragma unroll
            for (int q = 1; q < MAXK; ++q)
                if (p[k] == q) u = v[q];
        }
        if constexpr (STREAM) __builtin_nontemporal_store(u, reinterpret_cast<C*>(base + k * bytes + at));
        else *reinterpret_cast<C*>(base + k * bytes + at) = u;
    }
}

// STREAM: whole columns pass the caches by.
template <int MAXK, bool STREAM>
__global__ __launch_bounds__(kColumns) void beam_reorder_kernel(ReorderArgs a) {
    typedef uint32_t Even __attribute__((ext_vector_type(4)));
    struct __attribute__((packed)) Any { Even v; };
    extern __shared__ __align__(16) uint8_t slots[];
    for (int64_t id = blockIdx.x; id < a.first[a.count]; id += gridDim.x) {
        int t = 0;
        while (id >= a.first[t + 1]) ++t;
        const mssm_beam_state st = a.st[t];
        const int64_t blocks = (st.bytes + 16 * kColumns - 1) / (16 * kColumns), in = id - a.first[t];
        const int64_t lb = in / blocks, at = (in % blocks * kColumns + threadIdx.x) * 16;
        uint8_t* base = static_cast<uint8_t*>(st.data) + lb * a.K * st.bytes;
        const int32_t* par = a.parent + lb % a.B * a.K;
        int p[MAXK];
        uint32_t need = 0;
#pragma unroll
        for (int k = 0; k < MAXK; ++k) {
            p[k] = k < a.K ? __builtin_amdgcn_readfirstlane(par[k]) : k;
            if (p[k] < 0 || p[k] >= a.K) p[k] = k;
            if (p[k] != k) need |= 1u << p[k];
        }
        if (need == 0) continue;
        uint8_t* mine = slots + threadIdx.x * 16;
        if (at + 16 <= st.bytes) {
            if (st.bytes % 16 == 0)
                move_column<MAXK, STREAM, Even>(base, st.bytes, p, need, at, mine);
            else
                move_column<MAXK, false, Any>(base, st.bytes, p, need, at, mine);
        } else {
            for (int64_t i = at; i < st.bytes; ++i) move_column<MAXK, false, uint8_t>(base, st.bytes, p, need, i, mine);
        }
    }
}

}  // namespace

namespace {
// Parts of a row and the logits a thread holds: about 512 workgroups, two on each
// of 256 CUs (1,024 to 2,048 are up to 8 % slower at 512 x 50,280 and 512 x
// 131,072, by their shorter runs of spans).  32 logits a thread (spans of 8,192)
// where that many workgroups have a whole span, else 8 (2,048), which shortens
// the way of a few rows.
struct BeamPlan { int64_t parts, len; int per_thread; };
BeamPlan plan_beam(int64_t rows, int64_t V) {
    const bool many = V >= 4096 && rows * ((V + 8191) / 8192) >= 512;
    const int64_t span = many ? 8192 : 2048, spans = (V + span - 1) / span;
    int64_t parts = (512 + rows - 1) / rows;
    parts = parts < spans ? parts : spans;
    parts = parts < kMaxParts ? parts : kMaxParts;
    const int64_t len = ((V + parts - 1) / parts + 7) / 8 * 8;  // whole vectors
    return {(V + len - 1) / len, len, many ? 32 : 8};
}
}  // namespace

size_t beam_ws_bytes(int64_t B, int64_t K, int64_t V) {
    return static_cast<size_t>(B) * K * plan_beam(B * K, V).parts * (K * sizeof(uint64_t) + sizeof(PartStat));
}

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s) {
    const int64_t rows = a.B * a.K;
    const BeamPlan p = plan_beam(rows, a.V);
    uint64_t* best = static_cast<uint64_t*>(a.workspace);
    PartStat* stat = reinterpret_cast<PartStat*>(best + rows * p.parts * a.K);
    const int K = static_cast<int>(a.K);
    const bool even = a.V * (a.dtype == MSSM_F32 ? 4 : 2) % 16 == 0;
    // the second grid dimension holds 65,535 rows: more go in several launches
    for (int64_t r0 = 0; r0 < rows; r0 += 65535) {
        const dim3 grid(static_cast<uint32_t>(p.parts), static_cast<uint32_t>(imin64(65535, rows - r0)));
        const char* x = static_cast<const char*>(a.logits) + r0 * a.V * (a.dtype == MSSM_F32 ? 4 : 2);
        auto run = [&](auto kernel) {
            kernel<<<grid, kThreads, 0, s>>>(x, a.scores + r0, a.finished ? a.finished + r0 : nullptr, a.end_token, a.V, K,
                                             p.len, best + r0 * p.parts * a.K, stat + r0 * p.parts);
        };
        auto pick = [&](auto zero) {
            typedef decltype(zero) T;
            if (p.per_thread == 32)
                even ? run(beam_part_kernel<T, 32, true>) : run(beam_part_kernel<T, 32, false>);
            else
                even ? run(beam_part_kernel<T, 8, true>) : run(beam_part_kernel<T, 8, false>);
        };
        a.dtype == MSSM_F32 ? pick(0.0f) : pick(uint16_t{0});
    }
    // a launch has fewer than 2^32 threads: 2^22 batch rows at a time
    constexpr int64_t kBatch = int64_t{1} << 22;
    for (int64_t b0 = 0; b0 < a.B; b0 += kBatch) {
        const int64_t r0 = b0 * a.K;
        beam_merge_kernel<<<dim3(static_cast<uint32_t>(imin64(kBatch, a.B - b0))), 512, 0, s>>>(
            a.scores + r0, a.finished ? a.finished + r0 : nullptr, a.end_token, a.V, K, static_cast<int>(p.parts),
            best + r0 * p.parts * a.K, stat + r0 * p.parts, a.scores_out + r0, a.parent + r0, a.token + r0,
            a.finished_out ? a.finished_out + r0 : nullptr);
    }
    return hipGetLastError();
}

hipError_t launch_beam_reorder(int64_t B, int64_t K, const int32_t* parent, int count, const mssm_beam_state* st,
                               hipStream_t s) {
    ReorderArgs a{};
    a.B = B;
    a.K = static_cast<int>(K);
    a.count = count;
    a.parent = parent;
    double total = 0.0;  // bytes
    for (int i = 0; i < count; ++i) {
        total += static_cast<double>(st[i].layers) * B * K * st[i].bytes;
        a.st[i] = st[i];
        a.first[i + 1] = a.first[i] + st[i].layers * B * ((st[i].bytes + 16 * kColumns - 1) / (16 * kColumns));
    }
    const dim3 grid(static_cast<uint32_t>(imin64(a.first[count], int64_t{1} << 23)));  // below 2^32 threads; the kernel strides
    // States beyond the 256 MB last-level cache stream past it: 734 MB take 182 us
    // so and 201 us through it, but 245 MB 73 us so and 61 us through it (four beams).
    auto launch = [&](auto stream) {
        constexpr bool S = decltype(stream)::value;
        if (K <= 4)
            beam_reorder_kernel<4, S><<<grid, kColumns, 0, s>>>(a);
        else if (K <= 8)
            beam_reorder_kernel<8, S><<<grid, kColumns, 8 * 16 * kColumns, s>>>(a);
        else
            beam_reorder_kernel<16, S><<<grid, kColumns, 16 * 16 * kColumns, s>>>(a);
    };
    total > double{256 << 20} ? launch(std::true_type{}) : launch(std::false_type{});
    return hipGetLastError();
}

}  // namespace mssm
