// linear_plan.h -- how one product (linear.hip) is computed and cut.  Host
// arithmetic alone, without HIP, so that a test can ask for the variant of a size.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "mssm_block.h"

namespace mssm {

constexpr int kLinearStepBytes = 128;  // of k in a step of any variant

// How one product is computed and cut; the same rule sizes the workspace and launches.
enum class LinearPath { kRows, kColumns, kTile128, kTile256 };
struct LinearPlan {
    LinearPath path;
    int64_t full, rest;  // tiles computed whole, and tiles cut along in_dim
    int splits;          // parts of each of the latter, 1: none and no second pass
    size_t ws_bytes;
};

// The tile kernel's grid: a launch has fewer than 2^32 threads in a dimension,
// so 2^22 workgroups go in a row; number x + y * grid.x, those behind the last do
// nothing.
struct LinearGrid { uint32_t x, y; };
inline LinearGrid linear_grid(int64_t groups) {
    const int64_t x = std::min<int64_t>(groups, int64_t{1} << 22);
    return {static_cast<uint32_t>(x), static_cast<uint32_t>((groups + x - 1) / x)};
}

// Time of T tiles (us): a round of all the slots takes `depth` k steps of
// `step` us and `ends` us around them; a last round of few tiles is cut along k
// into `splits` when that saves more than a second pass (5 us) and the partial
// sums' traffic (written and read at about 4.5 TB/s, `tile_mb` each) cost.
struct LinearSchedule { int64_t full, rest; int splits; double us; };
inline LinearSchedule linear_schedule(int64_t T, int64_t depth, int64_t slots, double step, double ends, double tile_mb) {
    const int64_t rest = T % slots, full = T - rest;
    const double round = depth * step + ends;
    LinearSchedule best{T, 0, 1, static_cast<double>((T + slots - 1) / slots) * round};
    if (rest == 0) return best;
    for (int64_t s = 2; s <= slots / rest && s * 4 <= depth; ++s) {
        const double us = full / slots * round + (depth + s - 1) / s * step + ends + 5.0 + 2.0 * rest * s * tile_mb / 4.5;
        if (us < best.us) best = {full, rest, static_cast<int>(s), us};
    }
    return best;
}

// The variant and its cut, by estimated times (us) from measured step times.
// Tiles, on whole rounds at 16,384 x 2,560 x 10,240: a 256 x 256 tile takes 1.65
// us a 128-byte k step (float32 7 us), two 128 x 128 tiles on a CU 1.1 us
// together (float32 3.5 us); the large tile moves half the operand bytes, the
// small one fills the CUs with four times fewer outputs.  Few columns: 0.38 us
// a step of a round of 64-row workgroups (float32 0.22 + 0.11 for each 16
// columns, its matrix rate).  Few outputs: what they read, the operands once for
// each block of the other, comes at 6 TB/s, mostly from L2.
// Estimated and measured (us), bfloat16: 1 x 2,560 x 10,240 13.3 and 14.0; 100 x
// 1,000 x 1,000 6.8 and 6.4; 32 and 128 x 2,560 x 10,240 20.2 and 20.9, 29.3 and
// 27.8; 512 x 2,560 x 10,240 48 and 57.  The estimate of few outputs knows neither
// rows that are no multiple of 16 bytes, nor how few compute units a small grid
// fills, nor what it writes: 300 x 1,537 x 333 8.1 and 14.6, in 8 bits 2,500 x 17 x
// 4,001 6.2 and 74.  Nor does that of tiles know short uneven rows: 7,000 x 333 x
// 515 in 8 bits 9.1 and 19.8.
inline LinearPlan plan_linear(int64_t M, int64_t K, int64_t N, int dtype, int out_dtype, int64_t cus) {
    const int64_t kbytes = K * (dtype == MSSM_F32 ? 4 : dtype == MSSM_BF16 ? 2 : 1), depth = (kbytes + kLinearStepBytes - 1) / kLinearStepBytes;
    const bool f32 = dtype == MSSM_F32, even = kbytes % 16 == 0;
    const bool wide = dtype == MSSM_F8 && out_dtype == MSSM_F32;  // twice the fragment registers: no large tile
    auto mb = [&](int64_t t) { return 4e-6 * std::min(M, t) * std::min(N, t); };
    const LinearSchedule big = linear_schedule(((M + 255) / 256) * ((N + 255) / 256), depth, cus, f32 ? 7.0 : 1.65, 8.0, mb(256));
    const LinearSchedule small = linear_schedule(((M + 127) / 128) * ((N + 127) / 128), depth, 2 * cus, f32 ? 3.5 : even ? 1.1 : 1.7, 4.0, mb(128));
    const bool large = even && !wide && big.us < small.us;
    const LinearSchedule& s = large ? big : small;
    const int64_t tile = large ? 256 : 128;

    const int64_t block = M <= 16 ? 16 : M <= 32 ? 32 : 64, blocks_m = (M + block - 1) / block, blocks_n = (N + 15) / 16;
    const double read = static_cast<double>(blocks_n * M + blocks_m * N) * kbytes * 1e-6;
    const double flops = 2e-6 * blocks_m * block * blocks_n * 16 * K;
    const double rows = 4.0 + std::max(read / 6.0, flops / (f32 ? 100.0 : 500.0));
    const int64_t fn = (N + 15) / 16;
    const double columns = even && N <= 128 && M < (int64_t{1} << 28)
                               ? 3.0 + (M + 64 * cus - 1) / (64 * cus) * depth * (f32 ? 0.22 + 0.11 * fn : 0.38) : 1e30;
    // (a launch has fewer than 2^32 threads, and 65,535 row blocks)
    if (blocks_m < 65536 && blocks_n < (int64_t{1} << 22) && rows <= columns && rows <= s.us) return {LinearPath::kRows, 0, 0, 1, 0};
    if (columns <= s.us) return {LinearPath::kColumns, 0, 0, 1, 0};
    return {tile == 256 ? LinearPath::kTile256 : LinearPath::kTile128, s.full, s.rest, s.splits,
            s.splits > 1 ? static_cast<size_t>(s.splits) * s.rest * tile * tile * sizeof(float) : 0};
}

}  // namespace mssm
