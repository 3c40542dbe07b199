// gdr.h -- host-side interface between the C ABI of the gated delta rule
// (gdr_api.cpp) and its kernel launchers (gdr_prep.hip, gdr_fwd.hip,
// gdr_bwd.hip, gdr_step.hip), and the layout of what they hand over.  Internal.
// Element types are numbered as in the headers: 0 = float32, 1 = bfloat16.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mssm_gdr.h"

namespace mssm {

constexpr int kGdrChunk = 64;         // tokens of a chunk
constexpr float kGdrLeast = -200.0f;  // log decays below count as this: exp is 0 in float32
constexpr float kGdrNormEps = 1e-6f;  // added to the squared length of q and k

// Chunks are numbered without a sum over the sequences: sequence n that starts
// at token s has the slots s / 64 + n, s / 64 + n + 1, ... (the next sequence's
// first is at least ceil(length / 64) further), of T / 64 + N in all.
inline int64_t gdr_slots(int64_t tokens, int64_t seqs) { return tokens / kGdrChunk + seqs; }

// The pieces of the sequences that the forward's chains go through side by side:
// 2^shift tokens each, numbered as the chunks are, `count` in all; shift = 0: whole
// sequences.
struct GdrPieces {
    int shift = 0;
    int64_t count;
    GdrPieces(int64_t T, int64_t N, int64_t H, int64_t K, int64_t V, int dtype);
};

// Which piece of a sequence (`first`, `last`: of its pieces) reads h0 in which launch:
// the one that finds the pieces' ends (`ends`; it has no last pieces) or the one that
// goes through them.  h_final may be h0's buffer, and its last piece's workgroup writes
// it in the latter: there only a piece by itself reads h0, other first pieces take the
// copy that the former made.
constexpr bool gdr_reads_h0(bool ends, bool first, bool last) { return first && last != ends; }
constexpr bool gdr_writes_h_final(bool ends, bool last) { return !ends && last; }

// What the chunk-parallel pass leaves for each (slot, head), in bytes: of the
// matrices N and P their 6 blocks of 16 x 32 that are not zero, in the order of the
// matrix instructions' operands, N as three bfloat16 planes of 1 KB that add up to
// the float32 value, P in float32 (2 KB a block, cut into the same planes by who
// multiplies with it), 5 rows of 64 factors, and for the backward the transposes of
// both in planes.
constexpr int kGdrBlocks = 6;
constexpr int kGdrBlockBytes = 1024;
constexpr int kGdrFactors = 5;
struct GdrLayout {
    int64_t pm, n, factors, nt, pt, bytes;
    explicit GdrLayout(bool train) {
        pm = 0;  // the forward's P, N and factors and the backward's factors and transposes lie together
        n = pm + 2 * kGdrBlocks * kGdrBlockBytes;
        factors = n + 3 * kGdrBlocks * kGdrBlockBytes;
        nt = factors + kGdrFactors * kGdrChunk * 4;
        pt = nt + (train ? 3 * kGdrBlocks * kGdrBlockBytes : 0);
        bytes = pt + (train ? 3 * kGdrBlocks * kGdrBlockBytes : 0);
    }
};

struct GdrArgs {
    int64_t T, N, G, H, K, V;
    int dtype, norm;
    float scale;
    const void *q, *k, *v;
    const float *g, *beta;
    const float* h0;         // nullable
    const int32_t* offsets;  // nullable: equal lengths
    void* y;
    float* h_final;          // nullable
    // chunk matrices (slots, H, GdrLayout::bytes)
    uint8_t* mats;
    float* starts;           // (pieces, H, V, K) the state before a piece (none for a sequence of one)
    float* moves;            // (pieces, H, K, K) what a piece makes of a state's rows, transposed
    bool train;              // with the transposes, the states and the misses:
    float* states;           // (slots, H, V, K) before every chunk; null: not kept
    float* misses;           // (slots, H, 64, V) e; null: not kept
    // backward
    const void* dy;
    const float* dh_final;   // nullable
    void *dq, *dk, *dv;
    float *dg, *dbeta;
    float* dh0;              // nullable
    float* adjoints;         // (slots, H, V, K) of the state behind every chunk
    float* pulls;            // (slots, H, 64, V) Z, the adjoint of u with the chunk's later steps
};

hipError_t launch_gdr_prep(const GdrArgs& a, hipStream_t s);
hipError_t launch_gdr_fwd(const GdrArgs& a, hipStream_t s);
hipError_t launch_gdr_bwd(const GdrArgs& a, hipStream_t s);

struct GdrStepArgs {
    int64_t rows, pool, G, H, K, V;
    int dtype, norm;
    float scale;
    const void *q, *k, *v;
    const float *g, *beta;
    const int32_t* slots;  // nullable
    float* state;
    void* y;
};
hipError_t launch_gdr_step(const GdrStepArgs& a, hipStream_t s);

}  // namespace mssm
