// gdr_api.cpp -- the C ABI declared in include/mssm_gdr.h.
//
// Host-only layer, as mssm_api.cpp: every argument is checked before anything
// is enqueued, and a validated argument block goes to the kernel launchers.
#include "gdr.h"

#include <cmath>
#include <cstdint>
#include <initializer_list>

namespace {

using mssm::GdrArgs;
using mssm::GdrLayout;

mssm_status check_align(std::initializer_list<const void*> ptrs) {
    for (const void* q : ptrs)
        if (reinterpret_cast<uintptr_t>(q) & 15u) return MSSM_ERR_ALIGN;
    return MSSM_OK;
}

bool any_null(std::initializer_list<const void*> ptrs) {
    for (const void* q : ptrs)
        if (!q) return true;
    return false;
}

mssm_status from_hip(hipError_t e) { return e == hipSuccess ? MSSM_OK : MSSM_ERR_HIP; }

mssm_status check_problem(const mssm_gdr_problem* p) {
    if (!p) return MSSM_ERR_NULL;
    if (p->dtype != MSSM_F32 && p->dtype != MSSM_BF16) return MSSM_ERR_DTYPE;
    for (int64_t n : {p->tokens, p->seqs, p->qk_heads, p->heads, p->key_dim, p->value_dim})
        if (n < 1 || n >= (int64_t{1} << 31)) return MSSM_ERR_SHAPE;
    if (p->heads % p->qk_heads || !std::isfinite(p->scale)) return MSSM_ERR_SHAPE;
    if (p->key_dim % 16 || p->key_dim > MSSM_GDR_MAX_KEY_DIM || p->value_dim % 16 || p->value_dim > MSSM_GDR_MAX_VALUE_DIM)
        return MSSM_ERR_UNSUPPORTED;
    return MSSM_OK;
}

mssm_status check_chunked(const mssm_gdr_problem* p) {
    const mssm_status st = check_problem(p);
    if (st != MSSM_OK) return st;
    // byte offsets within a chunk stay below 2^31
    if (p->qk_heads * p->key_dim > (int64_t{1} << 22) || p->heads * p->value_dim > (int64_t{1} << 22)) return MSSM_ERR_SHAPE;
    // threads of a launch stay below 2^32: the chunks' kernels have up to 512 for each
    // chunk and head, the chains' 256 for 64 value columns of each sequence and head
    if (p->heads > (int64_t{1} << 20) || p->seqs > (int64_t{1} << 20) / p->heads) return MSSM_ERR_SHAPE;
    if (mssm::gdr_slots(p->tokens, p->seqs) >= (int64_t{1} << 23) / p->heads) return MSSM_ERR_SHAPE;
    return MSSM_OK;
}

// Device memory of a call, cut into 256-byte aligned parts.
struct Cut {
    uint8_t* at;
    size_t bytes = 0;
    explicit Cut(const void* p) : at(static_cast<uint8_t*>(const_cast<void*>(p))) {}
    void* take(size_t n) {
        void* p = at ? at + bytes : nullptr;
        bytes += (n + 255) / 256 * 256;
        return p;
    }
};

size_t cells(const mssm_gdr_problem* p) { return static_cast<size_t>(mssm::gdr_slots(p->tokens, p->seqs) * p->heads); }

// Sets the places of the forward's hand-over in `c`; train: of a ctx.
void place_forward(const mssm_gdr_problem* p, bool train, Cut& c, GdrArgs& a) {
    a.mats = static_cast<uint8_t*>(c.take(cells(p) * static_cast<size_t>(GdrLayout(train).bytes)));
    a.train = train;
    const mssm::GdrPieces pieces(p->tokens, p->seqs, p->heads, p->key_dim, p->value_dim, p->dtype);
    if (pieces.shift) {
        const size_t states = static_cast<size_t>(pieces.count * p->heads * p->key_dim) * 4;
        a.starts = static_cast<float*>(c.take(states * p->value_dim));
        a.moves = static_cast<float*>(c.take(states * p->key_dim));
    }
    if (!train) return;
    a.states = static_cast<float*>(c.take(cells(p) * p->value_dim * p->key_dim * 4));
    a.misses = static_cast<float*>(c.take(cells(p) * mssm::kGdrChunk * p->value_dim * 4));
}
void place_backward(const mssm_gdr_problem* p, Cut& c, GdrArgs& a) {
    a.adjoints = static_cast<float*>(c.take(cells(p) * p->value_dim * p->key_dim * 4));
    a.pulls = static_cast<float*>(c.take(cells(p) * mssm::kGdrChunk * p->value_dim * 4));
}

GdrArgs arguments(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g, const float* beta,
                  const float* h0, const int32_t* offsets) {
    GdrArgs a{};
    a.T = p->tokens; a.N = p->seqs; a.G = p->qk_heads; a.H = p->heads; a.K = p->key_dim; a.V = p->value_dim;
    a.dtype = p->dtype; a.norm = p->norm_qk != 0; a.scale = p->scale;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.h0 = h0; a.offsets = offsets;
    return a;
}

size_t ctx_size(const mssm_gdr_problem* p) {
    Cut c(nullptr);
    GdrArgs a{};
    place_forward(p, true, c, a);
    return c.bytes;
}
size_t saved_size(const mssm_gdr_problem* p) {
    Cut c(nullptr);
    GdrArgs a{};
    place_backward(p, c, a);
    return c.bytes;
}
size_t bwd_size(const mssm_gdr_problem* p) {
    Cut c(nullptr);
    GdrArgs a{};
    place_forward(p, true, c, a);
    place_backward(p, c, a);
    return c.bytes;
}
size_t fwd_size(const mssm_gdr_problem* p) {
    Cut c(nullptr);
    GdrArgs a{};
    place_forward(p, false, c, a);
    return c.bytes;
}

mssm_status run_forward(const GdrArgs& a, hipStream_t s) {
    const hipError_t e = mssm::launch_gdr_prep(a, s);
    return from_hip(e == hipSuccess ? mssm::launch_gdr_fwd(a, s) : e);
}

mssm_status forward(const mssm_gdr_problem* p, bool train, const void* q, const void* k, const void* v, const float* g,
                    const float* beta, const float* h0, const int32_t* offsets, void* y, float* h_final, void* mem,
                    size_t bytes, void* hip_stream) {
    mssm_status st = check_chunked(p);
    if (st != MSSM_OK) return st;
    if (any_null({q, k, v, g, beta, y})) return MSSM_ERR_NULL;
    if (!offsets && p->tokens % p->seqs) return MSSM_ERR_SHAPE;
    st = check_align({q, k, v, g, beta, h0, offsets, y, h_final, mem});
    if (st != MSSM_OK) return st;
    if (!mem || bytes < (train ? ctx_size(p) : fwd_size(p))) return MSSM_ERR_WORKSPACE;
    GdrArgs a = arguments(p, q, k, v, g, beta, h0, offsets);
    a.y = y; a.h_final = h_final;
    Cut c(mem);
    place_forward(p, train, c, a);
    return run_forward(a, static_cast<hipStream_t>(hip_stream));
}

mssm_status check_backward(const mssm_gdr_problem* p, const GdrArgs& a, const void* mem) {
    if (any_null({a.q, a.k, a.v, a.g, a.beta, a.dy, a.dq, a.dk, a.dv, a.dg, a.dbeta})) return MSSM_ERR_NULL;
    if (!a.offsets && p->tokens % p->seqs) return MSSM_ERR_SHAPE;
    return check_align({a.q, a.k, a.v, a.g, a.beta, a.h0, a.offsets, a.dy, a.dh_final, a.dq, a.dk, a.dv, a.dg, a.dbeta, a.dh0, mem});
}

}  // namespace

extern "C" {

size_t mssm_gdr_fwd_workspace_bytes(const mssm_gdr_problem* p) { return check_chunked(p) == MSSM_OK ? fwd_size(p) : 0; }

mssm_status mssm_gdr_fwd(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                         const float* beta, const float* h0, const int32_t* offsets, void* y, float* h_final,
                         void* workspace, size_t workspace_bytes, void* hip_stream) {
    return forward(p, false, q, k, v, g, beta, h0, offsets, y, h_final, workspace, workspace_bytes, hip_stream);
}

size_t mssm_gdr_ctx_bytes(const mssm_gdr_problem* p) { return check_chunked(p) == MSSM_OK ? ctx_size(p) : 0; }

mssm_status mssm_gdr_fwd_train(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const float* h0, const int32_t* offsets, void* y, float* h_final,
                               void* ctx, size_t ctx_bytes, void* hip_stream) {
    return forward(p, true, q, k, v, g, beta, h0, offsets, y, h_final, ctx, ctx_bytes, hip_stream);
}

size_t mssm_gdr_bwd_saved_workspace_bytes(const mssm_gdr_problem* p) { return check_chunked(p) == MSSM_OK ? saved_size(p) : 0; }

mssm_status mssm_gdr_bwd_saved(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const int32_t* offsets, const void* ctx, size_t ctx_bytes,
                               const void* dy, const float* dh_final, void* dq, void* dk, void* dv, float* dg,
                               float* dbeta, float* dh0, void* workspace, size_t workspace_bytes, void* hip_stream) {
    mssm_status st = check_chunked(p);
    if (st != MSSM_OK) return st;
    if (!ctx) return MSSM_ERR_NULL;
    GdrArgs a = arguments(p, q, k, v, g, beta, nullptr, offsets);
    a.dy = dy; a.dh_final = dh_final; a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0;
    st = check_backward(p, a, workspace);
    if (st == MSSM_OK) st = check_align({ctx});
    if (st != MSSM_OK) return st;
    if (ctx_bytes < ctx_size(p) || !workspace || workspace_bytes < saved_size(p)) return MSSM_ERR_WORKSPACE;
    Cut kept(ctx), c(workspace);
    place_forward(p, true, kept, a);
    place_backward(p, c, a);
    return from_hip(mssm::launch_gdr_bwd(a, static_cast<hipStream_t>(hip_stream)));
}

size_t mssm_gdr_bwd_workspace_bytes(const mssm_gdr_problem* p) { return check_chunked(p) == MSSM_OK ? bwd_size(p) : 0; }

mssm_status mssm_gdr_bwd(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                         const float* beta, const float* h0, const int32_t* offsets, const void* dy,
                         const float* dh_final, void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dh0,
                         void* workspace, size_t workspace_bytes, void* hip_stream) {
    mssm_status st = check_chunked(p);
    if (st != MSSM_OK) return st;
    GdrArgs a = arguments(p, q, k, v, g, beta, h0, offsets);
    a.dy = dy; a.dh_final = dh_final; a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0;
    st = check_backward(p, a, workspace);
    if (st != MSSM_OK) return st;
    if (!workspace || workspace_bytes < bwd_size(p)) return MSSM_ERR_WORKSPACE;
    Cut c(workspace);
    place_forward(p, true, c, a);
    place_backward(p, c, a);
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    st = run_forward(a, s);  // writes no y and no final state
    return st == MSSM_OK ? from_hip(mssm::launch_gdr_bwd(a, s)) : st;
}

mssm_status mssm_gdr_step(const mssm_gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                          const float* beta, const int32_t* slots, float* state, void* y, void* hip_stream) {
    mssm_status st = check_problem(p);
    if (st != MSSM_OK) return st;
    // a launch holds every value part of at least one row: up to 8 workgroups of 256 threads a head
    if (p->heads > (int64_t{1} << 20) || p->tokens >= (int64_t{1} << 31) / p->heads || (!slots && p->tokens > p->seqs)) return MSSM_ERR_SHAPE;
    if (any_null({q, k, v, g, beta, state, y})) return MSSM_ERR_NULL;
    st = check_align({q, k, v, g, beta, slots, state, y});
    if (st != MSSM_OK) return st;
    const mssm::GdrStepArgs a{p->tokens, p->seqs, p->qk_heads, p->heads, p->key_dim, p->value_dim, p->dtype,
                              p->norm_qk != 0, p->scale, q, k, v, g, beta, slots, state, y};
    return from_hip(mssm::launch_gdr_step(a, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
