// linear_api.hip - the C entry points of linear attention with a decay for each head and of pools of states: argument
// checks and launches.  Declarations and the contract of every entry point are in include/ssd.h.
#include "ssd.h"
#include "api_checks.hpp"
#include "common.hpp"
#include "kernels.hpp"

using namespace ssd;

namespace {

bool width_ok(int64_t w) { return w >= 16 && w <= 256 && w % 16 == 0; }

int check_heads(int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups)
{
    if (nheads < 1 || nheads > 65535 || !width_ok(headdim) || !width_ok(dstate)) return SSD_ERR_SHAPE;
    if (ngroups < 1 || nheads % ngroups != 0) return SSD_ERR_SHAPE;
    // 32 tokens of an operand are addressed by 32-bit offsets
    if (nheads * (headdim > dstate ? headdim : dstate) > (int64_t(1) << 20)) return SSD_ERR_SHAPE;
    return SSD_OK;
}

int check_linear(const DeltaDims& d, size_t es)
{
    int rc = check_heads(d.nheads, d.headdim, d.dstate, d.ngroups);
    if (rc != SSD_OK) return rc;
    if (d.seqs < 0 || d.seqs > (int64_t(1) << 24) || d.seqlen < 0 || d.tokens < 0) return SSD_ERR_SHAPE;
    if (d.tokens > INT32_MAX) return SSD_ERR_SHAPE;                      // cu_seqlens holds 32-bit offsets
    if (d.tokens * d.nheads * (d.headdim > d.dstate ? d.headdim : d.dstate) > (int64_t(1) << 40)) return SSD_ERR_SHAPE;
    if (d.seqs * d.nheads * d.headdim * d.dstate > (int64_t(1) << 40)) return SSD_ERR_SHAPE;
    // one-dimensional grids of fewer than 2^32 threads: the walks', the carry's (a thread for 4 elements of a row's
    // states) and the sums' over the heads that share a key
    if (linear_blocks(d, (int)es) >= (int64_t(1) << 24)) return SSD_ERR_SHAPE;
    if (d.seqs * d.nheads * (d.headdim * d.dstate / 4) >= (int64_t(1) << 32) - 256) return SSD_ERR_SHAPE;
    if (d.tokens * d.ngroups * ((d.headdim > d.dstate ? d.headdim : d.dstate) / 4) >= (int64_t(1) << 32) - 256)
        return SSD_ERR_SHAPE;
    return SSD_OK;
}

// The sizes of a batch of rows of seqlen tokens; sizes out of range leave tokens at -1 (refused by
// check_linear), so that no product overflows.
DeltaDims batch_dims(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups)
{
    const bool ok = batch >= 0 && batch <= 65535 && seqlen >= 0 && seqlen <= INT32_MAX;
    return DeltaDims{batch, seqlen, ok ? batch * seqlen : -1, nheads, headdim, dstate, ngroups, nullptr};
}

struct Spans {
    size_t q, y, k, v, state;
};
Spans spans(const DeltaDims& d, size_t es)
{
    return {(size_t)(d.tokens * d.nheads * d.dstate) * es, (size_t)(d.tokens * d.nheads * d.headdim) * es,
            (size_t)(d.tokens * d.ngroups * d.dstate) * es, (size_t)(d.tokens * d.ngroups * d.headdim) * es,
            (size_t)(d.seqs * d.nheads * d.headdim * d.dstate) * 4};
}

int linear_forward_impl(const void* v, const float* g, const void* k, const void* q, const float* init_states, void* y,
                        float* final_states, const DeltaDims& d, int dtype, void* workspace, size_t workspace_bytes,
                        void* stream)
{
    if (!valid_dtype(dtype)) return SSD_ERR_DTYPE;
    const size_t es = elem_size(dtype);
    int rc = check_linear(d, es);
    if (rc != SSD_OK) return rc;
    if (d.seqs == 0) return SSD_OK;
    if (!final_states || !g) return SSD_ERR_NULL;
    if (d.tokens > 0 && (!v || !k || !q || !y)) return SSD_ERR_NULL;
    const size_t need = linear_forward_workspace(d, (int)es);
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!workspace) return SSD_ERR_NULL;
    if (!aligned16(workspace) || !aligned16(v) || !aligned16(k) || !aligned16(q) || !aligned16(y) ||
        !aligned16(init_states) || !aligned16(final_states))
        return SSD_ERR_SHAPE;
    const Spans n = spans(d, es);
    if (any_overlap({{y, n.y}, {final_states, n.state}, {workspace, need}},
                    {{v, n.v}, {g, (size_t)d.nheads * 4}, {k, n.k}, {q, n.q}, {init_states, n.state},
                     {d.cu, (size_t)(d.seqs + 1) * 4}}))
        return SSD_ERR_ALIAS;
    hipStream_t s = (hipStream_t)stream;
    if (dtype == SSD_BF16)
        return hip_status(launch_linear_forward<bf16>((const bf16*)v, g, (const bf16*)k, (const bf16*)q, init_states,
                                                      (bf16*)y, final_states, d, workspace, s));
    return hip_status(launch_linear_forward<float>((const float*)v, g, (const float*)k, (const float*)q, init_states,
                                                   (float*)y, final_states, d, workspace, s));
}

}  // namespace

extern "C" {

size_t ssd_linear_forward_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                          int64_t dstate, int64_t ngroups, int dtype)
{
    const DeltaDims d = batch_dims(batch, seqlen, nheads, headdim, dstate, ngroups);
    if (!valid_dtype(dtype) || check_linear(d, elem_size(dtype)) != SSD_OK) return 0;
    return linear_forward_workspace(d, (int)elem_size(dtype));
}

int ssd_linear_forward(const void* v, const float* g, const void* k, const void* q, const float* init_states, void* y,
                       float* final_states, int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                       int64_t dstate, int64_t ngroups, int dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    return linear_forward_impl(v, g, k, q, init_states, y, final_states,
                               batch_dims(batch, seqlen, nheads, headdim, dstate, ngroups), dtype, workspace,
                               workspace_bytes, stream);
}

size_t ssd_linear_forward_varlen_workspace_bytes(int64_t total_tokens, int64_t nseq, int64_t nheads, int64_t headdim,
                                                 int64_t dstate, int64_t ngroups, int dtype)
{
    // the size depends on the offsets' presence, not on their content
    static const int32_t present = 0;
    const DeltaDims d{nseq, 0, total_tokens, nheads, headdim, dstate, ngroups, &present};
    if (!valid_dtype(dtype) || check_linear(d, elem_size(dtype)) != SSD_OK) return 0;
    return linear_forward_workspace(d, (int)elem_size(dtype));
}

int ssd_linear_forward_varlen(const void* v, const float* g, const void* k, const void* q, const int32_t* cu_seqlens,
                              int64_t nseq, const float* init_states, void* y, float* final_states,
                              int64_t total_tokens, int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups,
                              int dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!valid_dtype(dtype)) return SSD_ERR_DTYPE;
    static const int32_t present = 0;
    const int rc = check_linear(DeltaDims{nseq, 0, total_tokens, nheads, headdim, dstate, ngroups, &present},
                                elem_size(dtype));
    if (rc != SSD_OK) return rc;
    if (nseq == 0 && total_tokens > 0) return SSD_ERR_SHAPE;
    if (nseq > 0 && !cu_seqlens) return SSD_ERR_NULL;
    return linear_forward_impl(v, g, k, q, init_states, y, final_states,
                               DeltaDims{nseq, 0, total_tokens, nheads, headdim, dstate, ngroups, cu_seqlens}, dtype,
                               workspace, workspace_bytes, stream);
}

size_t ssd_linear_backward_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                           int64_t dstate, int64_t ngroups, int dtype)
{
    const DeltaDims d = batch_dims(batch, seqlen, nheads, headdim, dstate, ngroups);
    if (!valid_dtype(dtype) || check_linear(d, elem_size(dtype)) != SSD_OK) return 0;
    return linear_backward_workspace(d, (int)elem_size(dtype));
}

int ssd_linear_backward(const void* v, const float* g, const void* k, const void* q, const float* init_states,
                        const void* dy, const float* dfinal, void* dv, float* dg, void* dk, void* dq, float* dinit,
                        int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t dstate,
                        int64_t ngroups, int dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    const DeltaDims d = batch_dims(batch, seqlen, nheads, headdim, dstate, ngroups);
    if (!valid_dtype(dtype)) return SSD_ERR_DTYPE;
    const size_t es = elem_size(dtype);
    int rc = check_linear(d, es);
    if (rc != SSD_OK) return rc;
    if (!g || !dg) return SSD_ERR_NULL;                                  // (dg is written without rows too: zeros)
    if (batch > 0 && !dinit) return SSD_ERR_NULL;
    if (d.tokens > 0 && (!v || !k || !q || !dy || !dv || !dk || !dq)) return SSD_ERR_NULL;
    const size_t need = linear_backward_workspace(d, (int)es);
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!workspace) return SSD_ERR_NULL;
    if (!aligned16(workspace) || !aligned16(v) || !aligned16(k) || !aligned16(q) || !aligned16(dy) || !aligned16(dv) ||
        !aligned16(dk) || !aligned16(dq) || !aligned16(init_states) || !aligned16(dfinal) || !aligned16(dinit))
        return SSD_ERR_SHAPE;
    const Spans n = spans(d, es);
    const size_t ng = (size_t)nheads * 4;
    if (any_overlap({{dv, n.v}, {dg, ng}, {dk, n.k}, {dq, n.q}, {dinit, n.state}, {workspace, need}},
                    {{v, n.v}, {g, ng}, {k, n.k}, {q, n.q}, {init_states, n.state}, {dy, n.y}, {dfinal, n.state}}))
        return SSD_ERR_ALIAS;
    hipStream_t s = (hipStream_t)stream;
    if (dtype == SSD_BF16)
        return hip_status(launch_linear_backward<bf16>((const bf16*)v, g, (const bf16*)k, (const bf16*)q, init_states,
                                                       (const bf16*)dy, dfinal, (bf16*)dv, dg, (bf16*)dk, (bf16*)dq,
                                                       dinit, d, workspace, s));
    return hip_status(launch_linear_backward<float>((const float*)v, g, (const float*)k, (const float*)q, init_states,
                                                    (const float*)dy, dfinal, (float*)dv, dg, (float*)dk, (float*)dq,
                                                    dinit, d, workspace, s));
}

int ssd_linear_step(float* state, const int32_t* slots, int64_t nslots, const void* v, const float* g, const void* k,
                    const void* q, void* y, int64_t batch, int64_t nheads, int64_t headdim, int64_t dstate,
                    int64_t ngroups, int dtype, void* stream)
{
    if (!valid_dtype(dtype)) return SSD_ERR_DTYPE;
    int rc = check_heads(nheads, headdim, dstate, ngroups);
    if (rc != SSD_OK) return rc;
    if (batch < 0 || batch > 65535 || nslots < 0 || nslots > (int64_t(1) << 24)) return SSD_ERR_SHAPE;
    if (!slots && nslots != batch) return SSD_ERR_SHAPE;
    if (batch * nheads * (headdim / 16) >= (int64_t(1) << 24)) return SSD_ERR_SHAPE;      // a grid of fewer than 2^32 threads
    if (batch == 0) return SSD_OK;
    if (!v || !g || !k || !q || !y || (!state && nslots > 0)) return SSD_ERR_NULL;
    const size_t es = elem_size(dtype);
    if (!aligned16(state) || !aligned16(k) || !aligned16(q)) return SSD_ERR_SHAPE;
    const size_t nst = (size_t)(nslots * nheads * headdim * dstate) * 4;
    const size_t ny = (size_t)(batch * nheads * headdim) * es, nq = (size_t)(batch * nheads * dstate) * es;
    const size_t nv = (size_t)(batch * ngroups * headdim) * es, nk = (size_t)(batch * ngroups * dstate) * es;
    if (any_overlap({{y, ny}, {state, nst}},
                    {{v, nv}, {g, (size_t)nheads * 4}, {k, nk}, {q, nq}, {slots, (size_t)batch * 4}}))
        return SSD_ERR_ALIAS;
    const DeltaDims d{batch, 1, batch, nheads, headdim, dstate, ngroups, nullptr};
    hipStream_t s = (hipStream_t)stream;
    if (dtype == SSD_BF16)
        return hip_status(launch_linear_step<bf16>(state, slots, nslots, (const bf16*)v, g, (const bf16*)k,
                                                   (const bf16*)q, (bf16*)y, d, s));
    return hip_status(launch_linear_step<float>(state, slots, nslots, (const float*)v, g, (const float*)k,
                                                (const float*)q, (float*)y, d, s));
}

int ssd_state_move(float* states, const float* source, const int32_t* src, int64_t nlayers, int64_t nslots,
                   int64_t nsource, int64_t slot_floats, void* stream)
{
    if (nlayers < 0 || nlayers > 65535 || nslots < 0 || nslots > 65535 || nsource < 0 || nsource > (int64_t(1) << 24))
        return SSD_ERR_SHAPE;
    if (slot_floats < 4 || slot_floats % 4 != 0 || slot_floats > (int64_t(1) << 32)) return SSD_ERR_SHAPE;
    // in place a strip of all moves is held at once
    if (!source && (nsource != nslots || nslots > 2048)) return SSD_ERR_SHAPE;
    if (nlayers == 0 || nslots == 0) return SSD_OK;
    if (!states || !src) return SSD_ERR_NULL;
    if (!aligned16(states) || !aligned16(source)) return SSD_ERR_SHAPE;
    const size_t bytes = (size_t)(nlayers * slot_floats) * 4;
    if (any_overlap({{states, bytes * nslots}}, {{source, bytes * nsource}, {src, (size_t)nslots * 4}}))
        return SSD_ERR_ALIAS;
    return hip_status(launch_state_move(states, source, src, nlayers, nslots, nsource, slot_floats,
                                        (hipStream_t)stream));
}

}  // extern "C"
