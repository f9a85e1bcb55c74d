// delta_api.hip - the C entry points of the gated delta rule: argument checks and launches.
// Declarations and the contract of every entry point are in include/ssd.h.
#include "ssd.h"
#include "api_checks.hpp"
#include "common.hpp"
#include "kernels.hpp"

using namespace ssd;

namespace {

int check_delta(const DeltaDims& d)
{
    int rc = check_common(0, d.nheads, d.headdim, d.dstate, d.ngroups);
    if (rc != SSD_OK) return rc;
    if (d.seqs < 0 || d.seqs > (int64_t(1) << 24) || d.seqlen < 0 || d.tokens < 0) return SSD_ERR_SHAPE;
    if (d.tokens > INT32_MAX) return SSD_ERR_SHAPE;                      // cu_seqlens holds 32-bit offsets
    // one-dimensional grids of fewer than 2^32 threads: 256 a (block of 32 tokens, head); a (row, head) 128 to 192 for
    // each 16 or 32 columns of v, which the first limit covers, or 80 for each 16, for which there is the second
    if ((d.tokens / 32 + d.seqs) * d.nheads >= (int64_t(1) << 24)) return SSD_ERR_SHAPE;
    if (d.seqs * d.nheads * d.headdim >= (int64_t(1) << 29)) return SSD_ERR_SHAPE;
    if (d.tokens * d.nheads * (d.headdim > d.dstate ? d.headdim : d.dstate) > (int64_t(1) << 40)) return SSD_ERR_SHAPE;
    if (d.seqs * d.nheads * d.headdim * d.dstate > (int64_t(1) << 40)) return SSD_ERR_SHAPE;
    return SSD_OK;
}

// The sizes of a batch of rows of seqlen tokens; sizes out of range leave tokens at -1 (refused by
// check_delta), so that no product overflows.
DeltaDims batch_dims(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups)
{
    const bool ok = batch >= 0 && batch <= 65535 && seqlen >= 0 && seqlen <= INT32_MAX;
    return DeltaDims{batch, seqlen, ok ? batch * seqlen : -1, nheads, headdim, dstate, ngroups, nullptr};
}

int delta_forward_impl(const void* v, const float* g, const float* beta, const void* k, const void* q,
                       const float* init_states, void* y, float* final_states, const DeltaDims& d, int dtype,
                       void* workspace, size_t workspace_bytes, void* stream)
{
    if (!valid_dtype(dtype)) return SSD_ERR_DTYPE;
    int rc = check_delta(d);
    if (rc != SSD_OK) return rc;
    if (d.seqs == 0) return SSD_OK;
    if (!final_states) return SSD_ERR_NULL;
    if (d.tokens > 0 && (!v || !g || !beta || !k || !q || !y)) return SSD_ERR_NULL;
    const size_t es = elem_size(dtype);
    const size_t need = delta_forward_workspace(d, (int)es);
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!workspace) return SSD_ERR_NULL;
    if (!aligned16(workspace) || !aligned16(v) || !aligned16(k) || !aligned16(q) || !aligned16(y) ||
        !aligned16(init_states) || !aligned16(final_states))
        return SSD_ERR_SHAPE;
    const size_t nv = (size_t)(d.tokens * d.nheads * d.headdim) * es;
    const size_t nk = (size_t)(d.tokens * d.ngroups * d.dstate) * es;
    const size_t ng = (size_t)(d.tokens * d.nheads) * 4;
    const size_t nst = (size_t)(d.seqs * d.nheads * d.headdim * d.dstate) * 4;
    if (any_overlap({{y, nv}, {final_states, nst}, {workspace, need}},
                    {{v, nv}, {g, ng}, {beta, ng}, {k, nk}, {q, nk}, {init_states, nst},
                     {d.cu, (size_t)(d.seqs + 1) * 4}}))
        return SSD_ERR_ALIAS;
    hipStream_t s = (hipStream_t)stream;
    if (dtype == SSD_BF16)
        return hip_status(launch_delta_forward<bf16>((const bf16*)v, g, beta, (const bf16*)k, (const bf16*)q,
                                                     init_states, (bf16*)y, final_states, d, workspace, s));
    return hip_status(launch_delta_forward<float>((const float*)v, g, beta, (const float*)k, (const float*)q,
                                                  init_states, (float*)y, final_states, d, workspace, s));
}

}  // namespace

extern "C" {

size_t ssd_delta_forward_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                         int64_t dstate, int64_t ngroups, int dtype)
{
    const DeltaDims d = batch_dims(batch, seqlen, nheads, headdim, dstate, ngroups);
    if (!valid_dtype(dtype) || check_delta(d) != SSD_OK) return 0;
    return delta_forward_workspace(d, (int)elem_size(dtype));
}

int ssd_delta_forward(const void* v, const float* g, const float* beta, const void* k, const void* q,
                      const float* init_states, void* y, float* final_states, int64_t batch, int64_t seqlen,
                      int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups, int dtype, void* workspace,
                      size_t workspace_bytes, void* stream)
{
    return delta_forward_impl(v, g, beta, k, q, init_states, y, final_states,
                              batch_dims(batch, seqlen, nheads, headdim, dstate, ngroups), dtype, workspace,
                              workspace_bytes, stream);
}

size_t ssd_delta_forward_varlen_workspace_bytes(int64_t total_tokens, int64_t nseq, int64_t nheads, int64_t headdim,
                                                int64_t dstate, int64_t ngroups, int dtype)
{
    // the size depends on the offsets' presence, not on their content
    static const int32_t present = 0;
    const DeltaDims d{nseq, 0, total_tokens, nheads, headdim, dstate, ngroups, &present};
    if (!valid_dtype(dtype) || check_delta(d) != SSD_OK) return 0;
    return delta_forward_workspace(d, (int)elem_size(dtype));
}

int ssd_delta_forward_varlen(const void* v, const float* g, const float* beta, const void* k, const void* q,
                             const int32_t* cu_seqlens, int64_t nseq, const float* init_states, void* y,
                             float* final_states, int64_t total_tokens, int64_t nheads, int64_t headdim,
                             int64_t dstate, int64_t ngroups, int dtype, void* workspace, size_t workspace_bytes,
                             void* stream)
{
    const DeltaDims d{nseq, 0, total_tokens, nheads, headdim, dstate, ngroups, cu_seqlens};
    if (!valid_dtype(dtype)) return SSD_ERR_DTYPE;
    int rc = check_delta(d);
    if (rc != SSD_OK) return rc;
    if (nseq == 0 && total_tokens > 0) return SSD_ERR_SHAPE;
    if (nseq > 0 && !cu_seqlens) return SSD_ERR_NULL;
    return delta_forward_impl(v, g, beta, k, q, init_states, y, final_states, d, dtype, workspace, workspace_bytes,
                              stream);
}

size_t ssd_delta_backward_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                          int64_t dstate, int64_t ngroups, int dtype)
{
    const DeltaDims d = batch_dims(batch, seqlen, nheads, headdim, dstate, ngroups);
    if (!valid_dtype(dtype) || check_delta(d) != SSD_OK) return 0;
    return delta_backward_workspace(d, (int)elem_size(dtype));
}

int ssd_delta_backward(const void* v, const float* g, const float* beta, const void* k, const void* q,
                       const float* init_states, const void* dy, const float* dfinal, void* dv, float* dg,
                       float* dbeta, void* dk, void* dq, float* dinit, int64_t batch, int64_t seqlen, int64_t nheads,
                       int64_t headdim, int64_t dstate, int64_t ngroups, int dtype, void* workspace,
                       size_t workspace_bytes, void* stream)
{
    const DeltaDims d = batch_dims(batch, seqlen, nheads, headdim, dstate, ngroups);
    if (!valid_dtype(dtype)) return SSD_ERR_DTYPE;
    int rc = check_delta(d);
    if (rc != SSD_OK) return rc;
    if (batch == 0) return SSD_OK;
    if (!dinit) return SSD_ERR_NULL;
    if (seqlen > 0 && (!v || !g || !beta || !k || !q || !dy || !dv || !dg || !dbeta || !dk || !dq)) return SSD_ERR_NULL;
    const size_t es = elem_size(dtype);
    const size_t need = delta_backward_workspace(d, (int)es);
    if (workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!workspace) return SSD_ERR_NULL;
    if (!aligned16(workspace) || !aligned16(v) || !aligned16(k) || !aligned16(q) || !aligned16(dy) || !aligned16(dv) ||
        !aligned16(dk) || !aligned16(dq) || !aligned16(init_states) || !aligned16(dfinal) || !aligned16(dinit))
        return SSD_ERR_SHAPE;
    const size_t nv = (size_t)(d.tokens * nheads * headdim) * es;
    const size_t nk = (size_t)(d.tokens * ngroups * dstate) * es;
    const size_t ng = (size_t)(d.tokens * nheads) * 4;
    const size_t nst = (size_t)(batch * nheads * headdim * dstate) * 4;
    if (any_overlap({{dv, nv}, {dg, ng}, {dbeta, ng}, {dk, nk}, {dq, nk}, {dinit, nst}, {workspace, need}},
                    {{v, nv}, {g, ng}, {beta, ng}, {k, nk}, {q, nk}, {init_states, nst}, {dy, nv}, {dfinal, nst}}))
        return SSD_ERR_ALIAS;
    hipStream_t s = (hipStream_t)stream;
    if (dtype == SSD_BF16)
        return hip_status(launch_delta_backward<bf16>((const bf16*)v, g, beta, (const bf16*)k, (const bf16*)q,
                                                      init_states, (const bf16*)dy, dfinal, (bf16*)dv, dg, dbeta,
                                                      (bf16*)dk, (bf16*)dq, dinit, d, workspace, s));
    return hip_status(launch_delta_backward<float>((const float*)v, g, beta, (const float*)k, (const float*)q,
                                                   init_states, (const float*)dy, dfinal, (float*)dv, dg, dbeta,
                                                   (float*)dk, (float*)dq, dinit, d, workspace, s));
}

int ssd_delta_step(float* state, const void* v, const float* g, const float* beta, const void* k, const void* q,
                   void* y, int64_t batch, int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups,
                   int dtype, void* stream)
{
    if (!valid_dtype(dtype)) return SSD_ERR_DTYPE;
    int rc = check_common(batch, nheads, headdim, dstate, ngroups);
    if (rc != SSD_OK) return rc;
    if (batch * nheads >= (int64_t(1) << 24)) return SSD_ERR_SHAPE;      // a grid of fewer than 2^32 threads
    if (batch == 0) return SSD_OK;
    if (!state || !v || !g || !beta || !k || !q || !y) return SSD_ERR_NULL;
    if (!aligned16(state)) return SSD_ERR_SHAPE;
    const size_t es = elem_size(dtype);
    const size_t nst = (size_t)(batch * nheads * headdim * dstate) * 4;
    const size_t nv = (size_t)(batch * nheads * headdim) * es;
    const size_t nk = (size_t)(batch * ngroups * dstate) * es;
    const size_t ng = (size_t)(batch * nheads) * 4;
    if (any_overlap({{y, nv}, {state, nst}}, {{v, nv}, {g, ng}, {beta, ng}, {k, nk}, {q, nk}})) return SSD_ERR_ALIAS;
    const DeltaDims d{batch, 1, batch, nheads, headdim, dstate, ngroups, nullptr};
    hipStream_t s = (hipStream_t)stream;
    if (dtype == SSD_BF16)
        return hip_status(launch_delta_step<bf16>(state, (const bf16*)v, g, beta, (const bf16*)k, (const bf16*)q,
                                                  (bf16*)y, d, s));
    return hip_status(launch_delta_step<float>(state, (const float*)v, g, beta, (const float*)k, (const float*)q,
                                               (float*)y, d, s));
}

}  // extern "C"
