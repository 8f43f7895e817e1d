// Host side of the C ABI, continued: the balance loss.
#include <hip/hip_runtime.h>

#include <cmath>
#include <vector>

#include "api.hpp"
#include "balance.hpp"
#include "dlm.h"
#include "route.hpp"

using namespace dlm;

extern "C" {

// --------------------------------------------------------------- balance ----

// Checks and arguments shared by dlm_balance and dlm_balance_backward.
static int balance_args(const char* call, const void* logits, int64_t ld, const int32_t* offsets, int32_t n_seq, int64_t T,
                        int32_t E, int32_t dtype, const dlm_balance_cfg* c, BalanceArgs* a) {
    if (!c) return fail(DLM_EINVAL, "%s: cfg is null", call);
    if (T < 0 || T >= ((int64_t)1 << 31)) return fail(DLM_ESHAPE, "%s: T=%lld out of range", call, (long long)T);
    if (E < 1 || E > DLM_MAX_ROUTE_EXPERTS)
        return fail(DLM_ESHAPE, "%s: E=%d not in [1, %d]", call, E, DLM_MAX_ROUTE_EXPERTS);
    if (n_seq < 1 || n_seq > DLM_MAX_BALANCE_SEQS)
        return fail(DLM_ESHAPE, "%s: %d sequences, not in [1, %d]", call, n_seq, DLM_MAX_BALANCE_SEQS);
    if (!offsets && n_seq != 1) return fail(DLM_EINVAL, "%s: %d sequences without offsets", call, n_seq);
    if (!valid_dtype(dtype)) return fail(DLM_EDTYPE, "%s: unknown dtype %d", call, dtype);
    if (ld < E || ld > kMaxDim) return fail(DLM_ESHAPE, "%s: row pitch %lld of rows of %d", call, (long long)ld, E);
    if (c->k < 1 || c->k > DLM_MAX_ROUTE_K) return fail(DLM_ESHAPE, "%s: k=%d not in [1, %d]", call, c->k, DLM_MAX_ROUTE_K);
    if (c->score != DLM_SOFTMAX && c->score != DLM_SIGMOID) return fail(DLM_EINVAL, "%s: unknown score %d", call, c->score);
    if (!std::isfinite(c->alpha) || !std::isfinite(c->zeta))
        return fail(DLM_EINVAL, "%s: alpha=%g, zeta=%g are not both finite", call, c->alpha, c->zeta);
    if (c->score == DLM_SIGMOID && c->zeta != 0.f)
        return fail(DLM_EINVAL, "%s: zeta=%g with sigmoid scores, which have no log sum", call, c->zeta);
    if ((uintptr_t)logits % esize(dtype) || (uintptr_t)offsets % 4)
        return fail(DLM_EALIGN, "%s: a pointer is not a multiple of its element's size", call);
    *a = BalanceArgs{};
    a->logits = logits;
    a->ld = ld;
    a->T = T;
    a->offsets = offsets;
    a->S = n_seq;
    a->E = E;
    a->k = c->k;
    a->score = c->score;
    a->alpha = c->alpha;
    a->zeta = c->zeta;
    const int64_t w = 16 / (int64_t)esize(dtype);
    a->vec = aligned16(logits) && ld % w == 0 && E % w == 0;
    return DLM_OK;
}

int dlm_balance_workspace_size(int64_t T, int32_t E, int32_t n_seq, size_t* bytes) {
    if (!bytes) return fail(DLM_EINVAL, "balance_workspace_size: bytes is null");
    if (T < 0 || T >= ((int64_t)1 << 31) || E < 1 || E > DLM_MAX_ROUTE_EXPERTS || n_seq < 1 || n_seq > DLM_MAX_BALANCE_SEQS)
        return fail(DLM_ESHAPE, "balance_workspace_size: T=%lld, E=%d, n_seq=%d out of range", (long long)T, E, n_seq);
    *bytes = balance_layout(T, E, n_seq).bytes;
    return ok();
}

int dlm_balance(const void* logits, int64_t ld, const int32_t* idx, const int32_t* offsets, int32_t n_seq, int64_t T,
                int32_t E, int32_t dtype, const dlm_balance_cfg* cfg, float* loss, int32_t* counts, int32_t* rows,
                float* probs, void* workspace, size_t ws_bytes, void* stream) {
    BalanceArgs a;
    const int rc = balance_args("balance", logits, ld, offsets, n_seq, T, E, dtype, cfg, &a);
    if (rc != DLM_OK) return rc;
    if ((T > 0 && (!logits || !idx)) || !loss || !counts || !rows || !probs) return fail(DLM_EINVAL, "balance: null pointer");
    const BalanceLayout w = balance_layout(T, E, n_seq);
    if (!workspace || ws_bytes < w.bytes)
        return fail(DLM_EWORKSPACE, "balance: workspace of %zu bytes, %zu needed", workspace ? ws_bytes : (size_t)0, w.bytes);
    if ((uintptr_t)workspace % 256) return fail(DLM_EALIGN, "balance: workspace is not 256-byte aligned");
    if ((uintptr_t)idx % 4 || (uintptr_t)loss % 4 || (uintptr_t)counts % 4 || (uintptr_t)rows % 4 || (uintptr_t)probs % 4)
        return fail(DLM_EALIGN, "balance: a pointer is not a multiple of its element's size");
    const size_t se = (size_t)n_seq * E * 4;
    const Span v[] = {span(logits, T ? rows_bytes(T, ld, E, esize(dtype)) : 0, false, "logits", 0),
                      span(idx, (size_t)T * a.k * 4, false, "idx", 0),
                      span(offsets, offsets ? (size_t)(n_seq + 1) * 4 : 0, false, "offsets", 0),
                      span(loss, 8, true, "loss", 0), span(counts, se, true, "counts", 0),
                      span(rows, (size_t)n_seq * 4, true, "rows", 0), span(probs, se, true, "probs", 0),
                      span(workspace, w.bytes, true, "workspace", 0)};
    Span p, q;
    if (pair_conflict(v, &p, &q)) return conflict_fail("balance", p, q);
    char* ws = (char*)workspace;
    a.idx = idx;
    a.per = w.per;
    a.blocks = w.blocks;
    a.part_p = (double*)(ws + w.p);
    a.part_z = (double*)(ws + w.z);
    a.seq = (double*)(ws + w.seq);
    a.part_c = (int32_t*)(ws + w.c);
    a.part_n = (int32_t*)(ws + w.n);
    a.ticket = (uint32_t*)(ws + w.ticket);
    a.loss = loss;
    a.counts = counts;
    a.rows = rows;
    a.probs = probs;
    const hipError_t e = launch_balance(a, dtype, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "balance launch");
    return ok();
}

int dlm_balance_backward(const void* logits, int64_t ld, const int32_t* counts, const int32_t* rows, const int32_t* offsets,
                         int32_t n_seq, int64_t T, int32_t E, int32_t dtype, const dlm_balance_cfg* cfg, const float* dloss,
                         int32_t accumulate, void* dlogits, int64_t ldd, void* stream) {
    BalanceArgs a;
    const int rc = balance_args("balance_backward", logits, ld, offsets, n_seq, T, E, dtype, cfg, &a);
    if (rc != DLM_OK) return rc;
    if (ldd < E || ldd > kMaxDim)
        return fail(DLM_ESHAPE, "balance_backward: row pitch %lld of dlogits rows of %d", (long long)ldd, E);
    if (T == 0) return ok();
    if (!logits || !counts || !rows || !dlogits) return fail(DLM_EINVAL, "balance_backward: null pointer");
    const size_t es = esize(dtype);
    if ((uintptr_t)counts % 4 || (uintptr_t)rows % 4 || (uintptr_t)dloss % 4 || (uintptr_t)dlogits % es)
        return fail(DLM_EALIGN, "balance_backward: a pointer is not a multiple of its element's size");
    const Span v[] = {span(logits, rows_bytes(T, ld, E, es), false, "logits", 0),
                      span(dlogits, rows_bytes(T, ldd, E, es), true, "dlogits", 0),
                      span(counts, (size_t)n_seq * E * 4, false, "counts", 0), span(rows, (size_t)n_seq * 4, false, "rows", 0),
                      span(offsets, offsets ? (size_t)(n_seq + 1) * 4 : 0, false, "offsets", 0),
                      span(dloss, dloss ? 8 : 0, false, "dloss", 0)};
    Span p, q;
    if (pair_conflict(v, &p, &q)) return conflict_fail("balance_backward", p, q);
    a.in_counts = counts;
    a.in_rows = rows;
    a.dloss = dloss;
    a.accumulate = accumulate ? 1 : 0;
    a.dlogits = dlogits;
    a.ldd = ldd;
    const int64_t w = 16 / (int64_t)es;
    a.vec_out = aligned16(dlogits) && ldd % w == 0 && E % w == 0;
    const hipError_t e = launch_balance_grad(a, dtype, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "balance_backward launch");
    return ok();
}

}  // extern "C"
