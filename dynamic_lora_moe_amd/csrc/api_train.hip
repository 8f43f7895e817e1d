// Host side of the C ABI, continued: the balance loss, the orthogonalised
// momentum step and the 8-bit products.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <new>
#include <set>
#include <utility>
#include <vector>

#include "api.hpp"
#include "balance.hpp"
#include "dlm.h"
#include "int8.hpp"
#include "muon.hpp"
#include "route.hpp"

using namespace dlm;

// --------------------------------------------------------------- handles ----

struct dlm_muon {
    void* d_tables = nullptr;  // descriptors, work tables, error word
    void* d_work = nullptr;    // scratch of a step
    int32_t* d_err = nullptr;
    int32_t p_dtype = 0, g_dtype = 0;
    MuonArgs small[3] = {};  // small sides up to 16, 32, 64
    MuonArgs big{};
    int64_t big_elems = 0;  // of the largest tensor with big matrices
};

// One direction of the 8-bit products: its tables on the device.
struct I8Tables {
    void* d = nullptr;
    I8Args args{};
};

struct dlm_i8_group {
    std::vector<dlm_i8_problem> probs;
    int32_t dtype = 0;
    char* d_w = nullptr;              // packed weights, then their scales
    std::vector<size_t> w_at, s_at;   // of every problem
    I8Tables fwd, bwd;
    char* d_wt = nullptr;             // packed transposes
    std::vector<const void*> dy;      // bound buffers
    std::vector<void*> dx;
    bool bound = false;
    int64_t checked_fwd = 0, checked_bwd = 0;  // rows up to which the buffers are known not to overlap
};

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

// -------------------------------------------------------------------- muon ----

int dlm_muon_create(const dlm_muon_param* params, int32_t n, int32_t p_dtype, int32_t g_dtype, dlm_muon** out) {
    static_assert(kMuonMaxSide == DLM_MAX_MUON_SIDE && kMuonMaxSteps == DLM_MAX_MUON_STEPS, "muon limits");
    if (!out) return fail(DLM_EINVAL, "muon_create: out is null");
    *out = nullptr;
    if (!params || n < 1 || n > (1 << 20)) return fail(DLM_EINVAL, "muon_create: bad tensor list (n=%d)", n);
    if (!valid_dtype(p_dtype) || !valid_dtype(g_dtype))
        return fail(DLM_EDTYPE, "muon_create: unknown dtype (p %d, g %d)", p_dtype, g_dtype);
    const size_t ps = esize(p_dtype), gs = esize(g_dtype);
    dlm_muon* h = nullptr;
    std::vector<char> blob;
    size_t work = 0;
    // where a class's or the big matrices' tables and scratch lie: offsets until the memory is there
    struct Slot {
        size_t items, mats, part, pm, bad;
    };
    Slot slots[3] = {};
    size_t descs_at = 0, err_at = 0, big_at = 0, big_items = 0, big_pair = 0, big_sum = 0, big_sump = 0, big_mul = 0, big_mula = 0,
           big_out = 0, big_outa = 0, big_part = 0, big_sq = 0, big_meta = 0, big_bad = 0;
    std::vector<size_t> u_at;
    try {
        h = new dlm_muon();
        std::vector<MuDesc> descs(n);
        std::vector<Span> v;
        std::vector<int> nbs(n);
        u_at.assign(n, 0);
        for (int i = 0; i < n; ++i) {
            const dlm_muon_param& q = params[i];
            MuDesc& d = descs[i];
            const auto bad = [&](int rc) {
                delete h;
                return rc;
            };
            if (q.rows < 1 || q.cols < 1 || q.count < 0 || q.rows > kMaxDim || q.cols > kMaxDim || q.count > kMaxDim ||
                (double)q.rows * (double)q.cols * (double)q.count > (double)((int64_t)1 << 40))
                return bad(fail(DLM_ESHAPE, "muon_create: tensor %d: %lld matrices of %lld x %lld", i, (long long)q.count,
                                (long long)q.rows, (long long)q.cols));
            const bool wide = q.rows <= q.cols;
            const int64_t side = wide ? q.rows : q.cols, elems = q.count * q.rows * q.cols;
            if (side > kMuonMaxSide)
                return bad(fail(DLM_ESHAPE, "muon_create: tensor %d: the smaller side of %lld x %lld is above %d", i,
                                (long long)q.rows, (long long)q.cols, kMuonMaxSide));
            if (elems > 0 && (!q.p || !q.g || !q.m)) return bad(fail(DLM_EINVAL, "muon_create: tensor %d: null pointer", i));
            if (q.master && p_dtype == DLM_F32)
                return bad(fail(DLM_EINVAL, "muon_create: tensor %d: an fp32 parameter has no master", i));
            if (!std::isfinite(q.weight_decay) || !std::isfinite(q.scale))
                return bad(fail(DLM_EINVAL, "muon_create: tensor %d: weight_decay or scale is not finite", i));
            if ((uintptr_t)q.p % ps || (uintptr_t)q.g % gs || (uintptr_t)q.m % 4 || (uintptr_t)q.master % 4)
                return bad(fail(DLM_EALIGN, "muon_create: tensor %d: a pointer is not a multiple of its element's size", i));
            d = MuDesc{};
            d.p = q.p;
            d.g = q.g;
            d.master = q.master;
            d.m = q.m;
            d.d = wide ? q.cols : q.rows;
            d.n = (int32_t)side;
            d.wide = wide ? 1 : 0;
            d.count = q.count;
            d.vec = q.cols % 4 == 0 && (uintptr_t)q.p % (4 * ps) == 0 && (uintptr_t)q.g % (4 * gs) == 0 &&
                    (uintptr_t)q.m % 16 == 0 && (uintptr_t)q.master % 16 == 0;
            d.wd = q.weight_decay;
            d.scale = q.scale;
            nbs[i] = side <= 16 ? 1 : side <= 32 ? 2 : side <= kMuonTileSide ? 4 : 0;
            v.push_back(span(q.p, elems * ps, true, "p", i));
            v.push_back(span(q.g, elems * gs, false, "g", i));
            v.push_back(span(q.m, (size_t)elems * 4, true, "m", i));
            if (q.master) v.push_back(span(q.master, (size_t)elems * 4, true, "master", i));
        }
        Span a, b;
        if (write_conflict(std::move(v), &a, &b)) {
            delete h;
            return conflict_fail("muon_create", a, b);
        }
        const auto table = [&](size_t bytes) {
            const size_t at = blob.size();
            blob.resize((at + bytes + 255) & ~(size_t)255);
            return at;
        };
        const auto put32 = [&](const std::vector<int32_t>& t) {
            const size_t at = table(t.size() * 4 + 4);
            if (!t.empty()) std::memcpy(blob.data() + at, t.data(), t.size() * 4);
            return at;
        };
        const auto scratch = [&](size_t bytes) {
            const size_t at = work;
            work = (at + bytes + 255) & ~(size_t)255;
            return at;
        };
        err_at = table(4);
        // tensors by their small side
        for (int k = 0; k < 3; ++k) {
            const int nb = 1 << k;
            int64_t items = 0, mats = 0;
            for (int i = 0; i < n; ++i)
                if (nbs[i] == nb) items += descs[i].count * ((descs[i].d + muon_chunk(nb, false) - 1) / muon_chunk(nb, false));
            const int chunk = muon_chunk(nb, items < 256);
            items = 0;
            std::vector<int32_t> item_desc, mat_desc;
            for (int i = 0; i < n; ++i) {
                MuDesc& d = descs[i];
                if (nbs[i] != nb || d.count == 0) continue;
                d.chunks = (int32_t)((d.d + chunk - 1) / chunk);
                d.item0 = items;
                d.mat0 = mats;
                items += d.count * d.chunks;
                mats += d.count;
                if (!grid_fits(items, 256) || !grid_fits(mats, 640)) {
                    delete h;
                    return fail(DLM_ESHAPE, "muon_create: the sizes need a launch grid of more than 2^32 - 1 work-items");
                }
                item_desc.insert(item_desc.end(), (size_t)(d.count * d.chunks), i);
                mat_desc.insert(mat_desc.end(), (size_t)d.count, i);
            }
            if (!mats) continue;
            h->small[k].items = items;
            h->small[k].chunk = chunk;
            h->small[k].mats = mats;
            Slot& s = slots[k];
            s.items = put32(item_desc);
            s.mats = put32(mat_desc);
            s.part = scratch((size_t)items * muon_part(nb) * 8);
            s.pm = scratch((size_t)mats * nb * nb * 256 * 8);
            s.bad = scratch((size_t)mats * 4);
        }
        std::vector<MuBig> bigs;
        std::vector<int32_t> ti, tp, ts, tsp, tm, tma, to, toa;
        int64_t off = 0;
        for (int i = 0; i < n; ++i) {
            MuDesc& d = descs[i];
            if (nbs[i] || d.count == 0) continue;
            ti.push_back(i);
            d.chunks = (int32_t)((d.d + kMuonBigChunk - 1) / kMuonBigChunk);
            if (ti.size() > 65535) {
                delete h;
                return fail(DLM_ESHAPE, "muon_create: more than 65535 tensors of a smaller side above %d", kMuonTileSide);
            }
            const int nb = (d.n + 63) / 64 * 4, groups = nb / 4, pairs = groups * (groups + 1) / 2;
            if (!grid_fits((int64_t)tp.size() + d.count * d.chunks * pairs, 256) ||
                !grid_fits((int64_t)to.size() + d.count * ((d.d + 63) / 64) * groups, 256) ||
                !grid_fits((int64_t)tm.size() + (int64_t)bigs.size() + d.count * (nb * nb + 1), 256) ||
                !grid_fits(((int64_t)ts.size() + d.count * pairs) * 16, 256)) {
                delete h;
                return fail(DLM_ESHAPE, "muon_create: the sizes need a launch grid of more than 2^32 - 1 work-items");
            }
            h->big_elems = std::max(h->big_elems, d.count * d.n * d.d);
            for (int64_t m = 0; m < d.count; ++m) {
                const int32_t at = (int32_t)bigs.size();
                bigs.push_back(MuBig{i, nb, m, (int64_t)tp.size(), off});
                off += (int64_t)nb * nb * 256;
                tp.insert(tp.end(), (size_t)d.chunks * pairs, at);
                for (int p = 0; p < pairs; ++p) {
                    ts.push_back(at);
                    tsp.push_back(p);
                }
                for (int blk = 0; blk < nb * nb; ++blk) {
                    tm.push_back(at);
                    tma.push_back(blk);
                }
                for (int o = 0; o < (d.d + 63) / 64 * groups; ++o) {
                    to.push_back(at);
                    toa.push_back(o);
                }
            }
        }
        if (!bigs.empty()) {
            MuonArgs& g = h->big;
            g.n_big = (int64_t)bigs.size();
            g.only = bigs[0];
            g.items = (int64_t)ti.size();
            g.n_pair = (int64_t)tp.size();
            g.n_sum = (int64_t)ts.size();
            g.n_mul = (int64_t)tm.size();
            g.n_out = (int64_t)to.size();
            g.sq = off;
            big_at = table(bigs.size() * sizeof(MuBig));
            std::memcpy(blob.data() + big_at, bigs.data(), bigs.size() * sizeof(MuBig));
            big_items = put32(ti);
            big_pair = put32(tp);
            big_sum = put32(ts);
            big_sump = put32(tsp);
            big_mul = put32(tm);
            big_mula = put32(tma);
            big_out = put32(to);
            big_outa = put32(toa);
            big_part = scratch((size_t)g.n_pair * kMuonBigPart * 8);
            big_sq = scratch((size_t)off * 6 * 8);
            big_meta = scratch((size_t)g.n_big * 16);
            big_bad = scratch((size_t)g.n_big * 4);
            for (int i : ti) u_at[i] = scratch((size_t)(descs[i].count * descs[i].n * descs[i].d) * 4);
        }
        descs_at = table(sizeof(MuDesc) * n);
        hipError_t e = hipSuccess;
        if (work) e = hipMalloc(&h->d_work, work);
        if (e == hipSuccess) e = hipMalloc(&h->d_tables, blob.size());
        for (int i = 0; i < n; ++i)
            if (!nbs[i] && descs[i].count) descs[i].u = (float*)((char*)h->d_work + u_at[i]);
        std::memcpy(blob.data() + descs_at, descs.data(), sizeof(MuDesc) * n);
        if (e == hipSuccess) e = hipMemcpy(h->d_tables, blob.data(), blob.size(), hipMemcpyHostToDevice);
        if (e == hipSuccess) e = prepare_muon();
        if (e != hipSuccess) {
            if (h->d_work) (void)hipFree(h->d_work);
            if (h->d_tables) (void)hipFree(h->d_tables);
            delete h;
            return hip_fail(e, "muon_create");
        }
    } catch (const std::bad_alloc&) {
        if (h) {
            if (h->d_work) (void)hipFree(h->d_work);
            if (h->d_tables) (void)hipFree(h->d_tables);
            delete h;
        }
        return fail(DLM_ENOMEM, "muon_create: host allocation failed");
    }
    const auto t32 = [&](size_t at) { return (int32_t*)((char*)h->d_tables + at); };
    const auto w = [&](size_t at) { return (char*)h->d_work + at; };
    h->p_dtype = p_dtype;
    h->g_dtype = g_dtype;
    h->d_err = t32(err_at);
    for (int k = 0; k < 3; ++k) {
        MuonArgs& a = h->small[k];
        if (!a.items) continue;
        a.descs = (const MuDesc*)t32(descs_at);
        a.item_desc = t32(slots[k].items);
        a.mat_desc = t32(slots[k].mats);
        a.part = (double*)w(slots[k].part);
        a.pm = (double*)w(slots[k].pm);
        a.bad = (int32_t*)w(slots[k].bad);
        a.err = h->d_err;
    }
    if (h->big.n_big) {
        MuonArgs& a = h->big;
        a.descs = (const MuDesc*)t32(descs_at);
        a.big = (const MuBig*)t32(big_at);
        a.item_desc = t32(big_items);
        a.pair_big = t32(big_pair);
        a.sum_big = t32(big_sum);
        a.sum_pair = t32(big_sump);
        a.mul_big = t32(big_mul);
        a.mul_at = t32(big_mula);
        a.out_big = t32(big_out);
        a.out_at = t32(big_outa);
        a.part = (double*)w(big_part);
        a.square = (double*)w(big_sq);
        a.meta = (double*)w(big_meta);
        a.bad = (int32_t*)w(big_bad);
        a.err = h->d_err;
    }
    *out = h;
    return ok();
}

int dlm_muon_destroy(dlm_muon* h) {
    if (!h) return fail(DLM_EINVAL, "muon_destroy: null handle");
    const hipError_t e = hipDeviceSynchronize();
    if (h->d_work) (void)hipFree(h->d_work);
    (void)hipFree(h->d_tables);
    delete h;
    if (e != hipSuccess) return hip_fail(e, "muon_destroy");
    return ok();
}

int dlm_muon_step(dlm_muon* h, const dlm_muon_cfg* c, const float* lr_scale, const float* grad_scale, void* stream) {
    if (!h || !c) return fail(DLM_EINVAL, "muon_step: null argument");
    if (!std::isfinite(c->lr)) return fail(DLM_EINVAL, "muon_step: lr is not finite");
    if (!(c->momentum >= 0.0 && c->momentum < 1.0)) return fail(DLM_EINVAL, "muon_step: momentum=%g not in [0, 1)", c->momentum);
    if (!(c->eps > 0.f) || !std::isfinite(c->eps)) return fail(DLM_EINVAL, "muon_step: eps=%g is not positive", c->eps);
    if (c->steps < 1 || c->steps > DLM_MAX_MUON_STEPS)
        return fail(DLM_EINVAL, "muon_step: steps=%d not in [1, %d]", c->steps, DLM_MAX_MUON_STEPS);
    for (int k = 0; k < c->steps; ++k)
        for (int j = 0; j < 3; ++j)
            if (!std::isfinite(c->coefs[k][j])) return fail(DLM_EINVAL, "muon_step: coefficient %d of step %d is not finite", j, k);
    if ((uintptr_t)lr_scale % 4 || (uintptr_t)grad_scale % 4) return fail(DLM_EALIGN, "muon_step: a pointer is not a multiple of 4");
    const auto set = [&](MuonArgs& a) {
        a.beta = c->momentum;
        a.lr = c->lr;
        a.eps = c->eps;
        a.nesterov = c->nesterov ? 1 : 0;
        a.steps = c->steps;
        std::memcpy(a.coefs, c->coefs, sizeof a.coefs);
        a.lr_scale = lr_scale;
        a.grad_scale = grad_scale;
    };
    MuonArgs small[3];
    for (int k = 0; k < 3; ++k) {
        small[k] = h->small[k];
        set(small[k]);
    }
    const hipError_t e = launch_muon(small, h->p_dtype, h->g_dtype, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "muon_step launch");
    if (h->big.n_big) {
        MuonArgs a = h->big;
        set(a);
        const hipError_t e = launch_muon_big(a, h->big_elems, h->p_dtype, h->g_dtype, (hipStream_t)stream);
        if (e != hipSuccess) return hip_fail(e, "muon_step launch");
    }
    return ok();
}

int dlm_muon_status(dlm_muon* h, int32_t* code, void* stream) {
    if (!h || !code) return fail(DLM_EINVAL, "muon_status: null argument");
    int32_t err = 0;
    hipError_t e = hipStreamSynchronize((hipStream_t)stream);
    if (e == hipSuccess) e = hipMemcpy(&err, h->d_err, sizeof err, hipMemcpyDeviceToHost);
    if (e == hipSuccess && err) e = hipMemset(h->d_err, 0, sizeof err);
    if (e != hipSuccess) return hip_fail(e, "muon_status");
    *code = err ? DLM_EDEVICE : DLM_OK;
    return ok();
}

// -------------------------------------------------------------------- int8 ----

static int i8_pieces(int64_t d) { return (int)((d + 127) / 128 * 2); }

int dlm_i8_quantize(const void* x, int64_t T, int64_t d, int32_t dtype, int8_t* q, float* scale, void* stream) {
    if (T < 0 || T >= ((int64_t)1 << 31)) return fail(DLM_ESHAPE, "i8_quantize: T=%lld out of range", (long long)T);
    if (d < 1 || d > kMaxDim) return fail(DLM_ESHAPE, "i8_quantize: d=%lld out of range", (long long)d);
    if (!valid_dtype(dtype)) return fail(DLM_EDTYPE, "i8_quantize: unknown dtype %d", dtype);
    if (T == 0) return ok();
    if (!x || !q || !scale) return fail(DLM_EINVAL, "i8_quantize: null pointer");
    if ((uintptr_t)x % esize(dtype) || (uintptr_t)scale % 4)
        return fail(DLM_EALIGN, "i8_quantize: a pointer is not a multiple of its element's size");
    const Span v[] = {span(x, (size_t)T * d * esize(dtype), false, "x", 0), span(q, (size_t)T * d, true, "q", 0),
                      span(scale, (size_t)T * 4, true, "scale", 0)};
    Span a, b;
    if (pair_conflict(v, &a, &b)) return conflict_fail("i8_quantize", a, b);
    const hipError_t e = launch_i8_quantize(x, T, d, dtype, q, scale, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "i8_quantize launch");
    return ok();
}

// Copies a direction's tables to the device and fills in its arguments.
static hipError_t i8_upload(const std::vector<I8Seg>& segs, const std::vector<I8Rows>& rows, std::vector<I8Prod>& prods, I8Tables* t) {
    // the longest sums first: what is left at the end of a launch is short
    std::stable_sort(prods.begin(), prods.end(), [](const I8Prod& x, const I8Prod& y) { return x.pieces > y.pieces; });
    I8Args& a = t->args;
    a = I8Args{};
    a.n_rows = (int32_t)rows.size();
    a.n_prods = (int32_t)prods.size();
    for (I8Prod& p : prods) {
        for (int k = 0; k < 6; ++k) {
            p.tile[k] = a.tiles[k];
            a.tiles[k] += (int32_t)((p.d + kI8Cols[k] - 1) / kI8Cols[k]);
        }
    }
    for (const I8Rows& r : rows) {
        a.pieces += r.pieces;
        a.max_pieces = std::max(a.max_pieces, r.pieces);
    }
    const size_t b0 = (segs.size() * sizeof(I8Seg) + 255) & ~(size_t)255, b1 = b0 + ((rows.size() * sizeof(I8Rows) + 255) & ~(size_t)255);
    std::vector<char> blob(b1 + prods.size() * sizeof(I8Prod));
    std::memcpy(blob.data(), segs.data(), segs.size() * sizeof(I8Seg));
    std::memcpy(blob.data() + b0, rows.data(), rows.size() * sizeof(I8Rows));
    std::memcpy(blob.data() + b1, prods.data(), prods.size() * sizeof(I8Prod));
    hipError_t e = hipMalloc(&t->d, blob.size());
    if (e == hipSuccess) e = hipMemcpy(t->d, blob.data(), blob.size(), hipMemcpyHostToDevice);
    a.segs = (const I8Seg*)t->d;
    a.rows = (const I8Rows*)((char*)t->d + b0);
    a.prods = (const I8Prod*)((char*)t->d + b1);
    return e;
}

static size_t i8_workspace(const I8Args& a, int64_t T, size_t* scale_at) {
    const size_t t16 = (size_t)(T + 15) / 16, q = t16 * a.pieces * kI8Piece;
    if (scale_at) *scale_at = q;
    return (q + t16 * 16 * 4 * a.n_rows + 255) & ~(size_t)255;
}

int dlm_i8_group_create(const dlm_i8_problem* probs, int32_t n, int32_t dtype, dlm_i8_group** out) {
    if (!out) return fail(DLM_EINVAL, "i8_group_create: out is null");
    *out = nullptr;
    if (!probs || n < 1 || n > 65535) return fail(DLM_EINVAL, "i8_group_create: bad problem list (n=%d)", n);
    if (!valid_dtype(dtype)) return fail(DLM_EDTYPE, "i8_group_create: unknown dtype %d", dtype);
    const size_t es = esize(dtype);
    int64_t tiles = 0;
    for (int i = 0; i < n; ++i) {
        const dlm_i8_problem& q = probs[i];
        if (!q.x || !q.W || !q.w_scale || !q.y) return fail(DLM_EINVAL, "i8_group_create: problem %d: null pointer", i);
        if (q.d_in < 1 || q.d_in > kI8MaxK)
            return fail(DLM_ESHAPE, "i8_group_create: problem %d: d_in=%lld not in [1, %lld]", i, (long long)q.d_in, (long long)kI8MaxK);
        if (q.d_out < 1 || q.d_out > kMaxDim)
            return fail(DLM_ESHAPE, "i8_group_create: problem %d: d_out=%lld out of range", i, (long long)q.d_out);
        if ((uintptr_t)q.x % es || (uintptr_t)q.y % es || (uintptr_t)q.w_scale % 4)
            return fail(DLM_EALIGN, "i8_group_create: problem %d: a pointer is not a multiple of its element's size", i);
        tiles += (q.d_out + 15) / 16;
    }
    if (!grid_fits(tiles, 512))
        return fail(DLM_ESHAPE, "i8_group_create: the sizes need a launch grid of more than 2^32 - 1 work-items");
    dlm_i8_group* h = nullptr;
    hipError_t e = hipSuccess;
    try {
        h = new dlm_i8_group();
        h->probs.assign(probs, probs + n);
        h->dtype = dtype;
        size_t bytes = 0;
        for (const dlm_i8_problem& q : h->probs) {
            h->w_at.push_back(bytes);
            bytes += (size_t)(q.d_out + 15) / 16 * i8_pieces(q.d_in) * kI8Piece;
        }
        for (const dlm_i8_problem& q : h->probs) {
            h->s_at.push_back(bytes);
            bytes += (size_t)(q.d_out + 15) / 16 * 64;
        }
        std::vector<I8Seg> segs;
        std::vector<I8Rows> rows;
        std::vector<I8Prod> prods;
        int64_t q0 = 0;
        e = hipDeviceSynchronize();  // W may still be written, on any stream
        if (e == hipSuccess) e = hipMalloc((void**)&h->d_w, bytes);
        if (e == hipSuccess) e = hipMemset(h->d_w + h->s_at[0], 0, bytes - h->s_at[0]);  // the scales' padding
        for (int i = 0; i < n && e == hipSuccess; ++i) {
            const dlm_i8_problem& q = h->probs[i];
            const int pieces = i8_pieces(q.d_in);
            // problems that read one x share its codes
            int r = 0;
            while (r < (int)rows.size() && !(segs[r].x == q.x && segs[r].d == q.d_in)) ++r;
            if (r == (int)rows.size()) {
                segs.push_back(I8Seg{q.x, nullptr, q.d_in, 0, aligned16(q.x) && q.d_in % (16 / (int64_t)es) == 0});
                rows.push_back(I8Rows{r, r + 1, pieces, 0, q0, r});
                q0 += pieces;
            }
            I8Prod p{};
            p.w = (const int8_t*)h->d_w + h->w_at[i];
            p.w_scale = (const float*)(h->d_w + h->s_at[i]);
            p.out = q.y;
            p.d = q.d_out;
            p.pieces = pieces;
            p.vec = q.d_out % 4 == 0 && (uintptr_t)q.y % (4 * es) == 0;
            p.q0 = rows[r].q0;
            p.rows = r;
            prods.push_back(p);
            e = launch_i8_pack(q.W, q.d_out, q.d_in, pieces, (int8_t*)h->d_w + h->w_at[i], nullptr);
            if (e == hipSuccess) e = hipMemcpy(h->d_w + h->s_at[i], q.w_scale, (size_t)q.d_out * 4, hipMemcpyDeviceToDevice);
        }
        if (e == hipSuccess) e = i8_upload(segs, rows, prods, &h->fwd);
        if (e == hipSuccess) e = prepare_i8();
        if (e == hipSuccess) e = hipDeviceSynchronize();
    } catch (const std::bad_alloc&) {
        e = hipErrorOutOfMemory;
    }
    if (e != hipSuccess) {
        if (h) {
            if (h->d_w) (void)hipFree(h->d_w);
            if (h->fwd.d) (void)hipFree(h->fwd.d);
            delete h;
        }
        return hip_fail(e, "i8_group_create");
    }
    *out = h;
    return ok();
}

int dlm_i8_group_destroy(dlm_i8_group* h) {
    if (!h) return fail(DLM_EINVAL, "i8_group_destroy: null handle");
    const hipError_t e = hipDeviceSynchronize();
    for (void* p : {(void*)h->d_w, h->fwd.d, (void*)h->d_wt, h->bwd.d})
        if (p) (void)hipFree(p);
    delete h;
    if (e != hipSuccess) return hip_fail(e, "i8_group_destroy");
    return ok();
}

int dlm_i8_group_workspace_size(const dlm_i8_group* h, int64_t T, size_t* bytes) {
    if (!h || !bytes) return fail(DLM_EINVAL, "i8_group_workspace_size: null argument");
    if (T < 0 || T >= ((int64_t)1 << 31)) return fail(DLM_ESHAPE, "i8_group_workspace_size: T=%lld out of range", (long long)T);
    *bytes = i8_workspace(h->fwd.args, T, nullptr);
    return ok();
}

// Refuses a call whose written buffers overlap others: looked up when it has more rows than any before.
static int i8_overlap(const char* call, dlm_i8_group* h, bool back, int64_t T, const void* ws, size_t ws_bytes) {
    const size_t es = esize(h->dtype);
    const int n = (int)h->probs.size();
    const auto in = [&](int i) { return back ? span(h->dy[i], (size_t)T * h->probs[i].d_out * es, false, "dy", i)
                                             : span(h->probs[i].x, (size_t)T * h->probs[i].d_in * es, false, "x", i); };
    const auto out = [&](int i) { return back ? span(h->dx[i], (size_t)T * h->probs[i].d_in * es, true, "dx", i)
                                              : span(h->probs[i].y, (size_t)T * h->probs[i].d_out * es, true, "y", i); };
    const Span w = span(ws, ws_bytes, true, "workspace", 0);
    for (int i = 0; i < n; ++i) {
        if (back && !h->dx[i]) continue;
        for (const Span& s : {in(i), out(i)})
            if (s.hi > w.lo && w.hi > s.lo) return conflict_fail(call, w, s);
    }
    int64_t& checked = back ? h->checked_bwd : h->checked_fwd;
    if (T <= checked) return DLM_OK;
    try {
        std::vector<Span> v;
        std::set<const void*> shared;  // a dx that several problems share is one buffer
        for (int i = 0; i < n; ++i) {
            if (back && !h->dx[i]) continue;
            v.push_back(in(i));
            if (!back || shared.insert(h->dx[i]).second) v.push_back(out(i));
        }
        Span a, b;
        if (write_conflict(std::move(v), &a, &b)) return conflict_fail(call, a, b);
    } catch (const std::bad_alloc&) {
        return fail(DLM_ENOMEM, "%s: host allocation failed", call);
    }
    checked = T;
    return DLM_OK;
}

static int i8_launch(const char* call, dlm_i8_group* h, bool back, int64_t T, int32_t accumulate, void* workspace, size_t ws_bytes, void* stream) {
    if (T < 0 || T >= ((int64_t)1 << 31)) return fail(DLM_ESHAPE, "%s: T=%lld out of range", call, (long long)T);
    I8Args a = back ? h->bwd.args : h->fwd.args;
    if (T == 0 || a.n_prods == 0) return ok();
    size_t scale_at;
    const size_t need = i8_workspace(a, T, &scale_at);
    if (!workspace || ws_bytes < need)
        return fail(DLM_EWORKSPACE, "%s: workspace of %zu bytes, %zu needed", call, workspace ? ws_bytes : (size_t)0, need);
    if ((uintptr_t)workspace % 256) return fail(DLM_EALIGN, "%s: workspace is not 256-byte aligned", call);
    const int rc = i8_overlap(call, h, back, T, workspace, need);
    if (rc != DLM_OK) return rc;
    a.T = T;
    a.T16 = (T + 15) / 16;
    a.q = (int8_t*)workspace;
    a.scale = (float*)((char*)workspace + scale_at);
    a.accumulate = accumulate ? 1 : 0;
    a.plain = back ? 0 : 1;
    hipError_t e;
    if (i8_one_launch(a)) {
        e = launch_i8_token(a, h->dtype, (hipStream_t)stream);
        return e == hipSuccess ? ok() : hip_fail(e, call);
    }
    e = launch_i8_rows(a, h->dtype, (hipStream_t)stream);
    if (e == hipSuccess) e = launch_i8_products(a, h->dtype, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, call);
    return ok();
}

int dlm_i8_group_run(dlm_i8_group* h, int64_t T, void* workspace, size_t ws_bytes, void* stream) {
    if (!h) return fail(DLM_EINVAL, "i8_group_run: null handle");
    return i8_launch("i8_group_run", h, false, T, 0, workspace, ws_bytes, stream);
}

int dlm_i8_group_bind_grads(dlm_i8_group* h, const void* const* dy, void* const* dx) {
    if (!h || !dy || !dx) return fail(DLM_EINVAL, "i8_group_bind_grads: null argument");
    const int n = (int)h->probs.size();
    const size_t es = esize(h->dtype);
    for (int i = 0; i < n; ++i) {
        if (!dx[i]) continue;
        if (!dy[i]) return fail(DLM_EINVAL, "i8_group_bind_grads: problem %d: dx without dy", i);
        if ((uintptr_t)dy[i] % es || (uintptr_t)dx[i] % es)
            return fail(DLM_EALIGN, "i8_group_bind_grads: problem %d: a pointer is not a multiple of its element's size", i);
        for (int j = 0; j < i; ++j)
            if (dx[j] == dx[i] && h->probs[j].d_in != h->probs[i].d_in)
                return fail(DLM_EINVAL, "i8_group_bind_grads: problems %d and %d share a dx and differ in d_in", j, i);
    }
    I8Tables t;
    char* wt = nullptr;
    hipError_t e = hipDeviceSynchronize();
    std::vector<const void*> new_dy;
    std::vector<void*> new_dx;
    try {
        new_dy.assign(dy, dy + n);
        new_dx.assign(dx, dx + n);
        std::vector<I8Seg> segs;
        std::vector<I8Rows> rows;
        std::vector<I8Prod> prods;
        std::vector<size_t> at;
        std::vector<std::vector<int>> of;
        size_t bytes = 0;
        int64_t q0 = 0;
        for (int i = 0; i < n; ++i) {
            if (!dx[i]) continue;
            bool first = true;
            for (int j = 0; j < i; ++j) first = first && dx[j] != dx[i];
            if (!first) continue;
            const int64_t d_in = h->probs[i].d_in;
            const int seg0 = (int)segs.size();
            int k0 = 0;
            of.emplace_back();
            for (int j = i; j < n; ++j) {
                if (dx[j] != dx[i]) continue;
                const int64_t d = h->probs[j].d_out;
                if (((int64_t)k0 + (d + 63) / 64) * 64 > kI8MaxK)
                    return fail(DLM_ESHAPE, "i8_group_bind_grads: problem %d: more than %lld output channels share its dx", j,
                                (long long)kI8MaxK);
                segs.push_back(I8Seg{dy[j], (const float*)(h->d_w + h->s_at[j]), d, k0,
                                     aligned16(dy[j]) && d % (16 / (int64_t)es) == 0});
                k0 += (int)((d + 63) / 64);
                of.back().push_back(j);
            }
            const int pieces = (k0 + 1) / 2 * 2, r = (int)rows.size();
            rows.push_back(I8Rows{seg0, (int)segs.size(), pieces, 0, q0, r});
            I8Prod p{};
            p.out = dx[i];
            p.d = d_in;
            p.pieces = pieces;
            p.vec = d_in % 4 == 0 && (uintptr_t)dx[i] % (4 * es) == 0;
            p.q0 = q0;
            p.rows = r;
            prods.push_back(p);
            at.push_back(bytes);
            q0 += pieces;
            bytes += (size_t)(d_in + 15) / 16 * pieces * kI8Piece;
        }
        if (e == hipSuccess && bytes) e = hipMalloc((void**)&wt, bytes);
        if (e == hipSuccess && bytes) e = hipMemset(wt, 0, bytes);
        for (size_t r = 0; r < rows.size() && e == hipSuccess; ++r) {
            prods[r].w = (const int8_t*)wt + at[r];
            for (size_t s = 0; s < of[r].size() && e == hipSuccess; ++s) {
                const dlm_i8_problem& q = h->probs[of[r][s]];
                e = launch_i8_transpose((const int8_t*)h->d_w + h->w_at[of[r][s]], q.d_out, q.d_in, i8_pieces(q.d_in), (int8_t*)wt + at[r],
                                        rows[r].pieces, segs[rows[r].seg0 + s].k0, nullptr);
            }
        }
        if (e == hipSuccess) e = i8_upload(segs, rows, prods, &t);
        if (e == hipSuccess) e = hipDeviceSynchronize();
    } catch (const std::bad_alloc&) {
        e = hipErrorOutOfMemory;
    }
    if (e != hipSuccess) {
        if (wt) (void)hipFree(wt);
        if (t.d) (void)hipFree(t.d);
        return hip_fail(e, "i8_group_bind_grads");
    }
    if (h->d_wt) (void)hipFree(h->d_wt);
    if (h->bwd.d) (void)hipFree(h->bwd.d);
    h->d_wt = wt;
    h->bwd = t;
    h->dy.swap(new_dy);
    h->dx.swap(new_dx);
    h->bound = true;
    h->checked_bwd = 0;
    return ok();
}

int dlm_i8_group_backward_workspace_size(const dlm_i8_group* h, int64_t T, size_t* bytes) {
    if (!h || !bytes) return fail(DLM_EINVAL, "i8_group_backward_workspace_size: null argument");
    if (!h->bound) return fail(DLM_EINVAL, "i8_group_backward_workspace_size: no gradients are bound");
    if (T < 0 || T >= ((int64_t)1 << 31))
        return fail(DLM_ESHAPE, "i8_group_backward_workspace_size: T=%lld out of range", (long long)T);
    *bytes = i8_workspace(h->bwd.args, T, nullptr);
    return ok();
}

int dlm_i8_group_backward(dlm_i8_group* h, int64_t T, int32_t accumulate, void* workspace, size_t ws_bytes, void* stream) {
    if (!h) return fail(DLM_EINVAL, "i8_group_backward: null handle");
    if (!h->bound) return fail(DLM_EINVAL, "i8_group_backward: no gradients are bound");
    return i8_launch("i8_group_backward", h, true, T, accumulate, workspace, ws_bytes, stream);
}

}  // extern "C"
