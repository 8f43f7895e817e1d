// Host side of the C ABI declared in include/dlm.h: argument validation (no GPU
// call before it passes), device descriptor tables, launches and status words.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "dlm.h"
#include "adamw.hpp"
#include "api.hpp"
#include "internal.hpp"
#include "route.hpp"
#include "sgmm.hpp"

using namespace dlm;

// --------------------------------------------------------------- handles ----

struct dlm_layers {
    SwDesc* d_descs = nullptr;
    int32_t* d_err = nullptr;
    void* d_pack = nullptr;       // packed A images of every weight, then the zero image (wide tiles)
    void* d_zimg = nullptr;
    float* d_part = nullptr;      // partial products of the fused switch + product (bound vectors)
    float* d_vpart = nullptr;     // rank-vector partials of the unmerged product (bound vectors)
    int64_t n_ks = 0;             // their K slices over all weights
    bool bound = false;           // dlm_layers_bind_vectors has been called
    int64_t n_blocks = 0, n_bands = 0;  // product blocks (kGemvRows rows) and 256-row bands over all weights
    std::vector<SwDesc> h_descs;
    int32_t n = 0;
    int32_t E = 0, r = 0;
    float scale = 1.f;
    int32_t dtype = 0;
    SwTile tile{};
    int64_t n_tiles = 0, n_elems = 0, per_xcd = 0;
    std::vector<std::pair<uintptr_t, uintptr_t>> w_spans;  // every W, sorted, disjoint
};

// Whether [p, p + bytes) touches any weight the handle writes.
static bool hits_weights(const dlm_layers* h, const void* p, size_t bytes) {
    if (!p) return false;
    const uintptr_t lo = (uintptr_t)p, hi = lo + bytes;
    auto it = std::upper_bound(h->w_spans.begin(), h->w_spans.end(), std::make_pair(lo, UINTPTR_MAX));
    if (it != h->w_spans.begin() && std::prev(it)->second > lo) return true;
    return it != h->w_spans.end() && it->first < hi;
}

static int check_sets(const dlm_layers* h, const int32_t* old_idx, const float* old_g, const int32_t* new_idx,
                      const float* new_g, const char* call) {
    if ((old_idx && !old_g) || (new_idx && !new_g)) return fail(DLM_EINVAL, "%s: a set has indices but no gates", call);
    if (hits_weights(h, old_idx, 8) || hits_weights(h, old_g, 8) || hits_weights(h, new_idx, 8) ||
        hits_weights(h, new_g, 8))
        return fail(DLM_EINVAL, "%s: a set lies inside a weight the switch writes", call);
    return DLM_OK;
}

struct dlm_sgmm_group {
    SgDesc* d_descs = nullptr;          // device block: descriptors, then their per-unit copies
    const SgDesc* d_ks_desc = nullptr;
    const SgDesc* d_cb_desc = nullptr;
    std::vector<SgDesc> h_descs;
    int32_t n = 0;
    int32_t E = 0, r = 0;
    float scale = 1.f;
    int32_t dtype = 0;
    int64_t total_cb = 0, total_ks = 0, d_out_max = 0, d_in_max = 0;
    int32_t w_max = 0;  // largest K slices + column groups of one problem
    // packed copies of the distinct A banks (bf16 groups), owned by the handle
    struct Pack {
        const void* A;
        void* Ap;
        int64_t d_in;
    };
    std::vector<Pack> packs;
    int64_t checked_T = 0;  // largest row count whose buffers were checked for overlaps
    // gradients (dlm_sgmm_group_bind_grads)
    struct Grads {
        char* d_tab = nullptr;   // device block: every table below
        char* d_pack = nullptr;  // the banks' transposes
        struct Wave {            // expands that run in one launch: no dx twice
            const SgDesc* descs;
            const SgDesc* cb_desc;
            int32_t n;
            int64_t total_cb, d_max;
            int32_t w_max;
        };
        // the tables that go by the shrink's K slice width: one set for
        // kSgmmKSlice, one for kSgmmKSliceFew
        struct Slices {
            int32_t width = 0;
            int64_t total_ks = 0;
            const SgDesc* descs = nullptr;    // 2n shrink problems: (x, A), then (dy, B^T)
            const SgDesc* ks_desc = nullptr;
            std::vector<Wave> waves;
            const SgGrad* probs = nullptr;
        } slices[2];
        const SgOuter* outers = nullptr;
        const int32_t* unit_outer = nullptr;
        int32_t n_units = 0;
        int64_t pk_total = 0;
        std::vector<const void*> dy;
        std::vector<void*> dx;
        std::vector<float*> dA, dB;
        int64_t checked_T = -1;
        bool bound = false;
        // fp32 has one slice per side, whatever its width
        const Slices& for_rows(int64_t T) const { return slices[slices[0].total_ks * ((T + 31) / 32) < kSgmmFewItems ? 1 : 0]; }
    } grads;
};

struct dlm_adamw {
    AdDesc* d_descs = nullptr;  // device block: descriptors, the tensor of every chunk, every chunk's step count, the error word
    const int32_t* d_chunk_tensor = nullptr;
    int32_t* d_steps = nullptr;
    int32_t* d_err = nullptr;
    int64_t step0 = 0;
    int64_t n_chunks = 0;
    int32_t p_dtype = 0, g_dtype = 0, bits = 32;
    uint32_t seed = 0;
};

// Scratch memory of dlm_sgmm_noalloc: one file-scope device array, which each
// device that loads the library holds until the process ends.  In host code
// its name stands for a host-side shadow, not for device memory: the device
// address is looked up once per device (hipGetSymbolAddress, with that device
// current) and only that address is ever handed to a kernel.
constexpr size_t kNoAllocScratchBytes = DLM_SGMM_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) char scratch[kNoAllocScratchBytes];

extern "C" {

const char* dlm_last_error(void) { return g_err; }

const char* dlm_version(void) { return "dlm 0.1.0 (gfx950)"; }

// ---------------------------------------------------------------- router ----

int dlm_pregate(const void* x, const void* Wr, int64_t T, int64_t d, int32_t E, int32_t dtype,
                int32_t* idx, float* g, void* stream) {
    if (T < 0 || T >= ((int64_t)1 << 31)) return fail(DLM_ESHAPE, "pregate: T=%lld out of range", (long long)T);
    if (d < 1 || d > kMaxDim) return fail(DLM_ESHAPE, "pregate: d=%lld out of range", (long long)d);
    if (E < 2 || E > DLM_MAX_EXPERTS) return fail(DLM_ESHAPE, "pregate: E=%d not in [2, %d]", E, DLM_MAX_EXPERTS);
    if (!valid_dtype(dtype)) return fail(DLM_EDTYPE, "pregate: unknown dtype %d", dtype);
    if (T == 0) return ok();
    if (!x || !Wr || !idx || !g) return fail(DLM_EINVAL, "pregate: null pointer");
    hipError_t e = launch_pregate(x, Wr, T, d, E, dtype, idx, g, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "pregate launch");
    return ok();
}

int dlm_pregate_centroid(const void* x, const void* C, int64_t T, int64_t d, int32_t E, int32_t J, int32_t dtype,
                         int32_t* idx, float* g, void* stream) {
    if (T < 0 || T >= ((int64_t)1 << 31)) return fail(DLM_ESHAPE, "pregate_centroid: T=%lld out of range", (long long)T);
    if (d < 1 || d > kMaxDim) return fail(DLM_ESHAPE, "pregate_centroid: d=%lld out of range", (long long)d);
    if (E < 1 || E > DLM_MAX_EXPERTS)
        return fail(DLM_ESHAPE, "pregate_centroid: E=%d not in [1, %d]", E, DLM_MAX_EXPERTS);
    if (J < 1 || J > DLM_MAX_CENTROIDS)
        return fail(DLM_ESHAPE, "pregate_centroid: J=%d not in [1, %d]", J, DLM_MAX_CENTROIDS);
    if (!valid_dtype(dtype)) return fail(DLM_EDTYPE, "pregate_centroid: unknown dtype %d", dtype);
    if (T == 0) return ok();
    if (!x || !C || !idx || !g) return fail(DLM_EINVAL, "pregate_centroid: null pointer");
    hipError_t e = launch_pregate_centroid(x, C, T, d, E, J, dtype, idx, g, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "pregate_centroid launch");
    return ok();
}

// Checks and arguments shared by dlm_route and dlm_route_backward.
static int route_args(const char* call, const void* logits, int64_t ld, int64_t T, int32_t E, int32_t dtype,
                      const dlm_route_cfg* c, RouteArgs* a) {
    static_assert(kRouteMaxExperts == DLM_MAX_ROUTE_EXPERTS && kRouteMaxK == DLM_MAX_ROUTE_K, "route limits");
    static_assert(kRouteSoftmax == DLM_SOFTMAX && kRouteSigmoid == DLM_SIGMOID, "score codes");
    if (!c) return fail(DLM_EINVAL, "%s: cfg is null", call);
    if (T < 0 || T >= ((int64_t)1 << 31)) return fail(DLM_ESHAPE, "%s: T=%lld out of range", call, (long long)T);
    if (E < 1 || E > DLM_MAX_ROUTE_EXPERTS)
        return fail(DLM_ESHAPE, "%s: E=%d not in [1, %d]", call, E, DLM_MAX_ROUTE_EXPERTS);
    if (!valid_dtype(dtype)) return fail(DLM_EDTYPE, "%s: unknown dtype %d", call, dtype);
    if (ld < E || ld > kMaxDim) return fail(DLM_ESHAPE, "%s: row pitch %lld of rows of %d", call, (long long)ld, E);
    if (c->score != DLM_SOFTMAX && c->score != DLM_SIGMOID) return fail(DLM_EINVAL, "%s: unknown score %d", call, c->score);
    if (!std::isfinite(c->scale)) return fail(DLM_EINVAL, "%s: scale is not finite", call);
    if (c->n_groups < 1 || c->n_groups > DLM_MAX_ROUTE_GROUPS || E % c->n_groups != 0)
        return fail(DLM_ESHAPE, "%s: %d groups of %d experts (at most %d groups, of equal size)", call, c->n_groups, E,
                    DLM_MAX_ROUTE_GROUPS);
    if (c->keep_groups < 1 || c->keep_groups > c->n_groups)
        return fail(DLM_ESHAPE, "%s: keep_groups=%d not in [1, %d]", call, c->keep_groups, c->n_groups);
    if (c->group_top != 1 && c->group_top != 2) return fail(DLM_EINVAL, "%s: group_top=%d is not 1 or 2", call, c->group_top);
    const int gs = E / c->n_groups;
    if (c->k < 1 || c->k > DLM_MAX_ROUTE_K || c->k > c->keep_groups * gs)
        return fail(DLM_ESHAPE, "%s: k=%d of %d experts in the kept groups (at most %d)", call, c->k, c->keep_groups * gs,
                    DLM_MAX_ROUTE_K);
    *a = RouteArgs{};
    a->logits = logits;
    a->ld = ld;
    a->T = T;
    a->E = E;
    a->k = c->k;
    a->score = c->score;
    a->renorm = c->renorm ? 1 : 0;
    a->scale = c->scale;
    a->n_groups = c->n_groups;
    a->group_size = gs;
    a->keep_groups = c->keep_groups;
    a->group_top = c->group_top;
    a->gs_magic = (uint32_t)((1u << 20) / gs + 1);
    const int64_t w = 16 / (int64_t)esize(dtype);
    a->vec = aligned16(logits) && ld % w == 0 && E % w == 0;
    return DLM_OK;
}

int dlm_route(const void* logits, int64_t ld, const float* bias, int64_t T, int32_t E, int32_t dtype,
              const dlm_route_cfg* cfg, int32_t* idx, float* g, int32_t* counts, void* stream) {
    RouteArgs a;
    const int rc = route_args("route", logits, ld, T, E, dtype, cfg, &a);
    if (rc != DLM_OK) return rc;
    if (T == 0) return ok();
    if (!logits || !idx || !g) return fail(DLM_EINVAL, "route: null pointer");
    const Span v[] = {span(logits, rows_bytes(T, ld, E, esize(dtype)), false, "logits", 0),
                      span(idx, (size_t)T * a.k * 4, true, "idx", 0), span(g, (size_t)T * a.k * 4, true, "g", 0),
                      span(bias, bias ? (size_t)E * 4 : 0, false, "bias", 0),
                      span(counts, counts ? (size_t)E * 4 : 0, true, "counts", 0)};
    Span p, q;
    if (pair_conflict(v, &p, &q)) return conflict_fail("route", p, q);
    a.bias = bias;
    a.vec_bias = bias && aligned16(bias) && E % 4 == 0;
    a.scores_order = bias || (a.n_groups > 1 && a.group_top == 2) ? 1 : 0;
    a.need_scores = a.scores_order || (a.score == kRouteSoftmax && !a.renorm) ? 1 : 0;
    a.idx = idx;
    a.g = g;
    a.counts = counts;
    const hipError_t e = launch_route(a, dtype, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "route launch");
    return ok();
}

int dlm_route_backward(const void* logits, int64_t ld, const int32_t* idx, const float* dg, int64_t T, int32_t E,
                       int32_t dtype, const dlm_route_cfg* cfg, void* dlogits, int64_t ldd, void* stream) {
    RouteArgs a;
    const int rc = route_args("route_backward", logits, ld, T, E, dtype, cfg, &a);
    if (rc != DLM_OK) return rc;
    if (ldd < E || ldd > kMaxDim)
        return fail(DLM_ESHAPE, "route_backward: row pitch %lld of dlogits rows of %d", (long long)ldd, E);
    if (T == 0) return ok();
    if (!logits || !idx || !dg || !dlogits) return fail(DLM_EINVAL, "route_backward: null pointer");
    const size_t es = esize(dtype);
    Span p, q;
    const Span v[] = {span(logits, rows_bytes(T, ld, E, es), false, "logits", 0),
                      span(dlogits, rows_bytes(T, ldd, E, es), true, "dlogits", 0),
                      span(idx, (size_t)T * a.k * 4, false, "idx", 0), span(dg, (size_t)T * a.k * 4, false, "dg", 0)};
    if (pair_conflict(v, &p, &q)) return conflict_fail("route_backward", p, q);
    a.in_idx = idx;
    a.dg = dg;
    a.dlogits = dlogits;
    a.ldd = ldd;
    const int64_t w = 16 / (int64_t)es;
    a.vec_out = aligned16(dlogits) && ldd % w == 0 && E % w == 0;
    const hipError_t e = launch_route_grad(a, dtype, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "route_backward launch");
    return ok();
}

// ---------------------------------------------------------------- switch ----

int dlm_layers_create(const dlm_proj* projs, int32_t n, int32_t E, int32_t r, float scale,
                      int32_t dtype, dlm_layers** out) {
    if (!out) return fail(DLM_EINVAL, "layers_create: out is null");
    *out = nullptr;
    if (!projs) return fail(DLM_EINVAL, "layers_create: projs is null");
    if (n < 1) return fail(DLM_EINVAL, "layers_create: n=%d", n);
    if (E < 1 || E > DLM_MAX_EXPERTS) return fail(DLM_ESHAPE, "layers_create: E=%d not in [1, %d]", E, DLM_MAX_EXPERTS);
    if (r < 1 || r > DLM_MAX_RANK) return fail(DLM_ESHAPE, "layers_create: r=%d not in [1, %d]", r, DLM_MAX_RANK);
    if (!valid_dtype(dtype)) return fail(DLM_EDTYPE, "layers_create: unknown dtype %d", dtype);
    if (!std::isfinite(scale)) return fail(DLM_EINVAL, "layers_create: scale is not finite");
    const SwTile tile = switch_tile_for_rank(r);
    std::vector<SwDesc> h(n);
    int64_t tiles = 0, elems = 0, blocks = 0, bands = 0;
    for (int i = 0; i < n; ++i) {
        const dlm_proj& p = projs[i];
        if (!p.W || !p.A || !p.B) return fail(DLM_EINVAL, "layers_create: proj %d has a null pointer", i);
        if (p.d_out < 1 || p.d_in < 1 || p.d_out > kMaxDim || p.d_in > kMaxDim)
            return fail(DLM_ESHAPE, "layers_create: proj %d shape %lldx%lld out of range", i,
                        (long long)p.d_out, (long long)p.d_in);
        if (dtype == DLM_BF16) {
            if (!aligned16(p.W) || !aligned16(p.A) || !aligned16(p.B))
                return fail(DLM_EALIGN, "layers_create: proj %d pointer not 16-byte aligned", i);
            if (p.d_in % 8 != 0)
                return fail(DLM_EALIGN, "layers_create: proj %d d_in=%lld not a multiple of 8", i, (long long)p.d_in);
        }
        SwDesc& d = h[i];
        d.W = p.W;
        d.A = p.A;
        d.B = p.B;
        d.d_out = (int32_t)p.d_out;
        d.d_in = (int32_t)p.d_in;
        d.n_rt = (int32_t)((p.d_out + tile.rt - 1) / tile.rt);
        d.n_ct = (int32_t)((p.d_in + tile.ct - 1) / tile.ct);
        d.tile0 = tiles;
        d.elem0 = elems;
        d.Ap = nullptr;
        d.xv = nullptr;
        d.yv = nullptr;
        d.part = nullptr;
        d.rb0 = blocks;
        d.rt0 = bands;
        blocks += (p.d_out + kGemvRows - 1) / kGemvRows;
        bands += (p.d_out + 255) / 256;
        tiles += (int64_t)d.n_rt * d.n_ct;
        elems += p.d_out * p.d_in;
    }
    {
        std::vector<Span> v;
        const size_t es = esize(dtype);
        for (int i = 0; i < n; ++i) {
            const dlm_proj& p = projs[i];
            v.push_back(span(p.W, (size_t)p.d_out * p.d_in * es, true, "weight W", i));
            v.push_back(span(p.A, (size_t)E * r * p.d_in * es, false, "bank A", i));
            v.push_back(span(p.B, (size_t)E * p.d_out * r * es, false, "bank B", i));
        }
        Span a, b;
        if (write_conflict(std::move(v), &a, &b)) return conflict_fail("layers_create", a, b);
    }
    dlm_layers* hd = new (std::nothrow) dlm_layers();
    if (!hd) return fail(DLM_ENOMEM, "layers_create: host allocation failed");
    hd->n = n;
    hd->E = E;
    hd->r = r;
    hd->scale = scale;
    hd->dtype = dtype;
    hd->tile = tile;
    hd->n_tiles = tiles;
    hd->n_elems = elems;
    hd->per_xcd = (tiles + 7) / 8;
    hd->n_blocks = blocks;
    hd->n_bands = bands;
    hipError_t e = dtype == DLM_BF16 ? prepare_switch_bf16(tile) : hipSuccess;
    if (e == hipSuccess && dtype == DLM_BF16 && switch_packs_a(tile)) {
        // ranks 17..64: packed A images for the copy-staged tiles, one block
        size_t elems_total = 0;
        std::vector<size_t> off(n);
        for (int i = 0; i < n; ++i) {
            off[i] = elems_total;
            elems_total += switch_packed_a_elems(h[i].d_in, E, tile);
        }
        const size_t zero_off = elems_total;
        elems_total += switch_zero_image_elems(tile);
        e = hipMalloc(&hd->d_pack, elems_total * 2);
        if (e == hipSuccess) {
            uint16_t* base = (uint16_t*)hd->d_pack;
            hd->d_zimg = base + zero_off;
            e = hipMemset(hd->d_zimg, 0, switch_zero_image_elems(tile) * 2);
            for (int i = 0; i < n && e == hipSuccess; ++i) {
                h[i].Ap = base + off[i];
                e = launch_switch_pack_a(h[i].A, base + off[i], h[i].d_in, E, r, tile, nullptr);
            }
            if (e == hipSuccess) e = hipDeviceSynchronize();
        }
    }
    if (e == hipSuccess) e = hipMalloc((void**)&hd->d_descs, sizeof(SwDesc) * n);
    if (e == hipSuccess) e = hipMalloc((void**)&hd->d_err, 256);
    if (e == hipSuccess) e = hipMemcpy(hd->d_descs, h.data(), sizeof(SwDesc) * n, hipMemcpyHostToDevice);
    if (e == hipSuccess) e = hipMemset(hd->d_err, 0, 256);
    if (e != hipSuccess) {
        if (hd->d_descs) (void)hipFree(hd->d_descs);
        if (hd->d_err) (void)hipFree(hd->d_err);
        if (hd->d_pack) (void)hipFree(hd->d_pack);
        delete hd;
        return hip_fail(e, "layers_create");
    }
    for (const SwDesc& q : h)
        hd->w_spans.emplace_back((uintptr_t)q.W, (uintptr_t)q.W + (size_t)q.d_out * q.d_in * esize(dtype));
    std::sort(hd->w_spans.begin(), hd->w_spans.end());
    hd->h_descs = std::move(h);
    *out = hd;
    return ok();
}

int dlm_layers_repack(dlm_layers* h, void* stream) {
    if (!h) return fail(DLM_EINVAL, "layers_repack: null handle");
    if (!h->d_pack) return ok();
    for (const SwDesc& d : h->h_descs) {
        hipError_t e = launch_switch_pack_a(d.A, (void*)d.Ap, d.d_in, h->E, h->r, h->tile, (hipStream_t)stream);
        if (e != hipSuccess) return hip_fail(e, "layers_repack launch");
    }
    return ok();
}

int dlm_layers_destroy(dlm_layers* h) {
    if (!h) return fail(DLM_EINVAL, "layers_destroy: null handle");
    hipError_t e = hipDeviceSynchronize();
    if (h->d_descs) (void)hipFree(h->d_descs);
    if (h->d_err) (void)hipFree(h->d_err);
    if (h->d_pack) (void)hipFree(h->d_pack);
    if (h->d_part) (void)hipFree(h->d_part);
    if (h->d_vpart) (void)hipFree(h->d_vpart);
    delete h;
    if (e != hipSuccess) return hip_fail(e, "layers_destroy");
    return ok();
}

static SwitchArgs switch_args(const dlm_layers* h, const int32_t* old_idx, const float* old_g,
                              const int32_t* new_idx, const float* new_g) {
    SwitchArgs a;
    a.descs = h->d_descs;
    a.n_desc = h->n;
    a.E = h->E;
    a.r = h->r;
    a.scale = h->scale;
    a.old_idx = old_idx;
    a.old_g = old_g;
    a.new_idx = new_idx;
    a.new_g = new_g;
    a.err = h->d_err;
    a.zimg = h->d_zimg;
    a.vpart = h->d_vpart;
    if (h->dtype == DLM_BF16) {
        a.n_units = h->n_tiles;
        a.per_xcd = h->per_xcd;
    } else {
        a.n_units = h->n_elems;
        a.per_xcd = 0;
    }
    return a;
}

int dlm_switch(dlm_layers* h, const int32_t* old_idx, const float* old_g, const int32_t* new_idx,
               const float* new_g, void* stream) {
    if (!h) return fail(DLM_EINVAL, "switch: null handle");
    const int rc = check_sets(h, old_idx, old_g, new_idx, new_g, "switch");
    if (rc != DLM_OK) return rc;
    const SwitchArgs a = switch_args(h, old_idx, old_g, new_idx, new_g);
    const hipError_t e = h->dtype == DLM_BF16 ? launch_switch_bf16(a, h->tile, (hipStream_t)stream)
                                              : launch_switch_generic(a, h->dtype, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "switch launch");
    return ok();
}

int dlm_switch_launches(const dlm_layers* h) { return h ? 1 : 0; }

// ------------------------------------------------- merged-weight products ----

int dlm_layers_bind_vectors(dlm_layers* h, const void* const* x, float* const* y) {
    if (!h || !x || !y) return fail(DLM_EINVAL, "bind_vectors: null argument");
    std::vector<SwDesc> d = h->h_descs;
    for (int i = 0; i < h->n; ++i) {
        if (!x[i] || !y[i]) return fail(DLM_EINVAL, "bind_vectors: vector %d is null", i);
        if (h->dtype == DLM_BF16 && !aligned16(x[i]))
            return fail(DLM_EALIGN, "bind_vectors: x %d not 16-byte aligned", i);
        if (((uintptr_t)y[i] & 3u) != 0) return fail(DLM_EALIGN, "bind_vectors: y %d not 4-byte aligned", i);
        d[i].xv = x[i];
        d[i].yv = y[i];
    }
    {
        // the product reads W, x (and the switch + product also writes W and
        // reads A, B); y is written
        std::vector<Span> v;
        const size_t es = esize(h->dtype);
        for (int i = 0; i < h->n; ++i) {
            v.push_back(span(d[i].W, (size_t)d[i].d_out * d[i].d_in * es, true, "weight W", i));
            v.push_back(span(d[i].A, (size_t)h->E * h->r * d[i].d_in * es, false, "bank A", i));
            v.push_back(span(d[i].B, (size_t)h->E * d[i].d_out * h->r * es, false, "bank B", i));
            v.push_back(span(x[i], (size_t)d[i].d_in * es, false, "vector x", i));
            v.push_back(span(y[i], (size_t)d[i].d_out * 4, true, "vector y", i));
        }
        Span a, b;
        if (write_conflict(std::move(v), &a, &b)) return conflict_fail("bind_vectors", a, b);
    }
    float* part = nullptr;
    float* vpart = nullptr;
    // the unmerged product's K slices: per weight a prefix and a count
    int64_t n_ks = 0;
    for (int i = 0; i < h->n; ++i) {
        d[i].ks0 = n_ks;
        d[i].n_ks = (int32_t)((d[i].d_in + kLoraKSlice - 1) / kLoraKSlice);
        n_ks += d[i].n_ks;
    }
    // launches still in flight on any stream read the current table and
    // partial buffers: let them finish before any is replaced
    hipError_t e = hipDeviceSynchronize();
    if (e == hipSuccess) e = hipMalloc((void**)&vpart, (size_t)n_ks * 2 * h->r * sizeof(float));
    if (e == hipSuccess && switch_gemv_fused(h->tile, h->dtype)) {
        size_t total = 0;
        for (const SwDesc& q : d) total += (size_t)q.n_ct * q.d_out;
        e = hipMalloc((void**)&part, total * sizeof(float));
        size_t off = 0;
        for (int i = 0; i < h->n && e == hipSuccess; ++i) {
            d[i].part = part + off;
            off += (size_t)d[i].n_ct * d[i].d_out;
        }
    }
    if (e == hipSuccess) e = hipMemcpy(h->d_descs, d.data(), sizeof(SwDesc) * h->n, hipMemcpyHostToDevice);
    if (e != hipSuccess) {
        if (part) (void)hipFree(part);
        if (vpart) (void)hipFree(vpart);
        return hip_fail(e, "bind_vectors");
    }
    if (h->d_part) (void)hipFree(h->d_part);
    if (h->d_vpart) (void)hipFree(h->d_vpart);
    h->d_part = part;
    h->d_vpart = vpart;
    h->n_ks = n_ks;
    h->h_descs = std::move(d);
    h->bound = true;
    return ok();
}

int dlm_gemv(dlm_layers* h, void* stream) {
    if (!h) return fail(DLM_EINVAL, "gemv: null handle");
    if (!h->bound) return fail(DLM_EINVAL, "gemv: no vectors bound (dlm_layers_bind_vectors)");
    const SwitchArgs a = switch_args(h, nullptr, nullptr, nullptr, nullptr);
    hipError_t e = launch_gemv(a, h->n_blocks, h->dtype, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "gemv launch");
    return ok();
}

int dlm_switch_gemv(dlm_layers* h, const int32_t* old_idx, const float* old_g, const int32_t* new_idx,
                    const float* new_g, void* stream) {
    if (!h) return fail(DLM_EINVAL, "switch_gemv: null handle");
    if (!h->bound) return fail(DLM_EINVAL, "switch_gemv: no vectors bound (dlm_layers_bind_vectors)");
    const int rc = check_sets(h, old_idx, old_g, new_idx, new_g, "switch_gemv");
    if (rc != DLM_OK) return rc;
    const SwitchArgs a = switch_args(h, old_idx, old_g, new_idx, new_g);
    hipStream_t s = (hipStream_t)stream;
    hipError_t e;
    if (switch_gemv_fused(h->tile, h->dtype)) {
        e = launch_switch_gemv_bf16(a, s);
        if (e == hipSuccess) e = launch_gemv_reduce(a, h->n_bands, s);
    } else {
        e = h->dtype == DLM_BF16 ? launch_switch_bf16(a, h->tile, s) : launch_switch_generic(a, h->dtype, s);
        if (e == hipSuccess) e = launch_gemv(a, h->n_blocks, h->dtype, s);
    }
    if (e != hipSuccess) return hip_fail(e, "switch_gemv launch");
    return ok();
}

int dlm_switch_gemv_launches(const dlm_layers* h) { return h ? 2 : 0; }

int dlm_gemv_unmerged(dlm_layers* h, const int32_t* idx, const float* g, void* stream) {
    if (!h) return fail(DLM_EINVAL, "gemv_unmerged: null handle");
    if (!h->bound) return fail(DLM_EINVAL, "gemv_unmerged: no vectors bound (dlm_layers_bind_vectors)");
    if (!idx || !g) return fail(DLM_EINVAL, "gemv_unmerged: idx or g is null");
    const int rc = check_sets(h, nullptr, nullptr, idx, g, "gemv_unmerged");
    if (rc != DLM_OK) return rc;
    const SwitchArgs a = switch_args(h, nullptr, nullptr, idx, g);
    const hipError_t e = launch_gemv_unmerged(a, h->n_ks, h->n_blocks, h->dtype, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "gemv_unmerged launch");
    return ok();
}

int dlm_gemv_unmerged_launches(const dlm_layers* h) { return h ? 2 : 0; }

int dlm_layers_status(dlm_layers* h, int32_t* code, void* stream) {
    if (!h || !code) return fail(DLM_EINVAL, "layers_status: null argument");
    hipError_t e = hipStreamSynchronize((hipStream_t)stream);
    int32_t v = 0;
    if (e == hipSuccess) e = hipMemcpy(&v, h->d_err, sizeof v, hipMemcpyDeviceToHost);
    if (e == hipSuccess && v != 0) e = hipMemset(h->d_err, 0, sizeof v);
    if (e != hipSuccess) return hip_fail(e, "layers_status");
    *code = v ? DLM_EDEVICE : DLM_OK;
    return ok();
}

// ------------------------------------------------------------------ SGMM ----

int dlm_sgmm_workspace_size(int64_t T, int64_t d_in_max, int32_t E, int32_t r, int32_t n_problems,
                            size_t* bytes) {
    if (!bytes) return fail(DLM_EINVAL, "sgmm_workspace_size: bytes is null");
    if (T < 0 || T > ((int64_t)1 << 30)) return fail(DLM_ESHAPE, "sgmm_workspace_size: T=%lld", (long long)T);
    if (d_in_max < 1 || d_in_max > kMaxDim)
        return fail(DLM_ESHAPE, "sgmm_workspace_size: d_in_max=%lld", (long long)d_in_max);
    if (E < 1 || E > DLM_MAX_EXPERTS) return fail(DLM_ESHAPE, "sgmm_workspace_size: E=%d", E);
    if (r < 1 || r > DLM_MAX_RANK) return fail(DLM_ESHAPE, "sgmm_workspace_size: r=%d", r);
    if (n_problems < 1) return fail(DLM_EINVAL, "sgmm_workspace_size: n_problems=%d", n_problems);
    *bytes = sgmm_layout(T, d_in_max, E, r, n_problems).total;
    return ok();
}

namespace {

int check_problem(const dlm_sgmm_problem& p, int dtype, int i) {
    if (!p.x || !p.A || !p.B || !p.y) return fail(DLM_EINVAL, "sgmm: problem %d has a null pointer", i);
    if (p.d_in < 1 || p.d_out < 1 || p.d_in > kMaxDim || p.d_out > kMaxDim)
        return fail(DLM_ESHAPE, "sgmm: problem %d shape d_in=%lld d_out=%lld", i, (long long)p.d_in,
                    (long long)p.d_out);
    if (dtype == DLM_BF16) {
        if (!aligned16(p.x) || !aligned16(p.A) || !aligned16(p.B) || !aligned16(p.y))
            return fail(DLM_EALIGN, "sgmm: problem %d pointer not 16-byte aligned", i);
        if (p.d_in % 8 != 0 || p.d_out % 8 != 0)
            return fail(DLM_EALIGN, "sgmm: problem %d d_in/d_out not multiples of 8", i);
    }
    return DLM_OK;
}

int check_ws(void* ws, size_t ws_bytes, const SgLayout& L) {
    if (!ws) return fail(DLM_EWORKSPACE, "sgmm: workspace is null");
    if (((uintptr_t)ws & 255u) != 0) return fail(DLM_EALIGN, "sgmm: workspace not 256-byte aligned");
    if (ws_bytes < L.total)
        return fail(DLM_EWORKSPACE, "sgmm: workspace %zu bytes < %zu needed", ws_bytes, L.total);
    return DLM_OK;
}

int run_sgmm(const SgDesc* d_descs, const SgDesc* ks_desc, const SgDesc* cb_desc,
             const SgDesc& single, int n_prob, int64_t total_cb,
             int64_t total_ks, int64_t d_out_max, int32_t w_max, const int32_t* idx, const float* g, int64_t T,
             int E, int r, float scale, int dtype, int packed, void* ws, const SgLayout& L, hipStream_t s,
             int32_t* status_out = nullptr) {
    SgmmArgs a{};
    a.w_max = w_max;
    a.kslice = kSgmmKSlice;
    a.status_out = status_out;
    a.inline_seg = 0;  // launch_sgmm decides
    a.descs = d_descs;
    a.ks_desc = ks_desc;
    a.cb_desc = cb_desc;
    a.packed = packed;
    a.single = single;
    a.n_prob = n_prob;
    a.n_expand_units = L.tiles_max * total_cb;
    a.total_cb = total_cb;
    a.total_ks = total_ks;
    a.d_out_max = d_out_max;
    a.idx = idx;
    a.g = g;
    a.T = T;
    a.E = E;
    a.r = r;
    a.scale = scale;
    a.ws = (char*)ws;
    a.L = L;
    hipError_t e = launch_sgmm(a, dtype, s);
    if (e != hipSuccess) return hip_fail(e, "sgmm launch");
    return ok();
}

// Host checks shared by dlm_sgmm and dlm_sgmm_noalloc (everything but the
// workspace).  *done = true: T == 0, nothing to enqueue.
int check_sgmm_args(const void* x, const int32_t* idx, const float* g, const void* A, const void* B, void* y,
                    int64_t T, int64_t d_in, int64_t d_out, int32_t E, int32_t r, float scale, int32_t dtype,
                    const void* ws, size_t ws_bytes, bool* done) {
    *done = false;
    if (T < 0 || T > ((int64_t)1 << 30)) return fail(DLM_ESHAPE, "sgmm: T=%lld out of range", (long long)T);
    if (E < 1 || E > DLM_MAX_EXPERTS) return fail(DLM_ESHAPE, "sgmm: E=%d not in [1, %d]", E, DLM_MAX_EXPERTS);
    if (r < 1 || r > DLM_MAX_RANK) return fail(DLM_ESHAPE, "sgmm: r=%d not in [1, %d]", r, DLM_MAX_RANK);
    if (!valid_dtype(dtype)) return fail(DLM_EDTYPE, "sgmm: unknown dtype %d", dtype);
    if (!std::isfinite(scale)) return fail(DLM_EINVAL, "sgmm: scale is not finite");
    if (T == 0) {  // nothing to do; the (possibly empty) buffers are not looked at
        if (d_in < 1 || d_out < 1 || d_in > kMaxDim || d_out > kMaxDim)
            return fail(DLM_ESHAPE, "sgmm: shape d_in=%lld d_out=%lld", (long long)d_in, (long long)d_out);
        *done = true;
        return DLM_OK;
    }
    dlm_sgmm_problem p{x, A, B, y, d_in, d_out};
    int rc = check_problem(p, dtype, 0);
    if (rc != DLM_OK) return rc;
    if (!idx || !g) return fail(DLM_EINVAL, "sgmm: idx or g is null");
    const size_t es = esize(dtype);
    std::vector<Span> v = {span(x, (size_t)T * d_in * es, false, "x", 0), span(y, (size_t)T * d_out * es, true, "y", 0),
                           span(A, (size_t)E * r * d_in * es, false, "A", 0), span(B, (size_t)E * d_out * r * es, false, "B", 0),
                           span(idx, (size_t)T * 8, false, "idx", 0), span(g, (size_t)T * 8, false, "g", 0)};
    if (ws) v.push_back(span(ws, ws_bytes, true, "workspace", 0));
    Span a, b;
    if (write_conflict(std::move(v), &a, &b)) return conflict_fail("sgmm", a, b);
    return DLM_OK;
}

SgDesc single_desc(const void* x, const void* A, const void* B, void* y, int64_t d_in, int64_t d_out) {
    SgDesc d{};
    d.x = x;
    d.A = A;
    d.B = B;
    d.y = y;
    d.d_in = (int32_t)d_in;
    d.d_out = (int32_t)d_out;
    d.n_cb = (int32_t)((d_out + kSgmmExpandCols - 1) / kSgmmExpandCols);
    d.unit0 = 0;
    d.n_ks = (int32_t)((d_in + kSgmmKSlice - 1) / kSgmmKSlice);
    d.ks0 = 0;
    return d;
}

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// Device address of `scratch` on the current device (looked up on its first use there).
int scratch_on_current_device(void** out) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "sgmm_noalloc: hipGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(DLM_EDEVICE, "sgmm_noalloc: device %d out of range", dev);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return hip_fail(e, "sgmm_noalloc: hipGetSymbolAddress(scratch)");
        if (!p) return fail(DLM_EHIP, "sgmm_noalloc: scratch has no device address");
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return DLM_OK;
}

}  // namespace

int dlm_sgmm(const void* x, const int32_t* idx, const float* g, const void* A, const void* B,
             void* y, int64_t T, int64_t d_in, int64_t d_out, int32_t E, int32_t r, float scale,
             int32_t dtype, void* workspace, size_t ws_bytes, void* stream) {
    bool done = false;
    int rc = check_sgmm_args(x, idx, g, A, B, y, T, d_in, d_out, E, r, scale, dtype, workspace, ws_bytes, &done);
    if (rc != DLM_OK) return rc;
    if (done) return ok();
    const SgLayout L = sgmm_layout(T, d_in, E, r, 1);
    rc = check_ws(workspace, ws_bytes, L);
    if (rc != DLM_OK) return rc;
    const SgDesc d = single_desc(x, A, B, y, d_in, d_out);
    return run_sgmm(nullptr, nullptr, nullptr, d, 1, d.n_cb, d.n_ks, d_out, d.n_cb + d.n_ks, idx, g, T, E, r, scale,
                    dtype, 0, workspace, L,
                    (hipStream_t)stream);
}

int dlm_sgmm_noalloc(const void* x, const int32_t* idx, const float* g, const void* A, const void* B,
                     void* y, int64_t T, int64_t d_in, int64_t d_out, int32_t E, int32_t r, float scale,
                     int32_t dtype, int32_t* status, void* stream) {
    bool done = false;
    int rc = check_sgmm_args(x, idx, g, A, B, y, T, d_in, d_out, E, r, scale, dtype, status, status ? 4 : 0, &done);
    if (rc != DLM_OK) return rc;
    if (done) return ok();
    const SgLayout L = sgmm_layout(T, d_in, E, r, 1);
    if (L.total > kNoAllocScratchBytes)
        return fail(DLM_EWORKSPACE, "sgmm_noalloc: needs %zu bytes of scratch, the library's maximum is %zu "
                    "(use dlm_sgmm with a caller workspace)", L.total, kNoAllocScratchBytes);
    int sdev = -1, cdev = -1;
    hipError_t e = hipStreamGetDevice((hipStream_t)stream, &sdev);
    if (e == hipSuccess) e = hipGetDevice(&cdev);
    if (e != hipSuccess) return hip_fail(e, "sgmm_noalloc: stream device");
    if (sdev != cdev) return fail(DLM_EINVAL, "sgmm_noalloc: the stream belongs to device %d, not the current %d", sdev, cdev);
    void* ws = nullptr;
    rc = scratch_on_current_device(&ws);
    if (rc != DLM_OK) return rc;
    const SgDesc d = single_desc(x, A, B, y, d_in, d_out);
    return run_sgmm(nullptr, nullptr, nullptr, d, 1, d.n_cb, d.n_ks, d_out, d.n_cb + d.n_ks, idx, g, T, E, r, scale,
                    dtype, 0, ws, L,
                    (hipStream_t)stream, status);
}

int dlm_sgmm_group_create(const dlm_sgmm_problem* probs, int32_t n, int32_t E, int32_t r,
                          float scale, int32_t dtype, dlm_sgmm_group** out) {
    if (!out) return fail(DLM_EINVAL, "sgmm_group_create: out is null");
    *out = nullptr;
    if (!probs || n < 1 || n > 65535) return fail(DLM_EINVAL, "sgmm_group_create: bad problem list (n=%d)", n);
    if (E < 1 || E > DLM_MAX_EXPERTS) return fail(DLM_ESHAPE, "sgmm_group_create: E=%d", E);
    if (r < 1 || r > DLM_MAX_RANK) return fail(DLM_ESHAPE, "sgmm_group_create: r=%d", r);
    if (!valid_dtype(dtype)) return fail(DLM_EDTYPE, "sgmm_group_create: unknown dtype %d", dtype);
    if (!std::isfinite(scale)) return fail(DLM_EINVAL, "sgmm_group_create: scale is not finite");
    dlm_sgmm_group* h = new (std::nothrow) dlm_sgmm_group();
    if (!h) return fail(DLM_ENOMEM, "sgmm_group_create: host allocation failed");
    h->h_descs.resize(n);
    int64_t cb = 0, ks = 0, dmax = 0, dimax = 0;
    for (int i = 0; i < n; ++i) {
        const int rc = check_problem(probs[i], dtype, i);
        if (rc != DLM_OK) {
            delete h;
            return rc;
        }
        SgDesc& d = h->h_descs[i];
        d = SgDesc{};
        d.x = probs[i].x;
        d.A = probs[i].A;
        d.B = probs[i].B;
        d.y = probs[i].y;
        d.d_in = (int32_t)probs[i].d_in;
        d.d_out = (int32_t)probs[i].d_out;
        d.n_cb = (int32_t)((probs[i].d_out + kSgmmExpandCols - 1) / kSgmmExpandCols);
        d.unit0 = cb;
        cb += d.n_cb;
        d.n_ks = (int32_t)((probs[i].d_in + kSgmmKSlice - 1) / kSgmmKSlice);
        d.ks0 = ks;
        ks += d.n_ks;
        if (probs[i].d_out > dmax) dmax = probs[i].d_out;
        if (probs[i].d_in > dimax) dimax = probs[i].d_in;
        if (d.n_ks + d.n_cb > h->w_max) h->w_max = d.n_ks + d.n_cb;
    }
    h->n = n;
    h->E = E;
    h->r = r;
    h->scale = scale;
    h->dtype = dtype;
    h->total_cb = cb;
    h->total_ks = ks;
    h->d_out_max = dmax;
    h->d_in_max = dimax;
    hipError_t e = hipSuccess;
    if (dtype == DLM_BF16) {
        // one packed copy per distinct (A, d_in); problems sharing a bank share it
        std::map<std::pair<const void*, int64_t>, void*> seen;
        for (int i = 0; i < n && e == hipSuccess; ++i) {
            SgDesc& d = h->h_descs[i];
            const auto key = std::make_pair(d.A, (int64_t)d.d_in);
            auto it = seen.find(key);
            if (it == seen.end()) {
                void* ap = nullptr;
                e = hipMalloc(&ap, (size_t)E * r * d.d_in * 2);
                if (e != hipSuccess) break;
                h->packs.push_back({d.A, ap, d.d_in});
                e = launch_sgmm_pack_a(d.A, ap, E, r, d.d_in, nullptr);
                it = seen.emplace(key, ap).first;
            }
            d.Ap = it->second;
        }
        if (e == hipSuccess) e = hipStreamSynchronize(nullptr);
    }
    // one device block: the descriptors, then a copy of the owning problem's
    // descriptor for every K slice and every expand column group (a work item
    // reads its problem with one load, not an owner index and then the table)
    const size_t desc_bytes = (sizeof(SgDesc) * n + 255) & ~(size_t)255;
    const size_t ks_bytes = (sizeof(SgDesc) * (size_t)ks + 255) & ~(size_t)255;
    std::vector<char> blob(desc_bytes + ks_bytes + sizeof(SgDesc) * (size_t)cb);
    std::memcpy(blob.data(), h->h_descs.data(), sizeof(SgDesc) * n);
    SgDesc* ks_desc = (SgDesc*)(blob.data() + desc_bytes);
    SgDesc* cb_desc = (SgDesc*)(blob.data() + desc_bytes + ks_bytes);
    for (int i = 0; i < n; ++i) {
        const SgDesc& d = h->h_descs[i];
        for (int k = 0; k < d.n_ks; ++k) ks_desc[d.ks0 + k] = d;
        for (int k = 0; k < d.n_cb; ++k) cb_desc[d.unit0 + k] = d;
    }
    if (e == hipSuccess) e = hipMalloc((void**)&h->d_descs, blob.size());
    if (e == hipSuccess) e = hipMemcpy(h->d_descs, blob.data(), blob.size(), hipMemcpyHostToDevice);
    if (e != hipSuccess) {
        if (h->d_descs) (void)hipFree(h->d_descs);
        for (auto& pk : h->packs) (void)hipFree(pk.Ap);
        delete h;
        return hip_fail(e, "sgmm_group_create");
    }
    h->d_ks_desc = (const SgDesc*)((const char*)h->d_descs + desc_bytes);
    h->d_cb_desc = (const SgDesc*)((const char*)h->d_descs + desc_bytes + ks_bytes);
    *out = h;
    return ok();
}

int dlm_sgmm_group_destroy(dlm_sgmm_group* h) {
    if (!h) return fail(DLM_EINVAL, "sgmm_group_destroy: null handle");
    hipError_t e = hipDeviceSynchronize();
    if (h->d_descs) (void)hipFree(h->d_descs);
    for (auto& pk : h->packs) (void)hipFree(pk.Ap);
    if (h->grads.d_tab) (void)hipFree(h->grads.d_tab);
    if (h->grads.d_pack) (void)hipFree(h->grads.d_pack);
    delete h;
    if (e != hipSuccess) return hip_fail(e, "sgmm_group_destroy");
    return ok();
}

int dlm_sgmm_group_repack(dlm_sgmm_group* h, void* stream) {
    if (!h) return fail(DLM_EINVAL, "sgmm_group_repack: null handle");
    for (auto& pk : h->packs) {
        const hipError_t e = launch_sgmm_pack_a(pk.A, pk.Ap, h->E, h->r, pk.d_in, (hipStream_t)stream);
        if (e != hipSuccess) return hip_fail(e, "sgmm_group_repack");
    }
    return ok();
}

int dlm_sgmm_group_run(dlm_sgmm_group* h, const int32_t* idx, const float* g, int64_t T,
                       void* workspace, size_t ws_bytes, void* stream) {
    if (!h) return fail(DLM_EINVAL, "sgmm_group_run: null handle");
    if (T < 0 || T > ((int64_t)1 << 30)) return fail(DLM_ESHAPE, "sgmm_group_run: T=%lld", (long long)T);
    if (T == 0) return ok();
    if (!idx || !g) return fail(DLM_EINVAL, "sgmm_group_run: idx or g is null");
    const size_t es = esize(h->dtype);
    const SgLayout L = sgmm_layout(T, h->d_in_max, h->E, h->r, h->n);
    const int rc = check_ws(workspace, ws_bytes, L);
    if (rc != DLM_OK) return rc;
    {
        // every problem's ranges, the sets and the workspace: a written one (y,
        // workspace) may overlap nothing else.  The problems' extents grow with
        // T, so a row count up to one already checked needs only the per-call
        // pointers (sets, workspace) checked again.
        std::vector<Span> v;
        const int64_t Tc = T > h->checked_T ? T : h->checked_T;
        for (int i = 0; i < h->n; ++i) {
            const SgDesc& d = h->h_descs[i];
            v.push_back(span(d.x, (size_t)Tc * d.d_in * es, false, "problem x", i));
            v.push_back(span(d.y, (size_t)Tc * d.d_out * es, true, "problem y", i));
            v.push_back(span(d.A, (size_t)h->E * h->r * d.d_in * es, false, "problem A", i));
            v.push_back(span(d.B, (size_t)h->E * d.d_out * h->r * es, false, "problem B", i));
        }
        if (T > h->checked_T) {
            Span a, b;
            if (write_conflict(v, &a, &b)) return conflict_fail("sgmm_group_run", a, b);
            h->checked_T = T;
        }
        const Span call[3] = {span(idx, (size_t)T * 8, false, "idx", 0), span(g, (size_t)T * 8, false, "g", 0),
                              span(workspace, ws_bytes, true, "workspace", 0)};
        for (const Span& c : call)
            for (const Span& q : v)
                if (c.hi > q.lo && q.hi > c.lo && (c.write || q.write)) return conflict_fail("sgmm_group_run", c, q);
        if (overlap(workspace, ws_bytes, idx, (size_t)T * 8) || overlap(workspace, ws_bytes, g, (size_t)T * 8))
            return fail(DLM_EINVAL, "sgmm_group_run: the workspace overlaps the sets");
    }
    return run_sgmm(h->d_descs, h->d_ks_desc, h->d_cb_desc, h->h_descs[0], h->n, h->total_cb, h->total_ks, h->d_out_max,
                    h->w_max, idx, g, T, h->E,
                    h->r, h->scale, h->dtype, h->packs.empty() ? 0 : 1, workspace, L, (hipStream_t)stream);
}

// ------------------------------------------------------- SGMM gradients ----

static SgGradLayout grad_layout(const dlm_sgmm_group* h, int64_t T) {
    const auto& G = h->grads;
    return sgmm_grad_layout(T, G.for_rows(T).total_ks, h->E, h->r, h->n, G.n_units, h->dtype);
}

int dlm_sgmm_group_backward_workspace_size(const dlm_sgmm_group* h, int64_t T, size_t* bytes) {
    if (!h || !bytes) return fail(DLM_EINVAL, "sgmm_group_backward_workspace_size: null argument");
    if (!h->grads.bound) return fail(DLM_EINVAL, "sgmm_group_backward_workspace_size: no gradients are bound");
    if (T < 0 || T > ((int64_t)1 << 29))
        return fail(DLM_ESHAPE, "sgmm_group_backward_workspace_size: T=%lld", (long long)T);
    // enough for fewer rows too: those that take the narrower K slices have more of them
    const int64_t few = 32 * ((kSgmmFewItems - 1) / h->grads.slices[0].total_ks);
    *bytes = grad_layout(h, T).total;
    if (few > 0 && few < T) *bytes = std::max(*bytes, grad_layout(h, few).total);
    return ok();
}

int dlm_sgmm_group_bind_grads(dlm_sgmm_group* h, const void* const* dy, void* const* dx, float* const* dA,
                              float* const* dB) {
    if (!h) return fail(DLM_EINVAL, "sgmm_group_bind_grads: null handle");
    if (!dy || !dA || !dB) return fail(DLM_EINVAL, "sgmm_group_bind_grads: null pointer list");
    const int n = h->n, E = h->E, r = h->r;
    const bool bf = h->dtype == DLM_BF16;
    const size_t es = esize(h->dtype);
    if (n > 32767) return fail(DLM_ESHAPE, "sgmm_group_bind_grads: %d problems (at most 32767)", n);
    for (int i = 0; i < n; ++i) {
        if (!dy[i] || !dA[i] || !dB[i]) return fail(DLM_EINVAL, "sgmm_group_bind_grads: problem %d has a null pointer", i);
        const uintptr_t m = bf ? 15 : 3;
        if (((uintptr_t)dy[i] & m) || (dx && ((uintptr_t)dx[i] & m)) || ((uintptr_t)dA[i] & m) || ((uintptr_t)dB[i] & m))
            return fail(DLM_EALIGN, "sgmm_group_bind_grads: problem %d pointer not %d-byte aligned", i, (int)m + 1);
    }
    dlm_sgmm_group::Grads G;
    hipError_t e = hipSuccess;
    try {
        auto a256 = [](size_t v) { return (v + 255) & ~(size_t)255; };
        // per problem: the place of its dx in the order of the problems that share
        // it, and its transposes' offsets
        std::vector<int> wave(n, -1);
        std::map<void*, std::pair<int, int>> uses;  // dx -> (d_in, problems so far)
        int n_waves = 0;
        std::vector<size_t> o_at(n), o_bt(n);
        size_t pack_bytes = 0;
        for (int i = 0; i < n; ++i) {
            const SgDesc& p = h->h_descs[i];
            o_at[i] = pack_bytes;
            pack_bytes += a256((size_t)E * (bf ? (r + 15) / 16 * 16 : r) * p.d_in * es);
            o_bt[i] = pack_bytes;
            pack_bytes += a256((size_t)E * r * p.d_out * es);
            if (!dx || !dx[i]) continue;
            auto it = uses.emplace(dx[i], std::make_pair(p.d_in, 0)).first;
            if (it->second.first != p.d_in)  // with another width it would be another layout
                return fail(DLM_EINVAL, "sgmm_group_bind_grads: problem %d shares a dx with one of another d_in", i);
            wave[i] = it->second.second++;
            n_waves = std::max(n_waves, wave[i] + 1);
        }
        // outer products: side 0 has x's columns, side 1 dy's
        std::vector<SgOuter> outers(2 * (size_t)n);
        int64_t units = 0;
        const int cols = grad_cols(h->dtype);
        for (int i = 0; i < 2 * n; ++i) {
            const SgDesc& p = h->h_descs[i % n];
            SgOuter& o = outers[i];
            o = SgOuter{};
            o.act = i < n ? p.x : dy[i - n];
            o.out = i < n ? dA[i] : dB[i - n];
            o.d = i < n ? p.d_in : p.d_out;
            o.side = i < n ? 0 : 1;
            o.prob = i % n;
            o.unit0 = (int32_t)units;
            units += (o.d + cols - 1) / cols;
            if (units > ((int64_t)1 << 24)) return fail(DLM_ESHAPE, "sgmm_group_bind_grads: too many columns");
        }
        G.n_units = (int32_t)units;
        std::vector<int32_t> unit_outer(units);
        for (int i = 0; i < 2 * n; ++i)
            std::fill(unit_outer.begin() + outers[i].unit0,
                      i + 1 < 2 * n ? unit_outer.begin() + outers[i + 1].unit0 : unit_outer.end(), i);
        G.dy.assign(dy, dy + n);
        G.dx.assign(n, nullptr);
        if (dx) G.dx.assign(dx, dx + n);
        G.dA.assign(dA, dA + n);
        G.dB.assign(dB, dB + n);

        e = hipDeviceSynchronize();  // launches in flight read the current tables
        if (e == hipSuccess) e = hipMalloc((void**)&G.d_pack, pack_bytes);
        // the transposes' padding ranks, which no call writes
        if (e == hipSuccess && bf && r % 16 != 0) e = hipMemset(G.d_pack, 0, pack_bytes);
        std::vector<char> tab;
        auto put = [&](const void* src, size_t bytes) {
            const size_t o = tab.size();
            tab.resize(a256(o + bytes));
            std::memcpy(tab.data() + o, src, bytes);
            return o;
        };
        auto owners = [](const std::vector<SgDesc>& v, bool cb) {
            std::vector<SgDesc> o;
            for (const SgDesc& d : v) o.insert(o.end(), cb ? d.n_cb : d.n_ks, d);
            return o;
        };
        const size_t o_outers = put(outers.data(), sizeof(SgOuter) * outers.size());
        const size_t o_units = put(unit_outer.data(), sizeof(int32_t) * unit_outer.size());
        size_t o_descs[2], o_ks[2], o_probs[2];
        std::vector<std::pair<size_t, size_t>> o_waves[2];
        for (int w2 = 0; w2 < 2 && e == hipSuccess; ++w2) {
            auto& S = G.slices[w2];
            S.width = w2 ? kSgmmKSliceFew : kSgmmKSlice;
            std::vector<SgDesc> descs(2 * (size_t)n);
            for (int i = 0; i < 2 * n; ++i) {
                const SgDesc& p = h->h_descs[i % n];
                SgDesc& d = descs[i];
                d = SgDesc{};
                d.x = i < n ? p.x : dy[i - n];
                d.A = i < n ? p.A : G.d_pack + o_bt[i - n];
                d.Ap = i < n ? p.Ap : G.d_pack + o_bt[i - n];
                d.d_in = i < n ? p.d_in : p.d_out;
                d.n_ks = bf ? (d.d_in + S.width - 1) / S.width : 1;
                d.ks0 = S.total_ks;
                S.total_ks += d.n_ks;
            }
            std::vector<SgGrad> probs(n);
            int64_t pk = 0;
            for (int i = 0; i < n; ++i) {
                const SgDesc& p = h->h_descs[i];
                SgGrad& q = probs[i];
                q = SgGrad{};
                q.A = p.A;
                q.B = p.B;
                q.x = p.x;
                q.dy = dy[i];
                q.Ap = const_cast<void*>(p.Ap);
                q.At = G.d_pack + o_at[i];
                q.Bt = G.d_pack + o_bt[i];
                q.d_in = p.d_in;
                q.d_out = p.d_out;
                q.pk0 = pk;
                pk += (int64_t)E * r * (bf ? p.d_in / 8 + p.d_out / 8 : p.d_in + p.d_out);
                q.ks_u = descs[i].ks0;
                q.ks_w = descs[n + i].ks0;
                // above kSgmmFoldRank the K-slice sum launch has added the slices
                const bool summed = (r + 15) / 16 * 16 > kSgmmFoldRank;
                q.n_ks_u = summed ? 1 : descs[i].n_ks;
                q.n_ks_w = summed ? 1 : descs[n + i].n_ks;
            }
            G.pk_total = pk;
            const std::vector<SgDesc> ks = owners(descs, false);
            o_descs[w2] = put(descs.data(), sizeof(SgDesc) * descs.size());
            o_ks[w2] = put(ks.data(), sizeof(SgDesc) * ks.size());
            o_probs[w2] = put(probs.data(), sizeof(SgGrad) * n);
            for (int w = 0; w < n_waves; ++w) {
                std::vector<SgDesc> v;
                dlm_sgmm_group::Grads::Wave W{};
                for (int i = 0; i < n; ++i) {
                    if (wave[i] != w) continue;
                    SgDesc d = descs[n + i];  // its K slices: w = B^T dy
                    d.B = probs[i].At;
                    d.y = dx[i];
                    d.d_out = h->h_descs[i].d_in;
                    d.n_cb = (d.d_out + kSgmmExpandCols - 1) / kSgmmExpandCols;
                    d.unit0 = W.total_cb;
                    W.total_cb += d.n_cb;
                    W.d_max = std::max<int64_t>(W.d_max, d.d_out);
                    W.w_max = std::max(W.w_max, d.n_ks + d.n_cb);
                    v.push_back(d);
                }
                W.n = (int32_t)v.size();
                const std::vector<SgDesc> cb = owners(v, true);
                const size_t ow = put(v.data(), sizeof(SgDesc) * v.size());
                o_waves[w2].push_back({ow, put(cb.data(), sizeof(SgDesc) * cb.size())});
                S.waves.push_back(W);
            }
        }
        if (e == hipSuccess) e = hipMalloc((void**)&G.d_tab, tab.size());
        if (e == hipSuccess) e = hipMemcpy(G.d_tab, tab.data(), tab.size(), hipMemcpyHostToDevice);
        if (e == hipSuccess) {
            G.outers = (const SgOuter*)(G.d_tab + o_outers);
            G.unit_outer = (const int32_t*)(G.d_tab + o_units);
            for (int w2 = 0; w2 < 2; ++w2) {
                auto& S = G.slices[w2];
                S.descs = (const SgDesc*)(G.d_tab + o_descs[w2]);
                S.ks_desc = (const SgDesc*)(G.d_tab + o_ks[w2]);
                S.probs = (const SgGrad*)(G.d_tab + o_probs[w2]);
                for (size_t w = 0; w < S.waves.size(); ++w) {
                    S.waves[w].descs = (const SgDesc*)(G.d_tab + o_waves[w2][w].first);
                    S.waves[w].cb_desc = (const SgDesc*)(G.d_tab + o_waves[w2][w].second);
                }
            }
        }
    } catch (const std::bad_alloc&) {
        if (G.d_tab) (void)hipFree(G.d_tab);
        if (G.d_pack) (void)hipFree(G.d_pack);
        return fail(DLM_ENOMEM, "sgmm_group_bind_grads: host allocation failed");
    }
    if (e != hipSuccess) {
        if (G.d_tab) (void)hipFree(G.d_tab);
        if (G.d_pack) (void)hipFree(G.d_pack);
        return hip_fail(e, "sgmm_group_bind_grads");
    }
    if (h->grads.d_tab) (void)hipFree(h->grads.d_tab);
    if (h->grads.d_pack) (void)hipFree(h->grads.d_pack);
    G.bound = true;
    h->grads = std::move(G);
    return ok();
}

int dlm_sgmm_group_backward(dlm_sgmm_group* h, const int32_t* idx, const float* g, float* dg, int64_t T,
                            int32_t accumulate, void* workspace, size_t ws_bytes, void* stream) {
    if (!h) return fail(DLM_EINVAL, "sgmm_group_backward: null handle");
    dlm_sgmm_group::Grads& G = h->grads;
    if (!G.bound) return fail(DLM_EINVAL, "sgmm_group_backward: no gradients are bound");
    if (T < 0 || T > ((int64_t)1 << 29)) return fail(DLM_ESHAPE, "sgmm_group_backward: T=%lld", (long long)T);
    hipStream_t s = (hipStream_t)stream;
    const auto& S = G.for_rows(T);
    const bool bf = h->dtype == DLM_BF16;
    SgGradArgs b{};
    b.probs = S.probs;
    b.outers = G.outers;
    b.unit_outer = G.unit_outer;
    b.ks_desc = S.ks_desc;
    b.total_ks = S.total_ks;
    b.kslice = S.width;
    b.n_prob = h->n;
    b.n_units = G.n_units;
    b.pk_total = G.pk_total;
    b.E = h->E;
    b.r = h->r;
    b.scale = h->scale;
    b.accumulate = accumulate ? 1 : 0;
    if (T == 0) {
        if (accumulate) return ok();
        const hipError_t e = launch_grad_zero(b, h->dtype, s);
        return e == hipSuccess ? ok() : hip_fail(e, "sgmm_group_backward");
    }
    if (!idx || !g) return fail(DLM_EINVAL, "sgmm_group_backward: idx or g is null");
    if (!workspace) return fail(DLM_EWORKSPACE, "sgmm_group_backward: workspace is null");
    if (((uintptr_t)workspace & 255u) != 0) return fail(DLM_EALIGN, "sgmm_group_backward: workspace not 256-byte aligned");
    const SgGradLayout L = grad_layout(h, T);
    if (ws_bytes < L.total)
        return fail(DLM_EWORKSPACE, "sgmm_group_backward: workspace %zu bytes < %zu needed", ws_bytes, L.total);
    try {
        // a written range overlaps nothing, but that problems may share one dx
        // (added to in launches of their own); checked again when T grows
        const size_t es = esize(h->dtype);
        const int64_t Tc = T > G.checked_T ? T : G.checked_T;
        std::vector<Span> v;
        std::map<void*, int> seen;
        for (int i = 0; i < h->n; ++i) {
            const SgDesc& d = h->h_descs[i];
            const size_t na = (size_t)h->E * h->r * d.d_in, nb = (size_t)h->E * h->r * d.d_out;
            v.push_back(span(d.x, (size_t)Tc * d.d_in * es, false, "problem x", i));
            v.push_back(span(G.dy[i], (size_t)Tc * d.d_out * es, false, "problem dy", i));
            v.push_back(span(d.A, na * es, false, "problem A", i));
            v.push_back(span(d.B, nb * es, false, "problem B", i));
            v.push_back(span(G.dA[i], na * 4, true, "problem dA", i));
            v.push_back(span(G.dB[i], nb * 4, true, "problem dB", i));
            if (G.dx[i] && seen.emplace(G.dx[i], i).second)
                v.push_back(span(G.dx[i], (size_t)Tc * d.d_in * es, true, "problem dx", i));
        }
        if (T > G.checked_T) {
            Span p, q;
            if (write_conflict(v, &p, &q)) return conflict_fail("sgmm_group_backward", p, q);
            G.checked_T = T;
        }
        std::vector<Span> call = {span(idx, (size_t)T * 8, false, "idx", 0), span(g, (size_t)T * 8, false, "g", 0),
                                  span(workspace, ws_bytes, true, "workspace", 0)};
        if (dg) call.push_back(span(dg, (size_t)T * 8, true, "dg", 0));
        for (const Span& c : call)
            for (const Span& q : v)
                if (c.hi > q.lo && q.hi > c.lo && (c.write || q.write)) return conflict_fail("sgmm_group_backward", c, q);
        Span p, q;
        if (write_conflict(call, &p, &q)) return conflict_fail("sgmm_group_backward", p, q);
    } catch (const std::bad_alloc&) {
        return fail(DLM_ENOMEM, "sgmm_group_backward: host allocation failed");
    }
    SgmmArgs a{};
    a.descs = S.descs;
    a.ks_desc = S.ks_desc;
    a.packed = bf ? 1 : 0;
    a.n_prob = 2 * h->n;
    a.total_ks = S.total_ks;
    a.kslice = S.width;
    a.idx = idx;
    a.g = g;
    a.T = T;
    a.E = h->E;
    a.r = h->r;
    a.scale = h->scale;
    a.ws = (char*)workspace;
    a.L = L.L;
    b.idx = idx;
    b.T = T;
    b.ws = (char*)workspace;
    b.G = L;
    b.dg = dg;
    auto expand_args = [&](const dlm_sgmm_group::Grads::Wave& w) {
        SgmmArgs x = a;
        x.descs = w.descs;
        x.cb_desc = w.cb_desc;
        x.ks_desc = nullptr;
        x.n_prob = w.n;
        x.total_cb = w.total_cb;
        x.n_expand_units = L.L.tiles_max * w.total_cb;
        x.d_out_max = w.d_max;
        x.w_max = w.w_max;
        x.total_ks = 0;
        return x;
    };
    bool fits = sgmm_grad_fits(b, h->dtype) && sgmm_launches_fit(a, h->dtype);
    for (const auto& w : S.waves) fits = fits && grad_expand_fits(b, expand_args(w), h->dtype);
    if (!fits) return hip_fail(hipErrorInvalidConfiguration, "sgmm_group_backward");
    hipError_t e = launch_grad_prep(b, g, h->dtype, s);
    if (bf && h->r >= kGradListRank) {
        if (e == hipSuccess) e = launch_grad_shrink(b, s);
        if (e == hipSuccess) e = launch_sgmm_vsum(a, s);
    } else if (e == hipSuccess) {
        e = bf ? launch_sgmm_shrink(a, s) : launch_grad_shrink_f32(b, s);
    }
    if (e == hipSuccess && S.waves.empty()) e = launch_grad_coefs(b, h->dtype, s);
    for (const auto& w : S.waves)  // the first also writes the coefficients
        if (e == hipSuccess) e = launch_grad_expand(b, expand_args(w), &w == &S.waves[0], h->dtype, s);
    if (e == hipSuccess) e = launch_grad_outer(b, h->dtype, s);
    if (e != hipSuccess) return hip_fail(e, "sgmm_group_backward");
    return ok();
}

int dlm_sgmm_status(void* workspace, int32_t* code, void* stream) {
    if (!workspace || !code) return fail(DLM_EINVAL, "sgmm_status: null argument");
    hipError_t e = hipStreamSynchronize((hipStream_t)stream);
    int32_t v = 0;
    if (e == hipSuccess) e = hipMemcpy(&v, (char*)workspace + SG_ERR * 4, sizeof v, hipMemcpyDeviceToHost);
    if (e == hipSuccess && v != 0) e = hipMemset((char*)workspace + SG_ERR * 4, 0, sizeof v);
    if (e != hipSuccess) return hip_fail(e, "sgmm_status");
    *code = v ? DLM_EDEVICE : DLM_OK;
    return ok();
}

int dlm_sgmm_launches(int64_t T, int64_t d_in_max, int32_t r, int32_t n_problems, int32_t dtype) {
    if (T < 0 || d_in_max < 1 || r < 1 || r > DLM_MAX_RANK || n_problems < 1 ||
        (dtype != DLM_F32 && dtype != DLM_BF16)) {
        fail(DLM_EINVAL, "sgmm_launches: T < 0, d_in_max < 1, r outside [1, DLM_MAX_RANK], n_problems < 1 or unknown dtype");
        return -1;
    }
    if (T == 0) return 0;
    if (dtype == DLM_BF16 && T <= kSgmmSmallT) return n_problems == 1 ? 1 : 2;
    const int seg = T > kSgmmSegFewRows ? 2 : 1;
    if (dtype == DLM_F32) return seg + 2;
    const int vsum = d_in_max > kSgmmKSlice && r > kSgmmFoldRank ? 1 : 0;
    const bool fold = (r + 15) / 16 * 16 <= kSgmmFoldRank;
    const bool fused_ks = (d_in_max + kSgmmKSlice - 1) / kSgmmKSlice <= kSgmmFusedMaxKs;
    const bool fused_pairs = (int64_t)n_problems * ((T + 31) / 32) >= kSgmmFusedMinPairs;
    if (fold && r % 8 == 0 && fused_ks && fused_pairs && kSgmmFused > 0 && (kSgmmFused > 1 || T > kSgmmInlineRows))
        return seg + 1;  // one launch after the segmentation
    if (T <= kSgmmInlineRows && !vsum) return 2;  // the rows ordered inside the shrink and expand
    return seg + 2 + vsum;
}

// ----------------------------------------------------------------- AdamW ----

int dlm_adamw_create(const dlm_adamw_param* params, int32_t n, int32_t p_dtype, int32_t g_dtype, int32_t state_bits,
                     int64_t step, uint32_t seed, dlm_adamw** out) {
    if (!out) return fail(DLM_EINVAL, "adamw_create: out is null");
    *out = nullptr;
    if (!params || n < 1 || n > (1 << 20)) return fail(DLM_EINVAL, "adamw_create: bad tensor list (n=%d)", n);
    if (!valid_dtype(p_dtype) || !valid_dtype(g_dtype))
        return fail(DLM_EDTYPE, "adamw_create: unknown dtype (p %d, g %d)", p_dtype, g_dtype);
    if (state_bits != 32 && state_bits != 8) return fail(DLM_EINVAL, "adamw_create: state_bits=%d is not 32 or 8", state_bits);
    if (step < 0 || step >= ((int64_t)1 << 31)) return fail(DLM_EINVAL, "adamw_create: step=%lld", (long long)step);
    const size_t ps = esize(p_dtype), gs = esize(g_dtype), ss = state_bits == 32 ? 4 : 1;
    std::vector<AdDesc> descs;
    std::vector<Span> v;
    std::vector<char> blob;
    dlm_adamw* h = nullptr;
    int64_t chunks = 0;
    size_t desc_bytes = 0;
    try {
        descs.resize(n);
        for (int i = 0; i < n; ++i) {
            const dlm_adamw_param& q = params[i];
            AdDesc& d = descs[i];
            if (q.n < 0 || q.n > ((int64_t)1 << 40)) return fail(DLM_ESHAPE, "adamw_create: tensor %d: n=%lld", i, (long long)q.n);
            if (q.n > 0 && (!q.p || !q.g || !q.m || !q.v || (state_bits == 8 && (!q.m_scale || !q.v_scale))))
                return fail(DLM_EINVAL, "adamw_create: tensor %d: null pointer", i);
            if (q.master && p_dtype == DLM_F32)
                return fail(DLM_EINVAL, "adamw_create: tensor %d: an fp32 parameter has no master", i);
            if (!std::isfinite(q.weight_decay)) return fail(DLM_EINVAL, "adamw_create: tensor %d: weight_decay is not finite", i);
            if ((uintptr_t)q.p % ps || (uintptr_t)q.g % gs || (uintptr_t)q.m % ss || (uintptr_t)q.v % ss ||
                (uintptr_t)q.master % 4 || (uintptr_t)q.m_scale % 4 || (uintptr_t)q.v_scale % 4)
                return fail(DLM_EALIGN, "adamw_create: tensor %d: a pointer is not a multiple of its element's size", i);
            d = AdDesc{};
            d.p = q.p;
            d.g = q.g;
            d.master = q.master;
            d.m = q.m;
            d.v = q.v;
            d.ms = q.m_scale;
            d.vs = q.v_scale;
            d.n = q.n;
            d.wd = q.weight_decay;
            d.vec = (uintptr_t)q.p % (4 * ps) == 0 && (uintptr_t)q.g % (4 * gs) == 0 && (uintptr_t)q.m % (4 * ss) == 0 &&
                    (uintptr_t)q.v % (4 * ss) == 0 && (uintptr_t)q.master % 16 == 0;
            d.chunk0 = chunks;
            chunks += (q.n + kAdamChunk - 1) / kAdamChunk;
            const size_t nb = (size_t)(q.n + kAdamBlock - 1) / kAdamBlock * 4;
            v.push_back(span(q.p, q.n * ps, true, "p", i));
            v.push_back(span(q.g, q.n * gs, false, "g", i));
            v.push_back(span(q.m, q.n * ss, true, "m", i));
            v.push_back(span(q.v, q.n * ss, true, "v", i));
            if (q.master) v.push_back(span(q.master, (size_t)q.n * 4, true, "master", i));
            if (state_bits == 8) {
                v.push_back(span(q.m_scale, nb, true, "m_scale", i));
                v.push_back(span(q.v_scale, nb, true, "v_scale", i));
            }
        }
        if (!grid_fits(chunks, 256)) return fail(DLM_ESHAPE, "adamw_create: the sizes need a launch grid of more than 2^32 - 1 work-items");
        Span a, b;
        if (write_conflict(std::move(v), &a, &b)) return conflict_fail("adamw_create", a, b);
        desc_bytes = (sizeof(AdDesc) * n + 255) & ~(size_t)255;
        blob.resize(desc_bytes + sizeof(int32_t) * (2 * (size_t)chunks + 1));
        std::memcpy(blob.data(), descs.data(), sizeof(AdDesc) * n);
        int32_t* map = (int32_t*)(blob.data() + desc_bytes);
        for (int i = 0; i < n; ++i) {
            const int64_t end = i + 1 < n ? descs[i + 1].chunk0 : chunks;
            for (int64_t c = descs[i].chunk0; c < end; ++c) map[c] = i;
        }
        std::fill(map + chunks, map + 2 * chunks, (int32_t)step);
        map[2 * chunks] = 0;
        h = new dlm_adamw();
    } catch (const std::bad_alloc&) {
        return fail(DLM_ENOMEM, "adamw_create: host allocation failed");
    }
    hipError_t e = hipMalloc((void**)&h->d_descs, blob.size());
    if (e == hipSuccess) e = hipMemcpy(h->d_descs, blob.data(), blob.size(), hipMemcpyHostToDevice);
    if (e != hipSuccess) {
        if (h->d_descs) (void)hipFree(h->d_descs);
        delete h;
        return hip_fail(e, "adamw_create");
    }
    h->d_chunk_tensor = (const int32_t*)((const char*)h->d_descs + desc_bytes);
    h->d_steps = const_cast<int32_t*>(h->d_chunk_tensor) + chunks;
    h->d_err = h->d_steps + chunks;
    h->step0 = step;
    h->n_chunks = chunks;
    h->p_dtype = p_dtype;
    h->g_dtype = g_dtype;
    h->bits = state_bits;
    h->seed = seed;
    *out = h;
    return ok();
}

int dlm_adamw_destroy(dlm_adamw* h) {
    if (!h) return fail(DLM_EINVAL, "adamw_destroy: null handle");
    const hipError_t e = hipDeviceSynchronize();
    (void)hipFree(h->d_descs);
    delete h;
    if (e != hipSuccess) return hip_fail(e, "adamw_destroy");
    return ok();
}

int dlm_adamw_step(dlm_adamw* h, const dlm_adamw_cfg* c, const float* lr_scale, const float* grad_scale, void* stream) {
    if (!h || !c) return fail(DLM_EINVAL, "adamw_step: null argument");
    if (!std::isfinite(c->lr)) return fail(DLM_EINVAL, "adamw_step: lr is not finite");
    if (!(c->beta1 >= 0.0 && c->beta1 < 1.0) || !(c->beta2 >= 0.0 && c->beta2 < 1.0))
        return fail(DLM_EINVAL, "adamw_step: beta1=%g, beta2=%g not in [0, 1)", c->beta1, c->beta2);
    if (!(c->eps > 0.f) || !std::isfinite(c->eps)) return fail(DLM_EINVAL, "adamw_step: eps=%g is not positive", c->eps);
    if (h->bits == 8 && c->eps < FLT_MIN)  // the kernel's reciprocal of such a number is infinite
        return fail(DLM_EINVAL, "adamw_step: eps=%g is below 2^-126, the least with 8-bit moments", c->eps);
    if (h->n_chunks == 0) return ok();
    AdamArgs a{};
    a.descs = h->d_descs;
    a.chunk_tensor = h->d_chunk_tensor;
    a.steps = h->d_steps;
    a.err = h->d_err;
    a.n_chunks = h->n_chunks;
    a.beta1 = c->beta1;
    a.beta2 = c->beta2;
    a.lb1 = std::log(c->beta1);
    a.lb2 = std::log(c->beta2);
    a.lr = c->lr;
    a.eps = c->eps;
    a.seed = h->seed;
    a.lr_scale = lr_scale;
    a.grad_scale = grad_scale;
    const hipError_t e = launch_adamw(a, h->p_dtype, h->g_dtype, h->bits, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "adamw_step launch");
    return ok();
}

int dlm_adamw_status(dlm_adamw* h, int64_t* step, int32_t* code, void* stream) {
    if (!h || !step || !code) return fail(DLM_EINVAL, "adamw_status: null argument");
    uint32_t t = (uint32_t)h->step0;  // a handle of empty tensors counts nothing
    int32_t err = 0;
    hipError_t e = hipStreamSynchronize((hipStream_t)stream);
    if (e == hipSuccess && h->n_chunks > 0) e = hipMemcpy(&t, h->d_steps, sizeof t, hipMemcpyDeviceToHost);
    if (e == hipSuccess) e = hipMemcpy(&err, h->d_err, sizeof err, hipMemcpyDeviceToHost);
    if (e == hipSuccess && err) e = hipMemset(h->d_err, 0, sizeof err);
    if (e != hipSuccess) return hip_fail(e, "adamw_status");
    *step = t;
    *code = err ? DLM_EDEVICE : DLM_OK;
    return ok();
}

int dlm_adamw_read_state(const int8_t* m, const uint8_t* v, const float* m_scale, const float* v_scale, int64_t n,
                         float* m_out, float* v_out, void* stream) {
    if (n < 0 || n > ((int64_t)1 << 40)) return fail(DLM_ESHAPE, "adamw_read_state: n=%lld", (long long)n);
    if (n == 0) return ok();
    if (!m || !v || !m_scale || !v_scale || !m_out || !v_out) return fail(DLM_EINVAL, "adamw_read_state: null pointer");
    const size_t nb = (size_t)(n + kAdamBlock - 1) / kAdamBlock * 4;
    Span a, b;
    const Span v8[] = {span(m, n, false, "m", 0), span(v, n, false, "v", 0), span(m_scale, nb, false, "m_scale", 0),
                       span(v_scale, nb, false, "v_scale", 0), span(m_out, (size_t)n * 4, true, "m_out", 0),
                       span(v_out, (size_t)n * 4, true, "v_out", 0)};
    if (pair_conflict(v8, &a, &b)) return conflict_fail("adamw_read_state", a, b);
    const hipError_t e = launch_adamw_read_state(m, v, m_scale, v_scale, n, m_out, v_out, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "adamw_read_state launch");
    return ok();
}

}  // extern "C"
