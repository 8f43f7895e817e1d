// Structures shared between the host API (api.hip) and the SGMM kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dlm {

// ---- SGMM -----------------------------------------------------------------

struct SgDesc {
    const void* x;
    const void* A;
    const void* Ap;     // packed copy of A ([E][d_in / 8][r][8]), or nullptr
    const void* B;
    void* y;
    int32_t d_in, d_out;
    int32_t n_cb;       // column groups of the expand (kSgmmExpandCols each)
    int32_t n_ks;       // kSgmmKSlice-wide K slices of the shrink
    int64_t ks0;        // first K slice of this problem (prefix sum of n_ks)
    int64_t unit0;      // first column block of this problem (prefix sum of n_cb)
};

// Workspace sections (byte offsets, each 256-aligned).
struct SgLayout {
    // perm: row at each sorted position (-1 = padding); epk: its expert pair
    // (slot 0 in the low 16 bits, slot 1 in the high, -1 = empty); gpk: its two
    // gates; hist, cerr: each segmentation chunk's key counts and bad-set flag;
    // v: the shrink's results
    // dep, xcd: the one-launch shrink + expand's per-(problem, tile) counts of
    // finished shrink items and its per-XCD work ranges
    size_t hdr, perm, epk, gpk, hist, cerr, v, dep, xcd, total;
    int64_t T, T_pad, tiles_max, n_chunks;
    int r_pad;
    int max_ks;  // K slices of the widest problem
};
// Width of one shrink K slice (one work item; its fp32 partial v is summed
// with the other slices' afterwards).
constexpr int kSgmmKSlice = 2048;
// The gradients take narrower slices while kSgmmKSlice would leave fewer than
// kSgmmFewItems shrink items, one per CU: 256 rows of a 4096 x 4096 projection
// make 32 items, 18 us, or 128, 9 us.  With many rows the narrow slices cost more,
// as every slice's sums are written and read back: one layer's seven projections at
// 4096 rows 197 us of shrink against 145, and 43 us more in what adds the slices.
constexpr int kSgmmKSliceFew = 512;
constexpr int kSgmmFewItems = 256;
// Up to this rank the expand adds a tile's K-slice partials itself; above it a
// K-slice sum launch runs between the shrink and the expand.
constexpr int kSgmmFoldRank = 64;
SgLayout sgmm_layout(int64_t T, int64_t d_in_max, int E, int r, int n_prob);

// Rows per segmentation chunk (one workgroup of the segmentation kernels).
constexpr int kSgmmSegRows = 1024;
// Up to this many rows the segmentation is one launch (each workgroup counts
// every chunk's rows); above it a count launch runs first.
constexpr int kSgmmSegFewRows = 8192;

// Output columns one SGMM expand work item covers (4 waves x 4 x 64).
constexpr int kSgmmExpandCols = 1024;

// Single-problem calls with at most this many rows (bf16) take one launch:
// each column group computes the rank vectors itself instead of a
// segmentation, a shrink and a K-slice sum running first.
constexpr int kSgmmSmallT = 4;

// Up to this many rows (one wave's lanes) the shrink and expand workgroups
// order the rows themselves (the segmentation's order, computed by one wave),
// so there is no segmentation launch; batches that need the K-slice sum launch
// keep it.
constexpr int kSgmmInlineRows = 64;

// Header words of the workspace.
enum { SG_ERR = 0, SG_NPOS = 1, SG_NTILES = 2 };
// Words per XCD of the one-launch shrink + expand's work ranges.
constexpr int kSgmmXcdWords = 16;
// One-launch shrink + expand after the segmentation (bf16, ranks up to
// kSgmmFoldRank that are multiples of 8: the others' loads of B leave it no
// registers, 4096 rows of a layer's seven projections at rank 12 477 us against
// 421 in two launches): 0 off, 1 for segmented batches, 2 also for batches of up to
// kSgmmInlineRows rows (segmented first instead of ordered in the kernels).
#ifndef DLM_SGMM_FUSED
#define DLM_SGMM_FUSED 2
#endif
constexpr int kSgmmFused = DLM_SGMM_FUSED;
// Its counts hold K slices in 16 bits and K slices x (XCD id + 1) in 15: up to
// this many K slices per problem.
constexpr int kSgmmFusedMaxKs = 4095;
// It pays from this many (problem, tile) pairs on (32 per XCD); smaller batches,
// whose few items would mostly wait on each other, keep two launches.
constexpr int64_t kSgmmFusedMinPairs = 256;

struct SgmmArgs {
    const SgDesc* descs;    // device table, or nullptr to use `single`
    const SgDesc* ks_desc;  // the owning problem's descriptor per K slice (device; with descs)
    const SgDesc* cb_desc;  // the owning problem's descriptor per expand column group (device; with descs)
    SgDesc single;
    int32_t n_prob;
    int64_t n_expand_units;  // tiles_max * total_cb
    int64_t total_cb;        // sum over problems of their expand column groups
    int64_t total_ks;        // sum over problems of their shrink K slices
    int64_t d_out_max;       // largest d_out over the problems
    int32_t packed;          // 1: the shrink reads every problem's packed A (Ap)
    const int32_t* idx;
    const float* g;
    int64_t T;
    int32_t E, r;
    float scale;
    char* ws;
    SgLayout L;
    int32_t* status_out;   // device word that also receives the set-validity flag, or nullptr
    int32_t inline_seg;    // 1: the shrink and expand order the rows themselves (launch_sgmm sets it)
    int32_t w_max;         // largest K slices + column groups of one problem
    int32_t kslice;        // K slice width of the shrink (the owners' n_ks goes by it)
};

hipError_t launch_sgmm(const SgmmArgs& a, int dtype, hipStream_t s);
// Ap[e][k / 8][rho][0..8) = A[e][rho][k..k+8) for k = 0, 8, ..., d_in - 8 (bf16).
hipError_t launch_sgmm_pack_a(const void* A, void* Ap, int E, int r, int64_t d_in, hipStream_t s);

// The shrink of every problem of a segmented batch (bf16, ranks below kGradListRank).
hipError_t launch_sgmm_shrink(const SgmmArgs& a, hipStream_t s);
hipError_t launch_sgmm_vsum(const SgmmArgs& a, hipStream_t s);  // the K-slice sum alone
bool sgmm_launches_fit(const SgmmArgs& a, int dtype);

// ---- gradients ----------------------------------------------------------------

// From this rank on the gradients' shrink goes by the experts' slot lists, not by
// tiles of expert pairs: a tile's bank rows then serve 128 slots of one expert, not 32
// rows of two or more, and every row is read once per expert.  The shrink at rank 64,
// 4096 rows, 8192 columns on either side, 16 experts: 53 us against 113; at rank 128,
// 4096 columns, 8 experts: 47 against 82.  Whole calls at ranks 33, 40, 48, 56 and 64:
// those 16 experts' 206, 201, 205, 239, 244 us against 258, 250, 257, 299, 303; 4096
// rows of 4096 columns, 8 experts, 120, 120, 120, 139, 140 against 132, 132, 132, 146,
// 146; 512 rows and 32 experts, and 64 rows and 8, are 13 to 25% shorter too.  At rank
// 32 reading the rows twice no longer pays: the shrink of 4096 rows of 4096 columns 34
// us against 25.
constexpr int kGradListRank = 33;
// Slots of one list tile.
constexpr int kGradTile = 32;

// A run of one expert's list tiles: what one workgroup of the outer products sums.
struct SgChunk {
    int32_t e, t0, t1;  // tiles [t0, t1)
    int32_t part;       // its partial sums' place (expert-major), or -1: the expert's only chunk
};
// The experts' slot lists as the segmentation writes them: every expert's slots
// in sorted-position order, padded to whole tiles (a padding slot repeats a row
// of its expert), the lists one after another, and their chunks.
struct SgLists {
    int32_t* eoff;    // [E + 1] first list position
    int32_t* slot;    // 2 * position + k, or -1 (padding)
    int32_t* srow;    // the slot's row
    SgChunk* chunk;   // in the order they run
    int32_t* echunk;  // [E + 1] first chunk, expert-major
    int32_t chunk_tiles;  // most tiles of a chunk
};

// One projection and its gradients in the device table.
struct SgGrad {
    const void* A;   // [E][r][d_in]
    const void* B;   // [E][d_out][r]
    const void* x;   // [T][d_in]
    const void* dy;  // [T][d_out]
    void* Ap;        // A packed for the shrink (bf16), else unused
    // A transposed, the dx expand's up matrix: [E][rank chunk of 16][d_in][16], the
    // last chunk's padding ranks 0 (bf16), or [E][d_in][r] (fp32)
    void* At;
    void* Bt;        // B transposed: [E][d_out / 8][r][8] (bf16) or [E][r][d_out] (fp32)
    int32_t d_in, d_out;
    int64_t pk0;     // first group (bf16: 8 elements, fp32: one) of its banks (prefix sum)
    int64_t ks_u, ks_w;      // first K slice of u = A x and of w = B^T dy in the workspace's v
    int32_t n_ks_u, n_ks_w;  // and how many there are to add
};
// One side of a projection's bank gradients: dA from x, dB from dy.
struct SgOuter {
    const void* act;  // x [T][d] or dy [T][d]
    float* out;       // dA [E][r][d] or dB [E][d][r]
    int32_t d;
    int32_t side;     // 0: dA, 1: dB
    int32_t prob;
    int32_t unit0;    // first column block (prefix sum)
};
// Columns of one column block of the outer products.
int grad_cols(int dtype);

// Workspace of a backward call.
struct SgGradLayout {
    SgLayout L;     // a segmented SGMM's, its v for every K slice of both sides
    size_t eoff, slot, srow, chunk, echunk;  // the lists (SgLists)
    // coefficients: bf16 [prob][side][list tile][rank block][3 terms][16 ranks][kGradTile],
    // fp32 [prob][side][list tile][r_pad][kGradTile]
    size_t coef;
    size_t part;    // bf16: partial sums of experts with several chunks, [unit][rank chunk][chunk][ranks][columns] (dB: [columns][ranks])
    size_t dgp;     // [prob][T][2] fp32
    size_t total;
    int64_t cap;    // list positions at most
    int chunk_tiles, max_chunks;
};
SgGradLayout sgmm_grad_layout(int64_t T, int64_t total_ks, int E, int r, int n_prob, int n_units, int dtype);

struct SgGradArgs {
    const SgGrad* probs;
    const SgOuter* outers;       // 2 * n_prob
    const int32_t* unit_outer;   // the owning entry of every column block
    const SgDesc* ks_desc;       // the shrink problem (x, A or dy, B^T) of every K slice
    int64_t total_ks;
    int32_t kslice;
    int32_t n_prob, n_units;
    int64_t pk_total;
    const int32_t* idx;
    int64_t T;
    int32_t E, r;
    float scale;
    char* ws;
    SgGradLayout G;
    float* dg;           // [T][2] or nullptr
    int32_t accumulate;  // add to dA and dB instead of writing them
};
// T = 0: the gradients of no rows.
hipError_t launch_grad_zero(const SgGradArgs& a, int dtype, hipStream_t s);
// Segmentation, lists and the banks' transposes.
bool grad_prep_fits(const SgGradArgs& a);
hipError_t launch_grad_prep(const SgGradArgs& a, const float* g, int dtype, hipStream_t s);
// u and w over the experts' slot lists (bf16).
hipError_t launch_grad_shrink(const SgGradArgs& a, hipStream_t s);
hipError_t launch_grad_shrink_f32(const SgGradArgs& a, hipStream_t s);
// The expand of a set of problems whose v (ks0, n_ks) the shrink has left in the
// workspace and whose B is packed as SgGrad::At, with the coefficients of all
// projections in the same launch if asked.
bool grad_expand_fits(const SgGradArgs& b, const SgmmArgs& a, int dtype);
hipError_t launch_grad_expand(const SgGradArgs& b, const SgmmArgs& a, bool coefs, int dtype, hipStream_t s);
// The coefficients alone.
hipError_t launch_grad_coefs(const SgGradArgs& a, int dtype, hipStream_t s);
// dA, dB and dg.
hipError_t launch_grad_outer(const SgGradArgs& a, int dtype, hipStream_t s);
bool sgmm_grad_fits(const SgGradArgs& a, int dtype);

}  // namespace dlm
