// Gradients of the SGMM y[t] += sum_k s g_k B_{e_k} (A_{e_k} x[t]).  With
// u = A_e x and w = B_e^T dy per row and slot:
//   dx[t] += sum_k s g_k A_{e_k}^T w        dg[t][k] = s u . w
//   dA_e   = sum s g w x[t]^T               dB_e     = sum s g dy[t] u^T
// (sums over the slots (t, k) that chose e).
//
// dx is itself an SGMM, of dy through the banks' transposes.  Launches:
//   prep   (in sgmm.hip) the segmentation; every expert's slot list, whose
//          places follow from the segmentation's counts; and in the other
//          workgroups the banks' transposes (and A as the shrink reads it),
//          every call: the banks change with every training step.
//   shrink u and w of all projections, (x, A) and (dy, B^T) together: the SGMM's
//          own shrink up to rank 32, above it one over the slot lists.
//   expand (in sgmm.hip) two things that need u and w and not each other:
//          - w through A^T into dx, the SGMM's expand;
//          - the coefficients, per (32-slot tile, projection): u and w (their K
//            slices added in order), s u . w for dg, and s g w and s g u, each
//            as three bf16 terms (8 + 8 + 8 bits: fp32 whole), transposed so that
//            eight slots of one rank are one 16-byte operand.  With two terms the
//            gradients lose a factor of three to fp32 sums; the third costs matrix
//            instructions where memory is the bound.
//          As a launch of their own the coefficients took 8 us of latency more.
//          Problems that share a dx add to it in launches one after another.
//   outer  dA and dB: per (projection, side, 512-column block, chunk of an
//          expert's list) a product with M = ranks (64 at most), N = columns and
//          K = slots, bf16 MFMA 16x16x32 with fp32 sums.  The four waves take 128
//          columns each and share a tile's coefficients through LDS (global to
//          LDS directly, two tiles in turn): read by every wave on its own they
//          were as much L2 traffic as the rows at rank 64 (134 us against 77 for
//          4096 rows of 8192 columns on either side, 16 experts).  A lane reads
//          eight columns of eight rows and transposes the block in registers, one
//          v_perm per two values: x and dy go from memory to the matrix cores
//          without LDS.
//          Its last workgroups write dg.
//   sum    experts with several chunks: their partial sums in chunk order.
//
// Measured (us)                            prep  shrink  expand  outer  sum
//   256 rows, 4096 x 4096, 8 x rank 16        9       9       9      9    -   latency
//   4096 rows, a 7B-shaped layer, 8 x 16     20     138     142    188   22
//   4096 rows, 8192 x 8192, 16 x rank 64     26      53      79     83   11
// The layer's shrink reads x and dy at 4.6 TB/s, its expand reads and writes dx at
// 4.1 and its outer products read x and dy once per expert, 1.26 GB at 6.7 TB/s, of
// which the L2s find almost nothing: a row's two experts come to it at different
// times.  At rank 64 the bank rows' and coefficients' traffic through L2 and LDS
// weighs as much as the memory's.
// Every gradient element has one owner per launch: no atomics, bitwise
// reproducible.
//
// Chunks.  Routing is skewed (Zipf 1.1 over 8 experts: the first is in 60% of the
// rows), and one workgroup per (block, expert) would wait for the longest list.
// An expert's list is cut into chunks of at most chunk_tiles tiles, chosen so
// that a call has about kTargetItems of them, several rounds of what the chip
// holds, but none so short that its partial sums (4 bytes a rank, column and
// chunk, written and read back) outweigh the 2 bytes a slot and column that it reads.
// A row is read once for each of its experts.  (Reading it once, with the sums of
// all 8 experts of rank 16 in a workgroup's registers, was tried: half the bytes
// at a third of the bytes in flight, 235 us against 190 for a layer's seven
// projections at 4096 rows.)
#include <algorithm>

#include "gfx950.hpp"
#include "internal.hpp"
#include "sgmm.hpp"
#include "sgmm_coefs.hpp"

namespace dlm {

namespace {

size_t a256(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int kTargetItems = 1536;

constexpr int kCPL = 8;                // columns per lane of the outer products
constexpr int kOuterCols = 64 * kCPL;  // per workgroup
constexpr int kSumPer = 4;             // gradient quads per thread of the sum

int rank_chunks(const SgLayout& L) { return (L.r_pad + 63) / 64; }
int outer_r16(const SgLayout& L) { return L.r_pad <= 64 ? L.r_pad / 16 : 4; }

}  // namespace

int grad_cols(int dtype) { return dtype == 1 ? kOuterCols : 64; }

SgGradLayout sgmm_grad_layout(int64_t T, int64_t total_ks, int E, int r, int n_prob, int n_units, int dtype) {
    SgGradLayout G;
    G.L = sgmm_layout(T, 1, E, r, (int)total_ks);  // one slice each of total_ks problems
    G.cap = (2 * T + (int64_t)E * (kGradTile - 1) + kGradTile - 1) / kGradTile * kGradTile;
    const int64_t tiles = G.cap / kGradTile, units = (int64_t)n_units * rank_chunks(G.L);
    const int64_t least = 8 * outer_r16(G.L), even = std::min((units * tiles + kTargetItems - 1) / kTargetItems, tiles);
    G.chunk_tiles = (int)(even > least ? even : least);
    // full chunks (by bounds that do not fall as T grows) and one more per expert
    const int64_t by_tiles = tiles / least, by_items = kTargetItems / units;
    G.max_chunks = (int)(by_tiles < by_items ? by_tiles : by_items) + E;
    // few rows, whose longest list makes two short chunks at most: one chunk an
    // expert, and no launch to add them (256 rows of 4096 x 4096: 39.7 us to 37.3)
    const int64_t longest = (2 * T + kGradTile - 1) / kGradTile;
    if (longest <= 2 * least) {
        G.chunk_tiles = (int)std::max<int64_t>(longest, least);
        G.max_chunks = E;
    }
    size_t o = G.L.total;
    G.eoff = o;    o += a256((size_t)(E + 1) * 4);
    G.slot = o;    o += a256((size_t)G.cap * 4);
    G.srow = o;    o += a256((size_t)G.cap * 4);
    G.chunk = o;   o += a256((size_t)(tiles / least + 2 * E + 2) * sizeof(SgChunk));
    G.echunk = o;  o += a256((size_t)(E + 1) * 4);
    G.coef = o;
    if (dtype == 0) o += a256((size_t)n_prob * 2 * G.cap * G.L.r_pad * 4);
    else o += (size_t)n_prob * 2 * tiles * (G.L.r_pad / 16) * kCoefTerms * kKB * 2;
    G.part = o;
    if (dtype == 1) o += (size_t)units * G.max_chunks * (16 * outer_r16(G.L)) * kOuterCols * 4;
    G.dgp = o;     o += a256((size_t)n_prob * T * 8);
    G.total = o;
    return G;
}

namespace {

// ---- u, w over the lists (bf16) -----------------------------------------------------

// D = A(16x32) B(32x16) + C: lane l supplies row (l % 16) of A and column
// (l % 16) of B, k = 8 (l / 16) + [0, 8); register i holds D[4 (l / 16) + i][l % 16].
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// One work item = (K slice, rank chunk, kListSlots slots of one expert's list): a
// product with M = ranks, N = slots, K = columns.  The waves take 32 slots each and
// share the bank's rows.  Both come through LDS, copied directly, two steps in turn:
// a lane that loads its operand's 16 bytes of a row by itself makes one cache access
// of them, and those accesses were the bound.
constexpr int kListSlots = 128;
constexpr int kListK = 64;  // columns per step

template <int R16>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3)))
void grad_shrink_list(SgGradArgs a, int n_ch) {
    constexpr int NR = 16 * R16;
    const SgLayout& L = a.G.L;
    if (rejected(a)) return;
    const int lane = lane_id(), w = wave_id(), n = lane & 15, kg = lane >> 4, r = a.r, E = a.E;
    // the experts' groups of kListSlots slots: lane e holds expert e's
    const int32_t* eoff = (const int32_t*)(a.ws + a.G.eoff);
    const int e_l = lane < E ? lane : E - 1;
    const int my0 = gld(eoff + e_l), my1 = gld(eoff + e_l + 1);
    const int ng = lane < E ? (my1 - my0 + kListSlots - 1) / kListSlots : 0;
    int incl = ng;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up(incl, o, kWave);
        if (lane >= o) incl += y;
    }
    const int n_groups = __shfl(incl, E - 1, kWave);
    // XCD b % 8 takes a contiguous share, the groups of one slice next to each other
    const int64_t n_live = a.total_ks * n_ch * n_groups, per = (n_live + 7) / 8;
    const int64_t j = blockIdx.x >> 3, item = (int64_t)(blockIdx.x & 7) * per + j;
    if (j >= per || item >= n_live) return;
    const int group = uniform((int)(item % n_groups));
    const int ch = uniform((int)(item / n_groups % n_ch));
    const int64_t gks = item / n_groups / n_ch;
    const int e = __popcll(__ballot(lane < E && incl <= group));
    const int p0 = uniform(__shfl(my0, e, kWave) + (group - __shfl(incl - ng, e, kWave)) * kListSlots + 32 * w);
    const int p1 = uniform(__shfl(my1, e, kWave));
    const bool mine = p0 < p1;  // (else this wave only helps with the bank)

    const SgDesc D = a.ks_desc[gks];
    const int d = uniform(D.d_in), nq = d / 8, k0 = (int)(gks - D.ks0) * a.kslice;
    const int n_steps = ((d - k0 < a.kslice ? d - k0 : a.kslice) + kListK - 1) / kListK;
    const uint16_t* bank = (const uint16_t*)D.Ap + (int64_t)e * nq * r * 8;
    int entry[2];  // of the slots whose sums this lane holds
    const uint16_t* row[4];  // of the slots whose rows it copies
    const int32_t* srow = (const int32_t*)(a.ws + a.G.srow);
    auto place = [&](int i) { return mine ? (p0 + i < p1 ? p0 + i : p1 - 1) : 0; };
#pragma unroll
    for (int m = 0; m < 2; ++m)
        entry[m] = mine && p0 + 16 * m + n < p1 ? gld((const int32_t*)(a.ws + a.G.slot) + place(16 * m + n)) : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = (const uint16_t*)D.x + (int64_t)gld(srow + place(8 * i + lane / 8)) * d;
    __shared__ __attribute__((aligned(16))) uint16_t s_a[2][kListK / 8][NR][8];
    // 16-byte piece c of slot n is at piece c ^ (n & 7): the reads of a piece of
    // eight slots fall on different banks
    __shared__ __attribute__((aligned(16))) uint16_t s_x[2][4][32][kListK];
    const int xc = 8 * ((lane % 8) ^ (lane / 8));  // the column of a step that this lane copies
    auto copy = [&](int s) {
        const int kb = k0 + s * kListK;
        if (mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i) copy16_to_lds(row[i] + (kb + xc < d ? kb + xc : 0), s_x[s & 1][w][8 * i]);
        }
        // the bank's packed rows: 16-byte pieces (k group, rank); ranks and groups
        // past the end repeat the last
#pragma unroll
        for (int i = 0; i < (2 * R16 + 3) / 4; ++i) {
            const int c = w + 4 * i, piece = c * kWave + lane, kq = kb / 8 + piece / NR, rho = 64 * ch + piece % NR;
            if (c < 2 * R16)
                copy16_to_lds(bank + ((int64_t)(kq < nq ? kq : nq - 1) * r + (rho < r ? rho : r - 1)) * 8,
                              &s_a[s & 1][0][0][0] + c * kWave * 8);
        }
    };
    f32x4 acc[R16][2];
#pragma unroll
    for (int b = 0; b < R16; ++b) acc[b][0] = acc[b][1] = f32x4{};
    copy(0);
#pragma unroll 1
    for (int s = 0; s < n_steps; ++s) {
        // this step's rows and bank have landed, in every wave, and every wave is
        // done with the step before, whose half of the buffers is free again
        wait_vmcnt<0>();
        __syncthreads();
        if (s + 1 < n_steps) copy(s + 1);
        if (!mine) continue;
        const int kb = k0 + s * kListK;
        const bool full = kb + kListK <= d;
#pragma unroll
        for (int i = 0; i < kListK / 32; ++i) {
            const bool in = full || kb + 32 * i + 8 * kg < d;
            u32x4 x[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                x[m] = *(const u32x4*)&s_x[s & 1][w][16 * m + n][8 * ((4 * i + kg) ^ (n & 7))];
                if (!in) x[m] = u32x4{};
            }
#pragma unroll
            for (int b = 0; b < R16; ++b) {
                u32x4 h = *(const u32x4*)s_a[s & 1][4 * i + kg][16 * b + n];
                if (!in) h = u32x4{};  // the repeated group may hold an infinity
#pragma unroll
                for (int m = 0; m < 2; ++m) acc[b][m] = mfma16(h, x[m], acc[b][m]);
            }
        }
    }
    if (!mine) return;
    // register i of block b: rank 16 b + 4 kg + i of slot n (ranks r .. r_pad - 1 are not read)
    float* v = (float*)(a.ws + L.v) + gks * L.T_pad * 2 * L.r_pad + 64 * ch + 4 * kg;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if (entry[m] < 0) continue;
#pragma unroll
        for (int b = 0; b < R16; ++b)
            if (64 * ch + 16 * b < L.r_pad) gst((f32x4*)(v + (int64_t)entry[m] * L.r_pad + 16 * b), acc[b][m]);
    }
}

// ---- u, w in fp32 -------------------------------------------------------------------

// One wave per (projection side, position, slot): eight ranks' products at a
// time over the row, lanes along it, then a butterfly sum.
__global__ __launch_bounds__(256) void grad_shrink_f32(SgGradArgs a) {
    const SgLayout& L = a.G.L;
    if (rejected(a)) return;
    const int64_t q = (int64_t)blockIdx.x * 4 + wave_id();  // 2 * position + k
    if (q >= 2 * (int64_t)gld((const int32_t*)(a.ws + L.hdr) + SG_NPOS)) return;
    const uint32_t ep = gld((const uint32_t*)(a.ws + L.epk) + q / 2);
    const int e = uniform((q & 1) ? (int16_t)(ep >> 16) : (int16_t)(ep & 0xffffu));
    if (e < 0) return;
    const int64_t row = uniform(gld((const int32_t*)(a.ws + L.perm) + q / 2));
    const int side = blockIdx.y & 1, lane = lane_id(), r = a.r;
    const SgGrad P = a.probs[blockIdx.y / 2];
    const int d = side ? P.d_out : P.d_in;
    const float* act = (const float*)(side ? P.dy : P.x) + row * d;
    const float* bank = (const float*)(side ? P.Bt : P.A) + (int64_t)e * r * d;
    float* v = (float*)(a.ws + L.v) + (side ? P.ks_w : P.ks_u) * L.T_pad * 2 * L.r_pad + q * L.r_pad;
    for (int r0 = 0; r0 < r; r0 += 8) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int j = lane; j < d; j += kWave) {
            const float x = gld(act + j);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int rho = r0 + i < r ? r0 + i : r - 1;
                acc[i] = fmaf(x, gld(bank + (int64_t)rho * d + j), acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s = acc[i];
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, kWave);
            if (lane == i && r0 + i < r) gst(v + r0 + i, s);
        }
    }
}

template <bool BF>
__global__ __launch_bounds__(256) void grad_coefs(SgGradArgs a) {
    if (rejected(a)) return;
    __shared__ CoefLds<BF> sm;
    coefs_tile<BF>(a, blockIdx.x, blockIdx.y, sm);
}

// dg[t][k] = the projections' parts, added in order; 0 for an empty slot.
__device__ __forceinline__ void write_dg(const SgGradArgs& a, int64_t i) {
    if (i >= 2 * a.T) return;
    const float* p = (const float*)(a.ws + a.G.dgp) + i;
    float v = 0.f;
    if (gld(a.idx + i) >= 0)
        for (int k = 0; k < a.n_prob; ++k) v += gld(p + (int64_t)k * 2 * a.T);
    gst(a.dg + i, v);
}

// ---- dA, dB -------------------------------------------------------------------------

// Stores (or adds) columns 4h .. 4h + 3 of a lane's eight, rank block b: acc[j]
// holds four ranks of column 4h + j.
__device__ __forceinline__ void store_quad(const SgGradArgs& a, const SgOuter& O, int e, int r0, int col, int kg, int b,
                                           const f32x4 (&acc)[4]) {
    const int r = a.r, d = O.d, rho = r0 + 16 * b + 4 * kg;  // this lane's four ranks
    if (col >= d) return;
    if (O.side == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (rho + i >= r) continue;
            f32x4* p = (f32x4*)(O.out + ((int64_t)e * r + rho + i) * d + col);
            f32x4 o = {acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
            if (a.accumulate) o += gld(p);
            gst(p, o);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float* p = O.out + ((int64_t)e * d + col + j) * r + rho;
            if ((r & 3) == 0) {
                if (rho >= r) continue;
                f32x4 o = acc[j];
                if (a.accumulate) o += gld((const f32x4*)p);
                gst((f32x4*)p, o);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (rho + i < r) gst(p + i, a.accumulate ? gld(p + i) + acc[j][i] : acc[j][i]);
            }
        }
    }
}

// The same into a partial tile of NR ranks and NC columns: [rank][column] for
// dA, [column][rank] for dB (lc: the quad's first column in the tile).
__device__ __forceinline__ void store_part(float* part, int side, int NR, int NC, int lc, int rho, const f32x4 (&acc)[4]) {
    if (side == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            gst((f32x4*)(part + (int64_t)(rho + i) * NC + lc), f32x4{acc[0][i], acc[1][i], acc[2][i], acc[3][i]});
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) gst((f32x4*)(part + (int64_t)(lc + j) * NR + rho), acc[j]);
    }
}

// Column j of the 8x8 block whose row i is v[i]: one v_perm per two values.
__device__ __forceinline__ u32x4 column(const u32x4 (&v)[8], int j) {
    u32x4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        o[q] = __builtin_amdgcn_perm(v[2 * q + 1][j / 2], v[2 * q][j / 2], (j & 1) ? 0x07060302u : 0x05040100u);
    return o;
}

template <int R16>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(R16 == 1 ? 3 : 2)))
void grad_outer_bf16(SgGradArgs a, int n_ch, int64_t n_blocks) {
    constexpr int CPL = kCPL, kCols = kOuterCols, NR = 16 * R16;
    if (rejected(a)) return;
    if (blockIdx.x >= n_blocks) {
        write_dg(a, (blockIdx.x - n_blocks) * 256 + threadIdx.x);
        return;
    }
    // XCD b % 8 takes every eighth column block, its chunks (and rank chunks) one after another
    const int per_unit = a.G.max_chunks * n_ch;
    const int64_t jj = blockIdx.x / 8;
    const int64_t unit = jj / per_unit * 8 + blockIdx.x % 8;
    if (unit >= a.n_units) return;
    const int sub = (int)(jj % per_unit), c = sub % a.G.max_chunks, ch = sub / a.G.max_chunks;
    if (c >= gld((const int32_t*)(a.ws + a.G.echunk) + a.E)) return;
    const SgChunk K = ((const SgChunk*)(a.ws + a.G.chunk))[c];
    const SgOuter O = a.outers[a.unit_outer[unit]];
    const int32_t* srow = (const int32_t*)(a.ws + a.G.srow);
    const int lane = lane_id(), w = wave_id(), n = lane & 15, kg = lane >> 4;
    const int d = uniform(O.d), t0 = uniform(K.t0), t1 = uniform(K.t1);
    const int lc = w * 16 * CPL + CPL * n, col = (int)(unit - O.unit0) * kCols + lc;
    const int lcol = col < d ? col : 0;          // columns past the end read the first ones and are not stored
    const bool mine = col - CPL * n < d;         // this wave has columns (else it only helps with the coefficients)
    const uint16_t* __restrict__ act = (const uint16_t*)O.act + lcol;
    const int nb = a.G.L.r_pad / 16, b0 = ch * 4, my_b = nb - b0 < R16 ? nb - b0 : R16;
    const uint16_t* __restrict__ coef = (const uint16_t*)(a.ws + a.G.coef) +
                                        ((int64_t)O.prob * 2 + O.side) * (a.G.cap / kGradTile) * nb * kCoefTerms * kKB;

    __shared__ __attribute__((aligned(16))) uint16_t s_c[2][R16 * kCoefTerms * kKB];
    f32x4 acc[R16][CPL];
#pragma unroll
    for (int b = 0; b < R16; ++b)
#pragma unroll
        for (int j = 0; j < CPL; ++j) acc[b][j] = f32x4{};
    u32x4 v[8];
    int rows[8];
    auto load_rows = [&](int t) {
        const u32x4 a0 = ld128(srow + t * kGradTile + 8 * kg), a1 = ld128(srow + t * kGradTile + 8 * kg + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rows[i] = (int)a0[i];
            rows[4 + i] = (int)a1[i];
        }
    };
    auto load_x = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = ld128(act + (int64_t)rows[i] * d);
    };
    auto copy_coefs = [&](int t) {
        const uint16_t* src = coef + ((int64_t)t * nb + b0) * kCoefTerms * kKB + 8 * lane;
#pragma unroll
        for (int i = 0; i < (R16 * kCoefTerms + 3) / 4; ++i) {
            const int k = w + 4 * i;
            if (k < my_b * kCoefTerms) copy16_to_lds(src + k * kKB, s_c[t & 1] + k * kKB);
        }
    };
    if (t0 < t1) {
        load_rows(t0);
        copy_coefs(t0);
        if (mine) load_x();
        if (t0 + 1 < t1) load_rows(t0 + 1);
    }
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
        // everything loaded for this tile has landed, in every wave, and every
        // wave is done with the tile before, whose half of s_c is free again
        wait_vmcnt<0>();
        __syncthreads();
        u32x4 x[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) x[j] = column(v, j);
        if (t + 1 < t1) {
            copy_coefs(t + 1);
            if (mine) load_x();
            if (t + 2 < t1) load_rows(t + 2);
        }
        if (mine) {
            const uint16_t* s = s_c[t & 1] + n * kGradTile + 8 * kg;
#pragma unroll
            for (int b = 0; b < R16; ++b) {
                if (R16 == 4 && b >= my_b) break;  // the last rank chunk may have fewer blocks
#pragma unroll
                for (int m = 0; m < kCoefTerms; ++m) {
                    const u32x4 h = *(const u32x4*)(s + (b * kCoefTerms + m) * kKB);
#pragma unroll
                    for (int j = 0; j < CPL; ++j) acc[b][j] = mfma16(h, x[j], acc[b][j]);
                }
            }
        }
    }
    if (!mine) return;
    float* part = (float*)(a.ws + a.G.part) + ((unit * n_ch + ch) * a.G.max_chunks + (K.part < 0 ? 0 : K.part)) * (int64_t)(NR * kCols);
#pragma unroll
    for (int b = 0; b < R16; ++b)
#pragma unroll
        for (int h = 0; h < CPL / 4; ++h) {
            const f32x4 q[4] = {acc[b][4 * h], acc[b][4 * h + 1], acc[b][4 * h + 2], acc[b][4 * h + 3]};
            if (K.part < 0) store_quad(a, O, K.e, ch * 64, col + 4 * h, kg, b, q);
            else store_part(part, O.side, NR, kCols, lc + 4 * h, 16 * b + 4 * kg, q);
        }
}

// ---- partial sums

// Four gradient elements (a quad) at a time of (unit, rank chunk, expert): the
// expert's partial tiles added in chunk order, kSumPer quads per thread, whose
// loads go out together.
__global__ __launch_bounds__(256) void grad_sum_bf16(SgGradArgs a, int n_ch, int per_item) {
    if (rejected(a)) return;
    const int64_t item = blockIdx.x / per_item;
    const int e = (int)(item % a.E), ch = (int)(item / a.E) % n_ch;
    const int64_t unit = item / a.E / n_ch;
    const int32_t* echunk = (const int32_t*)(a.ws + a.G.echunk);
    const int c0 = uniform(gld(echunk + e)), nc = uniform(gld(echunk + e + 1)) - c0;
    if (nc < 2) return;
    constexpr int cols = kOuterCols;
    const int r = a.r, nb = a.G.L.r_pad / 16, NR = 16 * (nb < 4 ? nb : 4);  // ranks of a partial tile
    const SgOuter O = a.outers[a.unit_outer[unit]];
    const int64_t step = (int64_t)NR * cols;
    const float* p = (const float*)(a.ws + a.G.part) + ((unit * n_ch + ch) * a.G.max_chunks + c0) * step;
    const int u0 = (int)(unit - O.unit0) * cols;  // the tile's first column
    f32x4 acc[kSumPer];
    int i[kSumPer];
#pragma unroll
    for (int q = 0; q < kSumPer; ++q) {
        i[q] = ((int)(blockIdx.x % per_item) * kSumPer + q) * 256 + threadIdx.x;
        if (i[q] >= NR * cols / 4) i[q] = -1;
        acc[q] = gld((const f32x4*)p + (i[q] < 0 ? 0 : i[q]));
    }
    for (int c = 1; c < nc; c += 2) {
        f32x4 y[kSumPer], z[kSumPer];
#pragma unroll
        for (int q = 0; q < kSumPer; ++q) {
            const int at = i[q] < 0 ? 0 : i[q];
            y[q] = gld((const f32x4*)(p + c * step) + at);
            z[q] = gld((const f32x4*)(p + (c + 1 < nc ? c + 1 : c) * step) + at);
        }
#pragma unroll
        for (int q = 0; q < kSumPer; ++q) {
            acc[q] += y[q];
            if (c + 1 < nc) acc[q] += z[q];
        }
    }
#pragma unroll
    for (int q = 0; q < kSumPer; ++q) {
        // the quad's place: four columns of a rank (dA), four ranks of a column (dB)
        const int rho = 64 * ch + (O.side == 0 ? i[q] / (cols / 4) : 4 * (i[q] % (NR / 4)));
        const int col = u0 + (O.side == 0 ? 4 * (i[q] % (cols / 4)) : i[q] / (NR / 4));
        if (i[q] < 0 || rho >= r || col >= O.d) continue;
        if (O.side == 0) {
            f32x4* o = (f32x4*)(O.out + ((int64_t)e * r + rho) * O.d + col);
            if (a.accumulate) acc[q] += gld(o);
            gst(o, acc[q]);
        } else {
            float* o = O.out + ((int64_t)e * O.d + col) * r + rho;
            if ((r & 3) == 0) {
                if (a.accumulate) acc[q] += gld((const f32x4*)o);
                gst((f32x4*)o, acc[q]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (rho + k < r) gst(o + k, a.accumulate ? gld(o + k) + acc[q][k] : acc[q][k]);
            }
        }
    }
}

// fp32: 64 columns per workgroup and eight ranks (blockIdx.z), the four waves
// taking every fourth list tile; the coefficients of a wave's slots are the
// same for its lanes.  The last grid row writes dg.
__global__ __launch_bounds__(256) void grad_outer_f32(SgGradArgs a, int n_units) {
    if (rejected(a)) return;
    if ((int)blockIdx.x >= n_units) {
        if (blockIdx.y == 0 && blockIdx.z == 0) write_dg(a, (int64_t)(blockIdx.x - n_units) * 256 + threadIdx.x);
        return;
    }
    const int unit = blockIdx.x, e = blockIdx.y, r0 = 8 * blockIdx.z, r = a.r, RPAD = a.G.L.r_pad;
    const SgOuter O = a.outers[a.unit_outer[unit]];
    const int lane = lane_id(), w = wave_id();
    const int col = (unit - O.unit0) * 64 + lane, lcol = col < O.d ? col : 0;
    const int32_t* eoff = (const int32_t*)(a.ws + a.G.eoff);
    const int32_t* srow = (const int32_t*)(a.ws + a.G.srow);
    const float* __restrict__ coef = (const float*)(a.ws + a.G.coef) + ((int64_t)O.prob * 2 + O.side) * a.G.cap * RPAD;
    const float* __restrict__ act = (const float*)O.act + lcol;
    const int t0 = uniform(gld(eoff + e)) / kGradTile, t1 = uniform(gld(eoff + e + 1)) / kGradTile;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int t = t0 + w; t < t1; t += 4) {
        const float* ct = coef + ((int64_t)t * RPAD + r0) * kGradTile;
#pragma unroll 1
        for (int s = 0; s < kGradTile; s += 8) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = gld(act + (int64_t)uniform(gld(srow + t * kGradTile + s + i)) * O.d);
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[k] = fmaf(ct[k * kGradTile + s + i], x[i], acc[k]);
        }
    }
    __shared__ float s_red[4][8][kWave];
#pragma unroll
    for (int k = 0; k < 8; ++k) s_red[w][k][lane] = acc[k];
    __syncthreads();
    // wave w sums and stores ranks w and w + 4
    if (col >= O.d) return;
    for (int k = w; k < 8; k += 4) {
        if (r0 + k >= r) break;
        const float v = (s_red[0][k][lane] + s_red[1][k][lane]) + (s_red[2][k][lane] + s_red[3][k][lane]);
        float* p = O.side == 0 ? O.out + ((int64_t)e * r + r0 + k) * O.d + col : O.out + ((int64_t)e * O.d + col) * r + r0 + k;
        gst(p, a.accumulate ? gld(p) + v : v);
    }
}

__global__ __launch_bounds__(kWave) void grad_zero(SgGradArgs a, int cols) {
    const int unit = blockIdx.x, e = blockIdx.y;
    const SgOuter O = a.outers[a.unit_outer[unit]];
    for (int c = threadIdx.x; c < cols; c += kWave) {
        const int col = (unit - O.unit0) * cols + c;
        if (col >= O.d) return;
        for (int rho = 0; rho < a.r; ++rho)
            gst(O.side == 0 ? O.out + ((int64_t)e * a.r + rho) * O.d + col : O.out + ((int64_t)e * O.d + col) * a.r + rho, 0.f);
    }
}

// Work items of grad_shrink_list at most, a multiple of 8.
int64_t list_blocks(const SgGradArgs& a) {
    const int64_t items = a.total_ks * rank_chunks(a.G.L) * (a.G.cap / kListSlots + a.E);
    return (items + 7) / 8 * 8;
}
int64_t dg_blocks(const SgGradArgs& a) { return a.dg ? (2 * a.T + 255) / 256 : 0; }
int64_t outer_blocks(const SgGradArgs& a) {
    return 8ll * a.G.max_chunks * rank_chunks(a.G.L) * ((a.n_units + 7) / 8);
}
// Items of the sum (none where no expert can have a second chunk) and workgroups per item.
int64_t sum_items(const SgGradArgs& a) {
    if (a.G.max_chunks <= a.E) return 0;
    return (int64_t)a.n_units * rank_chunks(a.G.L) * a.E;
}
int sum_blocks(const SgGradArgs& a) { return (16 * outer_r16(a.G.L) * kOuterCols / 4 + 256 * kSumPer - 1) / (256 * kSumPer); }

}  // namespace

bool sgmm_grad_fits(const SgGradArgs& a, int dtype) {
    return grad_prep_fits(a) && grid_fits(a.G.cap / kGradTile, 256) && grid_fits((a.T + 1) / 2, 256) &&
           grid_fits(a.n_units + dg_blocks(a), 256) &&
           (dtype == 0 || (grid_fits(list_blocks(a), 256) && grid_fits(outer_blocks(a) + dg_blocks(a), 256) &&
                           grid_fits(sum_items(a) * sum_blocks(a), 256)));
}

hipError_t launch_grad_zero(const SgGradArgs& a, int dtype, hipStream_t s) {
    hipLaunchKernelGGL(grad_zero, dim3((unsigned)a.n_units, (unsigned)a.E), dim3(kWave), 0, s, a,
                       grad_cols(dtype));
    return hipGetLastError();
}

hipError_t launch_grad_shrink(const SgGradArgs& a, hipStream_t s) {
    const int n_ch = rank_chunks(a.G.L);
    const dim3 g((unsigned)list_blocks(a));
    static_assert(kGradListRank > 32, "ranks padded to 48 at least");
    if (outer_r16(a.G.L) == 3) hipLaunchKernelGGL(grad_shrink_list<3>, g, dim3(256), 0, s, a, n_ch);
    else hipLaunchKernelGGL(grad_shrink_list<4>, g, dim3(256), 0, s, a, n_ch);
    return hipGetLastError();
}

hipError_t launch_grad_shrink_f32(const SgGradArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(grad_shrink_f32, dim3((unsigned)((a.T + 1) / 2), (unsigned)(2 * a.n_prob)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_coefs(const SgGradArgs& a, int dtype, hipStream_t s) {
    const dim3 g((unsigned)(a.G.cap / kGradTile), (unsigned)a.n_prob);
    if (dtype == 1) hipLaunchKernelGGL(grad_coefs<true>, g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(grad_coefs<false>, g, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_outer(const SgGradArgs& a, int dtype, hipStream_t s) {
    if (dtype == 0) {
        hipLaunchKernelGGL(grad_outer_f32, dim3((unsigned)(a.n_units + dg_blocks(a)), (unsigned)a.E, (unsigned)((a.r + 7) / 8)),
                           dim3(256), 0, s, a, a.n_units);
        return hipGetLastError();
    }
    const int n_ch = rank_chunks(a.G.L);
    const int64_t n = outer_blocks(a);
    const dim3 g((unsigned)(n + dg_blocks(a)));
    switch (outer_r16(a.G.L)) {
        case 1: hipLaunchKernelGGL(grad_outer_bf16<1>, g, dim3(256), 0, s, a, n_ch, n); break;
        case 2: hipLaunchKernelGGL(grad_outer_bf16<2>, g, dim3(256), 0, s, a, n_ch, n); break;
        case 3: hipLaunchKernelGGL(grad_outer_bf16<3>, g, dim3(256), 0, s, a, n_ch, n); break;
        default: hipLaunchKernelGGL(grad_outer_bf16<4>, g, dim3(256), 0, s, a, n_ch, n); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks = sum_items(a) * sum_blocks(a);
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(grad_sum_bf16, dim3((unsigned)blocks), dim3(256), 0, s, a, n_ch, sum_blocks(a));
    return hipGetLastError();
}

}  // namespace dlm
