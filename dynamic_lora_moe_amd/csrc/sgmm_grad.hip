// Gradients of the SGMM y[t] += sum_k s g_k B_{e_k} (A_{e_k} x[t]).  With
// u = A_e x and w = B_e^T dy per row and slot:
//   dx[t] += sum_k s g_k A_{e_k}^T w        dg[t][k] = s u . w
//   dA_e   = sum s g w x[t]^T               dB_e     = sum s g dy[t] u^T
// (sums over the slots (t, k) that chose e).
//
// dx is itself an SGMM, of dy through the banks' transposes, so it runs the
// SGMM's own kernels: one shrink launch over the projections' (x, A) and
// (dy, B^T) together, which leaves u and w in the workspace, and the expand of w
// through A^T into dx.  Launches:
//   prep   (in sgmm.hip) the segmentation; every expert's slot list, whose
//          places follow from the segmentation's counts; and in the other
//          workgroups the banks' transposes (and A as the shrink reads it),
//          every call: the banks change with every training step.
//   shrink the SGMM's.
//   coefs  per (32-slot tile, projection): u and w (their K slices added in
//          order), s u . w for dg, and the coefficients s g w and s g u, each as
//          three bf16 terms (8 + 8 + 8 bits: fp32 whole), transposed so
//          that eight slots of one rank are one 16-byte operand.  With two terms
//          the gradients lose a factor of three to fp32 sums; the third costs
//          matrix instructions where memory is the bound.
//   expand the SGMM's.
//   outer  dA and dB: per (projection, side, column block, chunk of an expert's
//          list) a product with M = ranks, N = columns and K = slots, bf16 MFMA
//          16x16x32 with fp32 sums.  A lane reads CPL columns of eight rows and
//          transposes the block in registers, one v_perm per two values: x and dy
//          go from memory to the matrix cores without LDS.  The four waves take
//          every fourth tile and add up through LDS in a fixed order.
//   sum    experts with several chunks: their partial sums in chunk order; dg.
// Every gradient element has one owner per launch: no atomics, bitwise
// reproducible.
//
// Chunks.  Routing is skewed (Zipf 1.1 over 8 experts: the first is in 60% of the
// rows), and one workgroup per (block, expert) would wait for the longest list.
// An expert's list is cut into chunks of at most chunk_tiles tiles, chosen so
// that a call has about kTargetItems chunks, several rounds of what the chip
// holds; only experts with more than one chunk pay for partial sums.
#include <type_traits>

#include "gfx950.hpp"
#include "internal.hpp"
#include "sgmm.hpp"

namespace dlm {

namespace {

size_t a256(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int kTargetItems = 4096;
constexpr int kMinChunkTiles = 16;  // four per wave: fewer would be mostly the sum at its end
constexpr int kCoefTerms = 3;

// Rank blocks (of 16) and columns per lane of the outer products.  From 48
// ranks on a lane takes four columns instead of eight: accumulators, rows and
// coefficients together then leave room for three waves per SIMD (one at 64
// ranks x 8 columns).
constexpr int outer_cpl(int r16) { return r16 <= 2 ? 8 : 4; }

int rank_chunks(const SgLayout& L) { return (L.r_pad + 63) / 64; }
int outer_r16(const SgLayout& L) { return L.r_pad <= 64 ? L.r_pad / 16 : 4; }

}  // namespace

int grad_cols(int r, int dtype) {
    const int r16 = (r + 15) / 16;
    return dtype == 1 ? 16 * outer_cpl(r16 < 4 ? r16 : 4) : 64;
}

SgGradLayout sgmm_grad_layout(int64_t T, int64_t total_ks, int E, int r, int n_prob, int n_units, int dtype) {
    SgGradLayout G;
    G.L = sgmm_layout(T, 1, E, r, (int)total_ks);  // one slice each of total_ks problems
    G.cap = (2 * T + (int64_t)E * (kGradTile - 1) + kGradTile - 1) / kGradTile * kGradTile;
    G.rc_pad = rank_chunks(G.L) * 16 * outer_r16(G.L);
    const int64_t tiles = G.cap / kGradTile, items = (int64_t)n_units * rank_chunks(G.L) * tiles;
    int64_t ct = (items + kTargetItems - 1) / kTargetItems;
    ct = ct < kMinChunkTiles ? kMinChunkTiles : ct;
    G.chunk_tiles = (int)(dtype == 1 ? (ct < (1 << 30) ? ct : 1 << 30) : 1 << 30);
    // full chunks (the bounds, not the count, so that it does not fall as T grows), and one more per expert
    const int64_t by_tiles = tiles / kMinChunkTiles, by_items = kTargetItems / ((int64_t)n_units * rank_chunks(G.L));
    G.max_chunks = (int)(dtype == 1 ? (by_tiles < by_items ? by_tiles : by_items) + E : E);
    size_t o = G.L.total;
    G.eoff = o;    o += a256((size_t)(E + 1) * 4);
    G.slot = o;    o += a256((size_t)G.cap * 4);
    G.srow = o;    o += a256((size_t)G.cap * 4);
    G.chunk = o;   o += a256((size_t)G.max_chunks * sizeof(SgChunk));
    G.echunk = o;  o += a256((size_t)(E + 1) * 4);
    G.coef = o;
    o += a256(dtype == 1 ? (size_t)n_prob * 2 * kCoefTerms * G.cap * G.rc_pad * 2 : (size_t)n_prob * 2 * G.cap * G.L.r_pad * 4);
    G.part = o;
    if (dtype == 1)
        o += (size_t)n_units * rank_chunks(G.L) * G.max_chunks * (16 * outer_r16(G.L)) * grad_cols(r, dtype) * 4;
    G.dgp = o;     o += a256((size_t)n_prob * T * 8);
    G.total = o;
    return G;
}

namespace {

__device__ __forceinline__ bool rejected(const SgGradArgs& a) { return gld((const int32_t*)(a.ws + a.G.L.hdr) + SG_ERR) != 0; }

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

// ---- coefficients -------------------------------------------------------------------

// Eight threads per slot, 16 ranks at a time.  Padding ranks and slots get 0
// (their v was never written: selected away, not multiplied).
template <bool BF>
__global__ __launch_bounds__(256) void grad_coefs(SgGradArgs a) {
    const SgLayout& L = a.G.L;
    if (rejected(a)) return;
    const int64_t tile = blockIdx.x;
    if (tile * kGradTile >= gld((const int32_t*)(a.ws + a.G.eoff) + a.E)) return;
    const int prob = blockIdx.y;
    const SgGrad P = a.probs[prob];
    const int tid = threadIdx.x, s = tid / 8, j = tid % 8, RPAD = L.r_pad, r = a.r;
    const int entry = gld((const int32_t*)(a.ws + a.G.slot) + tile * kGradTile + s);
    const bool live = entry >= 0;
    const int64_t q = live ? entry : 0;
    const float gate = live ? gld((const float*)(a.ws + L.gpk) + q) : 0.f;
    const float c = a.scale * gate;
    const int64_t stride = L.T_pad * 2 * RPAD;  // floats per K slice
    const float* vu = (const float*)(a.ws + L.v) + P.ks_u * stride + q * RPAD;
    const float* vw = (const float*)(a.ws + L.v) + P.ks_w * stride + q * RPAD;
    constexpr int kParts = BF ? 2 * kCoefTerms : 2;
    typedef typename std::conditional<BF, uint16_t, float>::type C;
    __shared__ __attribute__((aligned(16))) C s_c[kParts][16][kGradTile];
    float dot = 0.f;
    const int rc = BF ? a.G.rc_pad : RPAD;
    C* coef = (C*)(a.ws + a.G.coef);
    const int64_t part = a.G.cap * rc;  // elements of one (prob, side, term)
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    for (int r0 = 0; r0 < rc; r0 += 16) {
        const int rho = r0 + 2 * j;
        float u[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
        if (live && rho < r) {
            for (int k = 0; k < P.n_ks_u; ++k) {
                const f32x2_t v = gld((const f32x2_t*)(vu + k * stride + rho));
                u[0] = k ? u[0] + v.x : v.x;
                u[1] = k ? u[1] + v.y : v.y;
            }
            for (int k = 0; k < P.n_ks_w; ++k) {
                const f32x2_t v = gld((const f32x2_t*)(vw + k * stride + rho));
                w[0] = k ? w[0] + v.x : v.x;
                w[1] = k ? w[1] + v.y : v.y;
            }
            if (rho + 1 >= r) u[1] = w[1] = 0.f;
        }
        dot = fmaf(u[0], w[0], dot);
        dot = fmaf(u[1], w[1], dot);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float x = c * w[k], y = c * u[k];
            if constexpr (BF) {
#pragma unroll
                for (int m = 0; m < kCoefTerms; ++m) {
                    const uint16_t xm = f_to_bf(x), ym = f_to_bf(y);
                    s_c[m][2 * j + k][s] = xm;
                    s_c[kCoefTerms + m][2 * j + k][s] = ym;
                    x -= bf_to_f(xm);
                    y -= bf_to_f(ym);
                }
            } else {
                s_c[0][2 * j + k][s] = x;
                s_c[1][2 * j + k][s] = y;
            }
        }
        __syncthreads();
        constexpr int W = 16 / (int)sizeof(C), kRow = kGradTile / W;  // 16-byte stores per rank row
        for (int i = tid; i < kParts * 16 * kRow; i += 256) {
            const int m = i / (16 * kRow), rr = i / kRow % 16, o = W * (i % kRow);
            st128(coef + ((int64_t)prob * kParts + m) * part + (tile * rc + r0 + rr) * kGradTile + o,
                  *(const u32x4*)&s_c[m][rr][o]);
        }
    }
    // the slot's eight partial sums, in a fixed order
    dot += __shfl_xor(dot, 1, kWave);
    dot += __shfl_xor(dot, 2, kWave);
    dot += __shfl_xor(dot, 4, kWave);
    if (live && j == 0) {
        const int row = gld((const int32_t*)(a.ws + a.G.srow) + tile * kGradTile + s);
        gst((float*)(a.ws + a.G.dgp) + ((int64_t)prob * a.T + row) * 2 + (q & 1), a.scale * dot);
    }
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

// D = A(16x32) B(32x16) + C: lane l supplies row (l % 16) of A and column
// (l % 16) of B, k = 8 (l / 16) + [0, 8); register i holds D[4 (l / 16) + i][l % 16].
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
template <int CPL> struct RowRegs;
template <> struct RowRegs<8> { typedef u32x4 type; };
template <> struct RowRegs<4> { typedef u32x2v type; };

// The outer product's gradient element(s) of accumulators acc[b][j] (rank block
// b, column j of the lane): written or added to.
template <int R16, int CPL>
__device__ __forceinline__ void store_block(const SgGradArgs& a, const SgOuter& O, int e, int r0, int col, int kg, int b,
                                            const f32x4 (&acc)[CPL]) {
    const int r = a.r, d = O.d, rho = r0 + 16 * b + 4 * kg;  // this lane's four ranks
    if (col >= d) return;
    if (O.side == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (rho + i >= r) continue;
            f32x4* p = (f32x4*)(O.out + ((int64_t)e * r + rho + i) * d + col);
#pragma unroll
            for (int h = 0; h < CPL / 4; ++h) {
                f32x4 o = {acc[4 * h][i], acc[4 * h + 1][i], acc[4 * h + 2][i], acc[4 * h + 3][i]};
                if (a.accumulate) o += gld(p + h);
                gst(p + h, o);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
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

// Partial sums of item (unit, rank chunk, chunk): [b][j][lane] f32x4.
template <int R16, int CPL> __device__ __forceinline__ f32x4* part_of(const SgGradArgs& a, int64_t unit, int n_ch, int ch, int c) {
    return (f32x4*)(a.ws + a.G.part) + ((unit * n_ch + ch) * a.G.max_chunks + c) * (R16 * CPL * kWave);
}

template <int R16>
__global__ __launch_bounds__(256) void grad_outer_bf16(SgGradArgs a, int n_ch) {
    constexpr int CPL = outer_cpl(R16);
    typedef typename RowRegs<CPL>::type Row;
    if (rejected(a)) return;
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
    const int d = uniform(O.d), rc = a.G.rc_pad, r0 = ch * 64, t1 = K.t1;
    const int col = (int)(unit - O.unit0) * (16 * CPL) + CPL * n;
    const int lcol = col < d ? col : 0;  // columns past the end read the first ones and are not stored
    const uint16_t* __restrict__ act = (const uint16_t*)O.act + lcol;
    const int64_t part = a.G.cap * rc;
    const uint16_t* __restrict__ coef = (const uint16_t*)(a.ws + a.G.coef) +
                                        ((int64_t)O.prob * 2 + O.side) * kCoefTerms * part +
                                        (r0 + n) * kGradTile + 8 * kg;

    f32x4 acc[R16][CPL];
#pragma unroll
    for (int b = 0; b < R16; ++b)
#pragma unroll
        for (int j = 0; j < CPL; ++j) acc[b][j] = f32x4{};
    Row v[8];
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
        for (int i = 0; i < 8; ++i) v[i] = gld((const Row*)(act + (int64_t)rows[i] * d));
    };
    int t = K.t0 + w;
    if (t < t1) {
        load_rows(t);
        load_x();
        if (t + 4 < t1) load_rows(t + 4);
    }
#pragma unroll 1
    for (; t < t1; t += 4) {
        // this tile's coefficients go out before the next tile's rows, so
        // waiting for them does not wait for those
        u32x4 h[R16][kCoefTerms];
#pragma unroll
        for (int b = 0; b < R16; ++b)
#pragma unroll
            for (int m = 0; m < kCoefTerms; ++m)
                h[b][m] = ld128(coef + m * part + ((int64_t)t * rc + 16 * b) * kGradTile);
        // column j of the 8 x CPL block: one v_perm per two values
        u32x4 x[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                x[j][q] = __builtin_amdgcn_perm(v[2 * q + 1][j / 2], v[2 * q][j / 2], (j & 1) ? 0x07060302u : 0x05040100u);
        if (t + 4 < t1) {
            load_x();
            if (t + 8 < t1) load_rows(t + 8);
        }
#pragma unroll
        for (int b = 0; b < R16; ++b)
#pragma unroll
            for (int m = 0; m < kCoefTerms; ++m)
#pragma unroll
                for (int j = 0; j < CPL; ++j) acc[b][j] = mfma16(h[b][m], x[j], acc[b][j]);
    }
    // the four waves' sums: (0 + 2) + (1 + 3)
    __shared__ f32x4 s_red[2][R16 * CPL][kWave];
    if (w >= 2) {
#pragma unroll
        for (int b = 0; b < R16; ++b)
#pragma unroll
            for (int j = 0; j < CPL; ++j) s_red[w - 2][b * CPL + j][lane] = acc[b][j];
    }
    __syncthreads();
    if (w < 2) {
#pragma unroll
        for (int b = 0; b < R16; ++b)
#pragma unroll
            for (int j = 0; j < CPL; ++j) acc[b][j] += s_red[w][b * CPL + j][lane];
    }
    __syncthreads();
    if (w == 1) {
#pragma unroll
        for (int b = 0; b < R16; ++b)
#pragma unroll
            for (int j = 0; j < CPL; ++j) s_red[0][b * CPL + j][lane] = acc[b][j];
    }
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int b = 0; b < R16; ++b) {
#pragma unroll
        for (int j = 0; j < CPL; ++j) acc[b][j] += s_red[0][b * CPL + j][lane];
        if (K.alone) {
            store_block<R16, CPL>(a, O, K.e, r0, col, kg, b, acc[b]);
        } else {
            f32x4* p = part_of<R16, CPL>(a, unit, n_ch, ch, c) + b * CPL * kWave + lane;
#pragma unroll
            for (int j = 0; j < CPL; ++j) gst(p + j * kWave, acc[b][j]);
        }
    }
}

// Item (unit, rank chunk, expert): an expert with several chunks gets the sum of
// their partials in chunk order, one rank block per wave and turn.  The
// workgroups past the items write dg.
template <int R16>
__global__ __launch_bounds__(256) void grad_sum_bf16(SgGradArgs a, int n_ch, int64_t n_items) {
    constexpr int CPL = outer_cpl(R16);
    if (rejected(a)) return;
    if (blockIdx.x >= n_items) {
        write_dg(a, (blockIdx.x - n_items) * 256 + threadIdx.x);
        return;
    }
    const int e = blockIdx.x % a.E, ch = blockIdx.x / a.E % n_ch;
    const int64_t unit = blockIdx.x / a.E / n_ch;
    const int32_t* echunk = (const int32_t*)(a.ws + a.G.echunk);
    const int c0 = uniform(gld(echunk + e)), c1 = uniform(gld(echunk + e + 1));
    if (c1 - c0 < 2) return;
    const SgOuter O = a.outers[a.unit_outer[unit]];
    const int lane = lane_id(), n = lane & 15, kg = lane >> 4;
    const int col = (int)(unit - O.unit0) * (16 * CPL) + CPL * n;
    for (int b = wave_id(); b < R16; b += 4) {
        f32x4 acc[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) acc[j] = f32x4{};
        for (int c = c0; c < c1; ++c) {
            const f32x4* p = part_of<R16, CPL>(a, unit, n_ch, ch, c) + b * CPL * kWave + lane;
#pragma unroll
            for (int j = 0; j < CPL; ++j) acc[j] += gld(p + j * kWave);
        }
        store_block<R16, CPL>(a, O, e, ch * 64, col, kg, b, acc);
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

int64_t dg_blocks(const SgGradArgs& a) { return a.dg ? (2 * a.T + 255) / 256 : 0; }
int64_t outer_blocks(const SgGradArgs& a) {
    return 8ll * a.G.max_chunks * rank_chunks(a.G.L) * ((a.n_units + 7) / 8);
}
int64_t sum_items(const SgGradArgs& a) { return (int64_t)a.n_units * rank_chunks(a.G.L) * a.E; }

template <int R16> hipError_t launch_outer(const SgGradArgs& a, hipStream_t s) {
    const int n_ch = rank_chunks(a.G.L);
    hipLaunchKernelGGL(grad_outer_bf16<R16>, dim3((unsigned)outer_blocks(a)), dim3(256), 0, s, a, n_ch);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // no expert can have a second chunk while a chunk holds every tile
    const int64_t items = a.G.max_chunks > a.E ? sum_items(a) : 0;
    if (items + dg_blocks(a) == 0) return hipSuccess;
    hipLaunchKernelGGL(grad_sum_bf16<R16>, dim3((unsigned)(items + dg_blocks(a))), dim3(256), 0, s, a, n_ch, items);
    return hipGetLastError();
}

}  // namespace

bool sgmm_grad_fits(const SgGradArgs& a, int dtype) {
    return grad_prep_fits(a) && grid_fits(a.G.cap / kGradTile, 256) && grid_fits((a.T + 1) / 2, 256) &&
           grid_fits(a.n_units + dg_blocks(a), 256) &&
           (dtype == 0 || (grid_fits(outer_blocks(a), 256) && grid_fits(sum_items(a) + dg_blocks(a), 256)));
}

hipError_t launch_grad_zero(const SgGradArgs& a, int dtype, hipStream_t s) {
    hipLaunchKernelGGL(grad_zero, dim3((unsigned)a.n_units, (unsigned)a.E), dim3(kWave), 0, s, a, grad_cols(a.r, dtype));
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
    switch (outer_r16(a.G.L)) {
        case 1: return launch_outer<1>(a, s);
        case 2: return launch_outer<2>(a, s);
        case 3: return launch_outer<3>(a, s);
        default: return launch_outer<4>(a, s);
    }
}

}  // namespace dlm
