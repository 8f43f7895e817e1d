// Gradients of the SGMM y[t] += sum_k s g_k B_{e_k} (A_{e_k} x[t]).  With
// u = A_e x and w = B_e^T dy per row and slot:
//   dx[t] += sum_k s g_k A_{e_k}^T w        dg[t][k] = s u . w
//   dA_e   = sum s g w x[t]^T               dB_e     = sum s g dy[t] u^T
// (sums over the slots (t, k) that chose e).
//
// dx is itself an SGMM, of dy through the banks' transposes, so it runs the
// SGMM's own kernels: one segmentation, one shrink launch over the projections'
// (x, A) and (dy, B^T) together, which leaves u and w in the workspace, and the
// expand of w through A^T into dx.  The rest is here:
//   pack   the banks' transposes (and A as the shrink reads it), every call:
//          the banks change with every training step.
//   lists  every expert's slots in sorted-position order, padded to whole
//          tiles of 32 (a padding slot repeats a row of its expert with
//          coefficients 0, so it brings in no row's infinities that are not
//          the expert's own); one workgroup per expert.
//   coefs  per (32-slot tile, projection): u and w (their K slices added in
//          order), s u . w for dg, and the products' coefficients s g w and
//          s g u, each as two bf16 terms (hi + lo hold 16 bits of it, as the
//          expand's do: one bf16 alone would cost 2^-9), transposed so that
//          eight slots of one rank are one 16-byte operand.
//   outer  dA and dB: per (projection, side, 128 columns, expert) a product
//          with M = ranks, N = columns and K = the expert's slots, bf16 MFMA
//          16x16x32 with fp32 sums.  A lane reads eight columns of eight rows
//          (16 bytes each; a quarter wave reads 256 contiguous bytes of a row)
//          and transposes the 8x8 block in registers, one v_perm per two
//          values: x and dy go from memory to the matrix cores without LDS.
//          The four waves take every fourth tile and add up through LDS in a
//          fixed order.  Every gradient element has one owner: no atomics,
//          bitwise reproducible.
// The x and dy rows are read by the shrink and, once per chosen slot, by the
// outer product: the experts of one column block run next to each other on one
// XCD so that the second slot's read finds the row in L2 or the memory-side cache.
#include "gfx950.hpp"
#include "internal.hpp"
#include "sgmm.hpp"

namespace dlm {

static size_t a256(size_t v) { return (v + 255) & ~(size_t)255; }

SgGradLayout sgmm_grad_layout(int64_t T, int64_t d_max, int E, int r, int n_prob) {
    SgGradLayout G;
    G.L = sgmm_layout(T, d_max, E, r, 2 * n_prob);
    G.cap = (2 * T + (int64_t)E * (kGradTile - 1) + kGradTile - 1) / kGradTile * kGradTile;
    G.rc_pad = G.L.r_pad <= 64 ? G.L.r_pad : (G.L.r_pad + 63) / 64 * 64;
    size_t o = G.L.total;
    G.eoff = o;  o += a256((size_t)(E + 1) * 4);
    G.slot = o;  o += a256((size_t)G.cap * 4);
    G.srow = o;  o += a256((size_t)G.cap * 4);
    G.coef = o;  o += a256((size_t)n_prob * 4 * G.cap * G.rc_pad * 2);
    G.dgp = o;   o += a256((size_t)n_prob * T * 8);
    G.total = o;
    return G;
}

namespace {

// ---- banks' transposes ----------------------------------------------------------

// One thread per eight elements of a projection's A (then of its B).  A: eight
// columns of one rank row, written as the packed group the shrink reads and as
// eight elements of the transpose; B: element [e][o][rho] of eight consecutive o.
// Groups are numbered so that neighbouring threads read and write neighbours.
__global__ __launch_bounds__(256) void grad_pack_bf16(SgGradArgs a) {
    const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (q >= a.pk_total) return;
    int p = 0;
    for (int lo = 0, hi = a.n_prob - 1; lo <= hi;) {  // the last projection that starts at or before q
        const int mid = (lo + hi) / 2;
        if (a.probs[mid].pk0 <= q) p = mid, lo = mid + 1;
        else hi = mid - 1;
    }
    const SgGrad P = a.probs[p];
    const int r = a.r;
    const int64_t i = q - P.pk0, na = (int64_t)a.E * r * (P.d_in / 8);
    if (i < na) {
        const int64_t nq = P.d_in / 8, rho = i % r, kq = (i / r) % nq, e = i / (r * nq);
        const u32x4 v = ld128((const uint16_t*)P.A + ((e * r + rho) * nq + kq) * 8);
        st128((uint16_t*)P.Ap + 8 * i, v);
        uint16_t* t = (uint16_t*)P.At + (e * P.d_in + 8 * kq) * r + rho;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            gst(t + (2 * j) * r, (uint16_t)(v[j] & 0xffffu));
            gst(t + (2 * j + 1) * r, (uint16_t)(v[j] >> 16));
        }
    } else {
        const int64_t b = i - na, nq = P.d_out / 8, rho = b % r, kq = (b / r) % nq, e = b / (r * nq);
        const uint16_t* src = (const uint16_t*)P.B + (e * P.d_out + 8 * kq) * r + rho;
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (uint32_t)gld(src + (2 * j) * r) | ((uint32_t)gld(src + (2 * j + 1) * r) << 16);
        st128((uint16_t*)P.Bt + 8 * b, v);
    }
}

// fp32: one thread per element; At [E][d_in][r], Bt [E][r][d_out].
__global__ __launch_bounds__(256) void grad_pack_f32(SgGradArgs a) {
    const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (q >= a.pk_total) return;
    int p = 0;
    for (int lo = 0, hi = a.n_prob - 1; lo <= hi;) {
        const int mid = (lo + hi) / 2;
        if (a.probs[mid].pk0 <= q) p = mid, lo = mid + 1;
        else hi = mid - 1;
    }
    const SgGrad P = a.probs[p];
    const int r = a.r;
    const int64_t i = q - P.pk0, na = (int64_t)a.E * r * P.d_in;
    if (i < na) {
        const int64_t rho = i % r, j = (i / r) % P.d_in, e = i / ((int64_t)r * P.d_in);
        gst((float*)P.At + i, gld((const float*)P.A + (e * r + rho) * P.d_in + j));
    } else {
        const int64_t b = i - na, o = b % P.d_out, rho = (b / P.d_out) % r, e = b / ((int64_t)r * P.d_out);
        gst((float*)P.Bt + b, gld((const float*)P.B + (e * P.d_out + o) * r + rho));
    }
}

// ---- the experts' slot lists ------------------------------------------------------

constexpr int kListThreads = 1024;
constexpr int kListWaves = kListThreads / kWave;

// Workgroup e: counts every expert's slots (its list starts behind the earlier
// experts' padded lists), then writes its own list in position order.
__global__ __launch_bounds__(kListThreads) void grad_lists(SgGradArgs a) {
    const SgLayout& L = a.G.L;
    const int32_t* hdr = (const int32_t*)(a.ws + L.hdr);
    const int32_t* perm = (const int32_t*)(a.ws + L.perm);
    const uint32_t* epk = (const uint32_t*)(a.ws + L.epk);
    int32_t* eoff = (int32_t*)(a.ws + a.G.eoff);
    int32_t* slot = (int32_t*)(a.ws + a.G.slot);
    int32_t* srow = (int32_t*)(a.ws + a.G.srow);
    if (gld(hdr + SG_ERR)) return;
    const int n_pos = gld(hdr + SG_NPOS);
    const int e = blockIdx.x, E = a.E, tid = threadIdx.x, lane = lane_id(), w = wave_id();
    __shared__ int s_cnt[32], s_wave[kListWaves], s_last;
    if (tid < 32) s_cnt[tid] = 0;
    if (tid == 0) s_last = -1;
    __syncthreads();
    for (int p0 = 0; p0 < n_pos; p0 += kListThreads) {
        const int p = p0 + tid;
        const uint32_t ep = p < n_pos ? gld(epk + p) : 0xffffffffu;
        const int e0 = (int16_t)(ep & 0xffffu), e1 = (int16_t)(ep >> 16);
        for (int x = 0; x < E; ++x) {
            const int n = (int)(__popcll(__ballot(e0 == x)) + __popcll(__ballot(e1 == x)));
            if (lane == 0 && n) atomicAdd(&s_cnt[x], n);
        }
    }
    __syncthreads();
    int off = 0;
    for (int x = 0; x < E; ++x) {
        if (e == 0 && tid == 0) gst(eoff + x, off);
        if (x < e || e == 0) off += (s_cnt[x] + kGradTile - 1) / kGradTile * kGradTile;
    }
    if (e == 0) {
        if (tid == 0) gst(eoff + E, off);
        off = 0;
    }
    const int cnt = s_cnt[e];
    int done = 0;
    for (int p0 = 0; p0 < n_pos; p0 += kListThreads) {
        const int p = p0 + tid;
        const uint32_t ep = p < n_pos ? gld(epk + p) : 0xffffffffu;
        const bool k0 = (int16_t)(ep & 0xffffu) == e, k1 = (int16_t)(ep >> 16) == e;
        const uint64_t b0 = __ballot(k0), b1 = __ballot(k1), lt = (1ull << lane) - 1ull;
        if (lane == 0) s_wave[w] = (int)(__popcll(b0) + __popcll(b1));
        __syncthreads();
        int at = done, all = 0;
        for (int i = 0; i < kListWaves; ++i) {
            at += i < w ? s_wave[i] : 0;
            all += s_wave[i];
        }
        at += (int)(__popcll(b0 & lt) + __popcll(b1 & lt));
        if (k0 || k1) {
            const int row = gld(perm + p);
            if (k0) {
                gst(slot + off + at, 2 * p);
                gst(srow + off + at, row);
            }
            if (k1) {
                gst(slot + off + at + (k0 ? 1 : 0), 2 * p + 1);
                gst(srow + off + at + (k0 ? 1 : 0), row);
            }
            if (at + (k0 && k1 ? 2 : 1) == cnt) s_last = row;
        }
        done += all;
        __syncthreads();
    }
    const int pad = (cnt + kGradTile - 1) / kGradTile * kGradTile;
    if (tid < pad - cnt) {
        gst(slot + off + cnt + tid, -1);
        gst(srow + off + cnt + tid, s_last);
    }
}

// ---- coefficients -------------------------------------------------------------------

// Eight threads per slot, kRank ranks at a time.  Padding ranks and slots get 0
// (their v was never written: selected away, not multiplied).
template <bool BF>
__global__ __launch_bounds__(256) void grad_coefs(SgGradArgs a) {
    const SgLayout& L = a.G.L;
    const int32_t* hdr = (const int32_t*)(a.ws + L.hdr);
    if (gld(hdr + SG_ERR)) return;
    const int32_t* eoff = (const int32_t*)(a.ws + a.G.eoff);
    const int64_t tile = blockIdx.x;
    if (tile * kGradTile >= gld(eoff + a.E)) return;
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
    __shared__ __attribute__((aligned(16))) uint16_t s_c[4][16][kGradTile];  // side x (hi, lo), 16 ranks
    float dot = 0.f;
    const int rc = BF ? a.G.rc_pad : RPAD;
    uint16_t* coef = (uint16_t*)(a.ws + a.G.coef);
    const int64_t part = a.G.cap * rc;  // elements of one (prob, side, term)
    for (int r0 = 0; r0 < rc; r0 += 16) {
        const int rho = r0 + 2 * j;
        float u[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
        typedef float f32x2_t __attribute__((ext_vector_type(2)));
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
        if constexpr (BF) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float x = c * w[k], y = c * u[k];
                const uint16_t xh = f_to_bf(x), yh = f_to_bf(y);
                s_c[0][2 * j + k][s] = xh;
                s_c[1][2 * j + k][s] = f_to_bf(x - bf_to_f(xh));
                s_c[2][2 * j + k][s] = yh;
                s_c[3][2 * j + k][s] = f_to_bf(y - bf_to_f(yh));
            }
            __syncthreads();
            // 4 parts x 16 ranks x 64 bytes: one 16-byte store per thread
            const int part_i = tid / 64, rr = (tid / 4) % 16, o = 8 * (tid % 4);
            st128(coef + ((int64_t)prob * 4 + part_i) * part + (tile * rc + r0 + rr) * kGradTile + o,
                  *(const u32x4*)&s_c[part_i][rr][o]);
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
__global__ __launch_bounds__(256) void grad_dg(SgGradArgs a) {
    if (gld((const int32_t*)(a.ws + a.G.L.hdr) + SG_ERR)) return;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
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

// Column c of the 8x8 bf16 block whose row i is v[i]: one v_perm per two values.
__device__ __forceinline__ u32x4 column(const u32x4 (&v)[8], int c) {
    u32x4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        o[q] = __builtin_amdgcn_perm(v[2 * q + 1][c / 2], v[2 * q][c / 2], (c & 1) ? 0x07060302u : 0x05040100u);
    return o;
}

template <int R16>
__global__ __launch_bounds__(256) void grad_outer_bf16(SgGradArgs a, int rank_chunks) {
    const SgLayout& L = a.G.L;
    const int32_t* hdr = (const int32_t*)(a.ws + L.hdr);
    if (gld(hdr + SG_ERR)) return;
    // XCD b % 8 takes every eighth column block, its experts (and rank chunks) one after another
    const int per_unit = a.E * rank_chunks;
    const int64_t jj = blockIdx.x / 8;
    const int64_t unit = jj / per_unit * 8 + blockIdx.x % 8;
    if (unit >= a.n_units) return;
    const int sub = (int)(jj % per_unit), e = sub % a.E, ch = sub / a.E;
    const SgOuter O = a.outers[a.unit_outer[unit]];
    const int c0 = (int)(unit - O.unit0) * kGradCols;
    const int32_t* eoff = (const int32_t*)(a.ws + a.G.eoff);
    const int32_t* srow = (const int32_t*)(a.ws + a.G.srow);
    const int t0 = uniform(gld(eoff + e)) / kGradTile, t1 = uniform(gld(eoff + e + 1)) / kGradTile;
    const int lane = lane_id(), w = wave_id(), n = lane & 15, kg = lane >> 4;
    const int d = uniform(O.d), rc = a.G.rc_pad, r0 = ch * 64;
    const uint16_t* __restrict__ act = (const uint16_t*)O.act;
    const int64_t part = a.G.cap * rc;
    const uint16_t* __restrict__ hi = (const uint16_t*)(a.ws + a.G.coef) + ((int64_t)O.prob * 4 + 2 * O.side) * part;
    const uint16_t* __restrict__ lo = hi + part;
    const int col = c0 + 8 * n;
    const int lcol = col < d ? col : 0;  // columns past the end read the first ones and are not stored

    f32x4 acc[R16][8];
#pragma unroll
    for (int b = 0; b < R16; ++b)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[b][j] = f32x4{};
    u32x4 v[8], ch_[R16], cl_[R16];
    int rows[8];
    auto load_rows = [&](int t) {
        const u32x4 a0 = ld128(srow + t * kGradTile + 8 * kg), a1 = ld128(srow + t * kGradTile + 8 * kg + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rows[i] = (int)a0[i];
            rows[4 + i] = (int)a1[i];
        }
    };
    auto load_tile = [&](int t) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = ld128(act + (int64_t)rows[i] * d + lcol);
#pragma unroll
        for (int b = 0; b < R16; ++b) {
            const int64_t o = ((int64_t)t * rc + r0 + 16 * b + n) * kGradTile + 8 * kg;
            ch_[b] = ld128(hi + o);
            cl_[b] = ld128(lo + o);
        }
    };
    int t = t0 + w;
    if (t < t1) {
        load_rows(t);
        load_tile(t);
        if (t + 4 < t1) load_rows(t + 4);
    }
#pragma unroll 1
    for (; t < t1; t += 4) {
        u32x4 x[8], h[R16], l[R16];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v[i];
#pragma unroll
        for (int b = 0; b < R16; ++b) {
            h[b] = ch_[b];
            l[b] = cl_[b];
        }
        if (t + 4 < t1) {
            load_tile(t + 4);
            if (t + 8 < t1) load_rows(t + 8);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const u32x4 bx = column(x, j);
#pragma unroll
            for (int b = 0; b < R16; ++b) {
                acc[b][j] = mfma16(h[b], bx, acc[b][j]);
                acc[b][j] = mfma16(l[b], bx, acc[b][j]);
            }
        }
    }
    // the four waves' sums: (0 + 2) + (1 + 3)
    __shared__ f32x4 s_red[2][R16 * 8][kWave];
    if (w >= 2) {
#pragma unroll
        for (int b = 0; b < R16; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j) s_red[w - 2][b * 8 + j][lane] = acc[b][j];
    }
    __syncthreads();
    if (w < 2) {
#pragma unroll
        for (int b = 0; b < R16; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[b][j] += s_red[w][b * 8 + j][lane];
    }
    __syncthreads();
    if (w == 1) {
#pragma unroll
        for (int b = 0; b < R16; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j) s_red[0][b * 8 + j][lane] = acc[b][j];
    }
    __syncthreads();
    if (w != 0 || col >= d) return;
    const int r = a.r;
#pragma unroll
    for (int b = 0; b < R16; ++b) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[b][j] += s_red[0][b * 8 + j][lane];
        const int rho = r0 + 16 * b + 4 * kg;  // this lane's four ranks
        if (O.side == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (rho + i >= r) continue;
                float* p = O.out + ((int64_t)e * r + rho + i) * d + col;
                f32x4 o0 = {acc[b][0][i], acc[b][1][i], acc[b][2][i], acc[b][3][i]};
                f32x4 o1 = {acc[b][4][i], acc[b][5][i], acc[b][6][i], acc[b][7][i]};
                if (a.accumulate) {
                    o0 += gld((const f32x4*)p);
                    o1 += gld((const f32x4*)p + 1);
                }
                gst((f32x4*)p, o0);
                gst((f32x4*)p + 1, o1);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float* p = O.out + ((int64_t)e * d + col + j) * r + rho;
                if ((r & 3) == 0) {
                    if (rho >= r) continue;
                    f32x4 o = acc[b][j];
                    if (a.accumulate) o += gld((const f32x4*)p);
                    gst((f32x4*)p, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (rho + i < r) gst(p + i, a.accumulate ? gld(p + i) + acc[b][j][i] : acc[b][j][i]);
                }
            }
        }
    }
}

// fp32: one thread per column, eight ranks at a time over the expert's slots in list order.
__global__ __launch_bounds__(kGradCols) void grad_outer_f32(SgGradArgs a) {
    const SgLayout& L = a.G.L;
    if (gld((const int32_t*)(a.ws + L.hdr) + SG_ERR)) return;
    const int unit = blockIdx.x, e = blockIdx.y, r = a.r, RPAD = L.r_pad;
    const SgOuter O = a.outers[a.unit_outer[unit]];
    const SgGrad P = a.probs[O.prob];
    const int col = (unit - O.unit0) * kGradCols + threadIdx.x;
    if (col >= O.d) return;
    const int32_t* eoff = (const int32_t*)(a.ws + a.G.eoff);
    const int32_t* slot = (const int32_t*)(a.ws + a.G.slot);
    const int32_t* srow = (const int32_t*)(a.ws + a.G.srow);
    const float* gpk = (const float*)(a.ws + L.gpk);
    const float* v = (const float*)(a.ws + L.v) + (O.side == 0 ? P.ks_w : P.ks_u) * L.T_pad * 2 * RPAD;
    const float* act = (const float*)O.act;
    const int s0 = gld(eoff + e), s1 = gld(eoff + e + 1);
    for (int r0 = 0; r0 < r; r0 += 8) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int s = s0; s < s1; ++s) {
            const int q = gld(slot + s);
            if (q < 0) break;
            const float x = gld(act + (int64_t)gld(srow + s) * O.d + col), c = a.scale * gld(gpk + q);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r0 + i < r) acc[i] = fmaf(c * gld(v + (int64_t)q * RPAD + r0 + i), x, acc[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (r0 + i >= r) break;
            float* p = O.side == 0 ? O.out + ((int64_t)e * r + r0 + i) * O.d + col
                                   : O.out + ((int64_t)e * O.d + col) * r + r0 + i;
            gst(p, a.accumulate ? gld(p) + acc[i] : acc[i]);
        }
    }
}

__global__ __launch_bounds__(kGradCols) void grad_zero(SgGradArgs a) {
    const int unit = blockIdx.x, e = blockIdx.y;
    const SgOuter O = a.outers[a.unit_outer[unit]];
    const int col = (unit - O.unit0) * kGradCols + threadIdx.x;
    if (col >= O.d) return;
    for (int rho = 0; rho < a.r; ++rho)
        gst(O.side == 0 ? O.out + ((int64_t)e * a.r + rho) * O.d + col : O.out + ((int64_t)e * O.d + col) * a.r + rho, 0.f);
}

int64_t outer_blocks(const SgGradArgs& a) {
    const int chunks = (a.G.L.r_pad + 63) / 64;
    return 8ll * a.E * chunks * ((a.n_units + 7) / 8);
}

}  // namespace

bool sgmm_grad_fits(const SgGradArgs& a, int dtype) {
    return grid_fits((a.pk_total + 255) / 256, 256) && grid_fits(a.G.cap / kGradTile, 256) &&
           grid_fits((2 * a.T + 255) / 256, 256) && grid_fits(a.n_units, kGradCols) && (dtype == 0 || grid_fits(outer_blocks(a), 256));
}

hipError_t launch_grad_zero(const SgGradArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(grad_zero, dim3((unsigned)a.n_units, (unsigned)a.E), dim3(kGradCols), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_pack(const SgGradArgs& a, int dtype, hipStream_t s) {
    const dim3 g((unsigned)((a.pk_total + 255) / 256));
    if (dtype == 1) hipLaunchKernelGGL(grad_pack_bf16, g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(grad_pack_f32, g, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_lists(const SgGradArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(grad_lists, dim3((unsigned)a.E), dim3(kListThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_coefs(const SgGradArgs& a, int dtype, hipStream_t s) {
    const dim3 g((unsigned)(a.G.cap / kGradTile), (unsigned)a.n_prob);
    if (dtype == 1) hipLaunchKernelGGL(grad_coefs<true>, g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(grad_coefs<false>, g, dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dg) return e;
    hipLaunchKernelGGL(grad_dg, dim3((unsigned)((2 * a.T + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_outer(const SgGradArgs& a, int dtype, hipStream_t s) {
    if (dtype == 0) {
        hipLaunchKernelGGL(grad_outer_f32, dim3((unsigned)a.n_units, (unsigned)a.E), dim3(kGradCols), 0, s, a);
        return hipGetLastError();
    }
    const int chunks = (a.G.L.r_pad + 63) / 64;
    const dim3 g((unsigned)outer_blocks(a));
    switch (a.G.L.r_pad <= 64 ? a.G.L.r_pad / 16 : 4) {
        case 1: hipLaunchKernelGGL(grad_outer_bf16<1>, g, dim3(256), 0, s, a, chunks); break;
        case 2: hipLaunchKernelGGL(grad_outer_bf16<2>, g, dim3(256), 0, s, a, chunks); break;
        case 3: hipLaunchKernelGGL(grad_outer_bf16<3>, g, dim3(256), 0, s, a, chunks); break;
        default: hipLaunchKernelGGL(grad_outer_bf16<4>, g, dim3(256), 0, s, a, chunks); break;
    }
    return hipGetLastError();
}

}  // namespace dlm
