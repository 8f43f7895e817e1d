// One step of momentum orthogonalised by Newton-Schulz products, over many matrices:
//   m <- b m + (1 - b) g,  u = b m + (1 - b) g (or m)
//   X = u / (|u| + eps), K times X <- a X + (b A + c A^2) X with A = X X^T
//   w <- w (1 - lr wd) - lr s X
//
// Every factor of the K products is a polynomial of one Gram matrix, G = u u^T over
// the small side n of a matrix n x d (u^T u for the other way round: the same X): with
//   Q = a + b G + c G^2,  P <- Q P,  G <- Q G Q     X = P u / (|u| + eps)
// u is read twice, not 2 K times, and what lies between is n x n.  Squaring u loses
// its weak directions in fp32 (a direction 10^-4 of the strongest is 10^-8 of G, and
// each of the K steps makes it, and its error, a^2 = 12 times larger): G, P and the
// sums are binary64, on the binary64 matrix instructions, whose products of fp32
// values are exact.  Their rate (66 TFLOP/s in a large product) and a copy's, 4.6 TB/s,
// meet near a small side of 80; at rank 16 they are a fifth of the memory's time.
//
// Launches per class of matrices (small sides up to 16, 32, 64): the Gram matrices of
// pieces of the long side, the n x n steps (a workgroup per matrix, a wave per 16 x 16
// block), and the product with the update.  A symmetric block's accumulators are its
// operands of the next product: entry (4 v + l / 16, l % 16) in register v of lane l is
// also what an operand wants there.  The product takes four neighbouring elements of u
// per lane and access, with the order of rows or columns within a tile (which the
// sum does not see) chosen so that each lane's results are the elements it loaded.
//
// Small sides from 65 to 512 (routers of many experts): the same with 64 x 64 tiles, u
// in scratch memory, and a launch per n x n product.
//
// A matrix whose u is not finite, or whose X would leave fp32's range, is left as it was,
// momentum too, and the handle's error word is set.
//
// Measured: 322 million bf16 weights at rank 16, fp32 gradients and masters, 1.6 to 1.74 ms:
// the Gram pass 0.44-0.47, the steps 0.026, the update 1.12-1.21; both passes move 5.6 to 6
// TB/s (with u read twice that is 4.05 to 4.4 TB/s of the bytes that a step cannot do
// without).  10 million: 18, 8 and 42-45 us.  Rank 64, 16.8 million: 53, 42 and 87 us, where
// neither memory (2.9 and 4.6 TB/s) nor the matrix cores (12 and 29 % of the cycles) are
// busy: two waves a SIMD, each in a chain of loads, products and stores, and a 64 x 64 tile's
// u and m beside its products' operands do not fit their registers: 29 are spilled in the
// Gram kernel, 28 or 38 (bf16 or fp32 gradients) in the update.  8192 x 256: 145 to 160 us
// in 18 launches.
#include <utility>

#include "gfx950.hpp"
#include "internal.hpp"
#include "muon.hpp"

namespace dlm {

namespace {

constexpr int kNT = 256;
constexpr int kWaves = kNT / kWave;

typedef double d4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ d4 mfma(double a, double b, d4 c) { return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0); }

__device__ __forceinline__ float read1(const float* p) { return gld(p); }
__device__ __forceinline__ float read1(const uint16_t* p) { return bf_to_f(gld(p)); }
__device__ __forceinline__ void store1(float* p, float f) { gst(p, f); }
__device__ __forceinline__ void store1(uint16_t* p, float f) { gst(p, f_to_bf(f)); }

__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
    const u32x4 r = ld128(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&f)[4]) {
    const u32x2 r = gld((const u32x2*)p);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        f[2 * j] = bf_lo(r[j]);
        f[2 * j + 1] = bf_hi(r[j]);
    }
}
template <typename T> __device__ __forceinline__ void store4(T* p, const float (&f)[4]) {
    if constexpr (sizeof(T) == 4) st128(p, u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])});
    else gst((u32x2*)p, u32x2{pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3])});
}
// The same for what is used for the last time, past the caches (which keep what a later
// launch reads again).
__device__ __forceinline__ void load4_nt(const float* p, float (&f)[4]) {
    const u32x4 r = ld128_nt(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void load4_nt(const uint16_t* p, float (&f)[4]) {
    const u32x2 r = __builtin_nontemporal_load((gcptr<u32x2>)p);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        f[2 * j] = bf_lo(r[j]);
        f[2 * j + 1] = bf_hi(r[j]);
    }
}
__device__ __forceinline__ void store4_nt(float* p, const float (&f)[4]) {
    st128_nt(p, u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])});
}
__device__ __forceinline__ void store4_nt(uint16_t* p, const float (&f)[4]) {
    __builtin_nontemporal_store(u32x2{pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3])}, (gptr<u32x2>)p);
}
// Four neighbours of which nv are inside (vec: all or none), 0 for the others.
template <bool NT = false, typename T>
__device__ __forceinline__ void read4(const T* p, int64_t i, int nv, bool vec, float (&f)[4]) {
    if (vec && nv >= 4) {
        if constexpr (NT) load4_nt(p + i, f);
        else load4(p + i, f);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = !vec && j < nv ? read1(p + i + j) : 0.f;
    }
}
template <bool NT = false, typename T>
__device__ __forceinline__ void write4(T* p, int64_t i, int nv, bool vec, const float (&f)[4]) {
    if (vec && nv >= 4) {
        if constexpr (NT) store4_nt(p + i, f);
        else store4(p + i, f);
    } else if (!vec) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < nv) store1(p + i + j, f[j]);
    }
}

// The momentum's step: fp32, as it is stored.
struct Mom {
    float b, r, gs;
    bool nesterov;
    __device__ __forceinline__ explicit Mom(const MuonArgs& a)
        : b((float)a.beta), r((float)(1.0 - a.beta)), gs(a.grad_scale ? gld(a.grad_scale) : 1.f), nesterov(a.nesterov != 0) {}
    __device__ __forceinline__ float m(float m0, float g) const { return fmaf(b, m0, r * (g * gs)); }
    __device__ __forceinline__ float u(float m1, float g) const { return nesterov ? fmaf(b, m1, r * (g * gs)) : m1; }
};

// Where an element of the matrix at `base` lies.
struct Place {
    int64_t base, d;
    int n;
    bool wide, vec;
    __device__ __forceinline__ Place(const MuDesc& D, int64_t mat) : base(mat * D.n * D.d), d(D.d), n(D.n), wide(D.wide != 0), vec(D.vec != 0) {}
    __device__ __forceinline__ int64_t at(int i, int64_t j) const { return wide ? base + i * d + j : base + j * n + i; }
};

// ---- u --------------------------------------------------------------------------------

// From the gradient and the momentum,
template <typename G> struct FromState {
    struct Raw {
        float g[4], m[4];
    };
    const G* g;
    const float* m;
    Mom mom;
    __device__ __forceinline__ void load4(int64_t i, int nv, bool vec, Raw& r) const {
        read4(g, i, nv, vec, r.g);
        read4(m, i, nv, vec, r.m);
    }
    __device__ __forceinline__ float u(const Raw& r, int c) const { return mom.u(mom.m(r.m[c], r.g[c]), r.g[c]); }
};
// or from the scratch where a launch has left it.
struct FromScratch {
    struct Raw {
        float u[4];
    };
    const float* p;
    __device__ __forceinline__ void load4(int64_t i, int nv, bool vec, Raw& r) const { read4(p, i, nv, vec, r.u); }
    __device__ __forceinline__ void load1(int64_t i, bool in, int c, Raw& r) const { r.u[c] = in ? gld(p + i) : 0.f; }
    __device__ __forceinline__ float u(const Raw& r, int c) const { return r.u[c]; }
};

// The lane's place of its v-th (wide) or x-th (tall) group of four in block b.
template <bool WIDE>
__device__ __forceinline__ int group_at(const Place& q, int b, int k, int64_t j0, int64_t hi, int lane, int64_t* at) {
    const int i = WIDE ? 16 * b + 4 * k + lane / 16 : 16 * b + 4 * (lane / 16);
    const int64_t j = WIDE ? j0 + 4 * (lane % 16) : j0 + 16 * k + lane % 16;
    *at = WIDE ? q.base + i * q.d + j : q.base + j * q.n + i;
    if (i >= q.n || j >= hi) return 0;
    const int64_t left = WIDE ? hi - j : q.n - i;
    return left < 4 ? (int)left : 4;
}
// ---- Gram matrices of pieces ------------------------------------------------------------

// Operands of columns [lo, hi) of the long side for one wave, for NB blocks of the
// small side from i0 on, handed to `use(a)` four columns at a time; the loads of the next 16 S
// columns are out while these are used (three such ahead leave a SIMD one wave: 44 us for 8192 x 256,
// against 30).  Wide: a lane loads
// four neighbours of its row; tall: the small side is contiguous, and a wave's lanes are.
template <bool WIDE, int NB, int S, typename SRC, typename F>
__device__ __forceinline__ void long_side(const SRC& src, const Place& q, const int (&i0)[NB], int64_t lo, int64_t hi, F use) {
    const int lane = lane_id();
    constexpr int STEP = 16 * S;
    typename SRC::Raw raw[2][NB][S];
    const auto load = [&](int64_t j0, typename SRC::Raw (&r)[NB][S]) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if constexpr (WIDE) {
                    const int64_t j = j0 + 16 * s + 4 * (lane / 16), left = hi - j;
                    const int i = i0[b] + lane % 16;
                    src.load4(q.at(i, j), i < q.n && left > 0 ? (left < 4 ? (int)left : 4) : 0, q.vec, r[b][s]);
                } else {
                    const int i = i0[b] + lane % 16;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int64_t j = j0 + 16 * s + 4 * c + lane / 16;
                        src.load1(q.at(i, j), i < q.n && j < hi, c, r[b][s]);
                    }
                }
            }
    };
    const auto spend = [&](const typename SRC::Raw (&r)[NB][S]) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                double a[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) a[b] = (double)src.u(r[b][s], c);
                use(a);
            }
    };
    if (lo >= hi) return;
    load(lo, raw[0]);
    for (int64_t j0 = lo; j0 < hi; j0 += 2 * STEP) {
        if (j0 + STEP < hi) load(j0 + STEP, raw[1]);
        spend(raw[0]);
        if (j0 + STEP >= hi) break;
        if (j0 + 2 * STEP < hi) load(j0 + 2 * STEP, raw[0]);
        spend(raw[1]);
    }
}

// Adds the waves' tiles, in their order, and stores them: tile t, register v, lane l at
// out[256 t + 64 v + l].
template <int N> __device__ __forceinline__ void store_tiles(const d4 (&acc)[N], double* s, double* out) {
    const int lane = lane_id(), w = wave_id();
#pragma unroll
    for (int k = 1; k < kWaves; ++k) {
        if (w == k) {
#pragma unroll
            for (int t = 0; t < N; ++t)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    double* p = s + 256 * t + 64 * v + lane;
                    *p = k == 1 ? acc[t][v] : *p + acc[t][v];
                }
        }
        __syncthreads();
    }
    if (w == 0) {
#pragma unroll
        for (int t = 0; t < N; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) gst(out + 256 * t + 64 * v + lane, acc[t][v] + s[256 * t + 64 * v + lane]);
    }
}

// One workgroup: one piece of one matrix; its blocks on and above the diagonal.  A wave
// takes 64 UN columns of the long side at a time, loaded as the apply launch does (whole
// cache lines: straight into operands, 64 bytes a row or 4 an element, the loads were half
// as fast) and turned round in its own part of LDS.
template <int NB> constexpr int gram_in_flight() { return NB == 1 ? 2 : 1; }
template <int NB> constexpr int gram_tall_pitch() { return NB == 1 ? 16 : 16 * NB + 16; }  // floats: LDS banks
constexpr int kGramWidePitch = 68;
template <int NB> constexpr int gram_floats() {  // of a wave's 64 columns
    return 64 * gram_tall_pitch<NB>() > 16 * NB * kGramWidePitch ? 64 * gram_tall_pitch<NB>() : 16 * NB * kGramWidePitch;
}
template <int NB> constexpr size_t gram_lds() { return (size_t)kWaves * gram_in_flight<NB>() * gram_floats<NB>() * 4; }

template <int NB, bool WIDE, typename SRC, int T>
__device__ __forceinline__ void gram_piece(const SRC& src, const Place& q, int64_t lo, int64_t hi, float* s_u, d4 (&acc)[T]) {
    constexpr int UN = gram_in_flight<NB>(), F = gram_floats<NB>(), TP = gram_tall_pitch<NB>();
    const int lane = lane_id();
    for (int64_t j0 = lo + wave_id() * 64 * UN; j0 < hi; j0 += kWaves * 64 * UN) {
        typename SRC::Raw raw[UN][NB][4];
#pragma unroll
        for (int n = 0; n < UN; ++n)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    int64_t at;
                    const int nv = group_at<WIDE>(q, b, k, j0 + 64 * n, hi, lane, &at);
                    src.load4(at, nv, q.vec, raw[n][b][k]);
                }
#pragma unroll
        for (int n = 0; n < UN; ++n)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f32x4 u;
#pragma unroll
                    for (int c = 0; c < 4; ++c) u[c] = src.u(raw[n][b][k], c);
                    const int at = WIDE ? (16 * b + 4 * k + lane / 16) * kGramWidePitch + 4 * (lane % 16)
                                        : (16 * k + lane % 16) * TP + 16 * b + 4 * (lane / 16);
                    *(f32x4*)(s_u + n * F + at) = u;
                }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int n = 0; n < UN; ++n)
#pragma unroll
            for (int s = 0; s < 4; ++s) {  // 16 columns
                float o[NB][4];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if constexpr (WIDE) {
                        const f32x4 r = *(const f32x4*)(s_u + n * F + (16 * b + lane % 16) * kGramWidePitch + 16 * s + 4 * (lane / 16));
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[b][c] = r[c];
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[b][c] = s_u[n * F + (16 * s + 4 * c + lane / 16) * TP + 16 * b + lane % 16];
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    int t = 0;
#pragma unroll
                    for (int bi = 0; bi < NB; ++bi)
#pragma unroll
                        for (int bj = bi; bj < NB; ++bj, ++t) acc[t] = mfma((double)o[bi][c], (double)o[bj][c], acc[t]);
                }
            }
        __builtin_amdgcn_wave_barrier();
    }
}
template <int NB, typename G> __device__ __forceinline__ void gram_item(const MuonArgs& a, int64_t item, float* s_all) {
    constexpr int T = NB * (NB + 1) / 2;
    static_assert(gram_lds<NB>() >= T * 256 * 8, "the waves' sums fit where the columns were");
    const MuDesc D = a.descs[gld(a.item_desc + item)];
    const int64_t local = item - D.item0;
    const Place q(D, local / D.chunks);
    const int64_t lo = local % D.chunks * a.chunk, end = lo + a.chunk, hi = end < q.d ? end : q.d;
    const FromState<G> src{(const G*)D.g, D.m, Mom(a)};
    float* s_u = s_all + wave_id() * gram_in_flight<NB>() * gram_floats<NB>();
    d4 acc[T];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = d4{0.0, 0.0, 0.0, 0.0};
    if (q.wide) gram_piece<NB, true>(src, q, lo, hi, s_u, acc);
    else gram_piece<NB, false>(src, q, lo, hi, s_u, acc);
    __syncthreads();
    store_tiles(acc, (double*)s_all, a.part + item * muon_part(NB));
}
template <int NB, typename G> __global__ __launch_bounds__(kNT, NB == 4 ? 2 : 1) void muon_gram(MuonArgs a) {
    extern __shared__ __align__(16) float s_all[];
    gram_item<NB, G>(a, blockIdx.x, s_all);
}

// Whether the products P u of an entry of P, with its 1 / norm, and of others like it stay within
// fp32: |X| is at most n max|P| |u|, and |u| 1 / norm at most 1.  (False for NaN.)
__device__ __forceinline__ bool in_range(double p, int n, double inv) { return fabs(p) * n <= 3.402823466e38 * inv; }

// ---- the n x n steps ----------------------------------------------------------------------

// Of block (bi, bj), element (row, col) as register v of lane l: (4 v + l / 16, l % 16).
__device__ __forceinline__ bool on_diagonal(int v, int lane) { return 4 * v + lane / 16 == lane % 16; }
// The place of that element's mirror image in block (bj, bi).
__device__ __forceinline__ int mirrored(int v, int lane) { return lane % 16 / 4 * 64 + lane % 16 % 4 * 16 + 4 * v + lane / 16; }

// One workgroup per matrix, a wave for each block (bi, bj) on or above the diagonal, which
// holds that block of every square matrix in registers; the operands of products lie in LDS
// whole, block after block as they are in registers (one block alone is its own operand).
// A workgroup of more waves (WAVES, shared with wider classes): those without a block only
// take part in the barriers, which every wave of a workgroup has to reach.
template <int NB, int WAVES = NB * (NB + 1) / 2> __device__ __forceinline__ void steps_matrix(const MuonArgs& a, int64_t mat, double* smem) {
    constexpr int SQ = NB * NB * 256, BLOCKS = NB * (NB + 1) / 2;
    double *LG = smem, *LQ = smem + SQ, *LP = smem + 2 * SQ, *LR = smem + 3 * SQ, *s_tr = smem + (NB > 1 ? 4 * SQ : 0);
    const int lane = lane_id(), w = wave_id();
    const bool on = WAVES == BLOCKS || w < BLOCKS;
    int bi = 0, bj = on ? w : 0;
    while (bj >= NB) bj -= NB - 1 - bi++;  // row after row: (0, 0 ..), (1, 1 ..), ..
    const MuDesc D = a.descs[gld(a.mat_desc + mat)];
    // the pieces' sums, in their order
    d4 g = {0.0, 0.0, 0.0, 0.0};
    if (on) {
        const double* part = a.part + (D.item0 + (mat - D.mat0) * D.chunks) * muon_part(NB) + w * 256 + lane;
#pragma unroll 4
        for (int c = 0; c < D.chunks; ++c, part += muon_part(NB))
#pragma unroll
            for (int v = 0; v < 4; ++v) g[v] += gld(part + 64 * v);
    }
    // |u|^2 is the trace
    double tr = 0.0;
    if (on && bi == bj) {
#pragma unroll
        for (int v = 0; v < 4; ++v) tr += on_diagonal(v, lane) ? g[v] : 0.0;
        tr = wave_sum(tr);
    }
    if (lane == 0 && on && bi == bj) s_tr[bi] = tr;
    __syncthreads();
    tr = 0.0;
#pragma unroll
    for (int b = 0; b < NB; ++b) tr += s_tr[b];
    const double inv = 1.0 / (sqrt(tr) + (double)a.eps);
    g *= inv * inv;

    d4 eye;
#pragma unroll
    for (int v = 0; v < 4; ++v) eye[v] = bi == bj && on_diagonal(v, lane) ? 1.0 : 0.0;
    // the block and its mirror image
    const auto put = [&](double* L, const d4& x) {
        if (NB > 1 && on) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                L[(bi * NB + bj) * 256 + 64 * v + lane] = x[v];
                if (bi != bj) L[(bj * NB + bi) * 256 + mirrored(v, lane)] = x[v];
            }
        }
    };
    // X Y of symmetric X, Y (all are polynomials of G): an operand's block (bi, bk) is read as (bk, bi)
    const auto mul = [&](const double* LX, const d4& x, const double* LY, const d4& y) {
        d4 r = {0.0, 0.0, 0.0, 0.0};
        if (!on) return r;
#pragma unroll
        for (int bk = 0; bk < NB; ++bk)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                if constexpr (NB > 1)
                    r = mfma(LX[(bk * NB + bi) * 256 + 64 * v + lane], LY[(bk * NB + bj) * 256 + 64 * v + lane], r);
                else
                    r = mfma(x[v], y[v], r);
            }
        return r;
    };
    const auto sync = [] {
        if constexpr (NB > 1) __syncthreads();
    };
    d4 p = eye;
    put(LG, g);
    sync();
    for (int k = 0; k < a.steps; ++k) {
        const d4 s = mul(LG, g, LG, g);
        const d4 q = a.coefs[k][0] * eye + a.coefs[k][1] * g + a.coefs[k][2] * s;
        put(LQ, q);
        sync();
        if (k + 1 == a.steps) {
            p = k == 0 ? q : mul(LP, p, LQ, q);
            break;
        }
        const d4 r = mul(LG, g, LQ, q);
        p = k == 0 ? q : mul(LP, p, LQ, q);
        put(LR, r);
        sync();  // R is there, G and P are read
        put(LP, p);
        g = mul(LR, r, LQ, q);
        put(LG, g);
        sync();
    }
    p *= inv;
    bool fin = true;
    if (on) {
        double* out = a.pm + mat * SQ;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            fin = fin && in_range(p[v], 16 * NB, inv);
            gst(out + (bi * NB + bj) * 256 + 64 * v + lane, p[v]);
            if (bi != bj) gst(out + (bj * NB + bi) * 256 + mirrored(v, lane), p[v]);
        }
    }
    const bool ok = __syncthreads_and(fin && __builtin_isfinite(tr));
    if (threadIdx.x == 0) {
        gst(a.bad + mat, ok ? 0 : 1);
        if (!ok) gst(a.err, 1);
    }
}
template <int NB> __global__ __launch_bounds__(NB*(NB + 1) / 2 * kWave) void muon_steps(MuonArgs a) {
    extern __shared__ double smem[];
    steps_matrix<NB>(a, blockIdx.x, smem);
}

// ---- the product and the update ---------------------------------------------------------

// A lane's tile of 64 of the long side (16 NB of the small): wide, rows 16 b + 4 v + l / 16
// of four columns 4 (l % 16) + c; tall, four of the small side 16 b + 4 (l / 16) + c of
// columns 16 x + l % 16.
struct Rate {
    float lr, keep;
    __device__ __forceinline__ Rate(const MuonArgs& a, const MuDesc& D) {
        const float l = a.lr_scale ? a.lr * gld(a.lr_scale) : a.lr;
        keep = (float)(1.0 - (double)l * (double)D.wd);
        lr = l * D.scale;
    }
};
// Four neighbours' weights, and what their four products make of them.
template <bool NT, typename P>
__device__ __forceinline__ void weights4(const MuDesc& D, int64_t at, int nv, bool vec, float (&w)[4]) {
    if (D.master) read4<NT>((const float*)D.master, at, nv, vec, w);
    else read4<NT>((const P*)D.p, at, nv, vec, w);
}
template <bool NT, typename P>
__device__ __forceinline__ void update4(const MuDesc& D, const Rate& r, int64_t at, int nv, bool vec, const double (&x)[4], float (&w)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = w[j] * r.keep - r.lr * (float)x[j];
    if (D.master) write4<NT>(D.master, at, nv, vec, w);
    write4<NT>((P*)D.p, at, nv, vec, w);
}
// Entry of a square matrix's block that a tall product's first operand wants: row
// sigma(l % 16), column 4 (l / 16) + k, of a symmetric block pair.
__device__ __forceinline__ int tall_entry(int k, int lane) {
    return lane / 16 * 64 + k * 16 + 4 * (lane % 4) + lane % 16 / 4;
}

// A wave's share of a piece: 64 UN of the long side at a time.  Loads do not move up past
// stores (the compiler cannot know that they differ), so all of g and m comes first (block
// by block a 64 x 64 tile waited eight times for memory, 30 us) and a block's weights come
// before its products, which hide them.
template <int NB, bool WIDE, typename P, typename G>
__device__ __forceinline__ void apply_piece(const MuonArgs& a, const MuDesc& D, const Place& q, int64_t lo, int64_t hi, const double* pm, const double* s_p) {
    constexpr int UN = NB == 1 ? 2 : 1;
    // an access covers whole cache lines (tall rows of more than one block take several)
    constexpr bool LAST = WIDE || NB == 1;
    const int lane = lane_id();
    double own[4];
    if constexpr (NB == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) own[k] = gld(pm + (WIDE ? 64 * k + lane : tall_entry(k, lane)));
    }
    const Mom mom(a);
    const Rate rate(a, D);
    for (int64_t j0 = lo + wave_id() * 64 * UN; j0 < hi; j0 += kWaves * 64 * UN) {
        float u[UN][NB][4][4], m[UN][NB][4][4];
        const auto each = [&](int n, int b, auto f) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                int64_t at;
                const int nv = group_at<WIDE>(q, b, k, j0 + 64 * n, hi, lane, &at);
                f(k, at, nv);
            }
        };
#pragma unroll
        for (int n = 0; n < UN; ++n)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                each(n, b, [&](int k, int64_t at, int nv) {
                    read4<LAST>((const G*)D.g, at, nv, q.vec, u[n][b][k]);
                    read4<LAST>((const float*)D.m, at, nv, q.vec, m[n][b][k]);
                });
#pragma unroll
        for (int n = 0; n < UN; ++n)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                each(n, b, [&](int k, int64_t at, int nv) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float g = u[n][b][k][c];
                        m[n][b][k][c] = mom.m(m[n][b][k][c], g);
                        u[n][b][k][c] = mom.u(m[n][b][k][c], g);
                    }
                    write4<LAST>(D.m, at, nv, q.vec, m[n][b][k]);
                });
#pragma unroll
        for (int n = 0; n < UN; ++n)
#pragma unroll
            for (int ib = 0; ib < NB; ++ib) {
                float w[4][4];
                each(n, ib, [&](int k, int64_t at, int nv) { weights4<LAST, P>(D, at, nv, q.vec, w[k]); });
                d4 acc[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c] = d4{0.0, 0.0, 0.0, 0.0};
#pragma unroll
                for (int kb = 0; kb < NB; ++kb)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        double x;
                        if constexpr (NB > 1) x = s_p[(kb * NB + ib) * 256 + (WIDE ? 64 * k + lane : tall_entry(k, lane))];
                        else x = own[k];
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[c] = mfma(x, (double)(WIDE ? u[n][kb][k][c] : u[n][kb][c][k]), acc[c]);
                    }
                each(n, ib, [&](int k, int64_t at, int nv) {
                    const double x[4] = {WIDE ? acc[0][k] : acc[k][0], WIDE ? acc[1][k] : acc[k][1], WIDE ? acc[2][k] : acc[k][2],
                                         WIDE ? acc[3][k] : acc[k][3]};
                    update4<LAST, P>(D, rate, at, nv, q.vec, x, w[k]);
                });
            }
    }
}

template <int NB, typename P, typename G> __device__ __forceinline__ void apply_item(const MuonArgs& a, int64_t item, double* s_p) {
    const MuDesc D = a.descs[gld(a.item_desc + item)];
    const int64_t local = item - D.item0, index = local / D.chunks, mat = D.mat0 + index;
    if (gld(a.bad + mat)) return;
    const Place q(D, index);
    const int64_t lo = local % D.chunks * a.chunk, end = lo + a.chunk, hi = end < q.d ? end : q.d;
    const double* pm = a.pm + mat * NB * NB * 256;
    if constexpr (NB > 1) {
        for (int i = threadIdx.x; i < NB * NB * 256; i += kNT) s_p[i] = gld(pm + i);
        __syncthreads();
    }
    if (q.wide) apply_piece<NB, true, P, G>(a, D, q, lo, hi, pm, s_p);
    else apply_piece<NB, false, P, G>(a, D, q, lo, hi, pm, s_p);
}
// One workgroup: one piece of one matrix, the last first (the pieces that the Gram launch
// read last are the likeliest to be in a cache still).
template <int NB, typename P, typename G> __global__ __launch_bounds__(kNT, NB == 4 ? 2 : 1) void muon_apply(MuonArgs a) {
    __shared__ double s_p[NB > 1 ? NB * NB * 256 : 1];
    apply_item<NB, P, G>(a, (int64_t)gridDim.x - 1 - blockIdx.x, s_p);
}

// ---- all classes in one set of launches --------------------------------------------------

// Tensors of several classes that together are few pieces: a launch each after the other
// would wait for one another's latencies (three tensors of odd sizes 133 us
// against 96 when they were joined; 76 now).
struct MuonAll {
    MuonArgs a[3];  // small sides up to 16, 32, 64; a class without matrices has no items
};
template <typename G> __global__ __launch_bounds__(kNT) void muon_gram_all(MuonAll m) {
    extern __shared__ __align__(16) float s_all[];
    int64_t i = blockIdx.x;  // the widest first: they take longest
    if (i < m.a[2].items) return gram_item<4, G>(m.a[2], i, s_all);
    i -= m.a[2].items;
    if (i < m.a[1].items) return gram_item<2, G>(m.a[1], i, s_all);
    gram_item<1, G>(m.a[0], i - m.a[1].items, s_all);
}
__global__ __launch_bounds__(10 * kWave) void muon_steps_all(MuonAll m) {
    extern __shared__ double smem[];
    int64_t i = blockIdx.x;
    if (i < m.a[2].mats) return steps_matrix<4>(m.a[2], i, smem);
    i -= m.a[2].mats;
    if (i < m.a[1].mats) return steps_matrix<2, 10>(m.a[1], i, smem);
    steps_matrix<1, 10>(m.a[0], i - m.a[1].mats, smem);
}
// WIDEST: some small side is above 32.  Such calls are few pieces of long chains: one wave a
// SIMD and no spilled registers (8 x 16 x 8192, 8 x 8192 x 16, 8192 x 64 and 8 x 64 x 4096 98 us,
// against 106 with two; without such sides two waves, 49 against 56).
template <bool WIDEST, typename P, typename G> __global__ __launch_bounds__(kNT, WIDEST ? 1 : 2) void muon_apply_all(MuonAll m) {
    __shared__ double s_p[WIDEST ? 16 * 256 : 4 * 256];
    int64_t i = blockIdx.x;
    if constexpr (WIDEST) {
        if (i < m.a[2].items) return apply_item<4, P, G>(m.a[2], i, s_p);
        i -= m.a[2].items;
    }
    if (i < m.a[1].items) return apply_item<2, P, G>(m.a[1], i, s_p);
    apply_item<1, P, G>(m.a[0], i - m.a[1].items, s_p);
}

// ---- small sides above 64 -----------------------------------------------------------------

// u of the big matrices' tensors, element by element.
template <typename G> __global__ __launch_bounds__(kNT) void muon_big_u(MuonArgs a) {
    const MuDesc D = a.descs[gld(a.item_desc + blockIdx.y)];
    const Mom mom(a);
    const int64_t n = D.count * D.n * D.d;
    for (int64_t i = ((int64_t)blockIdx.x * kNT + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * kNT * 4) {
        const int nv = n - i < 4 ? (int)(n - i) : 4;
        float g[4], m[4], u[4];
        read4((const G*)D.g, i, nv, D.vec != 0, g);
        read4((const float*)D.m, i, nv, D.vec != 0, m);
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = mom.u(mom.m(m[j], g[j]), g[j]);
        write4(D.u, i, nv, D.vec != 0, u);
    }
}

// A workgroup's matrix: the only one comes with the arguments, which saves two dependent
// loads in each of the launches.
__device__ __forceinline__ MuBig big_of(const MuonArgs& a, const int32_t* table) { return a.n_big == 1 ? a.only : a.big[gld(table)]; }

// The 64 x 64 blocks on and above the diagonal, by number: (bi, bj), bi <= bj.
__device__ __forceinline__ void pair_of(int t, int groups, int* bi, int* bj) {
    int i = 0;
    while (t >= groups - i) t -= groups - i++;
    *bi = i;
    *bj = i + t;
}
// One workgroup: one 64 x 64 of one piece's Gram matrix (rows 64 bi .., columns 64 bj ..),
// 16 rows of it a wave.
__global__ __launch_bounds__(kNT) void muon_big_gram(MuonArgs a) {
    const MuBig B = big_of(a, a.pair_big + blockIdx.x);
    const MuDesc D = a.descs[B.desc];
    const int groups = B.nb / 4, pairs = groups * (groups + 1) / 2;
    const int64_t local = (int64_t)blockIdx.x - B.part0;
    int bi, bj;
    pair_of((int)(local % pairs), groups, &bi, &bj);
    const Place q(D, B.index);
    const int64_t lo = local / pairs * kMuonBigChunk, end = lo + kMuonBigChunk, hi = end < q.d ? end : q.d;
    const FromScratch src{D.u};
    const int w = wave_id(), lane = lane_id();
    const int i0[5] = {64 * bi + 16 * w, 64 * bj, 64 * bj + 16, 64 * bj + 32, 64 * bj + 48};
    d4 acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = d4{0.0, 0.0, 0.0, 0.0};
    const auto add = [&](const double (&u)[5]) {
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = mfma(u[0], u[1 + t], acc[t]);
    };
    if (q.wide) long_side<true, 5, 1>(src, q, i0, lo, hi, add);
    else long_side<false, 5, 1>(src, q, i0, lo, hi, add);
    double* out = a.part + (int64_t)blockIdx.x * kMuonBigPart + w * 1024;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) gst(out + 256 * t + 64 * v + lane, acc[t][v]);
}

// The pieces' sums of one 16 x 16, in their order, into G and its mirror image.
__global__ __launch_bounds__(kNT) void muon_big_sum(MuonArgs a) {
    const MuBig B = big_of(a, a.sum_big + blockIdx.x / 16);
    const MuDesc D = a.descs[B.desc];
    const int groups = B.nb / 4, pairs = groups * (groups + 1) / 2, pair = gld(a.sum_pair + blockIdx.x / 16);
    int bi, bj;
    pair_of(pair, groups, &bi, &bj);
    double* G = a.square + B.off;
    const int t = blockIdx.x % 16, e = threadIdx.x, v = e / 64, lane = e % 64;
    const double* part = a.part + (B.part0 + pair) * kMuonBigPart + t * 256 + e;
    double s = 0.0;
#pragma unroll 16
    for (int c = 0; c < D.chunks; ++c, part += (int64_t)pairs * kMuonBigPart) s += gld(part);
    const int r = 4 * bi + t / 4, k = 4 * bj + t % 4;
    gst(G + ((int64_t)r * B.nb + k) * 256 + e, s);
    if (bi != bj) gst(G + ((int64_t)k * B.nb + r) * 256 + mirrored(v, lane), s);
}

// The trace of big matrix i and what follows from it, by one workgroup.
__device__ __forceinline__ void big_norm(const MuonArgs& a, int i) {
    __shared__ double s_tr[kWaves];
    const MuBig B = a.n_big == 1 ? a.only : a.big[i];
    const double* G = a.square + B.off;
    double tr = 0.0;
    for (int e = threadIdx.x; e < 16 * B.nb; e += kNT) {
        const int b = e / 16, r = e % 16;  // entry (r, r): register r / 4 of lane 16 (r % 4) + r
        tr += gld(G + ((int64_t)b * B.nb + b) * 256 + r / 4 * 64 + r % 4 * 16 + r);
    }
    tr = wave_sum(tr);
    if (lane_id() == 0) s_tr[wave_id()] = tr;
    __syncthreads();
    if (threadIdx.x != 0) return;
    tr = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) tr += s_tr[w];
    const double inv = 1.0 / (sqrt(tr) + (double)a.eps);
    gst(a.meta + 2 * i, inv);
    gst(a.meta + 2 * i + 1, inv * inv);
    const bool ok = __builtin_isfinite(tr);
    gst(a.bad + i, ok ? 0 : 1);
    if (!ok) gst(a.err, 1);
}

// Products of the square matrices, a workgroup per 16 x 16 block of the result: its waves
// take every fourth block of the sum and add up in their order.  G's factor 1 / norm^2 is
// applied in the first step, P's 1 / norm too.
//   MUL_S  S = G G  (in the first step the norms beside it, in workgroups of their own)
//   MUL_RP  R = G Q, and (blockIdx.y 1, or alone in the last step) P' = P Q
//   MUL_G  G' = R Q       with Q = a + b G + c S of this step's G and S
enum { MUL_S = 0, MUL_RP = 1, MUL_G = 2 };
struct BigMats {
    double *G, *S, *R, *P, *G2, *P2;
};
template <int MODE> __global__ __launch_bounds__(kNT) void muon_big_mul(MuonArgs a, BigMats M, int step, int only_p) {
    __shared__ double s_sum[kWaves][256];
    if (MODE == MUL_S && (int64_t)blockIdx.x >= a.n_mul) return big_norm(a, (int)(blockIdx.x - a.n_mul));
    const int bigi = a.n_big == 1 ? 0 : gld(a.mul_big + blockIdx.x);
    const MuBig B = a.n_big == 1 ? a.only : a.big[bigi];
    const int nb = B.nb, lane = lane_id(), w = wave_id(), block = a.n_big == 1 ? (int)blockIdx.x : gld(a.mul_at + blockIdx.x), bi = block / nb, bj = block % nb;
    const double f = MODE != MUL_S && step == 0 ? gld(a.meta + 2 * bigi + 1) : 1.0;  // G is f times what is stored
    const double ca = a.coefs[step][0], cb = a.coefs[step][1] * f, cc = a.coefs[step][2] * f * f;
    const auto frag = [&](const double* X, int r, int c, int v) { return gld(X + B.off + ((int64_t)r * nb + c) * 256 + 64 * v + lane); };
    const bool want_p = MODE == MUL_RP && (only_p || blockIdx.y == 1);
    double* out = (MODE == MUL_S ? M.S : MODE == MUL_G ? M.G2 : want_p ? M.P2 : M.R) + B.off + (int64_t)block * 256;
    if (want_p && step == 0) {
        if (w != 0) return;
        const double inv = gld(a.meta + 2 * bigi);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const double q = (bi == bj && on_diagonal(v, lane) ? ca : 0.0) + cb * frag(M.G, bi, bj, v) + cc * frag(M.S, bi, bj, v);
            gst(out + 64 * v + lane, inv * q);
            if (a.steps == 1 && !in_range(inv * q, 16 * nb, inv)) {
                gst(a.bad + bigi, 1);
                gst(a.err, 1);
            }
        }
        return;
    }
    const double* X = MODE == MUL_G ? M.R : want_p ? M.P : M.G;
    d4 r = {0.0, 0.0, 0.0, 0.0};
    // two blocks of the sum's loads at a time
    for (int b0 = w; b0 < nb; b0 += 2 * kWaves) {
        double x[2][4], y[2][4], z[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int bk = b0 + h * kWaves;
            if (bk < nb) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    x[h][v] = frag(X, bk, bi, v);
                    y[h][v] = frag(M.G, bk, bj, v);
                    z[h][v] = MODE == MUL_S ? 0.0 : frag(M.S, bk, bj, v);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int bk = b0 + h * kWaves;
            if (bk < nb) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    double q = y[h][v];
                    if constexpr (MODE != MUL_S) q = (bk == bj && on_diagonal(v, lane) ? ca : 0.0) + cb * q + cc * z[h][v];
                    r = mfma(x[h][v], q, r);
                }
            }
        }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) s_sum[w][64 * v + lane] = r[v];
    __syncthreads();
    double s = s_sum[0][threadIdx.x];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) s += s_sum[k][threadIdx.x];
    // (R and S keep the stored G's scale; G' takes it from R)
    gst(out + threadIdx.x, MODE == MUL_G ? s * f : s);
    if (MODE == MUL_RP && step + 1 == a.steps && !in_range(s, 16 * nb, gld(a.meta + 2 * bigi))) {
        gst(a.bad + bigi, 1);
        gst(a.err, 1);
    }
}

// One workgroup: 64 of the long side, 64 of the small side, 16 of them a wave.
template <bool WIDE, typename P, typename G>
__device__ __forceinline__ void big_apply(const MuonArgs& a, const MuDesc& D, const MuBig& B, const double* PM, int ib, int64_t j0) {
    const int lane = lane_id();
    const Place q(D, B.index);
    const int64_t hi = q.d;
    const Mom mom(a);
    const Rate rate(a, D);
    d4 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = d4{0.0, 0.0, 0.0, 0.0};
    const auto load = [&](int kb, float (&u)[4][4], double (&x)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            int64_t at;
            const int nv = group_at<WIDE>(q, kb, k, j0, hi, lane, &at);
            read4((const float*)D.u, at, nv, q.vec, u[k]);
            x[k] = gld(PM + B.off + ((int64_t)kb * B.nb + ib) * 256 + (WIDE ? 64 * k + lane : tall_entry(k, lane)));
        }
    };
    const auto spend = [&](const float (&u)[4][4], const double (&x)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[c] = mfma(x[k], (double)(WIDE ? u[k][c] : u[c][k]), acc[c]);
    };
    float u[2][4][4];
    double x[2][4];
    load(0, u[0], x[0]);
    for (int kb = 0; kb < B.nb; kb += 2) {  // nb is a multiple of 4
        load(kb + 1, u[1], x[1]);
        spend(u[0], x[0]);
        if (kb + 2 < B.nb) load(kb + 2, u[0], x[0]);
        spend(u[1], x[1]);
    }
    float g[4][4], m[4][4], wt[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        int64_t at;
        const int nv = group_at<WIDE>(q, ib, k, j0, hi, lane, &at);
        read4((const G*)D.g, at, nv, q.vec, g[k]);
        read4((const float*)D.m, at, nv, q.vec, m[k]);
        weights4<false, P>(D, at, nv, q.vec, wt[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        int64_t at;
        const int nv = group_at<WIDE>(q, ib, k, j0, hi, lane, &at);
#pragma unroll
        for (int c = 0; c < 4; ++c) m[k][c] = mom.m(m[k][c], g[k][c]);
        write4(D.m, at, nv, q.vec, m[k]);
        const double y[4] = {WIDE ? acc[0][k] : acc[k][0], WIDE ? acc[1][k] : acc[k][1], WIDE ? acc[2][k] : acc[k][2],
                             WIDE ? acc[3][k] : acc[k][3]};
        update4<false, P>(D, rate, at, nv, q.vec, y, wt[k]);
    }
}
template <typename P, typename G> __global__ __launch_bounds__(kNT) void muon_big_apply(MuonArgs a, const double* PM) {
    const int bigi = a.n_big == 1 ? 0 : gld(a.out_big + blockIdx.x);
    if (gld(a.bad + bigi)) return;
    const MuBig B = a.n_big == 1 ? a.only : a.big[bigi];
    const MuDesc D = a.descs[B.desc];
    const int groups = B.nb / 4, at = gld(a.out_at + blockIdx.x), ib = at % groups * 4 + wave_id();
    const int64_t j0 = (int64_t)(at / groups) * 64;
    if (D.wide) big_apply<true, P, G>(a, D, B, PM, ib, j0);
    else big_apply<false, P, G>(a, D, B, PM, ib, j0);
}

// ---- launches ---------------------------------------------------------------------------

constexpr size_t steps_lds(int nb) { return nb > 1 ? (size_t)(4 * nb * nb * 256 + nb) * 8 : 64; }

template <int NB, typename P, typename G> hipError_t launch_class(const MuonArgs& a, hipStream_t s) {
    const dim3 items((unsigned)a.items), n(kNT);
    hipLaunchKernelGGL((muon_gram<NB, G>), items, n, gram_lds<NB>(), s, a);
    hipLaunchKernelGGL((muon_steps<NB>), dim3((unsigned)a.mats), dim3(NB * (NB + 1) / 2 * kWave), steps_lds(NB), s, a);
    hipLaunchKernelGGL((muon_apply<NB, P, G>), items, n, 0, s, a);
    return hipGetLastError();
}
template <typename P, typename G> hipError_t launch_pg(const MuonArgs (&a)[3], hipStream_t s) {
    const int64_t items = a[0].items + a[1].items + a[2].items, mats = a[0].mats + a[1].mats + a[2].mats;
    const int classes = (a[0].items > 0) + (a[1].items > 0) + (a[2].items > 0);
    if (classes > 1 && items <= kMuonFewItems) {
        MuonAll m;
        for (int k = 0; k < 3; ++k) m.a[k] = a[k];
        const bool wide = a[2].items > 0;
        const size_t gl = wide ? gram_lds<4>() : gram_lds<2>(), sl = wide ? steps_lds(4) : steps_lds(2);
        hipLaunchKernelGGL((muon_gram_all<G>), dim3((unsigned)items), dim3(kNT), gl, s, m);
        hipLaunchKernelGGL(muon_steps_all, dim3((unsigned)mats), dim3(10 * kWave), sl, s, m);
        if (wide) hipLaunchKernelGGL((muon_apply_all<true, P, G>), dim3((unsigned)items), dim3(kNT), 0, s, m);
        else hipLaunchKernelGGL((muon_apply_all<false, P, G>), dim3((unsigned)items), dim3(kNT), 0, s, m);
        return hipGetLastError();
    }
    hipError_t e = hipSuccess;
    if (a[0].items) e = launch_class<1, P, G>(a[0], s);
    if (a[1].items && e == hipSuccess) e = launch_class<2, P, G>(a[1], s);
    if (a[2].items && e == hipSuccess) e = launch_class<4, P, G>(a[2], s);
    return e;
}
template <typename P, typename G> hipError_t launch_big_pg(const MuonArgs& a, int64_t u_elems, hipStream_t s) {
    const dim3 n(kNT);
    const int64_t ublocks = (u_elems + 4 * kNT - 1) / (4 * kNT);
    hipLaunchKernelGGL((muon_big_u<G>), dim3((unsigned)(ublocks < 4096 ? ublocks : 4096), (unsigned)a.items), n, 0, s, a);
    hipLaunchKernelGGL(muon_big_gram, dim3((unsigned)a.n_pair), n, 0, s, a);
    hipLaunchKernelGGL(muon_big_sum, dim3((unsigned)(a.n_sum * 16)), n, 0, s, a);
    double* at = a.square;
    BigMats M{at, at + a.sq, at + 2 * a.sq, at + 3 * a.sq, at + 4 * a.sq, at + 5 * a.sq};
    const unsigned mul = (unsigned)a.n_mul;
    for (int k = 0; k < a.steps; ++k) {
        const bool last = k + 1 == a.steps;
        hipLaunchKernelGGL((muon_big_mul<MUL_S>), dim3(k == 0 ? mul + (unsigned)a.n_big : mul), n, 0, s, a, M, k, 0);
        hipLaunchKernelGGL((muon_big_mul<MUL_RP>), dim3(mul, last ? 1 : 2), n, 0, s, a, M, k, last ? 1 : 0);
        if (!last) hipLaunchKernelGGL((muon_big_mul<MUL_G>), dim3(mul), n, 0, s, a, M, k, 0);
        std::swap(M.P, M.P2);
        std::swap(M.G, M.G2);
    }
    hipLaunchKernelGGL((muon_big_apply<P, G>), dim3((unsigned)a.n_out), n, 0, s, a, (const double*)M.P);
    return hipGetLastError();
}

}  // namespace

hipError_t prepare_muon() {
    hipError_t e = hipSuccess;
    for (const void* f : {(const void*)muon_steps<4>, (const void*)muon_steps_all})
        if (e == hipSuccess) e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)steps_lds(4));
    for (const void* f : {(const void*)muon_gram<4, float>, (const void*)muon_gram<4, uint16_t>, (const void*)muon_gram_all<float>,
                          (const void*)muon_gram_all<uint16_t>})
        if (e == hipSuccess) e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)gram_lds<4>());
    return e;
}

hipError_t launch_muon(const MuonArgs (&a)[3], int p_dtype, int g_dtype, hipStream_t s) {
    for (int k = 0; k < 3; ++k)
        if (!grid_fits(a[k].items, kNT) || !grid_fits(a[k].mats, 10 * kWave)) return hipErrorInvalidConfiguration;
    if (p_dtype == 0) return g_dtype == 0 ? launch_pg<float, float>(a, s) : launch_pg<float, uint16_t>(a, s);
    return g_dtype == 0 ? launch_pg<uint16_t, float>(a, s) : launch_pg<uint16_t, uint16_t>(a, s);
}
hipError_t launch_muon_big(const MuonArgs& a, int64_t u_elems, int p_dtype, int g_dtype, hipStream_t s) {
    if (!grid_fits(a.n_pair, kNT) || !grid_fits(a.n_mul + a.n_big, kNT) || !grid_fits(a.n_sum * 16, kNT) || !grid_fits(a.n_out, kNT)) return hipErrorInvalidConfiguration;
    if (p_dtype == 0) return g_dtype == 0 ? launch_big_pg<float, float>(a, u_elems, s) : launch_big_pg<float, uint16_t>(a, u_elems, s);
    return g_dtype == 0 ? launch_big_pg<uint16_t, float>(a, u_elems, s) : launch_big_pg<uint16_t, uint16_t>(a, u_elems, s);
}

}  // namespace dlm
