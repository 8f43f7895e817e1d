// The coefficients of the gradients' outer products, one (list tile, projection)
// per workgroup: a launch of its own, or workgroups of the expand's launch.
#pragma once

#include <type_traits>

#include "gfx950.hpp"
#include "internal.hpp"
#include "sgmm.hpp"

namespace dlm {
namespace {

constexpr int kCoefTerms = 3;
constexpr int kKB = 512;  // elements of one coefficient block: 16 ranks x kGradTile slots, 1 KB

__device__ __forceinline__ bool rejected(const SgGradArgs& a) { return gld((const int32_t*)(a.ws + a.G.L.hdr) + SG_ERR) != 0; }

// Two neighbouring ranks' K slices, eight loads in flight, added in order.
__device__ __forceinline__ void slice_sum(const float* p, int64_t stride, int n, float (&o)[2]) {
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    for (int k0 = 0; k0 < n; k0 += 8) {
        f32x2_t v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = gld((const f32x2_t*)(p + (k0 + k < n ? k0 + k : n - 1) * stride));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k0 + k >= n) break;
            o[0] = k0 + k ? o[0] + v[k].x : v[k].x;
            o[1] = k0 + k ? o[1] + v[k].y : v[k].y;
        }
    }
}

// x as three bf16 terms (hi, the rest's hi, ...), one to each array's [rank][slot].
__device__ __forceinline__ void put_terms(uint16_t (*s_c)[16][kGradTile], int rank, int slot, float x) {
#pragma unroll
    for (int m = 0; m < kCoefTerms; ++m) {
        const uint16_t t = f_to_bf(x);
        s_c[m][rank][slot] = t;
        x -= bf_to_f(t);
    }
}

// Eight threads per slot, 16 ranks at a time.  Padding ranks and
// slots get 0 (their v was never written: selected away, not multiplied).
template <bool BF> struct CoefLds {
    typedef typename std::conditional<BF, uint16_t, float>::type C;
    __attribute__((aligned(16))) C c[2 * (BF ? kCoefTerms : 1)][16][kGradTile];
};
template <bool BF>
__device__ __forceinline__ void coefs_tile(const SgGradArgs& a, int64_t tile, int prob, CoefLds<BF>& sm) {
    const SgLayout& L = a.G.L;
    if (tile * kGradTile >= gld((const int32_t*)(a.ws + a.G.eoff) + a.E)) return;
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
    typedef typename CoefLds<BF>::C C;
    constexpr int kTerms = BF ? kCoefTerms : 1;
    auto& s_c = sm.c;
    float dot = 0.f;
    C* coef = (C*)(a.ws + a.G.coef);
    const int64_t list_tiles = a.G.cap / kGradTile, nb = RPAD / 16;
    for (int b = 0; b < nb; ++b) {
        const int rho = 16 * b + 2 * j;
        float u[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
        if (live && rho < r) {
            slice_sum(vu + rho, stride, P.n_ks_u, u);
            slice_sum(vw + rho, stride, P.n_ks_w, w);
            if (rho + 1 >= r) u[1] = w[1] = 0.f;
        }
        dot = fmaf(u[0], w[0], dot);
        dot = fmaf(u[1], w[1], dot);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if constexpr (BF) {
                put_terms(s_c, 2 * j + k, s, c * w[k]);
                put_terms(s_c + kTerms, 2 * j + k, s, c * u[k]);
            } else {
                s_c[0][2 * j + k][s] = c * w[k];
                s_c[1][2 * j + k][s] = c * u[k];
            }
        }
        __syncthreads();
        constexpr int W = 16 / (int)sizeof(C), kRow = kGradTile / W;  // 16-byte stores per rank row
        for (int i = tid; i < 2 * kTerms * 16 * kRow; i += 256) {
            const int m = i / (16 * kRow), rr = i / kRow % 16, o = W * (i % kRow), side = m / kTerms;
            const int64_t at = ((((int64_t)prob * 2 + side) * list_tiles + tile) * nb + b) * kTerms + m % kTerms;
            st128(coef + at * kKB + rr * kGradTile + o, *(const u32x4*)&s_c[m][rr][o]);
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

}  // namespace
}  // namespace dlm
