// One AdamW step over many tensors in one launch:
//   m <- b1 m + (1 - b1) g      v <- b2 v + (1 - b2) g^2
//   w <- w (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
// with w the fp32 master where there is one (the parameter is then its
// rounding) and the parameter itself otherwise.  The step is a stream over the
// tensors, bound by memory: every element of every array is read and written
// once, four elements per lane and access.  One workgroup takes one
// kAdamChunk-element chunk of one tensor, found through a table of chunks, so
// tensors of any sizes share a launch.
//
// The step count t lives on the device (a captured step counts on replay): a
// one-thread launch moves it and works out the bias corrections, and the step
// reads them with ordinary cached loads.  Counting in the step itself, by a
// ticket that the last workgroup to end finds complete, took 8.0 ms where this
// takes 1.8 (322 million weights, 78 thousand workgroups): every workgroup's
// atomics on one address go past the XCD's L2 and queue up.
//
// 8-bit moments.  Blocks of 256 consecutive elements share an fp32 scale, the
// block's largest |m| and largest v:
//   m = ms sign(q) (q / 127)^2, q = -127..127      v = vs (c / 255)^4, c = 0..255
// The powers spend the codes where moments lie: steps of 1.6% at the top, and a
// range of 1.6e4 for m and 4.2e9 for v.  Rounding is stochastic: of the two
// neighbouring codes the upper is taken with the probability that makes the
// stored value's mean the exact one.  To the nearest code v would never decay:
// a step takes 0.1% off it (b2 = 0.999), half a code is 0.8%.  The noise is a
// hash of (seed, t, tensor, block, element), so a step is reproducible.  A
// positive v keeps a code of at least 1: sqrt(v) is then at least 1.5e-5 of the
// block's largest while m's smallest nonzero code is 6.2e-5 of its own, so no
// element's m / sqrt(v) grows past about four times the block's.
// Which code is taken turns on values next to a border, so the moments are
// binary64 between their codes (a binary64 FMA issues like an unpacked fp32
// one here); the weights take fp32 roundings of them.
//
// An element whose new v is not finite in fp32 (a gradient that is infinite,
// NaN, or past 1.8e19) is left as it was, with 8-bit moments its whole block,
// and the handle's error word is set.
#include "adamw.hpp"
#include "gfx950.hpp"
#include "internal.hpp"

namespace dlm {

namespace {

constexpr int kNT = 256;
constexpr int kPer = kAdamChunk / (kNT * 4);  // rounds of four elements per thread
static_assert(kAdamBlock == 4 * kWave, "a wave's four elements per lane are one block");

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Four consecutive elements as loaded.
template <typename T> struct Raw4;
template <> struct Raw4<float> { u32x4 r; };
template <> struct Raw4<uint16_t> { u32x2 r; };

__device__ __forceinline__ void load4(Raw4<float>& o, const float* p) { o.r = *(gcptr<u32x4>)p; }
__device__ __forceinline__ void load4(Raw4<uint16_t>& o, const uint16_t* p) { o.r = *(gcptr<u32x2>)p; }
__device__ __forceinline__ void widen(const Raw4<float>& o, float (&f)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(o.r[j]);
}
__device__ __forceinline__ void widen(const Raw4<uint16_t>& o, float (&f)[4]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        f[2 * j] = bf_lo(o.r[j]);
        f[2 * j + 1] = bf_hi(o.r[j]);
    }
}
__device__ __forceinline__ void store4(float* p, const float (&f)[4]) {
    *(gptr<u32x4>)p = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&f)[4]) {
    *(gptr<u32x2>)p = u32x2{pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3])};
}
// One element (tensors whose pointers or end do not allow four).
__device__ __forceinline__ float load1(const float* p) { return gld(p); }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf_to_f(gld(p)); }
__device__ __forceinline__ void store1(float* p, float f) { gst(p, f); }
__device__ __forceinline__ void store1(uint16_t* p, float f) { gst(p, f_to_bf(f)); }

// Four elements i .. i+3 of an array of n: one access where vec allows it, else
// element by element, 0 past the end.
template <typename T> __device__ __forceinline__ void get4(const T* p, int64_t i, int64_t n, bool vec, float (&f)[4]) {
    if (vec && i + 4 <= n) {
        Raw4<T> r;
        load4(r, p + i);
        widen(r, f);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = i + j < n ? load1(p + i + j) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void put4(T* p, int64_t i, int64_t n, bool vec, const float (&f)[4]) {
    if (vec && i + 4 <= n) {
        store4(p + i, f);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) store1(p + i + j, f[j]);
    }
}
__device__ __forceinline__ uint32_t get4b(const uint8_t* p, int64_t i, int64_t n, bool vec) {
    if (vec && i + 4 <= n) return gld((const uint32_t*)(p + i));
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (i + j < n) w |= (uint32_t)gld(p + i + j) << (8 * j);
    return w;
}
__device__ __forceinline__ void put4b(uint8_t* p, int64_t i, int64_t n, bool vec, uint32_t w) {
    if (vec && i + 4 <= n) {
        gst((uint32_t*)(p + i), w);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) gst(p + i + j, (uint8_t)(w >> (8 * j)));
    }
}

// A step's first launch, one thread: counts the step and works out what its
// elements share.
__global__ void adamw_begin(AdamArgs a) {
    AdWords w = *a.words;
    w.t += 1;
    w.gs = a.grad_scale ? *a.grad_scale : 1.f;
    w.lr = a.lr_scale ? a.lr * *a.lr_scale : a.lr;
    w.ic1 = (float)(-1.0 / expm1((double)w.t * a.lb1));
    w.ic2 = (float)(-1.0 / expm1((double)w.t * a.lb2));
    *a.words = w;
}

struct Step {
    uint32_t t;
    float gs, lr, keep, ic1, ic2;  // keep = 1 - lr wd
};
__device__ __forceinline__ Step step_of(const AdamArgs& a, float wd) {
    const AdWords w = *a.words;
    return Step{(uint32_t)w.t, w.gs, w.lr, (float)(1.0 - (double)w.lr * (double)wd), w.ic1, w.ic2};
}

__device__ __forceinline__ float updated(float w, float m, float v, const Step& s, float eps) {
    const float step = (m * s.ic1) / (sqrtf(v * s.ic2) + eps);
    return w * s.keep - s.lr * step;
}

// ---- fp32 moments --------------------------------------------------------------

template <typename P, typename G>
__global__ __launch_bounds__(kNT) void adamw_f32(AdamArgs a) {
    const AdDesc D = a.descs[a.chunk_tensor[blockIdx.x]];
    const Step s = step_of(a, D.wd);
    const float b1 = (float)a.beta1, b2 = (float)a.beta2, r1 = (float)(1.0 - a.beta1), r2 = (float)(1.0 - a.beta2);
    const int64_t base = ((int64_t)blockIdx.x - D.chunk0) * kAdamChunk + 4 * threadIdx.x;
    const bool vec = D.vec;
    P* __restrict__ p = (P*)D.p;
    const G* __restrict__ gp = (const G*)D.g;
    float* __restrict__ mp = (float*)D.m;
    float* __restrict__ vp = (float*)D.v;
    bool bad = false;
    float g[kPer][4], m[kPer][4], v[kPer][4], w[kPer][4];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t i = base + k * kNT * 4;
        get4(gp, i, D.n, vec, g[k]);
        get4(mp, i, D.n, vec, m[k]);
        get4(vp, i, D.n, vec, v[k]);
        if (D.master) get4(D.master, i, D.n, vec, w[k]);
        else get4(p, i, D.n, vec, w[k]);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t i = base + k * kNT * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float gj = g[k][j] * s.gs;
            const float mj = fmaf(b1, m[k][j], r1 * gj), vj = fmaf(b2, v[k][j], r2 * (gj * gj));
            const bool fin = __builtin_isfinite(vj);
            if (!fin) {
                bad = true;
            } else {
                m[k][j] = mj;
                v[k][j] = vj;
                w[k][j] = updated(w[k][j], mj, vj, s, a.eps);
            }
        }
        put4(mp, i, D.n, vec, m[k]);
        put4(vp, i, D.n, vec, v[k]);
        if (D.master) put4(D.master, i, D.n, vec, w[k]);
        put4(p, i, D.n, vec, w[k]);
    }
    if (bad) gst(&a.words->err, 1);
}

// ---- 8-bit moments -------------------------------------------------------------

// The 32-bit finaliser of MurmurHash3 (A. Appleby, public domain).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
    x = (x ^ (x >> 13)) * 0xC2B2AE35u;
    return x ^ (x >> 16);
}

constexpr double kM2 = 127.0 * 127.0, kV4 = 255.0 * 255.0 * 255.0 * 255.0;

__device__ __forceinline__ double m_value(int q, double unit) { return unit * (double)(q * (q < 0 ? -q : q)); }
__device__ __forceinline__ double v_value(uint32_t c, double unit) { return unit * (double)((c * c) * (c * c)); }

// The code of x = (|m| / ms) 127^2: floor(sqrt x), or one more where x lies
// further up its step of 2c + 1 than the noise (2h + 1) / 2^17.  The fp32 root
// may miss the floor by one next to a square; it is put right exactly.
__device__ __forceinline__ int m_code(double x, uint32_t h) {
    int c = (int)sqrtf((float)x);
    double d = x - (double)(c * c);
    if (d < 0.0) {
        --c;
        d = x - (double)(c * c);
    } else if (d >= (double)(2 * c + 1)) {
        ++c;
        d = x - (double)(c * c);
    }
    return c + (d * 131072.0 > (double)((2 * (int)h + 1) * (2 * c + 1)) ? 1 : 0);
}
// The same for v with steps between fourth powers.
__device__ __forceinline__ double pow4(int c) {
    const double s = (double)(c * c);
    return s * s;
}
__device__ __forceinline__ uint32_t v_code(double x, uint32_t h, bool positive) {
    int c = (int)sqrtf(sqrtf((float)x));
    double lo = pow4(c), hi = pow4(c + 1);
    if (x < lo) {
        --c;
        hi = lo;
        lo = pow4(c);
    } else if (x >= hi) {
        ++c;
        lo = hi;
        hi = pow4(c + 1);
    }
    c += (x - lo) * 131072.0 > (double)(2 * (int)h + 1) * (hi - lo) ? 1 : 0;
    return (uint32_t)(positive && c < 1 ? 1 : c);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
    return v;
}

template <typename P, typename G>
__global__ __launch_bounds__(kNT) void adamw_q8(AdamArgs a) {
    const int tensor = a.chunk_tensor[blockIdx.x];
    const AdDesc D = a.descs[tensor];
    const Step s = step_of(a, D.wd);
    constexpr int kBlocks = kAdamChunk / kAdamBlock / (kNT / kWave);  // blocks per wave
    const int lane = lane_id();
    const int64_t blk0 = ((int64_t)blockIdx.x - D.chunk0) * (kAdamChunk / kAdamBlock) + wave_id() * kBlocks;
    const bool vec = D.vec;
    P* __restrict__ p = (P*)D.p;
    const G* __restrict__ gp = (const G*)D.g;
    const double r1 = 1.0 - a.beta1, r2 = 1.0 - a.beta2;
    bool bad = false;
    float g[kBlocks][4], w[kBlocks][4], ms[kBlocks], vs[kBlocks];
    uint32_t q[kBlocks], c[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const int64_t blk = blk0 + b, i = blk * kAdamBlock + 4 * lane;
        const bool in = blk * kAdamBlock < D.n;
        get4(gp, i, D.n, vec, g[b]);
        q[b] = get4b((const uint8_t*)D.m, i, D.n, vec);
        c[b] = get4b((const uint8_t*)D.v, i, D.n, vec);
        ms[b] = in ? gld(D.ms + blk) : 0.f;
        vs[b] = in ? gld(D.vs + blk) : 0.f;
        if (D.master) get4(D.master, i, D.n, vec, w[b]);
        else get4(p, i, D.n, vec, w[b]);
    }
    const uint32_t key_t = mix(mix(a.seed + s.t * 0x9E3779B1u) + (uint32_t)tensor * 0x85EBCA77u);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const int64_t blk = blk0 + b, i = blk * kAdamBlock + 4 * lane;
        if (blk * kAdamBlock >= D.n) break;  // the same for the whole wave
        const double mu = (double)ms[b] / kM2, vu = (double)vs[b] / kV4;
        double m[4], v[4];
        float mm = 0.f, vm = 0.f;
        bool fin = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double gj = (double)(g[b][j] * s.gs);
            m[j] = a.beta1 * m_value((int)(int8_t)(q[b] >> (8 * j)), mu) + r1 * gj;
            v[j] = a.beta2 * v_value((c[b] >> (8 * j)) & 255u, vu) + r2 * (gj * gj);
            mm = fmaxf(mm, fabsf((float)m[j]));
            vm = fmaxf(vm, (float)v[j]);
            fin = fin && __builtin_isfinite((float)v[j]);
        }
        if (__ballot(!fin)) {  // a NaN does not reach the maxima: the ballot decides
            bad = true;
            continue;
        }
        mm = wave_max(mm);
        vm = wave_max(vm);
        const double mi = mm > 0.f ? kM2 / (double)mm : 0.0, vi = vm > 0.f ? kV4 / (double)vm : 0.0;
        const uint32_t key = mix(key_t + (uint32_t)blk * 0xC2B2AE3Du);
        uint32_t nq = 0, nc = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t h = mix(key + (uint32_t)(4 * lane + j) * 0x9E3779B1u);
            const double xm = fabs(m[j]) * mi, xv = v[j] * vi;
            int k = m_code(xm < kM2 ? xm : kM2, h & 0xffffu);
            k = m[j] < 0.0 ? -k : k;
            nq |= ((uint32_t)k & 255u) << (8 * j);
            nc |= v_code(xv < kV4 ? xv : kV4, h >> 16, v[j] > 0.0 && vm > 0.f) << (8 * j);
            w[b][j] = updated(w[b][j], (float)m[j], (float)v[j], s, a.eps);
        }
        put4b((uint8_t*)D.m, i, D.n, vec, nq);
        put4b((uint8_t*)D.v, i, D.n, vec, nc);
        if (lane == 0) {
            gst(D.ms + blk, mm);
            gst(D.vs + blk, vm);
        }
        if (D.master) put4(D.master, i, D.n, vec, w[b]);
        put4(p, i, D.n, vec, w[b]);
    }
    if (bad) gst(&a.words->err, 1);
}

// The moments that the codes stand for.
__global__ __launch_bounds__(kNT) void adamw_read(const int8_t* __restrict__ m, const uint8_t* __restrict__ v,
                                                  const float* __restrict__ ms, const float* __restrict__ vs, int64_t n,
                                                  int vec, float* __restrict__ m_out, float* __restrict__ v_out) {
    const int64_t i = ((int64_t)blockIdx.x * kNT + threadIdx.x) * 4;
    if (i >= n) return;
    const int64_t blk = i / kAdamBlock;
    const uint32_t q = get4b((const uint8_t*)m, i, n, vec), c = get4b(v, i, n, vec);
    const double mu = (double)gld(ms + blk) / kM2, vu = (double)gld(vs + blk) / kV4;
    float mo[4], vo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        mo[j] = (float)m_value((int)(int8_t)(q >> (8 * j)), mu);
        vo[j] = (float)v_value((c >> (8 * j)) & 255u, vu);
    }
    put4(m_out, i, n, vec, mo);
    put4(v_out, i, n, vec, vo);
}

template <typename P, typename G> hipError_t launch_pg(const AdamArgs& a, int bits, hipStream_t s) {
    if (bits == 32) hipLaunchKernelGGL((adamw_f32<P, G>), dim3((unsigned)a.n_chunks), dim3(kNT), 0, s, a);
    else hipLaunchKernelGGL((adamw_q8<P, G>), dim3((unsigned)a.n_chunks), dim3(kNT), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(const AdamArgs& a, int p_dtype, int g_dtype, int bits, hipStream_t s) {
    if (!grid_fits(a.n_chunks, kNT)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(adamw_begin, dim3(1), dim3(1), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p_dtype == 0) return g_dtype == 0 ? launch_pg<float, float>(a, bits, s) : launch_pg<float, uint16_t>(a, bits, s);
    return g_dtype == 0 ? launch_pg<uint16_t, float>(a, bits, s) : launch_pg<uint16_t, uint16_t>(a, bits, s);
}

hipError_t launch_adamw_read_state(const int8_t* m, const uint8_t* v, const float* ms, const float* vs, int64_t n,
                                   float* m_out, float* v_out, hipStream_t s) {
    const int64_t blocks = (n + 4 * kNT - 1) / (4 * kNT);
    if (!grid_fits(blocks, kNT)) return hipErrorInvalidConfiguration;
    const uintptr_t all = (uintptr_t)m_out | (uintptr_t)v_out, codes = (uintptr_t)m | (uintptr_t)v;
    const int vec = (all & 15) == 0 && (codes & 3) == 0;
    hipLaunchKernelGGL(adamw_read, dim3((unsigned)blocks), dim3(kNT), 0, s, m, v, ms, vs, n, vec, m_out, v_out);
    return hipGetLastError();
}

}  // namespace dlm
