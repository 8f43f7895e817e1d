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
// The step count t lives on the device, so that a captured step counts on
// replay, and once per chunk: a workgroup reads, uses and moves its own, and none
// waits for another.  (One count moved by the last workgroup to end, found by a
// ticket, took 8.0 ms where this takes 1.8 -- 322 million weights, 78 thousand
// workgroups whose atomics on one address queue up past their XCD's L2; moved by
// a one-thread launch before the step it took the same time and a second launch.)
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
// Measured: 322 million bf16 weights with fp32 masters and moments in 448 tensors,
// 1.69 ms, 5.7 TB/s (a large copy reaches 4.7); one layer's 10 million 54 us; with
// 8-bit moments 48 us, where the binary64 codes and hashes bound it as much as the
// memory; 80 million fp32 weights with 8-bit moments 306 us (420 with the read-back's
// 114), 4.2 TB/s.
//
// An element whose new v is not finite in fp32 (a gradient that is infinite, NaN,
// or past 1.8e19 / sqrt(1 - b2)) is left as it was, with 8-bit moments its whole
// block, and the handle's error word is set.
#include "adamw.hpp"
#include "gfx950.hpp"
#include "internal.hpp"

namespace dlm {

namespace {

constexpr int kNT = 256;
constexpr int kPer = kAdamChunk / (kNT * 4);  // rounds of four elements per thread
constexpr int kReadPer = 4;  // quads per thread of the read-back
static_assert(kAdamBlock == 4 * kWave, "a wave's four elements per lane are one block");

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Four consecutive elements as loaded.  Loads and stores are nontemporal: every
// array is touched once, and kept out of the caches it leaves them to whatever
// comes next (322 million weights 1.69 ms against 1.79, one layer's 54 us against 63).
template <typename T> struct Raw4;
template <> struct Raw4<float> { u32x4 r; };
template <> struct Raw4<uint16_t> { u32x2 r; };

__device__ __forceinline__ void load4(Raw4<float>& o, const float* p) { o.r = __builtin_nontemporal_load((gcptr<u32x4>)p); }
__device__ __forceinline__ void load4(Raw4<uint16_t>& o, const uint16_t* p) { o.r = __builtin_nontemporal_load((gcptr<u32x2>)p); }
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
    const u32x4 o = {__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    __builtin_nontemporal_store(o, (gptr<u32x4>)p);
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&f)[4]) {
    const u32x2 o = {pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3])};
    __builtin_nontemporal_store(o, (gptr<u32x2>)p);
}
// One element (tensors whose pointers or end do not allow four).
__device__ __forceinline__ float load1(const float* p) { return gld(p); }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf_to_f(gld(p)); }
__device__ __forceinline__ void store1(float* p, float f) { gst(p, f); }
__device__ __forceinline__ void store1(uint16_t* p, float f) { gst(p, f_to_bf(f)); }

// Four elements i .. i+3 of an array of n: one access (FULL: the workgroup's
// whole chunk is inside and aligned), else element by element, 0 past the end.
template <bool FULL, typename T> __device__ __forceinline__ void get4(const T* p, int64_t i, int64_t n, float (&f)[4]) {
    if constexpr (FULL) {
        Raw4<T> r;
        load4(r, p + i);
        widen(r, f);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = i + j < n ? load1(p + i + j) : 0.f;
    }
}
template <bool FULL, typename T>
__device__ __forceinline__ void put4(T* p, int64_t i, int64_t n, const float (&f)[4]) {
    if constexpr (FULL) {
        store4(p + i, f);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) store1(p + i + j, f[j]);
    }
}
template <bool FULL> __device__ __forceinline__ uint32_t get4b(const uint8_t* p, int64_t i, int64_t n) {
    if constexpr (FULL) return gld((const uint32_t*)(p + i));
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (i + j < n) w |= (uint32_t)gld(p + i + j) << (8 * j);
    return w;
}
template <bool FULL> __device__ __forceinline__ void put4b(uint8_t* p, int64_t i, int64_t n, uint32_t w) {
    if constexpr (FULL) {
        gst((uint32_t*)(p + i), w);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) gst(p + i + j, (uint8_t)(w >> (8 * j)));
    }
}

struct Step {
    uint32_t t;
    float gs, lr, keep, ic1, rc2;  // gradient scale, rate, 1 - lr wd, 1 / (1 - b1^t), sqrt(1 / (1 - b2^t))
};
// Counts the chunk's step and shares what its elements need (called by the whole
// workgroup, once its loads are out: one thread works, the others wait).
__device__ __forceinline__ Step begin_step(const AdamArgs& a, float wd, Step* s_step) {
    if (threadIdx.x == 0) {
        Step s;
        s.t = (uint32_t)gld(a.steps + blockIdx.x) + 1u;
        gst(a.steps + blockIdx.x, (int32_t)s.t);
        s.gs = a.grad_scale ? gld(a.grad_scale) : 1.f;
        s.lr = a.lr_scale ? a.lr * gld(a.lr_scale) : a.lr;
        s.keep = (float)(1.0 - (double)s.lr * (double)wd);
        s.ic1 = (float)(-1.0 / expm1((double)s.t * a.lb1));
        s.rc2 = (float)sqrt(-1.0 / expm1((double)s.t * a.lb2));
        *s_step = s;
    }
    __syncthreads();
    return *s_step;
}

__device__ __forceinline__ float updated(float w, float m, float v, const Step& s, float eps) {
    const float step = (m * s.ic1) / (sqrtf(v) * s.rc2 + eps);
    return w * s.keep - s.lr * step;
}

// ---- fp32 moments --------------------------------------------------------------

template <bool FULL, typename P, typename G>
__device__ __forceinline__ void step_f32(const AdamArgs& a, const AdDesc& D, Step* s_step) {
    const float b1 = (float)a.beta1, b2 = (float)a.beta2, r1 = (float)(1.0 - a.beta1), r2 = (float)(1.0 - a.beta2);
    const int64_t base = ((int64_t)blockIdx.x - D.chunk0) * kAdamChunk + 4 * threadIdx.x;
    P* __restrict__ p = (P*)D.p;
    const G* __restrict__ gp = (const G*)D.g;
    float* __restrict__ mp = (float*)D.m;
    float* __restrict__ vp = (float*)D.v;
    bool bad = false;
    float g[kPer][4], m[kPer][4], v[kPer][4], w[kPer][4];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t i = base + k * kNT * 4;
        get4<FULL>(gp, i, D.n, g[k]);
        get4<FULL>((const float*)mp, i, D.n, m[k]);
        get4<FULL>((const float*)vp, i, D.n, v[k]);
        if (D.master) get4<FULL>((const float*)D.master, i, D.n, w[k]);
        else get4<FULL>((const P*)p, i, D.n, w[k]);
    }
    const Step s = begin_step(a, D.wd, s_step);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t i = base + k * kNT * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float gj = g[k][j] * s.gs;
            // g'^2 may pass fp32 where v's share of it does not
            const float g2 = gj * gj, inc = __builtin_isfinite(g2) ? r2 * g2 : (r2 * gj) * gj;
            const float mj = fmaf(b1, m[k][j], r1 * gj), vj = fmaf(b2, v[k][j], inc);
            const bool fin = __builtin_isfinite(vj);
            if (!fin) {
                bad = true;
            } else {
                m[k][j] = mj;
                v[k][j] = vj;
                w[k][j] = updated(w[k][j], mj, vj, s, a.eps);
            }
        }
        put4<FULL>(mp, i, D.n, m[k]);
        put4<FULL>(vp, i, D.n, v[k]);
        if (D.master) put4<FULL>(D.master, i, D.n, w[k]);
        put4<FULL>(p, i, D.n, w[k]);
    }
    if (bad) gst(a.err, 1);
}

// A chunk that lies whole in its tensor, with pointers for four elements at a time.
__device__ __forceinline__ bool whole(const AdDesc& D) {
    return D.vec && ((int64_t)blockIdx.x - D.chunk0 + 1) * kAdamChunk <= D.n;
}

template <typename P, typename G> __global__ __launch_bounds__(kNT) void adamw_f32(AdamArgs a) {
    const AdDesc D = a.descs[a.chunk_tensor[blockIdx.x]];
    __shared__ Step s_step;
    if (whole(D)) step_f32<true, P, G>(a, D, &s_step);
    else step_f32<false, P, G>(a, D, &s_step);
}

// ---- 8-bit moments -------------------------------------------------------------

// The 32-bit finaliser of MurmurHash3 (A. Appleby, public domain).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
    x = (x ^ (x >> 13)) * 0xC2B2AE35u;
    return x ^ (x >> 16);
}

constexpr double kM2 = 127.0 * 127.0, kV4 = 255.0 * 255.0 * 255.0 * 255.0;

// The codes' values over their block's scale: sign(q) (q / 127)^2 and (c / 255)^4,
// 1 exactly at the top (a block's largest moment goes on as it was stored: its
// decayed value often lies next to the middle of two fp32 scales, and the last
// bit of binary64 decides).  A table of each in LDS, looked up by code.
__device__ __forceinline__ void value_tables(double* s_m, double* s_v) {
    for (int i = threadIdx.x; i < 256; i += blockDim.x) {
        const int q = (int8_t)i;
        s_m[i] = (double)(q * (q < 0 ? -q : q)) / kM2;
        s_v[i] = (double)((uint32_t)(i * i) * (uint32_t)(i * i)) / kV4;
    }
    __syncthreads();
}

// The code of x = (|m| / ms) 127^2: with c = floor(sqrt x), c, or c + 1 where x
// lies further up its step of 2c + 1 than the noise u = (2h + 1) / 2^17.  So it
// is the first n with x <= border(n) = n^2 + u (2n + 1), borders and x times 2^17
// being whole numbers below 2^32 (x rounded up, which changes no comparison).
// The fp32 root, made a little smaller, starts at c or c - 1: two comparisons.
__device__ __forceinline__ uint32_t m_code(double x, uint32_t h) {
    const uint32_t xi = (uint32_t)__builtin_ceil(x * 131072.0);
    const uint32_t c = (uint32_t)(__builtin_amdgcn_sqrtf((float)x) * 0.9999997f);
    const uint32_t u = 2 * h + 1;
    const uint32_t b0 = ((c * c) << 17) + u * (2 * c + 1), b1 = (((c + 1) * (c + 1)) << 17) + u * (2 * c + 3);
    return c + (xi > b0 ? 1u : 0u) + (xi > b1 ? 1u : 0u);
}
// The same for v with steps between fourth powers; root = sqrt x over shrink^2 (a
// power of two, times the little).
__device__ __forceinline__ double pow4(uint32_t c) {
    const double s = (double)(c * c);
    return s * s;
}
__device__ __forceinline__ uint32_t v_code(double x, float root, float shrink, uint32_t h) {
    const uint32_t c = (uint32_t)(__builtin_amdgcn_sqrtf(root) * shrink);
    const double u = (double)(2 * h + 1) * (1.0 / 131072.0);
    const double p0 = pow4(c), p1 = pow4(c + 1), p2 = pow4(c + 2);
    return c + (x > __builtin_fma(u, p1 - p0, p0) ? 1u : 0u) + (x > __builtin_fma(u, p2 - p1, p1) ? 1u : 0u);
}

// The largest of the wave's values (none a NaN), as a scalar.
__device__ __forceinline__ float wave_max(float v) {
    int x = __float_as_int(v);
#define DLM_STEP(CTRL, ROWS) \
    x = __float_as_int(fmaxf(__int_as_float(x), __int_as_float(__builtin_amdgcn_update_dpp(x, x, CTRL, ROWS, 0xf, false))))
    DLM_STEP(0xB1, 0xf);   // quad_perm: within pairs
    DLM_STEP(0x4E, 0xf);   // between pairs
    DLM_STEP(0x141, 0xf);  // half rows mirrored
    DLM_STEP(0x140, 0xf);  // rows mirrored
    DLM_STEP(0x142, 0xa);  // row 0 to 1, 2 to 3
    DLM_STEP(0x143, 0xc);  // rows 0..1 to 2..3
#undef DLM_STEP
    return __int_as_float(__builtin_amdgcn_readlane(x, kWave - 1));
}

template <bool FULL, typename P, typename G>
__device__ __forceinline__ void step_q8(const AdamArgs& a, const AdDesc& D, int tensor, double* s_m, double* s_v, Step* s_step) {
    constexpr int kBlocks = kAdamChunk / kAdamBlock / (kNT / kWave);  // blocks per wave
    const int lane = lane_id();
    const int64_t blk0 = ((int64_t)blockIdx.x - D.chunk0) * (kAdamChunk / kAdamBlock) + wave_id() * kBlocks;
    P* __restrict__ p = (P*)D.p;
    const G* __restrict__ gp = (const G*)D.g;
    const double r1 = 1.0 - a.beta1, r2 = 1.0 - a.beta2;
    bool bad = false;
    float g[kBlocks][4], w[kBlocks][4], ms[kBlocks], vs[kBlocks];
    uint32_t q[kBlocks], c[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const int64_t blk = blk0 + b, i = blk * kAdamBlock + 4 * lane;
        const bool in = FULL || blk * kAdamBlock < D.n;
        get4<FULL>(gp, i, D.n, g[b]);
        q[b] = get4b<FULL>((const uint8_t*)D.m, i, D.n);
        c[b] = get4b<FULL>((const uint8_t*)D.v, i, D.n);
        ms[b] = in ? gld(D.ms + blk) : 0.f;
        vs[b] = in ? gld(D.vs + blk) : 0.f;
        if (D.master) get4<FULL>((const float*)D.master, i, D.n, w[b]);
        else get4<FULL>((const P*)p, i, D.n, w[b]);
    }
    value_tables(s_m, s_v);
    const Step s = begin_step(a, D.wd, s_step);
    const uint32_t key_t = mix(mix(a.seed + s.t * 0x9E3779B1u) + (uint32_t)tensor * 0x85EBCA77u);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const int64_t blk = blk0 + b, i = blk * kAdamBlock + 4 * lane;
        if (!FULL && blk * kAdamBlock >= D.n) break;  // the same for the whole wave
        double m[4], v[4];
        float mm = 0.f, vm = 0.f;
        bool fin = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double gj = (double)(g[b][j] * s.gs);
            const double mo = (double)ms[b] * s_m[(q[b] >> (8 * j)) & 255u], vo = (double)vs[b] * s_v[(c[b] >> (8 * j)) & 255u];
            m[j] = a.beta1 * mo + r1 * gj;
            v[j] = a.beta2 * vo + r2 * (gj * gj);
            const float vj = (float)v[j];
            mm = fmaxf(mm, fabsf((float)m[j]));
            vm = fmaxf(vm, vj);
            fin = fin && vj < __builtin_huge_valf();  // false for a NaN too
        }
        if (__ballot(!fin)) {  // a NaN does not reach the maxima: the ballot decides
            bad = true;
            continue;
        }
        mm = wave_max(mm);
        vm = wave_max(vm);
        const double mi = mm > 0.f ? kM2 / (double)mm : 0.0, vi = vm > 0.f ? kV4 / (double)vm : 0.0;
        // sqrt(v / (1 - b2^t)) from the root of v's place in the block.  Beside a large
        // vm the place of a v that counts may lie below fp32's normal numbers: its
        // root is taken 2^46 times as large (vm <= 1: such a v is 0 in fp32 too)
        const bool high = vm > 1.f;
        const double up = high ? 0x1p92 : 1.0;
        const float shrink = high ? 0.9999997f * 0x1p-23f : 0.9999997f;
        const float vroot = sqrtf(vm) * s.rc2 * (1.f / (255.f * 255.f)) * (high ? 0x1p-46f : 1.f);
        const uint32_t key = mix(key_t + (uint32_t)blk * 0xC2B2AE3Du);
        const uint32_t least = vm > 0.f ? 1u : 0u;
        uint32_t nq = 0, nc = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t h = mix(key + (uint32_t)(4 * lane + j) * 0x9E3779B1u);
            const double xm = fabs(m[j]) * mi, xv = v[j] * vi;
            const uint32_t k = m_code(xm < kM2 ? xm : kM2, h & 0xffffu);
            nq |= ((m[j] < 0.0 ? 0u - k : k) & 255u) << (8 * j);
            const double xc = xv < kV4 ? xv : kV4;
            const float root = __builtin_amdgcn_sqrtf((float)(xc * up));
            uint32_t cv = v_code(xc, root, shrink, h >> 16);
            cv = cv < least && v[j] > 0.0 ? least : cv;
            nc |= cv << (8 * j);
            // the quotient by the reciprocal's estimate (1 ulp): the step is lr of a weight
            const float step = ((float)m[j] * s.ic1) * __builtin_amdgcn_rcpf(root * vroot + a.eps);
            w[b][j] = w[b][j] * s.keep - s.lr * step;
        }
        put4b<FULL>((uint8_t*)D.m, i, D.n, nq);
        put4b<FULL>((uint8_t*)D.v, i, D.n, nc);
        if (lane == 0) {
            gst(D.ms + blk, mm);
            gst(D.vs + blk, vm);
        }
        if (D.master) put4<FULL>(D.master, i, D.n, w[b]);
        put4<FULL>(p, i, D.n, w[b]);
    }
    if (bad) gst(a.err, 1);
}

template <typename P, typename G> __global__ __launch_bounds__(kNT) void adamw_q8(AdamArgs a) {
    const int tensor = a.chunk_tensor[blockIdx.x];
    const AdDesc D = a.descs[tensor];
    __shared__ double s_m[256], s_v[256];
    __shared__ Step s_step;
    if (whole(D)) step_q8<true, P, G>(a, D, tensor, s_m, s_v, &s_step);
    else step_q8<false, P, G>(a, D, tensor, s_m, s_v, &s_step);
}

// The moments that the codes stand for.
template <bool FULL>
__device__ __forceinline__ void read_state(const int8_t* m, const uint8_t* v, const float* ms, const float* vs, int64_t i,
                                           int64_t n, float* m_out, float* v_out, const double* s_m, const double* s_v) {
    const int64_t blk = i / kAdamBlock;
    const uint32_t q = get4b<FULL>((const uint8_t*)m, i, n), c = get4b<FULL>(v, i, n);
    const double mu = (double)gld(ms + blk), vu = (double)gld(vs + blk);
    float mo[4], vo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        mo[j] = (float)(mu * s_m[(q >> (8 * j)) & 255u]);
        vo[j] = (float)(vu * s_v[(c >> (8 * j)) & 255u]);
    }
    put4<FULL>(m_out, i, n, mo);
    put4<FULL>(v_out, i, n, vo);
}
__global__ __launch_bounds__(kNT) void adamw_read(const int8_t* __restrict__ m, const uint8_t* __restrict__ v,
                                                  const float* __restrict__ ms, const float* __restrict__ vs, int64_t n,
                                                  int vec, float* __restrict__ m_out, float* __restrict__ v_out) {
    __shared__ double s_m[256], s_v[256];
    value_tables(s_m, s_v);
#pragma unroll
    for (int k = 0; k < kReadPer; ++k) {
        const int64_t i = (((int64_t)blockIdx.x * kReadPer + k) * kNT + threadIdx.x) * 4;
        if (i >= n) return;
        if (vec && i + 4 <= n) read_state<true>(m, v, ms, vs, i, n, m_out, v_out, s_m, s_v);
        else read_state<false>(m, v, ms, vs, i, n, m_out, v_out, s_m, s_v);
    }
}

template <typename P, typename G> hipError_t launch_pg(const AdamArgs& a, int bits, hipStream_t s) {
    if (bits == 32) hipLaunchKernelGGL((adamw_f32<P, G>), dim3((unsigned)a.n_chunks), dim3(kNT), 0, s, a);
    else hipLaunchKernelGGL((adamw_q8<P, G>), dim3((unsigned)a.n_chunks), dim3(kNT), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(const AdamArgs& a, int p_dtype, int g_dtype, int bits, hipStream_t s) {
    if (!grid_fits(a.n_chunks, kNT)) return hipErrorInvalidConfiguration;
    if (p_dtype == 0) return g_dtype == 0 ? launch_pg<float, float>(a, bits, s) : launch_pg<float, uint16_t>(a, bits, s);
    return g_dtype == 0 ? launch_pg<uint16_t, float>(a, bits, s) : launch_pg<uint16_t, uint16_t>(a, bits, s);
}

hipError_t launch_adamw_read_state(const int8_t* m, const uint8_t* v, const float* ms, const float* vs, int64_t n,
                                   float* m_out, float* v_out, hipStream_t s) {
    const int64_t blocks = (n + 4 * kNT * kReadPer - 1) / (4 * kNT * kReadPer);
    if (!grid_fits(blocks, kNT)) return hipErrorInvalidConfiguration;
    const uintptr_t all = (uintptr_t)m_out | (uintptr_t)v_out, codes = (uintptr_t)m | (uintptr_t)v;
    const int vec = (all & 15) == 0 && (codes & 3) == 0;
    hipLaunchKernelGGL(adamw_read, dim3((unsigned)blocks), dim3(kNT), 0, s, m, v, ms, vs, n, vec, m_out, v_out);
    return hipGetLastError();
}

}  // namespace dlm
