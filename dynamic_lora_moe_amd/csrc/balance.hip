// The router's balance loss over packed sequences, its counts, and its gradient.
//
//   p      softmax(l), or sigmoid(l) over its sum in the row, of the available experts
//   per sequence of n rows that have any:  c_e slots that chose e,  f_e = E c_e / (k n),
//   P_e = mean p_e,  balance = sum_e f_e P_e,  z = mean (log sum exp l)^2
//   loss   alpha mean balance, zeta mean z (over the sequences)
//   dl_e   p_e (1 - s_e) (u_e - sum_j u_j p_j) with u = alpha f / (S n), the choice held
//          (softmax: without 1 - s_e), and 2 zeta lse p_e / (S n) on top
//
// The gradient needs the counts but not the means, so each direction reads the
// logits once.  L lanes hold a row, eight experts each.  The forward launch adds p
// over a block's rows of one sequence, in binary64 (a lane has per L / 256 of them, as
// many as the batch makes it; fp32 sums cost as much), and stores the sums as a part; the
// second launch adds the parts in their order, and the last of its workgroups (a ticket
// that the first launch clears) adds the sequences: no atomics on values, the same bits
// every time.
// (One block of one sequence needs no second launch.)
//
// 16384 rows of 256 fp32 logits, sigmoid, 8 sequences: 14 us, 9 and 15 for the gradient that
// joins one that is there (3.4 TB/s; the forward's 1.2 are its waits: two waves a SIMD, whose
// next row is loaded once this one's sums are done, and a slot's logit once its idx is there).
// 256 rows of 8: 5.4 and 2.8, a launch and a chain of loads each.  512 blocks at most: the
// second launch reads every block's part, and more of them cost it what the first gains.
#include "balance.hpp"
#include "gfx950.hpp"
#include "internal.hpp"
#include "route.hpp"

namespace dlm {

namespace {

constexpr int kNT = 256;
constexpr int kV = 8;                // experts per lane
constexpr int kPiece = 16;           // experts of one sequence that a workgroup of the second launch adds
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float from(float v) { return v; }
__device__ __forceinline__ float from(uint16_t v) { return bf_to_f(v); }
// +inf counts as the largest fp32 value, NaN as not available, as for the routing.
__device__ __forceinline__ float clean(float l) { return l == l ? fminf(l, 3.402823466e38f) : -kInf; }

// The peer of a step of a reduction over L lanes: every lane ends with the same bits.
template <int STEP> __device__ __forceinline__ float peer(float v) {
    if constexpr (STEP > 8) return __shfl_xor(v, STEP, kWave);
    constexpr int ctrl = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
    const int x = __float_as_int(v);
    return __int_as_float(__builtin_amdgcn_update_dpp(x, x, ctrl, 0xf, 0xf, false));
}
template <int L> __device__ __forceinline__ float row_sum(float v) {
    if constexpr (L > 1) v += peer<1>(v);
    if constexpr (L > 2) v += peer<2>(v);
    if constexpr (L > 4) v += peer<4>(v);
    if constexpr (L > 8) v += peer<8>(v);
    if constexpr (L > 16) v += peer<16>(v);
    if constexpr (L > 32) v += peer<32>(v);
    return v;
}
template <int L> __device__ __forceinline__ float row_max(float v) {
    if constexpr (L > 1) v = fmaxf(v, peer<1>(v));
    if constexpr (L > 2) v = fmaxf(v, peer<2>(v));
    if constexpr (L > 4) v = fmaxf(v, peer<4>(v));
    if constexpr (L > 8) v = fmaxf(v, peer<8>(v));
    if constexpr (L > 16) v = fmaxf(v, peer<16>(v));
    if constexpr (L > 32) v = fmaxf(v, peer<32>(v));
    return v;
}

// e^x for x <= 0 as 2^(x log2 e): the product's rounding is carried to the result
// to first order (by itself it would cost |x| 2^-24 of it).  0 below 2^-126.
__device__ __forceinline__ float exp_neg(float x) {
    const float t = x * 1.44269502f;
    const float lo = fmaf(x, 1.44269502f, -t) + x * 1.92596303e-8f;
    const float e = __builtin_amdgcn_exp2f(t);
    return x > -88.f ? fmaf(e, lo * 0.693147182f, e) : 0.f;
}

// Lane `lane`'s experts of a row: eight neighbours, loaded 16 bytes at a time.
template <typename T> struct Raw {
    u32x4 c[kV * sizeof(T) / 16];
};
template <typename T> __device__ __forceinline__ void load_raw(const T* row, int e0, int E, Raw<T>& r) {
    constexpr int W = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < kV / W; ++i) r.c[i] = e0 + i * W < E ? ld128(row + e0 + i * W) : u32x4{0u, 0u, 0u, 0u};
}
__device__ __forceinline__ void unpack(const Raw<float>& r, float (&f)[kV]) {
#pragma unroll
    for (int v = 0; v < kV; ++v) f[v] = __uint_as_float(r.c[v / 4][v % 4]);
}
__device__ __forceinline__ void unpack(const Raw<uint16_t>& r, float (&f)[kV]) {
#pragma unroll
    for (int v = 0; v < kV; ++v) f[v] = v & 1 ? bf_hi(r.c[0][v / 2]) : bf_lo(r.c[0][v / 2]);
}
// Values of a row that the lane holds, as stored (0 past E).
template <typename T> __device__ __forceinline__ void load_values(const T* row, int e0, int E, bool vec, float (&f)[kV]) {
    if (vec) {
        Raw<T> r;
        load_raw(row, e0, E, r);
        unpack(r, f);
    } else {
#pragma unroll
        for (int v = 0; v < kV; ++v) f[v] = e0 + v < E ? from(gld(row + e0 + v)) : 0.f;
    }
}
template <typename T> __device__ __forceinline__ void load_logits(const T* row, int e0, int E, bool vec, float (&l)[kV]) {
    load_values(row, e0, E, vec, l);
#pragma unroll
    for (int v = 0; v < kV; ++v) l[v] = e0 + v < E ? clean(l[v]) : -kInf;
}

struct Row {
    bool live;
    float lse;  // softmax only
};
// p of the row's experts, and for the sigmoid 1 - s.  A row without an available expert has p = 0.
template <int L, int SCORE> __device__ __forceinline__ Row row_probs(const float (&l)[kV], float (&p)[kV], float (&slope)[kV]) {
    float m = l[0];
#pragma unroll
    for (int v = 1; v < kV; ++v) m = fmaxf(m, l[v]);
    m = row_max<L>(m);
    Row r;
    r.live = m > -kInf;
    const float top = r.live ? m : 0.f;
    float sum = 0.f;
    if constexpr (SCORE == kRouteSoftmax) {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            p[v] = exp_neg(l[v] - top);
            sum += p[v];
        }
    } else {
        // s = (l >= 0 ? 1 : z) / (1 + z), z = e^-|l|.  A row of very negative logits takes
        // e^(l - top) above the line instead: the common factor cancels in p
        const bool small = __any(r.live && top < -40.f);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const float z = exp_neg(-fabsf(l[v])), over = __builtin_amdgcn_rcpf(1.f + z);
            float up = l[v] >= 0.f ? 1.f : z;
            if (small && top < -40.f) up = exp_neg(l[v] - top);
            p[v] = up * over;
            slope[v] = (l[v] >= 0.f ? z : 1.f) * over;
            sum += p[v];
        }
    }
    sum = row_sum<L>(sum);
    const float inv = r.live ? 1.f / sum : 0.f;
#pragma unroll
    for (int v = 0; v < kV; ++v) p[v] *= inv;
    r.lse = r.live ? top + __logf(sum) : 0.f;
    return r;
}

// Sequence q's rows, kept inside the batch whatever the offsets hold.
__device__ __forceinline__ int64_t first_row(const BalanceArgs& a, int q) {
    if (!a.offsets) return q == 0 ? 0 : a.T;
    const int64_t t = gld(a.offsets + q);
    return t < 0 ? 0 : t > a.T ? a.T : t;
}
// The last sequence that begins at or before row t (0 if none does): of a lane's own row,
__device__ __forceinline__ int sequence_of(const BalanceArgs& a, int64_t t) {
    if (!a.offsets) return 0;
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (gld(a.offsets + mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
// and of a row that the wave shares, 64 places at a time (all lanes there).
__device__ __forceinline__ int sequence_of_wave(const BalanceArgs& a, int64_t t) {
    if (!a.offsets) return 0;
    int lo = 0, n = a.S;  // it is one of lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + kWave - 1) / kWave, q = lo + lane_id() * step;
        const uint64_t below = __ballot(lane_id() * step < n && gld(a.offsets + (q < a.S ? q : a.S - 1)) <= t);
        const int i = below ? 63 - __builtin_clzll(below) : 0;
        lo += i * step;
        n = n - i * step < step ? n - i * step : step;
    }
    return uniform(lo);
}

// A row's lanes' values, added over the wave's rows (in binary64, a fixed order): every
// lane l ends with the sum of lanes l % L.
template <int L> __device__ __forceinline__ double rows_sum(double v) {
#pragma unroll
    for (int o = L; o < kWave; o *= 2) v += __shfl_xor(v, o, kWave);
    return v;
}
// Sums over the workgroup, in a fixed order; the result in every thread.
__device__ __forceinline__ double block_sum(double v, double* s) {
    v = wave_sum(v);
    __syncthreads();
    if (lane_id() == 0) s[wave_id()] = v;
    __syncthreads();
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kNT / kWave; ++w) sum += s[w];
    return sum;
}

// One workgroup: `per` rows, kNT / L at a time, sequence by sequence.  The only one of the
// only sequence finishes it by itself.
template <typename T, int L, int SCORE> __global__ __launch_bounds__(kNT) void balance_parts(BalanceArgs a) {
    constexpr int TPB = kNT / L, WAVES = kNT / kWave;
    __shared__ double s_p[WAVES][L * kV];
    __shared__ int s_cnt[kRouteMaxExperts];
    __shared__ double s_z[WAVES], s_n[WAVES];
    const int tid = threadIdx.x, tl = tid / L, lane = tid % L, e0 = lane * kV, E = a.E, k = a.k;
    const int64_t b0 = (int64_t)blockIdx.x * a.per, b1 = b0 + a.per < a.T ? b0 + a.per : a.T;
    const bool alone = a.S == 1 && gridDim.x == 1;
    if (blockIdx.x == 0 && tid == 0) gst(a.ticket, 0u);
    for (int q = sequence_of_wave(a, b0); q < a.S; ++q) {
        const int64_t q0 = first_row(a, q), q1 = first_row(a, q + 1);
        if (q0 >= b1 && !alone) break;
        const int64_t lo = q0 > b0 ? q0 : b0, hi = q1 < b1 ? q1 : b1;
        if (lo >= hi && !alone) continue;
        for (int e = tid; e < E; e += kNT) s_cnt[e] = 0;
        __syncthreads();
        double acc[kV] = {};
        double z = 0.0;
        int n = 0;
        for (int64_t t = lo + tl; t < hi; t += TPB) {
            const T* row = (const T*)a.logits + t * a.ld;
            float l[kV], p[kV], slope[kV];
            load_logits(row, e0, E, a.vec, l);
            for (int s = lane; s < k; s += L) {
                const int e = gld(a.idx + t * k + s);
                if ((uint32_t)e < (uint32_t)E && clean(from(gld(row + e))) > -kInf) atomicAdd(&s_cnt[e], 1);
            }
            const Row r = row_probs<L, SCORE>(l, p, slope);
#pragma unroll
            for (int v = 0; v < kV; ++v) acc[v] += (double)p[v];
            n += r.live ? 1 : 0;
            if constexpr (SCORE == kRouteSoftmax) z += (double)r.lse * (double)r.lse;
        }
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const double sum = rows_sum<L>(acc[v]);
            if (tid % kWave < L) s_p[wave_id()][e0 + v] = sum;
        }
        const double zw = rows_sum<L>(z), nw = rows_sum<L>((double)n);  // (whole numbers below 2^53)
        if (tid % kWave == 0) {
            s_z[wave_id()] = zw;
            s_n[wave_id()] = nw;
        }
        __syncthreads();
        double zs = 0.0, ns = 0.0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            zs += s_z[w];
            ns += s_n[w];
        }
        const int64_t slot = (int64_t)blockIdx.x + q;
        double part = 0.0;
        for (int e = tid; e < E; e += kNT) {
            double sum = 0.0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) sum += s_p[w][e];
            if (alone) {
                const double mean = ns > 0.0 ? sum / ns : 0.0;
                gst(a.probs + e, (float)mean);
                gst(a.counts + e, s_cnt[e]);
                if (ns > 0.0) part += (double)E * s_cnt[e] / ((double)k * ns) * mean;
            } else {
                gst(a.part_p + slot * E + e, sum);
                gst(a.part_c + slot * E + e, s_cnt[e]);
            }
        }
        if (alone) {
            const double bal = block_sum(part, s_z);
            if (tid == 0) {
                gst(a.rows, (int)ns);
                gst(a.loss, (float)((double)a.alpha * bal));
                gst(a.loss + 1, ns > 0.0 ? (float)((double)a.zeta * (zs / ns)) : 0.f);
            }
            return;
        }
        if (tid == 0) {
            gst(a.part_z + slot, zs);
            gst(a.part_n + slot, (int)ns);
        }
        __syncthreads();  // the shared sums are read
    }
}

// One workgroup: kPiece experts of one sequence, kNT / kPiece runs over its parts.
__global__ __launch_bounds__(kNT) void balance_sum(BalanceArgs a) {
    constexpr int RUNS = kNT / kPiece;
    __shared__ double s_p[RUNS][kPiece];
    __shared__ int s_c[RUNS][kPiece];
    __shared__ double s_w[kNT / kWave];
    __shared__ int s_last;
    const int tid = threadIdx.x, E = a.E;
    const int pieces = (E + kPiece - 1) / kPiece;
    const int q = blockIdx.x / pieces, piece = blockIdx.x % pieces;
    const int64_t q0 = first_row(a, q), q1 = first_row(a, q + 1);
    const int64_t f = q0 / a.per, l = q1 > q0 ? (q1 - 1) / a.per + 1 : f;  // its blocks
    const int e = piece * kPiece + tid % kPiece, run = tid / kPiece;
    double p = 0.0;
    int c = 0;
    if (e < E) {
#pragma unroll 8
        for (int64_t b = f + run; b < l; b += RUNS) {
            p += gld(a.part_p + (b + q) * E + e);
            c += gld(a.part_c + (b + q) * E + e);
        }
    }
    double z = 0.0;
    int n = 0;
#pragma unroll 4
    for (int64_t b = f + tid; b < l; b += kNT) {
        z += gld(a.part_z + b + q);
        n += gld(a.part_n + b + q);
    }
    s_p[run][tid % kPiece] = p;
    s_c[run][tid % kPiece] = c;
    z = block_sum(z, s_w);
    n = (int)block_sum((double)n, s_w);  // whole numbers below 2^53
    double part = 0.0;
    if (tid < kPiece && e < E) {
#pragma unroll
        for (int j = 1; j < RUNS; ++j) {
            p += s_p[j][tid];
            c += s_c[j][tid];
        }
        const double mean = n > 0 ? p / n : 0.0;
        gst(a.probs + (int64_t)q * E + e, (float)mean);
        gst(a.counts + (int64_t)q * E + e, c);
        if (n > 0) part = (double)E * c / ((double)a.k * n) * mean;
    }
    part = block_sum(part, s_w);
    if (tid == 0) {
        double* mine = a.seq + 2 * (int64_t)blockIdx.x;
        if (piece == 0) gst(a.rows + q, n);
        __hip_atomic_store(mine, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(mine + 1, piece == 0 && n > 0 ? z / n : 0.0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    double bal = 0.0, zz = 0.0;
    for (uint32_t i = tid; i < gridDim.x; i += kNT) {
        bal += __hip_atomic_load(a.seq + 2 * (int64_t)i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        zz += __hip_atomic_load(a.seq + 2 * (int64_t)i + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    bal = block_sum(bal, s_w);
    zz = block_sum(zz, s_w);
    if (tid == 0) {
        gst(a.loss, (float)((double)a.alpha * bal / a.S));
        gst(a.loss + 1, (float)((double)a.zeta * zz / a.S));
    }
}

// One workgroup: `per` rows, kNT / L at a time.
template <typename T, int L, int SCORE> __global__ __launch_bounds__(kNT) void balance_grad(BalanceArgs a) {
    constexpr int TPB = kNT / L;
    const int tl = threadIdx.x / L, e0 = threadIdx.x % L * kV, E = a.E;
    const int64_t b0 = (int64_t)blockIdx.x * a.per, b1 = b0 + a.per < a.T ? b0 + a.per : a.T;
    const double wb = (double)a.alpha * (a.dloss ? (double)gld(a.dloss) : 1.0) / a.S;
    const double wz = 2.0 * (double)a.zeta * (a.dloss ? (double)gld(a.dloss + 1) : 1.0) / a.S;
    int q = sequence_of_wave(a, b0);
    bool fresh = true;
    int64_t q0 = first_row(a, q), q1 = first_row(a, q + 1);  // the rows that u and zc hold for
    float u[kV] = {}, zc = 0.f;
    for (int64_t t = b0 + tl; t < b1; t += TPB) {
        if (fresh || t >= q1) {
            if (t >= q1) {
                q = sequence_of(a, t);
                q0 = first_row(a, q);
                q1 = first_row(a, q + 1);
            }
            fresh = false;
            const int n = gld(a.in_rows + q);
            const double by = n > 0 ? 1.0 / n : 0.0;
            zc = (float)(wz * by);
            const double uc = wb * E * by * by / a.k;
#pragma unroll
            for (int v = 0; v < kV; ++v) u[v] = e0 + v < E ? (float)(uc * gld(a.in_counts + (int64_t)q * E + e0 + v)) : 0.f;
        }
        if (t < q0 || t >= q1) continue;  // the same for the row's lanes: no sequence's row
        const T* row = (const T*)a.logits + t * a.ld;
        T* out = (T*)a.dlogits + t * a.ldd;
        float l[kV], p[kV], slope[kV], d[kV] = {};
        load_logits(row, e0, E, a.vec, l);
        if (a.accumulate) load_values((const T*)out, e0, E, a.vec_out, d);
        const Row r = row_probs<L, SCORE>(l, p, slope);
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < kV; ++v) dot = fmaf(u[v], p[v], dot);
        dot = row_sum<L>(dot);
        const float zl = zc * r.lse;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            float g = p[v] * (u[v] - dot);
            if constexpr (SCORE == kRouteSoftmax) g = fmaf(zl, p[v], g);
            else g *= slope[v];
            // where the expert is not available, exactly nothing (lse may be infinite)
            d[v] += l[v] > -kInf ? g : 0.f;
        }
        if (a.vec_out) {
            constexpr int W = 16 / (int)sizeof(T);
#pragma unroll
            for (int i = 0; i < kV / W; ++i) {
                u32x4 o;
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = __float_as_uint(d[i * 4 + j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = pack2_bf16(d[2 * j], d[2 * j + 1]);
                }
                if (e0 + i * W < E) st128(out + e0 + i * W, o);
            }
        } else {
#pragma unroll
            for (int v = 0; v < kV; ++v)
                if (e0 + v < E) {
                    if constexpr (sizeof(T) == 4) gst(out + e0 + v, d[v]);
                    else gst(out + e0 + v, f_to_bf(d[v]));
                }
        }
    }
}

template <bool GRAD, typename T, int L> hipError_t launch_one(const BalanceArgs& a, hipStream_t s) {
    const bool soft = a.score == kRouteSoftmax;
    const dim3 g((unsigned)a.blocks), n(kNT);
    if constexpr (GRAD) {
        if (soft) hipLaunchKernelGGL((balance_grad<T, L, kRouteSoftmax>), g, n, 0, s, a);
        else hipLaunchKernelGGL((balance_grad<T, L, kRouteSigmoid>), g, n, 0, s, a);
    } else {
        if (soft) hipLaunchKernelGGL((balance_parts<T, L, kRouteSoftmax>), g, n, 0, s, a);
        else hipLaunchKernelGGL((balance_parts<T, L, kRouteSigmoid>), g, n, 0, s, a);
    }
    return hipGetLastError();
}
template <bool GRAD, typename T> hipError_t launch_t(const BalanceArgs& a, hipStream_t s) {
    if (a.E <= 8) return launch_one<GRAD, T, 1>(a, s);
    if (a.E <= 16) return launch_one<GRAD, T, 2>(a, s);
    if (a.E <= 32) return launch_one<GRAD, T, 4>(a, s);
    if (a.E <= 64) return launch_one<GRAD, T, 8>(a, s);
    if (a.E <= 128) return launch_one<GRAD, T, 16>(a, s);
    if (a.E <= 256) return launch_one<GRAD, T, 32>(a, s);
    return launch_one<GRAD, T, 64>(a, s);
}

// Lanes of a row of E experts.
int lanes_of(int E) {
    int L = 1;
    while (L * kV < E) L *= 2;
    return L;
}

}  // namespace

BalanceLayout balance_layout(int64_t T, int E, int S) {
    BalanceLayout w;
    // no more than 512 blocks: the second launch reads every part
    const int64_t round = kNT / lanes_of(E);
    w.per = round;
    while ((T + w.per - 1) / w.per > 512) w.per *= 2;
    w.blocks = T > 0 ? (T + w.per - 1) / w.per : 1;
    w.slots = w.blocks + S;
    const int64_t pieces = (E + kPiece - 1) / kPiece;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at = (at + n + 255) & ~(size_t)255;
        return o;
    };
    w.ticket = take(4);
    w.p = take((size_t)w.slots * E * 8);
    w.z = take((size_t)w.slots * 8);
    w.seq = take((size_t)S * pieces * 16);
    w.c = take((size_t)w.slots * E * 4);
    w.n = take((size_t)w.slots * 4);
    w.bytes = at;
    return w;
}

hipError_t launch_balance(const BalanceArgs& a, int dtype, hipStream_t s) {
    const int64_t pieces = (a.E + kPiece - 1) / kPiece;
    if (!grid_fits(a.blocks, kNT) || !grid_fits(a.S * pieces, kNT)) return hipErrorInvalidConfiguration;
    const hipError_t e = dtype == 0 ? launch_t<false, float>(a, s) : launch_t<false, uint16_t>(a, s);
    if (e != hipSuccess || (a.S == 1 && a.blocks == 1)) return e;
    hipLaunchKernelGGL(balance_sum, dim3((unsigned)(a.S * pieces)), dim3(kNT), 0, s, a);
    return hipGetLastError();
}
hipError_t launch_balance_grad(const BalanceArgs& a0, int dtype, hipStream_t s) {
    BalanceArgs a = a0;
    const int64_t round = kNT / lanes_of(a.E);
    a.per = a.T > 1024 * round ? 4 * round : round;  // what a sequence's rows share is read once
    a.blocks = (a.T + a.per - 1) / a.per;
    if (!grid_fits(a.blocks, kNT)) return hipErrorInvalidConfiguration;
    return dtype == 0 ? launch_t<true, float>(a, s) : launch_t<true, uint16_t>(a, s);
}

}  // namespace dlm
