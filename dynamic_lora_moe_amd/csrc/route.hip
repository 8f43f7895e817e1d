// Routing to experts from router logits, and the gradient of its weights.
//
//   score   s = softmax(l) over the available experts, or sigmoid(l)
//   key     s + bias (the bias only selects; without one the logits themselves
//           order the experts, softmax and sigmoid being increasing)
//   groups  E / n_groups consecutive experts each, ranked by their best key or
//           the sum of their best two; the best keep_groups stay in the race
//   weights g = scale * s_i, or scale * s_i / sum_j s_j over the chosen
//
// The order of two close scores decides which expert runs, so scores, keys and
// sums are binary64 and the weights are rounded once, to fp32; on this machine
// a binary64 FMA issues at the rate of an unpacked fp32 one.
//
// L lanes hold one token's row, V experts each (L x V >= E), so a wave holds
// 64 / L tokens and a reduction over a token takes log2(L) DPP steps for all of
// them at once.  The kernels are bound by instruction issue (binary64 scores of
// every expert, then the selection), so few lanes with many experts each are the
// cheaper split.
//
// A key carries its expert in its nine lowest mantissa bits (the complement
// for a positive key), so one binary64 maximum is an argmax with ties to the
// lower index, and all keys differ.  Logits leave those bits empty (24
// significant bits of 53); of a score plus bias they cut what lies 2^-43 below
// it.  The k largest: each lane sorts its keys in lists of 4, 8 or 16 (k rounded
// up; Batcher's odd-even network) and merges them, then the lanes' lists merge
// pairwise; of two descending lists the largest are max(a[i], b[N - 1 - i]).
//
// Measured: 64 tokens of 8 experts, top 2: 2.8 us.  4099 tokens of 60 experts, bf16,
// softmax, top 6: 5.2 us, the gradient 6.1 (few workgroups: latency).  32768 tokens
// of 256 experts, fp32, sigmoid with bias, 4 of 8 groups, top 8: 26 us, 1.4 TB/s,
// three and a half times what reading the logits takes (softmax without bias and
// groups: 16 us); 16384 of them in bf16 15 us and their gradient, which needs the
// sigmoid of the chosen only, 7 us (2.4 TB/s).  The former on 8 lanes with 32
// experts each, which merges less across lanes: 28 us, as fewer waves hide less.
#include <type_traits>

#include "gfx950.hpp"
#include "internal.hpp"
#include "route.hpp"

namespace dlm {

namespace {

constexpr int kIdxBits = 9;
constexpr int kIdxMask = (1 << kIdxBits) - 1;
static_assert(kRouteMaxExperts <= kIdxMask + 1, "an expert fits the key's index bits");

// No operand is ever a NaN here (checked where keys are made).  As instructions
// of their own: the compiler's fmax first quiets both operands, an instruction each.
__device__ __forceinline__ double max2(double a, double b) {
    double d;
    asm("v_max_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
__device__ __forceinline__ double min2(double a, double b) {
    double d;
    asm("v_min_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}

// A double from another lane of the row.  A DPP operand must have been written
// two wait states before; the compiler does not see that those above write one,
// so the wait is here.
#define DLM_DPP_F64(NAME, CTRL)                                                             \
    __device__ __forceinline__ double NAME(double v) {                                      \
        const uint64_t b = __builtin_bit_cast(uint64_t, v);                                 \
        uint32_t lo, hi;                                                                    \
        asm("s_nop 1\n\tv_mov_b32_dpp %0, %2 " CTRL " row_mask:0xf bank_mask:0xf\n\t"        \
            "v_mov_b32_dpp %1, %3 " CTRL " row_mask:0xf bank_mask:0xf"                      \
            : "=&v"(lo), "=&v"(hi)                                                          \
            : "v"((uint32_t)b), "v"((uint32_t)(b >> 32)));                                  \
        return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);                       \
    }
DLM_DPP_F64(dpp_xor1, "quad_perm:[1,0,3,2]")
DLM_DPP_F64(dpp_xor2, "quad_perm:[2,3,0,1]")
DLM_DPP_F64(dpp_half_mirror, "row_half_mirror")
DLM_DPP_F64(dpp_mirror, "row_mirror")
#undef DLM_DPP_F64

// The other operand of step STEP of a reduction over a row of lanes: within a
// quad, between quads (half-row mirror), between half rows (row mirror) and
// between rows.  Every lane ends with the same bits (the operands of a step
// are the same two partial results in either order).
template <int STEP> __device__ __forceinline__ double peer(double v) {
    if constexpr (STEP == 1) return dpp_xor1(v);
    else if constexpr (STEP == 2) return dpp_xor2(v);
    else if constexpr (STEP == 4) return dpp_half_mirror(v);
    else if constexpr (STEP == 8) return dpp_mirror(v);
    else return __shfl_xor(v, STEP, kWave);
}

// Comparators of Batcher's odd-even merge sort of N = 4, 8 or 16 values.
template <int N> struct Network {
    int n = 0;
    int8_t lo[64] = {}, hi[64] = {};
    constexpr Network() {
        for (int p = 1; p < N; p *= 2)
            for (int k = p; k >= 1; k /= 2)
                for (int j = k % p; j <= N - 1 - k; j += 2 * k)
                    for (int i = 0; i < k && i < N - j - k; ++i)
                        if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                            lo[n] = (int8_t)(i + j);
                            hi[n] = (int8_t)(i + j + k);
                            ++n;
                        }
    }
};
template <int N> __device__ __forceinline__ void sort_descending(double* k) {
    constexpr Network<N> net;
#pragma unroll
    for (int c = 0; c < net.n; ++c) {
        const double a = k[net.lo[c]], b = k[net.hi[c]];
        k[net.lo[c]] = max2(a, b);
        k[net.hi[c]] = min2(a, b);
    }
}
// a <- the largest N of two descending lists of N, descending: the larger of
// a[i] and b[N - 1 - i] are those N as a bitonic sequence, which log2(N) steps sort.
template <int N> __device__ __forceinline__ void merge_top(double* a, const double (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = max2(a[i], b[N - 1 - i]);
#pragma unroll
    for (int h = N / 2; h >= 1; h /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((i & h) == 0) {
                const double x = a[i], y = a[i + h];
                a[i] = max2(x, y);
                a[i + h] = min2(x, y);
            }
}
template <int N, int STEP> __device__ __forceinline__ void merge_peer(double* a) {
    double b[N];
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = peer<STEP>(a[i]);
    merge_top<N>(a, b);
}
// A lane's largest D keys, descending, in key[0 .. D).
template <int V, int D> __device__ __forceinline__ void lane_keys(double (&key)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += D) sort_descending<D>(key + i);
#pragma unroll
    for (int i = D; i < V; i += D) {
        double b[D];
#pragma unroll
        for (int j = 0; j < D; ++j) b[j] = key[i + j];
        merge_top<D>(key, b);
    }
}
// From those, the token's in each of its lanes.
template <int L, int V, int D> __device__ __forceinline__ void row_keys(double (&key)[V]) {
    if constexpr (L > 1) merge_peer<D, 1>(key);
    if constexpr (L > 2) merge_peer<D, 2>(key);
    if constexpr (L > 4) merge_peer<D, 4>(key);
    if constexpr (L > 8) merge_peer<D, 8>(key);
    if constexpr (L > 16) merge_peer<D, 16>(key);
}

template <int L> __device__ __forceinline__ double row_max(double v) {
    if constexpr (L > 1) v = max2(v, peer<1>(v));
    if constexpr (L > 2) v = max2(v, peer<2>(v));
    if constexpr (L > 4) v = max2(v, peer<4>(v));
    if constexpr (L > 8) v = max2(v, peer<8>(v));
    if constexpr (L > 16) v = max2(v, peer<16>(v));
    return v;
}
template <int L> __device__ __forceinline__ double row_sum(double v) {
    if constexpr (L > 1) v += peer<1>(v);
    if constexpr (L > 2) v += peer<2>(v);
    if constexpr (L > 4) v += peer<4>(v);
    if constexpr (L > 8) v += peer<8>(v);
    if constexpr (L > 16) v += peer<16>(v);
    return v;
}

constexpr double kNone = -__builtin_huge_val();

// A key with its index in the low bits.  -inf or NaN (not available) gives
// -inf.  Straight-line code: the key is made either way and then selected.
__device__ __forceinline__ double with_index(double k, int e, bool on = true) {
    const double f = min2(k, 1.7976931348623157e308);  // +inf -> largest
    const uint64_t b = __builtin_bit_cast(uint64_t, f);
    const uint32_t lo = ((uint32_t)b & ~(uint32_t)kIdxMask) | (uint32_t)(f < 0.0 ? e : kIdxMask - e);
    const double r = __builtin_bit_cast(double, (b & 0xffffffff00000000ull) | lo);
    return on && k > kNone ? r : kNone;
}
__device__ __forceinline__ int index_of(double k) {
    const int b = (int)(__builtin_bit_cast(uint64_t, k) & kIdxMask);
    return k < 0.0 ? b : kIdxMask - b;
}

__device__ __forceinline__ double without_index(double k) {
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~(uint64_t)kIdxMask);
}
// A group's key from its best two: the best, or the sum of both (without their index bits).
__device__ __forceinline__ double group_key(double b1, double b2, int top, int g) {
    if (!(b1 > kNone)) return kNone;
    double k = without_index(b1);
    if (top == 2 && b2 > kNone) k += without_index(b2);
    return with_index(k + 0.0, g);
}
// (b1 >= b2) <- the best two of this lane's pair and the peer's, of other keys.
template <int STEP> __device__ __forceinline__ void merge_pair(double& b1, double& b2) {
    const double p1 = peer<STEP>(b1), p2 = peer<STEP>(b2);
    b2 = max2(min2(b1, p1), max2(b2, p2));
    b1 = max2(b1, p1);
}

template <typename T> __device__ __forceinline__ float logit_of(T v);
template <> __device__ __forceinline__ float logit_of<float>(float v) { return v; }
template <> __device__ __forceinline__ float logit_of<uint16_t>(uint16_t v) { return bf_to_f(v); }

// A logit as the routing sees it: +inf counts as the largest finite value, a
// NaN as not available (-inf).  Where an operand is a NaN the median instruction
// answers min(min(a, b), c): a quiet one drops out of the inner minimum, of a
// signalling one that makes a quiet NaN, which drops out of the outer.  With -inf
// as the last operand the answer is -inf for both.  (The builtin of it is folded to
// a minimum of two.)
__device__ __forceinline__ float clean(float l) {
    float r;
    asm("v_med3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(l), "v"(3.402823466e38f), "v"(-__builtin_huge_valf()));
    return r;
}

// a b + c with c a constant: one instruction with c in scalar registers.  (Left
// to itself the compiler moves c into a vector register first, two more each.)
__device__ __forceinline__ double fma_c(double a, double b, double c) {
    double d;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
    return d;
}
// e^x for |x| <= 750 (0 and infinity past binary64's range): x = n ln 2 + r, the
// Taylor series of e^r to r^13 (|r| <= 0.347: the rest is below 5e-18 of it), times 2^n.
__device__ __forceinline__ double exp_small(double x) {
    const double n = __builtin_rint(x * 1.4426950408889634);
    double r = __builtin_fma(n, -0.69314718036912381649, x);  // ln 2's upper 32 bits, then the rest
    r = __builtin_fma(n, -1.9082149292705877000e-10, r);
    double p = fma_c(r, 1.0 / 6227020800.0, 1.0 / 479001600.0);
    p = fma_c(p, r, 1.0 / 39916800.0);
    p = fma_c(p, r, 1.0 / 3628800.0);
    p = fma_c(p, r, 1.0 / 362880.0);
    p = fma_c(p, r, 1.0 / 40320.0);
    p = fma_c(p, r, 1.0 / 5040.0);
    p = fma_c(p, r, 1.0 / 720.0);
    p = fma_c(p, r, 1.0 / 120.0);
    p = fma_c(p, r, 1.0 / 24.0);
    p = fma_c(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}
// 1 / x for normal x: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double recip(double x) {
    double y = __builtin_amdgcn_rcp(x);
    y = __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
    return __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
}
// The softmax's numerator: 0 for -inf.
__device__ __forceinline__ double exp_of(float l, double mx) {
    const double d = (double)l - mx;
    return exp_small(d > -750.0 ? d : -750.0);
}
// e^-700 for anything below, which every use takes for 0 (keys: next to nothing;
// weights: weight_of).
__device__ __forceinline__ double sigmoid(float l) {
    return recip(1.0 + exp_small(-(double)__builtin_amdgcn_fmed3f(l, -700.f, 700.f)));
}
// A chosen expert's score.
__device__ __forceinline__ double weight_of(bool soft, float l, double mx, double inv) {
    if (soft) return exp_of(l, mx) * inv;
    const double s = sigmoid(l);
    return l < -700.f ? 0.0 : s;
}

// Lane `lane` of a token's L lanes holds experts W * (L * c + lane) + j of its
// 16-byte chunks c: a chunk of the L lanes is one contiguous run.  RUN: V
// neighbouring experts, so that a group of V or more is a run of whole lanes.
template <typename T, int L, int V, bool RUN = false> __device__ __forceinline__ int expert_of(int v, int lane) {
    constexpr int W = 16 / (int)sizeof(T);
    return RUN ? lane * V + v : (v / W) * (W * L) + lane * W + v % W;
}

template <typename T, int L, int V, bool RUN = false>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int E, int lane, bool live, bool vec, float (&l)[V]) {
    constexpr int W = 16 / (int)sizeof(T);
    static_assert(V % W == 0, "whole chunks");
    if (vec) {  // rows 16-byte aligned and E a multiple of W: a chunk is all in or all out
        u32x4 c[V / W];
#pragma unroll
        for (int i = 0; i < V / W; ++i) {
            const int e = expert_of<T, L, V, RUN>(i * W, lane);
            c[i] = live && e < E ? ld128(row + e) : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int i = 0; i < V / W; ++i) {
            const bool in = live && expert_of<T, L, V, RUN>(i * W, lane) < E;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float f;
                if constexpr (sizeof(T) == 4) f = __uint_as_float(c[i][j]);
                else f = (j & 1) ? bf_hi(c[i][j / 2]) : bf_lo(c[i][j / 2]);
                l[i * W + j] = in ? clean(f) : -__builtin_huge_valf();
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert_of<T, L, V, RUN>(v, lane);
            l[v] = live && e < E ? clean(logit_of<T>(gld(row + e))) : -__builtin_huge_valf();
        }
    }
}

// One workgroup: NT / L tokens.  Dynamic LDS: the chosen experts [tokens][k]
// and their scores, then (with groups) keys, group keys and the kept flags.
template <typename T, int L, int V, int NT, int SCORE, bool RUN>
__global__ __launch_bounds__(NT) void route_kernel(RouteArgs a) {
    constexpr int TPB = NT / L, W = 16 / (int)sizeof(T);
    extern __shared__ char smem[];
    const int tid = threadIdx.x, tl = tid / L, lane = tid % L;
    const int E = a.E, k = a.k, G = a.n_groups, gs = a.group_size;
    const int64_t t = (int64_t)blockIdx.x * TPB + tl;
    const bool live = t < a.T;
    double* s_w = (double*)smem;
    int* s_idx = (int*)(s_w + TPB * k);
    int* s_cnt = s_idx + TPB * k;

    const T* row = (const T*)a.logits + (live ? t : 0) * a.ld;
    float l[V];
    load_row<T, L, V, RUN>(row, E, lane, live, a.vec, l);

    // softmax: the largest logit (0 for a row with none), and with it the
    // denominator where the weights or the keys need it
    double mx = 0.0, inv = 1.0;
    if constexpr (SCORE == kRouteSoftmax) {
        float m = l[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
        mx = row_max<L>((double)m);
        if (!(mx > kNone)) mx = 0.0;
    }
    double key[V];
    if (a.need_scores) {
        if constexpr (SCORE == kRouteSoftmax) {
            double sum = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                key[v] = exp_of(l[v], mx);
                sum += key[v];
            }
            sum = row_sum<L>(sum);
            inv = sum > 0.0 ? 1.0 / sum : 0.0;
        }
        if (a.scores_order) {
            float bias[V] = {};
            if (RUN && a.vec_bias) {
#pragma unroll
                for (int v = 0; v < V; v += 4) {
                    const int e = expert_of<T, L, V, RUN>(v, lane);
                    const u32x4 q = ld128(a.bias + (e < E ? e : 0));
#pragma unroll
                    for (int j = 0; j < 4; ++j) bias[v + j] = __uint_as_float(q[j]);
                }
            } else if (a.bias) {
#pragma unroll
                for (int c = 0; c < V / W; ++c) {
                    const int e0 = expert_of<T, L, V, RUN>(c * W, lane);
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        if (a.vec ? e0 < E : e0 + j < E) bias[c * W + j] = gld(a.bias + e0 + j);
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const double s = SCORE == kRouteSoftmax ? key[v] * inv : sigmoid(l[v]);
                key[v] = with_index(s + (double)bias[v], expert_of<T, L, V, RUN>(v, lane), l[v] > -__builtin_huge_valf());
            }
        }
    }
    if (!a.scores_order) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = with_index((double)l[v] + 0.0, expert_of<T, L, V, RUN>(v, lane));  // -0 -> +0
    }

    if (a.counts) {
        for (int e = tid; e < E; e += NT) s_cnt[e] = 0;
    }
    if (!RUN && G > 1 && a.group_lanes) {
        // a group is group_lanes neighbouring lanes' part of one chunk: its best two
        // keys by merging sorted pairs over those lanes
        constexpr int C = V / W;
        const int gl = a.group_lanes;
        double gk[C];
        int above[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            double b1 = kNone, b2 = kNone;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const double x = key[c * W + j];
                b2 = max2(b2, min2(b1, x));
                b1 = max2(b1, x);
            }
            if (L > 1 && gl > 1) merge_pair<1>(b1, b2);
            if (L > 2 && gl > 2) merge_pair<2>(b1, b2);
            if (L > 4 && gl > 4) merge_pair<4>(b1, b2);
            if (L > 8 && gl > 8) merge_pair<8>(b1, b2);
            if (L > 16 && gl > 16) merge_pair<16>(b1, b2);
            gk[c] = group_key(b1, b2, a.group_top, c * (L / gl) + lane / gl);
            above[c] = 0;
        }
        for (int o = 0; o < L; o += gl) {  // this run of lanes, then the token's others
#pragma unroll
            for (int q = 0; q < C; ++q) {
                const double x = o ? __shfl_xor(gk[q], o, kWave) : gk[q];
#pragma unroll
                for (int c = 0; c < C; ++c) above[c] += x > gk[c] ? 1 : 0;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (above[v / W] >= a.keep_groups) key[v] = kNone;
    } else if (!RUN && G > 1) {
        const int S = G * (gs + 1);  // a token's keys, a gap behind each group (LDS banks)
        double* s_key = (double*)(smem + a.lds_groups);
        double* s_gk = s_key + TPB * S;
        uint8_t* s_keep = (uint8_t*)(s_gk + TPB * G);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert_of<T, L, V, RUN>(v, lane);
            if (e < E) s_key[tl * S + e + (int)(((uint32_t)e * a.gs_magic) >> 20)] = key[v];
        }
        __syncthreads();
        for (int q = tid; q < TPB * G; q += NT) {
            const int tk = q / G, gi = q % G;
            const double* kp = s_key + tk * S + gi * (gs + 1);
            double b1 = kNone, b2 = kNone;
            for (int j = 0; j < gs; ++j) {
                const double x = kp[j];
                b2 = max2(b2, min2(b1, x));
                b1 = max2(b1, x);
            }
            s_gk[q] = group_key(b1, b2, a.group_top, gi);
        }
        __syncthreads();
        for (int q = tid; q < TPB * G; q += NT) {
            const int tk = q / G;
            const double mine = s_gk[q];
            int above = 0;
            for (int j = 0; j < G; ++j) above += s_gk[tk * G + j] > mine ? 1 : 0;
            s_keep[q] = mine > kNone && above < a.keep_groups ? 1 : 0;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert_of<T, L, V, RUN>(v, lane);
            const int gi = (int)(((uint32_t)e * a.gs_magic) >> 20);
            if (e < E && !s_keep[tl * G + gi]) key[v] = kNone;
        }
    }

    // the k largest keys: lists of 4, 8 or 16 merged
    auto choose = [&](auto depth) {
        constexpr int D = decltype(depth)::value;
        lane_keys<V, D>(key);
        if constexpr (RUN) {
            // a group is group_lanes lanes, whose lists begin with their best two
            double b1 = key[0], b2 = key[1];
            const int gl = a.group_lanes;
            if (L > 1 && gl > 1) merge_pair<1>(b1, b2);
            if (L > 2 && gl > 2) merge_pair<2>(b1, b2);
            if (L > 4 && gl > 4) merge_pair<4>(b1, b2);
            if (L > 8 && gl > 8) merge_pair<8>(b1, b2);
            const double gk = group_key(b1, b2, a.group_top, lane / gl);
            int above = 0;
            for (int o = gl; o < L; o += gl) above += __shfl_xor(gk, o, kWave) > gk ? 1 : 0;
#pragma unroll
            for (int q = 0; q < D; ++q)
                if (above >= a.keep_groups) key[q] = kNone;
        }
        row_keys<L, V, D>(key);
#pragma unroll
        for (int q = 0; q < D; ++q)
            if (q < k && lane == q % L) s_idx[tl * k + q] = key[q] > kNone ? index_of(key[q]) : -1;
    };
    if (k <= 4) choose(std::integral_constant<int, 4>());
    else if (k <= 8) choose(std::integral_constant<int, 8>());
    else if constexpr (V >= 16) choose(std::integral_constant<int, V>());  // (8 a lane: k <= 8)
    __syncthreads();

    // the chosen experts' scores, one slot per lane
    for (int s = lane; s < k; s += L) {
        const int e = s_idx[tl * k + s];
        double w = 0.0;
        if (e >= 0 && live) {
            const float le = clean(logit_of<T>(gld(row + e)));
            w = weight_of(SCORE == kRouteSoftmax, le, mx, inv);
        }
        s_w[tl * k + s] = w;
    }
    __syncthreads();
    for (int s = lane; s < k; s += L) {
        double w = s_w[tl * k + s];
        if (a.renorm) {
            double sum = 0.0;
            for (int j = 0; j < k; ++j) sum += s_w[tl * k + j];
            w = sum > 0.0 ? w / sum : 0.0;
        }
        if (live) {
            const int e = s_idx[tl * k + s];
            gst(a.idx + t * k + s, e);
            gst(a.g + t * k + s, (float)(w * (double)a.scale));
            if (a.counts && e >= 0) atomicAdd(&s_cnt[e], 1);
        }
    }
    if (a.counts) {
        // whole numbers: the order of the additions does not change the counts
        __syncthreads();
        for (int e = tid; e < E; e += NT)
            if (s_cnt[e]) atomicAdd(a.counts + e, s_cnt[e]);
    }
}

// The gradient: with q_j the weights over scale and d_j = scale * dg_j,
//   renormalised   ds_j = (d_j - sum_i d_i q_i) / sum_i s_i,  else ds_j = d_j
//   sigmoid        dl = ds s (1 - s)
//   softmax        dl_e = s_e (ds_e - sum_j ds_j s_j) over every expert; with
//                  renormalised weights the sum is 0 and the weights are the
//                  softmax over the chosen alone: dl_j = q_j (d_j - sum_i d_i q_i)
// and dl = 0 where nothing depends on the logit.  One workgroup holds NT / L
// rows of ds in LDS; a slot whose expert an earlier slot has already named adds
// to that slot, in slot order.
template <typename T, int L, int V, int NT>
__global__ __launch_bounds__(NT) void route_grad_kernel(RouteArgs a) {
    constexpr int TPB = NT / L;
    extern __shared__ char smem[];
    const int tid = threadIdx.x, tl = tid / L, lane = tid % L;
    const int E = a.E, k = a.k;
    const int64_t t = (int64_t)blockIdx.x * TPB + tl;
    const bool live = t < a.T;
    constexpr int EP = L * V;
    double* s_row = (double*)smem;          // [TPB][EP] d per expert
    double* s_w = s_row + TPB * EP;         // [TPB][k] scores
    double* s_d = s_w + TPB * k;            // [TPB][k] d
    int* s_idx = (int*)(s_d + TPB * k);     // [TPB][k]
    const T* row = (const T*)a.logits + (live ? t : 0) * a.ld;
    const bool soft = a.score == kRouteSoftmax, full = soft && !a.renorm;

    float l[V];
    double mx = 0.0, inv = 1.0;
    if (soft) {
        load_row<T, L, V>(row, E, lane, live, a.vec, l);
        float m = l[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
        mx = row_max<L>((double)m);
        if (!(mx > kNone)) mx = 0.0;
    }
    double p[V];
    if (full) {
        double sum = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = exp_of(l[v], mx);
            sum += p[v];
        }
        sum = row_sum<L>(sum);
        inv = sum > 0.0 ? 1.0 / sum : 0.0;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s_row[tl * EP + lane + L * v] = 0.0;
    for (int s = lane; s < k; s += L) {
        int e = live ? gld(a.in_idx + t * k + s) : -1;
        if (e < 0 || e >= E) e = -1;
        double w = 0.0, d = 0.0;
        if (e >= 0) {
            const float lf = clean(logit_of<T>(gld(row + e)));
            if (lf > -__builtin_huge_valf()) {
                w = weight_of(soft, lf, mx, inv);
                d = (double)a.scale * (double)gld(a.dg + t * k + s);
            } else {
                e = -1;
            }
        }
        s_idx[tl * k + s] = e;
        s_w[tl * k + s] = w;
        s_d[tl * k + s] = d;
    }
    __syncthreads();
    // per token: the sums over its slots (every lane, in slot order)
    double sw = 0.0, sdw = 0.0;
    for (int j = 0; j < k; ++j) {
        const double w = s_w[tl * k + j];
        sw += w;
        sdw += s_d[tl * k + j] * w;
    }
    if (a.renorm) {
        __syncthreads();  // the sums are read
        for (int s = lane; s < k; s += L) s_d[tl * k + s] = sw > 0.0 ? (s_d[tl * k + s] - sdw / sw) / sw : 0.0;
        __syncthreads();
    }
    for (int s = lane; s < k; s += L) {
        const int e = s_idx[tl * k + s];
        bool first = e >= 0;
        double d = 0.0;
        for (int j = 0; j < k; ++j) {
            if (s_idx[tl * k + j] != e) continue;
            if (j < s) first = false;
            d += s_d[tl * k + j];
        }
        if (!first) continue;
        if (!full) {
            const double w = s_w[tl * k + s];
            if (soft) {
                d *= w;
            } else {
                // s (1 - s) without the cancellation of 1 - s
                const double z = exp_of(-fabsf(clean(logit_of<T>(gld(row + e)))), 0.0);
                d *= z * recip((1.0 + z) * (1.0 + z));
            }
        }
        s_row[tl * EP + e] = d;
    }
    __syncthreads();
    if (!live) return;
    T* out = (T*)a.dlogits + t * a.ldd;
    constexpr int W = 16 / (int)sizeof(T);
#pragma unroll
    for (int c = 0; c < V / W; ++c) {
        const int e0 = expert_of<T, L, V>(c * W, lane);
        float r[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int e = e0 + j;
            double d = e < EP ? s_row[tl * EP + e] : 0.0;
            if (full) {
                const double pe = p[c * W + j] * inv;
                d = l[c * W + j] > -__builtin_huge_valf() ? pe * (d - sdw) : 0.0;
            }
            r[j] = (float)d;
        }
        if (a.vec_out) {
            if (e0 < E) {
                u32x4 o;
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = __float_as_uint(r[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = pack2_bf16(r[2 * j], r[2 * j + 1]);
                }
                st128(out + e0, o);
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (e0 + j < E) {
                    if constexpr (sizeof(T) == 4) gst(out + e0 + j, r[j]);
                    else gst(out + e0 + j, f_to_bf(r[j]));
                }
            }
        }
    }
}

template <bool GRAD, typename T, int L, int V, int NT>
hipError_t launch_one(RouteArgs a, hipStream_t s) {
    constexpr int TPB = NT / L;
    const int64_t blocks = (a.T + TPB - 1) / TPB;
    if (!grid_fits(blocks, NT)) return hipErrorInvalidConfiguration;
    if constexpr (GRAD) {
        const size_t lds = (size_t)TPB * (L * V * 8 + a.k * 20);
        hipLaunchKernelGGL((route_grad_kernel<T, L, V, NT>), dim3((unsigned)blocks), dim3(NT), lds, s, a);
    } else {
        size_t lds = (size_t)TPB * a.k * 12 + (a.counts ? (size_t)a.E * 4 : 0);
        const dim3 g((unsigned)blocks), n(NT);
        auto is_run = [](int lanes) { return lanes > 0 && (lanes & (lanes - 1)) == 0 && lanes <= L; };
        if constexpr (L > 1) {
            // groups that are whole runs of 2^i lanes: V neighbouring experts a lane,
            // ranked by the heads of its sorted list (32768 rows of 256 experts in 8
            // groups: 26 us, where ranking chunk by chunk before the sort took 31)
            if (a.n_groups > 1 && a.group_size % V == 0 && is_run(a.group_size / V)) {
                a.group_lanes = a.group_size / V;
                if (a.score == kRouteSoftmax)
                    hipLaunchKernelGGL((route_kernel<T, L, V, NT, kRouteSoftmax, true>), g, n, lds, s, a);
                else
                    hipLaunchKernelGGL((route_kernel<T, L, V, NT, kRouteSigmoid, true>), g, n, lds, s, a);
                return hipGetLastError();
            }
        }
        // smaller ones that are whole runs of 2^i lanes of a chunk need no LDS either
        constexpr int W = 16 / (int)sizeof(T);
        a.group_lanes = a.n_groups > 1 && a.group_size % W == 0 && is_run(a.group_size / W) ? a.group_size / W : 0;
        if (a.n_groups > 1 && !a.group_lanes) {
            lds = (lds + 15) & ~(size_t)15;
            a.lds_groups = (int)lds;
            lds += (size_t)TPB * (a.n_groups * (a.group_size + 1) * 8 + a.n_groups * 9);
        }
        if (a.score == kRouteSoftmax)
            hipLaunchKernelGGL((route_kernel<T, L, V, NT, kRouteSoftmax, false>), g, n, lds, s, a);
        else
            hipLaunchKernelGGL((route_kernel<T, L, V, NT, kRouteSigmoid, false>), g, n, lds, s, a);
    }
    return hipGetLastError();
}

// Lanes and experts per lane by E: 16 a lane, the cheaper split, or 8 on twice the
// lanes, whose chains are shorter, while that makes at most two waves per SIMD: 512
// rows of 60 experts 6.0 us against 8.8 (sigmoid, bias), of 256 experts 6.5 against
// 8.6, but 65536 of 256 58 against 53.  Lists of more than 8 need 16.  The gradients
// of up to 64 experts always take 8, for the rows' smaller share of a workgroup's LDS:
// 65536 rows of 60 experts 11.5 us against 16.2.
constexpr int64_t kRouteFewLanes = 2 * 1024 * kWave;
template <bool GRAD, typename T> hipError_t launch_t(const RouteArgs& a, hipStream_t s) {
    const auto eight = [&](int lanes) { return (GRAD || a.k <= 8) && a.T * lanes <= kRouteFewLanes; };
    if (a.E <= 8) return launch_one<GRAD, T, 1, 8, 64>(a, s);
    if (a.E <= 16) return launch_one<GRAD, T, 1, 16, 64>(a, s);
    if constexpr (GRAD) {
        if (a.E <= 32) return launch_one<GRAD, T, 4, 8, 128>(a, s);
        if (a.E <= 64) return launch_one<GRAD, T, 8, 8, 128>(a, s);
    } else {
        if (a.E <= 32) return eight(4) ? launch_one<GRAD, T, 4, 8, 128>(a, s) : launch_one<GRAD, T, 2, 16, 128>(a, s);
        if (a.E <= 64) return eight(8) ? launch_one<GRAD, T, 8, 8, 128>(a, s) : launch_one<GRAD, T, 4, 16, 128>(a, s);
    }
    if (a.E <= 128) return eight(16) ? launch_one<GRAD, T, 16, 8, 256>(a, s) : launch_one<GRAD, T, 8, 16, 256>(a, s);
    if (a.E <= 256) return eight(32) ? launch_one<GRAD, T, 32, 8, 256>(a, s) : launch_one<GRAD, T, 16, 16, 256>(a, s);
    return launch_one<GRAD, T, 32, 16, 256>(a, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s) {
    return dtype == 0 ? launch_t<false, float>(a, s) : launch_t<false, uint16_t>(a, s);
}
hipError_t launch_route_grad(const RouteArgs& a, int dtype, hipStream_t s) {
    return dtype == 0 ? launch_t<true, float>(a, s) : launch_t<true, uint16_t>(a, s);
}

}  // namespace dlm
