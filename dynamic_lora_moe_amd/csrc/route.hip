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
// them at once.  Few lanes with many experts each are the cheaper split: a
// round of the top-k costs V compares and log2(L) steps per wave, 64 / L tokens.
//
// A key carries its expert in its nine lowest mantissa bits (the complement
// for a positive key), so one binary64 maximum is an argmax with ties to the
// lower index, all keys differ, and the next round's candidates are the keys
// below the last winner: nothing is removed or marked.  Logits leave those
// bits empty (24 significant bits of 53); of a score plus bias they cut what
// lies 2^-43 below it.
#include "gfx950.hpp"
#include "internal.hpp"
#include "route.hpp"

namespace dlm {

namespace {

constexpr int kIdxBits = 9;
constexpr int kIdxMask = (1 << kIdxBits) - 1;
static_assert(kRouteMaxExperts <= kIdxMask + 1, "an expert fits the key's index bits");

template <int CTRL> __device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// The other operand of step STEP of a reduction over a row of lanes: within a
// quad, between quads (half-row mirror), between half rows (row mirror) and
// between rows.  Every lane ends with the same bits (the operands of a step
// are the same two partial results in either order).
template <int STEP> __device__ __forceinline__ double peer(double v) {
    if constexpr (STEP == 1) return dpp_f64<0xB1>(v);
    else if constexpr (STEP == 2) return dpp_f64<0x4E>(v);
    else if constexpr (STEP == 4) return dpp_f64<0x141>(v);
    else if constexpr (STEP == 8) return dpp_f64<0x140>(v);
    else return __shfl_xor(v, STEP, kWave);
}

// No operand is ever a NaN here (checked where keys are made).
__device__ __forceinline__ double max2(double a, double b) { return __builtin_fmax(a, b); }

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

// A key with its index in the low bits.  -inf (not available) stays as it is.
__device__ __forceinline__ double with_index(double k, int e) {
    if (!(k > kNone)) return kNone;  // also a NaN
    k = k < 1.7976931348623157e308 ? k + 0.0 : 1.7976931348623157e308;  // -0 -> +0, +inf -> largest
    const uint64_t b = __builtin_bit_cast(uint64_t, k) & ~(uint64_t)kIdxMask;
    return __builtin_bit_cast(double, b | (uint64_t)(k < 0.0 ? e : kIdxMask - e));
}
__device__ __forceinline__ int index_of(double k) {
    const int b = (int)(__builtin_bit_cast(uint64_t, k) & kIdxMask);
    return k < 0.0 ? b : kIdxMask - b;
}

template <typename T> __device__ __forceinline__ float logit_of(T v);
template <> __device__ __forceinline__ float logit_of<float>(float v) { return v; }
template <> __device__ __forceinline__ float logit_of<uint16_t>(uint16_t v) { return bf_to_f(v); }

// A logit as the routing sees it: +inf counts as the largest finite value, a
// NaN as not available (-inf).
__device__ __forceinline__ float clean(float l) {
    l = l == l ? l : -__builtin_huge_valf();
    return l > 3.402823466e38f ? 3.402823466e38f : l;
}

__device__ __forceinline__ double sigmoid(double l) { return 1.0 / (1.0 + exp(-l)); }

// Lane `lane` of a token's L lanes holds experts W * (L * c + lane) + j of its
// 16-byte chunks c: a chunk of the L lanes is one contiguous run.
template <typename T, int L> __device__ __forceinline__ int expert_of(int v, int lane) {
    constexpr int W = 16 / (int)sizeof(T);
    return (v / W) * (W * L) + lane * W + v % W;
}

template <typename T, int L, int V>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int E, int lane, bool live, bool vec, float (&l)[V]) {
    constexpr int W = 16 / (int)sizeof(T);
    static_assert(V % W == 0, "whole chunks");
    if (vec) {  // rows 16-byte aligned and E a multiple of W: a chunk is all in or all out
        u32x4 c[V / W];
#pragma unroll
        for (int i = 0; i < V / W; ++i) {
            const int e = expert_of<T, L>(i * W, lane);
            c[i] = live && e < E ? ld128(row + e) : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int i = 0; i < V / W; ++i) {
            const bool in = live && expert_of<T, L>(i * W, lane) < E;
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
            const int e = expert_of<T, L>(v, lane);
            l[v] = live && e < E ? clean(logit_of<T>(gld(row + e))) : -__builtin_huge_valf();
        }
    }
}

// One workgroup: NT / L tokens.  Dynamic LDS: the chosen experts [tokens][k]
// and their scores, then (with groups) keys, group keys and the kept flags.
template <typename T, int L, int V, int NT>
__global__ __launch_bounds__(NT) void route_kernel(RouteArgs a) {
    constexpr int TPB = NT / L;
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
    load_row<T, L, V>(row, E, lane, live, a.vec, l);

    // softmax: the largest logit (0 for a row with none), and with it the
    // denominator where the weights or the keys need it
    double mx = 0.0, inv = 1.0;
    if (a.score == kRouteSoftmax) {
        float m = l[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
        mx = row_max<L>((double)m);
        if (!(mx > kNone)) mx = 0.0;
    }
    double key[V];
    if (a.need_scores) {
        if (a.score == kRouteSoftmax) {
            double sum = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                key[v] = l[v] > -__builtin_huge_valf() ? exp((double)l[v] - mx) : 0.0;
                sum += key[v];
            }
            sum = row_sum<L>(sum);
            inv = sum > 0.0 ? 1.0 / sum : 0.0;
        }
        if (a.scores_order) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = expert_of<T, L>(v, lane);
                const double s = a.score == kRouteSoftmax ? key[v] * inv : sigmoid((double)l[v]);
                const double b = a.bias && e < E ? (double)gld(a.bias + e) : 0.0;
                key[v] = l[v] > -__builtin_huge_valf() ? with_index(s + b, e) : kNone;
            }
        }
    }
    if (!a.scores_order) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = with_index((double)l[v], expert_of<T, L>(v, lane));
    }

    if (a.counts) {
        for (int e = tid; e < E; e += NT) s_cnt[e] = 0;
    }
    if (G > 1) {
        const int S = G * (gs + 1);  // a token's keys, a gap behind each group (LDS banks)
        double* s_key = (double*)(smem + a.lds_groups);
        double* s_gk = s_key + TPB * S;
        uint8_t* s_keep = (uint8_t*)(s_gk + TPB * G);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert_of<T, L>(v, lane);
            if (e < E) s_key[tl * S + e + (int)(((uint32_t)e * a.gs_magic) >> 20)] = key[v];
        }
        __syncthreads();
        for (int q = tid; q < TPB * G; q += NT) {
            const int tk = q / G, gi = q % G;
            const double* kp = s_key + tk * S + gi * (gs + 1);
            double b1 = kNone, b2 = kNone;
            for (int j = 0; j < gs; ++j) {
                const double x = kp[j];
                b2 = max2(b2, x < b1 ? x : b1);
                b1 = max2(b1, x);
            }
            // the sum is of the keys without their index bits
            if (a.group_top == 2 && b2 > kNone) {
                const uint64_t m = ~(uint64_t)kIdxMask;
                b1 = __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, b1) & m) +
                     __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, b2) & m);
            } else if (b1 > kNone) {
                b1 = __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, b1) & ~(uint64_t)kIdxMask);
            }
            s_gk[q] = with_index(b1, gi);
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
            const int e = expert_of<T, L>(v, lane);
            const int gi = (int)(((uint32_t)e * a.gs_magic) >> 20);
            if (e < E && !s_keep[tl * G + gi]) key[v] = kNone;
        }
    }

    // k rounds of an argmax over the keys below the last winner
    double last = __builtin_huge_val();
    for (int s = 0; s < k; ++s) {
        double m = kNone;
#pragma unroll
        for (int v = 0; v < V; ++v) m = max2(m, key[v] < last ? key[v] : kNone);
        m = row_max<L>(m);
        if (lane == s % L) s_idx[tl * k + s] = m > kNone ? index_of(m) : -1;
        last = m;
    }
    __syncthreads();

    // the chosen experts' scores, one slot per lane
    for (int s = lane; s < k; s += L) {
        const int e = s_idx[tl * k + s];
        double w = 0.0;
        if (e >= 0 && live) {
            const double le = (double)clean(logit_of<T>(gld(row + e)));
            w = a.score == kRouteSoftmax ? exp(le - mx) * inv : sigmoid(le);
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
            p[v] = l[v] > -__builtin_huge_valf() ? exp((double)l[v] - mx) : 0.0;
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
                w = soft ? exp((double)lf - mx) * inv : sigmoid((double)lf);
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
    for (int s = lane; s < k; s += L) {
        const int e = s_idx[tl * k + s];
        bool first = e >= 0;
        double d = 0.0;
        for (int j = 0; j < k; ++j) {
            if (s_idx[tl * k + j] != e) continue;
            if (j < s) first = false;
            double dj = s_d[tl * k + j];
            if (a.renorm) dj = sw > 0.0 ? (dj - sdw / sw) / sw : 0.0;
            d += dj;
        }
        if (!first) continue;
        if (!full) {
            const double w = s_w[tl * k + s];
            if (soft) {
                d *= w;
            } else {
                // s (1 - s) without the cancellation of 1 - s
                const double z = exp(-fabs((double)clean(logit_of<T>(gld(row + e)))));
                d *= z / ((1.0 + z) * (1.0 + z));
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
        const int e0 = expert_of<T, L>(c * W, lane);
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

template <typename T, int L, int V, int NT>
hipError_t launch_one(RouteArgs a, bool grad, hipStream_t s) {
    constexpr int TPB = NT / L;
    const int64_t blocks = (a.T + TPB - 1) / TPB;
    if (!grid_fits(blocks, NT)) return hipErrorInvalidConfiguration;
    if (grad) {
        const size_t lds = (size_t)TPB * (L * V * 8 + a.k * 20);
        hipLaunchKernelGGL((route_grad_kernel<T, L, V, NT>), dim3((unsigned)blocks), dim3(NT), lds, s, a);
    } else {
        size_t lds = (size_t)TPB * a.k * 12 + (a.counts ? (size_t)a.E * 4 : 0);
        if (a.n_groups > 1) {
            lds = (lds + 15) & ~(size_t)15;
            a.lds_groups = (int)lds;
            lds += (size_t)TPB * (a.n_groups * (a.group_size + 1) * 8 + a.n_groups * 9);
        }
        hipLaunchKernelGGL((route_kernel<T, L, V, NT>), dim3((unsigned)blocks), dim3(NT), lds, s, a);
    }
    return hipGetLastError();
}

// Lanes and experts per lane by E.
template <typename T> hipError_t launch_t(const RouteArgs& a, bool grad, hipStream_t s) {
    if (a.E <= 8) return launch_one<T, 1, 8, 64>(a, grad, s);
    if (a.E <= 16) return launch_one<T, 1, 16, 64>(a, grad, s);
    if (a.E <= 32) return launch_one<T, 2, 16, 128>(a, grad, s);
    if (a.E <= 64) return launch_one<T, 4, 16, 128>(a, grad, s);
    if (a.E <= 128) return launch_one<T, 8, 16, 256>(a, grad, s);
    if (a.E <= 256) return launch_one<T, 16, 16, 256>(a, grad, s);
    return launch_one<T, 32, 16, 256>(a, grad, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s) {
    return dtype == 0 ? launch_t<float>(a, false, s) : launch_t<uint16_t>(a, false, s);
}
hipError_t launch_route_grad(const RouteArgs& a, int dtype, hipStream_t s) {
    return dtype == 0 ? launch_t<float>(a, true, s) : launch_t<uint16_t>(a, true, s);
}

}  // namespace dlm
