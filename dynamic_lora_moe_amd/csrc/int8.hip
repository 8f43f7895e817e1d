// Products in 8-bit integers with a scale per row (token) and per column (channel).
//
//   codes   q = 127 x / max|x| of the row, to the nearest whole number (a half goes
//           towards 0), s = max|x| / 127; weights come as codes and scales
//   out     s_t w_o sum_k q_tk w_ok     sums exact in 32 bits, then three fp32 roundings
//
// The rounding is decided on the exact quotient: x 127 / max is one binary64 fma onto
// 1.5 * 2^52, whose low byte is the code (127 / max is taken a hair low, 2^-51, so that
// the only exact halves, which binary64 could put on either side, go one way).  A quotient of
// 24-bit numbers that is no half is farther than that from one.  The gradient's dy w_scale
// have up to 48 bits (32 where dy is bf16): of fp32 dy a quotient can lie closer to a half,
// and its code then be one off.
//
// The input gradient is the same product: codes of dy w_scale, whose runs from all the
// products of one input stand side by side in one row with one scale, against the
// transposed codes of W.
//
// Codes and weights are kept in 1 KB pieces that are the matrix instruction's operands
// (16 x 16 x 64): a wave copies a piece with one instruction, lane after lane, to
// registers or LDS, and reads it from there without bank conflicts.  W is the first
// operand, so a lane's four results are neighbouring columns of out.
//
// A 7B-shaped layer's seven products, bf16: one row 5.5 us for the codes and 30 for the
// products (6.7 TB/s, the rate at which memory is read), 64 rows 8.5 and 46, 4096 rows 88
// and 690-730 (2300-2400 TOP/s), and the gradient 195 and 630-645.  The matrix cores are busy
// 54 % of those cycles (61 % in the gradient) at a clock of about 2.0 GHz; a loop of these
// instructions in registers reaches 4010 TOP/s on such operands, 4870 on zeros: it is the
// operands' switching that costs the rest of the clock.
#include "gfx950.hpp"
#include "int8.hpp"
#include "internal.hpp"

namespace dlm {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4a8 __attribute__((aligned(8)));  // rows of a multiple of four bf16

__device__ __forceinline__ i32x4 mfma(u32x4 a, u32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// ---- codes of rows ---------------------------------------------------------------------

__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(uint16_t v) { return bf_to_f(v); }

// 16 neighbours of a row as stored, 0 past its end.
template <typename T> struct Raw16 {
    u32x4 r[sizeof(T)];
};
template <typename T> __device__ __forceinline__ void load16(const T* row, int64_t i, int64_t d, bool vec, Raw16<T>& o) {
    constexpr int W = 16 / (int)sizeof(T);
    if (vec) {  // d a multiple of W: all in or all out
#pragma unroll
        for (int c = 0; c < (int)sizeof(T); ++c) o.r[c] = i + c * W < d ? ld128(row + i + c * W) : u32x4{0u, 0u, 0u, 0u};
    } else {
#pragma unroll
        for (int c = 0; c < (int)sizeof(T); ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                constexpr int N = 4 / (int)sizeof(T);  // values in a register
                uint32_t b = 0;
#pragma unroll
                for (int h = 0; h < N; ++h) {
                    const int64_t at = i + c * W + j * N + h;
                    uint32_t v = 0;
                    if (at < d) {
                        if constexpr (sizeof(T) == 4) v = __float_as_uint(gld(row + at));
                        else v = gld(row + at);
                    }
                    b |= v << (16 * h);
                }
                o.r[c][j] = b;
            }
    }
}
template <typename T> __device__ __forceinline__ float value16(const Raw16<T>& o, int j) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(o.r[j / 4][j % 4]);
    else return j & 1 ? bf_hi(o.r[j / 8][j % 8 / 2]) : bf_lo(o.r[j / 8][j % 8 / 2]);
}
__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// The codes' factor and the scale of a row from the largest magnitude; 0 and NaN for one
// that is not finite (its codes are 0, its results NaN), 0 and 0 for zeros.
__device__ __forceinline__ void row_scale(double top, double* by, float* scale) {
    const bool fin = top <= 1.7976931348623157e308;
    *by = fin && top > 0.0 ? 127.0 / top * (1.0 - 0x1p-51) : 0.0;
    *scale = fin ? (float)(top / 127.0) : __builtin_nanf("");
}
__device__ __forceinline__ uint32_t code(double x, double by) {
    return (uint32_t)__builtin_bit_cast(uint64_t, __builtin_fma(x, by, 0x1.8p52));
}
// The factors of 16 neighbours (an array padded to a multiple of 16; 1 where there is none).
struct Scale16 {
    u32x4 r[4];
    bool on;
    __device__ __forceinline__ Scale16(const float* sc, int64_t i, int64_t d) : on(sc != nullptr) {
#pragma unroll
        for (int c = 0; c < 4; ++c) r[c] = on && i < d ? ld128(sc + i + 4 * c) : u32x4{0u, 0u, 0u, 0u};
    }
    __device__ __forceinline__ double at(int j) const { return (double)__uint_as_float(r[j / 4][j % 4]); }
};
// By value, not by address: 16 codes of one lane.
template <typename T> __device__ __forceinline__ u32x4 codes16(const Raw16<T>& f, const Scale16& sc, double by) {
    u32x4 o;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            double x = (double)value16(f, 4 * w + j);
            if (sc.on) x *= sc.at(4 * w + j);
            b[j] = code(x, by);
        }
        // the four low bytes
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
        o[w] = by > 0.0 ? lo | hi << 16 : 0u;
    }
    return o;
}
// The largest |x| of 16 values, each times its factor (infinite for one that is not finite).
template <typename T> __device__ __forceinline__ double top16(const Raw16<T>& f, const Scale16& sc) {
    if (!sc.on) {
        uint32_t b = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint32_t v = abs_bits(value16(f, j));
            b = b > v ? b : v;
        }
        return b >= 0x7f800000u ? __builtin_huge_val() : (double)__uint_as_float(b);
    }
    double m = 0.0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const double x = fabs((double)value16(f, j) * sc.at(j));
        m = x <= m ? m : x == x ? x : __builtin_huge_val();
    }
    return m;
}

// The largest of the workgroup's values, R at a time, in every thread.
template <int NT, int R> __device__ __forceinline__ void block_max(double (&v)[R], double (*s)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            const double p = __shfl_xor(v[r], o, kWave);
            v[r] = v[r] > p ? v[r] : p;
        }
        if (lane_id() == 0) s[wave_id()][r] = v[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        v[r] = s[0][r];
#pragma unroll
        for (int w = 1; w < NT / kWave; ++w) v[r] = v[r] > s[w][r] ? v[r] : s[w][r];
    }
}

// Block b's rows: those that share 16-row pieces, and with them cache lines, on one XCD.
template <int R> __device__ __forceinline__ int64_t rows_of_block(int64_t b, int64_t blocks) {
    constexpr int per = 16 / R;
    if (blocks % (8 * per)) return b * R;
    const int64_t local = b / 8;
    return ((local / per * 8 + b % 8) * per + local % per) * R;
}

// One workgroup: R rows of one matrix of codes.  A thread takes every NT-th group of 16
// values of the rows' runs, keeps its first KEEP groups in registers and reads what is
// longer again; the rows share a run's factors.  4096 rows of a layer's four inputs (191 MB
// in, 95 out) take 88 us, 3.3 TB/s: a row's codes wait for its largest value.  One row a
// workgroup, or 1024 threads, were slower.
template <typename T, int R, int NT, int KEEP> __global__ __launch_bounds__(NT) void i8_rows(I8Args a) {
    __shared__ double s_max[NT / kWave][R];
    const I8Rows M = a.rows[blockIdx.y];
    const int64_t t0 = rows_of_block<R>(blockIdx.x, gridDim.x);
    if (t0 >= a.T) return;
    const int groups = M.pieces * 4, last = a.T - t0 < R ? (int)(a.T - 1 - t0) : R - 1;
    struct Group {
        const T* x;       // the run's first row here
        const float* scale;
        int64_t i, d;     // its place in the run; past its end where the run is padded
        bool vec;
    };
    const auto group = [&](int g) {
        int s = M.seg0;
        while (s + 1 < M.seg1 && gld(&a.segs[s + 1].k0) <= g / 4) ++s;
        const I8Seg S = a.segs[s];
        return Group{(const T*)S.x + t0 * S.d, S.scale, (int64_t)(g - 4 * S.k0) * 16, S.d, S.vec != 0};
    };
    const auto load = [&](const Group& G, Raw16<T> (&f)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r) load16(G.x + (r < last ? r : last) * G.d, G.i, G.d, G.vec, f[r]);
    };
    double top[R];
#pragma unroll
    for (int r = 0; r < R; ++r) top[r] = 0.0;
    const auto raise = [&](const Raw16<T> (&f)[R], const Scale16& sc) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const double m = top16(f[r], sc);
            top[r] = top[r] > m ? top[r] : m;
        }
    };
    Raw16<T> keep[KEEP][R];
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int g = c * NT + threadIdx.x;
        if (g < groups) load(group(g), keep[c]);
    }
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int g = c * NT + threadIdx.x;
        if (g < groups) {
            const Group G = group(g);
            raise(keep[c], Scale16(G.scale, G.i, G.d));
        }
    }
    for (int g = KEEP * NT + threadIdx.x; g < groups; g += NT) {
        const Group G = group(g);
        Raw16<T> f[R];
        load(G, f);
        raise(f, Scale16(G.scale, G.i, G.d));
    }
    block_max<NT, R>(top, s_max);
    double by[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float scale;
        row_scale(top[r], &by[r], &scale);
        if (threadIdx.x == 0 && t0 + r < a.T) gst(a.scale + M.index * a.T16 * 16 + t0 + r, scale);
    }
    // (rows past the last write the place of a row that no result is read from)
    int8_t* out = a.q + (M.q0 * a.T16 + t0 / 16 * M.pieces) * kI8Piece + t0 % 16 * 16;
    const auto put = [&](int g, const Raw16<T> (&f)[R], const Scale16& sc) {
#pragma unroll
        for (int r = 0; r < R; ++r) st128(out + (int64_t)(g / 4) * kI8Piece + g % 4 * 256 + r * 16, codes16(f[r], sc, by[r]));
    };
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
        const int g = c * NT + threadIdx.x;
        if (g < groups) {
            const Group G = group(g);
            put(g, keep[c], Scale16(G.scale, G.i, G.d));
        }
    }
    for (int g = KEEP * NT + threadIdx.x; g < groups; g += NT) {
        const Group G = group(g);
        Raw16<T> f[R];
        load(G, f);
        put(g, f, Scale16(G.scale, G.i, G.d));
    }
}

// Rows to row-major codes (weights, when they are quantized).
constexpr int kQT = 256;
template <typename T> __global__ __launch_bounds__(kQT) void i8_quantize(const T* __restrict__ x, int64_t d, int vec, int8_t* q, float* scale) {
    __shared__ double s_max[kQT / kWave][1];
    const T* row = x + (int64_t)blockIdx.x * d;
    const Scale16 one(nullptr, 0, 0);
    double top[1] = {0.0};
    for (int64_t i = threadIdx.x * 16; i < d; i += kQT * 16) {
        Raw16<T> f;
        load16(row, i, d, vec, f);
        const double m = top16(f, one);
        top[0] = top[0] > m ? top[0] : m;
    }
    block_max<kQT, 1>(top, s_max);
    double by;
    float sc;
    row_scale(top[0], &by, &sc);
    if (threadIdx.x == 0) gst(scale + blockIdx.x, sc);
    for (int64_t i = threadIdx.x * 16; i < d; i += kQT * 16) {
        Raw16<T> f;
        load16(row, i, d, vec, f);
        const u32x4 o = codes16(f, one, by);
        int8_t* out = q + (int64_t)blockIdx.x * d + i;
        if (i + 16 <= d && ((uintptr_t)out & 15u) == 0) {
            st128(out, o);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (i + j < d) gst(out + j, (int8_t)(o[j / 4] >> (8 * (j % 4))));
        }
    }
}

// ---- weights -----------------------------------------------------------------------------

__global__ __launch_bounds__(256) void i8_pack(const int8_t* __restrict__ W, int64_t d_out, int64_t d_in, int pieces, int64_t groups,
                                               int8_t* out) {
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += (int64_t)gridDim.x * 256) {
        const int64_t piece = g / 64, o = piece / pieces * 16 + g % 16, k = piece % pieces * 64 + g % 64 / 16 * 16;
        u32x4 r = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint32_t b = o < d_out && k + j < d_in ? (uint8_t)gld(W + o * d_in + k + j) : 0u;
            r[j / 4] |= b << (8 * (j % 4));
        }
        st128(out + g * 16, r);
    }
}
// W's transpose: rows are W's columns, columns k0 * 64 .. its rows.
__global__ __launch_bounds__(256) void i8_transpose(const int8_t* __restrict__ Wp, int64_t d_out, int64_t d_in, int pieces,
                                                    int64_t groups, int own, int8_t* out, int out_pieces, int k0) {
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += (int64_t)gridDim.x * 256) {
        const int64_t piece = g / 64, i = piece / own * 16 + g % 16;
        const int kp = (int)(piece % own), k = kp * 64 + (int)(g % 64) / 16 * 16;
        u32x4 r = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int64_t o = k + j;
            uint32_t b = 0;
            if (i < d_in && o < d_out)
                b = (uint8_t)gld(Wp + (o / 16 * pieces + i / 64) * kI8Piece + (i % 64 / 16 * 16 + o % 16) * 16 + i % 16);
            r[j / 4] |= b << (8 * (j % 4));
        }
        st128(out + ((piece / own * out_pieces + k0 + kp) * 64 + g % 64) * 16, r);
    }
}

// ---- products ------------------------------------------------------------------------------

// Four results.  The channel's factor goes first: rows run up to the largest fp32 value, whose
// scale times a sum of codes is past it, weights are small.
__device__ __forceinline__ void scaled(const i32x4& acc, float s, const float (&w)[4], float (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (float)acc[j] * w[j] * s;
}
template <typename T> __device__ __forceinline__ void put1(T* out, float v, bool add) {
    if (add) v += value(gld(out));
    if constexpr (sizeof(T) == 4) gst(out, v);
    else gst(out, f_to_bf(v));
}
// Four neighbouring columns o .. o + 3 of row t, their scales in w.
template <typename T>
__device__ __forceinline__ void put4(const I8Prod& P, int64_t t, int64_t o, const i32x4& acc, float s, const float (&w)[4], bool add) {
    const int64_t left = P.d - o;
    if (left <= 0) return;
    T* out = (T*)P.out + t * P.d + o;
    float v[4];
    scaled(acc, s, w, v);
    if (P.vec) {
        if constexpr (sizeof(T) == 4) {
            if (add) {
                const u32x4 y = ld128(out);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += __uint_as_float(y[j]);
            }
            st128(out, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
        } else {
            if (add) {
                const u32x2 y = gld((const u32x2*)out);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += j & 1 ? bf_hi(y[j / 2]) : bf_lo(y[j / 2]);
            }
            gst((u32x2*)out, u32x2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])});
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) put1(out + j, v[j], add);
    }
}
// The same for bf16 and two tiles side by side (columns o0 .. o0 + 31): lanes 16 apart
// swap halves, so that each has eight neighbours and a row's 64 bytes go out in one
// instruction (as four's 32 bytes the writes took a fifth of the kernel).  All lanes of
// the wave call it; t may be past the end.
__device__ __forceinline__ void put8(const I8Prod& P, int64_t T, int64_t t, int64_t o0, const i32x4& a0, const i32x4& a1, float s,
                                     const float (&w0)[4], const float (&w1)[4], bool add) {
    float v0[4], v1[4];
    scaled(a0, s, w0, v0);
    scaled(a1, s, w1, v1);
    const int h = lane_id() / 16;
    if (add) {  // what is there, in the places where the results are now
        const int64_t o = o0 + 4 * h;
        if (t < T) {
            const uint16_t* out = (const uint16_t*)P.out + t * P.d;
            const u32x2 y0 = o < P.d ? gld((const u32x2*)(out + o)) : u32x2{0u, 0u};
            const u32x2 y1 = o + 16 < P.d ? gld((const u32x2*)(out + o + 16)) : u32x2{0u, 0u};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v0[j] += j & 1 ? bf_hi(y0[j / 2]) : bf_lo(y0[j / 2]);
                v1[j] += j & 1 ? bf_hi(y1[j / 2]) : bf_lo(y1[j / 2]);
            }
        }
    }
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const auto x = __builtin_amdgcn_permlane16_swap(pack2_bf16(v0[2 * j], v0[2 * j + 1]), pack2_bf16(v1[2 * j], v1[2 * j + 1]), false, false);
        q[j] = x[0];
        q[2 + j] = x[1];
    }
    // lanes 0..15 and 32..47 hold columns 0..7 and 8..15 of the first tile, the others the second's
    const int64_t o = o0 + 16 * (h & 1) + 8 * (h >> 1);
    if (t >= T || o >= P.d) return;
    uint16_t* out = (uint16_t*)P.out + t * P.d + o;
    if (o + 8 <= P.d) {
        *(gptr<u32x4a8>)out = q;
    } else {
        gst((u32x2*)out, u32x2{q[0], q[1]});  // d is a multiple of 4
    }
}
// The scales of columns o .. o + 3 (the array is padded to whole pieces).
__device__ __forceinline__ void column_scales(const I8Prod& P, int64_t o, float (&w)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = 1.f;
    if (P.w_scale && o < P.d) {
        const u32x4 r = ld128(P.w_scale + o);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __uint_as_float(r[j]);
    }
}

// All waves' LDS reads so far are done, and nothing moves across (unlike __syncthreads,
// it leaves the copies to LDS in flight).
__device__ __forceinline__ void step_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), the other counters at their largest
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The order of a step: its reads from LDS go between its products, two or three to each (all
// at once they fill the LDS's queue, and the products wait behind them).
template <int MB, int NB> __device__ __forceinline__ void between() {
    constexpr int READS = MB + NB, EACH = MB * NB / READS;
#pragma unroll
    for (int i = 0; i < READS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // a read
        __builtin_amdgcn_sched_group_barrier(0x008, EACH, 0);  // products
    }
    __builtin_amdgcn_sched_group_barrier(0x008, MB * NB - EACH * READS, 0);
}

// The product whose tiles of a kind hold tile `t`.
template <int KIND> __device__ __forceinline__ int product_of(const I8Prod* prods, int n, int t) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (gld(&prods[mid].tile[KIND]) <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Many rows.  A workgroup's tile: WM x WN waves of 16 MB columns of out x 16 NB rows each,
// and KG such groups of waves that take every KG-th piece of the sums (products with few
// tiles would else wait for one another's latencies step by step; their sums are joined
// through LDS).  Pieces go from memory to LDS directly, STAGES - 1 steps of 64 KG columns
// ahead of the products; a step's pieces are overwritten one barrier after all waves have
// read them.  Large tiles: 256 x 256, because a CU's LDS feeds two operands' 32 pieces to 256
// instructions; 256 x 128 with two workgroups a CU took 1211 us where these took 861.
template <typename T, int MB, int NB, int WM, int WN, int KG, int STAGES, int KIND>
__global__ __launch_bounds__(WM* WN* KG* kWave) void i8_many(I8Args a) {
    constexpr int WAVES = WM * WN, PA = MB * WM, PB = NB * WN, PER = (PA + PB) / WAVES, STAGE = (PA + PB) * KG * kI8Piece;
    static_assert(kI8Cols[KIND] == 16 * PA && (PA + PB) % WAVES == 0 && MB % 2 == 0, "every wave copies the same number of pieces");
    static_assert(KG == 1 || WAVES * KG * MB * NB * kI8Piece <= STAGES * STAGE, "the groups' sums fit LDS");
    extern __shared__ __align__(16) char smem[];
    const int lane = lane_id(), w = wave_id() % WAVES, kg = wave_id() / WAVES, wm = w % WM, wn = w / WM;
    const uint32_t lane16 = lane * 16;
    const uint32_t nt = (uint32_t)((a.T16 + PB - 1) / PB);
    const int p = uniform(product_of<KIND>(a.prods, a.n_prods, (int)(blockIdx.x / nt)));
    const I8Prod P = a.prods[p];
    // Consecutive workgroups go round the XCDs: each XCD takes a run of neighbouring tiles of every
    // product (of all products together one XCD would get the longest sums).  The tiles go in bands
    // of eight rows of tiles, column after column: neighbours share both operands.
    const uint32_t mt = (uint32_t)((P.d + 16 * PA - 1) / (16 * PA)), n = mt * nt;
    const uint32_t mine = blockIdx.x - (uint32_t)P.tile[KIND] * nt, x = mine % 8;
    const uint32_t local = x * (n / 8) + (x < n % 8 ? x : n % 8) + mine / 8;
    const uint32_t band = local / (8 * mt), in = local % (8 * mt), height = nt - band * 8 < 8 ? nt - band * 8 : 8;
    const int64_t tb = band * 8 + in % height, ob = in / height;
    // this wave's pieces of a step: the first PA are W's, the others the rows' (blocks past the end: the last)
    const int64_t o16 = (P.d + 15) / 16;
    const int8_t* src[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int piece = w * PER + i;
        int64_t b;
        if (piece < PA) {
            b = ob * PA + piece;
            src[i] = P.w + (b < o16 ? b : o16 - 1) * P.pieces * kI8Piece;
        } else {
            b = tb * PB + piece - PA;
            src[i] = a.q + (P.q0 * a.T16 + (b < a.T16 ? b : a.T16 - 1) * P.pieces) * kI8Piece;
        }
    }
    char* const lds = smem + kg * (PA + PB) * kI8Piece;
    const auto copy = [&](int k) {
        char* to = lds + (k % STAGES) * STAGE + w * PER * kI8Piece;
        int piece = k * KG + kg;  // (past the end: the last, which is not multiplied again)
        if (KG > 1 && piece >= P.pieces) piece = P.pieces - 1;
#pragma unroll
        for (int i = 0; i < PER; ++i) copy16_to_lds(src[i] + (int64_t)piece * kI8Piece + lane16, to + i * kI8Piece);
    };
    i32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    // Step k's operands are in registers while those of step k + 1 are read from LDS between its
    // products; one barrier a step: past it step k + 1's pieces are in LDS, and step k's, read by all
    // waves, make room for step k + STAGES.
    const int K = (P.pieces + KG - 1) / KG;
#pragma unroll
    for (int k = 0; k < STAGES; ++k)
        if (k < K) copy(k);
    u32x4 fa[2][MB], fb[2][NB];
    const auto read = [&](int k, int to) {
        const char* st = lds + (k % STAGES) * STAGE + lane16;
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[to][j] = *(const u32x4*)(st + (PA + wn * NB + j) * kI8Piece);
#pragma unroll
        for (int i = 0; i < MB; ++i) fa[to][i] = *(const u32x4*)(st + (wm * MB + i) * kI8Piece);
    };
    const auto multiply = [&](int of) {
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = mfma(fa[of][i], fb[of][j], acc[i][j]);
    };
    // (in flight when step k + 1 has to be there: k + 2 .. k + STAGES - 1)
    const auto ahead = [&](int k, int to) {
        wait_vmcnt_le<(STAGES - 2) * PER>((K - 2 - k < STAGES - 2 ? K - 2 - k : STAGES - 2) * PER);
        step_barrier();
        if (k + STAGES < K) copy(k + STAGES);
        read(k + 1, to);
    };
    wait_vmcnt_le<(STAGES - 1) * PER>((K - 1 < STAGES - 1 ? K - 1 : STAGES - 1) * PER);
    step_barrier();
    read(0, 0);
    int k = 0;
    for (; k + 2 < K; k += 2) {
        ahead(k, 1);
        multiply(0);
        between<MB, NB>();
        ahead(k + 1, 0);
        multiply(1);
        between<MB, NB>();
    }
    const bool whole = KG == 1 || (K - 1) * KG + kg < P.pieces;  // the last step has a piece for this group
    if (KG == 1 || k + 1 < K) {  // (KG == 1: K is even)
        ahead(k, 1);
        multiply(0);
        between<MB, NB>();
        if (whole) multiply(1);
    } else if (whole) {
        multiply(0);
    }
    if constexpr (KG > 1) {
        step_barrier();  // every wave has read its last pieces
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) *(i32x4*)(smem + ((wave_id() * MB + i) * NB + j) * kI8Piece + lane16) = acc[i][j];
        step_barrier();
    }
    // the sum of the groups' tile (i, j)
    const auto sum = [&](int i, int j) {
        i32x4 r = acc[i][j];
        if constexpr (KG > 1) {
            r = i32x4{0, 0, 0, 0};
#pragma unroll
            for (int g = 0; g < KG; ++g) r += *(const i32x4*)(smem + (((g * WAVES + w) * MB + i) * NB + j) * kI8Piece + lane16);
        }
        return r;
    };
    float sr[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int64_t t = (tb * PB + wn * NB + j) * 16 + lane % 16;
        sr[j] = t < a.T ? gld(a.scale + P.rows * a.T16 * 16 + t) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < MB; i += 2) {
        const int64_t o0 = (ob * PA + wm * MB + i) * 16;
        float w0[4], w1[4];
        column_scales(P, o0 + lane / 16 * 4, w0);
        column_scales(P, o0 + 16 + lane / 16 * 4, w1);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            if (KG > 1 && (i / 2 * NB + j) % KG != kg) continue;  // another group's to write
            const i32x4 a0 = sum(i, j), a1 = sum(i + 1, j);
            const int64_t t = (tb * PB + wn * NB + j) * 16 + lane % 16, o = o0 + lane / 16 * 4;
            if (sizeof(T) == 2 && P.vec) {
                put8(P, a.T, t, o0, a0, a1, sr[j], w0, w1, a.accumulate != 0);
            } else if (t < a.T) {
                put4<T>(P, t, o, a0, sr[j], w0, a.accumulate != 0);
                put4<T>(P, t, o + 16, a1, sr[j], w1, a.accumulate != 0);
            }
        }
    }
}

// Few rows (up to 16 TB): the weights are read once, straight into operands.  One
// workgroup: 16 CB columns of out, its waves every kFewWaves-th piece of the row; their sums
// are whole numbers, added up in LDS in any order.  A row's pieces are read once for
// CB blocks of columns.  Bound by the weights' way from memory: 202 MB in 30 us for one row,
// in 46 for 64, whose own pieces come from L2 for every CB blocks.
constexpr int kFewWaves = 8;
template <typename T, int TB, int CB, int KIND> __global__ __launch_bounds__(kFewWaves* kWave) void i8_few(I8Args a) {
    constexpr int UNROLL = TB * CB >= 16 ? 1 : TB * CB >= 8 ? 2 : TB * CB >= 4 ? 4 : 8, BLOCKS = TB * CB;
    static_assert(kI8Cols[KIND] == 16 * CB, "the kind's tiles");
    __shared__ int s_acc[BLOCKS * 256];
    for (int i = threadIdx.x; i < BLOCKS * 256; i += kFewWaves * kWave) s_acc[i] = 0;
    const int p = uniform(product_of<KIND>(a.prods, a.n_prods, blockIdx.x));
    const I8Prod P = a.prods[p];
    const int64_t ob = (int64_t)(blockIdx.x - P.tile[KIND]) * CB, last = (P.d + 15) / 16 - 1;
    const int lane = lane_id(), w = wave_id(), K = P.pieces;
    const int8_t* W[CB];
#pragma unroll
    for (int c = 0; c < CB; ++c) W[c] = P.w + (ob + c < last ? ob + c : last) * K * kI8Piece + lane * 16;
    const int8_t* X = a.q + P.q0 * a.T16 * kI8Piece + lane * 16;
    bool row[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) row[b] = b * 16 + lane % 16 < a.T;
    i32x4 acc[CB][TB];
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
        for (int b = 0; b < TB; ++b) acc[c][b] = i32x4{0, 0, 0, 0};
    for (int k0 = w; k0 < K; k0 += kFewWaves * UNROLL) {
        u32x4 fw[UNROLL][CB], fx[UNROLL][TB];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int k = k0 + u * kFewWaves;
#pragma unroll
            for (int c = 0; c < CB; ++c) fw[u][c] = k < K ? ld128_nt(W[c] + (int64_t)k * kI8Piece) : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int k = k0 + u * kFewWaves;
#pragma unroll
            for (int b = 0; b < TB; ++b)
                fx[u][b] = k < K && row[b] ? ld128(X + ((int64_t)b * K + k) * kI8Piece) : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int c = 0; c < CB; ++c)
#pragma unroll
                for (int b = 0; b < TB; ++b) acc[c][b] = mfma(fw[u][c], fx[u][b], acc[c][b]);
    }
    __syncthreads();  // the sums are clear
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
            for (int v = 0; v < 4; ++v) atomicAdd(&s_acc[(c * TB + b) * 256 + v * kWave + lane], acc[c][b][v]);
    __syncthreads();
    for (int i = w; i < BLOCKS; i += kFewWaves) {
        const int64_t t = i % TB * 16 + lane % 16, o = (ob + i / TB) * 16 + lane / 16 * 4;
        i32x4 sum;
#pragma unroll
        for (int v = 0; v < 4; ++v) sum[v] = s_acc[i * 256 + v * kWave + lane];
        float sw[4];
        column_scales(P, o, sw);
        if (t < a.T) put4<T>(P, t, o, sum, gld(a.scale + P.rows * a.T16 * 16 + t), sw, a.accumulate != 0);
    }
}

// One to four rows, codes and products in one launch: every workgroup makes the codes of its
// product's rows itself, in LDS, while its first weights are on their way.  ROWS: 1, 2 or 4,
// an equal number of waves for each.
constexpr int kTokenLds = 48 << 10;  // codes, a row's pieces and 64 bytes (LDS banks) each
template <typename T, int ROWS> __global__ __launch_bounds__(kFewWaves* kWave) void i8_token(I8Args a) {
    constexpr int UNROLL = 8, NT = kFewWaves * kWave / ROWS, KEEP = 2;
    extern __shared__ __align__(16) char smem[];
    __shared__ int s_acc[256];
    __shared__ double s_max[kFewWaves];
    __shared__ float s_scale[4];
    const int tid = threadIdx.x;
    if (tid < 256) s_acc[tid] = 0;
    const int p = uniform(product_of<kI8Few1>(a.prods, a.n_prods, blockIdx.x));
    const I8Prod P = a.prods[p];
    const int64_t ob = blockIdx.x - P.tile[kI8Few1];
    const int lane = lane_id(), w = wave_id(), K = P.pieces, pitch = K * 64 + 64;
    const int8_t* W = P.w + ob * K * kI8Piece + lane * 16;
    u32x4 fw[UNROLL];
    const auto weights = [&](int k0) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int k = k0 + u * kFewWaves;
            fw[u] = k < K ? ld128_nt(W + (int64_t)k * kI8Piece) : u32x4{0u, 0u, 0u, 0u};
        }
    };
    weights(w);
    {
        const int r = tid / NT, t = tid % NT, groups = K * 4;
        const I8Seg S = a.segs[a.rows[P.rows].seg0];
        const bool live = r < a.T;
        const T* x = (const T*)S.x + (live ? r : 0) * S.d;
        const Scale16 one(nullptr, 0, 0);
        Raw16<T> keep[KEEP];
        double top = 0.0;
        const auto raise = [&](const Raw16<T>& f) {
            const double m = top16(f, one);
            top = top > m ? top : m;
        };
#pragma unroll
        for (int c = 0; c < KEEP; ++c)
            if (c * NT + t < groups) load16(x, (int64_t)(c * NT + t) * 16, S.d, S.vec, keep[c]);
#pragma unroll
        for (int c = 0; c < KEEP; ++c)
            if (c * NT + t < groups) raise(keep[c]);
        for (int g = KEEP * NT + t; g < groups; g += NT) {
            Raw16<T> f;
            load16(x, (int64_t)g * 16, S.d, S.vec, f);
            raise(f);
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            const double q = __shfl_xor(top, o, kWave);
            top = top > q ? top : q;
        }
        if (lane == 0) s_max[w] = top;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kFewWaves / ROWS; ++v) {
            const double q = s_max[w / (kFewWaves / ROWS) * (kFewWaves / ROWS) + v];
            top = top > q ? top : q;
        }
        double by;
        float scale;
        row_scale(top, &by, &scale);
        if (t == 0) s_scale[r] = scale;
        char* out = smem + r * pitch;
#pragma unroll
        for (int c = 0; c < KEEP; ++c)
            if (c * NT + t < groups) *(u32x4*)(out + (c * NT + t) * 16) = codes16(keep[c], one, by);
        for (int g = KEEP * NT + t; g < groups; g += NT) {
            Raw16<T> f;
            load16(x, (int64_t)g * 16, S.d, S.vec, f);
            *(u32x4*)(out + g * 16) = codes16(f, one, by);
        }
        __syncthreads();
    }
    const bool row = lane % 16 < a.T;
    const char* X = smem + (row ? lane % 16 : 0) * pitch + lane / 16 * 16;
    i32x4 acc = {0, 0, 0, 0};
    for (int k0 = w; k0 < K; k0 += kFewWaves * UNROLL) {
        if (k0 != w) weights(k0);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int k = k0 + u * kFewWaves;
            const u32x4 fx = k < K && row ? *(const u32x4*)(X + k * 64) : u32x4{0u, 0u, 0u, 0u};
            acc = mfma(fw[u], fx, acc);
        }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) atomicAdd(&s_acc[v * kWave + lane], acc[v]);
    __syncthreads();
    if (w != 0 || !row) return;
    i32x4 sum;
#pragma unroll
    for (int v = 0; v < 4; ++v) sum[v] = s_acc[v * kWave + lane];
    float sw[4];
    column_scales(P, ob * 16 + lane / 16 * 4, sw);
    put4<T>(P, lane % 16, ob * 16 + lane / 16 * 4, sum, s_scale[lane % 16], sw, a.accumulate != 0);
}

constexpr int64_t kCus = 256;  // a workgroup of the large tiles' takes a CU
constexpr size_t kBigLds = 4 * (16 + 16) * kI8Piece, kMidLds = 4 * 2 * (8 + 8) * kI8Piece, kSmallLds = 4 * 4 * (4 + 4) * kI8Piece;
template <typename T> constexpr auto* kBigTile = &i8_many<T, 8, 4, 2, 4, 1, 4, kI8Big>;
template <typename T> constexpr auto* kMidTile = &i8_many<T, 4, 4, 2, 2, 2, 4, kI8Mid>;
template <typename T> constexpr auto* kSmallTile = &i8_many<T, 2, 2, 2, 2, 4, 4, kI8Small>;

template <typename T, int TB> hipError_t launch_few(const I8Args& a, hipStream_t s) {
    const dim3 n(kFewWaves * kWave);
    // as many columns a workgroup as leave two for every CU
    if constexpr (TB >= 4) {
        if (a.tiles[kI8Few4] >= 2 * kCus) {
            hipLaunchKernelGGL((i8_few<T, TB, 4, kI8Few4>), dim3((unsigned)a.tiles[kI8Few4]), n, 0, s, a);
            return hipGetLastError();
        }
    }
    if (a.T > 4 && a.tiles[kI8Few2] >= 2 * kCus)
        hipLaunchKernelGGL((i8_few<T, TB, 2, kI8Few2>), dim3((unsigned)a.tiles[kI8Few2]), n, 0, s, a);
    else
        hipLaunchKernelGGL((i8_few<T, TB, 1, kI8Few1>), dim3((unsigned)a.tiles[kI8Few1]), n, 0, s, a);
    return hipGetLastError();
}
template <typename T> hipError_t launch_products(const I8Args& a, hipStream_t s) {
    if (!grid_fits(a.tiles[kI8Few1], kFewWaves * kWave)) return hipErrorInvalidConfiguration;
    if (a.T <= kI8FewT) return a.T16 == 1 ? launch_few<T, 1>(a, s) : a.T16 == 2 ? launch_few<T, 2>(a, s) : launch_few<T, 4>(a, s);
    const auto tiles = [&](int kind) { return (a.T + kI8Cols[kind] - 1) / kI8Cols[kind] * a.tiles[kind]; };  // (square tiles)
    const int64_t big = tiles(kI8Big), mid = tiles(kI8Mid), small = tiles(kI8Small);
    // A CU takes one tile at a time, of 256, 128 or 64 square: rounds of a tile for every CU last as 24 : 10 : 4 (54, 22
    // and 9 us at 4096 columns summed).  512 rows of two 11008 x 4096 products: 58 us in large tiles, 67 in middle ones;
    // 2048 rows of one 4096 x 4096: 56 in middle ones, 65 in large, 81 in small; 128 rows 13.5 in small ones, 22 in middle.
    const auto rounds = [](int64_t n) { return (n + kCus - 1) / kCus; };
    const int64_t tb = 24 * rounds(big), tm = 10 * rounds(mid), ts = 4 * rounds(small);
    const auto go = [&](auto* kernel, int64_t n, int threads, size_t lds) {
        if (!grid_fits(n, threads)) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(threads), lds, s, a);
        return hipGetLastError();
    };
    if (tb <= tm && tb <= ts) return go(kBigTile<T>, big, 512, kBigLds);
    return tm <= ts ? go(kMidTile<T>, mid, 512, kMidLds) : go(kSmallTile<T>, small, 1024, kSmallLds);
}

}  // namespace

hipError_t prepare_i8() {
    static_assert(kMidLds == kBigLds && kSmallLds == kBigLds, "all tiles take the same LDS");
    for (const void* f : {(const void*)kBigTile<float>, (const void*)kBigTile<uint16_t>, (const void*)kMidTile<float>,
                          (const void*)kMidTile<uint16_t>, (const void*)kSmallTile<float>, (const void*)kSmallTile<uint16_t>}) {
        const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)kBigLds);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

bool i8_one_launch(const I8Args& a) {
    const int rows = a.T == 1 ? 1 : a.T == 2 ? 2 : 4;
    return a.T <= 4 && a.plain && rows * a.tiles[kI8Few1] <= 2048 && rows * (a.max_pieces * 64 + 64) <= kTokenLds;
}
hipError_t launch_i8_token(const I8Args& a, int dtype, hipStream_t s) {
    const int rows = a.T == 1 ? 1 : a.T == 2 ? 2 : 4;
    const dim3 g((unsigned)a.tiles[kI8Few1]), n(kFewWaves * kWave);
    if (!grid_fits(a.tiles[kI8Few1], kFewWaves * kWave)) return hipErrorInvalidConfiguration;
    const size_t lds = (size_t)rows * (a.max_pieces * 64 + 64);
    const auto go = [&](auto k1, auto k2, auto k4) { hipLaunchKernelGGL(rows == 1 ? k1 : rows == 2 ? k2 : k4, g, n, lds, s, a); };
    if (dtype == 0) go(i8_token<float, 1>, i8_token<float, 2>, i8_token<float, 4>);
    else go(i8_token<uint16_t, 1>, i8_token<uint16_t, 2>, i8_token<uint16_t, 4>);
    return hipGetLastError();
}
hipError_t launch_i8_rows(const I8Args& a, int dtype, hipStream_t s) {
    const auto go = [&](auto kernel, int rows, int threads) {
        // many rows: whole runs of 128, which go round the XCDs 16 at a time
        const int64_t blocks = a.T > 128 ? (a.T + 127) / 128 * (128 / rows) : (a.T + rows - 1) / rows;
        if (!grid_fits(blocks, threads)) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks, (unsigned)a.n_rows), dim3(threads), 0, s, a);
        return hipGetLastError();
    };
    // a row's values in registers where they fit
    const bool wide = a.max_pieces > 3 * 64;
    if (dtype == 0) return wide ? go(i8_rows<float, 1, 512, 3>, 1, 512) : go(i8_rows<float, 1, 256, 3>, 1, 256);
    if (a.T <= 128) return wide ? go(i8_rows<uint16_t, 1, 512, 3>, 1, 512) : go(i8_rows<uint16_t, 1, 256, 3>, 1, 256);
    return wide ? go(i8_rows<uint16_t, 2, 512, 3>, 2, 512) : go(i8_rows<uint16_t, 2, 256, 3>, 2, 256);
}
hipError_t launch_i8_products(const I8Args& a, int dtype, hipStream_t s) {
    return dtype == 0 ? launch_products<float>(a, s) : launch_products<uint16_t>(a, s);
}
hipError_t launch_i8_pack(const int8_t* W, int64_t d_out, int64_t d_in, int pieces, int8_t* out, hipStream_t s) {
    const int64_t groups = (d_out + 15) / 16 * pieces * 64, blocks = (groups + 255) / 256;
    hipLaunchKernelGGL(i8_pack, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, W, d_out, d_in, pieces, groups, out);
    return hipGetLastError();
}
hipError_t launch_i8_transpose(const int8_t* packed, int64_t d_out, int64_t d_in, int pieces, int8_t* out, int out_pieces, int k0,
                               hipStream_t s) {
    const int own = (int)((d_out + 63) / 64);
    const int64_t groups = (d_in + 15) / 16 * own * 64, blocks = (groups + 255) / 256;
    hipLaunchKernelGGL(i8_transpose, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, packed, d_out, d_in, pieces,
                       groups, own, out, out_pieces, k0);
    return hipGetLastError();
}
hipError_t launch_i8_quantize(const void* x, int64_t T, int64_t d, int dtype, int8_t* q, float* scale, hipStream_t s) {
    if (!grid_fits(T, kQT)) return hipErrorInvalidConfiguration;
    const int vec = ((uintptr_t)x & 15u) == 0 && d % (dtype == 0 ? 4 : 8) == 0;
    if (dtype == 0) hipLaunchKernelGGL(i8_quantize<float>, dim3((unsigned)T), dim3(kQT), 0, s, (const float*)x, d, vec, q, scale);
    else hipLaunchKernelGGL(i8_quantize<uint16_t>, dim3((unsigned)T), dim3(kQT), 0, s, (const uint16_t*)x, d, vec, q, scale);
    return hipGetLastError();
}

}  // namespace dlm
