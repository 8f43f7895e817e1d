// Structures shared between the host API (api_train.hip) and the balance kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dlm {

// Where the parts of a balance call's workspace lie.  The rows are cut in blocks of
// `per`; a block's rows of sequence q are one part, numbered block + q: along the
// rows each step raises one of the two or both, so no two parts share a number.
struct BalanceLayout {
    int64_t per, blocks, slots;
    size_t p, z, seq, c, n, ticket, bytes;  // byte offsets of the arrays, and the total
};

struct BalanceArgs {
    const void* logits;      // [T] rows of E, ld elements apart
    int64_t ld, T;
    const int32_t* idx;      // [T][k]
    const int32_t* offsets;  // [S + 1], or nullptr: one sequence of every row
    int32_t S, E, k, score;
    int32_t vec, vec_out;    // rows of logits / dlogits take 16-byte accesses
    float alpha, zeta;
    int64_t per, blocks;
    // parts: sums of p [slots][E], of lse^2 [slots], counts [slots][E], rows [slots];
    // then every sequence's two terms [S][pieces][2], and the count of pieces done
    double* part_p;
    double* part_z;
    double* seq;
    int32_t* part_c;
    int32_t* part_n;
    uint32_t* ticket;
    float* loss;             // [2]
    int32_t* counts;         // [S][E]
    int32_t* rows;           // [S]
    float* probs;            // [S][E]
    // gradient
    const int32_t* in_counts;
    const int32_t* in_rows;
    const float* dloss;      // [2], or nullptr: 1, 1
    void* dlogits;           // [T] rows of E, ldd elements apart
    int64_t ldd;
    int32_t accumulate;
};

BalanceLayout balance_layout(int64_t T, int E, int S);
hipError_t launch_balance(const BalanceArgs& a, int dtype, hipStream_t s);
hipError_t launch_balance_grad(const BalanceArgs& a, int dtype, hipStream_t s);

}  // namespace dlm
