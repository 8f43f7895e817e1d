// Structures shared between the host API (api_train.hip) and the kernels of the
// orthogonalised momentum step.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dlm {

constexpr int kMuonMaxSide = 512;   // the smaller side of a matrix
constexpr int kMuonMaxSteps = 10;
constexpr int kMuonTileSide = 64;   // up to here one workgroup holds a matrix's square ones

// One tensor: `count` matrices of a small side n and a long side d.
struct MuDesc {
    void* p;
    const void* g;
    float* master;    // or nullptr
    float* m;
    float* u;         // fp32 scratch of the tensor's layout (small side above kMuonTileSide)
    int64_t d, count;
    int32_t n;
    int32_t wide;     // element (i of n, j of d) lies at i d + j, else at j n + i
    int32_t vec;      // rows allow four elements per access
    int32_t chunks;   // pieces of the long side
    int64_t item0;    // its first piece of its class's launches
    int64_t mat0;     // its first matrix of its class
    float wd, scale;
};

// One matrix with a small side above kMuonTileSide.
struct MuBig {
    int32_t desc, nb;  // its tensor; 16-wide blocks of the small side, a multiple of 4
    int64_t index;     // its place in the tensor
    int64_t part0;     // its first part (64 x 64 sums of one chunk)
    int64_t off;       // doubles before its square matrices
};

struct MuonArgs {
    const MuDesc* descs;
    const int32_t* item_desc;  // of every piece
    double* part;              // sums of the pieces
    double* pm;                // [matrix] the product's square matrix, in fragments
    int32_t* bad;              // [matrix] 1: not finite
    int32_t* err;
    int64_t items, mats;
    int32_t chunk;             // long-side elements of a piece
    const int32_t* mat_desc;   // of every matrix
    // big matrices
    MuBig only;                // the first
    const MuBig* big;
    const int32_t* pair_big;   // per (matrix, chunk, pair of 64-blocks)
    const int32_t* sum_big;    // per (matrix, pair)
    const int32_t* sum_pair;   // the pair's number within its matrix
    const int32_t* mul_big;    // per 16 x 16 block
    const int32_t* mul_at;     // which of the matrix's
    const int32_t* out_big;    // per (matrix, 64 of its long side, 64 of its small side)
    const int32_t* out_at;     // which of them
    int64_t n_big, n_pair, n_sum, n_mul, n_out, sq;  // sq: doubles of one square matrix of all
    double* square;            // six square matrices of each
    double* meta;              // [matrix][2] 1 / norm, 1 / norm^2
    double beta;
    float lr, eps;
    int32_t nesterov, steps;
    double coefs[kMuonMaxSteps][3];
    const float* lr_scale;    // device, or nullptr
    const float* grad_scale;  // device, or nullptr
};

// Long-side elements of one piece, for nb 16-wide blocks of the small side (1, 2 or 4): of wider ones
// half as many where that leaves CUs without one (odd sizes 97 us against 75; 70B-shaped banks in halves
// 363 against 351).
constexpr int muon_chunk(int nb, bool few) { return nb == 1 || !few ? 512 : 256; }
// Doubles of one piece's sums: the blocks on and above the diagonal; 64 x 64 of a big matrix.
constexpr int muon_part(int nb) { return nb * (nb + 1) / 2 * 256; }
constexpr int kMuonBigPart = 16 * 256;
constexpr int64_t kMuonFewItems = 512;  // pieces that classes share launches up to
constexpr int kMuonBigChunk = 256;  // long-side elements of a big matrix's piece

// Once per handle on its device, before its first launch.
hipError_t prepare_muon();
// Matrices with a small side up to 16, 32 and 64 (no items: none).
hipError_t launch_muon(const MuonArgs (&a)[3], int p_dtype, int g_dtype, hipStream_t s);
hipError_t launch_muon_big(const MuonArgs& a, int64_t u_elems, int p_dtype, int g_dtype, hipStream_t s);

}  // namespace dlm
