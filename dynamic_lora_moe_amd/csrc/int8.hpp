// Structures shared between the host API (api_train.hip) and the kernels of the 8-bit
// products.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dlm {

// Codes are kept as the matrix instructions take them: a piece of 16 rows x 64 columns is
// 1 KB, 16 bytes (columns 16 h .. 16 h + 15 of row r) at 16 (16 h + r); the pieces of 16
// rows follow one another along the columns, an even number of them.
constexpr int kI8Piece = 1024;
constexpr int64_t kI8MaxK = 131072;  // 128 * 127 * kI8MaxK < 2^31: sums are exact

// One run of a row of codes: d values of x, times scale[.] where there is one.
struct I8Seg {
    const void* x;       // [T][d]
    const float* scale;  // [d] or nullptr
    int64_t d;
    int32_t k0;          // its first 64-column piece in the row
    int32_t vec;         // rows take 16-byte accesses
};
// One matrix of codes made from a call's inputs: runs seg0 .. seg1 - 1.
struct I8Rows {
    int32_t seg0, seg1, pieces, pad;
    int64_t q0;          // pieces (per 16 rows) before its codes
    int64_t index;       // its place among the row scales
};
// One product: out[t][o] = scale of row t * w_scale[o] * sum_k codes[t][k] w[o][k].
struct I8Prod {
    const int8_t* w;       // packed [ceil(d / 16)][pieces]
    const float* w_scale;  // [d, padded to a multiple of 16], or nullptr (1)
    void* out;             // [T][d]
    int64_t d;
    int32_t pieces;        // 64-column pieces of a row, even
    int32_t vec;           // rows of out take accesses of four elements
    int64_t q0;            // of its I8Rows
    int64_t rows;
    int32_t tile[6], pad[2];  // tiles of earlier products (per row tile), by kind
};

struct I8Args {
    const I8Seg* segs;
    const I8Rows* rows;
    const I8Prod* prods;
    int32_t n_rows, n_prods;
    int32_t tiles[6];     // of all products, by kind
    int64_t T, T16;       // rows, and 16-row blocks
    int64_t pieces;       // of all I8Rows together (per 16 rows)
    int32_t max_pieces;   // of the longest row
    int32_t plain;        // every row of codes is one run without factors
    int8_t* q;            // codes: matrix i at q0_i * T16 pieces
    float* scale;         // [n_rows][T16 * 16]
    int32_t accumulate;
};

// Kinds of tiles, and their columns of out: many rows, in three sizes; few rows, by how
// many 16-column blocks share a read of the rows.
enum { kI8Big = 0, kI8Mid = 1, kI8Small = 2, kI8Few1 = 3, kI8Few2 = 4, kI8Few4 = 5 };
constexpr int kI8Cols[6] = {256, 128, 64, 16, 32, 64};
constexpr int kI8FewT = 64;  // rows that count as few

hipError_t prepare_i8();
// Whether codes and products take one launch (few rows, codes that fit LDS), and that launch.
bool i8_one_launch(const I8Args& a);
hipError_t launch_i8_token(const I8Args& a, int dtype, hipStream_t s);
hipError_t launch_i8_rows(const I8Args& a, int dtype, hipStream_t s);
hipError_t launch_i8_products(const I8Args& a, int dtype, hipStream_t s);
// Weights: row-major codes to pieces, and from pieces to their transpose's at `k0`.
hipError_t launch_i8_pack(const int8_t* W, int64_t d_out, int64_t d_in, int pieces, int8_t* out, hipStream_t s);
hipError_t launch_i8_transpose(const int8_t* packed, int64_t d_out, int64_t d_in, int pieces, int8_t* out, int out_pieces,
                               int k0, hipStream_t s);
hipError_t launch_i8_quantize(const void* x, int64_t T, int64_t d, int dtype, int8_t* q, float* scale, hipStream_t s);

}  // namespace dlm
