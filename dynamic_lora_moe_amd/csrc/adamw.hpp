// Structures shared between the host API (api.hip) and the AdamW kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dlm {

// Elements one workgroup updates (of one tensor), and of one block of 8-bit moments.
constexpr int kAdamChunk = 4096;
constexpr int kAdamBlock = 256;

struct AdDesc {
    void* p;
    const void* g;
    float* master;   // or nullptr
    void* m;         // fp32, or int8 codes
    void* v;         // fp32, or uint8 codes
    float* ms;       // 8-bit moments: one scale per block
    float* vs;
    int64_t n;
    int64_t chunk0;  // first chunk of this tensor (prefix sum)
    float wd;
    int32_t vec;     // every pointer allows four elements per access
};

struct AdamArgs {
    const AdDesc* descs;
    const int32_t* chunk_tensor;  // the tensor of every chunk
    int32_t* steps;               // steps taken, one count per chunk
    int32_t* err;                 // set where a gradient is not finite
    int64_t n_chunks;
    double beta1, beta2, lb1, lb2;  // and their natural logarithms
    float lr, eps;
    uint32_t seed;
    const float* lr_scale;    // device, or nullptr
    const float* grad_scale;  // device, or nullptr
};

hipError_t launch_adamw(const AdamArgs& a, int p_dtype, int g_dtype, int bits, hipStream_t s);
hipError_t launch_adamw_read_state(const int8_t* m, const uint8_t* v, const float* ms, const float* vs, int64_t n,
                                   float* m_out, float* v_out, hipStream_t s);

}  // namespace dlm
