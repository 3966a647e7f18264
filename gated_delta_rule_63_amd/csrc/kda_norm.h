// kda_norm.h -- host/device interface of the residual's addition with an RMS norm (kda_norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kNormMaxC = 16384;

struct NormArgs {
    const void* x;
    const void* res;           // nullptr: the norm of x alone
    const float* weight;       // [C]
    float eps;
    void* y;                   // x's type, or one byte a value
    void* r;                   // the sum as it is stored
    float* scales;             // 8-bit outputs: [rows, C / group]
    // gradient
    const void* dy;
    const void* dr;            // nullptr: zero
    void* dx;
    void* dres;                // nullptr: not written
    float* dweight;
    float* part;               // workspace, norm_partials() rows of C
    long long rows;
    int C;
    int group;                 // 0: a row
    bool f32, res_f32, q8;
    int vec;                   // neighbours that make up every row: 8, 4, 2 or 1
};

int norm_partials(long long rows, int C);

hipError_t launch_add_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_add_norm_bwd(const NormArgs& a, hipStream_t s);

}  // namespace kda
