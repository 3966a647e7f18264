// kda_recurrent.h -- host/device interface of the recurrent kernel (kda_recurrent.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

struct RecurrentArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    const int32_t* cu;         // nullptr: N rows of T tokens
    const int32_t* slots;      // [N], nullptr: sequence n uses slot n
    const int32_t* out_slots;  // one per token, nullptr: the last state goes back to its slot
    void* pool;                // [num_slots, H, 128, 128] fp32 or bf16
    float* o;
    int T, H, N, num_slots;
    bool scalar_gate, f32, pool_bf16;
};

hipError_t launch_recurrent(const RecurrentArgs& a, int cus, hipStream_t stream);

}  // namespace kda
