// kda_block.h -- host/device interface of the kernels before and after the rule (kda_block.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct BlockInArgs {
    const void* q;
    const void* k;
    const void* f;             // raw gate [tokens, H, 128] or [tokens, H]
    const void* b;             // raw beta [tokens, H]
    const float* A_log;        // [H]
    const float* dt_bias;      // [H, 128] or [H]; nullptr: zero
    float lower_bound, eps;    // lower_bound 0: the softplus gate
    void* q_out;
    void* k_out;
    float* g;
    float* beta;
    // gradients (backward only): of the outputs, then of the inputs
    const void* dq_out;
    const void* dk_out;
    const float* dg;
    const float* dbeta;
    void* dq;
    void* dk;
    void* df;
    void* db;
    float* dA_log;
    float* ddt_bias;           // nullptr: not written
    float* part;               // workspace of block_in_partials() rows
    long long tokens;
    int H;
    bool scalar_gate, f32;
};

struct BlockOutArgs {
    const float* o;
    const void* z;
    const float* weight;       // [128]
    float eps;
    int silu;
    void* y;
    const void* dy;
    float* d_o;
    void* dz;
    float* dweight;
    float* part;               // workspace, block_out_partials() rows of 128
    long long rows;            // tokens * H
    bool f32;
};

// Rows of [H, 129] (scalar gate: [H, 2]) that the backward kernel leaves for its second stage.
int block_in_partials(long long tokens, int H);
int block_out_partials(long long rows);

hipError_t launch_block_in(const BlockInArgs& a, hipStream_t s);
hipError_t launch_block_in_bwd(const BlockInArgs& a, hipStream_t s);
hipError_t launch_block_out(const BlockOutArgs& a, hipStream_t s);
hipError_t launch_block_out_bwd(const BlockOutArgs& a, hipStream_t s);

}  // namespace kda
