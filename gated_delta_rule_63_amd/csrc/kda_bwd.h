// kda_bwd.h -- host/device interface of the gradient kernels (kda_bwd.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

constexpr int kBwdChunk = 32;

// Layouts: q, k, v, g, d_o and their gradients as in include/kda.h. A chunk of
// a (sequence, head) has the index ch = slot * H + h; the workspace arrays
// below are fp32 and indexed by it. Matrices are kept as 16 x 16 tiles of 1 KiB,
// row after row, so that a wave's fragment is one contiguous piece; "T" in a
// name: [channel][token], tiles in the order (channel tile, token tile).
struct BwdArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    const float* d_o;
    const int32_t* cu;
    const float* h0;     // nullptr: zero
    const float* dhT;    // nullptr: zero
    void* dq;
    void* dk;
    void* dv;
    float* dg;
    float* dbeta;
    float* dh0;          // nullptr: not written
    float* X;            // [32][32]
    float* MT;           // [32][32], M transposed; the block of tokens 0..15 by 16..31 is unset
    float* b;            // [32] beta, zero behind the last token
    float* decay;        // [128] exp(sum of g over the chunk)
    float* WT;           // 128 x 32
    float* eT;           // 128 x 32, e
    float* dDT;          // 128 x 32, dDelta
    float* KcT;          // 128 x 32
    float* QrT;          // 128 x 32
    float* S;            // 128 x 128, [v][k], tiles (v tile, k tile): state entering the chunk
    float* dS;           // the same: gradient of the state leaving it
    int B, T, H, N, nslots;
    bool scalar_gate, f32;
};

// Slots of a descriptor: ceil(T / 32) per row, or with cu_seqlens
// floor(T / 32) + N, sequence n starting at slot floor(cu[n] / 32) + n.
long long bwd_slots(int B, int T, int N, bool varlen);

// The three kernels in order.
hipError_t launch_bwd(const BwdArgs& a, int cus, hipStream_t stream);

}  // namespace kda
