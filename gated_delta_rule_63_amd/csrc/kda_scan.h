// kda_scan.h -- host/device interface of the rule with a vector state (kda_scan.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kScanChunk = 128;   // tokens between kept states
constexpr int kScanStrip = 64;    // channels of a workgroup

struct ScanArgs {
    const void* x;
    const float* g;
    const int32_t* cu;            // nullptr: N rows of T tokens
    const float* h0;              // [N, C], nullptr: zero
    void* y;
    float* hT;                    // [N, C], nullptr: not written
    float* states;                // [scan_slots(), C]; the forward writes them if there, the gradient reads them
    // gradient
    const void* dy;
    const float* dhT;             // [N, C], nullptr: zero
    void* dx;
    float* dg;
    float* dh0;                   // [N, C], nullptr: not written
    // workspace of the split form, [scan_slots(), C] each: a chunk's decay, what it adds to the state,
    // what it adds to the gradient, in whose place the gradient that leaves it is put, and decays past fp32's range
    float* decays;
    float* adds;
    float* grads;
    float* bigs;
    int T, C, N;
    long long slots;
    bool f32, leaky;
    int width;                    // scan_width()
    bool fold;                    // side by side: a chunk's workgroup folds those before it itself
    bool stream;                  // more bytes than the last-level cache holds
};

struct ScanPoolArgs {
    const void* x;
    const float* g;
    const int32_t* cu;
    const int32_t* slots;
    const int32_t* out_slots;
    void* pool;                   // [num_slots, C]
    void* y;
    int T, C, N, num_slots;
    bool f32, leaky, pool_bf16;
    bool vec;                     // four neighbouring channels can be read and written at once
};

// Rows of `states`: one for each chunk of each sequence; packed, sequence n's begin at row cu[n] / 128 + n.
long long scan_slots(int B, int T, int N, bool packed);
// How a call runs: channels of a workgroup that goes through a sequence (64, 32, 16), or 0:
// its chunks side by side, in three kernels.
struct ScanForm {
    int rows, T, C, N;            // rows of T tokens, sequences
    bool packed, f32, leaky;
    bool back, known;             // the gradient; with the forward's states
};
int scan_width(const ScanForm& f, int cus);

hipError_t launch_scan(const ScanArgs& a, hipStream_t s);
// known: `states` holds the forward's; else it is formed first.
hipError_t launch_scan_bwd(const ScanArgs& a, bool known, hipStream_t s);
hipError_t launch_scan_recurrent(const ScanPoolArgs& a, hipStream_t s);

}  // namespace kda
