// kda_beam.h -- host/device interface of a step of beam search (kda_beam.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

constexpr int kBeamMax = 64;           // beams of a batch entry, and places selected

// A part of a row: its largest logit, or one at most one below it, sum of exp(logit - max), and its best
// candidates as keys (see kda_beam.hip), descending, zeros behind the last.
struct BeamPart {
    float max;
    int pad;
    double sum;
};

struct BeamArgs {
    const void* logits;                // [B, W, V]
    const float* scores;               // [B, W]
    const uint8_t* done;               // [B, W], nullptr: none
    float* out_scores;                 // [B, K]
    int32_t* parents;
    int32_t* tokens;
    BeamPart* parts;                   // workspace: [B * W, splits]
    uint64_t* keys;                    // workspace: [B * W, splits, K]
    int B, W, V, K, eos, splits;
    bool f32;
};

struct ReorderArgs {
    char* pool;
    size_t slot_bytes;
    const int32_t* slots;              // [B, W]
    const int32_t* parents;            // [B, W]
    int32_t* new_slots;                // [B, W]
    int B, W, num_slots;
    int unit;                          // bytes of a copied piece: 16, 4 or 1
};

// Parts that a row is cut into, each a workgroup's.
int beam_splits(int B, int W, int V, bool f32, int cus);

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s);
hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t s);

}  // namespace kda
