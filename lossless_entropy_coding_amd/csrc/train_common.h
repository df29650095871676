// Launch interface of the weight update.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ec {

constexpr uint32_t kAdamTensors = 56;       // a launch's, in its arguments
// State blocks of a step, more than a card's memory holds: a launch's chunks of
// four blocks, at most one begun a tensor, are then counted in 32 bits.
constexpr uint64_t kAdamBlocks = 1ull << 32;

struct AdamTensor {
    float *p;
    const void *g;
    uint16_t *copy;                         // bf16, or null
    uint64_t n, block;                      // block: the first of its state
    float decay;
    uint32_t grad_bf16;
};

struct AdamArgs {
    void *m, *v;
    float *m_scale, *v_scale;
    int32_t *steps;
    const float *lr_at, *grad_scale;        // or null
    float lr, b1, b2, rest1, rest2, log_b1, log_b2, eps;
    uint32_t seed;
    uint32_t e4m3;
};

struct AdamPart {                           // of a launch
    AdamTensor t[kAdamTensors];
    uint32_t first[kAdamTensors];           // chunk
    uint32_t count, chunks;
    AdamArgs a;
};
static_assert(sizeof(AdamPart) <= 4096, "kernel arguments");

// Collects tensors and launches whenever a launch is full.
struct AdamBatch {
    AdamPart part;
    hipStream_t stream;
    bool launched = false;

    AdamBatch(const AdamArgs &a, hipStream_t s) : stream(s) {
        part.a = a;
        part.count = part.chunks = 0;
    }
    hipError_t add(const AdamTensor &t);
    hipError_t launch(bool alone);           // alone: the only launch of the step
    hipError_t finish();                    // the last launch, and the step's number
};

uint64_t adamw_blocks(uint64_t n);

}  // namespace ec
