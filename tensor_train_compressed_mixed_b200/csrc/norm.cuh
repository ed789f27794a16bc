// The norm over all gradients of a list of tensors, on the device: what clipping and AdamW's clipped step share.
#pragma once

#include <vector>

#include "types.cuh"

namespace tt {

constexpr int kNormTensors = 128;   // tensors of one launch; their records travel as its parameters

struct NormRec {
    void* grad;
    const int32_t* guard;
    int64_t size;
    int64_t tile0;     // first tile of the tensor, counted over the launch
    int32_t type;      // tt_dtype
    int32_t lead;      // values before the first one that begins a vector of 16 bytes
};
struct NormList {
    int32_t count;
    int32_t first_slot;   // of the launch's partial sums
    int64_t tiles;
    NormRec r[kNormTensors];
};

// What a call leaves for the kernels behind it.
struct NormResult {
    uint32_t ticket;
    int32_t finite;    // whether the norm is a number
    float factor;      // of every gradient: bound / norm where the norm is above the bound, else 1
};

// The plan of one list (host).
struct NormPlan {
    std::vector<NormList> lists;
    std::vector<int> grids;
    int slots = 0;
    bool few = false;         // so little that one cluster clips in one launch
    char* mem = nullptr;      // the owner's device memory: a NormResult, and the partial sums from byte 256 on; cleared before the first call
    NormResult* result() const { return (NormResult*)mem; }
    size_t bytes() const { return 256 + (size_t)slots * sizeof(double); }
};

// For a device of `sms` SMs, the current one.  clips: gradients are to be scaled in place, too.  May throw std::bad_alloc.
void norm_plan(NormPlan& p, int sms, bool clips, int32_t count, const tt_emb_norm_tensor* tensors);
// Cleared device memory on the current device; waited for, as the first call may run on a stream that is not ordered behind this one.
cudaError_t cleared(void** mem, size_t bytes);
// Sums, the norm (rounded once to *norm, which may be null) and the factor for `bound`.
cudaError_t norm_launch(const NormPlan& p, float bound, float* norm, cudaStream_t s);
// The same, and every gradient times the factor, in place.
cudaError_t norm_clip(const NormPlan& p, float bound, float* norm, cudaStream_t s);

}  // namespace tt
