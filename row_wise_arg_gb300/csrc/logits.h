// Host-side declarations of the vocabulary-row operators (argreduce_logprobs,
// argreduce_distill and their gradients): the problem as the launchers see it,
// the planner and the launchers of each element type.
#pragma once

#include "internal.h"

namespace argr {

// Properties of the current device (api.cpp), cached per device.
argr_status current_caps(argr_caps* out);

struct LogitsProblem {
    const void* x;
    int dtype;
    int64_t rows;
    int cols;
    int64_t row_stride;  // elements
    float temperature, inv_t;  // and 1 / temperature
    // log probabilities
    const int64_t* tokens;
    int top_k;
    float* logprob;
    float* entropy;
    float* lse;
    int64_t* top_ids;
    float* top_logprobs;
    // distillation
    const int64_t* ids;
    const float* teacher;
    int slots;
    int tail;
    float* loss;
    // gradients
    float4* stats;  // written by the forward pass, read by the gradients
    const float* grad_logprob;  // grad_loss for the distillation
    const float* grad_entropy;
    const float* grad_lse;
    void* grad;
    int64_t grad_stride;
    cudaStream_t stream;
};

// Bytes of a row that a CTA of the step's kernel holds, at most: two CTAs per SM.
constexpr int64_t kStepMaxChunk = 108 * 1024;

// Shared memory of a CTA of the persistent forward kernel, for the planner: k
// alternatives (distill == false) or slots, `warps` in all.
size_t logits_stream_smem(bool distill, int64_t cols, int dtype, int k, int warps, int finishers);

// Planner (plan_logits.cpp): pure host code.
argr_status make_logits_plan(int what, int64_t rows, int64_t cols, int dtype, int k, const argr_caps& caps,
                             argr_plan* out);
argr_status check_logits_plan(int what, const argr_plan& p, int64_t rows, int64_t cols, int dtype, int k,
                              const argr_caps& caps);

#define ARGR_DECLARE_LOGITS(sfx)                                                         \
    cudaError_t launch_logprobs_##sfx(const argr_plan& p, const LogitsProblem& pr);      \
    cudaError_t launch_distill_##sfx(const argr_plan& p, const LogitsProblem& pr);       \
    cudaError_t read_and_clear_logits_error_##sfx(unsigned* out);                        \
    cudaError_t launch_distill_step_##sfx(const argr_plan& p, const LogitsProblem& pr);  \
    cudaError_t launch_logprobs_grad_##sfx(const argr_plan& p, const LogitsProblem& pr); \
    cudaError_t launch_distill_grad_##sfx(const argr_plan& p, const LogitsProblem& pr);
ARGR_DECLARE_LOGITS(f32)
ARGR_DECLARE_LOGITS(f16)
ARGR_DECLARE_LOGITS(bf16)
#undef ARGR_DECLARE_LOGITS

}  // namespace argr
