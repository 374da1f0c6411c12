// Internal declarations of the operators in include/mxfp8_step.h.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mxw {

struct TokenPlanArgs {
    const void* ids;
    int id64, first, local, align;
    int64_t pairs, rows;
    int32_t *offs, *slot, *src;
    int dev;
    int* status;
    cudaStream_t stream;
};

int launch_token_plan(const TokenPlanArgs& a);

// A plan and the buffers that it joins: `tok` [T][H] in token order, `sorted`
// [rows][H]; which one is read and which written is the operator's.
struct TokenArgs {
    int64_t T, rows;
    int H, top_k;
    const int32_t *slot, *src;
    const uint16_t *tok_in, *sorted_in;
    uint16_t *tok_out, *sorted_out;
    uint8_t *q, *s;        // dispatch to MXFP8 (q != nullptr)
    const float* weights;  // combine; nullptr: all one
    float* dweights;
    int num_sms;
    int* status;
    cudaStream_t stream;
};

int launch_token_dispatch(const TokenArgs& a);
int launch_token_combine(const TokenArgs& a);
int launch_token_combine_grad(const TokenArgs& a);

struct GradArgs {
    const void* const* grads;
    const int64_t* sizes;
    const int32_t* types;
    void* const* outs;  // nullptr: in place
    int n;
    bool clip;          // false: the norm only
    float max_norm, eps;
    const float* norm_in;
    float* norm;
    double* ws;
    int num_sms;
    cudaStream_t stream;
};

size_t grad_ws_bytes(int n);
int launch_grads(const GradArgs& a);

}  // namespace mxw
