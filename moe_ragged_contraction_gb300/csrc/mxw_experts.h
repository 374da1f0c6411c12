// Internal declarations of the operators in include/mxfp8_experts.h.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mxw {

struct MoeArgs {
    const uint16_t* x;
    const uint16_t* router;
    const float* bias;
    const uint8_t *w13, *s13, *w2, *s2;
    int T, experts, first, local, H, I, top_k, score, renormalize;
    float scale;
    uint16_t* out;
    int32_t* ids;
    float* weights;
    uint8_t* ws;
    int dev, num_sms, stall;
    uint64_t wait_limit_ns;
    int* status;
    cudaStream_t stream;
};

// Scratch of one call (bytes), the same for every routing of T tokens.
size_t moe_ws_bytes(int T, int experts, int local, int H, int I, int top_k, int num_sms);
int launch_moe(const MoeArgs& a);

struct MuonArgs {
    const void* grad;
    int grad_f32;
    float* momentum;
    int E, N, K, nesterov, steps;
    float mu, a, b, c, eps;
    uint16_t* out;
    uint8_t* ws;
    int dev, num_sms, stall;
    uint64_t wait_limit_ns;
    int* status;
    cudaStream_t stream;
};

size_t muon_ws_bytes(int E, int N, int K);
int launch_muon(const MuonArgs& a);

// Matrices that one cluster holds on chip (muon_small.cu): no scratch.
bool muon_fits_small(int N, int K);
int launch_muon_small(const MuonArgs& a);

}  // namespace mxw
