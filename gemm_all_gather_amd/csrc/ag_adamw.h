// Internal interface between the AdamW optimizer's host code (ag_adamw_host.cpp)
// and its kernels (ag_adamw.hip).  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ag {

// One tensor in the device table.
struct AdamwEntry {
    void* param;
    const void* grad;
    void* exp_avg;
    void* exp_avg_sq;
    float* exp_avg_scale;
    float* exp_avg_sq_scale;
    float* master;
    int64_t n;
    int64_t first_block;     // blocks of AG_ADAMW_BLOCK elements in the tensors before it
};

// One workgroup's elements: kAdamwChunk of one tensor.
struct AdamwChunk {
    uint32_t tensor;
    uint32_t chunk;
};
constexpr int kAdamwChunk = 4096;

// A step's scalars in fp32, each rounded once from fp64.
struct AdamwScalars {
    float b1, one_minus_b1, b2, one_minus_b2;
    float decay, rate, inv_bias2, eps;      // p decay - rate m / (sqrt(v inv_bias2) + eps)
    float grad_scale;
    uint64_t seed;                          // mixed
};

// A seed's 64 bits spread over all of them: a step of SplitMix64 (Steele, Lea and Flood 2014), with its constants.
__host__ __device__ inline uint64_t adamw_mix_seed(uint64_t z)
{
    z += 0x9E3779B97F4A7C15ull;
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

struct AdamwArgs {
    const AdamwEntry* entries;
    const AdamwChunk* chunks;
    AdamwScalars scalars;
    double beta1, beta2, one_minus_beta1, one_minus_beta2;
    double lr, weight_decay, grad_scale, bias1, bias2;
    const int64_t* dev_step;
    const float* dev_lr;
    const float* dev_grad_scale;
    uint64_t seed;                          // as given
    int32_t stochastic;
    int32_t reserved;
};

struct AdamwLaunch {
    AdamwArgs args;
    int64_t chunks;
    int param, grad;     // ag_dtype_t
    int master;
    int state8;
};
hipError_t launch_adamw(const AdamwLaunch& l, hipStream_t stream);

// fp32 outputs of the 8-bit states, kAdamwReadTensors tensors a launch.
constexpr int kAdamwReadTensors = 64;
struct AdamwReadArgs {
    const AdamwEntry* entries;       // of the first tensor
    float* exp_avg[kAdamwReadTensors];
    float* exp_avg_sq[kAdamwReadTensors];
    uint32_t first_group[kAdamwReadTensors + 1];   // workgroups before each tensor
    int32_t count;
    int32_t reserved;
};
hipError_t launch_adamw_read(const AdamwReadArgs& a, hipStream_t stream);

}  // namespace ag
