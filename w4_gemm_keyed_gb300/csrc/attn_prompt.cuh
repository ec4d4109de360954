// Causal attention of whole prompts, packed one after the other: declarations.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "attention.cuh"
#include "tf_ptx.cuh"

namespace tfk {

constexpr int kMaxSeqs = 1024;

struct AttnPromptArgs {
    const uint16_t *q, *k, *v;  // bf16 [rows][ldq], [rows][ldk], [rows][ldv]
    int ldq, ldk, ldv;
    int rows, n_kv, group;
    const int64_t *starts;      // [n_seq + 1]: sequence s holds rows starts[s] .. starts[s + 1] - 1
    int n_seq;
    uint16_t *out;              // bf16 [rows][ldo]
    int ldo;
    int *err;
    void *ws;                   // the status block (256 bytes)
};
// *why is set where the failure is not a CUDA call's.
cudaError_t launch_attn_prompt(const AttnPromptArgs &a, cudaStream_t s, const char **why);

}  // namespace tfk
