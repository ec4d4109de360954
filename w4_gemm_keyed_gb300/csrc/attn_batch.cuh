// Attention of a batch of sequences over a shared prefix and their own caches:
// declarations.
#pragma once
#include "kv_batch.cuh"

namespace tfk {

struct AttnBatchArgs {
    KvBatch own, prefix;    // prefix: n_seq = 1; not read when prefix_len == 0
    int prefix_len;
    int group, R;
    const uint16_t *q;      // bf16 [n_seq * R][ldq]
    int ldq;
    const int64_t *pos;     // [n_seq]
    uint16_t *out;          // bf16 [n_seq * R][ldo]
    int ldo;
    int *err;
    void *ws;               // attn_batch_bytes(): the status block (256 bytes), then scratch
};

size_t attn_batch_bytes(const KvBatch &own, int prefix_len, int group, int R);
// *why is set where the failure is not a CUDA call's.
cudaError_t launch_attn_batch(const AttnBatchArgs &a, cudaStream_t s, const char **why);

}  // namespace tfk
