// Attention of a batch of sequences whose rows are trees of drafted tokens: declarations.
#pragma once
#include "kv_batch.cuh"

namespace tfk {

struct AttnTreeArgs {
    KvBatch own, prefix;    // prefix: n_seq = 1; not read when prefix_len == 0
    int prefix_len;
    int group, n;           // query heads per KV head; nodes of a tree
    const uint16_t *q;      // bf16 [n_seq * n][ldq]
    int ldq;
    const int64_t *pos;     // [n_seq]
    const int32_t *parents; // [n_seq][n]
    uint16_t *out;          // bf16 [n_seq * n][ldo]
    int ldo;
    int *err;
    void *ws;               // attn_tree_bytes(); zero-filled once
};
size_t attn_tree_bytes(const KvBatch &own, int prefix_len, int group, int n);
// *why is set where the failure is not a CUDA call's.
cudaError_t launch_attn_tree(const AttnTreeArgs &a, cudaStream_t s, const char **why);

}  // namespace tfk
