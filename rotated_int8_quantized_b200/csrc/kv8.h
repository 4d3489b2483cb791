// kv8.h -- launch interface of the attention-side kernels: head norms with
// rotation, the paged INT8 key/value cache, and attention over it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace convrot {

constexpr int kKvBlock = 16;              // cached tokens that share a scale

// Rows of `heads` x `dim` BF16 values, strides in elements.
struct HeadRows {
    const uint16_t *p;
    int64_t ts, hs;
};
struct HeadRowsOut {
    uint16_t *p;
    int64_t ts, hs;
};

struct RopeArgs {
    const float *cs;                      // [rows][rot / 2][2], nullptr: no rotation
    int64_t rows;
    const uint8_t *axis;                  // [rot / 2] or nullptr
    const int32_t *pos;                   // [axes][tokens] or nullptr (the cache position)
    int32_t rot, adjacent, axes;
};

struct NormRopeArgs {
    int64_t tokens;
    int32_t q_heads, kv_heads, dim;
    HeadRows q, k;
    HeadRowsOut q_out, k_out;
    const uint16_t *qw, *kw;              // BF16 [dim] or nullptr
    float eps;
    RopeArgs rope;
};

// The sequences of a step and where their cached tokens lie.
struct KvSeqs {
    const int32_t *table;                 // [batch][max_pages]
    const int32_t *kv_len;                // [batch]
    const int32_t *cu;                    // [batch + 1] or nullptr: one token each
    int64_t tokens;                       // rows of the step's tensors
    int64_t pages;
    int32_t batch, max_pages, page_shift; // page_tokens = 1 << page_shift
};

struct KvCache {
    int8_t *k, *v;
    float *ks, *vs;
    int32_t heads, dim;
};

struct AppendArgs {
    KvCache c;
    KvSeqs s;
    int32_t q_heads;
    HeadRows q, k, v;
    HeadRowsOut q_out;
    const uint16_t *qw, *kw;
    float eps;
    RopeArgs rope;
};

struct ReadArgs {
    KvCache c;
    KvSeqs s;
    uint16_t *k_out, *v_out;              // [tokens][heads][dim], either may be nullptr
};

struct AttnArgs {
    KvCache c;
    KvSeqs s;
    int32_t q_heads;
    HeadRows q;
    uint16_t *out;                        // [tokens][q_heads][dim]
    float *lse;                           // [tokens][q_heads] or nullptr
    float scale;                          // softmax scale
    int32_t causal;
    void *ws;
};

cudaError_t launch_norm_rope(const NormRopeArgs &a, int sms, cudaStream_t stream);
cudaError_t launch_kv8_append(const AppendArgs &a, int sms, cudaStream_t stream);
cudaError_t launch_kv8_read(const ReadArgs &a, int sms, cudaStream_t stream);
cudaError_t launch_attn_kv8(const AttnArgs &a, int sms, cudaStream_t stream);
int64_t attn_kv8_workspace_bytes(const AttnArgs &a, int sms);

}  // namespace convrot
