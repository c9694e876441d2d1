// qz_serving.cuh -- launchers of what a batch of requests needs beside the packed
// weights: adapters and the 4-bit key/value cache.  Internal; not installed.
// (defined in the .cu files; arguments already validated)
#pragma once

#include "qz_internal.cuh"

namespace qz {

// Low-rank adapters beside a packed projection: launch_lora (qz_lora.cu) makes
// the first product h in `scratch` (lora_scratch_bytes), launch_gemv_lora
// (qz_gemv.cu) is the integer GEMV that adds the second one to its sums.
constexpr int64_t kLoraMaxRank = 128;
struct LoraUp {
    const uint16_t *up;        // adapters x N x rank
    const uint16_t *h;         // [2][M][rank]: bf16 hi, lo
    const int32_t *ids;        // adapter of each token
    int rank, adapters;
};
size_t lora_scratch_bytes(int64_t M);
qz_status launch_lora(const void *a, const void *lora_a, const void *lora_b, const void *adapters,
                      const void *lora_scales, int64_t n_adapters, int64_t rank, int64_t M,
                      int64_t K, void *scratch, LoraUp *up, cudaStream_t stream);
qz_status launch_gemv_lora(int bits, const void *a, const void *codes, const void *scales,
                           const void *zeros, int64_t M, int64_t N, int64_t K, int64_t group_size,
                           const LoraUp &up, void *y, void *workspace, uint32_t *counters,
                           const GemvPlan &plan, cudaStream_t stream);

// The paged 4-bit key/value cache (qz_kv4.cu).
struct Kv4Cache {
    void *cache;
    const void *page_table, *kv_lens, *cu;     // int32 [B][max_pages], [B], [B + 1]
    int64_t T, B, kv_heads, head_dim, group_size, page_size, num_pages, max_pages;
};
size_t kv4_record_bytes(int64_t head_dim, int64_t group_size);
size_t kv4_attention_workspace_bytes(int64_t head_dim);
qz_status launch_kv4_append(const Kv4Cache &c, const void *k, const void *v, int64_t k_stride,
                            int64_t v_stride, cudaStream_t stream);
qz_status launch_kv4_read(const Kv4Cache &c, void *k, void *v, cudaStream_t stream);
qz_status launch_kv4_attention(const Kv4Cache &c, const void *q, int64_t q_stride, int64_t q_heads,
                               float scale, int64_t window, void *out, int64_t out_stride,
                               void *workspace, cudaStream_t stream);

}  // namespace qz
