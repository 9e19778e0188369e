// kvq_around.h -- launch parameters and launchers of the operators around the cache: prompt
// attention, page weights and page eviction.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "kvq.h"

namespace kvq {

// let `kernel` take `bytes` of dynamic shared memory on the current device; `done`, one per kernel,
// remembers the devices (64 of them) that know it
template <typename K>
cudaError_t allow_smem(K *kernel, size_t bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// query heads per cache head that share a 128-row tile of prompt attention
constexpr int kMaxPromptGroup = 128;

struct PromptParams {
    const int32_t *cu;  // [num_seqs + 1]: sequence b's rows are cu[b] .. cu[b+1]-1
    uint16_t *out;      // [total][num_q_heads][128]
    float *lse;         // [total][num_q_heads] or null
    const uint16_t *v;  // rows of v (read again only where a value is not finite)
    int64_t v_stride;   // elements from one row of v to the next
    int32_t *status;
    int num_seqs, num_heads, num_q_heads, group, max_n;
    int64_t total;
    float score_scale;  // softmax_scale * log2(e)
    // a unit's two tiles of up to 128 rows = tile_tokens x tile_heads, tile 1 tile1_token tokens
    // and tile1_head heads after tile 0 (one of them 0)
    int tile_heads, tile_tokens, tile1_head, tile1_token, unit_tokens;
};

struct PageWeightsParams {
    const uint8_t *k_codes;
    const float *k_scales;
    const uint16_t *q;           // [total_q][num_q_heads][128]
    const int32_t *cu_q;         // [num_seqs + 1]
    const int32_t *seq_lens;     // [num_seqs]: lengths including the chunk
    const int32_t *block_table;  // [num_seqs][max_blocks]
    const float *weights_in;     // [num_seqs][max_blocks] or null (zero)
    float *weights_out;          // [num_seqs][max_blocks]
    int32_t *status;
    int num_seqs, num_heads, num_q_heads, group, num_pages, max_blocks, max_q;
    int64_t total_q;
    float score_scale;  // softmax_scale * log2(e)
    float decay;
    float *lse;   // total_q * num_q_heads * max_blocks log2-sums of a page's 2^score per query row
    float *part;  // [total_q * ceil(num_q_heads / 64)][max_blocks]: page masses of a chunk of rows
};

// query rows (tokens x heads) of a sequence that one CTA of page_sum_kernel sums
constexpr int kPwSumRows = 64;

struct EvictParams {
    const int32_t *table;     // [num_seqs][max_blocks]
    const int32_t *seq_lens;  // [num_seqs]
    const float *weights;     // [num_seqs][max_blocks]
    const int32_t *keep;      // [num_seqs]: pages to keep
    int32_t *table_out;
    int32_t *seq_lens_out;
    float *weights_out;
    int32_t *num_evicted;
    int32_t *status;
    int num_seqs, max_blocks, sink, recent;
};

// the longest block-table row an eviction takes (2 million tokens, four SMs)
constexpr int kMaxEvictBlocks = 32768;

cudaError_t launch_prompt(int dtype, const PromptParams &p, const uint16_t *q, int64_t q_stride, const uint16_t *k,
                          int64_t k_stride, int num_sms, cudaStream_t s);
size_t page_weights_lse_floats(int64_t total_q, int num_q_heads, int max_blocks);
size_t page_weights_workspace_bytes(int64_t total_q, int num_q_heads, int max_blocks);
cudaError_t launch_page_window(int fmt, const PageWeightsParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_page_weights(int fmt, const PageWeightsParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_evict(const EvictParams &p, cudaStream_t s);

}  // namespace kvq
