// kvq_weights.cuh -- what the two kernels of page weights share.
#pragma once

#include "kvq_around.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

// the byte formats' exact widening to fp16 pairs
template <int FMT>
__device__ __forceinline__ void widen_bytes(uint32_t w, __half2 c[2])
{
    if constexpr (FMT == KVQ_FP8_E4M3)
        widen_e4m3(w, c);
    else
        widen_int8(w, c);
}

// the largest of three binary32 values (one instruction)
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// what a sequence brings: its chunk's first row, rows, length; false (and flagged) when a bound is broken
struct PwSeq {
    int c0, n, L;
};
__device__ __forceinline__ bool pw_seq(const PageWeightsParams &p, int b, PwSeq &s)
{
    s.c0 = p.cu_q[b];
    s.n = p.cu_q[b + 1] - s.c0;
    s.L = p.seq_lens[b];
    return s.n >= 0 && s.n <= p.max_q && s.n <= s.L && s.L <= (int64_t)p.max_blocks * kPage && s.c0 >= 0 &&
           (int64_t)s.c0 + s.n <= p.total_q;
}

// The workspace of a sequence's log2-sums: [page][query row], its rows by cache head, then by token
// and head of the group, so that the rows of a tile lie side by side.
__device__ __forceinline__ float *pw_sums(const PageWeightsParams &p, const PwSeq &s)
{
    return p.lse + (int64_t)s.c0 * p.num_q_heads * p.max_blocks;
}

// the least factor of a raw score: a key scale or softmax scale of 0 scores 1e-38 * raw instead of
// 0 (no difference in binary32 once the maximum is subtracted), and a masked score stays -inf
constexpr float kPwMinScale = 1.17549435e-38f;

}  // namespace kvq
