// kvq_evict.cu -- pages of least accumulated attention weight leave the block
// tables (eviction from a paged cache; paging through a block table: ddd.cn
// section 4).  A page is the unit of both the block table and the quantizer's
// scale, so whole pages go: nothing is re-quantized and no code is touched.
//
// Per sequence of nb pages: the first `sink` and the last max(recent, 1) pages
// stay; of the others the `room` = max(0, min(keep, nb) - protected) with the
// largest weights stay, ties to the lower index.  The row of the block table is
// rewritten as [kept, in order][entries past the length][evicted, in order],
// a permutation of itself.
//
// One CTA per sequence, the row held on the SM (order-preserving integer keys
// of the weights in registers, table and weights in shared memory), so every
// output may be its input.  The smallest kept key is found by bits from the top, two at a
// time: each round counts the keys at or above three thresholds, 16 rounds of
// one barrier each whatever the weights are (a histogram by bytes would
// serialise its atomics: weights of one sequence share their exponent bytes).
// Two ordered scans over warp ballots then give every entry its place.  The
// call is bound by latency: one 16384-page row is 192 KB of traffic.
#include "kvq_around.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;

// float -> uint32 whose unsigned order is the weight's order; NaN below
// everything (as -inf), -0.0 equal to 0.0.  0 is free for "not a candidate".
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int inclusive_scan(int x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += v;
    }
    return x;
}

}  // namespace

// Items are striped (item k of thread t is entry k * 1024 + t), so ballots of
// item k, warp by warp, list the entries in order.
template <int ITEMS>
__global__ void __launch_bounds__(kEvictThreads, 1) evict_pages_kernel(EvictParams p)
{
    extern __shared__ int32_t row[];                 // the table row, max_blocks entries, ...
    float *w = reinterpret_cast<float *>(row + p.max_blocks);  // ... and the weights
    __shared__ int32_t cnt[2][3][kEvictWarps];       // a round's counts by warp (double-buffered)
    __shared__ int32_t before[ITEMS * kEvictWarps];  // entries counted before (item, warp) in its item
    __shared__ int32_t total[32];                    // entries counted in an item
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x, mb = p.max_blocks;
    const int32_t *tin = p.table + (int64_t)b * mb;
    const float *win = p.weights + (int64_t)b * mb;
    int32_t *tout = p.table_out + (int64_t)b * mb;
    float *wout = p.weights_out + (int64_t)b * mb;
    const int L = p.seq_lens[b];
    const int64_t cap = (int64_t)mb * kPage;
    const bool bad = L < 0 || L > cap;
    if (bad && tid == 0) set_flag(p.status, KVQ_FLAG_BAD_LENGTH);
    const int nb = bad ? mb : (L + kPage - 1) / kPage;  // (bad: the row is copied as it is)
    const int budget = bad ? nb : max(0, min(p.keep[b], nb));
    const int lo = min(p.sink, nb), hi = max(lo, nb - max(p.recent, 1));  // candidates [lo, hi)
    const int guarded = nb - (hi - lo);
    const int room = min(hi - lo, max(0, budget - guarded));

    uint32_t key[ITEMS];  // 0: no candidate
#pragma unroll
    for (int k = 0; k < ITEMS; k++) {
        const int j = k * kEvictThreads + tid;
        key[k] = 0;
        if (j < mb) {
            row[j] = tin[j];  // (read again by this thread only)
            const float x = j < nb ? win[j] : 0.0f;
            w[j] = x;
            if (j >= lo && j < hi) key[k] = weight_key(x);
        }
    }
    // T = the room-th largest candidate key: the largest T with #(key >= T) >= room
    uint32_t T = 0;
    int above = 0;  // #(key > T) once T is final
    if (room > 0 && room < hi - lo) {
        for (int sh = 30, r = 0; sh >= 0; sh -= 2, r ^= 1) {
            int c1 = 0, c2 = 0, c3 = 0;
            const uint32_t t1 = T + (1u << sh), t2 = T + (2u << sh), t3 = T + (3u << sh);
#pragma unroll
            for (int k = 0; k < ITEMS; k++) {
                c1 += key[k] >= t1;
                c2 += key[k] >= t2;
                c3 += key[k] >= t3;
            }
            c1 = __reduce_add_sync(kFull, c1);
            c2 = __reduce_add_sync(kFull, c2);
            c3 = __reduce_add_sync(kFull, c3);
            if (lane == 0) {
                cnt[r][0][warp] = c1;
                cnt[r][1][warp] = c2;
                cnt[r][2][warp] = c3;
            }
            __syncthreads();
            c1 = __reduce_add_sync(kFull, cnt[r][0][lane]);
            c2 = __reduce_add_sync(kFull, cnt[r][1][lane]);
            c3 = __reduce_add_sync(kFull, cnt[r][2][lane]);
            T = c3 >= room ? t3 : c2 >= room ? t2 : c1 >= room ? t1 : T;
        }
        int c = 0;
#pragma unroll
        for (int k = 0; k < ITEMS; k++) c += key[k] > T;
        c = __reduce_add_sync(kFull, c);
        if (lane == 0) cnt[0][0][warp] = c;
        __syncthreads();
        above = __reduce_add_sync(kFull, cnt[0][0][lane]);
    }
    // ordered counts of a predicate over the row: ballots by (item, warp), then one scan
    int item0 = 0;  // lane k: entries counted before item k
    auto count = [&](auto pred) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < ITEMS; k++) {
            const uint32_t m = __ballot_sync(kFull, pred(k));
            if (lane == 0) before[k * kEvictWarps + warp] = __popc(m);
        }
        __syncthreads();
        if (warp < ITEMS) {  // warp k scans item k's counts, ...
            const int c = before[warp * kEvictWarps + lane];
            const int s = inclusive_scan(c, lane);
            before[warp * kEvictWarps + lane] = s - c;
            if (lane == 31) total[warp] = s;
        }
        __syncthreads();
        // ... and every warp the items' totals
        const int tot = lane < ITEMS ? total[lane] : 0;
        item0 = inclusive_scan(tot, lane) - tot;
    };
    // entries counted before item k of this thread (x: its own predicate)
    auto rank = [&](int k, bool x) {
        return before[k * kEvictWarps + warp] + __shfl_sync(kFull, item0, k) +
               __popc(__ballot_sync(kFull, x) & ((1u << lane) - 1u));
    };
    const bool all = room >= hi - lo;
    const int ties = room - above;  // keys equal to T that stay: the first of them
    uint32_t kept = 0;  // bit k: item k stays
    if (room > 0 && !all) count([&](int k) { return key[k] == T; });
#pragma unroll
    for (int k = 0; k < ITEMS; k++) {
        const int j = k * kEvictThreads + tid;
        bool stays = j < lo || j >= hi || all;
        if (room > 0 && !all) {  // (the same for the whole CTA)
            const int r = rank(k, key[k] == T);
            stays = stays || key[k] > T || (key[k] == T && r < ties);
        }
        kept |= (uint32_t)(stays && j < nb) << k;
    }
    count([&](int k) { return (kept >> k & 1u) != 0; });
    const int stay = guarded + room, gone = nb - stay;
#pragma unroll
    for (int k = 0; k < ITEMS; k++) {
        const int j = k * kEvictThreads + tid;
        const bool stays = (kept >> k & 1u) != 0;
        const int r = rank(k, stays);
        if (j >= mb) continue;
        if (stays) {
            tout[r] = row[j];
            wout[r] = w[j];
        } else {  // evicted: behind everything, in order; past the length: moves up
            tout[j < nb ? mb - gone + (j - r) : j - gone] = row[j];
        }
        if (j >= stay) wout[j] = 0.0f;
    }
    if (tid == 0) {
        p.seq_lens_out[b] = L - kPage * gone;
        p.num_evicted[b] = gone;
    }
}

template <int ITEMS>
static cudaError_t launch_evict_items(const EvictParams &p, cudaStream_t s)
{
    const size_t smem = (size_t)p.max_blocks * (sizeof(int32_t) + sizeof(float));
    cudaError_t e = cudaFuncSetAttribute(evict_pages_kernel<ITEMS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(ITEMS * kEvictThreads * (sizeof(int32_t) + sizeof(float))));
    if (e != cudaSuccess) return e;
    return launch_plain(evict_pages_kernel<ITEMS>, dim3((unsigned)p.num_seqs), dim3(kEvictThreads), smem, s, p);
}

cudaError_t launch_evict(const EvictParams &p, cudaStream_t s)
{
    static_assert(kMaxEvictBlocks == 24 * kEvictThreads, "the longest row fits the largest instance");
    if (p.max_blocks <= kEvictThreads) return launch_evict_items<1>(p, s);
    if (p.max_blocks <= 4 * kEvictThreads) return launch_evict_items<4>(p, s);
    if (p.max_blocks <= 16 * kEvictThreads) return launch_evict_items<16>(p, s);
    return launch_evict_items<24>(p, s);
}

}  // namespace kvq
