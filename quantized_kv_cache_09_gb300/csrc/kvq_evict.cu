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
// One CTA per sequence, for long rows a cluster of four, an entry's key
// (order-preserving integer of its weight), weight and page in registers, so
// every output may be its input.  The smallest kept key is found a byte at a
// time from the top: four histograms of the keys that share the bytes found so
// far, each in eight copies by lane (weights of one sequence share their
// exponents, and atomics on one address run one after the other), summed over
// the cluster through distributed shared memory.  Ordered counts over warp
// ballots then give every entry its place.  Bound by latency: the longest row is
// 512 KB of traffic.
#include <cooperative_groups.h>

#include "kvq_around.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kEvictCluster = 4;  // CTAs of a long row
constexpr int kEvictCopies = 8;   // of a histogram

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

// CTA r of a row's CTAS has entries [r, r + 1) * THREADS * N, striped: item k of thread
// t is entry k * THREADS + t of them, so ballots of item k, warp by warp, list the entries in order.
template <int THREADS, int CTAS, int N>
__global__ void __launch_bounds__(THREADS, 1) evict_pages_kernel(EvictParams p)
{
    namespace cg = cooperative_groups;
    constexpr int W = THREADS / 32;
    __shared__ uint32_t hist[2][256 * kEvictCopies];  // a round's histogram in copies (two buffers in turn)
    __shared__ uint32_t bins[2][256];                 // the CTA's sums of the copies
    __shared__ __align__(16) uint32_t row_bins[2][256];  // the row's
    __shared__ int32_t before[N][W];          // entries counted before (item, warp) in its item
    __shared__ int32_t total[N];              // entries counted in an item
    __shared__ int32_t cta_total[2][CTAS];    // entries counted by a CTA (for the ties, for the kept)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / CTAS, rank_cta = blockIdx.x % CTAS, mb = p.max_blocks;
    const int32_t *tin = p.table + (int64_t)b * mb;
    const float *win = p.weights + (int64_t)b * mb;
    int32_t *tout = p.table_out + (int64_t)b * mb;
    float *wout = p.weights_out + (int64_t)b * mb;
    const int e0 = rank_cta * THREADS * N + tid;  // item k is entry e0 + k * THREADS
    if constexpr (CTAS > 1) cg::this_cluster().barrier_arrive();

    // all loads at once: none waits for the length
    const int L = p.seq_lens[b], want = p.keep[b];
    int32_t page[N];
    float w[N];
#pragma unroll
    for (int k = 0; k < N; k++) {
        const int j = e0 + k * THREADS;
        page[k] = j < mb ? tin[j] : 0;
        w[k] = j < mb ? win[j] : 0.0f;
    }
    const bool bad = L < 0 || L > (int64_t)mb * kPage;
    if (bad && tid == 0) set_flag(p.status, KVQ_FLAG_BAD_LENGTH);
    const int nb = bad ? mb : (L + kPage - 1) / kPage;  // (bad: the row is copied as it is)
    const int budget = bad ? nb : max(0, min(want, nb));
    const int lo = min(p.sink, nb), hi = max(lo, nb - max(p.recent, 1));  // candidates [lo, hi)
    const int guarded = nb - (hi - lo);
    const int room = min(hi - lo, max(0, budget - guarded));
    const bool some = room > 0 && room < hi - lo;  // (the same for the whole row)
    uint32_t key[N];                               // 0: no candidate
#pragma unroll
    for (int k = 0; k < N; k++) {
        const int j = e0 + k * THREADS;
        key[k] = j >= lo && j < hi ? weight_key(w[k]) : 0u;
    }
    __syncwarp();
    if constexpr (CTAS > 1) cg::this_cluster().barrier_wait();  // every CTA runs: its shared memory may be written

    // T = the room-th largest candidate key, `ties` of those equal to it stay
    uint32_t T = 0;
    int ties = room;
    if (some) {
        for (int i = tid; i < 2 * 256 * kEvictCopies; i += THREADS) (&hist[0][0])[i] = 0u;
        __syncthreads();
#pragma unroll 1
        for (int r = 0; r < 4; r++) {
            const int sh = 24 - 8 * r, buf = r & 1;
#pragma unroll
            for (int k = 0; k < N; k++)
                if (key[k] && (r == 0 || key[k] >> (sh + 8) == T >> (sh + 8)))
                    atomicAdd(&hist[buf][(key[k] >> sh & 255u) * kEvictCopies + lane % kEvictCopies], 1u);
            __syncthreads();
            for (int i = tid; i < 256; i += THREADS) {
                uint32_t c = 0;
#pragma unroll
                for (int x = 0; x < kEvictCopies; x++) {
                    c += hist[buf][i * kEvictCopies + x];
                    hist[buf][i * kEvictCopies + x] = 0u;  // (written again two rounds on)
                }
                if constexpr (CTAS > 1)
                    bins[buf][i] = c;
                else
                    row_bins[buf][i] = c;
            }
            if constexpr (CTAS > 1) {
                cg::cluster_group cluster = cg::this_cluster();
                __syncwarp();
                cluster.sync();
                for (int i = tid; i < 256; i += THREADS) {
                    uint32_t c = 0;
#pragma unroll
                    for (int x = 0; x < CTAS; x++) c += *cluster.map_shared_rank(&bins[buf][i], x);
                    row_bins[buf][i] = c;
                }
            }
            __syncthreads();
            // every warp: lane l holds bins 255 - 8 l .. 248 - 8 l; the bin where the count from the
            // top reaches `ties`
            const uint4 *v = reinterpret_cast<const uint4 *>(&row_bins[buf][248 - 8 * lane]);
            const uint4 v0 = v[0], v1 = v[1];
            const uint32_t c[8] = {v1.w, v1.z, v1.y, v1.x, v0.w, v0.z, v0.y, v0.x};
            int sum = 0;
#pragma unroll
            for (int x = 0; x < 8; x++) sum += (int)c[x];
            int run = inclusive_scan(sum, lane);
            const int at = __ffs(__ballot_sync(kFull, run >= ties)) - 1;
            run -= sum;
            int digit = -1, left = 0;
#pragma unroll
            for (int x = 0; x < 8; x++) {
                if (digit < 0 && run + (int)c[x] >= ties) {
                    digit = 255 - 8 * lane - x;
                    left = ties - run;
                }
                run += (int)c[x];
            }
            T |= (uint32_t)__shfl_sync(kFull, digit, at) << sh;
            ties = __shfl_sync(kFull, left, at);
        }
    }
    // ordered counts of a predicate over the row: ballots by (item, warp), scans, the CTAs' totals
    int base = 0, item0 = 0;  // entries counted in lower CTAs; lane k: before item k
    auto count = [&](auto pred, int which) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; k++) {
            const uint32_t m = __ballot_sync(kFull, pred(k));
            if (lane == 0) before[k][warp] = __popc(m);
        }
        __syncthreads();
        for (int k = warp; k < N; k += W) {  // a warp scans an item's counts, ...
            const int x = lane < W ? before[k][lane] : 0;
            const int s = inclusive_scan(x, lane);
            if (lane < W) before[k][lane] = s - x;
            if (lane == 31) total[k] = s;
        }
        __syncthreads();
        const int x = lane < N ? total[lane] : 0;  // ... every warp the items' totals
        const int s = inclusive_scan(x, lane);
        item0 = s - x;
        base = 0;
        if constexpr (CTAS > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            const int mine = __shfl_sync(kFull, s, N - 1);  // (by every lane: lane N - 1 holds the CTA's sum)
            if (warp == 0 && lane < CTAS) *cluster.map_shared_rank(&cta_total[which][rank_cta], lane) = mine;
            __syncwarp();
            cluster.sync();
            base = __reduce_add_sync(kFull, lane < rank_cta ? cta_total[which][lane] : 0);
        }
    };
    // entries counted before item k of this thread (x: its own predicate)
    auto rank = [&](int k, bool x) {
        return base + before[k][warp] + __shfl_sync(kFull, item0, k) +
               __popc(__ballot_sync(kFull, x) & ((1u << lane) - 1u));
    };
    const bool all = room >= hi - lo;
    uint32_t kept = 0;              // bit k: item k stays
    if (some) count([&](int k) { return key[k] == T; }, 0);
#pragma unroll
    for (int k = 0; k < N; k++) {
        const int j = e0 + k * THREADS;
        bool stays = j < lo || j >= hi || all;
        if (some) {
            const int r = rank(k, key[k] == T);
            stays = stays || key[k] > T || (key[k] == T && r < ties);
        }
        kept |= (uint32_t)(stays && j < nb) << k;
    }
    // (every CTA of the row has read its entries by the barriers in here: the outputs may be the inputs)
    count([&](int k) { return (kept >> k & 1u) != 0; }, 1);
    const int stay = guarded + room, gone = nb - stay;
#pragma unroll
    for (int k = 0; k < N; k++) {
        const int j = e0 + k * THREADS;
        const bool stays = (kept >> k & 1u) != 0;
        const int r = rank(k, stays);
        if (j >= mb) continue;
        if (stays) {
            tout[r] = page[k];
            wout[r] = w[k];
        } else {  // evicted: behind everything, in order; past the length: moves up
            tout[j < nb ? mb - gone + (j - r) : j - gone] = page[k];
        }
        if (j >= stay) wout[j] = 0.0f;
    }
    if (tid == 0 && rank_cta == 0) {
        p.seq_lens_out[b] = L - kPage * gone;
        p.num_evicted[b] = gone;
    }
    if constexpr (CTAS > 1) {
        __syncwarp();
        cg::this_cluster().sync();  // no CTA ends while another may write to it
    }
}

template <int THREADS, int CTAS, int N>
static cudaError_t launch_evict_rows(const EvictParams &p, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.num_seqs * CTAS);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CTAS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, evict_pages_kernel<THREADS, CTAS, N>, p);
}

// Few threads, many entries each: barriers cost more than instructions here.  A row of 16400
// entries (16 rows, event time with a launch): one CTA of 1024 threads 28 us, clusters of eight
// CTAs of 1024 / 256 threads 34 / 22 us, of four of 512 threads 20 us; rows of up to 512 entries
// 10 us with 128 threads.
cudaError_t launch_evict(const EvictParams &p, cudaStream_t s)
{
    static_assert(kMaxEvictBlocks == 512 * 16 * kEvictCluster, "the longest row fits the largest instance");
    if (p.max_blocks <= 128 * 4) return launch_evict_rows<128, 1, 4>(p, s);
    if (p.max_blocks <= 512 * 8) return launch_evict_rows<512, 1, 8>(p, s);
    if (p.max_blocks <= 512 * 9 * kEvictCluster) return launch_evict_rows<512, kEvictCluster, 9>(p, s);
    return launch_evict_rows<512, kEvictCluster, 16>(p, s);
}

}  // namespace kvq
