// kvq_window.cu -- page weights for windows of query rows: more than 16 rows of one cache head
// (the last tokens of a prompt, chunks).  The same numbers as page_lse_kernel of kvq_weights.cu
// -- S(row, page) = log2 sum_{t in page} 2^(score) -- on the 5th-generation tensor cores: 128
// query rows share one widening of a page's codes, and the widening, the MMAs and the softmax
// sums each run in their own warps.
//
// A persistent CTA per SM takes an equal contiguous share of all steps; a step is two pages (128
// keys) of one (sequence, cache head, tile of 128 query rows).  Roles:
//   warps 0, 1   one thread each issues the MMAs of the even and of the odd steps: S = Q K^T, M = N
//                = 128, Q (two tiles) and two S in tensor memory.  (A thread that has committed
//                its MMAs gets nothing back from shared memory for some 500 cycles, even a
//                barrier long complete: one thread for all steps took 1500 cycles a step.)
//   warps 2, 3   look pages up and issue the bulk copies of the even and of the odd steps, up to
//                four steps ahead (a copy of 8 KB holds its issuer ~450 cycles: one warp took
//                1450 cycles a step)
//   warps 4-7    the next tile's query rows into tensor memory, a row per thread
//   warps 8-11   widening: codes of a step from the copy ring to fp16 in shared memory (128-byte
//                swizzled, K-major).  int4 pairs come out as elements (0,4) (1,5) (2,6) (3,7) of a
//                word, and q is permuted alike
//   warps 12-19  softmax sums, warps 12-15 the even steps, 16-19 the odd ones: one thread per query
//                row reads its 64 scores of each page from tensor memory
// Every hand-off is an mbarrier, every wait bounded.
//
// Measured: the last 32 tokens of 16 prompts of 512 .. 16384 tokens, int8, 32 / 8 heads (20 GFLOP,
// 84 MB): 30 us (mma.sync with 16 rows a unit, which widens each page eight times: 116 us).  A step
// takes ~1350 cycles, of which the tensor pipe and the exponentials need ~512 each; without any
// softmax, widening and all but one MMA of a step it still takes ~900, the hand-offs from role to
// role.  (Letting S go page by page: 6% slower.)  Rows: 17 fill a tile of 128 as 128 do;
// up to 16 rows page_lse_kernel reads the codes at the rate of HBM.
#include "kvq_tc.cuh"
#include "kvq_weights.cuh"

namespace kvq {

namespace {

constexpr int kWinThreads = 20 * 32;
constexpr int kWinRows = 128;
constexpr int kWinKeys = 2 * kPage;
// Even numbers of stages: the even and the odd steps have their own copy warp, MMA thread and
// softmax warps, which run ahead of one another, so each keeps to its own stages (a wait by parity
// of a stage that both used would take the use before last for the last).  Two widened tiles: with
// four, the widening runs ahead and takes the sums' issue slots (33 us against 29).
constexpr int kCodeStages = 4, kKeyStages = 2, kScoreStages = 2, kMeta = 16;
static_assert(kCodeStages % 2 == 0 && kKeyStages % 2 == 0 && kScoreStages % 2 == 0, "stages by parity of the step");
// a step's record lives until its sums are done: the copies run at most the sum of the stages ahead
static_assert(kMeta >= kCodeStages + kKeyStages + kScoreStages + 2, "records outlive their steps");
constexpr int kWinTile = kWinKeys * kHeadDim * 2;
constexpr uint32_t kWinTmem = 512;    // S at columns 128 * stage, Q at 256 + 64 * buffer
constexpr uint32_t kWinIdesc = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);  // f32 += f16 x f16, M = N = 128

// what a step is: its sequence, cache head, first query row and page, key scales of its pages
struct WinStep {
    int32_t c0, n, L, h, row0, j, pages;
    int32_t tile, first, left;  // number of its tile in this CTA, whether it begins it, steps of it that follow
    float sk[2];
};

struct alignas(1024) WinSmem {
    uint8_t k[kKeyStages][kWinTile];
    uint8_t code[kCodeStages][2 * kPage * kHeadDim];
    uint64_t code_full[kCodeStages], code_free[kCodeStages];
    uint64_t k_full[kKeyStages], k_free[kKeyStages];
    uint64_t s_full[kScoreStages], s_free[kScoreStages];
    uint64_t q_full[2], q_free[2], mma_done;
    WinStep meta[kMeta];
    int64_t upto[kMaxSeqsPerLaunch + 1];
    uint32_t tmem;
};
static_assert(sizeof(WinSmem) <= 227 * 1024, "one CTA's shared memory");

// counter i of a ring of N stages: its stage and the parity of its use
template <int N>
struct Turn {
    uint32_t stage = 0, parity = 0;
    __device__ __forceinline__ void next()
    {
        if (++stage == N) {
            stage = 0;
            parity ^= 1u;
        }
    }
};

// byte offset of elements 8c .. 8c + 7 of row r in a K-major tile of 128 rows, 128-byte swizzled
__device__ __forceinline__ uint32_t tile_chunk(int r, int c)
{
    return (uint32_t)((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint32_t lop_and_xor(uint32_t x, uint32_t m, uint32_t c)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(x), "r"(m), "r"(c));  // (x & m) ^ c
    return d;
}

// 8 int4 codes (a word) as fp16, pairs (0,4) (1,5) (2,6) (3,7): a nibble with its top bit flipped
// is c + 8; as the low bits of 1024 it reads 1032 + c, four bits up 1024 + 16 (c + 8)
__device__ __forceinline__ uint4 widen8_pairs(uint32_t w)
{
    const __half2 k1032 = __float2half2_rn(1032.0f), k16 = __float2half2_rn(0.0625f), k72 = __float2half2_rn(-72.0f);
    const uint32_t x[4] = {lop_and_xor(w, 0x000f000fu, 0x64086408u), lop_and_xor(w, 0x00f000f0u, 0x64806480u),
                           lop_and_xor(w >> 8, 0x000f000fu, 0x64086408u),
                           lop_and_xor(w >> 8, 0x00f000f0u, 0x64806480u)};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __half2 h = *reinterpret_cast<const __half2 *>(&x[i]);
        r[i] = h2_bits(i & 1 ? __hfma2(h, k16, k72) : __hsub2(h, k1032));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// the order widen8_pairs gives, for 8 elements of a query row
__device__ __forceinline__ uint4 as_pairs(uint4 v)
{
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                      __byte_perm(v.y, v.w, 0x7632));
}

}  // namespace

template <int FMT>
__global__ void __launch_bounds__(kWinThreads, 1) page_window_kernel(PageWeightsParams p)
{
    constexpr int RB = FMT == KVQ_INT4_B64 ? 64 : 128;
    constexpr uint32_t kPageBytes = kPage * RB;
    extern __shared__ __align__(1024) uint8_t smem_win[];
    WinSmem &sm = *reinterpret_cast<WinSmem *>(smem_win);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = p.num_heads, G = p.group;
    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < kCodeStages; i++) {
            mbar_init(&sm.code_full[i], 1);
            mbar_init(&sm.code_free[i], 4);
        }
        for (int i = 0; i < kKeyStages; i++) {
            mbar_init(&sm.k_full[i], 4);
            mbar_init(&sm.k_free[i], 1);
        }
        for (int i = 0; i < kScoreStages; i++) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_free[i], 4);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&sm.q_full[i], 4);
            mbar_init(&sm.q_free[i], 2);
        }
        mbar_init(&sm.mma_done, 2);
        mbar_init_fence();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)),
                     "r"(kWinTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // steps of sequence b: (cache head, tile of query rows, page pair), the pages fastest
    auto steps_of = [&](const PwSeq &s) { return (s.L + kWinKeys - 1) / kWinKeys; };
    auto tiles_of = [&](const PwSeq &s) { return (s.n * G + kWinRows - 1) / kWinRows; };
    bool bad_seq = false;
    if (warp == 2) {
        int64_t run = 0;
        for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
            int64_t u = 0;
            if (b0 + lane < p.num_seqs) {
                PwSeq s;
                if (pw_seq(p, b0 + lane, s))
                    u = (int64_t)steps_of(s) * H * tiles_of(s);
                else
                    bad_seq = true;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(kFull, u, o);
                if (lane >= o) u += v;
            }
            if (b0 + lane < p.num_seqs) sm.upto[b0 + lane + 1] = run + u;
            run += __shfl_sync(kFull, u, 31);
        }
        if (lane == 0) sm.upto[0] = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();  // (the lengths are read before it, everything else after)
    if (bad_seq && blockIdx.x == 0) set_flag(p.status, KVQ_FLAG_BAD_LENGTH);
    const uint32_t tmem = sm.tmem;
    // step u of the launch: its sequence; of it the step's record, but for the scales and flags; and
    // its number among the tile's `all` steps
    auto place = [&](int64_t u, WinStep &m, int &k, int &all) {
        int lo = 0, hi = p.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm.upto[mid] <= u)
                lo = mid;
            else
                hi = mid;
        }
        PwSeq s;
        pw_seq(p, lo, s);
        all = steps_of(s);
        const int tiles = tiles_of(s);
        const uint32_t r = (uint32_t)(u - sm.upto[lo]), hr = r / (uint32_t)all;  // (under 2^31 of one sequence)
        k = (int)(r - hr * (uint32_t)all);
        m.c0 = s.c0;
        m.n = s.n;
        m.L = s.L;
        m.h = (int)(hr / (uint32_t)tiles);
        m.row0 = (int)(hr % (uint32_t)tiles) * kWinRows;
        m.j = 2 * k;
        m.pages = min(2, (s.L + kPage - 1) / kPage - m.j);
        return lo;
    };
    const int64_t U = sm.upto[p.num_seqs];
    const int64_t first = U * blockIdx.x / gridDim.x;
    const int steps = (int)(U * (blockIdx.x + 1) / gridDim.x - first);
    bool ok = true;

    if (warp >= 8 && warp < 12) {
        // ---- widening ----
        const int wt = tid - 8 * 32;
        Turn<kCodeStages> code;
        Turn<kKeyStages> key;
        for (int i = 0; i < steps; i++, code.next(), key.next()) {
            ok = mbar_wait_short(&sm.code_full[code.stage], code.parity);
            constexpr int kLd = 2 * kPageBytes / (16 * 128);  // 16-byte pieces per thread
            // int4: 8 threads take 4 keys x 2 pieces (16 bytes of a row), else 2 keys x 4 pieces: the
            // stores meet no bank conflict
            auto key_of = [&](int r) {
                return RB == 64 ? (r >> 1) * kPage + 4 * (wt >> 3) + ((wt & 7) >> 1)
                                : 32 * (r >> 1) + 2 * (wt >> 3) + ((wt & 7) >> 2);
            };
            auto piece_of = [&](int r) { return RB == 64 ? (wt & 1) + 2 * (r & 1) : (wt & 3) + 4 * (r & 1); };
            uint4 w[kLd];
#pragma unroll
            for (int r = 0; r < kLd; r++) w[r] = *reinterpret_cast<const uint4 *>(sm.code[code.stage] + key_of(r) * RB + 16 * piece_of(r));
            if (ok && i >= kKeyStages) ok = mbar_wait_short(&sm.k_free[key.stage], key.parity ^ 1u);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            uint8_t *dst = sm.k[key.stage];
#pragma unroll
            for (int r = 0; r < kLd; r++) {
                const int kk = key_of(r), pc = piece_of(r);
                const uint32_t x[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
                if constexpr (FMT == KVQ_INT4_B64) {
#pragma unroll
                    for (int y = 0; y < 4; y++)
                        *reinterpret_cast<uint4 *>(dst + tile_chunk(kk, 4 * pc + y)) = widen8_pairs(x[y]);
                } else {
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        __half2 a[2], b[2];
                        widen_bytes<FMT>(x[2 * y], a);
                        widen_bytes<FMT>(x[2 * y + 1], b);
                        *reinterpret_cast<uint4 *>(dst + tile_chunk(kk, 2 * pc + y)) =
                            make_uint4(h2_bits(a[0]), h2_bits(a[1]), h2_bits(b[0]), h2_bits(b[1]));
                    }
                }
            }
            fence_proxy_async_smem();  // the MMAs read through the async proxy, the next copy writes through it
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.k_full[key.stage]);
                mbar_arrive(&sm.code_free[code.stage]);
            }
        }
    } else if (warp >= 12) {
        // ---- softmax sums: one query row per thread ----
        const int row = (warp & 3) * 32 + lane;
        const float sabs = fmaxf(fabsf(p.score_scale), kPwMinScale);
        Turn<kScoreStages> score;
        for (int i = 0; i < steps; i++, score.next()) {
            if ((i & 1) != (warp - 12) >> 2) continue;
            const uint32_t ss = score.stage;
            ok = __all_sync(kFull, mbar_wait_short(&sm.s_full[ss], score.parity));
            if (!ok) break;
            tc_fence_after();
            const WinStep m = sm.meta[i % kMeta];
            const uint32_t tm = tmem + 128u * ss + ((uint32_t)((warp & 3) * 32) << 16);
            const int rr = m.row0 + row, pos0 = m.L - m.n, pos = pos0 + rr / G;
            const int64_t row_step = (int64_t)m.n * p.num_q_heads;  // from a page's sums to the next one's
            float *dst = pw_sums(p, PwSeq{m.c0, m.n, m.L}) + m.j * row_step + (int64_t)m.h * (m.n * G) + rr;
#pragma unroll
            for (int hh = 0; hh < 2; hh++) {
                uint32_t x[2][32];
                tmem_ld32_async(tm + 64 * hh, x[0]);
                tmem_ld32_async(tm + 64 * hh + 32, x[1]);
                tmem_ld_wait();
                if (hh == 1) {  // S may be written again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.s_free[ss]);
                }
                float s[64];
#pragma unroll
                for (int e = 0; e < 64; e++) s[e] = __uint_as_float(x[e >> 5][e & 31]);
                const int k0 = (m.j + hh) * kPage;
                if (k0 + kPage - 1 > pos0) {  // keys past some row's position
#pragma unroll
                    for (int e = 0; e < 64; e++)
                        if (k0 + e > pos) s[e] = -INFINITY;
                }
                float m8[8];
#pragma unroll
                for (int y = 0; y < 8; y++) {
                    const float *v = s + 8 * y;
                    m8[y] = max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), fmaxf(v[6], v[7]));
                }
                const float mx = max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                const float f = fmaxf(m.sk[hh] * sabs, kPwMinScale);
                const float off = mx == -INFINITY ? 0.0f : -f * mx;
                const uint64_t f2 = pk2(f, f), r2 = pk2(off, off);
                uint64_t sum[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < 32; e++) {
                    float x0, x1;
                    upk2(fma2(pk2(s[2 * e], s[2 * e + 1]), f2, r2), x0, x1);
                    sum[e & 3] = add2(sum[e & 3], pk2(ex2_approx(x0), ex2_approx(x1)));
                }
                float la, lb;
                upk2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), la, lb);
                if (hh < m.pages && rr < m.n * G) dst[hh * row_step] = f * mx + __log2f(la + lb);
            }
        }
    } else if (warp < 2) {
        if (lane == 0) {
            // ---- an MMA thread: steps warp, warp + 2, ... ----
            const uint32_t hi = (uint32_t)(umma_desc(smem_addr(sm.k[0])) >> 32);
            const uint32_t k_lo = (uint32_t)umma_desc(smem_addr(sm.k[0]));
            Turn<kKeyStages> key;
            Turn<kScoreStages> score;
            int have = -1;  // the query tile that was waited for
            for (int i = 0; i < steps && ok; i++, key.next(), score.next()) {
                if ((i & 1) != warp) continue;
                ok = mbar_wait_short(&sm.k_full[key.stage], key.parity);
                if (!ok) break;
                const int tile = sm.meta[i % kMeta].tile, first = sm.meta[i % kMeta].first, left = sm.meta[i % kMeta].left;
                if (tile != have) ok = mbar_wait_short(&sm.q_full[tile & 1], (uint32_t)(tile >> 1) & 1u);
                have = tile;
                if (ok && i >= kScoreStages) ok = mbar_wait_short(&sm.s_free[score.stage], score.parity ^ 1u);
                if (!ok) break;
                tc_fence_after();
                const uint32_t b = k_lo + key.stage * (kWinTile >> 4), a = tmem + 256 + 64 * (tile & 1);
#pragma unroll
                for (int k = 0; k < 8; k++)
                    umma_f16_ts(tmem + 128 * score.stage, a + 8 * k,
                                b + (uint32_t)(((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4), hi, kWinIdesc,
                                k > 0 ? 1u : 0u);
                // both threads let a tile go after their last step of it (one for both where it has one step)
                if (left <= 1) umma_commit(&sm.q_free[tile & 1]);
                if (left == 0 && first) umma_commit(&sm.q_free[tile & 1]);
                umma_commit(&sm.s_full[score.stage]);
                umma_commit(&sm.k_free[key.stage]);
            }
            umma_commit(&sm.mma_done);  // whatever was issued completes before tensor memory is freed
            if (!mbar_wait_short(&sm.mma_done, 0u)) ok = false;
        }
    } else if (warp < 4) {
        // ---- pages and copies of steps warp - 2, warp, ...: lane l looks up step l of 32, two rings in turn ----
        WinStep ring[2];
        uint32_t ph[2][2];
        auto look = [&](int i, WinStep &m, uint32_t (&at)[2]) {
            if (i + lane >= steps) return;
            int k, all;
            const int b = place(first + i + lane, m, k, all);
            m.first = k == 0 || i + lane == 0;
            m.left = min(all - 1 - k, steps - 1 - (i + lane));
#pragma unroll
            for (int x = 0; x < 2; x++) {
                at[x] = 0;
                m.sk[x] = 0.0f;
                if (x >= m.pages) continue;
                int pg = p.block_table[(int64_t)b * p.max_blocks + m.j + x];
                if (pg < 0 || pg >= p.num_pages) {
                    set_flag(p.status, KVQ_FLAG_BAD_PAGE);
                    pg = 0;
                }
                at[x] = (uint32_t)pg * (uint32_t)H + (uint32_t)m.h;
                m.sk[x] = p.k_scales[at[x]];  // (not waited for: the copies come first)
            }
        };
        look(0, ring[0], ph[0]);
        Turn<kCodeStages> code;
        int tile = -1, mine = 0;  // steps copied here
        for (int i = 0; i < steps; i++, code.next()) {
            if ((i & 31) == kCodeStages) {  // (once the stages are filled)
                if (i & 32)
                    look(i - kCodeStages + 32, ring[0], ph[0]);
                else
                    look(i - kCodeStages + 32, ring[1], ph[1]);
            }
            tile += i & 32 ? __shfl_sync(kFull, ring[1].first, i & 31) : __shfl_sync(kFull, ring[0].first, i & 31);
            if ((i & 1) != (warp & 1)) continue;
            if (i >= kCodeStages) ok = __all_sync(kFull, mbar_wait_short(&sm.code_free[code.stage], code.parity ^ 1u));
            if (!ok) break;
            auto issue = [&](WinStep &m, const uint32_t (&at)[2]) {
                if (lane == (i & 31)) {
                    uint64_t *bar = &sm.code_full[code.stage];
#pragma unroll
                    for (int x = 0; x < 2; x++)
                        if (x < m.pages)
                            bulk_copy_g2s(sm.code[code.stage] + x * kPageBytes, p.k_codes + (size_t)at[x] * kPageBytes,
                                          kPageBytes, bar);
                    m.tile = tile;
                    sm.meta[i % kMeta] = m;  // (the phase is not over before the arrival, whatever has come)
                    mbar_arrive_expect_tx(bar, m.pages * kPageBytes);
                }
            };
            if (i & 32)
                issue(ring[1], ph[1]);
            else
                issue(ring[0], ph[0]);
            mine = i + 1;
        }
        // no copy in flight when the CTA ends
        for (int i = mine - 1; i >= 0 && i > mine - 1 - kCodeStages; i -= 2)
            if (!mbar_wait_short(&sm.code_full[i % kCodeStages], (uint32_t)(i / kCodeStages) & 1u)) ok = false;
    } else {
        // ---- query rows ----
        const int row = (warp & 3) * 32 + lane;
        const __half2 flip = __float2half2_rn(p.score_scale < 0.0f ? -1.0f : 1.0f);
        Turn<2> query;
        int tiles = 0;
        for (int i = 0; i < steps; tiles++, query.next()) {
            WinStep m;
            int k, all;
            place(first + i, m, k, all);
            i += all - k;
            const int rr = m.row0 + row;
            const bool live = rr < m.n * G;
            const uint4 *q = reinterpret_cast<const uint4 *>(
                p.q + ((int64_t)(m.c0 + rr / G) * p.num_q_heads + m.h * G + rr % G) * kHeadDim);
            uint32_t x[2][32];
#pragma unroll
            for (int c = 0; c < 16; c++) {
                uint4 v = live ? q[c] : make_uint4(0u, 0u, 0u, 0u);
                if constexpr (FMT == KVQ_INT4_B64) v = as_pairs(v);
                const uint32_t y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; e++)
                    x[c >> 3][4 * (c & 7) + e] = h2_bits(__hmul2(*reinterpret_cast<const __half2 *>(&y[e]), flip));
            }
            if (tiles >= 2) ok = mbar_wait_short(&sm.q_free[query.stage], query.parity ^ 1u);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t tm = tmem + 256 + 64 * query.stage + ((uint32_t)((warp & 3) * 32) << 16);
            tmem_st32(tm, x[0]);
            tmem_st32(tm + 32, x[1]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_full[query.stage]);
        }
    }
    __syncwarp();
    if (!ok) set_flag(p.status, KVQ_FLAG_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kWinTmem));
}

template <int FMT>
static cudaError_t launch_page_window_fmt(const PageWeightsParams &p, int num_sms, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(page_window_kernel<FMT>, sizeof(WinSmem), done);
    if (e != cudaSuccess) return e;
    return launch_pdl(page_window_kernel<FMT>, dim3((unsigned)num_sms), dim3(kWinThreads), sizeof(WinSmem), s, p);
}

cudaError_t launch_page_window(int fmt, const PageWeightsParams &p, int num_sms, cudaStream_t s)
{
    if (fmt == KVQ_INT4_B64) return launch_page_window_fmt<KVQ_INT4_B64>(p, num_sms, s);
    if (fmt == KVQ_FP8_E4M3) return launch_page_window_fmt<KVQ_FP8_E4M3>(p, num_sms, s);
    return launch_page_window_fmt<KVQ_INT8_PAGE>(p, num_sms, s);
}

}  // namespace kvq
