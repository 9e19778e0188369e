// kvq_prompt.cu -- causal attention of whole prompts over their own fp16 or
// bf16 rows: packed sequences of different lengths, grouped query heads.  What
// a first prompt runs beside kvq_append, which quantizes the same rows (dynamic
// chunked attention, "R1 performance overview", aicoding.csdn.net; grouped
// heads as for decode, ddd.cn section 2).
//
//   out_i = sum_{t <= i} softmax_t(scale q_i . k_t) v_t,  lse_i = ln sum_{t <= i} e^(scale q_i . k_t)
//
// Bound by the tensor cores (4 * 128 flops per query head and key, every byte
// read about once from HBM): tcgen05 with S, P and O in tensor memory, operands
// brought by TMA.  One CTA per SM stays resident and takes units in turn; a unit
// is two tiles of 128 query rows of one (sequence, cache head).  A tile's rows
// are tokens x query heads of the group (row = token * heads + head), so that a
// group of any size reads its cache head's keys once and short prompts fill the
// tile with heads: an even group's tiles share the tokens, half of the heads
// each; an odd group's tiles have all heads of neighbouring tokens.  Keys go in
// steps of 128.
//
// Roles (warps), handing over through mbarriers:
//   0, 2      one thread each issues the MMAs of a tile: S = Q K^T, O += P V,
//             M = N = 128.  (An MMA holds its issuer until the tensor pipe takes it,
//             and a wait between MMAs costs ~100 cycles: with one thread for both
//             tiles the pipe was busy 49% of the time.)
//   1         takes units, tells the other roles and issues the copies of K and V
//             (TMA) into a ring of four 32 KB stages.
//   3         issues the copies of the Q tiles.  The last step(s) of a unit hold
//             keys past some row's position: of their V this warp zeroes the rows
//             past the sequence's end and takes out values that are not finite
//             (0 * inf would reach rows that do not see them; the epilogue adds
//             them to the rows that do).
//   4-7, 8-11 softmax of tile 0, tile 1: one thread per query row.  A row of S
//             (128 scores) is read into registers once; maximum, 2^(s - m), the
//             row sum in binary32; P rounded to the operands' type (the tensor
//             cores take nothing wider) goes over S in three parts.  The running
//             maximum is lazy: O is rescaled only when a row's maximum grows by
//             more than 2^8, so P stays in [0, 256].
//   12-15     the epilogue: O / l, while the tensor cores are on the next unit.
// While one tile's rows are in the softmax, the tensor cores work on the other:
// the MMA threads take turns, [O += P V, next S] of one tile after the other.
// Without the order both tiles' softmaxes fall together and the pipe idles (16384
// tokens x 64 heads: 3.8 ms against 2.9).
//
// Measured (GB300): 16384 tokens x 64 / 8 heads 2.9 ms alone, 3.0 - 3.1 ms back to
// back at the power cap (1.42 - 1.52 PFLOP/s, 0.74 - 0.79 of the measured bf16
// rate); 8 x 2048 tokens x 32 heads 248 - 265 us (1.04 - 1.11 PFLOP/s), where a unit
// has 8.5 steps: its first and last steps, O's way out and the turn between units
// cost about as much as two of them.  A steady step of both tiles takes ~2900 - 3300
// cycles for 2048 of MMAs: half as many loads or no exponentials at all gain 4% each.
//
// Unit order: cache heads in groups whose keys and values fit half of L2, since
// each level reads them again (8 x 2048 x 32 heads, 268 MB of them, inputs warm:
// 250 us; 263 with groups of 48 MB, 258 with 128 MB); of a group by the number of
// the unit in its sequence, the highest (most keys) first, over sequences and heads.
// Units go to the CTAs as they come free: the grid has a CTA for each (16 per SM at
// most, then a ticket is several units), and one that runs takes the places of those
// that have not started.  Dealt in a fixed order, forwards and backwards in turn, the
// busiest CTA had 4% (8 x 2048) to 6% (16 prompts of 65 .. 8192 tokens) more steps than
// the mean: 16 prompts 858 us, 829 so; 24 of 50 .. 4000 tokens 1145, 1085; 6 of 150 .. 2000
// x 32 / 32 heads 76, 72; against 980, 1065 where a ticket is six units (150 of 10 .. 1200
// tokens x 32 / 32 heads).
#include <cuda.h>

#include <type_traits>

#include "kvq_around.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_tc.cuh"

namespace kvq {

namespace {

constexpr int kTileRows = 128;
constexpr int kUnitTiles = 2;
constexpr int kKeys = 128;
constexpr int kStages = 4;
constexpr int kOutPitch = 144;  // bytes: 128 and a step of 16 that keeps the rows' banks apart
constexpr int kParts = 3;  // P is handed over as keys 0..63, 64..95, 96..127
constexpr int kTileBytes = kTileRows * kHeadDim * 2;
constexpr int64_t kGroupBytes = 64 << 20;  // half of L2
constexpr int kPromptThreads = 512;
constexpr uint32_t kPromptTmem = 512;  // tile t: S / P at columns 256 t, O at 256 t + 128
constexpr float kLazy = 8.0f;
constexpr float kLn2 = 0.693147180559945309f;
// a softmax scale of 0 scores 1e-38 * raw instead, so that a masked score stays -inf
constexpr float kMinScale = 1.17549435e-38f;
// registers per thread after the split: 2 * 184 + 80 + 64 = 4 * 128, the launch's (nothing is
// spilled; with 176, 104 and 56 the spills cost 7%)
constexpr int kRegsSoftmax = 184, kRegsEpilogue = 80, kRegsIssue = 64;
static_assert(2 * kRegsSoftmax + kRegsEpilogue + kRegsIssue <= 4 * (65536 / kPromptThreads), "register split");

template <int N>
using Int = std::integral_constant<int, N>;

// 16-bit element type: fp16 or bf16
template <bool BF>
struct Elem {
    // f32 += a x b, M = 128, N = 128, K-major A and B (PV: B MN-major)
    static constexpr uint32_t kIdescS =
        (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
    static constexpr uint32_t kIdescO = kIdescS | (1u << 16);
    static constexpr uint32_t kExp = BF ? 0x7F807F80u : 0x7C007C00u;  // exponent bits of a pair
    static constexpr uint32_t kOne = BF ? 0x00800080u : 0x04000400u;  // their last
    __device__ static __forceinline__ uint32_t pack(float a, float b)
    {
        if constexpr (BF) {
            uint32_t d;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
            return d;
        } else {
            return f16x2_rn(a, b);
        }
    }
    // the larger magnitudes of two pairs, a NaN if there is one
    __device__ static __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
    {
        uint32_t d;
        if constexpr (BF)
            asm("{\n\t.reg .b32 x;\n\tabs.bf16x2 x, %2;\n\tmax.NaN.bf16x2 %0, %1, x;\n\t}" : "=r"(d) : "r"(a), "r"(b));
        else
            asm("{\n\t.reg .b32 x;\n\tabs.f16x2 x, %2;\n\tmax.NaN.f16x2 %0, %1, x;\n\t}" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    // bit 15 / 31 set where the pair's low / high value is not finite
    __device__ static __forceinline__ uint32_t wild(uint32_t w) { return ((w & kExp) + kOne) & 0x80008000u; }
    __device__ static __forceinline__ float value(uint16_t x)
    {
        if constexpr (BF)
            return __uint_as_float((uint32_t)x << 16);
        else
            return __half2float(__ushort_as_half(x));
    }
};

struct PromptUnit {
    int32_t c0, n, h, tok0;  // first row and length of the sequence, cache head, first token; n < 0: no more units
};

struct alignas(1024) PromptSmem {
    uint8_t q[kUnitTiles][kTileBytes];
    uint8_t kv[kStages][kTileBytes];
    uint8_t o[4][32 * kOutPitch];  // by epilogue warp: 64 elements of its 32 rows on their way out
    uint64_t kv_full[kStages];   // a stage's copy done: K, or V of a step without masked keys
    uint64_t kv_raw[kStages];    // the same for V of a mixed step (then kv_clean)
    uint64_t kv_clean[kStages];  // that V cleaned
    uint64_t kv_free[kStages];   // the MMAs that read the stage complete
    uint64_t q_full[kUnitTiles], q_free[kUnitTiles];
    uint64_t s_full[kUnitTiles];   // S of a step complete, and every MMA before it
    uint64_t p_full[kUnitTiles][kParts];  // a part of P in tensor memory (the first: O rescaled too)
    uint64_t turn[kUnitTiles];     // the MMA thread of a tile may issue
    uint64_t o_full[kUnitTiles];   // a unit's last PV complete
    uint64_t o_free[kUnitTiles];   // O and ml read by the epilogue
    uint64_t ml_full[kUnitTiles];  // a unit's maxima and sums written
    uint64_t unit_full[2], unit_free[2];
    uint64_t ticket_full;
    uint64_t mma_done;
    uint4 ticket;  // the answer to a request for one
    float2 ml[kUnitTiles][kTileRows];
    PromptUnit unit[2];
    uint32_t wild[4];  // by unit: some value of a mixed step is not finite (warp 3 may be two units ahead)
    uint32_t tmem;
};
static_assert(sizeof(PromptSmem) <= 227 * 1024, "one CTA's shared memory");

// what a unit spans, from its record
struct Span {
    int active;             // tiles with a token
    int steps[kUnitTiles];  // key steps of a tile
    int total;              // of the unit
    int mixed;              // first step with keys past some row's position
    __device__ __forceinline__ Span(const PromptUnit &u, const PromptParams &p)
    {
        const int t1 = u.tok0 + p.tile1_token;  // tile 1's first token
        active = u.n > t1 ? 2 : 1;
        steps[0] = (min(u.tok0 + p.tile_tokens, u.n) - 1) / kKeys + 1;
        steps[1] = active == 2 ? (min(t1 + p.tile_tokens, u.n) - 1) / kKeys + 1 : 0;
        total = max(steps[0], steps[1]);
        mixed = (u.tok0 + 1) / kKeys;
    }
};

// a position in the ring of stages
struct Ring {
    uint32_t stage = 0, phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

template <int N>
__device__ __forceinline__ void regs_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Take the place of a CTA of this grid that has not started: the answer (16 bytes) comes to `dst`.
__device__ __forceinline__ void ask_ticket(uint4 *dst, uint64_t *bar)
{
    mbar_arrive_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_addr(dst)),
        "r"(smem_addr(bar))
        : "memory");
}
// Its block index, or -1: every CTA has started (and no further request may be made).
__device__ __forceinline__ int read_ticket(const uint4 *src)
{
    int id;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%1];\n\tmov.b32 %0, -1;\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
        : "=r"(id)
        : "r"(smem_addr(src))
        : "memory");
    return id;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

}  // namespace

template <bool BF, bool NEG>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_attn_kernel(PromptParams p, const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    using E = Elem<BF>;
    extern __shared__ __align__(1024) uint8_t smem_prompt[];
    PromptSmem &sm = *reinterpret_cast<PromptSmem *>(smem_prompt);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.group, tt = p.tile_tokens, th = p.tile_heads;

    pdl_launch_dependents();
    if (tid == 32) {
        prefetch_map(&map_k);
        prefetch_map(&map_v);
        prefetch_map(&map_q);
    }
    if (tid == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&sm.kv_full[s], 1);
            mbar_init(&sm.kv_free[s], 2);  // both MMA threads
            mbar_init(&sm.kv_raw[s], 1);
            mbar_init(&sm.kv_clean[s], 1);
        }
        for (int t = 0; t < kUnitTiles; t++) {
            mbar_init(&sm.q_full[t], 1);
            mbar_init(&sm.q_free[t], 1);
            mbar_init(&sm.s_full[t], 1);
            for (int x = 0; x < kParts; x++) mbar_init(&sm.p_full[t][x], 4);
            mbar_init(&sm.turn[t], 1);
            mbar_init(&sm.o_full[t], 1);
            mbar_init(&sm.o_free[t], 4);
            mbar_init(&sm.ml_full[t], 4);
        }
        for (int s = 0; s < 2; s++) {
            mbar_init(&sm.unit_full[s], 1);
            mbar_init(&sm.unit_free[s], 15);  // 8 softmax warps, 4 epilogue warps, 2 MMA threads, warp 3
        }
        mbar_init(&sm.ticket_full, 1);
        mbar_init(&sm.mma_done, 2);
        mbar_init_fence();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)),
                     "r"(kPromptTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();  // (nothing of global memory is read before it)
    const uint32_t tmem = sm.tmem;
    bool ok = true;

    // the r-th unit of this CTA, for every role but the loader's
    auto fetch = [&](int r, PromptUnit &u) {
        ok = mbar_wait_short(&sm.unit_full[r & 1], (uint32_t)(r >> 1) & 1u);
        if (ok) u = sm.unit[r & 1];
        return ok;
    };

    if (warp >= 4 && warp < 12) {
        // ---- softmax: tile t, one query row per thread (its lane of tensor memory) ----
        regs_inc<kRegsSoftmax>();
        const int t = (warp >> 2) - 1, row = tid & 127;
        const uint32_t tm = tmem + 256u * t + ((uint32_t)((warp & 3) * 32) << 16);
        const float sabs = fmaxf(fabsf(p.score_scale), kMinScale);
        uint32_t s_phase = 0, done = 0;  // steps of this tile, units of this tile
        for (int r = 0;; r++) {
            PromptUnit u;
            bool got = fetch(r, u);
            got = __all_sync(kFull, got);
            __syncwarp();
            if (lane == 0 && got) mbar_arrive(&sm.unit_free[r & 1]);
            if (!got) {
                ok = false;
                break;
            }
            if (u.n < 0) break;
            const Span sp(u, p);
            if (t >= sp.active) continue;
            const int nst = sp.steps[t], tok_t = u.tok0 + t * p.tile1_token;
            const int pos = row < th * tt ? tok_t + row / th : -1;
            float m_used = -INFINITY;
            uint64_t l2 = pk2(0.0f, 0.0f);
            for (int i = 0; i < nst; i++) {
                ok = __all_sync(kFull, mbar_wait_short(&sm.s_full[t], s_phase & 1u));
                s_phase++;
                if (!ok) break;
                tc_fence_after();
                float s[128];
                {
                    uint32_t x[4][32];
#pragma unroll
                    for (int c = 0; c < 4; c++) tmem_ld32_async(tm + 32 * c, x[c]);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; c++)
#pragma unroll
                        for (int e = 0; e < 32; e++) s[32 * c + e] = __uint_as_float(x[c][e]);
                }
                if constexpr (NEG) {  // a negative softmax scale
#pragma unroll
                    for (int e = 0; e < 128; e++) s[e] = -s[e];
                }
                if (i * kKeys + kKeys - 1 > tok_t) {
                    const int last = pos - i * kKeys;  // keys after it are masked
#pragma unroll
                    for (int e = 0; e < 128; e++)
                        if (e > last) s[e] = -INFINITY;
                }
                float m8[8];
#pragma unroll
                for (int x = 0; x < 8; x++) {
                    const float *v = s + 16 * x;
                    m8[x] = max3(v[0], v[1], v[2]);
#pragma unroll
                    for (int e = 3; e < 15; e += 2) m8[x] = max3(m8[x], v[e], v[e + 1]);
                    m8[x] = fmaxf(m8[x], v[15]);
                }
                const float raw = max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                const float mx = raw == -INFINITY ? -INFINITY : raw * sabs;
                float factor = 1.0f;
                if (i == 0) {
                    m_used = mx;
                } else if (mx > m_used + kLazy) {
                    factor = ex2_approx(m_used - mx);
                    m_used = mx;
                }
                // O holds the PV of the step before (complete before this S): rescale where a maximum moved
                if (__any_sync(kFull, factor != 1.0f)) {
#pragma unroll 1
                    for (int c = 0; c < 4; c++) {
                        uint32_t x[32];
                        tmem_ld32_async(tm + 128 + 32 * c, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; e++) x[e] = __float_as_uint(__uint_as_float(x[e]) * factor);
                        tmem_st32(tm + 128 + 32 * c, x);
                    }
                    l2 = mul2(l2, pk2(factor, factor));
                }
                // a row without a key in range (past its sequence): every score is -inf and P is 0
                const float off = m_used == -INFINITY ? 0.0f : -m_used;
                const uint64_t sc2 = pk2(sabs, sabs), off2 = pk2(off, off);
                uint64_t sum2[2] = {pk2(0.0f, 0.0f), pk2(0.0f, 0.0f)};
                auto part = [&](auto first, auto count, uint64_t *bar) {  // pairs of keys
                    constexpr int A = decltype(first)::value, N = decltype(count)::value;
                    uint32_t w[N];
#pragma unroll
                    for (int e = 0; e < N; e++) {
                        float x0, x1;
                        upk2(fma2(pk2(s[2 * (A + e)], s[2 * (A + e) + 1]), sc2, off2), x0, x1);
                        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                        sum2[e & 1] = add2(sum2[e & 1], pk2(p0, p1));
                        w[e] = E::pack(p0, p1);
                    }
                    if constexpr (N == 32)
                        tmem_st32(tm + A, w);
                    else
                        tmem_st16(tm + A, w);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                };
                part(Int<0>(), Int<32>(), &sm.p_full[t][0]);
                part(Int<32>(), Int<16>(), &sm.p_full[t][1]);
                part(Int<48>(), Int<16>(), &sm.p_full[t][2]);
                l2 = add2(l2, add2(sum2[0], sum2[1]));
            }
            if (!ok) break;
            // the epilogue has read the unit before's ml
            if (done > 0) ok = __all_sync(kFull, mbar_wait_short(&sm.o_free[t], (done - 1) & 1u));
            if (!ok) break;
            float la, lb;
            upk2(l2, la, lb);
            sm.ml[t][row] = make_float2(m_used, la + lb);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.ml_full[t]);
            done++;
        }
    } else if (warp >= 12) {
        // ---- the epilogue ----
        regs_dec<kRegsEpilogue>();
        const int row = tid & 127;
        const uint32_t lane_tm = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        uint32_t done[kUnitTiles] = {0, 0};
        for (int r = 0; ok; r++) {
            PromptUnit u;
            ok = __all_sync(kFull, fetch(r, u));
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(&sm.unit_free[r & 1]);
            if (!ok || u.n < 0) break;
            const Span sp(u, p);
#pragma unroll 1
            for (int t = 0; t < sp.active && ok; t++) {
                ok = __all_sync(kFull, mbar_wait_short(&sm.ml_full[t], done[t] & 1u));
                if (!ok) break;
                const float2 ml = sm.ml[t][row];
                const float inv = 1.0f / ml.y;
                const int tok = u.tok0 + t * p.tile1_token + row / th, hq = u.h * G + t * p.tile1_head + row % th;
                const bool live = row < th * tt && tok < u.n;
                ok = __all_sync(kFull, mbar_wait_short(&sm.o_full[t], done[t] & 1u));
                if (!ok) break;
                done[t]++;
                tc_fence_after();
                const bool wild = sm.wild[r & 3] != 0;
                const int64_t at = (int64_t)(u.c0 + tok) * p.num_q_heads + hq;
                // The rows leave through shared memory, 4 of 128 bytes an instruction: 16 bytes a lane of 32
                // rows straight from registers hold up every other warp's shared-memory access.
                const int64_t at0 = (int64_t)(u.c0 + u.tok0) * p.num_q_heads + u.h * G;
                const int rel = live ? (int)(at - at0) : -1;
                uint8_t *stage = sm.o[warp & 3];
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        uint32_t x[32], o[16];
                        tmem_ld32_async(lane_tm + 256 * t + 128 + 64 * half + 32 * c, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            o[e] = E::pack(__uint_as_float(x[2 * e]) * inv, __uint_as_float(x[2 * e + 1]) * inv);
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            *reinterpret_cast<uint4 *>(stage + lane * kOutPitch + 64 * c + 16 * e) =
                                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                    if (half == 1) tc_fence_before();
                    __syncwarp();
                    if (half == 1 && lane == 0) mbar_arrive(&sm.o_free[t]);  // O may be written again
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const int to = __shfl_sync(kFull, rel, 4 * k + (lane >> 3));
                        const uint4 x =
                            *reinterpret_cast<const uint4 *>(stage + (4 * k + (lane >> 3)) * kOutPitch + 16 * (lane & 7));
                        if (to >= 0)
                            *reinterpret_cast<uint4 *>(p.out + (at0 + to) * kHeadDim + 64 * half + 8 * (lane & 7)) = x;
                    }
                }
                __syncwarp();
                if (!live) continue;
                if (p.lse) p.lse[at] = (ml.x + __log2f(ml.y)) * kLn2;
                // (the lanes that stored this row did so before the barrier)
                if (wild) {  // what is not finite among the values this row sees in the mixed steps decides its element
#pragma unroll 1
                    for (int d = 0; d < kHeadDim; d++) {
                        float y = 0.0f;
#pragma unroll 1
                        for (int j = sp.mixed * kKeys; j <= tok; j++) {
                            const float x = E::value(p.v[(int64_t)(u.c0 + j) * p.v_stride + u.h * kHeadDim + d]);
                            if (!(fabsf(x) < INFINITY)) y += x;
                        }
                        if (!(y == 0.0f)) p.out[at * kHeadDim + d] = (uint16_t)E::pack(y, 0.0f);
                    }
                }
            }
        }
    } else {
        regs_dec<kRegsIssue>();
        if ((warp & 1) == 0 && lane == 0) {
            // ---- the MMA thread of tile t (warps 0 and 2) ----
            const int t = warp >> 1;
            const uint32_t tm = tmem + 256 * t;
            const uint32_t hi = (uint32_t)(umma_desc(smem_addr(sm.q[0])) >> 32);
            const uint32_t hi_v = (uint32_t)(umma_desc_mn(smem_addr(sm.kv[0]), kKeys * 128, 1024) >> 32);
            const uint32_t q_lo = (uint32_t)umma_desc(smem_addr(sm.q[t]));
            const uint32_t k_lo = (uint32_t)umma_desc(smem_addr(sm.kv[0]));
            const uint32_t v_lo = (uint32_t)umma_desc_mn(smem_addr(sm.kv[0]), kKeys * 128, 1024);
            constexpr uint32_t kStep = kTileBytes >> 4;
            Ring ring;                                 // the stage to read next, K and V alternating
            uint32_t p_phase = 0, turn_phase = 0, uses = 0;
            uint32_t full_phase = 0, clean_phase = 0;  // bit s: parity of stage s's next kv_full, kv_clean
            if (t == 0) mbar_arrive(&sm.turn[0]);  // tile 0 begins
            auto wait_full = [&](uint32_t stage) {
                const uint32_t parity = full_phase >> stage & 1u;
                full_phase ^= 1u << stage;
                return mbar_wait_short(&sm.kv_full[stage], parity);
            };
            auto wait_clean = [&](uint32_t stage) {
                const uint32_t parity = clean_phase >> stage & 1u;
                clean_phase ^= 1u << stage;
                return mbar_wait_short(&sm.kv_clean[stage], parity);
            };
            for (int r = 0; ok; r++) {
                PromptUnit u;
                if (!fetch(r, u)) break;
                mbar_arrive(&sm.unit_free[r & 1]);
                if (u.n < 0) break;
                const Span sp(u, p);
                const int nst = t == 0 ? sp.steps[0] : sp.steps[1];
                // S of a step goes over P of the step before, whose PV was issued before it: the
                // tensor pipe runs one thread's MMAs in order
                auto issue_s = [&](uint32_t stage, bool pass) {
                    const uint32_t b = k_lo + stage * kStep;
#pragma unroll
                    for (int ks = 0; ks < 8; ks++) {
                        const uint32_t d = (uint32_t)(((ks >> 2) * (kTileRows * 128) + (ks & 3) * 32) >> 4);
                        umma_f16_ss(tm, q_lo + d, hi, b + d, hi, E::kIdescS, ks > 0 ? 1u : 0u);
                        if (ks == 4 && pass) mbar_arrive(&sm.turn[t ^ 1]);  // the pipe is fed while it wakes
                    }
                    umma_commit(&sm.s_full[t]);
                };
                if (nst > 0) {
                    ok = mbar_wait_short(&sm.q_full[t], uses & 1u) && wait_full(ring.stage);
                    if (!ok) break;
                    tc_fence_after();
                    issue_s(ring.stage, false);
                    umma_commit(&sm.kv_free[ring.stage]);
                    if (nst == 1) umma_commit(&sm.q_free[t]);
                    ring.next();
                    if (uses > 0) ok = mbar_wait_short(&sm.o_free[t], (uses - 1) & 1u);
                } else {
                    ok = wait_full(ring.stage);
                    if (ok) mbar_arrive(&sm.kv_free[ring.stage]);
                    ring.next();
                }
                for (int i = 0; i < sp.total && ok; i++) {
                    // O += P(i) V(i), in the parts that the softmax hands over, then S(i + 1); the
                    // tiles take turns (one without this step passes its own on), so that one's softmax runs
                    // while the other's MMAs do
                    const bool live = i < nst, more = i + 1 < nst;
                    const uint32_t stage_v = ring.stage;
                    ring.next();
                    ok = i >= sp.mixed ? wait_clean(stage_v) : wait_full(stage_v);
                    // (the next K's wait ahead of the turn: nothing comes between this PV and the next S)
                    if (i + 1 < sp.total) ok = ok && wait_full(ring.stage);
                    if (live) ok = ok && mbar_wait_short(&sm.p_full[t][0], p_phase);
                    ok = ok && mbar_wait_short(&sm.turn[t], turn_phase);
                    turn_phase ^= 1u;
                    if (!ok) break;
                    if (live) {
                        const uint32_t c = v_lo + stage_v * kStep;
#pragma unroll
                        for (int x = 0; x < kParts; x++) {
                            if (x > 0) ok = ok && mbar_wait_short(&sm.p_full[t][x], p_phase);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int ks = x == 0 ? 0 : 2 + 2 * x; ks < 4 + 2 * x; ks++)
                                umma_f16_ts(tm + 128, tm + 8 * ks, c + (uint32_t)((ks * 16 * 128) >> 4), hi_v,
                                            E::kIdescO, i == 0 && ks == 0 ? 0u : 1u);
                        }
                        if (!ok) break;
                        p_phase ^= 1u;
                        if (more)
                            issue_s(ring.stage, true);
                        else
                            umma_commit(&sm.o_full[t]);
                        umma_commit(&sm.kv_free[stage_v]);
                    } else {
                        mbar_arrive(&sm.kv_free[stage_v]);
                    }
                    if (!more) mbar_arrive(&sm.turn[t ^ 1]);
                    if (i + 1 < sp.total) {
                        if (more)
                            umma_commit(&sm.kv_free[ring.stage]);
                        else  // the other tile's K, seen so that the phases stay in step
                            mbar_arrive(&sm.kv_free[ring.stage]);
                        ring.next();
                    }
                    if (i + 2 == nst) umma_commit(&sm.q_free[t]);
                }
                uses += nst > 0;
            }
            umma_commit(&sm.mma_done);  // whatever was issued completes before tensor memory is freed
            if (!mbar_wait_short(&sm.mma_done, 0u)) ok = false;
        } else if (warp == 1) {
            // ---- units and copies ----
            const int H = p.num_heads, ut = p.unit_tokens;
            // a sequence's length, -1 where its bounds are broken
            auto length = [&](int b) {
                const int c0 = p.cu[b], n = p.cu[b + 1] - c0;
                return n >= 0 && n <= p.max_n && c0 >= 0 && (int64_t)c0 + n <= p.total ? n : -1;
            };
            const bool few = p.num_seqs <= 32;  // lengths and first rows stay in registers
            const int mine = few && lane < p.num_seqs ? length(lane) : 0;
            const int mine_c0 = few && lane < p.num_seqs ? p.cu[lane] : 0;
            // sequences (of 32 from b0 on) with a unit number x, as a mask
            auto longer = [&](int b0, int x) {
                const int n = few ? mine : b0 + lane < p.num_seqs ? length(b0 + lane) : 0;
                return __ballot_sync(kFull, n > (int64_t)x * ut);
            };
            int longest = 0;
            int64_t tokens = 0, units = 0;
#pragma unroll 1
            for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
                const int n = few ? mine : b0 + lane < p.num_seqs ? length(b0 + lane) : 0;
                if (n < 0) set_flag(p.status, KVQ_FLAG_BAD_LENGTH);
                longest = max(longest, n);
                tokens += max(n, 0);
                units += (max(n, 0) + (int64_t)ut - 1) / ut * H;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                tokens += __shfl_xor_sync(kFull, tokens, o);
                units += __shfl_xor_sync(kFull, units, o);
            }
            const int top = (int)((__reduce_max_sync(kFull, longest) + (int64_t)ut - 1) / ut) - 1;
            // heads go in groups whose K and V stay in L2 while all levels read them
            const int64_t groups = (tokens * H * (kHeadDim * 4) + kGroupBytes - 1) / kGroupBytes;
            const int hg = groups > H ? 1 : groups > 1 ? (int)((H + groups - 1) / groups) : H;
            int x = top, h0 = 0, hn = hg;
            int64_t base = 0;        // units before level x of the heads from h0 on
            int count = 0, same = 0;  // sequences on level x; the last level with as many
            int at = 0, passed = 0;  // of the level's: `passed` come before sequence `at`, a multiple of 32
            auto enter = [&](int x) {
                int c = 0, below = 0;  // the longest sequence without a unit x
#pragma unroll 1
                for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
                    const int n = few ? mine : b0 + lane < p.num_seqs ? length(b0 + lane) : 0;
                    const bool on = n > (int64_t)x * ut;
                    c += __popc(__ballot_sync(kFull, on));
                    below = max(below, on ? 0 : n);
                }
                below = __reduce_max_sync(kFull, below);
                count = c;
                same = (int)((below + (int64_t)ut - 1) / ut);
                at = passed = 0;
            };
            if (units > 0) enter(x);
            // the unit of number `id`, a negative length behind the last one
            auto find = [&](int64_t id) {
                PromptUnit u = {0, -1, 0, 0};
                if (id >= units) return u;
                // (numbers come nearly in order: the search goes on where the last one ended, a few levels back at most)
                while (id < base) {
                    if (x == top) {
                        h0 -= hg;
                        hn = hg;
                        x = 0;
                    } else {
                        x++;
                    }
                    enter(x);
                    base -= (int64_t)count * hn;
                }
                while (id >= base + (int64_t)count * hn) {
                    const int64_t size = (int64_t)count * hn, past = (id - base) / size;
                    const int levels = x - same + 1, go = past < levels ? (int)past : levels;
                    base += go * size;
                    x -= go;
                    if (x < 0) {
                        h0 += hg;
                        hn = min(hg, H - h0);
                        x = top;
                    }
                    enter(x);
                }
                const uint32_t rank = (uint32_t)(id - base);  // (at most 65535 sequences x 65535 heads)
                const int k = (int)(rank / (uint32_t)hn);     // the k-th sequence of the level
                u.h = h0 + (int)(rank % (uint32_t)hn);
                if (k < passed) at = passed = 0;
                uint32_t m = longer(at, x);
#pragma unroll 1
                while (k >= passed + __popc(m) && at + 32 < p.num_seqs) {
                    passed += __popc(m);
                    at += 32;
                    m = longer(at, x);
                }
#pragma unroll 1
                for (int skip = k - passed; skip > 0; skip--) m &= m - 1u;
                const int b = min(at + max(__ffs(m) - 1, 0), p.num_seqs - 1);
                if (few) {
                    u.c0 = __shfl_sync(kFull, mine_c0, b);
                    u.n = __shfl_sync(kFull, mine, b);
                } else {
                    u.c0 = p.cu[b];
                    u.n = p.cu[b + 1] - u.c0;
                }
                u.tok0 = x * ut;
                return u;
            };
            // the r-th unit of this CTA to the other roles
            auto publish = [&](int r, const PromptUnit &u) {
                ok = __all_sync(kFull, r < 2 || mbar_wait_short(&sm.unit_free[r & 1], (uint32_t)((r >> 1) - 1) & 1u));
                if (lane == 0 && ok) {
                    sm.unit[r & 1] = u;
                    mbar_arrive(&sm.unit_full[r & 1]);
                }
            };
            // a ticket is `per` units; this CTA's own first, then those of CTAs that have not started
            const int64_t per = (units + gridDim.x - 1) / gridDim.x;
            int64_t id = (int64_t)blockIdx.x * per;
            int left = (int)per;  // of the ticket, with this one
            uint32_t answered = 0;
            bool more = true;  // no refusal yet
            auto answer = [&]() {
                const bool came = __all_sync(kFull, mbar_wait_short(&sm.ticket_full, answered++ & 1u));
                const int t = came ? read_ticket(&sm.ticket) : -1;
                if (!came) ok = false;
                more = t >= 0;
                return t;
            };
            Ring ring;
            uint32_t used = 0;  // stages filled so far, up to kStages
            // bit s: parity of stage s's next kv_full, kv_raw; whether its last fill was a mixed V
            uint32_t full_phase = 0, raw_phase = 0, last_raw = 0;
            PromptUnit u = find(id);
            for (int r = 0;; r++) {
                publish(r, u);
                if (!ok || u.n < 0) break;
                const bool last = left == 1 || id + 1 >= units;  // of the ticket
                const bool take = last && more;
                if (lane == 0) {
                    const Span sp(u, p);
                    auto stage = [&](const CUtensorMap *map, int key, bool raw) {
                        if (used >= kStages) ok = mbar_wait_short(&sm.kv_free[ring.stage], ring.phase ^ 1u);
                        if (!ok) return;
                        const uint32_t bit = 1u << ring.stage;
                        uint64_t *bar = raw ? &sm.kv_raw[ring.stage] : &sm.kv_full[ring.stage];
                        if (raw)
                            raw_phase ^= bit;
                        else
                            full_phase ^= bit;
                        last_raw = raw ? last_raw | bit : last_raw & ~bit;
                        uint8_t *dst = sm.kv[ring.stage];
                        mbar_arrive_expect_tx(bar, kTileBytes);
                        tma_load_3d(dst, map, 0, u.h, u.c0 + key, bar);
                        tma_load_3d(dst + kTileBytes / 2, map, 64, u.h, u.c0 + key, bar);
                        if (used < kStages) used++;
                        ring.next();
                    };
#pragma unroll 1
                    for (int i = 0; i < sp.total && ok; i++) {
                        // (an answer takes 1 - 2 us: asked for as late as the copies' waits cover it, so that a CTA
                        // takes a unit about when it is free)
                        if (take && i == max(sp.total - 2, 0)) ask_ticket(&sm.ticket, &sm.ticket_full);
#pragma unroll 1
                        for (int kv = 0; kv < 2 && ok; kv++)
                            stage(kv == 0 ? &map_k : &map_v, i * kKeys, kv == 1 && i >= sp.mixed);
                    }
                }
                ok = __all_sync(kFull, ok);
                if (!ok) break;  // (flagged; the answer, if one is on its way, comes long before the other waits run out)
                id++;
                left--;
                if (last) {
                    const int t = take ? answer() : -1;
                    id = t < 0 ? units : t * per;
                    left = (int)per;
                }
                u = find(id);
            }
            // the tickets behind the last unit, or each would start a CTA
            while (ok && more) {
                __syncwarp();  // (the last answer was read)
                if (lane == 0) ask_ticket(&sm.ticket, &sm.ticket_full);
                answer();
            }
            if (lane == 0) {  // no copy in flight when the CTA ends
                for (uint32_t s = 0; s < used; s++) {
                    const bool raw = last_raw >> s & 1u;
                    const uint32_t next = (raw ? raw_phase : full_phase) >> s & 1u;
                    if (!mbar_wait_short(raw ? &sm.kv_raw[s] : &sm.kv_full[s], next ^ 1u)) ok = false;
                }
            }
        } else if (warp == 3) {
            // ---- Q tiles (apart from K and V, whose copies would wait behind a tile in use), then
            // the V of the mixed steps ----
            uint32_t uses[kUnitTiles] = {0, 0};
            Ring ring;
            uint32_t raw_phase = 0;  // bit s: parity of stage s's next mixed V
            for (int r = 0; ok; r++) {
                PromptUnit u;
                ok = __all_sync(kFull, fetch(r, u));
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(&sm.unit_free[r & 1]);
                if (!ok || u.n < 0) break;
                const Span sp(u, p);
                if (lane == 0) {
                    sm.wild[r & 3] = 0u;
#pragma unroll
                    for (int t = 0; t < kUnitTiles; t++) {
                        if (t >= sp.active || !ok) continue;
                        if (uses[t] > 0) ok = mbar_wait_short(&sm.q_free[t], (uses[t] - 1) & 1u);
                        if (!ok) continue;
                        mbar_arrive_expect_tx(&sm.q_full[t], 2u * 128u * th * tt);
                        const int tok = u.c0 + u.tok0 + t * p.tile1_token, hq = u.h * G + t * p.tile1_head;
                        tma_load_3d(sm.q[t], &map_q, 0, hq, tok, &sm.q_full[t]);
                        tma_load_3d(sm.q[t] + kTileBytes / 2, &map_q, 64, hq, tok, &sm.q_full[t]);
                        uses[t]++;
                    }
                }
                ok = __all_sync(kFull, ok);
#pragma unroll 1
                for (int i = 0; i < sp.total && ok; i++) {
                    ring.next();
                    if (i >= sp.mixed) {
                        ok = __all_sync(kFull, mbar_wait_short(&sm.kv_raw[ring.stage], raw_phase >> ring.stage & 1u));
                        if (!ok) break;
                        raw_phase ^= 1u << ring.stage;
                        const int left = u.n - i * kKeys;  // keys of the step inside the sequence
                        uint4 *piece = reinterpret_cast<uint4 *>(sm.kv[ring.stage]);
                        auto key_of = [](int e) { return (e & 1023) >> 3; };  // 8 pieces a key, two halves of the elements
                        if (left < kKeys) {
#pragma unroll 1
                            for (int e = lane; e < kTileBytes / 16; e += 32)
                                if (key_of(e) >= left) piece[e] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        uint32_t top[2] = {0u, 0u};
#pragma unroll 8
                        for (int e = lane; e < kTileBytes / 16; e += 32) {
                            const uint4 x = piece[e];
                            top[0] = E::larger(E::larger(top[0], x.x), x.y);
                            top[1] = E::larger(E::larger(top[1], x.z), x.w);
                        }
                        const uint32_t odd = E::wild(top[0]) | E::wild(top[1]);
                        if (odd) {
                            uint32_t *word = reinterpret_cast<uint32_t *>(piece);
#pragma unroll 1
                            for (int e = lane; e < kTileBytes / 16; e += 32)
#pragma unroll 1
                                for (int c = 0; c < 4; c++) {
                                    const uint32_t m = E::wild(word[4 * e + c]);
                                    if (m & 0x8000u) word[4 * e + c] &= 0xFFFF0000u;
                                    if (m & 0x80000000u) word[4 * e + c] &= 0x0000FFFFu;
                                }
                        }
                        fence_proxy_async_smem();
                        const bool any = __any_sync(kFull, odd != 0);
                        if (lane == 0) {
                            if (any) sm.wild[r & 3] = 1u;
                            mbar_arrive(&sm.kv_clean[ring.stage]);
                        }
                    }
                    ring.next();
                }
            }
            if (lane == 0)
                for (int t = 0; t < kUnitTiles; t++)  // no copy in flight when the CTA ends
                    if (uses[t] > 0 && !mbar_wait_short(&sm.q_full[t], (uses[t] - 1) & 1u)) ok = false;
        }
    }
    __syncwarp();
    if (!ok) set_flag(p.status, KVQ_FLAG_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPromptTmem));
}

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// rows of [heads][128] 16-bit elements, `stride` elements apart: boxes of 64 elements x `box_heads` x `box_rows`,
// 128-byte swizzled (rows past the tensor read as zero)
bool make_map(CUtensorMap *m, bool bf, const uint16_t *x, int64_t rows, int heads, int64_t stride, int box_heads,
              int box_rows)
{
    const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {kHeadDim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, one[3] = {1, 1, 1};
    return encode_tiled()(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                          const_cast<uint16_t *>(x), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF>
cudaError_t launch_prompt_type(const PromptParams &p, const uint16_t *q, int64_t q_stride, const uint16_t *k,
                               int64_t k_stride, int num_sms, cudaStream_t s)
{
    CUtensorMap mq, mk, mv;
    if (!encode_tiled()) return cudaErrorNotSupported;
    if (!make_map(&mq, BF, q, p.total, p.num_q_heads, q_stride, p.tile_heads, p.tile_tokens) ||
        !make_map(&mk, BF, k, p.total, p.num_heads, k_stride, 1, kKeys) ||
        !make_map(&mv, BF, p.v, p.total, p.num_heads, p.v_stride, 1, kKeys))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done[2] = {0, 0};
    auto kernel = p.score_scale < 0.0f ? prompt_attn_kernel<BF, true> : prompt_attn_kernel<BF, false>;
    const cudaError_t e = allow_smem(kernel, sizeof(PromptSmem), done[p.score_scale < 0.0f]);
    if (e != cudaSuccess) return e;
    // a CTA for every unit there can be, up to 32 per SM (then a ticket is several units): the first
    // ones to run take the others' places
    const int64_t ut = p.unit_tokens;
    const int64_t by_max = (int64_t)p.num_seqs * ((p.max_n + ut - 1) / ut), by_total = p.total / ut + p.num_seqs;
    const int64_t units = (by_max < by_total ? by_max : by_total) * p.num_heads;
    const int64_t most = 16 * (int64_t)num_sms, grid = units < most ? units : most;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kPromptThreads), sizeof(PromptSmem), s, p,
                        mq, mk, mv);
}

}  // namespace

cudaError_t launch_prompt(int dtype, const PromptParams &p, const uint16_t *q, int64_t q_stride, const uint16_t *k,
                          int64_t k_stride, int num_sms, cudaStream_t s)
{
    return dtype == KVQ_BF16 ? launch_prompt_type<true>(p, q, q_stride, k, k_stride, num_sms, s)
                             : launch_prompt_type<false>(p, q, q_stride, k, k_stride, num_sms, s);
}

}  // namespace kvq
