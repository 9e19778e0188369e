// kvq_weights.cu -- the softmax weight that each page of the quantized paged
// cache receives from the newest queries of its sequence (what eviction by
// accumulated attention weight goes by; the cache and its pages as for decode:
// quantize_block, jsqmd.com/news/887038 section 2.1, and PagedAttention, ddd.cn
// section 4).
//
//   W[b][j] = decay * W_in[b][j] + sum_{i, hq} sum_{t in page j, t <= p_i} softmax_t(scale q_i,hq . k^_t)
//
// Only the keys are read.  With s in base 2 and S(row, j) = log2 sum_{t in page j} 2^s_t,
//   softmax mass of page j = 2^(S(row, j) - log2 sum_j' 2^S(row, j')),
// so one pass over the codes that keeps a single number per (query row, page)
// is enough:
//   page_lse_kernel   one warp per page of 64 keys of one cache head: the codes
//                     go straight into registers, are widened exactly to fp16
//                     and multiplied with the query rows as the 8-column
//                     operand of mma.sync (query rows of the group and of the
//                     chunk share a page's widening); a page's row maximum and
//                     sum stay in registers, S goes to the workspace.
//   page_sum_kernel   rows of one sequence: log2-sum over the pages, then the
//                     page masses summed over the rows in a fixed order (no
//                     atomics: equal inputs give equal bits).
//   page_join_kernel  adds the row chunks of long windows.
#include "kvq_around.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kPwWarps = 8;
constexpr int kSumThreads = 256;

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

// int4 codes widened exactly to fp16 subnormals, one lop3 per pair: an even element (low
// nibble n of its byte, c the signed code) becomes (c + 8) * 2^-24, an odd one
// (7 - c) * 2^-20; q's odd elements enter as -q / 16, so a raw score is
// 2^-24 (q . c + 8 sum_even q - 7 sum_odd q), and the sums come out afterwards.
struct Nibbles {
    uint32_t m_lo, m_hi, x_lo, x_hi;
    __device__ __forceinline__ Nibbles() : m_lo(0x000f000fu), m_hi(0x00f000f0u), x_lo(0x00080008u), x_hi(0x00700070u)
    {
        // held in registers, so that (x & m) ^ c is one instruction
        asm volatile("" : "+r"(m_lo), "+r"(m_hi), "+r"(x_lo), "+r"(x_hi));
    }
    __device__ __forceinline__ uint32_t lo(uint32_t x) const { return (x & m_lo) ^ x_lo; }
    __device__ __forceinline__ uint32_t hi(uint32_t x) const { return (x & m_hi) ^ x_hi; }
};

}  // namespace

// A chunk is 4 KiB of codes: 64 keys (int4, a page) or 32 keys (int8, FP8, half a page) =
// kTiles tiles of 16.  Lane (g, t) = (lane / 4, lane % 4) holds rows g and g + 8 of each
// tile, of each row the 16-byte pieces that the k index of the MMA is permuted for: a
// warp's load covers whole 64-byte runs of 8 rows.
template <int FMT>
struct PwFmt {
    static constexpr int kRowBytes = FMT == KVQ_INT4_B64 ? 64 : 128;
    static constexpr int kPieces = kRowBytes / 64;  // 16-byte pieces of a row per lane
    static constexpr int kTiles = 4 / kPieces;      // 16-key tiles per chunk
    static constexpr int kChunks = kPieces;         // chunks per page
};

template <int FMT, int NT>
__global__ void __launch_bounds__(kPwWarps * 32) page_lse_kernel(PageWeightsParams p)
{
    using F = PwFmt<FMT>;
    constexpr int kCols = 8 * NT;  // query rows per unit
    __shared__ int64_t upto[kMaxSeqsPerLaunch + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int H = p.num_heads, G = p.group;
    // units of sequence b: (cache head, block of kCols query rows, page), the page fastest
    if (warp == 0) {
        int64_t run = 0;
        for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
            int64_t u = 0;
            if (b0 + lane < p.num_seqs) {
                PwSeq s;
                if (pw_seq(p, b0 + lane, s))
                    u = (int64_t)((s.L + kPage - 1) / kPage) * H * (((int64_t)s.n * G + kCols - 1) / kCols);
                else if (blockIdx.x == 0)
                    set_flag(p.status, KVQ_FLAG_BAD_LENGTH);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(kFull, u, o);
                if (lane >= o) u += v;
            }
            if (b0 + lane < p.num_seqs) upto[b0 + lane + 1] = run + u;
            run += __shfl_sync(kFull, u, 31);
        }
        if (lane == 0) upto[0] = 0;
    }
    __syncthreads();
    const int64_t U = upto[p.num_seqs];
    const int64_t warps = (int64_t)gridDim.x * kPwWarps, id = (int64_t)warp * gridDim.x + blockIdx.x;
    int64_t u = U * id / warps;
    const int64_t end = U * (id + 1) / warps;
    const Nibbles nib;

    while (u < end) {
        // ---- one segment: pages [j0, j1) of one (sequence, cache head, row block) ----
        int lo = 0, hi = p.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (upto[mid] <= u)
                lo = mid;
            else
                hi = mid;
        }
        const int b = lo;
        PwSeq s;
        pw_seq(p, b, s);
        const int np = (s.L + kPage - 1) / kPage;
        const int rows = s.n * G, blocks = (rows + kCols - 1) / kCols;
        const int64_t r = u - upto[b];
        const int j0 = (int)(r % np);
        const int64_t hr = r / np;
        const int h = (int)(hr / blocks), row0 = (int)(hr % blocks) * kCols;
        const int j1 = (int)min((int64_t)np, j0 + (end - u));
        u += j1 - j0;
        const int32_t *bt = p.block_table + (int64_t)b * p.max_blocks;

        // the unit's query rows as the B operand: column g of tile nt is row row0 + 8 nt + g
        uint32_t qb[NT][8][2];
        float bias[NT][2];  // columns 2t, 2t + 1: minus the offset share of every raw score (int4)
        float *dst[NT][2];  // their rows of the workspace
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const int rr = row0 + 8 * nt + g;
            const bool live = rr < rows;
            const uint16_t *q = p.q + ((int64_t)(s.c0 + rr / G) * p.num_q_heads + h * G + rr % G) * kHeadDim;
            uint4 v[4];
            float off = 0.0f;
#pragma unroll
            for (int m = 0; m < 4; m++) {
                v[m] = make_uint4(0u, 0u, 0u, 0u);
                if (!live) continue;
                if constexpr (FMT == KVQ_INT4_B64)
                    v[m] = *reinterpret_cast<const uint4 *>(q + 32 * t + 8 * m);
                else
                    v[m] = *reinterpret_cast<const uint4 *>(q + 64 * (m >> 1) + 16 * t + 8 * (m & 1));
            }
            if constexpr (FMT == KVQ_INT4_B64) {
                const __half2 odd = __float2half2_rn(-0.0625f);
#pragma unroll
                for (int m = 0; m < 4; m++) {  // a word's 8 elements as pairs (0,4) (1,5) (2,6) (3,7)
                    const uint32_t e04 = __byte_perm(v[m].x, v[m].z, 0x5410), e15 = __byte_perm(v[m].x, v[m].z, 0x7632);
                    const uint32_t e26 = __byte_perm(v[m].y, v[m].w, 0x5410), e37 = __byte_perm(v[m].y, v[m].w, 0x7632);
                    const __half2 o15 = __hmul2(*reinterpret_cast<const __half2 *>(&e15), odd);
                    const __half2 o37 = __hmul2(*reinterpret_cast<const __half2 *>(&e37), odd);
                    qb[nt][2 * m][0] = e04;
                    qb[nt][2 * m][1] = h2_bits(o15);
                    qb[nt][2 * m + 1][0] = e26;
                    qb[nt][2 * m + 1][1] = h2_bits(o37);
                    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&e04));
                    const float2 c = __half22float2(*reinterpret_cast<const __half2 *>(&e26));
                    const float2 x = __half22float2(o15), y = __half22float2(o37);
                    off += 8.0f * ((a.x + a.y) + (c.x + c.y)) + 112.0f * ((x.x + x.y) + (y.x + y.y));
                }
                off += __shfl_xor_sync(kFull, off, 1);  // the four lanes t hold the row's four slices
                off += __shfl_xor_sync(kFull, off, 2);
            } else {
#pragma unroll
                for (int m = 0; m < 4; m++) {
                    qb[nt][2 * m][0] = v[m].x;
                    qb[nt][2 * m][1] = v[m].y;
                    qb[nt][2 * m + 1][0] = v[m].z;
                    qb[nt][2 * m + 1][1] = v[m].w;
                }
            }
#pragma unroll
            for (int e = 0; e < 2; e++) {
                bias[nt][e] = -__shfl_sync(kFull, off, (2 * t + e) * 4);
                const int rc = row0 + 8 * nt + 2 * t + e;
                dst[nt][e] = rc < rows ? p.lse + ((int64_t)(s.c0 + rc / G) * p.num_q_heads + h * G + rc % G) *
                                                     p.max_blocks
                                       : nullptr;
            }
        }

        // page ids and key scales of 32 pages at a time, lane l those of page ring0 + l
        int ring0 = j0, pg = 0;
        float sk = 0.0f;
        auto ring = [&](int j) {
            ring0 = j;
            if (j + lane < j1) {
                pg = bt[j + lane];
                if (pg < 0 || pg >= p.num_pages) {
                    set_flag(p.status, KVQ_FLAG_BAD_PAGE);
                    pg = 0;
                }
                sk = p.k_scales[(int64_t)pg * H + h];
            }
        };
        // chunk x of the page whose ring lane is l
        auto load = [&](int page, int x, uint4 (&d)[8]) {
            const uint8_t *base = p.k_codes + ((size_t)page * H + h) * (kPage * F::kRowBytes) + 4096 * x +
                                  g * F::kRowBytes + 16 * t;
#pragma unroll
            for (int i = 0; i < 8; i++) {  // (tile, row half, piece)
                const int tile = i / (2 * F::kPieces), half = i / F::kPieces % 2, piece = i % F::kPieces;
                d[i] = ld_stream_v4(base + (16 * tile + 8 * half) * F::kRowBytes + 64 * piece);
            }
        };
        ring(j0);
        uint4 cur[8];
        load(__shfl_sync(kFull, pg, 0), 0, cur);
        for (int j = j0; j < j1; j++) {
            float acc[4][NT][4];
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[i][nt][e] = 0.0f;
            const int page = __shfl_sync(kFull, pg, j - ring0);
            const float fac = __shfl_sync(kFull, sk, j - ring0) * p.score_scale;
#pragma unroll
            for (int x = 0; x < F::kChunks; x++) {
                uint4 c[8];
#pragma unroll
                for (int i = 0; i < 8; i++) c[i] = cur[i];
                if (x + 1 < F::kChunks) {
                    load(page, x + 1, cur);
                } else if (j + 1 < j1) {
                    if (j + 1 - ring0 == 32) ring(j + 1);
                    load(__shfl_sync(kFull, pg, j + 1 - ring0), 0, cur);
                }
#pragma unroll
                for (int ks = 0; ks < 4; ks++) {
#pragma unroll
                    for (int tile = 0; tile < F::kTiles; tile++) {
                        float(&a)[NT][4] = acc[x * F::kTiles + tile];
#pragma unroll
                        for (int pc = 0; pc < F::kPieces; pc++) {
                            const uint4 &wa = c[tile * 2 * F::kPieces + pc];
                            const uint4 &wb = c[tile * 2 * F::kPieces + F::kPieces + pc];
                            const uint32_t ua = ks == 0 ? wa.x : ks == 1 ? wa.y : ks == 2 ? wa.z : wa.w;
                            const uint32_t ub = ks == 0 ? wb.x : ks == 1 ? wb.y : ks == 2 ? wb.z : wb.w;
                            if constexpr (FMT == KVQ_INT4_B64) {
                                const uint32_t ah = ua >> 8, bh = ub >> 8;
#pragma unroll
                                for (int nt = 0; nt < NT; nt++) {
                                    mma16816(a[nt], nib.lo(ua), nib.lo(ub), nib.hi(ua), nib.hi(ub),
                                             qb[nt][2 * ks][0], qb[nt][2 * ks][1]);
                                    mma16816(a[nt], nib.lo(ah), nib.lo(bh), nib.hi(ah), nib.hi(bh),
                                             qb[nt][2 * ks + 1][0], qb[nt][2 * ks + 1][1]);
                                }
                            } else {
                                __half2 ra[2], rb[2];
                                if constexpr (FMT == KVQ_FP8_E4M3) {
                                    widen_e4m3(ua, ra);
                                    widen_e4m3(ub, rb);
                                } else {
                                    widen_int8(ua, ra);
                                    widen_int8(ub, rb);
                                }
#pragma unroll
                                for (int nt = 0; nt < NT; nt++)
                                    mma16816(a[nt], h2_bits(ra[0]), h2_bits(rb[0]), h2_bits(ra[1]), h2_bits(rb[1]),
                                             qb[nt][4 * pc + ks][0], qb[nt][4 * pc + ks][1]);
                            }
                        }
                    }
                }
            }
            // log2-sum of the page per query row; lanes (0..7, t) hold the rows 2t, 2t + 1 of a tile
            const int k0 = j * kPage;
            const bool cut = k0 + kPage - 1 > s.L - s.n;  // keys past some row's position
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float v[8], m = -INFINITY;
                    const int pos = s.L - s.n + (row0 + 8 * nt + 2 * t + e) / G;
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float raw = acc[i >> 1][nt][2 * (i & 1) + e];
                        v[i] = FMT == KVQ_INT4_B64 ? fmaf(raw, fac * 16777216.0f, bias[nt][e] * fac) : raw * fac;
                        if (cut && k0 + 16 * (i >> 1) + 8 * (i & 1) + g > pos) v[i] = -INFINITY;
                        m = fmaxf(m, v[i]);
                    }
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                    const float ref = m == -INFINITY ? 0.0f : m;
                    float l = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; i++) l += ex2_approx(v[i] - ref);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(kFull, l, o);
                    if (g == 0 && dst[nt][e]) dst[nt][e][j] = m == -INFINITY ? m : m + __log2f(l);
                }
        }
    }
}

// Rows [64 c, 64 c + 64) of sequence b (query rows, tokens x heads): the rows' log2-sums over
// the pages, then each page's mass over these rows, to the output (one chunk) or to `part`.
__global__ void __launch_bounds__(kSumThreads) page_sum_kernel(PageWeightsParams p)
{
    __shared__ float total[kPwSumRows];
    const int b = blockIdx.y, c = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    PwSeq s;
    if (!pw_seq(p, b, s)) return;
    const int np = (s.L + kPage - 1) / kPage, mb = p.max_blocks;
    const int64_t rows = (int64_t)s.n * p.num_q_heads, r0 = (int64_t)c * kPwSumRows;
    const float *in = p.weights_in ? p.weights_in + (int64_t)b * mb : nullptr;
    float *out = p.weights_out + (int64_t)b * mb;
    if (rows == 0) {  // no new row: the weights stay
        if (c == 0)
            for (int j = tid; j < mb; j += kSumThreads) out[j] = in && j < np ? in[j] : 0.0f;
        return;
    }
    if (r0 >= rows) return;
    const int nr = (int)min((int64_t)kPwSumRows, rows - r0);
    const float *lse = p.lse + ((int64_t)s.c0 * p.num_q_heads + r0) * mb;
    for (int r = warp; r < nr; r += kSumThreads / 32) {
        const float *x = lse + (int64_t)r * mb;
        float m = -INFINITY;
        for (int j = lane; j < np; j += 32) m = fmaxf(m, x[j]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        float l = 0.0f;
        for (int j = lane; j < np; j += 32) l += ex2_approx(x[j] - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
        if (lane == 0) total[r] = m + __log2f(l);
    }
    __syncthreads();
    const bool last = rows <= kPwSumRows;  // the sequence's only chunk
    const int per_token = (p.num_q_heads + kPwSumRows - 1) / kPwSumRows;
    float *part = p.part + ((int64_t)s.c0 * per_token + c) * mb;
    for (int j = tid; j < (last ? mb : np); j += kSumThreads) {
        float a = 0.0f;
        if (j < np) {
#pragma unroll 8
            for (int r = 0; r < nr; r++) a += ex2_approx(lse[(int64_t)r * mb + j] - total[r]);
        }
        if (!last)
            part[j] = a;
        else
            out[j] = j < np ? fmaf(p.decay, in ? in[j] : 0.0f, a) : 0.0f;
    }
}

__global__ void __launch_bounds__(kSumThreads) page_join_kernel(PageWeightsParams p)
{
    const int b = blockIdx.y, j = blockIdx.x * kSumThreads + threadIdx.x, mb = p.max_blocks;
    PwSeq s;
    if (!pw_seq(p, b, s) || j >= mb) return;
    const int64_t rows = (int64_t)s.n * p.num_q_heads;
    if (rows <= kPwSumRows) return;
    const int np = (s.L + kPage - 1) / kPage;
    const int chunks = (int)((rows + kPwSumRows - 1) / kPwSumRows);
    const int per_token = (p.num_q_heads + kPwSumRows - 1) / kPwSumRows;
    const float *part = p.part + (int64_t)s.c0 * per_token * mb;
    const int64_t at = (int64_t)b * mb + j;
    float a = 0.0f;
    if (j < np) {
#pragma unroll 8
        for (int c = 0; c < chunks; c++) a += part[(int64_t)c * mb + j];
        a = fmaf(p.decay, p.weights_in ? p.weights_in[at] : 0.0f, a);
    }
    p.weights_out[at] = a;
}

template <int FMT, int NT>
static cudaError_t launch_page_lse(const PageWeightsParams &p, int num_sms, cudaStream_t s)
{
    int ctas = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, page_lse_kernel<FMT, NT>, kPwWarps * 32, 0);
    if (e != cudaSuccess) return e;
    return launch_plain(page_lse_kernel<FMT, NT>, dim3((unsigned)(num_sms * ctas)), dim3(kPwWarps * 32), 0, s, p);
}

template <int FMT>
static cudaError_t launch_page_weights_fmt(const PageWeightsParams &p, int num_sms, cudaStream_t s)
{
    const int64_t rows = (int64_t)p.max_q * p.group;  // query rows of one cache head
    if (rows <= 8) return launch_page_lse<FMT, 1>(p, num_sms, s);
    if (rows <= 16) return launch_page_lse<FMT, 2>(p, num_sms, s);
    return launch_page_lse<FMT, 4>(p, num_sms, s);
}

size_t page_weights_lse_floats(int64_t total_q, int num_q_heads, int max_blocks)
{
    return (size_t)total_q * num_q_heads * max_blocks;
}

size_t page_weights_workspace_bytes(int64_t total_q, int num_q_heads, int max_blocks)
{
    const size_t part = (size_t)total_q * ((num_q_heads + kPwSumRows - 1) / kPwSumRows) * max_blocks;
    return (page_weights_lse_floats(total_q, num_q_heads, max_blocks) + part) * sizeof(float);
}

cudaError_t launch_page_weights(int fmt, const PageWeightsParams &p, int num_sms, cudaStream_t s)
{
    cudaError_t e = fmt == KVQ_INT4_B64   ? launch_page_weights_fmt<KVQ_INT4_B64>(p, num_sms, s)
                    : fmt == KVQ_FP8_E4M3 ? launch_page_weights_fmt<KVQ_FP8_E4M3>(p, num_sms, s)
                                          : launch_page_weights_fmt<KVQ_INT8_PAGE>(p, num_sms, s);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)p.max_q * p.num_q_heads;
    const int64_t chunks = rows == 0 ? 1 : (rows + kPwSumRows - 1) / kPwSumRows;
    e = launch_plain(page_sum_kernel, dim3((unsigned)chunks, (unsigned)p.num_seqs), dim3(kSumThreads), 0, s, p);
    if (e != cudaSuccess || chunks == 1) return e;
    return launch_plain(page_join_kernel, dim3((unsigned)((p.max_blocks + kSumThreads - 1) / kSumThreads),
                                               (unsigned)p.num_seqs),
                        dim3(kSumThreads), 0, s, p);
}

}  // namespace kvq
