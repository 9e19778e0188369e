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
//                     come by bulk copies, are widened exactly to fp16 in
//                     registers and multiplied with the query rows as the
//                     8-column operand of mma.sync (query rows of the group and
//                     of the chunk share a page's widening); a page's row
//                     maximum and sum stay in registers, S goes to the workspace.
//   page_sum_kernel   rows of one sequence: log2-sum over the pages, then the
//                     page masses summed over the rows in a fixed order (no
//                     atomics: equal inputs give equal bits).
//   page_join_kernel  adds the row chunks of long windows.
//
// Bound by HBM: 64 (int4) or 128 bytes per cached key and head.  Measured: 16 x
// 32K tokens x 32 heads int4 (1.04 GB) 168 us, 0.92 of the measured copy rate;
// 32 x 8K x 8 heads FP8 with 8 query heads each (250 MB) 45 us, 0.83; 8 x 8193 x
// 32 heads int4 (134 MB) 30 us, 0.67 -- a launch begins and ends in about 8 us --
// plus 2 - 4 us of page_sum_kernel (8 us, with page_join_kernel, for the 1024 rows of a
// window of 32 tokens).  The log2-sums lie [page][row]: a row sum reads 256 bytes of 64
// rows at once and the writers of a tile of rows lie side by side (laid out [row][page],
// windows of 32 tokens took 46 us against 38).  16 warps with a ring of three 4 KB copies
// each: 12 warps with four 57 us on 268 MB against 51, 18 with three 57.
#include "kvq_weights.cuh"

namespace kvq {

namespace {

constexpr int kPwWarps = 16;
constexpr int kPwStages = 3;
constexpr int kPwChunk = 4096;
constexpr int kSumThreads = 512;

// int4 codes widened exactly to fp16 subnormals, one lop3 per pair: an even element (low
// nibble n of its byte, c the signed code) becomes (c + 8) * 2^-24, an odd one
// (7 - c) * 2^-20; q's odd elements enter as -q / 16, so a raw score is
// 2^-24 (q . c + 8 sum_even q - 7 sum_odd q), and the sums come out afterwards.
struct Nibbles {
    uint32_t m_lo, m_hi, x_lo, x_hi;
    __device__ __forceinline__ Nibbles() : m_lo(0x000f000fu), m_hi(0x00f000f0u), x_lo(0x00080008u), x_hi(0x00700070u)
    {
        // held in registers: an instruction takes one immediate
        asm volatile("" : "+r"(m_lo), "+r"(m_hi), "+r"(x_lo), "+r"(x_hi));
    }
    // (x & m) ^ c as one lop3 (written as C, it became two: 531 -> 403 warp instructions a page)
    static __device__ __forceinline__ uint32_t flip(uint32_t x, uint32_t m, uint32_t c)
    {
        uint32_t d;
        asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(x), "r"(m), "r"(c));
        return d;
    }
    __device__ __forceinline__ uint32_t lo(uint32_t x) const { return flip(x, m_lo, x_lo); }
    __device__ __forceinline__ uint32_t hi(uint32_t x) const { return flip(x, m_hi, x_hi); }
};

}  // namespace

// A chunk is 4 KiB of codes: 64 keys (int4, a page) or 32 keys (int8, FP8, half a page) =
// kTiles tiles of 16.  Lane (g, t) = (lane / 4, lane % 4) reads of rows g and g + 8 of each
// tile the 16-byte pieces that the k index of the MMA is permuted for.
template <int FMT>
struct PwFmt {
    static constexpr int kRowBytes = FMT == KVQ_INT4_B64 ? 64 : 128;
    static constexpr int kPieces = kRowBytes / 64;  // 16-byte pieces of a row per lane
    static constexpr int kTiles = 4 / kPieces;      // 16-key tiles per chunk
    static constexpr int kChunks = kPieces;         // chunks per page
};

// D = A * B, m16n8k16, fp16 operands, fp32 result (no accumulator to clear first)
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

struct PwSmem {
    uint8_t ring[kPwWarps][kPwStages][kPwChunk];
    uint64_t full[kPwWarps][kPwStages];
    int64_t upto[kMaxSeqsPerLaunch + 1];
};

// Up to 8 NT query rows of one cache head.  A persistent warp owns a contiguous range of units
// (pages, the fastest index) and streams their chunks through its own ring of bulk copies.
template <int FMT, int NT>
__global__ void __launch_bounds__(kPwWarps * 32, 1) page_lse_kernel(PageWeightsParams p)
{
    using F = PwFmt<FMT>;
    constexpr int kCols = 8 * NT;  // query rows per unit
    extern __shared__ __align__(128) uint8_t smem_pw[];
    PwSmem &sm = *reinterpret_cast<PwSmem *>(smem_pw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int H = p.num_heads, G = p.group;
    pdl_launch_dependents();
    if (lane < kPwStages) mbar_init(&sm.full[warp][lane], 1);
    mbar_init_fence();
    // units of sequence b: (cache head, block of kCols query rows, page), the page fastest
    bool bad_seq = false, bad_page = false;
    if (warp == 0) {
        int64_t run = 0;
        for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
            int64_t u = 0;
            if (b0 + lane < p.num_seqs) {
                PwSeq s;
                if (pw_seq(p, b0 + lane, s))
                    u = (int64_t)((s.L + kPage - 1) / kPage) * H * (((int64_t)s.n * G + kCols - 1) / kCols);
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
    __syncthreads();
    const int64_t U = sm.upto[p.num_seqs];
    const int64_t warps = (int64_t)gridDim.x * kPwWarps, id = (int64_t)warp * gridDim.x + blockIdx.x;
    const int64_t first = U * id / warps;
    const int units = (int)(U * (id + 1) / warps - first);
    const Nibbles nib;

    // the place of unit u: its sequence (and what it brings), (head, row block) and page
    struct Place {
        PwSeq s;
        int b, h, row0, j;
    };
    auto place = [&](int64_t u) {
        Place x;
        int lo = 0, hi = p.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm.upto[mid] <= u)
                lo = mid;
            else
                hi = mid;
        }
        x.b = lo;
        pw_seq(p, lo, x.s);
        const int np = (x.s.L + kPage - 1) / kPage, blocks = (x.s.n * G + kCols - 1) / kCols;
        const uint32_t r = (uint32_t)(u - sm.upto[lo]), hr = r / (uint32_t)np;  // (under 2^31 of one sequence)
        x.j = (int)(r - hr * (uint32_t)np);
        x.h = (int)(hr / (uint32_t)blocks);
        x.row0 = (int)(hr % (uint32_t)blocks) * kCols;
        return x;
    };

    // the warp's next 64 units by lane, in two rings of 32 (one is loaded while the other is
    // used): (page, head) of the codes, key scale, page number
    uint32_t ph[2] = {0u, 0u};
    float sk[2] = {0.0f, 0.0f};
    int pj[2] = {0, 0};
    auto look = [&](int i, uint32_t &ph_, int &pj_) {
        if (i + lane >= units) return;
        const Place x = place(first + i + lane);
        int pg = p.block_table[(int64_t)x.b * p.max_blocks + x.j];
        if (pg < 0 || pg >= p.num_pages) {
            bad_page = true;
            pg = 0;
        }
        ph_ = (uint32_t)pg * (uint32_t)H + (uint32_t)x.h;
        pj_ = x.j;
    };
    auto scales = [&](int i, uint32_t ph_, float &sk_) {
        if (i + lane < units) sk_ = p.k_scales[ph_];
    };
    look(0, ph[0], pj[0]);
    pdl_wait();  // (the lengths and the block table are read before it, everything else after)
    if (bad_seq && blockIdx.x == 0) set_flag(p.status, KVQ_FLAG_BAD_LENGTH);
    const int chunks = units * F::kChunks;
    uint8_t *ring = sm.ring[warp][0];
    uint64_t *full = sm.full[warp];
    // bring chunk c into its stage (the ring that holds its unit is picked by a branch: a select
    // would wait for the other ring's loads)
    auto bring = [&](int c) {
        if (c >= chunks) return;
        const int i = c / F::kChunks, x = c % F::kChunks;
        const uint32_t at = i & 32 ? __shfl_sync(kFull, ph[1], i & 31) : __shfl_sync(kFull, ph[0], i & 31);
        if (lane == 0) {
            const int st = c % kPwStages;
            mbar_arrive_expect_tx(&full[st], kPwChunk);
            bulk_copy_g2s(ring + st * kPwChunk,
                          p.k_codes + (size_t)at * (kPage * F::kRowBytes) + (size_t)x * kPwChunk, kPwChunk, &full[st]);
        }
    };
    __syncwarp();
    for (int c = 0; c < kPwStages; c++) bring(c);
    scales(0, ph[0], sk[0]);
    look(32, ph[1], pj[1]);
    scales(32, ph[1], sk[1]);

    uint32_t qb[NT][8][2];       // the unit's query rows as the B operand: column g of tile nt is row row0 + 8 nt + g
    int pos[NT][2], pos0 = 0;    // columns 2t, 2t + 1: their positions; the least position of the chunk
    // of column 2t + g % 2, whose sums this lane ends up with:
    float bias[NT];              // minus the offset share of every raw score (int4)
    float *dst[NT];              // its place in the workspace; the next page's is row_step on
    uint32_t writes = 0;         // bit nt: a lane that writes one
    int64_t row_step = 0;
    const float sign = p.score_scale < 0.0f ? -1.0f : 1.0f;
    const float sabs = fmaxf(fabsf(p.score_scale), kPwMinScale);
    bool ok = true;
    int c = 0, st = 0;
    uint32_t phase = 0;
    for (int i = 0; i < units; i++) {
        if (i > 0 && (i & 31) == 0) {  // this ring's turn: the other looks 32 units ahead of it
            if (i & 32) {
                look(i + 32, ph[0], pj[0]);
                scales(i + 32, ph[0], sk[0]);
            } else {
                look(i + 32, ph[1], pj[1]);
                scales(i + 32, ph[1], sk[1]);
            }
        }
        float fac;
        int j;
        if (i & 32) {
            fac = __shfl_sync(kFull, sk[1], i & 31);
            j = __shfl_sync(kFull, pj[1], i & 31);
        } else {
            fac = __shfl_sync(kFull, sk[0], i & 31);
            j = __shfl_sync(kFull, pj[0], i & 31);
        }
        fac = fmaxf(fac * sabs, kPwMinScale);
        if (i == 0 || j == 0) {  // another (sequence, head, row block)
            const Place x = place(first + i);
            const int rows = x.s.n * G;
            pos0 = x.s.L - x.s.n;
            row_step = (int64_t)x.s.n * p.num_q_heads;
            writes = 0;
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const int rr = x.row0 + 8 * nt + g;
                const bool live = rr < rows;
                const uint16_t *q = p.q + ((int64_t)(x.s.c0 + rr / G) * p.num_q_heads + x.h * G + rr % G) * kHeadDim;
                const __half2 flip = __float2half2_rn(sign);
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
                    uint32_t *w = reinterpret_cast<uint32_t *>(&v[m]);
#pragma unroll
                    for (int e = 0; e < 4; e++) w[e] = h2_bits(__hmul2(*reinterpret_cast<__half2 *>(&w[e]), flip));
                }
                if constexpr (FMT == KVQ_INT4_B64) {
                    const __half2 odd = __float2half2_rn(-0.0625f);
#pragma unroll
                    for (int m = 0; m < 4; m++) {  // a word's 8 elements as pairs (0,4) (1,5) (2,6) (3,7)
                        const uint32_t e04 = __byte_perm(v[m].x, v[m].z, 0x5410);
                        const uint32_t e15 = __byte_perm(v[m].x, v[m].z, 0x7632);
                        const uint32_t e26 = __byte_perm(v[m].y, v[m].w, 0x5410);
                        const uint32_t e37 = __byte_perm(v[m].y, v[m].w, 0x7632);
                        const __half2 o15 = __hmul2(*reinterpret_cast<const __half2 *>(&e15), odd);
                        const __half2 o37 = __hmul2(*reinterpret_cast<const __half2 *>(&e37), odd);
                        qb[nt][2 * m][0] = e04;
                        qb[nt][2 * m][1] = h2_bits(o15);
                        qb[nt][2 * m + 1][0] = e26;
                        qb[nt][2 * m + 1][1] = h2_bits(o37);
                        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&e04));
                        const float2 d = __half22float2(*reinterpret_cast<const __half2 *>(&e26));
                        const float2 e = __half22float2(o15), y = __half22float2(o37);
                        off += 8.0f * ((a.x + a.y) + (d.x + d.y)) + 112.0f * ((e.x + e.y) + (y.x + y.y));
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
                const int rc = x.row0 + 8 * nt + 2 * t;
                bias[nt] = -__shfl_sync(kFull, off, (2 * t + (g & 1)) * 4);
                dst[nt] = pw_sums(p, x.s) + j * row_step + (int64_t)x.h * rows + rc + (g & 1);
                writes |= (uint32_t)(g < 2 && rc + (g & 1) < rows) << nt;
                pos[nt][0] = pos0 + rc / G;
                pos[nt][1] = pos0 + (rc + 1) / G;
            }
        }

        // raw scores of the page: acc[tile][nt] = rows g, g + 8 of the tile x columns 2t, 2t + 1
        float acc[4][NT][4];
#pragma unroll
        for (int x = 0; x < F::kChunks; x++, c++) {
            if (!mbar_wait_bounded(&full[st], phase)) ok = false;
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            const uint32_t base = smem_addr(ring) + st * kPwChunk + g * F::kRowBytes + 16 * t;
            uint4 w[8];
#pragma unroll
            for (int k = 0; k < 8; k++) {  // (tile, row half, piece)
                const int tile = k / (2 * F::kPieces), half = k / F::kPieces % 2, piece = k % F::kPieces;
                w[k] = lds128(base + (16 * tile + 8 * half) * F::kRowBytes + 64 * piece);
            }
            if (++st == kPwStages) {
                st = 0;
                phase ^= 1u;
            }
            __syncwarp();
            if (lane == 0) fence_proxy_async_smem();
            bring(c + kPwStages);
#pragma unroll
            for (int pc = 0; pc < F::kPieces; pc++)
#pragma unroll
                for (int ks = 0; ks < 4; ks++)
#pragma unroll
                    for (int tile = 0; tile < F::kTiles; tile++) {
                        float(&a)[NT][4] = acc[x * F::kTiles + tile];
                        const uint4 &wa = w[tile * 2 * F::kPieces + pc];
                        const uint4 &wb = w[tile * 2 * F::kPieces + F::kPieces + pc];
                        const uint32_t ua = ks == 0 ? wa.x : ks == 1 ? wa.y : ks == 2 ? wa.z : wa.w;
                        const uint32_t ub = ks == 0 ? wb.x : ks == 1 ? wb.y : ks == 2 ? wb.z : wb.w;
                        if constexpr (FMT == KVQ_INT4_B64) {
                            const uint32_t ah = ua >> 8, bh = ub >> 8;
#pragma unroll
                            for (int nt = 0; nt < NT; nt++) {
                                const uint32_t(&q)[8][2] = qb[nt];
                                if (ks == 0)
                                    mma16816_first(a[nt], nib.lo(ua), nib.lo(ub), nib.hi(ua), nib.hi(ub), q[0][0],
                                                   q[0][1]);
                                else
                                    mma16816(a[nt], nib.lo(ua), nib.lo(ub), nib.hi(ua), nib.hi(ub), q[2 * ks][0],
                                             q[2 * ks][1]);
                                mma16816(a[nt], nib.lo(ah), nib.lo(bh), nib.hi(ah), nib.hi(bh), q[2 * ks + 1][0],
                                         q[2 * ks + 1][1]);
                            }
                        } else {
                            __half2 ra[2], rb[2];
                            widen_bytes<FMT>(ua, ra);
                            widen_bytes<FMT>(ub, rb);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++) {
                                const uint32_t(&q)[2] = qb[nt][4 * pc + ks];
                                if (pc == 0 && ks == 0)
                                    mma16816_first(a[nt], h2_bits(ra[0]), h2_bits(rb[0]), h2_bits(ra[1]),
                                                   h2_bits(rb[1]), q[0], q[1]);
                                else
                                    mma16816(a[nt], h2_bits(ra[0]), h2_bits(rb[0]), h2_bits(ra[1]), h2_bits(rb[1]),
                                             q[0], q[1]);
                            }
                        }
                    }
        }
        if (!ok) break;

        // log2-sum of the page per query row: lanes (0..7, t) hold the 64 keys of columns 2t, 2t + 1
        const int k0 = j * kPage;
        if (k0 + kPage - 1 > pos0) {  // keys past some row's position
#pragma unroll
            for (int k = 0; k < 4; k++)
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (k0 + 16 * k + 8 * (e >> 1) + g > pos[nt][e & 1]) acc[k][nt][e] = -INFINITY;
        }
        const float f = FMT == KVQ_INT4_B64 ? fac * 16777216.0f : fac;
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            float m[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                m[e] = max3(acc[0][nt][e], acc[0][nt][2 + e], acc[1][nt][e]);
                m[e] = max3(m[e], acc[1][nt][2 + e], acc[2][nt][e]);
                m[e] = max3(m[e], acc[2][nt][2 + e], acc[3][nt][e]);
                m[e] = fmaxf(m[e], acc[3][nt][2 + e]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(kFull, m[e], o));
            }
            // 2^(s - m) with s - m = f (raw - raw max): the columns' pair in one instruction.  A row
            // whose keys are all masked keeps a sum of 0
            const uint64_t f2 = pk2(f, f);
            const uint64_t r2 = pk2(m[0] == -INFINITY ? 0.0f : -f * m[0], m[1] == -INFINITY ? 0.0f : -f * m[1]);
            uint64_t l2 = pk2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                float x0, x1;
                upk2(fma2(pk2(acc[k >> 1][nt][2 * (k & 1)], acc[k >> 1][nt][2 * (k & 1) + 1]), f2, r2), x0, x1);
                l2 = add2(l2, pk2(ex2_approx(x0), ex2_approx(x1)));
            }
            // sums over the 8 lanes of a column: the first exchange leaves column 2t to even g, 2t + 1
            // to odd g
            float la, lb;
            upk2(l2, la, lb);
            const bool odd = g & 1;
            float l = odd ? lb : la;
            l += __shfl_xor_sync(kFull, odd ? la : lb, 4);
            l += __shfl_xor_sync(kFull, l, 8);
            l += __shfl_xor_sync(kFull, l, 16);
            if (writes >> nt & 1u)
                *dst[nt] = fmaf(f, odd ? m[1] : m[0], FMT == KVQ_INT4_B64 ? bias[nt] * fac : 0.0f) + __log2f(l);
            dst[nt] += row_step;
        }
    }
    if (bad_page) set_flag(p.status, KVQ_FLAG_BAD_PAGE);
    if (!ok) {  // a copy did not come: flagged, and none is left in flight
        if (lane == 0) set_flag(p.status, KVQ_FLAG_TIMEOUT);
        for (int k = 0; k < kPwStages && c + k < chunks; k++) {
            mbar_wait_bounded(&full[st], phase);
            if (++st == kPwStages) {
                st = 0;
                phase ^= 1u;
            }
        }
    }
}

// Rows [64 c, 64 c + 64) of sequence b: the rows' log2-sums over the pages, then each page's mass
// over these rows, to the output (one chunk) or to `part`.  A lane has two rows, a warp every 16th
// page; the pages go in blocks of 256, the first one last, so that it is still in registers for
// the masses (up to 16K tokens are read once).
__global__ void __launch_bounds__(kSumThreads, 2) page_sum_kernel(PageWeightsParams p)
{
    constexpr int kWarps = kSumThreads / 32, kPages = 16, kBlock = kWarps * kPages;
    __shared__ float2 row_part[kWarps][kPwSumRows];  // maximum and sum of a warp's pages
    __shared__ float total[kPwSumRows];
    __shared__ float mass[kBlock];
    const int b = blockIdx.y, c = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    PwSeq s;
    const bool good = pw_seq(p, b, s);
    pdl_wait();  // (the lengths are read before it)
    if (!good) return;
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
    const bool have[2] = {lane < nr, lane + 32 < nr};
    const float *sums = pw_sums(p, s) + r0 + lane;
    float v[kPages][2];
    auto load = [&](int j0) {
#pragma unroll
        for (int i = 0; i < kPages; i++) {
            const int j = j0 + i * kWarps + warp;
            const float *at = sums + j * rows;
#pragma unroll
            for (int x = 0; x < 2; x++) v[i][x] = j < np && have[x] ? at[32 * x] : -INFINITY;
        }
    };
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    for (int j0 = (np - 1) / kBlock * kBlock; j0 >= 0; j0 -= kBlock) {
        load(j0);
#pragma unroll
        for (int x = 0; x < 2; x++) {
            float top = m[x];
#pragma unroll
            for (int i = 0; i < kPages; i += 2) top = max3(top, v[i][x], v[i + 1][x]);
            const float ref = top == -INFINITY ? 0.0f : top;
            l[x] *= ex2_approx(m[x] - ref);  // (m = -inf: the sum was 0)
#pragma unroll
            for (int i = 0; i < kPages; i++) l[x] += ex2_approx(v[i][x] - ref);
            m[x] = top;
        }
    }
    row_part[warp][lane] = make_float2(m[0], l[0]);
    row_part[warp][lane + 32] = make_float2(m[1], l[1]);
    __syncthreads();
    if (tid < kPwSumRows) {
        float top = -INFINITY, a = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; w++) top = fmaxf(top, row_part[w][tid].x);
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            const float2 y = row_part[w][tid];
            a += y.x == -INFINITY ? y.y : y.y * ex2_approx(y.x - top);  // (-inf: a sum of 0, or NaN)
        }
        total[tid] = tid < nr ? top + __log2f(a) : 0.0f;
    }
    __syncthreads();
    const float t0 = total[lane], t1 = total[lane + 32];
    const bool last = rows <= kPwSumRows;  // the sequence's only chunk
    const int per_token = (p.num_q_heads + kPwSumRows - 1) / kPwSumRows;
    float *part = p.part + ((int64_t)s.c0 * per_token + c) * mb;
    const int end = last ? mb : np;
    for (int j0 = 0; j0 < end; j0 += kBlock) {
        if (j0 > 0) load(j0);
        // over the lanes: every exchange halves a lane's pages, the last one adds two lanes' sums of
        // one page, (lane / 2) of the warp's 16
        float a[kPages];
#pragma unroll
        for (int i = 0; i < kPages; i++) a[i] = ex2_approx(v[i][0] - t0) + ex2_approx(v[i][1] - t1);
#pragma unroll
        for (int o = 16, half = kPages / 2; half > 0; o >>= 1, half >>= 1) {
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < half; i++) {
                const float mine = upper ? a[i + half] : a[i], other = upper ? a[i] : a[i + half];
                a[i] = mine + __shfl_xor_sync(kFull, other, o);
            }
        }
        a[0] += __shfl_xor_sync(kFull, a[0], 1);
        if ((lane & 1) == 0) mass[(lane >> 1) * kWarps + warp] = a[0];
        __syncthreads();
        const int j = j0 + tid;
        if (tid < kBlock && j < end) {
            const float w = j < np ? mass[tid] : 0.0f;
            if (!last)
                part[j] = w;
            else
                out[j] = j < np ? fmaf(p.decay, in ? in[j] : 0.0f, w) : 0.0f;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSumThreads) page_join_kernel(PageWeightsParams p)
{
    const int b = blockIdx.y, j = blockIdx.x * kSumThreads + threadIdx.x, mb = p.max_blocks;
    PwSeq s;
    const bool good = pw_seq(p, b, s);
    pdl_wait();
    if (!good || j >= mb) return;
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
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(page_lse_kernel<FMT, NT>, sizeof(PwSmem), done);
    if (e != cudaSuccess) return e;
    return launch_pdl(page_lse_kernel<FMT, NT>, dim3((unsigned)num_sms), dim3(kPwWarps * 32), sizeof(PwSmem), s, p);
}

template <int FMT>
static cudaError_t launch_page_weights_fmt(const PageWeightsParams &p, int num_sms, cudaStream_t s)
{
    const int64_t rows = (int64_t)p.max_q * p.group;  // query rows of one cache head
    if (rows <= 8) return launch_page_lse<FMT, 1>(p, num_sms, s);
    if (rows <= 16) return launch_page_lse<FMT, 2>(p, num_sms, s);
    return launch_page_window(FMT, p, num_sms, s);
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
    e = launch_pdl(page_sum_kernel, dim3((unsigned)chunks, (unsigned)p.num_seqs), dim3(kSumThreads), 0, s, p);
    if (e != cudaSuccess || chunks == 1) return e;
    return launch_pdl(page_join_kernel, dim3((unsigned)((p.max_blocks + kSumThreads - 1) / kSumThreads),
                                               (unsigned)p.num_seqs),
                        dim3(kSumThreads), 0, s, p);
}

}  // namespace kvq
