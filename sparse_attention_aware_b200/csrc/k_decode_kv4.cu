// Split-KV sparse decode over a 4-bit cache (records of kv4.cuh), on mma.sync
// tensor cores.
//
// Method: as k_decode.cu and k_decode_gqa.cu -- attention of one query token
// per sequence over a token list per query head ("Kascade稀疏注意力…", section
// "核心机制：Anchor + Reuse") or a list of page segments shared by the heads
// ("语言模型能自己决定该看哪里吗？", DA state machine section), cut into parts
// that the common combine pass merges ("稀疏注意力机制创新…", section
// "四、从外卖到AI": SplitKV-and-Combine).  A row of 128 channels is 144 bytes
// here instead of 512.
//
// Mathematics.  A code c enters the matrix instruction as the bf16 number
// u = 1 + c/16: its four bits are or'd below 1.0's exponent, so widening costs
// a shift and one logic operation for two codes and no conversion.  Scale s
// and zero z of a half row then act outside the product:
//   x = z + s c = 16 s u + (z - 16 s)
//   q . k = sum over halves of  16 s (q . u) + (z - 16 s) sum(q)
//   sum_t p_t v_t = sum_t p'_t u_t - sum_t p'_t + sum_t p_t z_t,
//                   p'_t = bf16(16 s_t p_t)
// sum(q) comes from a product with ones of the very bf16 parts of q that the
// first product uses, and sum p' likewise from the rounded p', so the offset
// 1 of u cancels but for fp32 sums and the rounding of p' acts on the codes'
// part of v alone (bf16: half a step, 2^-8 relative).
//
// One CTA = (split, kv head and up to 16 of its query heads -- or one query
// head for token lists --, sequence), kDW warps that run independently until
// the final merge.  A warp streams tiles of 16 rows through its own ring of
// kDST shared-memory stages by bulk copies (one copy per page segment, one
// per row of a token list), each stage on its own mbarrier with a bounded
// wait.  Rows are padded by their scales, so 8-row matrix loads touch 32
// distinct banks (kv4.cuh).  Per tile: S^T = K Q^T with the 16 tokens as M and
// the heads as N of m16n8k16, softmax per head column in the base-2 domain,
// P'^T into the B layout by movmatrix, O^T += V^T P'^T.
//
// The running maximum of a head is raised (and its sums rescaled) only when a
// score passes it by more than 2^8: weights stay below 2^8, far from any
// overflow, and most tiles need neither the max across lanes nor a rescale.
//
// Bound: HBM for long lists; the widening and the softmax take about 60% of
// the issue slots at that rate.
#include <cuda_bf16.h>

#include "kv4.cuh"
#include "tc_ptx.cuh"

namespace sa {
namespace {

constexpr int kDW = 4;                   // warps per CTA
constexpr int kDThreads = kDW * 32;
constexpr int kDR = 16;                  // rows per tile (the MMA's M)
constexpr int kDST = 4;                  // ring stages per warp
constexpr int kDWindow = 1024;           // token-list positions resolved at a time
constexpr float kLazy = 8.f;             // log2 of how far a score may pass the running maximum
constexpr uint64_t kDWaitNs = 1000ull * 1000 * 1000;   // 1 s

template <int D>
struct DSmem {
    static constexpr int STAGE = kDR * Kv4<D>::REC;
    static constexpr int RING = kDW * kDST * STAGE;
    static constexpr int MERGE = kDW * (16 * D + 32) * 4;   // per-warp O, m, l (up to 16 heads)
    static constexpr int BODY = RING > MERGE ? RING : MERGE;
    static constexpr int BARS = BODY;                        // mbarriers
    static constexpr int ROWS = BARS + kDW * kDST * 8 + 16;  // abort flag in between; then row numbers
    static constexpr int BYTES = ROWS;
    static constexpr int BYTES_TOKENS = ROWS + kDWindow * 4;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// transpose of an 8x8 b16 matrix held in the mma fragment layout
__device__ __forceinline__ uint32_t movm(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// D (16x8 fp32) += A (16x16 bf16, row) * B (16x8 bf16, col)
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// nibble I of each 16-bit half of w as the bf16 pair 1 + c/16
template <int I>
__device__ __forceinline__ uint32_t widen(uint32_t w)
{
    const uint32_t x = I == 0 ? w << 3 : w >> (4 * I - 3);
    return (x & 0x00780078u) | 0x3f803f80u;
}
constexpr uint32_t kOnes = 0x3f803f80u;

__device__ __forceinline__ uint32_t pack_pair(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Query channels c0 and c1 of one head: bf16 pair, and for an fp32 query the
// pair of the rest x - bf16(x) (so that the two carry ~16 bits of it)
template <bool QF32>
__device__ __forceinline__ void query_pair(const void *q, size_t row, bool valid, int c0, int c1, uint32_t &hi,
                                           uint32_t &lo)
{
    hi = lo = 0u;
    if (!valid) return;
    if (QF32) {
        const float *p = static_cast<const float *>(q) + row;
        const float x = p[c0], y = p[c1];
        hi = pack_pair(x, y);
        lo = pack_pair(x - bf_lo(hi), y - bf_hi(hi));
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(q) + row;
        hi = (uint32_t)p[c0] | ((uint32_t)p[c1] << 16);
    }
}

// NH = 8-head column blocks of the CTA (1 or 2); TOKENS: one query head and
// its token list, else a kv head's heads and the sequence's block list
template <int D, int NH, bool QF32, bool TOKENS>
__global__ void __launch_bounds__(kDThreads) k_decode_kv4(const DecodeArgs a)
{
    pdl_wait();
    pdl_trigger();
    using SM = DSmem<D>;
    constexpr int REC = Kv4<D>::REC;
    constexpr int CB = D / 32;           // 16-byte column blocks of a row's codes (32 channels each)
    constexpr int CBH = CB / 2;          // of a half
    constexpr int NQ = QF32 ? 2 : 1;
    extern __shared__ __align__(128) uint8_t sm[];
    const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(sm);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + SM::BARS);   // [kDW][kDST]
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + kDW * kDST);
    uint32_t *s_row = reinterpret_cast<uint32_t *>(sm + SM::ROWS);   // token lists: rows of a window

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gq = lane >> 2, tq = lane & 3;   // mma group id / thread in group
    const int s = blockIdx.x, b = blockIdx.z;
    const int HPG = a.Hq / a.c.Hkv;
    const int hblocks = (HPG + 15) / 16;
    const int g = TOKENS ? blockIdx.y / HPG : blockIdx.y / hblocks;
    const int h0 = TOKENS ? blockIdx.y : g * HPG + (blockIdx.y % hblocks) * 16;   // first query head
    const int nheads = TOKENS ? 1 : min(16, (g + 1) * HPG - h0);
    const uint8_t *pool = reinterpret_cast<const uint8_t *>(a.c.k);
    DevStatus *st = a.st;
    const bool reports = s == 0 && tid == 0;

    const int Lcap = a.c.max_pages << a.c.Plog2;
    int L = __ldg(a.c.sl + b);
    if (L < 0 || L > Lcap) {
        if (reports) fault(st, CHK_SEQ_LEN, L);
        L = L < 0 ? 0 : Lcap;
    }
    // this split's range [lo, hi) of list positions (tokens) or entries (blocks)
    int lo, hi;
    const int *pt = a.c.pt + (size_t)b * a.c.max_pages;
    const int4 *ent = nullptr;
    const int *idx = nullptr;
    if (TOKENS) {
        const size_t r = (size_t)b * a.Hq + h0;
        int n = __ldg(a.cnt + r);
        if (n < 0 || n > a.kcap) {
            if (reports) fault(st, CHK_COUNT, n);
            n = n < 0 ? 0 : a.kcap;
        }
        idx = a.idx + r * a.kcap;
        const int chunk = ((n + a.S - 1) / a.S + kDR - 1) / kDR * kDR;   // whole tiles
        lo = min(s * chunk, n);
        hi = min(lo + chunk, n);
    } else {
        int n = __ldg(a.ecnt + b);
        if (n < 0 || n > a.max_blocks) {
            if (reports) fault(st, CHK_BLOCK_ENTRY, n);
            n = n < 0 ? 0 : a.max_blocks;
        }
        ent = reinterpret_cast<const int4 *>(a.ent) + (size_t)b * a.max_blocks;
        lo = (int)((long long)n * s / a.S);
        hi = (int)((long long)n * (s + 1) / a.S);
    }
    if (lo >= hi) {   // nothing for this split: an empty partial, which the combine skips
        for (int j = tid; j < nheads; j += kDThreads) {
            const size_t row = (size_t)b * a.Hq + h0 + j;
            a.part_ml[(row * a.S + s) * 2 + 0] = -INFINITY;
            a.part_ml[(row * a.S + s) * 2 + 1] = 0.f;
        }
        return;
    }

    if (tid == 0) {
        for (int i = 0; i < kDW * kDST; ++i) tc::mbar_init(bars + i, 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
    }

    // query B fragments: column n is head h0 + n; the k-steps' channels follow
    // the order in which widen() hands out a code word (channels i and i + 4)
    uint32_t qb[NQ][NH][CB][2][2];
    float qs[2][NH][2];   // sum of the query over each half, heads nh*8 + 2tq + j
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        const int h = nh * 8 + gq;
        const size_t r = ((size_t)b * a.Hq + h0 + h) * D;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t x, y;
                const int c = cb * 32 + tq * 8 + i;
                query_pair<QF32>(a.q, r, h < nheads, c, c + 4, x, y);
                qb[0][nh][cb][i >> 1][i & 1] = x;
                if (QF32) qb[NQ - 1][nh][cb][i >> 1][i & 1] = y;
            }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int cb = half * CBH; cb < (half + 1) * CBH; ++cb)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int qi = 0; qi < NQ; ++qi)
                        mma(sum, kOnes, kOnes, kOnes, kOnes, qb[qi][nh][cb][ks][0], qb[qi][nh][cb][ks][1]);
            qs[half][nh][0] = sum[0];
            qs[half][nh][1] = sum[1];
        }
    }
    __syncthreads();   // mbarriers initialised

    // O^T fragments: o[cb][j][nh]: rows gq / gq + 8 are channels cb*32 + 4gq + 2j / + 1, columns heads 2tq, 2tq + 1
    float o[CB][2][NH][4];
    float op[2][NH][4];            // sum of p' per half (every row the same)
    float zs[2][NH][2];            // sum of p z per half, this thread's tokens
    float mh[NH][2], lh[NH][2];    // heads nh*8 + 2tq + j (l: this thread's tokens)
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int j = 0; j < 2; ++j) o[cb][j][nh][0] = o[cb][j][nh][1] = o[cb][j][nh][2] = o[cb][j][nh][3] = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            op[half][nh][0] = op[half][nh][1] = op[half][nh][2] = op[half][nh][3] = 0.f;
            zs[half][nh][0] = zs[half][nh][1] = 0.f;
        }
        mh[nh][0] = mh[nh][1] = -INFINITY;
        lh[nh][0] = lh[nh][1] = 0.f;
    }

    uint64_t *wbar = bars + warp * kDST;
    uint8_t *wring = sm + warp * kDST * SM::STAGE;
    const uint32_t wring_a = sbase + warp * kDST * SM::STAGE;
    const uint64_t deadline = tc::globaltimer() + kDWaitNs;
    int done = 0;          // tiles this warp has consumed (stage = done % kDST, parity = (done / kDST) & 1)
    bool alive = true;

    // one tile whose rows (those in `mask`) are in stage `stage`
    auto consume = [&](int stage, uint32_t mask) {
        const uint32_t base = wring_a + stage * SM::STAGE;
        const uint32_t quad = base + ((lane & 7) + ((lane >> 3) & 1) * 8) * REC + (lane >> 4) * 16;
        const uint8_t *gen = wring + stage * SM::STAGE;
        const bool ok0 = (mask >> gq) & 1, ok1 = (mask >> (gq + 8)) & 1;
        // scales and zeros {K half 0, K half 1, V half 0, V half 1} of rows gq, gq + 8; a row
        // outside the mask is whatever the stage held, and must not reach a product
        uint4 p0 = *reinterpret_cast<const uint4 *>(gen + gq * REC + Kv4<D>::PAR);
        uint4 p1 = *reinterpret_cast<const uint4 *>(gen + (gq + 8) * REC + Kv4<D>::PAR);
        if (!ok0) p0 = make_uint4(0, 0, 0, 0);
        if (!ok1) p1 = make_uint4(0, 0, 0, 0);

        // ---- S^T = K Q^T per half
        float sc[2][NH][4];
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
                sc[half][nh][0] = sc[half][nh][1] = sc[half][nh][2] = sc[half][nh][3] = 0.f;
#pragma unroll
        for (int c2 = 0; c2 < CB; c2 += 2) {
            // matrices: rows 0-7 / 8-15 of column block c2, then of c2 + 1
            uint32_t w[4];
            ldsm4(quad + c2 * 16, w);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t w0 = w[2 * u], w1 = w[2 * u + 1];
                const uint32_t f[2][4] = {{widen<0>(w0), widen<0>(w1), widen<1>(w0), widen<1>(w1)},
                                          {widen<2>(w0), widen<2>(w1), widen<3>(w0), widen<3>(w1)}};
                const int cb = c2 + u, half = cb / CBH;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                        for (int qi = 0; qi < NQ; ++qi)
                            mma(sc[half][nh], f[ks][0], f[ks][1], f[ks][2], f[ks][3], qb[qi][nh][cb][ks][0],
                                qb[qi][nh][cb][ks][1]);
            }
        }
        // ---- scores: rows gq (elements 0, 1) and gq + 8 (2, 3), base-2 domain
        const float k16 = 16.f * a.qscale;
        const float s00 = bf_lo(p0.x) * k16, s01 = bf_lo(p0.y) * k16, s10 = bf_lo(p1.x) * k16, s11 = bf_lo(p1.y) * k16;
        const float c00 = fmaf(bf_hi(p0.x), a.qscale, -s00), c01 = fmaf(bf_hi(p0.y), a.qscale, -s01);
        const float c10 = fmaf(bf_hi(p1.x), a.qscale, -s10), c11 = fmaf(bf_hi(p1.y), a.qscale, -s11);
        float x[NH][4];
        bool high = false;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float y0 = fmaf(s00, sc[0][nh][j], fmaf(s01, sc[1][nh][j],
                                      fmaf(c00, qs[0][nh][j], c01 * qs[1][nh][j])));
                const float y1 = fmaf(s10, sc[0][nh][2 + j], fmaf(s11, sc[1][nh][2 + j],
                                      fmaf(c10, qs[0][nh][j], c11 * qs[1][nh][j])));
                x[nh][j] = ok0 ? y0 : -INFINITY;
                x[nh][2 + j] = ok1 ? y1 : -INFINITY;
                // (also true for the first finite score of a head)
                high = high || fmaxf(x[nh][j], x[nh][2 + j]) > mh[nh][j] + kLazy;
            }
        }
        if (__any_sync(~0u, high)) {
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float m = fmaxf(mh[nh][j], fmaxf(x[nh][j], x[nh][2 + j]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, off));
                    const float al = m == -INFINITY ? 1.f : ex2(mh[nh][j] - m);   // 0 for a head that was empty
                    mh[nh][j] = m;
                    lh[nh][j] *= al;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        zs[half][nh][j] *= al;
                        op[half][nh][j] *= al;
                        op[half][nh][2 + j] *= al;
                    }
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            o[cb][i][nh][j] *= al;
                            o[cb][i][nh][2 + j] *= al;
                        }
                }
        }
        // ---- weights; P'^T (tokens x heads) per half as B fragments (k = tokens)
        const float v00 = 16.f * bf_lo(p0.z), v01 = 16.f * bf_lo(p0.w), v10 = 16.f * bf_lo(p1.z), v11 = 16.f * bf_lo(p1.w);
        const float z00 = bf_hi(p0.z), z01 = bf_hi(p0.w), z10 = bf_hi(p1.z), z11 = bf_hi(p1.w);
        uint32_t pb[2][NH][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float m = mh[nh][j] == -INFINITY ? 0.f : mh[nh][j];
                p[j] = ex2(x[nh][j] - m);
                p[2 + j] = ex2(x[nh][2 + j] - m);
                lh[nh][j] += p[j] + p[2 + j];
                zs[0][nh][j] = fmaf(p[j], z00, fmaf(p[2 + j], z10, zs[0][nh][j]));
                zs[1][nh][j] = fmaf(p[j], z01, fmaf(p[2 + j], z11, zs[1][nh][j]));
            }
            pb[0][nh][0] = movm(pack_pair(p[0] * v00, p[1] * v00));
            pb[0][nh][1] = movm(pack_pair(p[2] * v10, p[3] * v10));
            pb[1][nh][0] = movm(pack_pair(p[0] * v01, p[1] * v01));
            pb[1][nh][1] = movm(pack_pair(p[2] * v11, p[3] * v11));
#pragma unroll
            for (int half = 0; half < 2; ++half)
                mma(op[half][nh], kOnes, kOnes, kOnes, kOnes, pb[half][nh][0], pb[half][nh][1]);
        }
        // ---- O^T += V^T P'^T: transposed 8x8 loads of the code bytes give, per
        // register, 4 channels of tokens 2tq (low half) and 2tq + 1 (high half)
#pragma unroll
        for (int c2 = 0; c2 < CB; c2 += 2) {
            uint32_t w[4];
            ldsm4_t(quad + Kv4<D>::V + c2 * 16, w);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t w0 = w[2 * u], w1 = w[2 * u + 1];
                const uint32_t f[2][4] = {{widen<0>(w0), widen<1>(w0), widen<0>(w1), widen<1>(w1)},
                                          {widen<2>(w0), widen<3>(w0), widen<2>(w1), widen<3>(w1)}};
                const int cb = c2 + u, half = cb / CBH;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
                        mma(o[cb][j][nh], f[j][0], f[j][1], f[j][2], f[j][3], pb[half][nh][0], pb[half][nh][1]);
            }
        }
    };
    // waits for the warp's next stage; on expiry the warp records it and stops
    auto arrived = [&]() -> bool {
        const bool ok = __all_sync(~0u, tc::mbar_wait(wbar + done % kDST, (uint32_t)(done / kDST) & 1u, deadline,
                                                      abort_flag));
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) record(st, SA_ERR_TIMEOUT, CHK_WAIT, done);
            alive = false;
        }
        return ok;
    };
    // copies still in flight land before the CTA's shared memory is released
    auto drain = [&](int tiles) {
        const uint64_t dl = tc::globaltimer() + kDWaitNs;
        volatile int zero = 0;
        for (int i = 0; i < tiles; ++i, ++done)
            tc::mbar_wait(wbar + done % kDST, (uint32_t)(done / kDST) & 1u, dl, &zero);
    };

    if (TOKENS) {
        // a window of the list is resolved (index -> page -> row, validated)
        // into shared memory by the whole CTA; then each warp streams tiles
        // warp, warp + kDW, ... of it
        constexpr uint32_t kNone = 0xffffffffu;
        for (int w0 = lo; w0 < hi; w0 += kDWindow) {
            const int wn = min(kDWindow, hi - w0);
            __syncthreads();   // the previous window's rows have been used
            for (int i = tid; i < (wn + kDR - 1) / kDR * kDR; i += kDThreads) {
                uint32_t row = kNone;
                if (i < wn) {
                    const int t = __ldg(idx + w0 + i);
                    if (t < 0 || t >= L) {
                        fault(st, CHK_INDEX, t);
                    } else {
                        const int page = __ldg(pt + (t >> a.c.Plog2));
                        if (page < 0 || page >= a.c.num_pages) fault(st, CHK_PAGE, page);
                        else row = (((uint32_t)page * a.c.Hkv + g) << a.c.Plog2) + (t & ((1 << a.c.Plog2) - 1));
                    }
                }
                s_row[i] = row;
            }
            __syncthreads();
            const int tiles = ((wn + kDR - 1) / kDR - warp + kDW - 1) / kDW;   // of this warp
            auto issue = [&](int n, int stage) {
                const uint32_t row = lane < kDR ? s_row[(warp + n * kDW) * kDR + lane] : kNone;
                const uint32_t mask = __ballot_sync(~0u, row != kNone);
                if (lane == 0) tc::mbar_arrive_expect_tx(wbar + stage, (uint32_t)__popc(mask) * REC);
                __syncwarp();
                if (row != kNone)
                    tc::bulk_load(wring + stage * SM::STAGE + lane * REC, pool + (size_t)row * REC, REC, wbar + stage);
                return mask;
            };
            if (!alive) continue;
            // the masks of the tiles in flight: lane i of `held` keeps stage i's
            uint32_t held = 0;
            const int pre = min(tiles, kDST);
            for (int n = 0; n < pre; ++n) {
                const uint32_t m = issue(n, (done + n) % kDST);
                if (lane == (done + n) % kDST) held = m;
            }
            for (int n = 0; n < tiles; ++n) {
                const int stage = done % kDST;
                if (!arrived()) {
                    drain(min(tiles - n, kDST));
                    break;
                }
                consume(stage, __shfl_sync(~0u, held, stage));
                ++done;
                __syncwarp();   // every lane is done with this stage before it is refilled
                if (n + kDST < tiles) {
                    const uint32_t m = issue(n + kDST, stage);
                    if (lane == stage) held = m;
                }
            }
        }
    } else {
        // the warp's entries lo + warp + kDW * j, a window of 32 (one per lane) at a time
        for (int wb = lo + warp; wb < hi && alive; wb += 32 * kDW) {
            const int e = wb + kDW * lane;
            int first = 0, len = 0;   // the entry's first row within the page, and its rows (0 = skipped)
            uint32_t row = 0;
            if (e < hi) {
                const int4 en = ent[e];
                bool ok = en.y >= 0 && en.y < en.z && en.z <= (1 << a.c.Plog2) && en.x >= 0 && en.x < a.c.max_pages;
                if (!ok) fault(st, CHK_BLOCK_ENTRY, e);
                if (ok && (en.x << a.c.Plog2) + en.z > L) {
                    fault(st, CHK_INDEX, (en.x << a.c.Plog2) + en.z - 1);
                    ok = false;
                }
                if (ok) {
                    const int page = __ldg(pt + en.x);
                    if (page < 0 || page >= a.c.num_pages) {
                        fault(st, CHK_PAGE, page);
                    } else {
                        first = en.y;
                        len = en.z - en.y;
                        row = (((uint32_t)page * a.c.Hkv + g) << a.c.Plog2) + first;
                    }
                }
            }
            // tiles per entry, inclusive prefix over the lanes
            const int nt = (len + kDR - 1) / kDR;
            int incl = nt;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(~0u, incl, off);
                if (lane >= off) incl += y;
            }
            const int tiles = __shfl_sync(~0u, incl, 31);
            // tile n: rows of the entry that holds it; returns their number
            auto issue = [&](int n, int stage) -> int {
                const int src = __ffs(__ballot_sync(~0u, incl > n)) - 1;
                const uint32_t r = __shfl_sync(~0u, row, src);
                const int ln = __shfl_sync(~0u, len, src);
                const int at = (n - __shfl_sync(~0u, incl - nt, src)) * kDR;
                const int rows = min(kDR, ln - at);
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(wbar + stage, (uint32_t)rows * REC);
                    tc::bulk_load(wring + stage * SM::STAGE, pool + (size_t)(r + at) * REC, (uint32_t)rows * REC,
                                  wbar + stage);
                }
                return rows;
            };
            int held = 0;   // lane i: rows of the tile in stage i
            const int pre = min(tiles, kDST);
            for (int n = 0; n < pre; ++n) {
                const int r = issue(n, (done + n) % kDST);
                if (lane == (done + n) % kDST) held = r;
            }
            for (int n = 0; n < tiles; ++n) {
                const int stage = done % kDST;
                if (!arrived()) {
                    drain(min(tiles - n, kDST));
                    break;
                }
                consume(stage, (1u << __shfl_sync(~0u, held, stage)) - 1u);
                ++done;
                __syncwarp();   // every lane is done with this stage before it is refilled
                if (n + kDST < tiles) {
                    const int r = issue(n + kDST, stage);
                    if (lane == stage) held = r;
                }
            }
        }
    }

    // ---- merge the warps' states through shared memory
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                lh[nh][j] += __shfl_xor_sync(~0u, lh[nh][j], off);
                zs[0][nh][j] += __shfl_xor_sync(~0u, zs[0][nh][j], off);
                zs[1][nh][j] += __shfl_xor_sync(~0u, zs[1][nh][j], off);
            }
    __syncthreads();
    float *mo = reinterpret_cast<float *>(sm);                 // [warp][16][D]
    float *mm = mo + kDW * 16 * D;                              // [warp][16]
    float *ml = mm + kDW * 16;                                  // [warp][16]
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int h = nh * 8 + 2 * tq + (i & 1), half = cb / CBH;
                    const int c = cb * 32 + 4 * gq + 2 * j + (i >> 1);
                    mo[(warp * 16 + h) * D + c] = o[cb][j][nh][i] + (zs[half][nh][i & 1] - op[half][nh][i & 1]);
                }
    if (gq == 0) {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mm[warp * 16 + nh * 8 + 2 * tq + j] = mh[nh][j];
                ml[warp * 16 + nh * 8 + 2 * tq + j] = lh[nh][j];
            }
    }
    __syncthreads();
    for (int i = tid; i < nheads * D; i += kDThreads) {
        const int j = i / D, c = i % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kDW; ++w) M = fmaxf(M, mm[w * 16 + j]);
        float O = 0.f, Ls = 0.f;
#pragma unroll
        for (int w = 0; w < kDW; ++w) {
            const float lw = ml[w * 16 + j];
            if (lw == 0.f) continue;   // no token (a sum that is not a number is taken along)
            const float wgt = ex2(mm[w * 16 + j] - M);
            O = fmaf(wgt, mo[(w * 16 + j) * D + c], O);
            Ls = fmaf(wgt, lw, Ls);
        }
        const size_t row = (size_t)b * a.Hq + h0 + j;
        a.part_o[(row * a.S + s) * D + c] = O;
        if (c == 0) {
            a.part_ml[(row * a.S + s) * 2 + 0] = M;
            a.part_ml[(row * a.S + s) * 2 + 1] = Ls;
        }
    }
}

// Merge of the splits, as k_decode_combine, except that a split whose sum is
// not a number (a selected row was stored as NaN) makes the result NaN.
template <int D>
__global__ void __launch_bounds__(D) k_kv4_combine(const float *__restrict__ part_o, const float *__restrict__ part_ml,
                                                    int S, uint16_t *__restrict__ out, float *__restrict__ lse)
{
    pdl_wait();
    pdl_trigger();
    const int row = blockIdx.x, c = threadIdx.x;
    const float *ml = part_ml + (size_t)row * S * 2;
    float M = -INFINITY;
    for (int s = 0; s < S; ++s)
        if (ml[2 * s + 1] != 0.f) M = fmaxf(M, ml[2 * s]);
    float o = 0.f, Ls = 0.f;
    for (int s = 0; s < S; ++s) {
        const float ls = ml[2 * s + 1];
        if (ls == 0.f) continue;
        const float w = ex2(ml[2 * s] - M);
        Ls = fmaf(w, ls, Ls);
        o = fmaf(w, part_o[((size_t)row * S + s) * D + c], o);
    }
    const bool some = Ls != 0.f;
    out[(size_t)row * D + c] = f2bf(some ? o / Ls : 0.f);
    if (lse && c == 0) lse[row] = some ? (M + lg2(Ls)) * kLn2 : -INFINITY;
}

template <int D, int NH, bool QF32, bool TOKENS>
cudaError_t launch_kv4(const DecodeArgs &a, cudaStream_t s)
{
    constexpr int smem = TOKENS ? DSmem<D>::BYTES_TOKENS : DSmem<D>::BYTES;
    auto kern = k_decode_kv4<D, NH, QF32, TOKENS>;
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
    const int hpg = a.Hq / a.c.Hkv;
    const dim3 grid((unsigned)a.S, (unsigned)(TOKENS ? a.Hq : a.c.Hkv * ((hpg + 15) / 16)), (unsigned)a.c.B);
    return launch_pdl(kern, grid, dim3(kDThreads), smem, s, a);
}

template <int D, bool QF32>
cudaError_t launch_kind(const DecodeArgs &a, cudaStream_t s)
{
    if (!a.blocks) return launch_kv4<D, 1, QF32, true>(a, s);
    return a.Hq / a.c.Hkv <= 8 ? launch_kv4<D, 1, QF32, false>(a, s) : launch_kv4<D, 2, QF32, false>(a, s);
}

}  // namespace

// Enough CTAs to fill the device about twice over (ragged lists even out), but
// no split below 256 tokens of the longest possible list.
int decode_kv4_splits(int B, int rows, long long list)
{
    const long long units = (long long)B * rows;
    if (units <= 0) return 1;
    const long long want = (2 * 148 * 4 + units - 1) / units, most = (list + 255) / 256;
    const long long s = want < most ? want : most;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

cudaError_t launch_decode_kv4(const DecodeArgs &a, cudaStream_t s)
{
    if (a.c.B * a.Hq == 0) return cudaSuccess;
    cudaError_t e;
    if (a.c.D == 64) e = a.q_f32 ? launch_kind<64, true>(a, s) : launch_kind<64, false>(a, s);
    else e = a.q_f32 ? launch_kind<128, true>(a, s) : launch_kind<128, false>(a, s);
    if (e != cudaSuccess) return e;
    auto comb = a.c.D == 64 ? k_kv4_combine<64> : k_kv4_combine<128>;
    return launch_pdl(comb, dim3((unsigned)(a.c.B * a.Hq)), dim3((unsigned)a.c.D), 0, s, a.part_o, a.part_ml, a.S, a.out,
                      a.lse);
}

}  // namespace sa
