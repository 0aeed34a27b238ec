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
// Mathematics.  A half row is x = z + s c with codes c in [0, 15]:
//   q . k = sum over halves of  s (q . c) + z sum(q)
//   sum_t p_t v_t = sum_t p'_t c_t + sum_t p_t z_t,     p'_t = fp16(s_t p_t)
// so scales and zeros act outside the products, and sum(q) comes from a
// product with ones of the very parts of q that the first product uses.
// The codes enter the matrix instruction as they are: a nibble alone in the low
// bits of a 16-bit word is the subnormal number c 2^-24 in fp16 and c 2^-133 in
// bf16, one in bits 4-7 is 16 times that (in bf16 half of them are past the
// subnormals, where the numbers go on in the same steps), and the products are
// exact, so eight codes cost one shift and four masks.  The 16 goes into the query
// (a sixteenth of those channels) or out of the sums (those rows of O), the power
// of two into the factors.
// Before, at 32 sequences x 8 kv heads of up to 16384 tokens: 146 us with bf16
// numbers 1 + c/16 (one logic operation and one shift a pair, all on the
// integer pipe), 118 us with fp16 numbers c - 8 (a mask-or and an fma a pair),
// 95 us with the codes as they are, all else equal.
//
// Ranges.  The matrix instruction lines products up by their operands' exponents,
// of which a subnormal's is the type's least, and drops what then lies below the
// 24 bits of fp32: a code of 1 loses products below 2^-15 of the largest one's in
// fp16, 2^-18 in bf16.  So a bf16 query meets its keys' codes as bf16, exactly and
// scaled by a power of two per head; only elements below 2^-10 of the head's
// largest lose bits (in fp16, scores of queries with a few large channels were off
// by up to 6e-5 of themselves, now 1.0 to 1.7 times a plain fp32 form's error on
// Gaussian ones).  Codes times 16 by a bf16 product first would keep 2^-22, at 2%
// more time.  An fp32 query is scaled to a largest element in [2^10, 2^11) and
// enters as fp16 in two parts: the nearest whole numbers, whose products with codes
// add up without any loss, and the rest, to 2^-23 of the largest element, with sums
// of their own.  Scores are finite while the largest element times |scale| is below
// 2^112.  s_t p_t is scaled by a power of two per half (raised scales
// rescale the sums, as a raised maximum does) to at most 2^15: a weight keeps
// 11 bits down to 2^-21 of the largest scale seen, 8 to 2^-24, and is within
// 2^-32 of that scale below.  Its rounding acts on scale times code, about 2.7
// times the value where values are spread around 0: next to the rounding of the bf16
// output it makes the error 2 to 5% larger than that of weights in fp32.
//
// One CTA = (split, kv head and up to 16 of its query heads -- or one query
// head for token lists --, sequence), kDW warps that run independently until
// the final merge.  A warp streams stages of 32 rows through its own ring of
// kDST shared-memory buffers by 16-byte asynchronous copies, one commit group
// a stage: a token list's rows are gathered 3 (or 6) rows an instruction with
// 9 (or 5) lanes a row; page segments are copied as the contiguous bytes they
// are.  (One bulk copy per row of a list costs more instructions: each lane's
// copy is issued on its own.)  What a stage copies is resolved -- list entry,
// page table, row -- two steps ahead, so the ring never waits for that chain.
// Rows are padded by their scales, so 8-row matrix loads touch 32 distinct
// banks (kv4.cuh).  Per 16 rows: S^T = K Q^T with the tokens as M and the heads
// as N of m16n8k16, softmax per head column in the base-2 domain, P'^T into the
// B layout by movmatrix, O^T += V^T P'^T.
//
// The running maximum of a head is raised (and its sums rescaled) only when a
// score passes it by more than 8 in the base-2 domain: weights stay below 2^8,
// and most tiles need neither the max across lanes nor a rescale.
//
// A group of at most 4 heads fills half of the 8 columns, a token list's head one.
// Two tiles of 16 rows then share a softmax: the heads stand in columns 0-3 for the
// one and again in 4-7 for the other, as two states that the merge joins; a tile's
// products see zeros in the other's columns (whole context 90 -> 81 us, token lists
// 142.5 -> 138).
//
// Measured (B200, 6.55 TB/s copy): every page of 32 sequences of up to 16384
// tokens, 32 heads on 8 kv heads (421 MB) 82 us, 0.79 of HBM; 1024 lists of 4096
// of 65536 tokens 139 us (0.56 by the 506 MB of distinct rows and lists; 794 MB are
// read, since a row's 144 bytes touch 192 in 64-byte pieces and rows that heads share
// come again, and by those it is 0.87); a masked step of 4 sequences 10 us, 256 of
// 4096 tokens of 4 heads, fp32 queries, 5 us.  The copies alone take 67 and 134
// us, the arithmetic alone 76 and 123: about 230 instructions per 16 rows (267 with
// a list), of which widening the codes is a third, with 12 to 16 warps an SM.  Short
// calls are bound by the dependent trips length -> entry -> page -> rows -> merge.
// Farther from their floors: groups of 5 to 8 heads (16 x 8 groups of up to 16384
// tokens 54 us, 0.67 of HBM) and of 9 to 16 (8 x 4 of up to 65536 81 us, 0.44: one
// tile at a time, 8 warps an SM); fp32 queries (the first case 95 us).
//
// Measured and not kept (whole context, 81 us at that stage): a page segment by
// bulk copies 88; the next tiles' scores between a tile's weights and its products
// 80; rings of 4 stages 81; 4 CTAs an SM 82; all rows' entries shared evenly
// over one wave of CTAs 80, but 53 us and not 50 with 16 sequences of 64/8 heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv4.cuh"

namespace sa {
namespace {

constexpr int kDW = 4;                   // warps per CTA
constexpr int kDThreads = kDW * 32;
constexpr int kDR = 32;                  // rows per stage (two of the MMA's M)
constexpr int kDST = 3;                   // ring stages per warp
constexpr int kLeast = 256;              // tokens of a split at least
constexpr float kLazy = 8.f;             // log2 of how far a score may pass the running maximum

template <int D>
struct DSmem {
    static constexpr int STAGE = kDR * Kv4<D>::REC;
    static constexpr int RING = kDW * kDST * STAGE;
    // merge: per-warp O, m, l of up to 16 heads.  Two rows of ROW floats are 8
    // banks apart, so the warps' 16-byte writes (4 heads' rows, 2 runs of 4
    // channels) touch all banks once
    static constexpr int ROW = D + 4;
    static constexpr int MERGE = kDW * (16 * ROW + 32) * 4;
    static constexpr int BYTES = RING > MERGE ? RING : MERGE;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

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
// D (16x8 fp32) = A (16x16, row) * B (16x8, col), fp16 or bf16
template <bool BF>
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1)
{
    if (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D += A * B
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    if (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the 8 codes of a word as 4 fp16 pairs: f[i] holds nibble i of the low half
// word (low) and of the high half word (high), c 2^-24 for even i, 16 c 2^-24
// for odd i
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&f)[4])
{
    const uint32_t x = w >> 8;
    f[0] = w & 0x000f000fu;
    f[1] = w & 0x00f000f0u;
    f[2] = x & 0x000f000fu;
    f[3] = x & 0x00f000f0u;
}
// the same for sums from which the even codes can be taken out afterwards: f[i]
// holds c 2^-24 for even i, for odd i the byte (16 c + the even code before it)
// 2^-24, which needs no mask of its own
__device__ __forceinline__ void widen_bytes(uint32_t w, uint32_t (&f)[4])
{
    f[1] = w & 0x00ff00ffu;
    f[3] = __byte_perm(w, 0u, 0x4341);
    f[0] = w & 0x000f000fu;
    f[2] = f[3] & 0x000f000fu;
}
// pairs of 1 and of 16
template <bool BF>
constexpr uint32_t kOnes = BF ? 0x3f803f80u : 0x3c003c00u;
template <bool BF>
constexpr uint32_t kSixteens = BF ? 0x41804180u : 0x4c004c00u;

template <bool BF = false>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi)
{
    if (BF) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// 2^e as a float, e clamped to what a float holds
__device__ __forceinline__ float pow2(int e) { return __int_as_float(min(max(e + 127, 1), 254) << 23); }
__device__ __forceinline__ int exponent(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }

// 8 query channels from element i on (a multiple of 8)
template <bool F32>
__device__ __forceinline__ void query8(const void *q, size_t i, float (&x)[8])
{
    if (F32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(q) + i);
        const float4 u = __ldg(p), v = __ldg(p + 1);
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
        const uint4 w = ldg_nc_v4(static_cast<const uint16_t *>(q) + i);
        x[0] = bf_lo(w.x); x[1] = bf_hi(w.x); x[2] = bf_lo(w.y); x[3] = bf_hi(w.y);
        x[4] = bf_lo(w.z); x[5] = bf_hi(w.z); x[6] = bf_lo(w.w); x[7] = bf_hi(w.w);
    }
}

// Where split s of a list of n begins, in units of `unit` positions.  The list
// is cut into at most S splits of at least `least`.  Where the launch has more
// CTAs than run at once (`guided`) the cuts are at n (1 - (1 - s/S)^2), each
// split smaller than the one before it: CTAs are launched in order of s, so the
// long splits of all sequences go first and the short ones fill the device's
// slots as they fall free (equal splits left 16% of it idle at the end of a
// launch of ragged sequences).  Where all run at once the longest sets the time,
// and splits are equal.
__device__ __forceinline__ int split_at(int n, int s, int S, int least, bool guided, int unit)
{
    S = min(S, (n + least - 1) / least);
    if (s <= 0) return 0;
    if (s >= S) return n;
    // (fp32: only the order of the boundaries matters, and rounding keeps it)
    float left = (float)(S - s) / (float)S;
    if (guided) left *= left;
    return n - min(n, ((int)((float)n * left) + unit - 1) & ~(unit - 1));
}

// Columns c .. c + 3 of an output row from its whole state
__device__ __forceinline__ void finish(const DecodeArgs &a, size_t row, int D, int c, float M, float Ls, const float4 &O)
{
    const bool some = Ls != 0.f;
    const float f = some ? 1.f / Ls : 0.f;
    const __nv_bfloat162 u = __floats2bfloat162_rn(O.x * f, O.y * f), v = __floats2bfloat162_rn(O.z * f, O.w * f);
    *reinterpret_cast<uint2 *>(a.out + row * D + c) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
    if (a.lse && c == 0) a.lse[row] = some ? (M + log2f(Ls)) * kLn2 : -INFINITY;
}

// CTAs an SM holds (by registers; 4 of the token lists' fit with 128)
template <int NH, bool QF32, bool TOKENS>
constexpr int kOcc = NH == 1 ? (TOKENS && !QF32 ? 4 : 3) : 2;

// NH = 8-head column blocks of the CTA (1 or 2); TOKENS: one query head and
// its token list, else a kv head's heads and the sequence's block list; PACK: at
// most 4 heads, which stand in columns 0-3 for one 16-row tile and again in 4-7
// for the other, so that the softmax of both fills the 8 columns
template <int D, int NH, bool QF32, bool TOKENS, bool PACK>
__global__ void __launch_bounds__(kDThreads, kOcc<NH, QF32, TOKENS>) k_decode_kv4(const DecodeArgs a)
{
    pdl_wait();
    pdl_trigger();
    using SM = DSmem<D>;
    constexpr int REC = Kv4<D>::REC;
    constexpr int CB = D / 32;           // 16-byte column blocks of a row's codes (32 channels each)
    constexpr int CBH = CB / 2;          // of a half
    constexpr int TT = NH == 1 ? 2 : 1;  // 16-row tiles at a time
    constexpr int NQ = QF32 ? 2 : 1;     // fp16 parts of the query
    constexpr int TS = PACK ? 1 : TT;    // tiles whose softmax a lane does
    extern __shared__ __align__(128) uint8_t sm[];
    const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(sm);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gq = lane >> 2, tq = lane & 3;   // mma group id / thread in group
    const int own = PACK ? tq >> 1 : 0;        // PACK: the tile whose scores are in this lane's columns
    const int s = blockIdx.z, b = blockIdx.y;
    const int HPG = a.Hq / a.c.Hkv;
    const int hblocks = (HPG + 15) / 16;
    const int g = TOKENS ? blockIdx.x / HPG : blockIdx.x / hblocks;
    const int h0 = TOKENS ? blockIdx.x : g * HPG + (blockIdx.x % hblocks) * 16;   // first query head
    const int nheads = TOKENS ? 1 : min(16, (g + 1) * HPG - h0);
    const uint8_t *pool = reinterpret_cast<const uint8_t *>(a.c.k);
    DevStatus *st = a.st;
    const bool reports = s == 0 && tid == 0;

    // the query's channels first: they wait on nothing (column n is head h0 + n)
    float qx[NH][CB][8];
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        const int h = nh * 8 + (PACK ? gq & 3 : gq);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
#pragma unroll
            for (int i = 0; i < 8; ++i) qx[nh][cb][i] = 0.f;
            if (h < nheads) query8<QF32>(a.q, ((size_t)b * a.Hq + h0 + h) * D + cb * 32 + tq * 8, qx[nh][cb]);
        }
    }
    // (both lengths in one trip, before either is looked at)
    const int Lcap = a.c.max_pages << a.c.Plog2;
    int L = __ldg(a.c.sl + b), n = TOKENS ? __ldg(a.cnt + (size_t)b * a.Hq + h0) : __ldg(a.ecnt + b);
    if (L < 0 || L > Lcap) {
        if (reports) fault(st, CHK_SEQ_LEN, L);
        L = L < 0 ? 0 : Lcap;
    }
    const bool guided = (unsigned long long)gridDim.x * gridDim.y * gridDim.z > 148 * kOcc<NH, QF32, TOKENS>;
    // this split's range [lo, hi) of list positions (tokens) or entries (blocks)
    int lo, hi;
    const int *pt = a.c.pt + (size_t)b * a.c.max_pages;
    const int4 *ent = nullptr;
    const int *idx = nullptr;
    if (TOKENS) {
        const size_t r = (size_t)b * a.Hq + h0;
        if (n < 0 || n > a.kcap) {
            if (reports) fault(st, CHK_COUNT, n);
            n = n < 0 ? 0 : a.kcap;
        }
        idx = a.idx + r * a.kcap;
        lo = split_at(n, s, a.S, kLeast, guided, kDR);
        hi = split_at(n, s + 1, a.S, kLeast, guided, kDR);
    } else {
        if (n < 0 || n > a.max_blocks) {
            if (reports) fault(st, CHK_BLOCK_ENTRY, n);
            n = n < 0 ? 0 : a.max_blocks;
        }
        ent = reinterpret_cast<const int4 *>(a.ent) + (size_t)b * a.max_blocks;
        lo = split_at(n, s, a.S, kLeast >> a.c.Plog2, guided, 1);
        hi = split_at(n, s + 1, a.S, kLeast >> a.c.Plog2, guided, 1);
    }
    // what this CTA has of 4 columns of an output row: the output itself where there
    // is one split, else a part for the combine kernel
    auto leave = [&](int j, int c, float M, float Ls, const float4 &O) {
        const size_t row = (size_t)b * a.Hq + h0 + j;
        if (a.S == 1) {
            finish(a, row, D, c, M, Ls, O);
            return;
        }
        *reinterpret_cast<float4 *>(a.part_o + (row * a.S + s) * D + c) = O;
        if (c == 0) {
            a.part_ml[(row * a.S + s) * 2 + 0] = M;
            a.part_ml[(row * a.S + s) * 2 + 1] = Ls;
        }
    };
    if (lo >= hi) {   // nothing for this split (the combine skips an empty part's output)
        const int per = a.S == 1 ? D / 4 : 1;
        for (int i = tid; i < nheads * per; i += kDThreads)
            leave(i / per, i % per * 4, -INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }

    // query B fragments: the k-steps' channels follow the order in which widen() hands out a code word (channels i and i + 4)
    uint32_t qb[NQ][NH][CB][2][2];
    constexpr float kWhole = 12582912.f;   // 1.5 * 2^23
    constexpr bool BF = !QF32;             // type of the products with keys
    constexpr int kTop = BF ? 118 : 10;    // the scaled query's largest element is in [2^kTop, 2^(kTop + 1))
    constexpr int kUnit = BF ? 133 : 24;   // a code c stands as c 2^-kUnit
    float qs[2][NH][2];   // 2^-kUnit sum of the scaled query over each half, heads nh*8 + 2tq + j
    float kf[NH][2];      // scores' factor of those heads: 2^kUnit scale log2(e) / the query's power of two
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        float top = 0.f;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(qx[nh][cb][i]));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const float up = pow2(kTop - exponent(top));
#pragma unroll
        for (int j = 0; j < 2; ++j) kf[nh][j] = a.qscale * pow2(kUnit - kUnit / 2) * (pow2(kUnit / 2) / __shfl_sync(~0u, up, (2 * tq + j) * 4));
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = (i & 1) ? 0.0625f : 1.f;   // odd nibbles stand for 16 c
                float y = qx[nh][cb][i] * up, z = qx[nh][cb][i + 4] * up;
                if (QF32) {
                    const float u = y + kWhole - kWhole, v = z + kWhole - kWhole;   // to whole numbers
                    qb[0][nh][cb][i >> 1][i & 1] = pack_pair<BF>(u * f, v * f);
                    y -= u;
                    z -= v;
                }
                qb[NQ - 1][nh][cb][i >> 1][i & 1] = pack_pair<BF>(y * f, z * f);
            }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float sum[2][4] = {};   // (of the parts on their own, as the scores below)
#pragma unroll
            for (int cb = half * CBH; cb < (half + 1) * CBH; ++cb)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int qi = 0; qi < NQ; ++qi)
                        mma<BF>(sum[qi], kOnes<BF>, kOnes<BF>, kSixteens<BF>, kSixteens<BF>, qb[qi][nh][cb][ks][0],
                                qb[qi][nh][cb][ks][1]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                qs[half][nh][j] = (sum[0][j] + sum[1][j]) * pow2(-(kUnit / 2)) * pow2(-(kUnit - kUnit / 2));
        }
    }
    // O^T fragments: o[cb][j][nh]: rows gq / gq + 8 are channels cb*32 + 4gq + 2j / + 1, columns heads 2tq, 2tq + 1
    float o[CB][2][NH][4];
    float zs[2][NH][2];            // sum of p z per half, this thread's tokens
    float mh[NH][2], lh[NH][2];    // heads nh*8 + 2tq + j (l: this thread's tokens)
    float mz[NH][2];               // mh, 0 for a head without a score
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int j = 0; j < 2; ++j) o[cb][j][nh][0] = o[cb][j][nh][1] = o[cb][j][nh][2] = o[cb][j][nh][3] = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) zs[half][nh][0] = zs[half][nh][1] = 0.f;
        mh[nh][0] = mh[nh][1] = -INFINITY;
        mz[nh][0] = mz[nh][1] = 0.f;
        lh[nh][0] = lh[nh][1] = 0.f;
    }

    // per half: the largest value scale that fits, and the power of two p s is kept at
    float smax[2] = {pow2(-100), pow2(-100)}, keep[2] = {pow2(107), pow2(107)};

    uint8_t *ring = sm + warp * kDST * SM::STAGE;
    const uint32_t ring_a = sbase + warp * kDST * SM::STAGE;

    // TT * 16 rows (those in `mask`) at byte `at` of the ring.  The tiles are
    // independent up to the running sums, so with a group's 8 heads two at a
    // time hide each other's latencies.
    const uint32_t quad0 = ring_a + ((lane & 7) + ((lane >> 3) & 1) * 8) * REC + (lane >> 4) * 16;
    auto consume = [&](int at, uint32_t mask) {
        const bool partial = mask != (TT == 2 ? 0xffffffffu : 0xffffu);
        // scales and zeros {K half 0, K half 1, V half 0, V half 1} of rows gq, gq + 8; a row
        // outside the mask is whatever the stage held, and must not reach a product
        uint4 par[TS][2];
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = (t + own) * 16 + r * 8 + gq;
                par[t][r] = *reinterpret_cast<const uint4 *>(ring + at + row * REC + Kv4<D>::PAR);
                if (partial && !((mask >> row) & 1)) par[t][r] = make_uint4(0, 0, 0, 0);
            }

        // ---- S^T = K Q^T per half
        float sc[TT][2][NH][4];
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int c2 = 0; c2 < CB; c2 += 2) {
                // matrices: rows 0-7 / 8-15 of column block c2, then of c2 + 1
                uint32_t w[4];
                float low[NH][4];   // QF32: the sums of the query's second part
                ldsm4(quad0 + at + t * 16 * REC + c2 * 16, w);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t f0[4], f1[4];
                    widen(w[2 * u], f0);
                    widen(w[2 * u + 1], f1);
                    const int cb = c2 + u, half = cb / CBH;
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                            for (int qi = 0; qi < NQ; ++qi) {
                                float(&sum)[4] = qi ? low[nh] : sc[t][half][nh];
                                if (cb == half * CBH && ks == 0)
                                    mma0<BF>(sum, f0[0], f1[0], f0[1], f1[1], qb[qi][nh][cb][0][0],
                                             qb[qi][nh][cb][0][1]);
                                else
                                    mma<BF>(sum, f0[2 * ks], f1[2 * ks], f0[2 * ks + 1], f1[2 * ks + 1],
                                            qb[qi][nh][cb][ks][0], qb[qi][nh][cb][ks][1]);
                            }
                    if (QF32 && cb + 1 == (half + 1) * CBH) {
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                            for (int i = 0; i < 4; ++i) sc[t][half][nh][i] += low[nh][i];
                    }
                }
            }
        if (PACK) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[0][half][0][i] = own ? sc[TT - 1][half][0][i] : sc[0][half][0][i];
        }
        // ---- scores: rows gq (elements 0, 1) and gq + 8 (2, 3), base-2 domain
        float x[TS][NH][4], above = -INFINITY, vs[2] = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 &p = par[t][r];
                const float s0 = bf_lo(p.x), s1 = bf_lo(p.y);
                const float c0 = bf_hi(p.x), c1 = bf_hi(p.y);
                vs[0] = fmaxf(vs[0], bf_lo(p.z));
                vs[1] = fmaxf(vs[1], bf_lo(p.w));
#pragma unroll
                for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        x[t][nh][2 * r + j] = kf[nh][j] * fmaf(s0, sc[t][0][nh][2 * r + j],
                                                               fmaf(s1, sc[t][1][nh][2 * r + j],
                                                                    fmaf(c0, qs[0][nh][j], c1 * qs[1][nh][j])));
            }
        if (partial) {
#pragma unroll
            for (int t = 0; t < TS; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (!((mask >> ((t + own) * 16 + r * 8 + gq)) & 1)) {
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh) x[t][nh][2 * r] = x[t][nh][2 * r + 1] = -INFINITY;
                    }
        }
        // (the difference is +inf for the first score of a head, NaN, which
        // compares false, while it has none)
        float top[NH][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                top[nh][j] = fmaxf(x[0][nh][j], x[0][nh][2 + j]);
                if (TS == 2) top[nh][j] = fmaxf(top[nh][j], fmaxf(x[TS - 1][nh][j], x[TS - 1][nh][2 + j]));
                above = fmaxf(above, top[nh][j] - mh[nh][j]);
            }
        if (__any_sync(~0u, above > kLazy || vs[0] > smax[0] || vs[1] > smax[1])) {
            float re[2] = {1.f, 1.f};   // what the halves' sums are rescaled by
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float m = vs[half];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, off));
                if (m > smax[half]) {
                    const int e = exponent(m) + 1;   // m < 2^e
                    smax[half] = e > 127 ? INFINITY : pow2(e);
                    const float was = keep[half];
                    keep[half] = pow2(7 - e);
                    re[half] = keep[half] / was;
                }
            }
#pragma unroll
            for (int nh = 0; nh < NH; ++nh)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float m = fmaxf(mh[nh][j], top[nh][j]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, off));
                    const float al = m == -INFINITY ? 1.f : ex2(mh[nh][j] - m);   // 0 for a head that was empty
                    mh[nh][j] = m;
                    mz[nh][j] = m == -INFINITY ? 0.f : m;
                    lh[nh][j] *= al;
                    zs[0][nh][j] *= al;
                    zs[1][nh][j] *= al;
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            o[cb][i][nh][j] *= al * re[cb / CBH];
                            o[cb][i][nh][2 + j] *= al * re[cb / CBH];
                        }
                }
        }
        // ---- weights; P'^T (tokens x heads) per half as B fragments (k = tokens)
        uint32_t pb[TT][2][NH][2];
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 &pr = par[t][r];
                const float v0 = bf_lo(pr.z), v1 = bf_lo(pr.w);
                const float w0 = v0 * keep[0], w1 = v1 * keep[1];
                const float z0 = bf_hi(pr.z), z1 = bf_hi(pr.w);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) {
                    float p[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        p[j] = ex2(x[t][nh][2 * r + j] - mz[nh][j]);
                        lh[nh][j] += p[j];
                        zs[0][nh][j] = fmaf(p[j], z0, zs[0][nh][j]);
                        zs[1][nh][j] = fmaf(p[j], z1, zs[1][nh][j]);
                    }
                    pb[t][0][nh][r] = movm(pack_pair(p[0] * w0, p[1] * w0));
                    pb[t][1][nh][r] = movm(pack_pair(p[0] * w1, p[1] * w1));
                }
            }
        if (PACK) {   // each tile's own columns
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    pb[TT - 1][half][0][r] = gq < 4 ? 0u : pb[0][half][0][r];
                    pb[0][half][0][r] = gq < 4 ? pb[0][half][0][r] : 0u;
                }
        }
        // ---- O^T += V^T P'^T: transposed 8x8 loads of the code bytes give, per
        // register, 4 channels of tokens 2tq (low half) and 2tq + 1 (high half)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int c2 = 0; c2 < CB; c2 += 2) {
                uint32_t w[4];
                ldsm4_t(quad0 + at + t * 16 * REC + Kv4<D>::V + c2 * 16, w);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t f0[4], f1[4];
                    widen_bytes(w[2 * u], f0);
                    widen_bytes(w[2 * u + 1], f1);
                    const int cb = c2 + u, half = cb / CBH;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int nh = 0; nh < NH; ++nh)
                            mma<false>(o[cb][j][nh], f0[2 * j], f0[2 * j + 1], f1[2 * j], f1[2 * j + 1], pb[t][half][nh][0],
                                pb[t][half][nh][1]);
                }
            }
    };
    constexpr uint32_t kNone = 0xffffffffu;
    // ring step g: its mask is kept by lane g % kDST
    uint32_t held = 0;
    auto hold = [&](int stage, uint32_t mask) {
        copies_commit();
        if (lane == stage) held = mask;
    };
    // consumes `steps` stages that issue(step, stage) starts, in order
    auto stream = [&](int steps, auto &&issue) {
        int fill = 0;
#pragma unroll 1
        for (; fill < kDST; ++fill) {
            if (fill < steps) issue(fill, fill);
            else hold(fill, 0);
        }
        int stage = 0;
#pragma unroll 1
        for (int n = 0; n < steps; ++n) {
            copies_wait<kDST - 1>();
            __syncwarp();   // every lane's copies of this stage are there
            const uint32_t mask = __shfl_sync(~0u, held, stage);
#pragma unroll 1
            for (int t = 0; t < 2; t += TT) {
                const uint32_t m = TT == 2 ? mask : t ? mask >> 16 : mask & 0xffffu;
                if (m) consume(stage * SM::STAGE + t * 16 * REC, m);
            }
            __syncwarp();   // every lane is done with this stage before it is refilled
            if (n + kDST < steps) issue(n + kDST, stage);
            else hold(stage, 0);
            stage = stage + 1 == kDST ? 0 : stage + 1;
        }
    };

    if (TOKENS) {
        // step n: list positions lo + (n * kDW + warp) * 32 + lane
        constexpr int PARTS = REC / 16, ROWS = 32 / PARTS;   // lanes of a row, rows of an instruction
        const int part = lane % PARTS, sub = lane / PARTS;
        const int first = lo + warp * kDR + lane;
        const int steps = max(0, (hi - lo - warp * kDR + kDR * kDW - 1) / (kDR * kDW));
        auto index_at = [&](int n) -> int {
            const int i = first + n * kDR * kDW;
            return i < hi ? __ldg(idx + i) : -1;
        };
        // page of token t, -1 without one (recorded)
        auto page_of = [&](int n, int t) -> int {
            if (first + n * kDR * kDW >= hi) return -1;
            if (t < 0 || t >= L) {
                fault(st, CHK_INDEX, t);
                return -1;
            }
            return __ldg(pt + (t >> a.c.Plog2));
        };
        int t0 = index_at(0), t1 = index_at(1);
        int page = page_of(0, t0);
        stream(steps, [&](int n, int stage) {
            uint32_t row = kNone;
            if (first + n * kDR * kDW < hi && t0 >= 0 && t0 < L) {
                if (page < 0 || page >= a.c.num_pages) fault(st, CHK_PAGE, page);
                else row = (((uint32_t)page * a.c.Hkv + g) << a.c.Plog2) + (t0 & ((1 << a.c.Plog2) - 1));
            }
            t0 = t1;
            page = page_of(n + 1, t0);
            t1 = index_at(n + 2);
            const uint32_t mask = __ballot_sync(~0u, row != kNone);
            const uint32_t dst = ring_a + stage * SM::STAGE + part * 16;
#pragma unroll
            for (int i = 0; i < (kDR + ROWS - 1) / ROWS; ++i) {
                const int r = i * ROWS + sub;
                const uint32_t from = __shfl_sync(~0u, row, r & 31);
                if (sub < ROWS && r < kDR && from != kNone)
                    copy16(dst + r * REC, pool + (size_t)from * REC + part * 16);
            }
            hold(stage, mask);
        });
    } else {
        // the warp's entries lo + warp + kDW * j, a window of 32 (one per lane)
        // at a time.  A step is 32 rows of an entry of a 64-token page, or two
        // entries of 16-token pages, 16 rows each.
        const bool small = a.c.Plog2 == 4;
        const int mine = (hi - lo - warp + kDW - 1) / kDW;   // entries of this warp (0 or more)
        const int steps = small ? (mine + 1) / 2 : 2 * mine;
        auto entry_at = [&](int w) -> int4 {
            const int j = w * 32 + lane;
            return j < mine ? ent[lo + warp + kDW * j] : make_int4(0, 0, 0, 0);
        };
        // page of an entry, -1 for one that is malformed (recorded)
        auto page_of = [&](int w, const int4 &en) -> int {
            if (w * 32 + lane >= mine) return -1;
            if (en.y < 0 || en.y >= en.z || en.z > (1 << a.c.Plog2) || en.x < 0 || en.x >= a.c.max_pages) {
                fault(st, CHK_BLOCK_ENTRY, lo + warp + kDW * (w * 32 + lane));
                return -1;
            }
            if ((en.x << a.c.Plog2) + en.z > L) {
                fault(st, CHK_INDEX, (en.x << a.c.Plog2) + en.z - 1);
                return -1;
            }
            const int page = __ldg(pt + en.x);
            if (page < 0 || page >= a.c.num_pages) {
                fault(st, CHK_PAGE, page);
                return -1;
            }
            return page;
        };
        uint32_t row = 0;   // of this lane's entry of the window: its first row
        int len = 0;        // and its rows
        int4 e1 = make_int4(0, 0, 0, 0);
        if (steps > 0) e1 = entry_at(0);
        const int log_spw = small ? 4 : 6;   // log2 of steps per window
        stream(max(steps, 0), [&](int n, int stage) {
            const int w = n >> log_spw, i = n & ((1 << log_spw) - 1);
            if (i == 0) {
                const int page = page_of(w, e1);
                len = page < 0 ? 0 : e1.z - e1.y;
                row = (((uint32_t)max(page, 0) * a.c.Hkv + g) << a.c.Plog2) + e1.y;
                e1 = entry_at(w + 1);
            }
            // rows 0-15 and 16-31 of the step: where they come from, how many
            const int src = small ? 2 * i : i >> 1, skip = small ? 0 : (i & 1) * kDR;
            const int la = __shfl_sync(~0u, len, src) - skip, lb = small ? __shfl_sync(~0u, len, src + 1) : la - 16;
            const uint32_t ra = __shfl_sync(~0u, row, src) + skip, rb = small ? __shfl_sync(~0u, row, src + 1) : ra + 16;
            const int na = min(max(la, 0), 16), nb = min(max(lb, 0), 16);
            const uint32_t dst = ring_a + stage * SM::STAGE + lane * 16;
            const uint8_t *pa = pool + (size_t)ra * REC + lane * 16, *pb = pool + (size_t)rb * REC + lane * 16 - 16 * REC;
            constexpr int COPIES = kDR * REC / 512;   // 512 bytes an instruction (REC is a multiple of 16)
            if (na == 16 && nb == 16) {
#pragma unroll
                for (int c = 0; c < COPIES; ++c)
                    copy16(dst + c * 512, (c * 512 + lane * 16 >= 16 * REC ? pb : pa) + c * 512);
            } else {
                const int ea = na * REC, eb = (16 + nb) * REC;
#pragma unroll 1
                for (int c = 0; c < COPIES; ++c) {
                    const int at = c * 512 + lane * 16;
                    const bool second = at >= 16 * REC;
                    if (at < (second ? eb : ea)) copy16(dst + c * 512, (second ? pb : pa) + c * 512);
                }
            }
            hold(stage, ((1u << na) - 1u) | (((1u << nb) - 1u) << 16));
        });
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
    constexpr int ROW = SM::ROW;
    float *mo = reinterpret_cast<float *>(sm);                 // [warp][16][ROW]
    float *mm = mo + kDW * 16 * ROW;                            // [warp][16]
    float *ml = mm + kDW * 16;                                  // [warp][16]
    // (a token list has one head, columns 0 and 4)
    if (!TOKENS || (tq & 1) == 0) {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                for (int i = 0; i < (TOKENS ? 1 : 2); ++i) {
                    // channels 4gq .. 4gq + 3 of block cb; the odd ones (rows gq + 8) went in as
                    // 16 c and the even one's code
                    const int half = cb / CBH;
                    const float f = 16777216.f / keep[half], odd = f * 0.0625f, z = zs[half][nh][i];
                    *reinterpret_cast<float4 *>(mo + (warp * 16 + nh * 8 + 2 * tq + i) * ROW + cb * 32 + 4 * gq) =
                        make_float4(fmaf(o[cb][0][nh][i], f, z), fmaf(o[cb][0][nh][2 + i] - o[cb][0][nh][i], odd, z),
                                    fmaf(o[cb][1][nh][i], f, z), fmaf(o[cb][1][nh][2 + i] - o[cb][1][nh][i], odd, z));
                }
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
    for (int i = tid; i < nheads * (D / 4); i += kDThreads) {
        const int j = i / (D / 4), c = i % (D / 4) * 4;
        constexpr int PARTS = PACK ? 2 : 1;   // columns of a head
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kDW * PARTS; ++w) M = fmaxf(M, mm[w / PARTS * 16 + w % PARTS * 4 + j]);
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        float Ls = 0.f;
#pragma unroll
        for (int w = 0; w < kDW * PARTS; ++w) {
            const int at = w / PARTS * 16 + w % PARTS * 4 + j;
            const float lw = ml[at];
            if (lw == 0.f) continue;   // no token (a sum that is not a number is taken along)
            const float wgt = ex2(mm[at] - M);
            const float4 x = *reinterpret_cast<const float4 *>(mo + at * ROW + c);
            O.x = fmaf(wgt, x.x, O.x);
            O.y = fmaf(wgt, x.y, O.y);
            O.z = fmaf(wgt, x.z, O.z);
            O.w = fmaf(wgt, x.w, O.w);
            Ls = fmaf(wgt, lw, Ls);
        }
        leave(j, c, M, Ls, O);
    }
}

// Merge of the splits, as k_decode_combine, except that a split whose sum is
// not a number (a selected row was stored as NaN) makes the result NaN.
// (Joined by a cluster of the splits in the first kernel instead, a masked
// step took 13.2 us and not 11.8: CTAs of a cluster start and end together.)
template <int D>
__global__ void __launch_bounds__(128) k_kv4_combine(const DecodeArgs a, int rows)
{
    pdl_wait();
    pdl_trigger();
    constexpr int LANES = D / 4;   // of a row
    const int r = blockIdx.x * (128 / LANES) + threadIdx.x / LANES, c = threadIdx.x % LANES * 4;
    if (r >= rows) return;
    const size_t row = r;
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + row * a.S;
    const float *po = a.part_o + row * a.S * D + c;
    // 8 splits at a time, states and outputs in one trip (an empty split's output
    // is whatever the workspace held, and is not looked at)
    float M = -INFINITY, Ls = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < a.S; s0 += 8) {
        float2 x[8];
        float4 v[8];
        float top = M;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            x[u] = make_float2(-INFINITY, 0.f);
            if (s0 + u < a.S) {
                x[u] = ml[s0 + u];
                v[u] = *reinterpret_cast<const float4 *>(po + (size_t)(s0 + u) * D);
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (x[u].y != 0.f) top = fmaxf(top, x[u].x);
        const float al = top == M ? 1.f : ex2(M - top);
        M = top;
        Ls *= al;
        O.x *= al;
        O.y *= al;
        O.z *= al;
        O.w *= al;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (x[u].y == 0.f) continue;
            const float w = ex2(x[u].x - M);
            Ls = fmaf(w, x[u].y, Ls);
            O.x = fmaf(w, v[u].x, O.x);
            O.y = fmaf(w, v[u].y, O.y);
            O.z = fmaf(w, v[u].z, O.z);
            O.w = fmaf(w, v[u].w, O.w);
        }
    }
    finish(a, row, D, c, M, Ls, O);
}

template <int D, int NH, bool QF32, bool TOKENS, bool PACK>
cudaError_t launch_kv4(const DecodeArgs &a, cudaStream_t s)
{
    constexpr int smem = DSmem<D>::BYTES;
    auto kern = k_decode_kv4<D, NH, QF32, TOKENS, PACK>;
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
    const int hpg = a.Hq / a.c.Hkv;
    const dim3 grid((unsigned)(TOKENS ? a.Hq : a.c.Hkv * ((hpg + 15) / 16)), (unsigned)a.c.B, (unsigned)a.S);
    if (cudaError_t e = launch_pdl(kern, grid, dim3(kDThreads), smem, s, a)) return e;
    if (a.S == 1) return cudaSuccess;
    const int rows = a.c.B * a.Hq, per = 128 / (D / 4);
    return launch_pdl(k_kv4_combine<D>, dim3((unsigned)((rows + per - 1) / per)), dim3(128), 0, s, a, rows);
}

template <int D, bool QF32>
cudaError_t launch_kind(const DecodeArgs &a, cudaStream_t s)
{
    if (!a.blocks) return launch_kv4<D, 1, QF32, true, true>(a, s);
    const int hpg = a.Hq / a.c.Hkv;
    return hpg <= 4   ? launch_kv4<D, 1, QF32, false, true>(a, s)
           : hpg <= 8 ? launch_kv4<D, 1, QF32, false, false>(a, s)
                      : launch_kv4<D, 2, QF32, false, false>(a, s);
}

}  // namespace

// The split count that a simple model of the launch finds fastest.  A CTA costs
// `start` beside `each` a token when its SM is full, less when it is not; CTAs
// that all run at once take as long as one of the longest row, more of them fill
// the slots with falling sizes (split_at), the first of which must fit in as well,
// and leave a tail.  The rule sees the lists' capacity alone, not what they hold:
// a capacity far above that costs splits (a masked step of 4 sequences with 8 groups:
// 10.2 us with the 256 entries it needs, 13.3 with the 8194 of its whole context).
//
// `filled`, what a batch's block lists hold of it on average, stands between
// sequences of one length and ragged ones, because a count chosen for the one must not
// be bad for the other.  Measured over batches of equal lengths, of lengths spread
// over a factor of 2 and of lengths spread evenly from 2% up: with 1.0 the chosen
// counts are up to 23%, 47% and 73% slower than the best of each batch, with 0.76
// 7%, 5% and 18%.  Times (us, head_dim 128) of equal | ragged | evenly spread
// lengths, * the chosen count:
//   32 x 8 groups (4 heads) of 16384     4*, 6, 8         107 107 113 | 85 84 87 | 68 64 66
//   16 x 8 groups (8 heads) of 16384     3, 5, 8*, 10     69 66 64 65 | 66 62 54 56 | 58 52 41 40
//   16 x 2 groups (8) of 65536           13, 24, 32*      66 70 67 | 63 57 56 | 55 49 43
//   32 x 4 groups (8) of 16384           3, 5, 8*, 10     69 66 64 65 | 66 61 52 54 | 63 56 42 43
//    8 x 4 groups (12) of 65536          10, 16, 20, 22*  136 97 101 104 | 135 90 81 82 | 129 88 74 70
//  128 x 8 groups (4) of 4096            1*, 2, 3         104 111 123 | 93 91 97 | 70 68 75
//   64 x 8 groups (4) of 4096            1, 2*, 3         65 59 63 | 59 51 52 | 43 39 41
//    4 x 8 groups (8) of 32768           8, 13*, 24, 32   40 38 42 41 | 40 37 36 37 | 40 36 32 31
// and of lists of one sequence, and token lists:
//    1 x 8 groups of 131072 tokens       24, 37, 55, 64   41, 37, 37, 42
//    4 x 8 groups of a masked step       4, 8*, 13        11.9, 10.2, 12.2
//   32 x 32 lists of 4096 tokens         1, 2*, 3, 4      150, 141, 144, 151
//    8 x 32 lists of 2048 tokens         1, 2*, 3, 4      34, 27, 26, 27
int decode_kv4_splits(int B, int rows, long long list, int D, bool tokens, bool f32, bool wide)
{
    const double units = (double)B * rows, start = 4.0;
    if (units <= 0 || list <= 0) return 1;
    const double slots = 148.0 * (wide ? 2 : tokens && !f32 ? 4 : 3);
    const double each = (tokens ? 0.0176 : wide ? 0.013 : 0.0095) * (D + 32) / 160;
    const double filled = tokens || B == 1 ? 1.0 : 0.76;
    int best = 1;
    double least = 0;
    for (int S = 1; S <= 64; ++S) {
        const double n = (double)list / S, ctas = units * S;
        if (S > 1 && n < kLeast) break;
        double t;
        if (ctas <= slots) {
            t = start + each * n * (0.3 + 0.7 * ctas / slots);
        } else {
            const double first = start + each * list * (2.0 * S - 1) / ((double)S * S);
            t = (ctas * start + filled * units * list * each) / slots;
            t = (t > first ? t : first) + start + each * n / (4 * S);
        }
        if (S > 1) t += 1.2 + (S + 7) / 8;   // the combine: a trip to memory for 8 splits
        if (S == 1 || t < least) {
            least = t;
            best = S;
        }
    }
    return best;
}

cudaError_t launch_decode_kv4(const DecodeArgs &a, cudaStream_t s)
{
    if (a.c.B * a.Hq == 0) return cudaSuccess;
    if (a.c.D == 64) return a.q_f32 ? launch_kind<64, true>(a, s) : launch_kind<64, false>(a, s);
    return a.q_f32 ? launch_kind<128, true>(a, s) : launch_kind<128, false>(a, s);
}

}  // namespace sa
