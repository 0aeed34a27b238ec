// Pages of a 4-bit cache back to bf16 pages.
//
// value = zero + scale * code (kv4.cuh), rounded once to bf16: one bf16 fma of
// the code as a bf16 number.  The selections and
// the block-sparse prefill read bf16 pages ("RBS-Attention…", 关键技术点 2: the
// selection feeds an unchanged block-sparse path); a context held in 4 bits is
// expanded for them page by page.
//
// One thread turns a 4-byte code word into 8 channels (one 16-byte store), so
// a warp writes whole rows; D + 16 bytes are read and 4 D written per record.
// kUnroll words a thread are in flight.  Bound by HBM: 2048 pages of 64 tokens
// and 4 kv heads (344 MB) 59.7 us, 0.88 of it; with codes converted to fp32 one
// by one and one word a thread it was 71.7 us (integer pipe 65% busy).
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sa {
namespace {

constexpr int kExpandThreads = 256, kUnroll = 4;

template <int D>
__global__ void __launch_bounds__(kExpandThreads) k_kv4_expand(const ExpandArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int WPR = D / 4;   // code words of a record: D/8 of the key, then D/8 of the value
    const int i = blockIdx.x;
    const int page = a.pages[i];
    if (page < 0 || page >= a.num_pages) {
        if (threadIdx.x == 0 && blockIdx.y == 0 && page != -1) fault(a.st, CHK_PAGE, page);
        return;
    }
    const int rows = a.Hkv << a.Plog2, words = rows * WPR;
    const uint8_t *src = a.kv4 + (size_t)page * rows * Kv4<D>::REC;
    const size_t dst = (size_t)i * rows * D;
    const __nv_bfloat162 off = __halves2bfloat162(__ushort_as_bfloat16(0xc300), __ushort_as_bfloat16(0xc300));   // -128
    const int w0 = blockIdx.y * kExpandThreads * kUnroll + threadIdx.x;
    uint32_t codes[kUnroll], par[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int w = w0 + u * kExpandThreads;
        codes[u] = par[u] = 0;
        if (w < words) {
            const int row = w / WPR, j = w % WPR;
            const uint8_t *rec = src + (size_t)row * Kv4<D>::REC;
            codes[u] = *reinterpret_cast<const uint32_t *>(rec + j * 4);
            par[u] = *reinterpret_cast<const uint32_t *>(rec + Kv4<D>::PAR + j / (WPR / 4) * 4);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int w = w0 + u * kExpandThreads;
        if (w >= words) break;
        const int row = w / WPR, j = w % WPR;
        const uint32_t s2 = __byte_perm(par[u], 0, 0x1010), z2 = __byte_perm(par[u], 0, 0x3232);
        const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162 *>(&s2);
        const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162 *>(&z2);
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // channels 2e, 2e + 1: their nibbles into the mantissas of 128.0, less 128
            const uint32_t x = codes[u] >> (8 * e);
            const uint32_t c = (x & 15u) | ((x & 240u) << 12) | 0x43004300u;
            const __nv_bfloat162 v = __hfma2(s, __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&c), off), z);
            o[e] = *reinterpret_cast<const uint32_t *>(&v);
        }
        const int side = j >= WPR / 2, jj = side ? j - WPR / 2 : j;
        *reinterpret_cast<uint4 *>((side ? a.v : a.k) + dst + (size_t)row * D + jj * 8) =
            make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

cudaError_t launch_expand(const ExpandArgs &a, cudaStream_t s)
{
    if (a.n == 0) return cudaSuccess;
    const int words = (a.Hkv << a.Plog2) * (a.D / 4);
    const dim3 grid((unsigned)a.n, (unsigned)((words + kUnroll * kExpandThreads - 1) / (kUnroll * kExpandThreads)));
    if (a.D == 64) return launch_pdl(k_kv4_expand<64>, grid, dim3(kExpandThreads), 0, s, a);
    return launch_pdl(k_kv4_expand<128>, grid, dim3(kExpandThreads), 0, s, a);
}

}  // namespace sa
