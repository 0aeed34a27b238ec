// Pages of a 4-bit cache back to bf16 pages.
//
// value = zero + scale * code (kv4.cuh), rounded to bf16.  The selections and
// the block-sparse prefill read bf16 pages ("RBS-Attention…", 关键技术点 2: the
// selection feeds an unchanged block-sparse path); a context held in 4 bits is
// expanded for them page by page.
//
// One thread turns a 4-byte code word into 8 channels (one 16-byte store), so
// a warp writes whole rows; D + 16 bytes are read and 4 D written per record.
// Bound by HBM writes.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sa {
namespace {

constexpr int kExpandThreads = 256;

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
    const int rows = a.Hkv << a.Plog2;
    const uint8_t *src = a.kv4 + (size_t)page * rows * Kv4<D>::REC;
    const size_t dst = (size_t)i * rows * D;
    for (int w = blockIdx.y * kExpandThreads + threadIdx.x; w < rows * WPR; w += gridDim.y * kExpandThreads) {
        const int row = w / WPR, j = w % WPR;
        const bool v = j >= WPR / 2;
        const int jj = v ? j - WPR / 2 : j;
        const uint8_t *rec = src + (size_t)row * Kv4<D>::REC;
        const uint32_t codes = *reinterpret_cast<const uint32_t *>(rec + j * 4);
        const uint32_t par = *reinterpret_cast<const uint32_t *>(rec + Kv4<D>::PAR + (v ? 8 : 0) + (jj >= WPR / 4 ? 4 : 0));
        const float s = bf_lo(par), z = bf_hi(par);
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float lo = fmaf(s, (float)((codes >> (8 * e)) & 15u), z);
            const float hi = fmaf(s, (float)((codes >> (8 * e + 4)) & 15u), z);
            const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
            o[e] = *reinterpret_cast<const uint32_t *>(&p);
        }
        uint16_t *out = (v ? a.v : a.k) + dst + (size_t)row * D + jj * 8;
        *reinterpret_cast<uint4 *>(out) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

cudaError_t launch_expand(const ExpandArgs &a, cudaStream_t s)
{
    if (a.n == 0) return cudaSuccess;
    const int words = (a.Hkv << a.Plog2) * (a.D / 4);
    const dim3 grid((unsigned)a.n, (unsigned)((words + 4 * kExpandThreads - 1) / (4 * kExpandThreads)));
    if (a.D == 64) return launch_pdl(k_kv4_expand<64>, grid, dim3(kExpandThreads), 0, s, a);
    return launch_pdl(k_kv4_expand<128>, grid, dim3(kExpandThreads), 0, s, a);
}

}  // namespace sa
