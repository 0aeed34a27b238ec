// C-ABI entry points of libsa: host-side argument validation, workspace
// layout and kernel launches.  Every check here runs before any launch, so a
// rejected call enqueues nothing.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "sa.h"
#include "sa_internal.h"

using namespace sa;

namespace sa {
// status header + split-KV partial outputs + (m, l) pairs, each rounded up to
// 256 bytes (the layout sa_sparse_decode_attn carves out of its workspace)
size_t decode_workspace_bytes(const sa_kv_cache *kv, int Hq, int S)
{
    const size_t rows = (size_t)kv->batch * Hq;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    return sizeof(DevStatus) + up(rows * S * kv->head_dim * sizeof(float)) + up(rows * S * 2 * sizeof(float));
}
}  // namespace sa

namespace {

constexpr size_t kAlign = 256;
constexpr size_t kHeader = sizeof(DevStatus);

inline size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int ilog2(int x)
{
    int r = 0;
    while ((1 << r) < x) ++r;
    return (1 << r) == x ? r : -1;
}

// Validate the cache descriptor (host-visible fields and pointers).
// pools = false: the call reads neither k nor v, which may then be null.
sa_status check_cache(const sa_kv_cache *kv, CacheArgs *c, bool pools = true)
{
    if (!kv) return SA_ERR_INVALID_ARGUMENT;
    if (kv->batch < 0 || kv->num_kv_heads <= 0 || kv->head_dim <= 0 || kv->page_size <= 0 ||
        kv->max_pages_per_seq < 0 || kv->num_pages < 0)
        return SA_ERR_INVALID_ARGUMENT;
    if (kv->head_dim != 64 && kv->head_dim != 128) return SA_ERR_UNSUPPORTED;
    if (kv->page_size != 16 && kv->page_size != 64) return SA_ERR_UNSUPPORTED;
    if ((long long)kv->max_pages_per_seq * kv->page_size > (1LL << 30)) return SA_ERR_UNSUPPORTED;
    if (kv->batch > 0) {
        if ((pools && (!kv->k || !kv->v)) || !kv->page_table || !kv->seq_lens) return SA_ERR_INVALID_ARGUMENT;
        if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->page_table, 4) ||
            !aligned(kv->seq_lens, 4))
            return SA_ERR_INVALID_ARGUMENT;
    }
    if (c) {
        c->k = static_cast<const uint16_t *>(kv->k);
        c->v = static_cast<const uint16_t *>(kv->v);
        c->pt = kv->page_table;
        c->sl = kv->seq_lens;
        c->B = kv->batch;
        c->Hkv = kv->num_kv_heads;
        c->D = kv->head_dim;
        c->P = kv->page_size;
        c->Plog2 = ilog2(kv->page_size);
        c->max_pages = kv->max_pages_per_seq;
        c->num_pages = kv->num_pages;
    }
    return SA_OK;
}

// A 4-bit cache, as the CacheArgs whose k is the records' pool.
sa_status check_cache4(const sa_kv4_cache *kv, CacheArgs *c)
{
    if (!kv) return SA_ERR_INVALID_ARGUMENT;
    const sa_kv_cache as = {kv->kv, kv->kv, kv->page_table, kv->seq_lens, kv->batch, kv->num_kv_heads,
                            kv->head_dim, kv->page_size, kv->max_pages_per_seq, kv->num_pages};
    sa_status st = check_cache(&as, c);
    if (st != SA_OK) return st;
    // the kernels number records with 32 bits, all ones meaning none
    if ((unsigned long long)kv->num_pages * kv->num_kv_heads * kv->page_size >= 0xffffffffull)
        return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

// CTAs per (sequence, split) of a block-list decode over a 4-bit cache
int kv4_group_rows(const sa_kv4_cache *kv, int Hq) { return kv->num_kv_heads * ((Hq / kv->num_kv_heads + 15) / 16); }

// Most splits that are chosen for a caller: 2400 CTAs of groups, which is past
// where more splits help, so that the workspace stays in proportion
int kv4_most_splits(const sa_kv4_cache *kv, int Hq)
{
    const long long units = (long long)kv->batch * kv4_group_rows(kv, Hq);
    const long long s = units > 0 ? (2400 + units - 1) / units : 1;
    return (int)(s > 64 ? 64 : s < 1 ? 1 : s);
}

// Fields of a decode that both cache kinds share, checked and set.
sa_status check_decode(int B, int Hkv, const void *q, sa_dtype q_dtype, int Hq, const sa_selection *sel, float scale,
                       const void *out, const float *lse, DecodeArgs *a)
{
    if (Hq <= 0 || !sel) return SA_ERR_INVALID_ARGUMENT;
    if (q_dtype != SA_DTYPE_F32 && q_dtype != SA_DTYPE_BF16) return SA_ERR_INVALID_ARGUMENT;
    if (Hq % Hkv) return SA_ERR_UNSUPPORTED;
    if (!(scale == scale) || scale == INFINITY || scale == -INFINITY) return SA_ERR_INVALID_ARGUMENT;
    if (B > 0 && (!q || !out)) return SA_ERR_INVALID_ARGUMENT;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return SA_ERR_INVALID_ARGUMENT;
    if (sel->kind == SA_SEL_TOKENS) {
        if (sel->k_cap < 0 || (B > 0 && sel->k_cap > 0 && (!sel->idx || !sel->count)))
            return SA_ERR_INVALID_ARGUMENT;
        if (B > 0 && !sel->count) return SA_ERR_INVALID_ARGUMENT;
    } else if (sel->kind == SA_SEL_BLOCKS) {
        if (sel->max_blocks < 0 || (B > 0 && (!sel->block_counts || (sel->max_blocks > 0 && !sel->blocks))))
            return SA_ERR_INVALID_ARGUMENT;
        if (!aligned(sel->blocks, 16)) return SA_ERR_INVALID_ARGUMENT;
    } else {
        return SA_ERR_INVALID_ARGUMENT;
    }
    a->q = q;
    a->q_f32 = q_dtype == SA_DTYPE_F32;
    a->Hq = Hq;
    a->qscale = scale * kLog2e;
    a->blocks = sel->kind == SA_SEL_BLOCKS;
    a->idx = sel->idx;
    a->cnt = sel->count;
    a->kcap = sel->k_cap;
    a->ent = sel->blocks;
    a->ecnt = sel->block_counts;
    a->max_blocks = sel->max_blocks;
    return SA_OK;
}

sa_status check_ws(void *ws, size_t ws_bytes, size_t need)
{
    if (need == 0) return SA_ERR_INVALID_ARGUMENT;
    if (!ws || ws_bytes < need) return SA_ERR_WORKSPACE;
    if (!aligned(ws, kAlign)) return SA_ERR_WORKSPACE;
    return SA_OK;
}

sa_status cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return SA_OK;
    cudaGetLastError();  // clear the sticky-free launch error
    return SA_ERR_CUDA;
}

// ---------------- workspace sizes ----------------
size_t ws_topk(const sa_kv_cache *kv, int Hq)
{
    const size_t Lcap = (size_t)kv->max_pages_per_seq * kv->page_size;
    return kHeader + up((size_t)kv->batch * Hq * Lcap * sizeof(float));
}

size_t ws_decode(const sa_kv_cache *kv, int Hq, int S) { return sa::decode_workspace_bytes(kv, Hq, S); }

size_t ws_blocks(const sa_kv_cache *kv, const sa_block_select_args *a)
{
    if (!a) return 0;
    if (a->mode == SA_SEL_SPANS) return kHeader;
    if (a->mode != SA_SEL_RBS) return 0;
    if (a->num_q_heads <= 0 || a->num_tokens <= 0 || a->block_size <= 0) return 0;
    const int nB = (a->num_tokens + a->block_size - 1) / a->block_size;
    size_t offs[16];
    return kHeader + rbs_workspace_layout(a->num_q_heads, kv->num_kv_heads, kv->head_dim, nB,
                                          a->tau_c == nullptr, offs);
}

size_t ws_prefill(const sa_kv_cache *kv, int Hq, int T)
{
    const int nQB = (T + 63) / 64;
    return kHeader + up((size_t)prefill_items(Hq, kv->num_kv_heads, nQB) * sizeof(int4) + 16);
}

}  // namespace

extern "C" {

int32_t sa_version(void) { return 200; }

const char *sa_status_string(sa_status s)
{
    switch (s) {
    case SA_OK: return "SA_OK";
    case SA_ERR_INVALID_ARGUMENT: return "SA_ERR_INVALID_ARGUMENT: invalid argument";
    case SA_ERR_UNSUPPORTED: return "SA_ERR_UNSUPPORTED: configuration not supported";
    case SA_ERR_WORKSPACE: return "SA_ERR_WORKSPACE: workspace missing, misaligned or too small";
    case SA_ERR_CUDA: return "SA_ERR_CUDA: CUDA launch or runtime call failed";
    case SA_ERR_DEVICE_FAULT: return "SA_ERR_DEVICE_FAULT: kernel found invalid device data";
    case SA_ERR_TIMEOUT: return "SA_ERR_TIMEOUT: bounded device wait expired";
    case SA_ERR_CAPACITY: return "SA_ERR_CAPACITY: output capacity exceeded";
    default: return "unknown sa_status";
    }
}

size_t sa_workspace_bytes(sa_op op, const sa_kv_cache *kv, const sa_ws_query *q)
{
    const bool spans = op == SA_OP_SELECT_BLOCKS && q && q->block_args && q->block_args->mode == SA_SEL_SPANS;
    if (check_cache(kv, nullptr, !spans) != SA_OK || !q) return 0;
    switch (op) {
    case SA_OP_SELECT_TOPK:
        if (q->num_q_heads <= 0 || q->k <= 0) return 0;
        return ws_topk(kv, q->num_q_heads);
    case SA_OP_SELECT_BLOCKS:
        return ws_blocks(kv, q->block_args);
    case SA_OP_DECODE:
        if (q->num_q_heads <= 0 || q->num_splits <= 0 || q->num_splits > 64) return 0;
        return ws_decode(kv, q->num_q_heads, q->num_splits);
    case SA_OP_PREFILL:
        if (q->num_q_heads <= 0 || q->num_tokens < 0) return 0;
        if (q->num_q_heads % kv->num_kv_heads) return 0;
        return ws_prefill(kv, q->num_q_heads, q->num_tokens);
    default:
        return 0;
    }
}

sa_status sa_fetch_pages(const void *host_k, const void *host_v, void *dev_k, void *dev_v, const int32_t *pairs,
                         int32_t n, int64_t host_pages, int64_t dev_pages, size_t page_bytes, void *ws,
                         size_t ws_bytes, sa_stream_t stream)
{
    if (n < 0 || host_pages < 0 || dev_pages < 0 || page_bytes == 0 || page_bytes % 16) return SA_ERR_INVALID_ARGUMENT;
    if (n > 0 && (!host_k || !host_v || !dev_k || !dev_v || !pairs)) return SA_ERR_INVALID_ARGUMENT;
    if (!aligned(host_k, 16) || !aligned(host_v, 16) || !aligned(dev_k, 16) || !aligned(dev_v, 16) ||
        !aligned(pairs, 8))
        return SA_ERR_INVALID_ARGUMENT;
    sa_status st = check_ws(ws, ws_bytes, kHeader);
    if (st != SA_OK) return st;
    FetchArgs a{};
    a.host_k = host_k;
    a.host_v = host_v;
    a.dev_k = dev_k;
    a.dev_v = dev_v;
    a.pairs = pairs;
    a.n = n;
    a.host_pages = host_pages;
    a.dev_pages = dev_pages;
    a.page_bytes = page_bytes;
    a.st = static_cast<DevStatus *>(ws);
    return cuda_status(launch_fetch(a, (cudaStream_t)stream));
}

sa_status sa_workspace_init(void *ws, size_t ws_bytes, sa_stream_t stream)
{
    if (!ws || ws_bytes < kHeader || !aligned(ws, kAlign)) return SA_ERR_WORKSPACE;
    return cuda_status(cudaMemsetAsync(ws, 0, kHeader, (cudaStream_t)stream));
}

sa_status sa_check_bounded_wait(int64_t timeout_ns, void *ws, size_t ws_bytes, sa_stream_t stream)
{
    if (timeout_ns <= 0 || timeout_ns > 10000000000ll) return SA_ERR_INVALID_ARGUMENT;
    sa_status st = check_ws(ws, ws_bytes, kHeader);
    if (st != SA_OK) return st;
    return cuda_status(sa::launch_wait_diag(static_cast<DevStatus *>(ws), (unsigned long long)timeout_ns,
                                            (cudaStream_t)stream));
}

sa_status sa_read_device_status(void *ws, sa_stream_t stream, int32_t *detail)
{
    if (!ws || !aligned(ws, kAlign)) return SA_ERR_WORKSPACE;
    cudaStream_t s = (cudaStream_t)stream;
    DevStatus h;
    if (cudaMemcpyAsync(&h, ws, 16, cudaMemcpyDeviceToHost, s) != cudaSuccess) return cuda_status(cudaErrorUnknown);
    if (cudaStreamSynchronize(s) != cudaSuccess) return cuda_status(cudaErrorUnknown);
    if (h.code != 0) {
        if (cudaMemsetAsync(ws, 0, 16, s) != cudaSuccess) return cuda_status(cudaErrorUnknown);
        if (cudaStreamSynchronize(s) != cudaSuccess) return cuda_status(cudaErrorUnknown);
    }
    if (detail) {
        detail[0] = (int32_t)h.code;
        detail[1] = (int32_t)h.detail;
        detail[2] = h.value;
    }
    return (sa_status)h.code;
}

// ---------------------------------------------------------------------------
sa_status sa_select_topk(const sa_kv_cache *kv, const void *q, sa_dtype q_dtype, int32_t num_q_heads,
                         int32_t k, int32_t *idx_out, int32_t *count_out, void *ws, size_t ws_bytes,
                         sa_stream_t stream)
{
    TopkArgs a{};
    sa_status st = check_cache(kv, &a.c);
    if (st != SA_OK) return st;
    if (num_q_heads <= 0 || k <= 0 || k > 65536) return SA_ERR_INVALID_ARGUMENT;
    if (q_dtype != SA_DTYPE_F32 && q_dtype != SA_DTYPE_BF16) return SA_ERR_INVALID_ARGUMENT;
    if (num_q_heads % kv->num_kv_heads) return SA_ERR_UNSUPPORTED;
    const int hpg = num_q_heads / kv->num_kv_heads;
    if (hpg != 1 && hpg != 2 && hpg != 4 && hpg != 8) return SA_ERR_UNSUPPORTED;
    if (kv->batch > 0 && (!q || !idx_out || !count_out)) return SA_ERR_INVALID_ARGUMENT;
    if (!aligned(q, 16) || !aligned(idx_out, 4) || !aligned(count_out, 4)) return SA_ERR_INVALID_ARGUMENT;
    // the selection keeps two bitmaps of the context in shared memory
    if ((long long)kv->max_pages_per_seq * kv->page_size > (1LL << 19)) return SA_ERR_UNSUPPORTED;
    st = check_ws(ws, ws_bytes, ws_topk(kv, num_q_heads));
    if (st != SA_OK) return st;
    a.q = q;
    a.q_f32 = q_dtype == SA_DTYPE_F32;
    a.Hq = num_q_heads;
    a.k = k;
    a.Lcap = kv->max_pages_per_seq * kv->page_size;
    a.scores = reinterpret_cast<float *>(static_cast<char *>(ws) + kHeader);
    a.idx = idx_out;
    a.cnt = count_out;
    a.st = static_cast<DevStatus *>(ws);
    return cuda_status(launch_topk(a, (cudaStream_t)stream));
}

sa_status sa_sparse_decode_attn(const sa_kv_cache *kv, const void *q, sa_dtype q_dtype,
                                int32_t num_q_heads, const sa_selection *sel, float scale,
                                int32_t num_splits, void *out, float *lse_out, void *ws,
                                size_t ws_bytes, sa_stream_t stream)
{
    DecodeArgs a{};
    sa_status st = check_cache(kv, &a.c);
    if (st != SA_OK) return st;
    if (num_splits < 1 || num_splits > 64) return SA_ERR_INVALID_ARGUMENT;
    st = check_decode(kv->batch, kv->num_kv_heads, q, q_dtype, num_q_heads, sel, scale, out, lse_out, &a);
    if (st != SA_OK) return st;
    st = check_ws(ws, ws_bytes, ws_decode(kv, num_q_heads, num_splits));
    if (st != SA_OK) return st;
    char *w = static_cast<char *>(ws);
    const size_t rows = (size_t)kv->batch * num_q_heads;
    a.S = num_splits;
    a.part_o = reinterpret_cast<float *>(w + kHeader);
    a.part_ml = reinterpret_cast<float *>(w + kHeader + up(rows * num_splits * kv->head_dim * sizeof(float)));
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse_out;
    a.st = static_cast<DevStatus *>(ws);
    return cuda_status(launch_decode(a, (cudaStream_t)stream));
}

sa_status sa_select_blocks(const sa_kv_cache *kv, const sa_block_select_args *args, sa_block_list *out,
                           void *ws, size_t ws_bytes, sa_stream_t stream)
{
    CacheArgs c{};
    sa_status st = check_cache(kv, &c, !(args && args->mode == SA_SEL_SPANS));
    if (st != SA_OK) return st;
    if (!args || !out) return SA_ERR_INVALID_ARGUMENT;
    if (args->mode == SA_SEL_SPANS) {
        if (args->max_spans < 0 || args->max_spans > 1024 || out->max_blocks < 0) return SA_ERR_INVALID_ARGUMENT;
        if (kv->batch > 0 && (!args->span_counts || !out->block_counts)) return SA_ERR_INVALID_ARGUMENT;
        if (kv->batch > 0 && args->max_spans > 0 && (!args->spans || !args->span_round))
            return SA_ERR_INVALID_ARGUMENT;
        if (kv->batch > 0 && out->max_blocks > 0 && !out->blocks) return SA_ERR_INVALID_ARGUMENT;
        if (!aligned(out->blocks, 16)) return SA_ERR_INVALID_ARGUMENT;
        st = check_ws(ws, ws_bytes, ws_blocks(kv, args));
        if (st != SA_OK) return st;
        SpanArgs a{};
        a.c = c;
        a.spans = args->spans;
        a.span_counts = args->span_counts;
        a.span_round = args->span_round;
        a.max_spans = args->max_spans;
        a.ent = out->blocks;
        a.ecnt = out->block_counts;
        a.max_blocks = out->max_blocks;
        a.st = static_cast<DevStatus *>(ws);
        return cuda_status(launch_spans(a, (cudaStream_t)stream));
    }
    if (args->mode != SA_SEL_RBS) return SA_ERR_INVALID_ARGUMENT;
    // RBS
    const int Hq = args->num_q_heads, T = args->num_tokens, bs = args->block_size;
    if (Hq <= 0 || T <= 0 || bs <= 0) return SA_ERR_INVALID_ARGUMENT;
    if (bs != 64) return SA_ERR_UNSUPPORTED;
    if (Hq % kv->num_kv_heads) return SA_ERR_UNSUPPORTED;
    if (kv->batch < 1) return SA_ERR_INVALID_ARGUMENT;
    if ((long long)T > (long long)kv->max_pages_per_seq * kv->page_size) return SA_ERR_INVALID_ARGUMENT;
    if (!args->q || !aligned(args->q, 16)) return SA_ERR_INVALID_ARGUMENT;
    if ((args->tau_c == nullptr) != (args->tau_r == nullptr)) return SA_ERR_INVALID_ARGUMENT;
    if (!args->tau_c && !(args->p_c >= 0.f && args->p_c <= 1.f && args->p_r >= 0.f && args->p_r <= 1.f))
        return SA_ERR_INVALID_ARGUMENT;
    if (!(args->scale > 0.f) || args->scale == INFINITY) return SA_ERR_INVALID_ARGUMENT;
    if (!out->row_ptr || !out->cols || out->nnz_capacity < 0) return SA_ERR_INVALID_ARGUMENT;
    const int nB = (T + bs - 1) / bs;
    if (nB > 65536) return SA_ERR_UNSUPPORTED;
    st = check_ws(ws, ws_bytes, ws_blocks(kv, args));
    if (st != SA_OK) return st;
    size_t offs[16];
    const bool quant = args->tau_c == nullptr;
    rbs_workspace_layout(Hq, kv->num_kv_heads, kv->head_dim, nB, quant, offs);
    char *w = static_cast<char *>(ws) + kHeader;
    RbsArgs a{};
    a.c = c;
    a.q = static_cast<const uint16_t *>(args->q);
    a.Hq = Hq;
    a.T = T;
    a.bs = bs;
    a.nB = nB;
    a.scale = args->scale;
    a.tau_c = args->tau_c;
    a.tau_r = args->tau_r;
    a.p_c = args->p_c;
    a.p_r = args->p_r;
    a.force_diag = args->force_diag;
    a.force_first = args->force_first;
    a.cen = reinterpret_cast<uint8_t *>(w + offs[0]);
    a.rad = reinterpret_cast<float *>(w + offs[1]);
    a.qbar = reinterpret_cast<uint8_t *>(w + offs[2]);
    a.qnorm = reinterpret_cast<float *>(w + offs[3]);
    a.tau = reinterpret_cast<float *>(w + offs[4]);
    a.bits = reinterpret_cast<uint32_t *>(w + offs[5]);
    a.rowcnt = reinterpret_cast<int32_t *>(w + offs[6]);
    a.pair_sc = quant ? reinterpret_cast<float *>(w + offs[7]) : nullptr;
    a.qhist = quant ? reinterpret_cast<uint32_t *>(w + offs[8]) : nullptr;
    a.row_ptr = out->row_ptr;
    a.cols = out->cols;
    a.nnz_cap = out->nnz_capacity;
    a.tau_out = out->tau_out;
    a.st = static_cast<DevStatus *>(ws);
    cudaError_t e = launch_rbs(a, (cudaStream_t)stream);
    if (e == cudaErrorNotSupported) return SA_ERR_UNSUPPORTED;
    return cuda_status(e);
}

sa_status sa_sparse_prefill_attn(const sa_kv_cache *kv, const void *q, int32_t num_q_heads,
                                 int32_t num_tokens, const sa_block_list *csr, float scale,
                                 int32_t causal, void *out, float *lse_out, void *ws, size_t ws_bytes,
                                 sa_stream_t stream)
{
    PrefillArgs a{};
    sa_status st = check_cache(kv, &a.c);
    if (st != SA_OK) return st;
    if (num_q_heads <= 0 || num_tokens < 0) return SA_ERR_INVALID_ARGUMENT;
    if (causal != 1) return SA_ERR_UNSUPPORTED;
    if (kv->head_dim != 128 || kv->page_size != 64) return SA_ERR_UNSUPPORTED;
    if (num_q_heads % kv->num_kv_heads) return SA_ERR_UNSUPPORTED;
    if (kv->batch < 1) return SA_ERR_INVALID_ARGUMENT;
    if ((long long)num_tokens > (long long)kv->max_pages_per_seq * kv->page_size) return SA_ERR_INVALID_ARGUMENT;
    if (!(scale == scale)) return SA_ERR_INVALID_ARGUMENT;
    if (num_tokens > 0 && (!q || !csr || !csr->row_ptr || !csr->cols || !out)) return SA_ERR_INVALID_ARGUMENT;
    if (csr && csr->nnz_capacity < 0) return SA_ERR_INVALID_ARGUMENT;
    if ((long long)kv->num_pages * kv->num_kv_heads * 64 >= (1LL << 31)) return SA_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse_out, 4)) return SA_ERR_INVALID_ARGUMENT;
    if (!(scale > 0.f) || scale == INFINITY) return SA_ERR_INVALID_ARGUMENT;
    st = check_ws(ws, ws_bytes, ws_prefill(kv, num_q_heads, num_tokens));
    if (st != SA_OK) return st;
    a.q = static_cast<const uint16_t *>(q);
    a.Hq = num_q_heads;
    a.T = num_tokens;
    a.scale = scale;
    if (num_tokens == 0) return SA_OK;
    a.row_ptr = csr->row_ptr;
    a.cols = csr->cols;
    a.nnz_cap = csr->nnz_capacity;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse_out;
    a.items = reinterpret_cast<int4 *>(static_cast<char *>(ws) + kHeader);
    a.n_items = prefill_items(num_q_heads, kv->num_kv_heads, (num_tokens + 63) / 64);
    a.st = static_cast<DevStatus *>(ws);
    if (num_tokens == 0) return SA_OK;
    cudaError_t e = launch_prefill(a, (cudaStream_t)stream);
    if (e == cudaErrorNotSupported) return SA_ERR_UNSUPPORTED;
    return cuda_status(e);
}

// ---------------------------------------------------------------------------
sa_status sa_plan_append(const sa_plan_args *p, void *ws, size_t ws_bytes, sa_stream_t stream)
{
    if (!p || p->batch < 0 || p->max_pages_per_seq < 0 || p->num_pages < 0 || p->num_free < 0 || p->max_tokens < 0)
        return SA_ERR_INVALID_ARGUMENT;
    if (p->page_size != 16 && p->page_size != 64) return SA_ERR_UNSUPPORTED;
    if (p->batch > kPlanMaxBatch || (long long)p->max_pages_per_seq * p->page_size > (1LL << 30))
        return SA_ERR_UNSUPPORTED;
    // (the kernel counts tokens and pages, a few rows ahead, in 32 bits)
    if (p->max_tokens > (1 << 30) || p->num_free > (1 << 30)) return SA_ERR_UNSUPPORTED;
    if (!p->free_count || !p->free_count_out || !p->cu_tokens || (p->num_free > 0 && !p->free_pages))
        return SA_ERR_INVALID_ARGUMENT;
    if (p->batch > 0 && (!p->seq_lens || !p->new_lens || !p->seq_lens_out ||
                         (p->max_pages_per_seq > 0 && !p->page_table)))
        return SA_ERR_INVALID_ARGUMENT;
    if (p->max_tokens > 0 && (!p->positions || !p->slots)) return SA_ERR_INVALID_ARGUMENT;
    if (!aligned(p->page_table, 4) || !aligned(p->seq_lens, 4) || !aligned(p->new_lens, 4) ||
        !aligned(p->free_pages, 4) || !aligned(p->free_count, 4) || !aligned(p->seq_lens_out, 4) ||
        !aligned(p->free_count_out, 4) || !aligned(p->cu_tokens, 4) || !aligned(p->positions, 4) ||
        !aligned(p->slots, 8) || !aligned(p->seq_ids, 4))
        return SA_ERR_INVALID_ARGUMENT;
    sa_status st = check_ws(ws, ws_bytes, kHeader);
    if (st != SA_OK) return st;
    PlanArgs a{};
    a.B = p->batch;
    a.Plog2 = ilog2(p->page_size);
    a.max_pages = p->max_pages_per_seq;
    a.num_pages = p->num_pages;
    a.num_free = p->num_free;
    a.max_tokens = p->max_tokens;
    a.table = p->page_table;
    a.sl = p->seq_lens;
    a.add = p->new_lens;
    a.free = p->free_pages;
    a.count = p->free_count;
    a.sl_out = p->seq_lens_out;
    a.count_out = p->free_count_out;
    a.cu = p->cu_tokens;
    a.pos = p->positions;
    a.slots = p->slots;
    a.seq_ids = p->seq_ids;
    a.st = static_cast<DevStatus *>(ws);
    return cuda_status(launch_plan(a, (cudaStream_t)stream));
}

}  // extern "C"

namespace {

sa_status rope_append(const CacheArgs &c, bool kv4, const sa_append_args *p, void *ws, size_t ws_bytes,
                      sa_stream_t stream)
{
    if (!p || p->num_tokens < 0 || p->num_q_heads <= 0) return SA_ERR_INVALID_ARGUMENT;
    if (p->rot_dim < 0 || p->rot_dim > c.D || p->rot_dim % 16) return SA_ERR_INVALID_ARGUMENT;
    if (p->weight_dtype != SA_DTYPE_F32 && p->weight_dtype != SA_DTYPE_BF16) return SA_ERR_INVALID_ARGUMENT;
    if (!(p->eps >= 0.f) || p->eps == INFINITY) return SA_ERR_INVALID_ARGUMENT;
    if (p->rot_dim > 0 && !p->inv_freq) return SA_ERR_INVALID_ARGUMENT;
    if (p->num_tokens > 0 && (!p->q || !p->k || !p->v || !p->q_out || !p->positions || !p->slots || !c.k || !c.v))
        return SA_ERR_INVALID_ARGUMENT;
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return SA_ERR_INVALID_ARGUMENT;
    if (p->q_stride % 8 || p->k_stride % 8 || p->v_stride % 8 || p->q_out_stride % 8) return SA_ERR_INVALID_ARGUMENT;
    // output rows must not run into one another
    if (p->num_tokens > 1 && p->q_out_stride < (long long)p->num_q_heads * c.D) return SA_ERR_INVALID_ARGUMENT;
    if (p->q_out == p->q && p->num_tokens > 1 && p->q_out_stride != p->q_stride) return SA_ERR_INVALID_ARGUMENT;
    if (!aligned(p->q, 16) || !aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->q_out, 16) ||
        !aligned(p->q_weight, 16) || !aligned(p->k_weight, 16) || !aligned(p->positions, 4) ||
        !aligned(p->slots, 8) || !aligned(p->inv_freq, 4))
        return SA_ERR_INVALID_ARGUMENT;
    sa_status st = check_ws(ws, ws_bytes, kHeader);
    if (st != SA_OK) return st;
    AppendArgs a{};
    a.q = static_cast<const uint16_t *>(p->q);
    a.k = static_cast<const uint16_t *>(p->k);
    a.v = static_cast<const uint16_t *>(p->v);
    a.q_stride = p->q_stride;
    a.k_stride = p->k_stride;
    a.v_stride = p->v_stride;
    a.q_out_stride = p->q_out_stride;
    a.T = p->num_tokens;
    a.Hq = p->num_q_heads;
    a.Hkv = c.Hkv;
    a.D = c.D;
    a.Plog2 = c.Plog2;
    a.num_slots = (long long)c.num_pages << c.Plog2;
    a.pos = p->positions;
    a.slots = p->slots;
    a.inv_freq = p->inv_freq;
    a.rot = p->rot_dim;
    a.interleaved = p->interleaved != 0;
    a.q_weight = p->q_weight;
    a.k_weight = p->k_weight;
    a.w_f32 = p->weight_dtype == SA_DTYPE_F32;
    a.eps = p->eps;
    a.q_out = static_cast<uint16_t *>(p->q_out);
    if (kv4) {
        a.kv4 = reinterpret_cast<uint8_t *>(const_cast<uint16_t *>(c.k));
    } else {
        a.kp = const_cast<uint16_t *>(c.k);
        a.vp = const_cast<uint16_t *>(c.v);
    }
    a.st = static_cast<DevStatus *>(ws);
    return cuda_status(launch_append(a, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

sa_status sa_rope_append(const sa_kv_cache *kv, const sa_append_args *p, void *ws, size_t ws_bytes, sa_stream_t stream)
{
    CacheArgs c{};
    sa_status st = check_cache(kv, &c);
    return st != SA_OK ? st : rope_append(c, false, p, ws, ws_bytes, stream);
}

sa_status sa_rope_append_kv4(const sa_kv4_cache *kv, const sa_append_args *p, void *ws, size_t ws_bytes,
                             sa_stream_t stream)
{
    CacheArgs c{};
    sa_status st = check_cache4(kv, &c);
    return st != SA_OK ? st : rope_append(c, true, p, ws, ws_bytes, stream);
}

sa_status sa_expand_kv4(const sa_kv4_cache *kv, const int32_t *pages, int32_t n, void *k_out, void *v_out, void *ws,
                        size_t ws_bytes, sa_stream_t stream)
{
    CacheArgs c{};
    sa_status st = check_cache4(kv, &c);
    if (st != SA_OK) return st;
    if (n < 0 || (n > 0 && (!pages || !k_out || !v_out || !kv->kv))) return SA_ERR_INVALID_ARGUMENT;
    if (!aligned(kv->kv, 16) || !aligned(pages, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return SA_ERR_INVALID_ARGUMENT;
    st = check_ws(ws, ws_bytes, kHeader);
    if (st != SA_OK) return st;
    ExpandArgs a{};
    a.kv4 = static_cast<const uint8_t *>(kv->kv);
    a.pages = pages;
    a.n = n;
    a.Hkv = c.Hkv;
    a.D = c.D;
    a.Plog2 = c.Plog2;
    a.num_pages = c.num_pages;
    a.k = static_cast<uint16_t *>(k_out);
    a.v = static_cast<uint16_t *>(v_out);
    a.st = static_cast<DevStatus *>(ws);
    return cuda_status(launch_expand(a, (cudaStream_t)stream));
}

size_t sa_kv4_decode_workspace_bytes(const sa_kv4_cache *kv, int32_t num_q_heads, int32_t num_splits)
{
    if (check_cache4(kv, nullptr) != SA_OK || num_q_heads <= 0 || num_splits < 0 || num_splits > 64) return 0;
    if (num_q_heads % kv->num_kv_heads) return 0;
    sa_kv_cache as{};
    as.batch = kv->batch;
    as.head_dim = kv->head_dim;
    // (chosen splits: no more CTAs than make the partial states worth their bytes)
    const int most = num_splits > 0 ? num_splits : kv4_most_splits(kv, num_q_heads);
    return sa::decode_workspace_bytes(&as, num_q_heads, most);
}

sa_status sa_sparse_decode_attn_kv4_parts(const sa_kv4_cache *kv, const void *q, sa_dtype q_dtype,
                                          int32_t num_q_heads, const sa_selection *sel, float scale,
                                          int32_t num_splits, void *out, float *lse_out, void *parts,
                                          size_t parts_bytes, void *ws, size_t ws_bytes, sa_stream_t stream)
{
    DecodeArgs a{};
    sa_status st = check_cache4(kv, &a.c);
    if (st != SA_OK) return st;
    if (num_splits < 0 || num_splits > 64) return SA_ERR_INVALID_ARGUMENT;
    st = check_decode(kv->batch, kv->num_kv_heads, q, q_dtype, num_q_heads, sel, scale, out, lse_out, &a);
    if (st != SA_OK) return st;
    if (kv->batch > 65535 || num_q_heads > 65535) return SA_ERR_UNSUPPORTED;   // grid dimensions
    // (list positions, two steps ahead, are counted in 32 bits)
    if ((a.blocks ? a.max_blocks : a.kcap) > (1 << 30)) return SA_ERR_UNSUPPORTED;
    st = check_ws(ws, ws_bytes, kHeader);
    if (st != SA_OK) return st;
    if (!parts || !aligned(parts, 16) || parts_bytes < sa_kv4_decode_workspace_bytes(kv, num_q_heads, num_splits) - kHeader)
        return SA_ERR_WORKSPACE;
    if (num_splits == 0) {
        const bool wide = a.blocks && num_q_heads / kv->num_kv_heads > 8;
        num_splits = decode_kv4_splits(kv->batch, a.blocks ? kv4_group_rows(kv, num_q_heads) : num_q_heads,
                                       a.blocks ? (long long)a.max_blocks * kv->page_size : (long long)a.kcap,
                                       kv->head_dim, !a.blocks, a.q_f32, wide);
        const int most = kv4_most_splits(kv, num_q_heads);
        if (num_splits > most) num_splits = most;
    }
    char *w = static_cast<char *>(parts);
    const size_t rows = (size_t)kv->batch * num_q_heads;
    a.S = num_splits;
    a.part_o = reinterpret_cast<float *>(w);
    a.part_ml = reinterpret_cast<float *>(w + up(rows * num_splits * kv->head_dim * sizeof(float)));
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse_out;
    a.st = static_cast<DevStatus *>(ws);
    return cuda_status(launch_decode_kv4(a, (cudaStream_t)stream));
}

sa_status sa_sparse_decode_attn_kv4(const sa_kv4_cache *kv, const void *q, sa_dtype q_dtype, int32_t num_q_heads,
                                    const sa_selection *sel, float scale, int32_t num_splits, void *out,
                                    float *lse_out, void *ws, size_t ws_bytes, sa_stream_t stream)
{
    void *parts = ws && ws_bytes >= kHeader ? static_cast<char *>(ws) + kHeader : nullptr;
    return sa_sparse_decode_attn_kv4_parts(kv, q, q_dtype, num_q_heads, sel, scale, num_splits, out, lse_out, parts,
                                           parts ? ws_bytes - kHeader : 0, ws, ws_bytes, stream);
}

}  // extern "C"
