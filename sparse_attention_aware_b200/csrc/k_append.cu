// A step's queries, keys and values: per-head RMS norm, rotary positions and
// the store into the paged cache, in one pass over the projections.
//
//   y = x / sqrt(mean x^2 + eps) * w                  (a head's D channels)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t)  t = position * inv_freq
// for queries and keys; values are stored as they are.  A cached key is a
// rotated key, so the selections and the attention that read the cache need
// no positions ("语言模型能自己决定该看哪里吗？", DA state machine section:
// the paged cache the masks read from).
//
// bf16 pages take the rows rounded to bf16.  4-bit pages (kv4.cuh) take, for
// each half of a row, zero = bf16(min), scale = bf16((max - min) / 15) (each
// through fp32) and codes rint((y - zero) / scale), ties to even, clamped to
// [0, 15]; a half that holds a value that is not finite is stored with scale
// and zero NaN.  Keys and values for 4-bit pages are computed in fp64 up to
// the codes: an fp32 norm is a few ulps off, which next to a border between
// two codes stores another code, a full step away.  With fp64 the stored
// bytes are those of the definition, whatever the call's shape.
//
// Angles are formed in fp64 (position * inv_freq is exact below 2^29),
// reduced by 2 pi in two parts (Cody and Waite) and only then rounded for the
// fp32 sine: fp32 angles of positions near 2^20 would be off by up to 0.06.
//
// One CTA per token (and slice of its heads); a warp takes 32 / (D/8) heads of
// one kind, 8 channels a lane.  Bound by HBM for prompts (rows in, rows out),
// by latency for single steps.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sa {
namespace {

constexpr int kAppendThreads = 256;

template <typename F>
struct Angle {
    F cos, sin;
};

// angle reduced to [-pi, pi] (2 pi as the sum of two doubles)
__device__ __forceinline__ double reduce_2pi(double x)
{
    const double k = rint(x * 0.15915494309189535);
    const double r = fma(-k, 6.283185307179586, x);
    return fma(-k, 2.4492935982947064e-16, r);
}

template <int D, typename F>
__device__ __forceinline__ void norm_row(F (&x)[8], const F (&w)[8], bool has_w, float eps)
{
    F ss = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fma(x[e], x[e], ss);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
    if (has_w) {
        const F r = (F)1 / sqrt(ss / (F)D + (F)eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
    }
}

// cs: the lane's 8 angles (pairs apart: angle of channel e; pairs together:
// angle of pair e / 2, in entries 0..3)
template <int D, typename F>
__device__ __forceinline__ void rope_row(F (&x)[8], const Angle<F> (&cs)[8], int e0, int rot, bool interleaved)
{
    if (interleaved) {
        if (e0 < rot) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const F a = x[2 * p], b = x[2 * p + 1];
                x[2 * p] = a * cs[p].cos - b * cs[p].sin;
                x[2 * p + 1] = b * cs[p].cos + a * cs[p].sin;
            }
        }
    } else {
        const int n = rot / 2, lane = threadIdx.x & 31;
        const int src = e0 < n ? lane + n / 8 : e0 < rot ? lane - n / 8 : lane;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const F other = __shfl_sync(~0u, x[e], src);
            const F turned = x[e] * cs[e].cos + (e0 < n ? -other : other) * cs[e].sin;
            if (e0 < rot) x[e] = turned;
        }
    }
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&f)[8])
{
    f[0] = bf_lo(w.x); f[1] = bf_hi(w.x); f[2] = bf_lo(w.y); f[3] = bf_hi(w.y);
    f[4] = bf_lo(w.z); f[5] = bf_hi(w.z); f[6] = bf_lo(w.w); f[7] = bf_hi(w.w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// One row (16 or 8 lanes, 8 channels each) to 4 bits: the lane's code word,
// and the {scale, zero} of its half as bf16.  Exact for the fp64 values given.
template <int D>
__device__ __forceinline__ void quantize_row(const double (&y)[8], uint32_t &codes, uint32_t &par)
{
    constexpr int HL = D / 16;   // lanes of a half
    double lo = y[0], hi = y[0];
    bool fine = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        lo = fmin(lo, y[e]);
        hi = fmax(hi, y[e]);
        fine = fine && isfinite(y[e]);
    }
#pragma unroll
    for (int o = HL / 2; o > 0; o >>= 1) {
        lo = fmin(lo, __shfl_xor_sync(~0u, lo, o));
        hi = fmax(hi, __shfl_xor_sync(~0u, hi, o));
    }
    const unsigned half_lanes = ((1u << HL) - 1) << ((threadIdx.x & 31) & ~(HL - 1));
    const unsigned finite = __ballot_sync(~0u, fine);
    const __nv_bfloat16 zb = __float2bfloat16_rn((float)lo), sb = __float2bfloat16_rn((float)((hi - lo) / 15.0));
    const float zf = __bfloat162float(zb), sf = __bfloat162float(sb);
    codes = 0;
    if ((finite & half_lanes) != half_lanes || !isfinite(zf) || !isfinite(sf)) {
        par = 0x7fc07fc0u;
        return;
    }
    par = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(zb) << 16);
    if (!(sf > 0.f)) return;
    const double z = zf, s = sf, inv = 1.0 / s;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double d = y[e] - z;
        double c = fmin(fmax(floor(d * inv), -1.0), 16.0);
        // the sign of d - (c + 1/2) s is exact in one fma; a tie goes to the even code
        const double over = fma(-(c + 0.5), s, d);
        int code = (int)c;
        code += over > 0.0 || (over == 0.0 && (code & 1));
        codes |= (uint32_t)min(max(code, 0), 15) << (4 * e);
    }
}

template <int D, int BITS>
__global__ void __launch_bounds__(kAppendThreads) k_rope_append(const AppendArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int LPR = D / 8, RPW = 32 / LPR, WARPS = kAppendThreads / 32;
    __shared__ Angle<double> s_ang[D / 2];
    const long long t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gl = lane & (LPR - 1), sub = lane / LPR, e0 = gl * 8;
    const int qt = (a.Hq + RPW - 1) / RPW, kt = (a.Hkv + RPW - 1) / RPW;
    const int tasks = qt + 2 * kt;

    const int n = a.rot / 2;
    if ((int)threadIdx.x < n) {
        double s, c;
        sincos(reduce_2pi((double)a.pos[t] * (double)a.inv_freq[threadIdx.x]), &s, &c);
        s_ang[threadIdx.x] = {c, s};
    }
    const long long slot = a.slots[t];
    bool store = slot >= 0;
    if (slot < -1 || slot >= a.num_slots) {
        if (threadIdx.x == 0 && blockIdx.y == 0) fault(a.st, CHK_SLOT, (int)slot);
        store = false;
    }
    __syncthreads();
    Angle<float> cs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // pairs apart: channel e0 + e and its partner share angle (e0 + e) mod n
        const int i = a.interleaved ? e0 / 2 + (e & 3) : e0 < n ? e0 + e : e0 - n + e;
        const Angle<double> x = e0 < a.rot ? s_ang[i] : Angle<double>{1.0, 0.0};
        cs[e] = {(float)x.cos, (float)x.sin};
    }
    const int off = (int)(slot & ((1 << a.Plog2) - 1));
    const long long page = slot >> a.Plog2;

    for (int task = blockIdx.y * WARPS + warp; task < tasks; task += gridDim.y * WARPS) {
        const int kind = task < qt ? 0 : task < qt + kt ? 1 : 2;
        const int head = (task - (kind == 0 ? 0 : kind == 1 ? qt : qt + kt)) * RPW + sub;
        const bool act = head < (kind == 0 ? a.Hq : a.Hkv);
        if (kind != 0 && !store) continue;
        const uint16_t *src = kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (act) raw = *reinterpret_cast<const uint4 *>(src + (size_t)head * D + e0);
        const void *w = kind == 0 ? a.q_weight : a.k_weight;
        const bool normed = kind != 2 && w != nullptr;
        float wf[8];
        if (normed) {
            if (a.w_f32) {
                const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + e0);
                const float4 x = p[0], y = p[1];
                wf[0] = x.x; wf[1] = x.y; wf[2] = x.z; wf[3] = x.w;
                wf[4] = y.x; wf[5] = y.y; wf[6] = y.z; wf[7] = y.w;
            } else {
                unpack8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + e0), wf);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) wf[e] = 1.f;
        }
        float x[8];
        unpack8(raw, x);
        const size_t row = (((size_t)page * a.Hkv + head) << a.Plog2) + off;   // of the cache, for keys and values
        if (BITS == 4 && kind != 0) {
            double y[8], w8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e], w8[e] = wf[e];
            if (kind == 1) {
                norm_row<D>(y, w8, normed, a.eps);
                if (n > 0) {
                    Angle<double> c8[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = a.interleaved ? e0 / 2 + (e & 3) : e0 < n ? e0 + e : e0 - n + e;
                        c8[e] = e0 < a.rot ? s_ang[i] : Angle<double>{1.0, 0.0};
                    }
                    rope_row<D>(y, c8, e0, a.rot, a.interleaved);
                }
            }
            uint32_t codes, par;
            quantize_row<D>(y, codes, par);
            if (act) {
                uint8_t *rec = a.kv4 + row * Kv4<D>::REC;
                *reinterpret_cast<uint32_t *>(rec + (kind == 2 ? Kv4<D>::V : 0) + gl * 4) = codes;
                if ((gl & (LPR / 2 - 1)) == 0)
                    *reinterpret_cast<uint32_t *>(rec + Kv4<D>::PAR + (kind == 2 ? 8 : 0) + (gl ? 4 : 0)) = par;
            }
            continue;
        }
        if (kind != 2) {
            norm_row<D>(x, wf, normed, a.eps);
            if (n > 0) rope_row<D>(x, cs, e0, a.rot, a.interleaved);
            raw = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
        }
        if (act) {
            uint16_t *dst = kind == 0 ? a.q_out + t * a.q_out_stride + (size_t)head * D
                                      : (kind == 1 ? a.kp : a.vp) + row * D;
            *reinterpret_cast<uint4 *>(dst + e0) = raw;
        }
    }
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t s)
{
    if (a.T == 0) return cudaSuccess;
    const int rpw = 256 / a.D, warps = kAppendThreads / 32;
    const int tasks = (a.Hq + rpw - 1) / rpw + 2 * ((a.Hkv + rpw - 1) / rpw);
    // few tokens: spread a token's heads over CTAs, so that a step is not a
    // serial walk over its heads
    const int most = (tasks + warps - 1) / warps;
    const int slices = a.T >= 296 ? 1 : most;
    const dim3 grid((unsigned)a.T, (unsigned)slices);
    if (a.kv4) {
        if (a.D == 64) return launch_pdl(k_rope_append<64, 4>, grid, dim3(kAppendThreads), 0, s, a);
        return launch_pdl(k_rope_append<128, 4>, grid, dim3(kAppendThreads), 0, s, a);
    }
    if (a.D == 64) return launch_pdl(k_rope_append<64, 16>, grid, dim3(kAppendThreads), 0, s, a);
    return launch_pdl(k_rope_append<128, 16>, grid, dim3(kAppendThreads), 0, s, a);
}

}  // namespace sa
