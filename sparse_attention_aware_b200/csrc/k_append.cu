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
// and zero NaN.  The stored bytes are those of the definition in fp64, whatever
// the call's shape: rows are computed in fp32 with a bound on their error, and a
// warp one of whose rows has a code, scale or zero nearer to a border than that
// (about one in thirty with keys) computes it again in fp64.  (A code next to a
// border would otherwise come out a full step off; with all keys and values in
// fp64 the kernel took 237 us for 16391 tokens of 32 + 2 x 8 heads, now 104.)
//
// Angles are formed in fp64 (position * inv_freq is exact below 2^29),
// reduced by 2 pi in two parts (Cody and Waite) and only then rounded for the
// fp32 sine: fp32 angles of positions near 2^20 would be off by up to 0.06.
//
// A warp takes a token's heads (or a slice of them, when there are few tokens)
// 32 / (D/8) at a time, kBatch rows a lane in flight; its lanes share out the
// token's angles.  A lane holds two runs of 4 channels whose elements turn with
// one another (4g.. and rot/2 + 4g.., or 8g.. and 8g + 4.. where pairs are
// neighbours), so the rotation needs no exchange between lanes.
//
// Measured: 32768 tokens of 32 + 2 x 4 heads into bf16 pages 109 us, 671 MB, 0.94
// of HBM; 16391 tokens into 4-bit pages 104 us, 354 MB, 0.52 of HBM: bound by
// instructions (about 5000 a token, of which 1900 are the queries'); a step's 32
// tokens 3.1 us, bound by latency.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sa {
namespace {

// One warp a block: a warp that has rows to do again takes several times as
// long, and must not hold the places of others (blocks of 8 warps: 118 us for a
// 32768-token prompt into bf16 pages, 147 us for 16391 tokens into 4-bit pages
// and back; of one: 110 and 127 us).
constexpr int kAppendThreads = 32;

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

__device__ __forceinline__ float inv_root(float x) { return rsqrtf(x); }   // within 2 ulps
__device__ __forceinline__ double inv_root(double x) { return 1.0 / sqrt(x); }

// Returns mean x^2 + eps
template <int D, typename F>
__device__ __forceinline__ F norm_row(F (&x)[8], const F (&w)[8], float eps)
{
    F ss = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fma(x[e], x[e], ss);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
    const F mean = ss * (F)(1.0 / D) + (F)eps, r = inv_root(mean);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
    return mean;
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
        const int n = rot / 2, lane = threadIdx.x;
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

__device__ __forceinline__ void load_weight(const void *w, bool f32, int e0, float (&wf)[8])
{
    if (f32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + e0);
        const float4 x = p[0], y = p[1];
        wf[0] = x.x; wf[1] = x.y; wf[2] = x.z; wf[3] = x.w;
        wf[4] = y.x; wf[5] = y.y; wf[6] = y.z; wf[7] = y.w;
    } else {
        unpack8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + e0), wf);
    }
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
        lo = y[e] < lo ? y[e] : lo;
        hi = y[e] > hi ? y[e] : hi;
        fine = fine && fabs(y[e]) <= 1e300;
    }
#pragma unroll
    for (int o = HL / 2; o > 0; o >>= 1) {
        const double l = __shfl_xor_sync(~0u, lo, o), h = __shfl_xor_sync(~0u, hi, o);
        lo = l < lo ? l : lo;
        hi = h > hi ? h : hi;
    }
    const unsigned half_lanes = ((1u << HL) - 1) << (threadIdx.x & ~(HL - 1));
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
        // (the clamp of the quotient only keeps the conversion in range)
        int code = __double2int_rd(d * inv);
        code = min(max(code, -1), 16);
        // the sign of d - (c + 1/2) s is exact in one fma; a tie goes to the even code
        const double over = fma(-(code + 0.5), s, d);
        code += over > 0.0 || (over == 0.0 && (code & 1));
        codes |= (uint32_t)min(max(code, 0), 15) << (4 * e);
    }
}

// Codes (low word) and parameters of one kind of row (1: key, 2: value), in
// fp64 from the start.  Called by whole warps; src null: no row.  ang: room for
// the token's angles.
template <int D>
__device__ __noinline__ uint2 append_row64(const AppendArgs &a, const uint16_t *src, int kind, long long t,
                                           Angle<double> *ang)
{
    const int e0 = (threadIdx.x & (D / 8 - 1)) * 8;
    float x[8];
    unpack8(src ? *reinterpret_cast<const uint4 *>(src + e0) : make_uint4(0, 0, 0, 0), x);
    double y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e];
    if (kind == 1) {
        if (a.k_weight) {
            float wf[8];
            load_weight(a.k_weight, a.w_f32, e0, wf);
            double w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = wf[e];
            norm_row<D>(y, w, a.eps);
        }
        const int n = a.rot / 2;
        if (n > 0) {
            const double pos = a.pos[t];
            __syncwarp();
#pragma unroll 1
            for (int i = threadIdx.x; i < n; i += 32) {
                Angle<double> x;
                sincos(reduce_2pi(pos * (double)a.inv_freq[i]), &x.sin, &x.cos);
                ang[i] = x;
            }
            __syncwarp();
            Angle<double> cs[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                cs[e] = {1.0, 0.0};
                if (e0 < a.rot) cs[e] = ang[a.interleaved ? e0 / 2 + (e & 3) : e0 < n ? e0 + e : e0 - n + e];
            }
            rope_row<D>(y, cs, e0, a.rot, a.interleaved);
        }
    }
    uint2 r;
    quantize_row<D>(y, r.x, r.y);
    return r;
}

// The same from fp32 rows whose elements are off by at most 36 * 2^-24 of the row's
// largest (exact: not at all); row: the same 8 elements in memory.  Returns false in the lanes that see a border too
// near.
//
// The bound, u = 2^-24: the norm's sum of squares is off by 12 u, its inverse
// root by half of that and 4 u, each of two products by u: 12 u; sine and cosine
// by 2 u, and 2 u more from the angle's rounding; their products by u.  |a| + |b|
// is at most twice the row's largest element (the pair's length is kept), so
// a cos - b sin is off by 2 (12 + 4 + 1) u + u = 35 u of it: 36 u is taken.
template <int D>
__device__ __forceinline__ bool quantize_row32(const float (&y)[8], const float *row, bool exact, uint32_t &codes,
                                               uint32_t &par)
{
    constexpr int HL = D / 16;               // lanes of a half
    constexpr float MAGIC = 12582912.f;      // 1.5 * 2^23: x + MAGIC holds the nearest whole number in its low bits
    float lo = y[0], hi = y[0];   // (a NaN is passed over here and fails the test of its code)
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        lo = fminf(lo, y[e]);
        hi = fmaxf(hi, y[e]);
    }
#pragma unroll
    for (int o = HL / 2; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
    }
    const float top = fmaxf(fabsf(lo), fabsf(hi));
    const float err = exact ? 0.f : fmaxf(top, __shfl_xor_sync(~0u, top, HL)) * (36.f / 16777216.f);   // of the row
    auto bf = [](float x) { return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x)); };
    const float range = (hi - lo) * (1.f / 15.f), slack = fmaf(range, 4.8e-7f, 0.25f * err);   // 8 u, and 2 err / 15
    const uint32_t zb = bf(lo - err), sb = bf(range - slack);
    const float z = bf_lo(zb), s = bf_lo(sb);
    // (subnormal, huge and infinite rows are left to fp64)
    bool sure = zb == bf(lo + err) && sb == bf(range + slack) && s > 1e-30f && top < 1e30f;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));   // within 1 ulp
    // quotients y / s - z / s: each product and the quotient's reciprocal are within 4 u
    const float zi = z * inv, near = 0.5f - fmaf(err, 1.01f * inv, fmaf((fabsf(z) + top) * inv, 4.8e-7f, 4e-6f));
    codes = 0u;
    unsigned close = 0u;   // elements next to a border
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = fmaf(y[e], inv, -zi), m = t + MAGIC;
        if (!(fabsf(t - (m - MAGIC)) < near)) close |= 1u << e;
        codes += __float_as_uint(fminf(fmaxf(m, MAGIC), MAGIC + 15.f)) * (1u << (4 * e));
    }
    codes -= 0x4b400000u * 0x11111111u;   // MAGIC's own bits
    par = sb | (zb << 16);
    if (!exact) return sure && !close;
    // on a border itself are one in 500 bf16 numbers: the sign of the distance
    // from it is exact in one fma if x - z is
    while (__any_sync(~0u, close)) {
        if (close) {
            const int e = __ffs(close) - 1;
            const float x = row[e], d = x - z, f = floorf(d * inv);
            // (d inv is within 1e-5 of a half: f is the code below the border)
            const float over = fmaf(-(f + 0.5f), s, d);
            const int c = (int)f + (over > 0.f || (over == 0.f && ((int)f & 1)));
            sure = sure && d + z == x && x - d == z;
            codes = (codes & ~(15u << (4 * e))) | (uint32_t)min(max(c, 0), 15) << (4 * e);
            close &= close - 1;
        }
    }
    return sure;
}

// A row's code word and its half's parameters into its record
template <int D>
__device__ __forceinline__ void put4(uint8_t *rec, int kind, uint32_t codes, uint32_t par)
{
    const int gl = threadIdx.x & (D / 8 - 1);
    *reinterpret_cast<uint32_t *>(rec + (kind == 2 ? Kv4<D>::V : 0) + gl * 4) = codes;
    if ((gl & (D / 16 - 1)) == 0)
        *reinterpret_cast<uint32_t *>(rec + Kv4<D>::PAR + (kind == 2 ? 8 : 0) + (gl ? 4 : 0)) = par;
}

constexpr int kBatch = 4;   // rows a lane has in flight

// wpt warps share a token's heads
template <int D, int BITS>
__global__ void __launch_bounds__(kAppendThreads, BITS == 4 ? 24 : 32) k_rope_append(const AppendArgs a, int wpt)
{
    pdl_wait();
    pdl_trigger();
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    __shared__ Angle<float> s_ang[D / 2];
    __shared__ Angle<double> s_ang64[BITS == 4 ? D / 2 : 1];
    __shared__ float4 s_row[BITS == 4 ? 32 * 2 : 1];   // rows on their way to 4 bits: RPW of them
    const int lane = threadIdx.x;
    const long long t = blockIdx.x / wpt;
    const int first = (int)(blockIdx.x - t * wpt);
    const int gl = lane & (LPR - 1), sub = lane / LPR, e0 = gl * 8;
    const int qt = (a.Hq + RPW - 1) / RPW, kt = (a.Hkv + RPW - 1) / RPW;
    const int n = a.rot / 2;
    // the lane's two runs of channels, and whether they turn with each other
    const bool turns = gl < a.rot / 8, apart = turns && !a.interleaved;
    const int ca = apart ? 4 * gl : e0, cb = apart ? n + 4 * gl : e0 + 4;

    const long long slot = a.slots[t];
    bool store = slot >= 0;
    if (slot < -1 || slot >= a.num_slots) {
        if (lane == 0 && first == 0) fault(a.st, CHK_SLOT, (int)slot);
        store = false;
    }
    const size_t row0 = (((size_t)(slot >> a.Plog2) * a.Hkv) << a.Plog2) + (size_t)(slot & ((1 << a.Plog2) - 1));

    // the token's angles, shared out over the lanes
    Angle<float> cs[4] = {{1.f, 0.f}, {1.f, 0.f}, {1.f, 0.f}, {1.f, 0.f}};
    if (first < qt + kt && n > 0) {
        const double pos = a.pos[t];
        for (int i = lane; i < n; i += 32) {
            Angle<float> x;
            sincosf((float)reduce_2pi(pos * (double)a.inv_freq[i]), &x.sin, &x.cos);
            s_ang[i] = x;
        }
        __syncwarp();
        if (turns) {
#pragma unroll
            for (int e = 0; e < 4; ++e) cs[e] = s_ang[4 * gl + e];
        }
    }

    // norm and rotation of a row: x[0..3] at channel ca, x[4..7] at cb; false
    // where squares leave the range that fp32 holds well
    auto turn = [&](float (&x)[8], const void *w, const float (&wf)[8]) {
        bool held = true;
        if (w) {
            const float mean = norm_row<D>(x, wf, a.eps);
            held = mean > 1e-24f && mean < 1e30f;
        }
        if (a.interleaved) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float u = x[2 * p], v = x[2 * p + 1];
                if (turns) {
                    x[2 * p] = fmaf(u, cs[p].cos, -v * cs[p].sin);
                    x[2 * p + 1] = fmaf(v, cs[p].cos, u * cs[p].sin);
                }
            }
        } else if (turns) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float u = x[p], v = x[4 + p];
                x[p] = fmaf(u, cs[p].cos, -v * cs[p].sin);
                x[4 + p] = fmaf(v, cs[p].cos, u * cs[p].sin);
            }
        }
        return held;
    };
    // this warp's tasks of a kind whose tasks begin at `from` of all of them
    auto start = [&](int from) { return wpt == 1 ? 0 : (first + wpt - from % wpt) % wpt; };
    // heads of a kind, kBatch rows at a time: row(head, channels ca and cb)
    auto load = [&](const uint16_t *src, int head, int heads) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (head < heads) {
            const uint2 u = *reinterpret_cast<const uint2 *>(src + (size_t)head * D + ca);
            const uint2 v = *reinterpret_cast<const uint2 *>(src + (size_t)head * D + cb);
            r = make_uint4(u.x, u.y, v.x, v.y);
        }
        return r;
    };
    auto put = [&](uint16_t *dst, const float (&x)[8]) {
        *reinterpret_cast<uint2 *>(dst + ca) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
        *reinterpret_cast<uint2 *>(dst + cb) = make_uint2(pack2(x[4], x[5]), pack2(x[6], x[7]));
    };
    float wf[8];
    auto weight = [&](const void *w) {
        float half[8];
        load_weight(w, a.w_f32, ca & ~7, half);
#pragma unroll
        for (int e = 0; e < 4; ++e) wf[e] = (ca & 4) ? half[4 + e] : half[e];
        load_weight(w, a.w_f32, cb & ~7, half);
#pragma unroll
        for (int e = 0; e < 4; ++e) wf[4 + e] = (cb & 4) ? half[4 + e] : half[e];
    };

    // ---- queries
    const int q0 = start(0);
    if (q0 < qt) {
        if (a.q_weight) weight(a.q_weight);
        const uint16_t *src = a.q + t * a.q_stride;
        uint16_t *out = a.q_out + t * a.q_out_stride;
        for (int i = q0; i < qt; i += kBatch * wpt) {
            uint4 raw[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) raw[u] = load(src, (i + u * wpt) * RPW + sub, a.Hq);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int head = (i + u * wpt) * RPW + sub;
                if (head - sub >= a.Hq) break;
                float x[8];
                unpack8(raw[u], x);
                turn(x, a.q_weight, wf);
                if (head < a.Hq) put(out + (size_t)head * D, x);
            }
        }
    }
    if (!store) return;
    // ---- keys, then values: tasks qt .. qt + 2 kt - 1.  The rows of a batch go
    // through one copy of the code (unrolled, the 4-bit form waited for its
    // instructions)
    const uint16_t *kp = a.k + t * a.k_stride, *vp = a.v + t * a.v_stride;
    const bool plain = !a.k_weight && n == 0;   // keys as they came
    const int begin = start(qt);
    if (begin < kt && a.k_weight) weight(a.k_weight);
    unsigned long long redo = 0, bit = 1;   // tasks to be done again in fp64
    for (int i = begin; i < 2 * kt; i += kBatch * wpt) {
        uint4 raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int j = i + u * wpt, head = (j < kt ? j : j - kt) * RPW + sub;
            raw[u] = load(j < kt ? kp : vp, j < 2 * kt ? head : a.Hkv, a.Hkv);
        }
#pragma unroll 1
        for (int u = 0, j = i; u < kBatch && j < 2 * kt; ++u, j += wpt, bit <<= 1) {
            const bool key = j < kt;
            const int head = (key ? j : j - kt) * RPW + sub;
            const bool act = head < a.Hkv;
            const size_t at = row0 + ((size_t)head << a.Plog2);
            float x[8];
            unpack8(raw[0], x);
#pragma unroll
            for (int v = 0; v + 1 < kBatch; ++v) raw[v] = raw[v + 1];
            const bool held = key ? turn(x, a.k_weight, wf) : true;
            if (BITS == 16) {
                if (act) put((key ? a.kp : a.vp) + at * D, x);
                continue;
            }
            // back to 8 channels a lane, in order
            float *r = reinterpret_cast<float *>(s_row) + sub * D;
            __syncwarp();
            *reinterpret_cast<float4 *>(r + ca) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(r + cb) = make_float4(x[4], x[5], x[6], x[7]);
            __syncwarp();
            const float4 u4 = *reinterpret_cast<const float4 *>(r + e0), v4 = *reinterpret_cast<const float4 *>(r + e0 + 4);
            const float y[8] = {u4.x, u4.y, u4.z, u4.w, v4.x, v4.y, v4.z, v4.w};
            uint32_t codes, par;
            const bool sure = quantize_row32<D>(y, r + e0, !key || plain, codes, par) && held;
            if (act) put4<D>(a.kv4 + at * Kv4<D>::REC, key ? 1 : 2, codes, par);
            if (!__all_sync(~0u, sure || !act)) redo |= bit;
        }
    }
    if (BITS == 4) {
        // (at the end: a call between the rows would have their state moved to
        // memory around it)
#pragma unroll 1
        for (; redo; redo &= redo - 1) {
            const int j = begin + (__ffsll(redo) - 1) * wpt, kind = j < kt ? 1 : 2;
            const int head = (j < kt ? j : j - kt) * RPW + sub;
            const bool act = head < a.Hkv;
            const uint2 r = append_row64<D>(a, act ? (j < kt ? kp : vp) + (size_t)head * D : nullptr, kind, t,
                                            s_ang64);
            if (act) put4<D>(a.kv4 + (row0 + ((size_t)head << a.Plog2)) * Kv4<D>::REC, kind, r.x, r.y);
        }
    }
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t s)
{
    if (a.T == 0) return cudaSuccess;
    const int rpw = 256 / a.D;
    const int tasks = (a.Hq + rpw - 1) / rpw + 2 * ((a.Hkv + rpw - 1) / rpw);
    // a warp per token, or more up to 16 warps an SM: a token's heads are then
    // taken at once, at the price of its angles in each warp (512 and 2048 tokens
    // of 32 + 2 x 8 heads into bf16 pages: with 64 warps an SM 10.4 and 17.5 us,
    // 32: 7.3 and 16.1, 16: 6.5 and 13.2, 8: 5.8 and 15.7, 4: 6.3 and 15.7)
    long long wpt = (16 * 148 + a.T - 1) / a.T;
    // (a warp keeps marks of up to 64 tasks of keys and values)
    const int least = (a.Hkv + 32 * rpw - 1) / (32 * rpw);
    wpt = wpt < least ? least : wpt > tasks ? tasks : wpt;
    const dim3 grid((unsigned)(wpt * a.T));   // at most max(2368 + a.T, least a.T) blocks
    auto kern = a.kv4 ? (a.D == 64 ? k_rope_append<64, 4> : k_rope_append<128, 4>)
                      : (a.D == 64 ? k_rope_append<64, 16> : k_rope_append<128, 16>);
    return launch_pdl(kern, grid, dim3(kAppendThreads), 0, s, a, (int)wpt);
}

}  // namespace sa
