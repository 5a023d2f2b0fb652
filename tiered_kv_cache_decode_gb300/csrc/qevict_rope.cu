// Head norms and rotation of a projection's queries and keys, in one pass.
//
// For every token and head x (128 bf16 channels): y = x / sqrt(mean(x^2) + eps) * w
// (no w: y = x), then each channel pair (a, b) turns by the angle position *
// inv_freq[pair]: (a cos - b sin, b cos + a sin). Values are copied. The sums,
// the angle and the products are fp32, rounded to bf16 once at the store.
#include "qevict_internal.cuh"

namespace qevict {
namespace {

constexpr int kRopeRows = 16;     // heads of one token per warp

// inv_freq / (2 pi) turns per position as a fraction of 2^64, in integers: with
// inv_freq = m 2^(E - 150), m * round(2^66 / (2 pi)) * 2^(E - 152) mod 2^64. The
// product with a 64-bit position then wraps at whole turns exactly; what is left
// of an error is the fraction's own, about 2^-64 turns per position (2^-27
// turns, 4.7e-8 rad, at position 2^37).
__device__ __forceinline__ uint64_t turn_fraction(float f) {
    const uint32_t u = __float_as_uint(f);
    const int E = max(1, (int)((u >> 23) & 0xff));
    const uint64_t m = (u & 0x7fffff) | ((u & 0x7f800000) ? 0x800000u : 0u);
    constexpr uint64_t kInv2Pi = 0xA2F9836E4E44152Aull;   // 2^66 / (2 pi)
    const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
    const int s = 152 - E;
    uint64_t r;
    if (s >= 128) r = 0;
    else if (s >= 64) r = hi >> (s - 64);
    else if (s > 0) r = (lo >> s) | (hi << (64 - s));
    else r = -s < 64 ? lo << -s : 0;
    return (u >> 31) ? 0ull - r : r;
}

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// One warp, a CTA of its own, takes up to 16 heads of one token. Eight lanes hold a
// head: lane l its channels 8 l .. 8 l + 7 and 64 + 8 l .. + 7 (two 16-byte loads), so
// both members of every pair, half-split (i, i + 64) or interleaved (2 i, 2 i + 1),
// lie in one lane and only the sum of squares crosses lanes. The warp's lanes
// compute the token's 64 angles once, two each, and hand them round.
// Memory-bound: every byte is read and written once, four 32-byte reads per lane
// in flight. CTAs of one warp replace one another as each ends: a 32K prompt (32
// query, 8 KV heads, with norms and values, 805 MB) takes 122 us (6.6 TB/s), 133
// with two warps to a CTA, 136 with four, 157 with eight.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(32) rope_kernel(const RopeArgs a, const int32_t *ctr, int ctr_stride, int chunks) {
    const int lane = threadIdx.x;
    const int64_t u = blockIdx.x;
    const int64_t tok = u / chunks;
    const int r0 = (int)(u - tok * chunks) * kRopeRows;
    const int R = a.Hq + a.Hkv + (a.v ? a.Hkv : 0);
    const int l = lane & 7, g = lane >> 3;

    const int4 *src[4];
    int4 x[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * i + g;
        const __nv_bfloat16 *p = r < a.Hq ? a.q + tok * a.q_stride + (int64_t)r * kHeadDim
                                 : r < a.Hq + a.Hkv ? a.k + tok * a.k_stride + (int64_t)(r - a.Hq) * kHeadDim
                                                    : a.v + tok * a.v_stride + (int64_t)(r - a.Hq - a.Hkv) * kHeadDim;
        src[i] = reinterpret_cast<const int4 *>(p) + l;
        if (r < R) {
            x[i][0] = src[i][0];
            x[i][1] = src[i][8];
        } else {
            x[i][0] = x[i][1] = make_int4(0, 0, 0, 0);
        }
    }
    // angles: lane j computes pairs 2 j and 2 j + 1
    float cs[8], sn[8];   // of this lane's pairs: elements 0..3 of each half in turn when interleaved
    if (r0 < a.Hq + a.Hkv) {
        const int64_t pos = a.positions ? a.positions[tok]
                                        : (int64_t)ctr[(tok / a.n_tokens) * ctr_stride + CTR_LEN] + tok % a.n_tokens;
        const float2 f = *reinterpret_cast<const float2 *>(a.inv_freq + 2 * lane);
        float c0, s0, c1, s1;
        const int64_t t0 = (int64_t)((uint64_t)pos * turn_fraction(f.x));
        const int64_t t1 = (int64_t)((uint64_t)pos * turn_fraction(f.y));
        // all 64 bits, so that a small angle keeps fp32's relative accuracy
        sincospif((float)t0 * 0x1p-63f, &s0, &c0);
        sincospif((float)t1 * 0x1p-63f, &s1, &c1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // half-split: pairs 8 l + 2 j, + 1; interleaved: pairs 4 l + .. of the low half, 32 + 4 l + .. of the high
            const int from = INTERLEAVED ? (j < 2 ? 2 * l + j : 16 + 2 * l + j - 2) : 4 * l + j;
            cs[2 * j] = __shfl_sync(~0u, c0, from);
            sn[2 * j] = __shfl_sync(~0u, s0, from);
            cs[2 * j + 1] = __shfl_sync(~0u, c1, from);
            sn[2 * j + 1] = __shfl_sync(~0u, s1, from);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * i + g;
        const bool isq = r < a.Hq, isk = !isq && r < a.Hq + a.Hkv;
        const __nv_bfloat16 *w = isq ? a.q_weight : a.k_weight;
        float y[16];
        const uint32_t *xw = reinterpret_cast<const uint32_t *>(&x[i][0]);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[2 * e] = bf_lo(xw[e]);
            y[2 * e + 1] = bf_hi(xw[e]);
            ss = fmaf(y[2 * e], y[2 * e], ss);
            ss = fmaf(y[2 * e + 1], y[2 * e + 1], ss);
        }
#pragma unroll
        for (int o = 4; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        if (r >= R) continue;
        int4 z[2] = {x[i][0], x[i][1]};
        if (isq || isk) {
            if (w) {
                const float inv = 1.f / sqrtf(fmaf(ss, 1.f / kHeadDim, a.eps));
                const int4 wv[2] = {__ldg(reinterpret_cast<const int4 *>(w) + l),
                                    __ldg(reinterpret_cast<const int4 *>(w) + 8 + l)};
                const uint32_t *ww = reinterpret_cast<const uint32_t *>(&wv[0]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[2 * e] = y[2 * e] * inv * bf_lo(ww[e]);
                    y[2 * e + 1] = y[2 * e + 1] * inv * bf_hi(ww[e]);
                }
            }
            uint32_t *zw = reinterpret_cast<uint32_t *>(&z[0]);
            if (INTERLEAVED) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    zw[e] = pack(y[2 * e] * cs[e] - y[2 * e + 1] * sn[e], y[2 * e + 1] * cs[e] + y[2 * e] * sn[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    zw[e] = pack(y[2 * e] * cs[2 * e] - y[8 + 2 * e] * sn[2 * e],
                                 y[2 * e + 1] * cs[2 * e + 1] - y[9 + 2 * e] * sn[2 * e + 1]);
                    zw[4 + e] = pack(y[8 + 2 * e] * cs[2 * e] + y[2 * e] * sn[2 * e],
                                     y[9 + 2 * e] * cs[2 * e + 1] + y[2 * e + 1] * sn[2 * e + 1]);
                }
            }
        }
        __nv_bfloat16 *d = isq ? a.q_out + (tok * a.Hq + r) * kHeadDim
                           : isk ? a.k_out + (tok * a.Hkv + r - a.Hq) * kHeadDim
                                 : a.v_out + (tok * a.Hkv + r - a.Hq - a.Hkv) * kHeadDim;
        reinterpret_cast<int4 *>(d)[l] = z[0];
        reinterpret_cast<int4 *>(d)[8 + l] = z[1];
    }
}

}  // namespace

cudaError_t launch_rope(const LayerDev &L, const RopeArgs &a, cudaStream_t s) {
    const int R = a.Hq + a.Hkv + (a.v ? a.Hkv : 0);
    const int chunks = (R + kRopeRows - 1) / kRopeRows;
    const int64_t grid = a.tokens * chunks;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    auto kernel = a.interleaved ? rope_kernel<true> : rope_kernel<false>;
    kernel<<<(unsigned)grid, 32, 0, s>>>(a, L.ctr, L.hs * kCtrN, chunks);
    return cudaGetLastError();
}

}  // namespace qevict
