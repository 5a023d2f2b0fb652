// Attention over a layer's uncompressed keys, and the window scores it gives.
//
// Query i of sequence b sits at position p = kv_len[b] - q_len[b] + i and sees
// key j iff j <= p and (j > p - span or j < sinks).
#include "qevict_tc.cuh"

#include <math.h>

namespace qevict {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 128;                    // keys per tile
constexpr int kHalf = kTile * 128;            // bytes of 128 rows x 64 channels
constexpr int kTileBytes = 2 * kHalf;

// Key tiles a run of positions [p_lo, p_hi] sees: tiles [0, sink) and [main, end).
struct Tiles {
    int sink, main, end;
    __device__ __forceinline__ int count() const { return sink + end - main; }
    __device__ __forceinline__ int key(int i) const { return (i < sink ? i : main + i - sink) * kTile; }
};
__device__ __forceinline__ Tiles tiles_of(const SpanArgs &a, int p_lo, int p_hi) {
    const int lo = max(0, p_lo - a.span + 1);
    Tiles t;
    t.main = lo / kTile;
    t.end = p_hi < 0 ? t.main : p_hi / kTile + 1;
    t.sink = min((min(a.sinks, lo) + kTile - 1) / kTile, t.main);
    if (p_hi < 0) t.sink = 0;
    return t;
}
__device__ __forceinline__ bool visible(const SpanArgs &a, int j, int p) {
    return j <= p && (j > p - a.span || j < a.sinks);
}
// whether some pair of keys [k0, k0 + 128) and positions [p_lo, p_hi] is masked
__device__ __forceinline__ bool masked_tile(const SpanArgs &a, int k0, int p_lo, int p_hi) {
    return !(k0 + kTile - 1 <= p_lo && (k0 > p_hi - a.span || k0 + kTile <= a.sinks));
}

__device__ __forceinline__ int clamped(const int32_t *len, int b, int n) {
    return len ? min(max(len[b], 0), n) : n;
}

// One query tile (the rows of 128 / G tokens, token-major, of one KV head's
// group) against its key tiles one by one.
__global__ void __launch_bounds__(128) span_attention_simple(const SpanArgs a, const CacheDev C, int layer,
                                                             const __grid_constant__ CUtensorMap qmap,
                                                             const __grid_constant__ CUtensorMap kmap,
                                                             const __grid_constant__ CUtensorMap vmap,
                                                             __nv_bfloat16 *out, float *lse) {
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[3];   // q + k loaded, v loaded, products done
    __shared__ uint32_t slot;
    __shared__ int stop;
    const int b = blockIdx.z, kvh = blockIdx.y;
    const int T = span_tile_tokens(a.G), rows = T * a.G;
    const int i0 = blockIdx.x * T;
    const int q_len = clamped(a.q_len, b, a.n_q), kv_len = clamped(a.kv_len, b, a.n_kv);
    if (i0 >= q_len) return;
    const int n_tok = min(T, q_len - i0);
    const int shift = kv_len - q_len;
    const int p_lo = shift + i0, p_hi = p_lo + n_tok - 1;
    const Tiles tl = tiles_of(a, p_lo, p_hi);

    const uint32_t sm = (smem_u32(raw) + 1023) & ~1023u;
    const uint32_t sq = sm, sk = sm + kTileBytes, sv = sm + 2 * kTileBytes;
    uint8_t *gen = raw + (sm - smem_u32(raw));
    const int tid = threadIdx.x, warp = tid >> 5;
    const uint32_t b_k = smem_u32(&bars[0]), b_v = smem_u32(&bars[1]), b_m = smem_u32(&bars[2]);
    if (tid == 0) {
        tc_mbar_init(b_k, 1);
        tc_mbar_init(b_v, 1);
        tc_mbar_init(b_m, 1);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tc_alloc<256>(smem_u32(&slot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = slot, lane_tm = tm + ((uint32_t)(warp * 32) << 16);
    const uint32_t tS = 0, tO = 128;
    const float c = kLog2e * rsqrtf((float)kHeadDim);

    const int t = tid / a.G, pos = p_lo + t;
    const bool valid = tid < rows && t < n_tok;
    float m = -INFINITY, l = 0.f;
    uint32_t ph_k = 0, ph_m = 0;
    bool ok = true;
    for (int it = 0; it < tl.count() && ok; ++it) {
        const int k0 = tl.key(it);
        if (tid == 0) {
            tc_expect_tx(b_k, kTileBytes + (it == 0 ? rows * 256 : 0));
            if (it == 0)
                for (int h = 0; h < 2; ++h) tc_tma_4d(sq + h * kHalf, &qmap, 64 * h, kvh * a.G, i0, b, b_k);
            for (int h = 0; h < 2; ++h) tc_tma_4d(sk + h * kHalf, &kmap, 64 * h, kvh, k0, b, b_k);
            tc_expect_tx(b_v, kTileBytes);
            for (int h = 0; h < 2; ++h) tc_tma_4d(sv + h * kHalf, &vmap, 64 * h, kvh, k0, b, b_v);
        }
        ok = tc_wait(b_k, ph_k, &stop) && tc_wait(b_v, ph_k, &stop);
        ph_k ^= 1;
        const int j = k0 + tid;
        if (j > p_hi || (j <= p_lo - a.span && j >= a.sinks)) {   // a key no row sees may hold anything
            for (int x = 0; x < 8; ++x) {
                *reinterpret_cast<int4 *>(gen + 2 * kTileBytes + tid * 128 + x * 16) = make_int4(0, 0, 0, 0);
                *reinterpret_cast<int4 *>(gen + 2 * kTileBytes + kHalf + tid * 128 + x * 16) = make_int4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        ok = __syncthreads_and(ok);
        if (!ok) break;
        if (tid == 0) {
            for (int s = 0; s < 8; ++s) {
                const uint32_t o = (s >> 2) * kHalf + (s & 3) * 32;
                tc_mma_ss(tm + tS, tc_desc_k(sq + o), tc_desc_k(sk + o), tc_idesc(false), s > 0);
            }
            tc_commit(b_m);
        }
        ok = tc_wait(b_m, ph_m, &stop);
        ph_m ^= 1;
        tc_fence_after();
        float x[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tc_ld32(lane_tm + tS + 32 * q, x[q]);
        tc_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) tc_tie(x[q]);
        const bool mt = masked_tile(a, k0, p_lo, p_hi);
        float mx = m;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                if (mt && !visible(a, k0 + 32 * q + e, pos)) x[q][e] = -INFINITY;
                mx = fmaxf(mx, x[q][e]);
            }
        const float f = m == -INFINITY ? 0.f : tc_ex2((m - mx) * c);
        m = mx;
        const float mc = m == -INFINITY ? 0.f : m * c;
        l *= f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float u = tc_ex2(fmaf(x[q][2 * e], c, -mc)), v = tc_ex2(fmaf(x[q][2 * e + 1], c, -mc));
                l += u + v;
                const __nv_bfloat162 pk = __floats2bfloat162_rn(u, v);
                p[e] = *reinterpret_cast<const uint32_t *>(&pk);
            }
            tc_st16(lane_tm + tS + 16 * q, p);
        }
        if (it > 0) {   // the output so far moves to the new maximum
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float o[32];
                tc_ld32(lane_tm + tO + 32 * q, o);
                tc_wait_ld();
                tc_tie(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f;
                tc_st32(lane_tm + tO + 32 * q, o);
            }
        }
        tc_wait_st();
        tc_fence_before();
        ok = __syncthreads_and(ok);
        if (!ok) break;
        if (tid == 0) {
            tc_fence_after();
            for (int s = 0; s < 8; ++s)
                tc_mma_ts(tm + tO, tm + tS + 8 * s, tc_desc_mn(sv + s * 2048, kHalf), tc_idesc(true), it > 0 || s > 0);
            tc_commit(b_m);
        }
        ok = tc_wait(b_m, ph_m, &stop);
        ph_m ^= 1;
        tc_fence_after();
        ok = __syncthreads_and(ok);
    }
    const float inv = 1.f / l;
    const bool none = l == 0.f;   // no key seen
    __nv_bfloat16 *orow = out + (((int64_t)b * a.n_q + i0 + t) * a.Hq + kvh * a.G + tid % a.G) * kHeadDim;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float o[32];
        tc_ld32(lane_tm + tO + 32 * q, o);
        tc_wait_ld();
        tc_tie(o);
        if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 2)
                *reinterpret_cast<__nv_bfloat162 *>(orow + 32 * q + e) =
                    none ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
        }
        __syncwarp();
    }
    if (valid && lse)
        lse[((int64_t)b * a.Hq + kvh * a.G + tid % a.G) * a.n_q + i0 + t] =
            none ? -INFINITY : m * rsqrtf((float)kHeadDim) + logf(l);
    if (tid == 0 && (stop || !ok)) set_status(C, QEVICT_ERR_TIMEOUT, layer, b, kvh);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tc_free<256>(tm);
}

// Window scores: one CTA per (key tile, sequence), or per (key tile, sequence,
// KV head) with per-head units. The logits are computed transposed, keys as
// the 128 lanes and the rows of a query tile as the 128 columns, so that a key's
// mass is a sum over its own lane's registers.
__global__ void __launch_bounds__(128) span_scores_simple(const SpanArgs a, const CacheDev C, int layer,
                                                          const __grid_constant__ CUtensorMap qmap,
                                                          const __grid_constant__ CUtensorMap kmap, const float *lse,
                                                          float *scores, int w, int n_win, int per_head) {
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2];
    __shared__ uint32_t slot;
    __shared__ int stop;
    __shared__ float ls[kTile], keys[kTile];
    __shared__ int ps[kTile];
    const int b = blockIdx.y;
    const int tk = kTile / w * w;   // whole windows of one tile
    const int k0 = blockIdx.x * tk;
    const int T = span_tile_tokens(a.G), rows = T * a.G;
    const int q_len = clamped(a.q_len, b, a.n_q), kv_len = clamped(a.kv_len, b, a.n_kv);
    const int shift = kv_len - q_len;
    const int k_hi = min(k0 + tk, kv_len) - 1;
    // queries that see some key of the tile
    int i_lo = max(0, k0 - shift), i_hi = q_len;
    if (k0 >= a.sinks) i_hi = min(i_hi, k_hi + a.span - shift);
    if (k_hi < k0) i_hi = 0;

    const uint32_t sm = (smem_u32(raw) + 1023) & ~1023u;
    const uint32_t sk = sm, sq = sm + kTileBytes;
    uint8_t *gen = raw + (sm - smem_u32(raw));
    const int tid = threadIdx.x, warp = tid >> 5;
    const uint32_t b_l = smem_u32(&bars[0]), b_m = smem_u32(&bars[1]);
    if (tid == 0) {
        tc_mbar_init(b_l, 1);
        tc_mbar_init(b_m, 1);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tc_alloc<128>(smem_u32(&slot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = slot, lane_tm = tm + ((uint32_t)(warp * 32) << 16);
    const float c = kLog2e * rsqrtf((float)kHeadDim);
    const int j = k0 + tid;
    const bool mine = tid < tk && j < kv_len;
    float sum = 0.f;
    uint32_t ph = 0;
    bool ok = true;
    const int h0 = per_head ? blockIdx.z : 0, h1 = per_head ? h0 + 1 : a.Hkv;
    for (int kvh = h0; kvh < h1 && ok; ++kvh)
        for (int i0 = i_lo / T * T; i0 < i_hi && ok; i0 += T) {
            if (tid == 0) {
                const bool first = i0 == i_lo / T * T;
                tc_expect_tx(b_l, rows * 256 + (first ? kTileBytes : 0));
                for (int h = 0; h < 2; ++h) {
                    if (first) tc_tma_4d(sk + h * kHalf, &kmap, 64 * h, kvh, k0, b, b_l);
                    tc_tma_4d(sq + h * kHalf, &qmap, 64 * h, kvh * a.G, i0, b, b_l);
                }
            }
            {
                const int i = i0 + tid / a.G;
                const bool v = tid < rows && i < q_len;
                ps[tid] = v ? shift + i : -1;
                ls[tid] = v ? lse[((int64_t)b * a.Hq + kvh * a.G + tid % a.G) * a.n_q + i] * kLog2e : 0.f;
            }
            ok = tc_wait(b_l, ph, &stop);
            ok = __syncthreads_and(ok);
            if (!ok) break;
            if (tid == 0) {
                for (int s = 0; s < 8; ++s) {
                    const uint32_t o = (s >> 2) * kHalf + (s & 3) * 32;
                    tc_mma_ss(tm, tc_desc_k(sk + o), tc_desc_k(sq + o), tc_idesc(false), s > 0);
                }
                tc_commit(b_m);
            }
            ok = tc_wait(b_m, ph, &stop);
            ph ^= 1;
            tc_fence_after();
            for (int q = 0; q < 4; ++q) {
                float x[32];
                tc_ld32(lane_tm + 32 * q, x);
                tc_wait_ld();
                tc_tie(x);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float y = tc_ex2(fmaf(x[e], c, -ls[32 * q + e]));
                    if (visible(a, j, ps[32 * q + e])) sum += y;
                }
            }
            tc_fence_before();
            ok = __syncthreads_and(ok);
        }
    keys[tid] = mine ? sum : 0.f;
    __syncthreads();
    const int win = k0 / w + tid;
    if (tid < tk / w && win < n_win) {
        float y = 0.f;
        for (int e = 0; e < w; ++e) y += keys[tid * w + e];
        const int u = per_head ? b * a.Hkv + blockIdx.z : b;
        scores[(int64_t)u * n_win + win] = y / (per_head ? a.G : a.Hq);
    }
    if (tid == 0 && !ok) set_status(C, QEVICT_ERR_TIMEOUT, layer, b, k0);
    __syncthreads();
    if (warp == 0) tc_free<128>(tm);
    (void)gen;
}

}  // namespace

cudaError_t launch_span_attention(const SpanArgs &a, const CacheDev &C, int layer, const CUtensorMap &qmap,
                                  const CUtensorMap &kmap, const CUtensorMap &vmap, __nv_bfloat16 *out, float *lse,
                                  int num_sms, cudaStream_t s) {
    constexpr int smem = 3 * kTileBytes + 1024 + 32768;   // above half an SM's: one CTA per SM owns its tensor memory
    cudaError_t e = once_per_device(0, [&] {
        return cudaFuncSetAttribute(span_attention_simple, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    const int T = span_tile_tokens(a.G);
    const dim3 grid((a.n_q + T - 1) / T, a.Hkv, a.B);
    span_attention_simple<<<grid, 128, smem, s>>>(a, C, layer, qmap, kmap, vmap, out, lse);
    return cudaGetLastError();
}

cudaError_t launch_span_scores(const SpanArgs &a, const CacheDev &C, int layer, const CUtensorMap &qmap,
                               const CUtensorMap &kmap, const float *lse, float *scores, int w, bool per_head,
                               int num_sms, cudaStream_t s) {
    constexpr int smem = 2 * kTileBytes + 1024;
    cudaError_t e = once_per_device(0, [&] {
        return cudaFuncSetAttribute(span_scores_simple, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    const int tk = kTile / w * w;
    const int n_win = (a.n_kv + w - 1) / w;
    const dim3 grid((a.n_kv + tk - 1) / tk, a.B, per_head ? a.Hkv : 1);
    span_scores_simple<<<grid, 128, smem, s>>>(a, C, layer, qmap, kmap, lse, scores, w, n_win, per_head);
    return cudaGetLastError();
}

}  // namespace qevict
