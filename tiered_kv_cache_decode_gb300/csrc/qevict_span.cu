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

// ---- attention ----------------------------------------------------------------
//
// Rows are (token, query head of one KV head's group), token-major, 128 / G
// tokens to a tile of 128 rows, so every head of the group shares the tile's keys.
// Ten warps: two softmax warpgroups (a thread owns a row), one thread that
// issues the products, one that issues the copies. Tensor memory holds a logit
// tile S and an output tile O (fp32, 128 x 128) per softmax group; the
// probabilities overwrite their logits as bf16 and are the A operand of P V
// from there, so neither S nor P leaves the SM. While one group is in its
// softmax, the tensor cores work for the other.
//
// Wide: the groups take two neighbouring query tiles over the same keys.
// Split: both take one query tile, every other key tile each, and the key tiles
// are further divided over the CTAs of a cluster; the partial (max, sum, O)
// meet in shared memory. No scratch in device memory either way.
constexpr int kSoftmax = 256;                 // threads of the two softmax groups
constexpr int kAttThreads = kSoftmax + 128;   // and a group of four warps for copies and products
constexpr int kAttSlots = 7;                  // 32 KB slots of shared memory: query tiles, then the key/value ring
constexpr int kAttSmem = kAttSlots * kTileBytes + 1024;
constexpr float kRescale = 8.f;               // log2 growth of a row's maximum that moves its reference

template <bool SPLIT>
__global__ void __launch_bounds__(kAttThreads, 1)
    span_attention_kernel(const SpanArgs a, const CacheDev C, int layer, const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          __nv_bfloat16 *out, float *lse, int q_tiles, int cl) {
    constexpr int QT = SPLIT ? 1 : 2;              // query tiles of the CTA
    constexpr int NS = kAttSlots - QT;             // ring slots
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * NS + 7];
    __shared__ uint32_t slot;
    __shared__ int stop;

    const int T = span_tile_tokens(a.G), rows = T * a.G;
    const int unit = blockIdx.x / cl, rank = blockIdx.x - unit * cl;
    const int heads = a.B * a.Hkv;
    const int qt = q_tiles - 1 - unit / heads;     // the longest rows of keys first
    const int b = unit % heads / a.Hkv, kvh = unit % a.Hkv;
    const int i0 = qt * QT * T;
    const int q_len = clamped(a.q_len, b, a.n_q), kv_len = clamped(a.kv_len, b, a.n_kv);
    if (i0 >= q_len) return;                       // all CTAs of the cluster alike
    const int n_tok = min(QT * T, q_len - i0);
    const int p_lo = kv_len - q_len + i0, p_hi = p_lo + n_tok - 1;
    const Tiles tl = tiles_of(a, p_lo, p_hi);
    const int all = tl.count();
    const int first = SPLIT ? (int)((int64_t)all * rank / cl) : 0;
    const int n = (SPLIT ? (int)((int64_t)all * (rank + 1) / cl) : all) - first;   // key tiles of this CTA

    const uint32_t sm = (smem_u32(raw) + 1023) & ~1023u;
    uint8_t *gen = raw + (sm - smem_u32(raw));
    const uint32_t ring = sm + QT * kTileBytes;
    const int tid = threadIdx.x, warp = tid >> 5;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8 * s; };
    auto empty = [&](int s) { return bar0 + 8 * (NS + s); };
    auto s_full = [&](int t) { return bar0 + 8 * (2 * NS + t); };
    auto p_full = [&](int t) { return bar0 + 8 * (2 * NS + 2 + t); };
    auto o_full = [&](int t) { return bar0 + 8 * (2 * NS + 4 + t); };
    const uint32_t q_full = bar0 + 8 * (2 * NS + 6);
    if (tid == 0) {
        for (int i = 0; i < 2 * NS + 7; ++i) tc_mbar_init(bar0 + 8 * i, i == 2 * NS + 2 || i == 2 * NS + 3 ? 4 : 1);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tc_alloc<512>(smem_u32(&slot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = slot;                      // S of group t at column 128 t, O at 256 + 128 t
    // ring order: the order in which the products use the tiles
    auto k_item = [&](int j) { return SPLIT ? (j ? 2 * j - 1 : 0) : 2 * j; };
    auto v_item = [&](int j) { return SPLIT ? min(2 * j + 2, 2 * n - 1) : 2 * j + 1; };

    // 12 warps start with 168 registers a thread; the softmax groups take 224 and leave 40
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (tid == 9 * 32 && n > 0) {
            tc_expect_tx(q_full, QT * rows * 256);
            for (int t = 0; t < QT; ++t)
                for (int h = 0; h < 2; ++h)
                    tc_tma_4d(sm + t * kTileBytes + h * kHalf, &qmap, 64 * h, kvh * a.G, i0 + t * T, b, q_full);
            int i = 0;
            for (; i < 2 * n; ++i) {
                const int s = i % NS;
                if (i >= NS && !tc_wait(empty(s), (i / NS - 1) & 1, &stop)) break;
                const bool isk = SPLIT ? i == 0 || (i & 1 && i < 2 * n - 1) : !(i & 1);
                const int j = SPLIT ? (isk ? (i + 1) / 2 : i == 2 * n - 1 ? n - 1 : i / 2 - 1) : i / 2;
                tc_expect_tx(full(s), kTileBytes);
                for (int h = 0; h < 2; ++h)
                    tc_tma_4d(ring + s * kTileBytes + h * kHalf, isk ? &kmap : &vmap, 64 * h, kvh, tl.key(first + j), b,
                              full(s));
            }
            if (i < 2 * n) {   // gave up: the copies in flight land before the CTA ends
                for (int o = max(0, i - NS); o < i; ++o) {
                    const long long t0 = clock64();
                    while (!tc_try_wait(full(o % NS), (o / NS) & 1) && clock64() - t0 < kDefaultWaitCycles) {}
                }
            }
        }
        if (tid == 8 * 32 && n > 0) {
            bool ok = tc_wait(q_full, 0, &stop);
            auto logits = [&](int t, int j) {   // S_t = Q K_j^T
                const uint32_t k = ring + k_item(j) % NS * kTileBytes, q = sm + (SPLIT ? 0 : t * kTileBytes);
                for (int s = 0; s < 8; ++s) {
                    const uint32_t o = (s >> 2) * kHalf + (s & 3) * 32;
                    tc_mma_ss(tm + 128 * t, tc_desc_k(q + o), tc_desc_k(k + o), tc_idesc(false), s > 0);
                }
                tc_commit(s_full(t));
            };
            auto wait_item = [&](int i) {
                ok = ok && tc_wait(full(i % NS), (i / NS) & 1, &stop);
                return ok;
            };
            if (wait_item(k_item(0))) {
                logits(0, 0);
                if (!SPLIT) logits(1, 0);
                tc_commit(empty(k_item(0) % NS));
            }
            if (SPLIT && n > 1 && wait_item(k_item(1))) {
                logits(1, 1);
                tc_commit(empty(k_item(1) % NS));
            }
            for (int j = 0; j < n && ok; ++j) {
                if (!wait_item(v_item(j))) break;
                const uint32_t v = ring + v_item(j) % NS * kTileBytes;
                const int ahead = SPLIT ? j + 2 : j + 1;
                for (int x = 0; x < QT && ok; ++x) {
                    const int t = SPLIT ? j & 1 : x;
                    ok = tc_wait(p_full(t), (SPLIT ? j >> 1 : j) & 1, &stop);
                    if (!ok) break;
                    tc_fence_after();
                    for (int s = 0; s < 8; ++s)
                        tc_mma_ts(tm + 256 + 128 * t, tm + 128 * t + 8 * s, tc_desc_mn(v + s * 2048, kHalf), tc_idesc(true),
                                  j >= (SPLIT ? 2 : 1) || s > 0);
                    if (x == QT - 1) tc_commit(empty(v_item(j) % NS));
                    if (ahead < n) {
                        if (!wait_item(k_item(ahead))) break;
                        logits(t, ahead);
                        if (x == QT - 1) tc_commit(empty(k_item(ahead) % NS));
                    } else {
                        tc_commit(o_full(t));
                    }
                }
            }
            if (!ok) {   // gave up: the products in flight end before the tensor memory is freed
                tc_commit(q_full);
                const long long t0 = clock64();
                while (!tc_try_wait(q_full, 1) && clock64() - t0 < kDefaultWaitCycles) {}
            }
        }
        __syncwarp();
        if (SPLIT) {
            if (cl > 1) cl_sync(), cl_sync();
            else __syncthreads();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lane_tm = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lane_tm + 128 * t, tO = lane_tm + 256 + 128 * t;
        const float c = kLog2e * rsqrtf((float)kHeadDim);
        const int tok = (SPLIT ? 0 : t * T) + r / a.G;
        const int pos = p_lo + tok;
        const bool valid = r < rows && tok < n_tok;
        const int g_lo = p_lo + (SPLIT ? 0 : t * T), g_hi = min(p_hi, g_lo + T - 1);   // this group's positions
        float m = -INFINITY, l = 0.f;
        const uint64_t cc = pair2(c, c);
        bool ok = true;
        int done = 0;
        for (int j = SPLIT ? t : 0; j < n; j += SPLIT ? 2 : 1, ++done) {
            ok = __all_sync(~0u, tc_wait(s_full(t), done & 1, &stop));   // a warp stops as one
            if (!ok) break;
            tc_fence_after();
            const int k0 = tl.key(first + j);
            float x[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tc_ld32(tS + 32 * q, x[q]);
            tc_wait_ld();
#pragma unroll
            for (int q = 0; q < 4; ++q) tc_tie(x[q]);
            if (masked_tile(a, k0, g_lo, g_hi)) {
                const int hi = pos - k0, lo = hi - a.span, sk = a.sinks - k0;
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * q + e > hi || (32 * q + e <= lo && 32 * q + e >= sk)) x[q][e] = -INFINITY;
            }
            float mx[4] = {x[0][0], x[1][0], x[2][0], x[3][0]};
#pragma unroll
            for (int e = 1; e < 32; ++e)
#pragma unroll
                for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], x[q][e]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            // The reference follows the maximum only when it has grown by more than
            // kRescale in the exponent: probabilities stay below 2^kRescale, and O is
            // rarely touched between its products.
            if (__any_sync(~0u, (top - m) * c > kRescale)) {
                const float mn = fmaxf(m, top);
                const float f = m == -INFINITY ? 0.f : tc_ex2((m - mn) * c);
                m = mn;
                l *= f;
                if (done > 0) {   // the product before it has ended: its logits came after it
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float o[32];
                        tc_ld32(tO + 32 * q, o);
                        tc_wait_ld();
                        tc_tie(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tc_st32(tO + 32 * q, o);
                    }
                }
            }
            const float mc = m == -INFINITY ? 0.f : -m * c;
            const uint64_t mm = pair2(mc, mc);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float u, v;
                    split2(fma2(pair2(x[q][2 * e], x[q][2 * e + 1]), cc, mm), u, v);
                    u = tc_ex2(u);
                    v = tc_ex2(v);
                    sum[e & 1] = add2(sum[e & 1], pair2(u, v));
                    const __nv_bfloat162 pk = __floats2bfloat162_rn(u, v);
                    p[e] = *reinterpret_cast<const uint32_t *>(&pk);
                }
                tc_st16(tS + 16 * q, p);
            }
            float s0, s1;
            split2(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
            // Values of keys that no row of the CTA sees may be anything: as zeros they stay out of the product.
            if ((SPLIT || t == 0) && (k0 + kTile - 1 > p_hi || (k0 <= p_lo - a.span && k0 + kTile > a.sinks))) {
                const int i = v_item(j), s = i % NS;
                ok = __all_sync(~0u, tc_wait(full(s), (i / NS) & 1, &stop));
                if (!ok) break;
                const int key = k0 + r;
                if (key > p_hi || (key <= p_lo - a.span && key >= a.sinks)) {
                    uint8_t *v = gen + (QT + s) * kTileBytes + r * 128;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        *reinterpret_cast<int4 *>(v + 16 * y) = make_int4(0, 0, 0, 0);
                        *reinterpret_cast<int4 *>(v + kHalf + 16 * y) = make_int4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if ((tid & 31) == 0) tc_arrive(p_full(t));
        }
        if (ok && done > 0) ok = __all_sync(~0u, tc_wait(o_full(t), 0, &stop));
        tc_fence_after();
        if (!SPLIT) {
            const float inv = 1.f / l;
            const bool none = l == 0.f;   // no key seen
            const int64_t head = kvh * a.G + r % a.G;
            uint32_t *dst = reinterpret_cast<uint32_t *>(out + (((int64_t)b * a.n_q + i0 + tok) * a.Hq + head) * kHeadDim);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float o[32];
                tc_ld32(tO + 32 * q, o);
                tc_wait_ld();
                tc_tie(o);
                if (valid && ok) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t p[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const __nv_bfloat162 pk = __floats2bfloat162_rn(none ? 0.f : o[e + 2 * y] * inv,
                                                                            none ? 0.f : o[e + 2 * y + 1] * inv);
                            p[y] = *reinterpret_cast<const uint32_t *>(&pk);
                        }
                        *reinterpret_cast<uint4 *>(dst + 16 * q + e / 2) = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                }
                __syncwarp();
            }
            if (valid && ok && lse)
                lse[((int64_t)b * a.Hq + head) * a.n_q + i0 + tok] =
                    none ? -INFINITY : m * rsqrtf((float)kHeadDim) + logf(l);
        } else {
            // both groups' products have read the ring: it holds the partial outputs now
            asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory");
            float2 *stat = reinterpret_cast<float2 *>(gen + 5 * kTileBytes) + t * kTile;   // (max, sum) of the rows
            stat[r] = done > 0 ? make_float2(m * c, l) : make_float2(-INFINITY, 0.f);
            float4 *part = reinterpret_cast<float4 *>(gen + kTileBytes + t * 2 * kTileBytes) + r * 32;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float o[32];
                tc_ld32(tO + 32 * q, o);
                tc_wait_ld();
                tc_tie(o);
                if (valid && done > 0 && ok) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)   // the swizzle spreads a warp's rows over the banks
                        part[(8 * q + e) ^ (r & 31)] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
                __syncwarp();
            }
            __syncwarp();
            if (cl > 1) cl_sync();
            else __syncthreads();
            {
                const uint32_t st = ring + 4 * kTileBytes;
                for (int i = rank * kSoftmax + tid; i < n_tok * a.G * 32; i += cl * kSoftmax) {
                    const int r = i >> 5, ch = i & 31;
                    float top = -INFINITY;
                    for (int x = 0; x < 2 * cl; ++x)
                        top = fmaxf(top, cl_ld1(cl_addr(st + (x & 1) * kTile * 8 + r * 8, x >> 1)));
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    float l = 0.f;
                    for (int x = 0; x < 2 * cl; ++x) {
                        const float2 s = cl_ld2(cl_addr(st + (x & 1) * kTile * 8 + r * 8, x >> 1));
                        if (s.y == 0.f) continue;   // saw no key (a sum of NaN goes on)
                        const float f = s.x == -INFINITY ? 1.f : tc_ex2(s.x - top);
                        const float4 y = cl_ld4(cl_addr(ring + (x & 1) * 2 * kTileBytes + r * 512 + 16 * (ch ^ (r & 31)), x >> 1));
                        l = fmaf(s.y, f, l);
                        o.x = fmaf(y.x, f, o.x);
                        o.y = fmaf(y.y, f, o.y);
                        o.z = fmaf(y.z, f, o.z);
                        o.w = fmaf(y.w, f, o.w);
                    }
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    const int64_t head = kvh * a.G + r % a.G;
                    __nv_bfloat162 p[2] = {__floats2bfloat162_rn(o.x * inv, o.y * inv), __floats2bfloat162_rn(o.z * inv, o.w * inv)};
                    *reinterpret_cast<uint2 *>(out + (((int64_t)b * a.n_q + i0 + r / a.G) * a.Hq + head) * kHeadDim + 4 * ch) =
                        *reinterpret_cast<const uint2 *>(p);
                    if (ch == 0 && lse)
                        lse[((int64_t)b * a.Hq + head) * a.n_q + i0 + r / a.G] =
                            l == 0.f ? -INFINITY : (top == -INFINITY ? 0.f : top) * (1.f / kLog2e) + logf(l);
                }
            }
            __syncwarp();
            if (cl > 1) cl_sync();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && stop) set_status(C, QEVICT_ERR_TIMEOUT, layer, b, kvh);
    if (warp == 0) tc_free<512>(tm);
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
    cudaError_t e = once_per_device(0, [&] {
        cudaError_t r = cudaFuncSetAttribute(span_attention_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kAttSmem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(span_attention_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttSmem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(span_attention_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return r;
    });
    if (e != cudaSuccess) return e;
    const int T = span_tile_tokens(a.G);
    const int64_t heads = (int64_t)a.B * a.Hkv;
    // key tiles that a query tile sees at most
    const int64_t seen = ((int64_t)a.span + T < a.n_kv ? ((int64_t)a.span + T) / kTile + 2 + (a.sinks + kTile - 1) / kTile
                                                       : (a.n_kv + kTile - 1) / kTile);
    const int64_t wide = (a.n_q + 2 * T - 1) / (2 * T) * heads;
    int cl = 0;   // 0: wide
    if (wide < num_sms) {
        const int64_t tiles = (a.n_q + T - 1) / T * heads;
        cl = 1;
        while (cl < 16 && tiles * cl * 2 <= num_sms && seen >= 2 * cl) cl *= 2;
    }
    const int64_t q_tiles = cl ? (a.n_q + T - 1) / T : (a.n_q + 2 * T - 1) / (2 * T);
    const int64_t grid = q_tiles * heads * (cl ? cl : 1);
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kAttThreads);
    cfg.dynamicSmemBytes = kAttSmem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cl;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    if (cl > 1) {
        cfg.attrs = &at;
        cfg.numAttrs = 1;
    }
    return cl ? cudaLaunchKernelEx(&cfg, span_attention_kernel<true>, a, C, layer, qmap, kmap, vmap, out, lse,
                                   (int)q_tiles, cl)
              : cudaLaunchKernelEx(&cfg, span_attention_kernel<false>, a, C, layer, qmap, kmap, vmap, out, lse,
                                   (int)q_tiles, 1);
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
