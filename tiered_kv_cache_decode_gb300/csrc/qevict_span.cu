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
// whether some pair of keys [k0, k0 + 128) and positions [p_lo, p_hi] is masked
__device__ __forceinline__ bool masked_tile(const SpanArgs &a, int k0, int p_lo, int p_hi) {
    return !(k0 + kTile - 1 <= p_lo && (k0 > p_hi - a.span || k0 + kTile <= a.sinks));
}

// bits 0 .. n - 1 of a word
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

__device__ __forceinline__ int clamped(const int32_t *len, int b, int n) {
    return len ? min(max(len[b], 0), n) : n;
}

// ---- attention ----------------------------------------------------------------
//
// Rows are (token, query head of one KV head's group), token-major, 128 / G
// tokens to a tile of 128 rows, so every head of the group shares the tile's keys.
// Twelve warps: two softmax warpgroups (a thread owns a row), one warp that
// issues the products, one thread that issues the copies. Tensor memory holds a logit
// tile S and an output tile O (fp32, 128 x 128) per softmax group; the
// probabilities overwrite their logits as bf16 and are the A operand of P V
// from there, so neither S nor P leaves the SM. While one group is in its
// softmax, the tensor cores work for the other.
//
// Wide: the groups take two neighbouring query tiles over the same keys, and the
// CTA goes on with units of CTAs that have not started. Bound by the products and by
// the chain between them: a group's loads, maximum, exponentials (at 32 a cycle and
// SM half as long as the tile's products) and stores take a little longer than the
// other group's two products; 32 query heads on 8: a prompt of 8K 326 us
// (1,690 TFLOP/s; the tensor pipe active 74 % of the cycles), of 32K 5.05 to 5.35 ms
// (1,645 to 1,740; the clock falls under the power limit), four of 8K with
// a span of 4K 1.04 ms (1,585: some of its tiles are half masked).
// Split: both take one query tile, every other key tile each, and the key tiles
// are further divided over the CTAs of a cluster; the partial (max, sum, O)
// meet in shared memory. No scratch in device memory either way. Single tokens
// are bound by the keys and values: 8 sequences of 26K to 32K 146 us (6.6 TB/s);
// 16 with a span of 4K 27 us (5.0 TB/s: the first copies and the meeting, about
// 5 us, do not overlap the stream).
//
// Probabilities are rounded to bf16 for P V: a product takes both operands in one
// type, and a second one for what the rounding leaves off would double P V, half of the
// tensor work here. Each is off by half a step, 2^-8 of itself, at most; their sum is taken
// before it, in fp32. Exponentials are the hardware's, off by 2^-22.
constexpr int kSoftmax = 256;                 // threads of the two softmax groups
constexpr int kAttThreads = kSoftmax + 128;   // and a group of four warps for copies and products
constexpr int kAttSlots = 7;                  // 32 KB slots of shared memory: query tiles, then the key/value ring
constexpr int kAttSmem = kAttSlots * kTileBytes + 1024;
constexpr float kRescale = 8.f;               // log2 growth of a row's maximum that moves its reference

// A value row in shared memory, its halves of 64 channels kHalf bytes apart: whether no
// element is infinite or NaN (row r starts at its own 16 bytes, so that a warp's
// rows fall into all banks), and those elements, or all, set to 0.
__device__ __forceinline__ bool all_finite(const uint8_t *v, int r) {
    uint32_t top = 0;
#pragma unroll
    for (int y = 0; y < 16; ++y) {
        const uint4 u = *reinterpret_cast<const uint4 *>(v + (y >> 3) * kHalf + 16 * ((y + r) & 7));
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                     __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
    }
    return (top & 0xffffu) < 0x7f80u && (top >> 16) < 0x7f80u;
}
__device__ __forceinline__ void clear_not_finite(uint8_t *v) {
#pragma unroll 1
    for (int y = 0; y < 64; ++y) {
        uint32_t *w = reinterpret_cast<uint32_t *>(v + (y >> 5) * kHalf) + (y & 31);
        uint32_t u = *w;
        if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
        if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
        *w = u;
    }
}
__device__ __forceinline__ void clear_row(uint8_t *v, int r) {
#pragma unroll
    for (int y = 0; y < 16; ++y)
        *reinterpret_cast<int4 *>(v + (y >> 3) * kHalf + 16 * ((y + r) & 7)) = make_int4(0, 0, 0, 0);
}

// One or two neighbouring query tiles of one (sequence, KV head), and the key tiles
// [first, first + n) of theirs that this CTA takes.
struct __align__(16) AttUnit {
    int b, kvh, i0, n_tok, p_lo, p_hi, first, n;
    Tiles tl;
    int pad;
};
template <bool SPLIT>
__device__ __forceinline__ AttUnit att_unit(const SpanArgs &a, int u, int q_tiles, int T, int rank, int cl) {
    AttUnit U;
    const int heads = a.B * a.Hkv;
    U.b = u % heads / a.Hkv;
    U.kvh = u % a.Hkv;
    U.i0 = (q_tiles - 1 - u / heads) * (SPLIT ? T : 2 * T);   // the longest rows of keys first
    const int q_len = clamped(a.q_len, U.b, a.n_q), kv_len = clamped(a.kv_len, U.b, a.n_kv);
    U.n_tok = min(SPLIT ? T : 2 * T, q_len - U.i0);           // none: past the sequence's queries
    U.p_lo = kv_len - q_len + U.i0;
    U.p_hi = U.p_lo + U.n_tok - 1;
    U.tl = tiles_of(a, U.p_lo, U.p_hi);
    const int all = U.n_tok > 0 ? U.tl.count() : 0;
    U.first = SPLIT ? (int)((int64_t)all * rank / cl) : 0;
    U.n = (SPLIT ? (int)((int64_t)all * (rank + 1) / cl) : all) - U.first;
    return U;
}

// Adds to four outputs of position `pos`, from channel `ch`, the infinite and NaN values of the
// keys that it sees in the unit's masked tiles.
__device__ __forceinline__ void add_cleared(const SpanArgs &a, const AttUnit &U, const __nv_bfloat16 *values, int pos,
                                            int ch, __nv_bfloat16 *o) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    bool any = false;
#pragma unroll 1
    for (int it = 0; it < U.tl.count(); ++it) {
        const int k0 = U.tl.key(it);
        if (!masked_tile(a, k0, U.p_lo, U.p_hi)) continue;
#pragma unroll 1
        for (int j = k0; j <= min(k0 + kTile - 1, pos); ++j) {
            if (j <= pos - a.span && j >= a.sinks) continue;
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(
                values + (((int64_t)U.b * a.n_kv + j) * a.Hkv + U.kvh) * kHeadDim + ch));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = __uint_as_float(e & 1 ? (e < 2 ? u.x : u.y) & 0xffff0000u : (e < 2 ? u.x : u.y) << 16);
                if (!isfinite(y)) x[e] += y, any = true;
            }
        }
    }
    if (any)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __float2bfloat16_rn(__bfloat162float(o[e]) + x[e]);
}

// Four lanes, each with 64 bytes of a row of its own as four chunks, trade them by two
// exchanges: afterwards lane i of the four has chunk i of each of the four rows, and a store
// of the warp covers 8 rows x 64 bytes instead of 32 rows x 16 bytes, a quarter of the lines
// (stores of a lane's own row and these: three prompts of 2K 88 and 79 us, 8 of 8K with
// a span of 128 403 and 341 us; both halves of the row unrolled, so that the second loads
// under the first: 83 and 350, the code is run once a unit and comes from far).
__device__ __forceinline__ void trade_chunks(uint32_t (&w)[16]) {
    const bool b0 = threadIdx.x & 1, b1 = threadIdx.x & 2;
#pragma unroll
    for (int m = 0; m < 16; m += 8)
#pragma unroll
        for (int e = m; e < m + 4; ++e) {
            const uint32_t got = __shfl_xor_sync(~0u, b0 ? w[e] : w[e + 4], 1);
            w[e] = b0 ? got : w[e];
            w[e + 4] = b0 ? w[e + 4] : got;
        }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t got = __shfl_xor_sync(~0u, b1 ? w[e] : w[e + 8], 2);
        w[e] = b1 ? got : w[e];
        w[e + 8] = b1 ? w[e + 8] : got;
    }
}

template <bool SPLIT>
__global__ void __launch_bounds__(kAttThreads, 1)
    span_attention_kernel(const SpanArgs a, const CacheDev C, int layer, const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const __nv_bfloat16 *values, __nv_bfloat16 *out, float *lse, int q_tiles, int cl) {
    constexpr int QT = SPLIT ? 1 : 2;              // query tiles of the CTA
    constexpr int NS = kAttSlots - QT;             // ring slots
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * NS + 16];
    __shared__ uint4 ticket;                       // wide: the answer to the copy thread's last request
    __shared__ AttUnit given[2];                   // wide: units that the copy thread has worked out
    __shared__ uint32_t slot;
    __shared__ int stop;
    __shared__ int poison[8];                      // by unit: a value was infinite or NaN in a masked tile

    const int T = span_tile_tokens(a.G), rows = T * a.G;
    const int rank = SPLIT ? blockIdx.x % cl : 0;
    if (threadIdx.x < 3) tc_prefetch_map(threadIdx.x == 0 ? &qmap : threadIdx.x == 1 ? &kmap : &vmap);
    AttUnit U;
    if (SPLIT) {   // one unit
        U = att_unit<SPLIT>(a, blockIdx.x / cl, q_tiles, T, rank, cl);
        if (U.n_tok <= 0) return;   // the whole cluster alike
    }

    const uint32_t sm = (smem_u32(raw) + 1023) & ~1023u;
    uint8_t *gen = raw + (sm - smem_u32(raw));
    const uint32_t ring = sm + QT * kTileBytes;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8 * s; };
    auto empty = [&](int s) { return bar0 + 8 * (NS + s); };
    auto s_full = [&](int t) { return bar0 + 8 * (2 * NS + t); };
    auto p_full = [&](int t, int h) { return bar0 + 8 * (2 * NS + 5 + 2 * t + h); };   // h: half of the keys
    auto o_full = [&](int t) { return bar0 + 8 * (2 * NS + 2 + t); };
    const uint32_t q_full = bar0 + 8 * (2 * NS + 4), q_empty = bar0 + 8 * (2 * NS + 9);
    auto u_full = [&](int x) { return bar0 + 8 * (2 * NS + 10 + x); };
    auto u_empty = [&](int x) { return bar0 + 8 * (2 * NS + 12 + x); };
    const uint32_t asked = bar0 + 8 * (2 * NS + 14), drained = asked + 8;
    // The ring holds key and value tiles in the order in which the products use them: K0 V0 K1 V1 ..,
    // split K0 K1 V0 K2 V1 .. K(n-1) V(n-2) V(n-1). The copy thread's loads, of a unit's query tiles
    // and of its item x as the i-th of the ring:
    auto load_q = [&] {
        tc_expect_tx(q_full, QT * rows * 256);
        for (int t = 0; t < QT; ++t)
            for (int h = 0; h < 2; ++h)
                tc_tma_4d(sm + t * kTileBytes + h * kHalf, &qmap, 64 * h, U.kvh * a.G, U.i0 + t * T, U.b, q_full);
    };
    auto load_item = [&](int x, int i) {
        const int s = i % NS;
        const bool last = x == 2 * U.n - 1;
        const bool isk = SPLIT ? x == 0 || (x & 1 && !last) : !(x & 1);
        const int j = SPLIT ? (isk ? (x + 1) / 2 : last ? U.n - 1 : x / 2 - 1) : x / 2;
        tc_expect_tx(full(s), kTileBytes);
        for (int h = 0; h < 2; ++h)
            tc_tma_4d(ring + s * kTileBytes + h * kHalf, isk ? &kmap : &vmap, 64 * h, U.kvh, U.tl.key(U.first + j), U.b,
                      full(s));
    };
    if (tid == 9 * 32) {
        // p_full: the group's four warps; u_empty: the product warp and both groups' warps
        for (int i = 0; i < 2 * NS + 16; ++i) {
            const int x = i - 2 * NS;
            tc_mbar_init(bar0 + 8 * i, x == 12 || x == 13 ? 9 : x >= 5 && x < 9 ? 4 : 1);
        }
        stop = 0;
        for (int i = 0; i < 8; ++i) poison[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (SPLIT && U.n > 0) {   // a short unit's latency counts: its first copies do not wait for the set-up
            load_q();
            for (int x = 0; x < min(2 * U.n, NS); ++x) load_item(x, x);
        }
    }
    __syncwarp();
    if (warp == 0) tc_alloc<512>(smem_u32(&slot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = slot;                      // S of group t at column 128 t, O at 256 + 128 t

    // The next unit of a warp (c: how many it has had), false when there is none. Wide: the copy
    // thread, which is tiles ahead, has worked it out, so the other warps do not stall on it.
    auto next = [&](int c, bool &ok) {
        if (SPLIT) return c == 0;
        ok = __all_sync(~0u, tc_wait(u_full(c & 1), (c >> 1) & 1, &stop));
        if (!ok) return false;
        U = given[c & 1];
        __syncwarp();
        if ((tid & 31) == 0) tc_arrive(u_empty(c & 1));
        return U.n_tok > 0;
    };

    // 12 warps start with 168 registers a thread; the softmax groups take 224 and leave 56
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (tid == 9 * 32) {
            int i = 0, q = 0, c = 0;
            bool ok = true;
            auto give = [&](const AttUnit &X) {
                if (c >= 2 && !(ok = tc_wait(u_empty(c & 1), ((c >> 1) - 1) & 1, &stop))) return;
                given[c & 1] = X;
                tc_arrive(u_full(c & 1));
                ++c;
            };
            // A wide CTA goes on with the units of CTAs that have not started yet, longest first. It
            // asks once the copies of the unit before are issued: the SM that is done first gets the next.
            uint32_t at = blockIdx.x;
            int asks = 0;
            for (int k = 0; ok; ++k) {
                if (SPLIT) {
                    if (k) break;
                } else {
                    if (k) {
                        tc_ask(smem_u32(&ticket), asked);
                        ok = tc_wait(asked, asks++ & 1, &stop);
                        if (!ok) break;
                        if (!tc_answer(smem_u32(&ticket), at)) {
                            U.n_tok = 0;   // no more
                            give(U);
                            break;
                        }
                    }
                    U = att_unit<SPLIT>(a, at, q_tiles, T, rank, cl);
                    if (U.n_tok <= 0) continue;
                    give(U);
                    if (!ok) break;
                }
                if (U.n <= 0) continue;
                if (SPLIT) {
                    i = min(2 * U.n, NS);   // these are on their way
                } else {
                    if (q > 0 && !(ok = tc_wait(q_empty, (q - 1) & 1, &stop))) break;
                    load_q();
                }
                ++q;
                for (int x = SPLIT ? i : 0; x < 2 * U.n; ++x, ++i) {
                    if (i >= NS && !(ok = tc_wait(empty(i % NS), (i / NS - 1) & 1, &stop))) break;
                    load_item(x, i);
                }
            }
            // The copies in flight land before the CTA ends, whichever role gave up, now or later.
            const long long t0 = clock64();
            while (q > 0 && !tc_try_wait(q_full, (q - 1) & 1) && clock64() - t0 < kDefaultWaitCycles) {}
            for (int o = max(0, i - NS); o < i; ++o)
                while (!tc_try_wait(full(o % NS), (o / NS) & 1) && clock64() - t0 < kDefaultWaitCycles) {}
            while (asks > 0 && !tc_try_wait(asked, (asks - 1) & 1) && clock64() - t0 < kDefaultWaitCycles) {}
        }
        if (warp == 8) {   // the whole warp keeps step, one lane issues
            const bool lead = tc_elect();
            const uint32_t tmu = __shfl_sync(~0u, tm, 0);
            bool ok = true;
            auto wait = [&](uint32_t bar, int par) {
                ok = __all_sync(~0u, tc_wait(bar, par, &stop));
                return ok;
            };
            auto wait2 = [&](uint32_t bar, int par, uint32_t bar2, int par2) {
                ok = __all_sync(~0u, tc_wait2(bar, par, bar2, par2, &stop));
                return ok;
            };
            // The ring slots of the next key tile for S and of the next value tile; a slot's parity flips as it wraps.
            int ks = 0, kp = 0, vs = 1, vp = 0, q = 0, tiles = 0;
            auto ahead_of = [&](int &slot_, int &par, int by) {
                slot_ += by;
                if (slot_ >= NS) slot_ -= NS, par ^= 1;
            };
            // S_t = Q K^T; done: the key tile's slot is free after it, last: so are the query tiles
            auto logits = [&](int t, bool done, bool last) {
                if (lead) {
                    tc_mma_tile<kTile>(tmu + 128 * t, sm + (SPLIT ? 0 : t * kTileBytes), ring + ks * kTileBytes);
                    tc_commit(s_full(t));
                    if (done) tc_commit(empty(ks));
                    if (done && last) tc_commit(q_empty);
                }
                __syncwarp();
            };
            for (int c = 0; next(c, ok); ++c) {
                const int n = __shfl_sync(~0u, U.n, 0);
                if (n <= 0) continue;
                if (!wait2(q_full, q & 1, full(ks), kp)) break;
                ++q;
                if (SPLIT && n > 1) vs = 2;
                logits(0, SPLIT, n == 1);
                if (!SPLIT) logits(1, true, n == 1);
                ahead_of(ks, kp, SPLIT ? 1 : 2);
                if (SPLIT && n > 1) {
                    if (!wait(full(ks), kp)) break;
                    logits(1, true, n == 2);
                    ahead_of(ks, kp, 2);
                }
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t v = tc_desc_mn(ring + vs * kTileBytes, kHalf);
                    const bool more = j + (SPLIT ? 2 : 1) < n;
                    const int par = (SPLIT ? j >> 1 : tiles + j) & 1;
#pragma unroll
                    for (int x = 0; x < QT; ++x) {
                        const int t = SPLIT ? j & 1 : x;
                        // the values' and the next keys' tiles are waited for beside the probabilities
                        if (!(x == 0 ? wait2(full(vs), vp, p_full(t, 0), par) : wait(p_full(t, 0), par))) break;
                        tc_fence_after();
                        if (lead) {
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                tc_mma_ts(tmu + 256 + 128 * t, tmu + 128 * t + 8 * s, v + s * 128, tc_idesc(true),
                                          s > 0 || j >= (SPLIT ? 2 : 1));
                        }
                        __syncwarp();
                        if (!(x == 0 && more ? wait2(full(ks), kp, p_full(t, 1), par) : wait(p_full(t, 1), par))) break;
                        tc_fence_after();
                        if (lead) {
#pragma unroll
                            for (int s = 4; s < 8; ++s)
                                tc_mma_ts(tmu + 256 + 128 * t, tmu + 128 * t + 8 * s, v + s * 128, tc_idesc(true), 1);
                            if (x == QT - 1) tc_commit(empty(vs));
                            if (!more) tc_commit(o_full(t));
                        }
                        __syncwarp();
                        if (more) logits(t, x == QT - 1, j + (SPLIT ? 3 : 2) == n);
                    }
                    if (more) ahead_of(ks, kp, 2);
                    // split: the last value tile follows its predecessor directly
                    ahead_of(vs, vp, SPLIT && j == n - 2 ? 1 : 2);
                }
                if (!ok) break;
                tiles += n;
            }
            // The products in flight end before the tensor memory is freed, whichever role gave up.
            if (lead) tc_commit(drained);
            __syncwarp();
            const long long t0 = clock64();
            while (!tc_try_wait(drained, 0) && clock64() - t0 < kDefaultWaitCycles) {}
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
        const uint64_t cc = pair2(c, c);
        const int tok = (SPLIT ? 0 : t * T) + r / a.G, g = r % a.G;
        bool ok = true;
        int tiles = 0, item0 = 0, outs = 0;   // logit tiles, ring items and outputs before this unit
        for (int c_ = 0; ok && next(c_, ok); ++c_) {
            // the groups are less than two units apart, so a slot four ahead is out of use
            if (tid == 0) poison[(c_ + 4) & 7] = 0;
            const int b = U.b, kvh = U.kvh, i0 = U.i0, p_lo = U.p_lo, p_hi = U.p_hi, n = U.n;
            auto v_item = [&](int j) { return item0 + (SPLIT ? min(2 * j + 2, 2 * n - 1) : 2 * j + 1); };
            const int pos = p_lo + tok;
            const bool valid = r < rows && tok < U.n_tok;
            float m = -INFINITY, l = 0.f;
            int done = 0;
            for (int j = SPLIT ? t : 0; j < n; j += SPLIT ? 2 : 1, ++done) {
                ok = __all_sync(~0u, tc_wait(s_full(t), (tiles + done) & 1, &stop));   // a warp stops as one
                if (!ok) break;
                tc_fence_after();
                const int k0 = U.tl.key(U.first + j);
                // of the unit, for the mask and the clearing alike (a test of the group's own positions
                // beside it: 8K prompt 336 instead of 327 us, four of 8K with a span of 4K 1,070 and 1,047)
                const bool masked = masked_tile(a, k0, p_lo, p_hi);
                const int hi = pos - k0, lo = hi - a.span, sk = a.sinks - k0;
                float x[4][32], mx[4];
                tc_ld32(tS, x[0]);
                tc_ld32(tS + 32, x[1]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {   // the maximum of the first half is taken while the second is on its way
                    if ((q & 1) == 0) {
                        tc_wait_ld();
                        tc_tie(x[q]);
                        tc_tie(x[q + 1]);
                        if (q == 0) {
                            tc_ld32(tS + 64, x[2]);
                            tc_ld32(tS + 96, x[3]);
                        }
                    }
                    if (masked) {   // the quarter's visible keys as bits, so that no element needs a branch
                        const uint32_t w = below(hi + 1 - 32 * q) & (~below(lo + 1 - 32 * q) | below(sk - 32 * q));
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[q][e] = (w >> e & 1) ? x[q][e] : -INFINITY;
                    }
                    float y[2] = {fmaxf(x[q][0], x[q][1]), fmaxf(x[q][2], x[q][3])};
#pragma unroll
                    for (int e = 4; e < 32; e += 4) {
                        y[0] = max3(y[0], x[q][e], x[q][e + 1]);
                        y[1] = max3(y[1], x[q][e + 2], x[q][e + 3]);
                    }
                    mx[q] = fmaxf(y[0], y[1]);
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                // The reference follows the maximum only when it has grown by more than
                // kRescale in the exponent: probabilities stay below 2^kRescale, and O is
                // rarely touched between its products. A warp moves together, but each row's
                // reference by its own logits alone (a factor of 1 changes no bit): rows share
                // a warp with later queries, with rows that no query fills and whose part of the
                // query tile holds anything, and with rows past the sequence's end.
                const bool move = valid && (top - m) * c > kRescale;
                if (__any_sync(~0u, move)) {
                    const float f = !move ? 1.f : m == -INFINITY ? 0.f : tc_ex2((m - top) * c);
                    if (move) m = top;
                    l *= f;
                    if (done > 0) {   // the product before it has ended: its logits came after it
#pragma unroll 1
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
                // A probability of 0 does not keep an infinity or a NaN out of its product, so in a tile
                // that some row of the unit does not see in full they are set to 0 (as are keys that no
                // row of it sees, which may be anything); rows that do see them get them back at the
                // end. Wide: the first group does it, for both: no product reads the tile before that
                // group's probabilities have arrived, and none of the second group's is issued before
                // them, so nothing is written under a product.
                if (masked && (SPLIT || t == 0)) {
                    const int i = v_item(j), s = i % NS;
                    ok = __all_sync(~0u, tc_wait(full(s), (i / NS) & 1, &stop));
                    if (!ok) break;
                    const int key = k0 + r;
                    const bool dead = key > p_hi || (key <= p_lo - a.span && key >= a.sinks);
                    uint8_t *v = gen + (QT + s) * kTileBytes + r * 128;
                    const bool bad = !dead && !all_finite(v, r);
                    if (dead) clear_row(v, r);
                    if (bad) {
                        poison[c_ & 7] = 1;
                        clear_not_finite(v);
                    }
                    if (dead || bad) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                const float mc = m == -INFINITY ? 0.f : -m * c;
                const uint64_t mm = pair2(mc, mc);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {   // the product starts on the first half of the keys
#pragma unroll
                    for (int q = 2 * h; q < 2 * h + 2; ++q) {
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
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if ((tid & 31) == 0) tc_arrive(p_full(t, h));
                }
                float s0, s1;
                split2(add2(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
            }
            if (ok && done > 0) ok = __all_sync(~0u, tc_wait(o_full(t), outs++ & 1, &stop));
            tc_fence_after();
            tiles += n;
            item0 += 2 * n;
            if (!SPLIT) {
                const float inv = 1.f / l;
                const bool none = l == 0.f;   // no key seen
                const int64_t head = kvh * a.G + g;
                __nv_bfloat16 *base = out + (((int64_t)b * a.n_q + i0) * a.Hq + kvh * a.G) * kHeadDim;
                const int row = valid ? tok * a.Hq + g : -1;   // from base; -1: not written
                int at[4];                                     // of the lane's four
#pragma unroll
                for (int e = 0; e < 4; ++e) at[e] = __shfl_sync(~0u, row, (tid & 28) + e);
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    float o[32];
                    tc_ld32(tO + 32 * q, o);
                    tc_wait_ld();
                    tc_tie(o);
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const __nv_bfloat162 pk =
                            __floats2bfloat162_rn(none ? 0.f : o[2 * e] * inv, none ? 0.f : o[2 * e + 1] * inv);
                        p[e] = *reinterpret_cast<const uint32_t *>(&pk);
                    }
                    trade_chunks(p);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (at[e] >= 0 && ok)
                            *reinterpret_cast<uint4 *>(base + (int64_t)at[e] * kHeadDim + 32 * q + 8 * (tid & 3)) =
                                make_uint4(p[4 * e], p[4 * e + 1], p[4 * e + 2], p[4 * e + 3]);
                    __syncwarp();
                }
                if (poison[c_ & 7] && valid && ok) {
#pragma unroll 1
                    for (int ch = 0; ch < kHeadDim; ch += 4)
                        add_cleared(a, U, values, pos, ch, base + (int64_t)row * kHeadDim + ch);
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
                            part[(8 * q + e) ^ (r & 31)] =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                    __syncwarp();
                }
                __syncwarp();
                if (cl > 1) cl_sync();
                else __syncthreads();
                {
                    const uint32_t st = ring + 4 * kTileBytes;
                    int bad = 0;
                    for (int x = 0; x < cl; ++x) bad |= cl_ldi(cl_addr(smem_u32(&poison[0]), x));
                    for (int i = rank * kSoftmax + tid; i < U.n_tok * a.G * 32; i += cl * kSoftmax) {
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
                            const uint32_t at = ring + (x & 1) * 2 * kTileBytes + r * 512 + 16 * (ch ^ (r & 31));
                            const float4 y = cl_ld4(cl_addr(at, x >> 1));
                            l = fmaf(s.y, f, l);
                            o.x = fmaf(y.x, f, o.x);
                            o.y = fmaf(y.y, f, o.y);
                            o.z = fmaf(y.z, f, o.z);
                            o.w = fmaf(y.w, f, o.w);
                        }
                        const float inv = l == 0.f ? 0.f : 1.f / l;
                        const int64_t head = kvh * a.G + r % a.G;
                        __nv_bfloat162 p[2] = {__floats2bfloat162_rn(o.x * inv, o.y * inv),
                                               __floats2bfloat162_rn(o.z * inv, o.w * inv)};
                        __nv_bfloat16 *dst =
                            out + (((int64_t)b * a.n_q + i0 + r / a.G) * a.Hq + head) * kHeadDim + 4 * ch;
                        *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(p);
                        if (bad) add_cleared(a, U, values, p_lo + r / a.G, 4 * ch, dst);
                        if (ch == 0 && lse)
                            lse[((int64_t)b * a.Hq + head) * a.n_q + i0 + r / a.G] =
                                l == 0.f ? -INFINITY : (top == -INFINITY ? 0.f : top) * (1.f / kLog2e) + logf(l);
                    }
                }
                __syncwarp();
                if (cl > 1) cl_sync();
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && stop) set_status(C, QEVICT_ERR_TIMEOUT, layer, (int)blockIdx.x, 0);
    if (warp == 0) tc_free<512>(tm);
}

// ---- window scores --------------------------------------------------------------
//
// A thread owns a row (a query of one head) of a logit tile and so has its
// log-sum-exp in a register; it sums the row's masses over 16 keys at a time (a
// window is a multiple of 16) into eight registers that it keeps over all query
// tiles, and the rows meet once an item, by shuffles. Shared memory then feeds the
// products alone. (Keys as the rows, with a log-sum-exp for every column out of
// shared memory, came out equal at 8K and slower with a span of 1K over 4 x 8K, 310
// and 300 us.)
// An item is a run of 256 keys (rounded down to whole windows) of one sequence
// (of one KV head with per-head units); its steps are the (KV head, query tile)
// pairs that see some of them. Where the items are few, each is split into parts
// of as many steps, whose sums a second kernel adds in order. CTAs go on with the
// work of CTAs that have not started, the longest first, and the copies of the
// next item run under this one.
// Four groups of four warps take the masses, each of one key tile in every other
// step, so that their waits and loads fall at different times; one warp issues the
// products, both key tiles' in one of 256 columns, one the copies. (Two groups, a
// group then reading every step: 241 us at 8K and 130 us for 64 queries of 8 x 32K.
// Groups of half a tile's keys, which give their half back before the exponentials:
// 238 and 127 us. A product of its own for each tile: 203 and 117 us.)
// 32 query heads on 8: every query of 8K 199 us (1,380 TFLOP/s), 64 queries of
// 8 x 32K 116 us (1,180 TFLOP/s and 4.65 TB/s). Bound by the way round a logit
// buffer: product, load, half of the exponentials, release (about 1,600 cycles a step,
// the products of which take 1,024, as its exponentials do at 32 a cycle and SM).
constexpr int kScMass = 512;                  // threads of the four groups
constexpr int kScThreads = kScMass + 64;
constexpr int kScK = 2;                       // sets of two key tiles
constexpr int kScQ = 7 - 2 * kScK;            // query tile slots
struct ScoreItem {
    int b, h0, nh, k0;      // sequence, KV heads, first key
    int qa, nq;             // query tiles [qa, qa + nq)
    int q_len, kv_len;
};
// items of the first keys, which the most queries see, come first
__device__ __forceinline__ ScoreItem score_item(const SpanArgs &a, int item, int keys, int T, bool per_head) {
    ScoreItem it;
    const int units = per_head ? a.B * a.Hkv : a.B;
    const int u = item % units;
    it.b = per_head ? u / a.Hkv : u;
    it.h0 = per_head ? u % a.Hkv : 0;
    it.nh = per_head ? 1 : a.Hkv;
    it.k0 = item / units * keys;
    it.q_len = clamped(a.q_len, it.b, a.n_q);
    it.kv_len = clamped(a.kv_len, it.b, a.n_kv);
    const int shift = it.kv_len - it.q_len, k_hi = min(it.k0 + keys, it.kv_len) - 1;
    int lo = max(0, it.k0 - shift), hi = it.q_len;
    if (it.k0 >= a.sinks) hi = min(hi, k_hi + a.span - shift);
    it.qa = lo / T;
    it.nq = k_hi < it.k0 || hi <= lo ? 0 : (hi - 1) / T + 1 - it.qa;
    return it;
}
// The steps of one part of an item, as KV head h and query tile q.
struct ScoreSteps {
    int64_t left;
    int h, q, qa, qz;
    // true: the next step is another KV head's
    __device__ __forceinline__ bool next() {
        --left;
        if (++q < qz) return false;
        q = qa;
        ++h;
        return true;
    }
};
struct __align__(16) ScoreWork {
    ScoreItem it;
    ScoreSteps s;
    int part;
};
__device__ __forceinline__ ScoreSteps score_steps(const ScoreItem &it, int part, int parts) {
    ScoreSteps s;
    const int64_t steps = (int64_t)it.nh * it.nq, at = steps * part / parts;
    s.left = steps * (part + 1) / parts - at;
    s.qa = it.qa;
    s.qz = it.qa + it.nq;
    s.h = it.h0 + (it.nq ? (int)(at / it.nq) : 0);
    s.q = it.qa + (it.nq ? (int)(at % it.nq) : 0);
    return s;
}

// what lies behind the tiles in shared memory
struct ScoreTail {
    float segs[2][2][4][8];     // masses of 16 keys by key tile, parity of the item's steps, and warp
    ScoreWork given[2];         // items that the copy thread has worked out
    uint4 ticket;               // the answer to the copy thread's last request
    uint64_t bars[4 + 2 * kScQ + 10];
    uint32_t slot;
    int stop, go[2];
};
constexpr int kScSmem = (2 * kScK + kScQ) * kTileBytes + (int)sizeof(ScoreTail);
static_assert(kScSmem <= 227 * 1024, "shared memory of one CTA");

__global__ void __launch_bounds__(kScThreads, 1)
    span_scores_kernel(const SpanArgs a, const CacheDev C, int layer, const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap kmap, const float *lse, float *scores, float *part, int w,
                       int n_win, int per_head, int parts) {
    extern __shared__ __align__(1024) uint8_t gen[];
    ScoreTail &tail = *reinterpret_cast<ScoreTail *>(gen + (2 * kScK + kScQ) * kTileBytes);
    asm volatile("griddepcontrol.launch_dependents;");   // the sums' launch runs under this; it waits for the end
    const int T = span_tile_tokens(a.G), rows = T * a.G;
    const int tk = kTile / w * w;

    const uint32_t sm = smem_u32(gen), sq = sm + 2 * kScK * kTileBytes;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0);
    const uint32_t bar0 = smem_u32(tail.bars);
    auto k_full = [&](int s) { return bar0 + 8 * s; };
    auto k_empty = [&](int s) { return bar0 + 16 + 8 * s; };
    auto q_full = [&](int s) { return bar0 + 32 + 8 * s; };
    auto q_empty = [&](int s) { return bar0 + 32 + 8 * (kScQ + s); };
    auto s_full = [&](int x) { return bar0 + 32 + 8 * (2 * kScQ + x); };
    auto s_empty = [&](int x) { return bar0 + 32 + 8 * (2 * kScQ + 2 + x); };
    auto i_empty = [&](int x) { return bar0 + 32 + 8 * (2 * kScQ + 4 + x); };
    auto i_full = [&](int x) { return bar0 + 32 + 8 * (2 * kScQ + 6 + x); };
    const uint32_t drained = bar0 + 32 + 8 * (2 * kScQ + 8), asked = drained + 8;
    if (tid == 0) {
        // s_empty: each of the warps that read; i_empty: every warp but the copies'
        for (int i = 0; i < 4 + 2 * kScQ + 10; ++i) {
            const uint32_t bar = bar0 + 8 * i;
            tc_mbar_init(bar, bar >= i_full(0) ? 1 : bar >= i_empty(0) ? 17 : bar >= s_empty(0) ? 8 : 1);
        }
        tail.stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tc_alloc<512>(smem_u32(&tail.slot));
    // rows of a query tile that no query fills stay zero
    for (int i = tid; i < kScQ * 2 * (kTile - rows) * 8; i += kScThreads) {
        const int x = i & 7, r = (i >> 3) % (kTile - rows), h = (i >> 3) / (kTile - rows);
        uint8_t *at = gen + 2 * kScK * kTileBytes + h * kHalf + (rows + r) * 128 + 16 * x;
        *reinterpret_cast<int4 *>(at) = make_int4(0, 0, 0, 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tail.slot;   // logits of buffer x, key tile t at column 256 x + 128 t
    bool ok = true;
    // The next item of a warp (c: how many it has had), false when there is none: the copy
    // thread, which is steps ahead, has worked it out, so the other warps do not stall on it.
    ScoreWork W;
    auto next = [&](int c) {
        ok = ok && __all_sync(~0u, tc_wait(i_full(c & 1), (c >> 1) & 1, &tail.stop));
        if (!ok) return false;
        W = tail.given[c & 1];
        __syncwarp();
        if ((tid & 31) == 0) tc_arrive(i_empty(c & 1));
        return W.it.b >= 0;
    };

    if (warp == 17) {
        if (tid == 17 * 32) {
            int nk = 0, nq = 0, c = 0;   // runs of one KV head, query tiles and items so far
            int asks = 0;
            uint32_t at = blockIdx.x;
            for (; ok; ++c) {
                bool more = c == 0;
                if (c) {   // the CTA goes on with the work of CTAs that have not started yet
                    tc_ask(smem_u32(&tail.ticket), asked);
                    ok = tc_wait(asked, asks++ & 1, &tail.stop);
                    if (!ok) break;
                    more = tc_answer(smem_u32(&tail.ticket), at);
                }
                if (more) {
                    W.it = score_item(a, at / parts, 2 * tk, T, per_head);
                    W.part = at % parts;
                    W.s = score_steps(W.it, W.part, parts);
                } else {
                    W.it.b = -1;
                }
                if (c >= 2 && !(ok = tc_wait(i_empty(c & 1), ((c >> 1) - 1) & 1, &tail.stop))) break;
                tail.given[c & 1] = W;
                tc_arrive(i_full(c & 1));
                if (W.it.b < 0) break;
                const ScoreItem &it = W.it;
                ScoreSteps &s = W.s;
                for (bool head = true; s.left > 0; head = s.next()) {
                    if (head) {
                        const int set = nk % kScK;
                        if (nk >= kScK && !(ok = tc_wait(k_empty(set), (nk / kScK - 1) & 1, &tail.stop))) break;
                        tc_expect_tx(k_full(set), 2 * kTileBytes);
                        for (int t = 0; t < 2; ++t)
                            for (int h = 0; h < 2; ++h)
                                tc_tma_4d(sm + 2 * set * kTileBytes + (2 * h + t) * kHalf, &kmap, 64 * h, s.h, it.k0 + t * tk,
                                          it.b, k_full(set));
                        ++nk;
                    }
                    const int q = nq % kScQ;
                    if (nq >= kScQ && !(ok = tc_wait(q_empty(q), (nq / kScQ - 1) & 1, &tail.stop))) break;
                    tc_expect_tx(q_full(q), rows * 256);
                    for (int h = 0; h < 2; ++h)
                        tc_tma_4d(sq + q * kTileBytes + h * kHalf, &qmap, 64 * h, s.h * a.G, s.q * T, it.b, q_full(q));
                    ++nq;
                }
            }
            // The copies in flight land before the CTA ends, whichever role gave up, now or later.
            const long long t0 = clock64();
            for (int o = max(0, nk - kScK); o < nk; ++o)
                while (!tc_try_wait(k_full(o % kScK), (o / kScK) & 1) && clock64() - t0 < kDefaultWaitCycles) {}
            for (int o = max(0, nq - kScQ); o < nq; ++o)
                while (!tc_try_wait(q_full(o % kScQ), (o / kScQ) & 1) && clock64() - t0 < kDefaultWaitCycles) {}
            while (asks > 0 && !tc_try_wait(asked, (asks - 1) & 1) && clock64() - t0 < kDefaultWaitCycles) {}
        }
        __syncwarp();
    } else if (warp == 16) {
        // the whole warp keeps step, one lane issues
        const bool lead = tc_elect();
        const uint32_t tmu = __shfl_sync(~0u, tm, 0);
        int set = kScK - 1, kp = 1, qs = 0, qp = 0, buf = 0, sp = 1;   // slots and their parities
        for (int c = 0; next(c); ++c) {
            ScoreSteps &s = W.s;
            bool head = true;
            while (s.left > 0) {
                if (head && ++set == kScK) set = 0, kp ^= 1;
                const uint32_t q = sq + qs * kTileBytes, k = sm + 2 * set * kTileBytes;
                // s_empty passes at once the first time
                ok = __all_sync(~0u, tc_wait3(k_full(set), kp, q_full(qs), qp, s_empty(buf), sp, &tail.stop));
                if (!ok) break;
                tc_fence_after();
                head = s.next();
                if (lead) {
                    tc_mma_tile<2 * kTile>(tmu + 256 * buf, q, k);
                    tc_commit(s_full(buf));
                    tc_commit(q_empty(qs));
                    if (head || s.left == 0) tc_commit(k_empty(set));
                }
                __syncwarp();
                if (++qs == kScQ) qs = 0, qp ^= 1;
                buf ^= 1;
                sp ^= buf == 0;
            }
        }
        // The products in flight end before the tensor memory is freed, whichever role gave up.
        if (lead) tc_commit(drained);
        __syncwarp();
        const long long t0 = clock64();
        while (!tc_try_wait(drained, 0) && clock64() - t0 < kDefaultWaitCycles) {}
        __syncwarp();
    } else {
        const int t = warp >> 3, x = (warp >> 2) & 1, r = tid & 127;
        const uint32_t tS = tm + ((uint32_t)((warp & 3) * 32) << 16) + 256 * x + 128 * t;
        const int tok = r / a.G;
        const int64_t off = (int64_t)(r % a.G) * a.n_q + tok;   // the row's log-sum-exp in a query tile's
        const float c = kLog2e * rsqrtf((float)kHeadDim);
        const uint64_t cc = pair2(c, c);
        int nq = 0, turn = 0;   // steps so far, and the group's own
        for (int c_ = 0;; ++c_) {
            // the first warp of a key tile decides for the eight, so that their barriers match
            const bool first_warp = (warp & 7) == 0;
            if (first_warp) {
                const bool more = next(c_);
                if ((tid & 31) == 0) tail.go[t] = more;
            }
            asm volatile("bar.sync %0, 256;" ::"r"(t + 1) : "memory");
            if (!tail.go[t]) break;
            if (!first_warp) {
                W = tail.given[c_ & 1];
                __syncwarp();
                if ((tid & 31) == 0) tc_arrive(i_empty(c_ & 1));
            }
            const ScoreItem it = W.it;
            const int shift = it.kv_len - it.q_len, k0 = it.k0 + t * tk;
            float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            const float *l0 = lse + (int64_t)it.b * a.Hq * a.n_q + off;
            auto fetch = [&](const ScoreSteps &s) {   // rows that no query fills, or that see no key, take no part
                if (s.left <= 0 || r >= rows || s.q * T + tok >= it.q_len) return -INFINITY;
                return __ldg(l0 + (int64_t)s.h * a.G * a.n_q + s.q * T);
            };
            ScoreSteps s = W.s;
            // The CTA's steps alternate between the groups, so which of them has the item's even steps
            // depends on the items before it; their sums are added as even and odd, not by group.
            const int odd = (nq & 1) ^ x;
            if (odd && s.left > 0) s.next(), ++nq;   // the first step of the group's parity
            float ahead = fetch(s);
            while (s.left > 0) {
                const int i0 = s.q * T, p_lo = shift + i0;
                const float ls = ahead == -INFINITY ? ahead : -kLog2e * ahead;
                s.next();
                ++nq;
                if (s.left > 0) s.next(), ++nq;
                ahead = fetch(s);   // of the group's next step
                ok = ok && __all_sync(~0u, tc_wait(s_full(x), turn++ & 1, &tail.stop));
                if (!ok) continue;
                tc_fence_after();
                const uint64_t mm = pair2(ls, ls);   // (used first after a wait: the load is the group's last step old)
                float v[2][32];
                tc_ld32(tS, v[0]);
                tc_ld32(tS + 32, v[1]);
                const bool plain =
                    i0 + T <= it.q_len && k0 + tk - 1 <= p_lo && (k0 > p_lo + T - 1 - a.span || k0 + tk <= a.sinks);
                const int hi = i0 + tok < it.q_len ? p_lo + tok - k0 : -1, lo = p_lo + tok - k0 - a.span;
                const int sk = a.sinks - k0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if ((q & 1) == 0) {
                        if (q == 2) {
                            tc_ld32(tS + 64, v[0]);
                            tc_ld32(tS + 96, v[1]);
                        }
                        tc_wait_ld();
                        tc_tie(v[0]);
                        tc_tie(v[1]);
                        if (q == 2) {
                            tc_fence_before();
                            __syncwarp();
                            if ((tid & 31) == 0) tc_arrive(s_empty(x));
                        }
                    }
                    float(&y)[32] = v[q & 1];
                    if (!plain) {   // the quarter's visible keys as bits
                        const uint32_t m = below(hi + 1 - 32 * q) & (~below(lo + 1 - 32 * q) | below(sk - 32 * q));
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] = (m >> e & 1) ? y[e] : -INFINITY;
                    }
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint64_t sum[2] = {0, 0};
#pragma unroll
                        for (int e = 16 * g; e < 16 * g + 16; e += 2) {
                            float u, z;
                            split2(fma2(pair2(y[e], y[e + 1]), cc, mm), u, z);
                            sum[e >> 1 & 1] = add2(sum[e >> 1 & 1], pair2(tc_ex2(u), tc_ex2(z)));
                        }
                        float s0, s1;
                        split2(add2(sum[0], sum[1]), s0, s1);
                        acc[2 * q + g] += s0 + s1;
                    }
                }
            }
            // Rows of a query tile that no query fills are zeros and have the weight 0, but a zero times
            // an infinite key is NaN.
            if (r >= rows)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = 0.f;
            // Eight sums over the warp's 32 rows: three exchanges halve the sums that a lane keeps,
            // two add what is left; lane l has the sum of keys 16 (l / 4) .. + 15.
#pragma unroll
            for (int o = 16, n = 4; o >= 4; o >>= 1, n >>= 1)
#pragma unroll
                for (int e = 0; e < n; ++e) {
                    const bool up = tid & o;
                    const float give = up ? acc[e] : acc[e + n];
                    acc[e] = (up ? acc[e + n] : acc[e]) + __shfl_xor_sync(~0u, give, o);
                }
            acc[0] += __shfl_xor_sync(~0u, acc[0], 2);
            acc[0] += __shfl_xor_sync(~0u, acc[0], 1);
            if ((tid & 3) == 0) tail.segs[t][odd][warp & 3][(tid & 31) >> 2] = acc[0];
            asm volatile("bar.sync %0, 256;" ::"r"(t + 1) : "memory");
            const int win = k0 / w + r;
            float mass = 0.f;
            if (x == 0 && r < tk / w)
                for (int e = r * (w / 16); e < (r + 1) * (w / 16); ++e)
                    for (int y = 0; y < 8; ++y) mass += tail.segs[t][y >> 2][y & 3][e];
            if (x == 0 && r < tk / w && win < n_win) {
                const int units = per_head ? a.B * a.Hkv : a.B, u = per_head ? it.b * a.Hkv + it.h0 : it.b;
                if (parts == 1) scores[(int64_t)u * n_win + win] = mass / (per_head ? a.G : a.Hq);
                else part[((int64_t)W.part * units + u) * n_win + win] = mass;
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && tail.stop) set_status(C, QEVICT_ERR_TIMEOUT, layer, 0, 0);
    if (warp == 0) tc_free<512>(tm);
}

// The parts' window masses in order, one window a thread (256 KB at most). Its launch
// runs under the items, for whose end it waits (every query of 2K 40.0 us with a plain
// launch, 37.9 so).
__global__ void __launch_bounds__(128) span_scores_sum_kernel(const float *part, float *scores, int64_t n, int parts,
                                                              float heads) {
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (i >= n) return;
    float y = 0.f;
    for (int p = 0; p < parts; ++p) y += part[p * n + i];
    scores[i] = y / heads;
}

// How many clusters of each size the device holds at once (its SMs come in
// groups of unlike size, so 8 CTAs fill fewer SMs than 4 or 9 do).
constexpr int kMaxCluster = 16;
template <class K>
cudaError_t prepare_clusters(K kernel, int threads, int smem, int *active) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (int c = 2; c <= kMaxCluster && e == cudaSuccess; ++c) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(c * 256);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = c;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&active[c], kernel, &cfg);
    }
    return e;
}

// CTAs per query tile that finish `tiles` tiles of `seen` key tiles each first, and in how many us.
int best_cluster(int64_t tiles, int64_t seen, int num_sms, const int *active, double *least) {
    int best = 1;
    for (int c = 1; c <= kMaxCluster && (c == 1 || seen >= 2 * c); ++c) {
        const int n = c == 1 ? num_sms : active[c];
        if (n < 1) continue;
        const double t = (double)((tiles + n - 1) / n) * ((double)((seen + c - 1) / c) * 0.88 + (c == 1 ? 4 : 5));
        if (c == 1 || t < *least) {
            *least = t;
            best = c;
        }
    }
    return best;
}

}  // namespace

cudaError_t launch_span_attention(const SpanArgs &a, const CacheDev &C, int layer, const CUtensorMap &qmap,
                                  const CUtensorMap &kmap, const CUtensorMap &vmap, const __nv_bfloat16 *values,
                                  __nv_bfloat16 *out, float *lse, int num_sms, cudaStream_t s) {
    static int active[kOnceDevices][kMaxCluster + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev >= kOnceDevices) e = cudaErrorInvalidDevice;
    if (e != cudaSuccess) return e;
    e = once_per_device(0, [&] {
        const cudaError_t r = cudaFuncSetAttribute(span_attention_kernel<false>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kAttSmem);
        return r == cudaSuccess ? prepare_clusters(span_attention_kernel<true>, kAttThreads, kAttSmem, active[dev]) : r;
    });
    if (e != cudaSuccess) return e;
    const int T = span_tile_tokens(a.G);
    const int64_t heads = (int64_t)a.B * a.Hkv;
    // key tiles that a query tile sees at most
    const int64_t seen = ((int64_t)a.span + T < a.n_kv ? ((int64_t)a.span + T) / kTile + 2 + (a.sinks + kTile - 1) / kTile
                                                       : (a.n_kv + kTile - 1) / kTile);
    // The wide form where its units fill the SMs. Below that, whichever ends first: a wide CTA takes
    // about 1.45 us a key tile (two query tiles), a split one 0.88 us (one), and a unit about 4 us to
    // start and to write (512 tokens of 16K contexts, 2 x 8 KV heads: 183 and 221 us).
    const int64_t wide = (a.n_q + 2 * T - 1) / (2 * T) * heads;
    int cl = 0;   // 0: wide
    if (wide < num_sms) {
        double split = 0;
        cl = best_cluster((a.n_q + T - 1) / T * heads, seen, num_sms, active[dev], &split);
        if (seen * 1.45 + 4 < split) cl = 0;
    }
    const int64_t q_tiles = cl ? (a.n_q + T - 1) / T : (a.n_q + 2 * T - 1) / (2 * T);
    const int64_t units = q_tiles * heads;
    const int64_t grid = units * (cl ? cl : 1);
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
    return cl ? cudaLaunchKernelEx(&cfg, span_attention_kernel<true>, a, C, layer, qmap, kmap, vmap, values, out, lse,
                                   (int)q_tiles, cl)
              : cudaLaunchKernelEx(&cfg, span_attention_kernel<false>, a, C, layer, qmap, kmap, vmap, values, out, lse,
                                   (int)q_tiles, 1);
}

cudaError_t launch_span_scores(const SpanArgs &a, const CacheDev &C, int layer, const CUtensorMap &qmap,
                               const CUtensorMap &kmap, const float *lse, float *scores, float *part, int w,
                               bool per_head, int num_sms, cudaStream_t s) {
    cudaError_t e = once_per_device(0, [&] {
        return cudaFuncSetAttribute(span_scores_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kScSmem);
    });
    if (e != cudaSuccess) return e;
    const int keys = 2 * (kTile / w * w), T = span_tile_tokens(a.G);
    const int runs = (a.n_kv + keys - 1) / keys, n_win = (a.n_kv + w - 1) / w;
    const int units = per_head ? a.B * a.Hkv : a.B;
    const int64_t items = (int64_t)runs * units, wins = (int64_t)units * n_win;
    // Parts per item: enough that the longest (at the lengths that the host knows) does not
    // outlast an even share of the SMs, and no shorter than two steps. (At most 16, 32 or 64 parts:
    // every query of 2K 37.7, 26.6, 30.0 us, of 4K 62.8, 62.6, 68.8 us, 2 x 8K with a span of 1K
    // and sinks 159, 164, 164 us.)
    int parts = 1;
    if (items < 8 * num_sms) {
        int64_t heavy = 0, total = 0;
        for (int x = 0; x < runs; ++x) {
            const int k0 = x * keys, shift = a.n_kv - a.n_q;
            const int lo = max(0, k0 - shift);
            const int hi = k0 < a.sinks ? a.n_q : min(a.n_q, min(k0 + keys, a.n_kv) - 1 + a.span - shift);
            const int64_t steps = hi <= lo ? 0 : (int64_t)((hi - 1) / T + 1 - lo / T) * (per_head ? 1 : a.Hkv);
            heavy = steps > heavy ? steps : heavy;
            total += steps * units;
        }
        while (parts < kMaxSpanParts && 2 * parts * wins <= kSpanPartFloats && heavy >= 4 * parts &&
               heavy * num_sms * 2 > total * parts)
            parts *= 2;
    }
    const int64_t grid = items * parts;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    span_scores_kernel<<<(unsigned)grid, kScThreads, kScSmem, s>>>(a, C, layer, qmap, kmap, lse, scores, part, w, n_win,
                                                                   per_head ? 1 : 0, parts);
    e = cudaGetLastError();
    if (e != cudaSuccess || parts == 1) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((wins + 127) / 128));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, span_scores_sum_kernel, (const float *)part, scores, wins, parts,
                              (float)(per_head ? a.G : a.Hq));
}

}  // namespace qevict
