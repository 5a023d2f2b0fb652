// Attention of the last positions over the cache in 8 bits.
//
// Query i of n_q sits at p = kv_len - n_q + i and sees the keys j <= p: softmax(q k / sqrt(d)) V, with
// k = code * s of its block, v likewise, and bf16 rows in the block that is not full. A row is a (query, query
// head); the rows of one KV head read the same bytes, so that 4 G n_q 128 operations meet 256 bytes a token:
// memory-bound for single tokens.
//
// A unit is what one bulk copy pair brings: a block's codes, or 32 rows of an open block, 16 KiB either way. The
// units of all (sequence, KV head) pairs, in one row, are divided evenly over the CTAs, whatever the lengths; a
// CTA's run of one pair is a segment. Within a CTA each warp takes units of its own through a ring of its own
// (nothing but the end of a segment makes warps meet) and keeps a running maximum, sum and output for 8 rows:
//   S = Q K^T      m16n8k16, rows x tokens (8 of the 16 rows used): a key's row is the operand as it lies, each
//                  lane 32 consecutive channels of a token; the query's fragments follow that order of channels.
//   O^T += V^T P   m16n8k16, channels x rows: S's registers are P's operand; V comes transposed from ldmatrix
//                  (which moves pairs of channels; their bytes are put in order on the way to fp16).
// Codes become fp16 exactly (int8 and e4m3 alike). A query row is scaled by a power of two into fp16's range:
// exact down to 2^-28 of its largest channel. Scales of K go into the factor of the logits, scales of V into an
// FMA per output after a block's product. More than 8 rows: 2, 4 or 8 warps share a ring, 8 rows each.
// A segment's warps meet in shared memory; a pair that lies in several CTAs is joined by the last of them.
#include "qevict_block.cuh"
#include "qevict_tc.cuh"

namespace qevict {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kRows = kMaxBlkQueries * kMaxG;      // rows of a pair
constexpr int kHalf = kBlkBytes / 2;               // what one copy brings: K or V of a unit
constexpr int kSlots = 24;                         // of kHalf bytes, 3 for each warp
constexpr int kOStride = kHeadDim + 4;             // floats of a row in shared memory and in a partial result
constexpr int kLeastUnits = 4;                     // a CTA takes no fewer units than this, where there are few
constexpr int kSmemBytes = kSlots * kHalf + kWarps * 8 * kOStride * 4 + kWarps * 8 * 8 + 2 * kSlots * 8 + 64;

__device__ __forceinline__ int units_of(int len) { return (len >> 6) + (((len & (kBlk - 1)) + kOpenHalf - 1) / kOpenHalf); }

// The units of all pairs in a row: where position `at` lies, moving forwards only.
struct Walk {
    int base;       // of sequence b
    int b, len, n;  // n: units of each of its pairs
    __device__ __forceinline__ void start(const BlockDev &D, const int32_t *kv_len) {
        base = 0;
        b = 0;
        len = blk_len(D, kv_len, 0);
        n = units_of(len);
    }
    __device__ __forceinline__ void to(const BlockDev &D, const int32_t *kv_len, int at) {
        while (at >= base + n * D.Hkv && b + 1 < D.B) {
            base += n * D.Hkv;
            len = blk_len(D, kv_len, ++b);
            n = units_of(len);
        }
    }
};

__device__ __forceinline__ void copy_half(uint32_t dst, const uint8_t *src, uint32_t bar) {
    tc_expect_tx(bar, kHalf);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(kHalf), "r"(bar)
                 : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 ldsm_t(uint32_t addr) {
    uint4 v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t bits(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }
// a word from ldmatrix (two channels of a token, the same of the next): the tokens' first channel, their second
template <int FMT>
__device__ __forceinline__ void pair_halves(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == QEVICT_BLOCK_INT8) {
        const __half2 off = __half2half2(__ushort_as_half(0x6480));
        const uint32_t l = __byte_perm(w, 0x64646464u, 0x5240), h = __byte_perm(w, 0x64646464u, 0x5341);
        lo = bits(__hsub2(*reinterpret_cast<const __half2 *>(&l), off));
        hi = bits(__hsub2(*reinterpret_cast<const __half2 *>(&h), off));
    } else {
        const uint32_t x = __byte_perm(w, 0, 0x3120);
        lo = bits(blk_half2<FMT>(x));
        hi = bits(blk_half2<FMT, true>(x));
    }
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
    return fmaxf(x, __shfl_xor_sync(~0u, x, 2));
}

// What a warp keeps of its 8 rows: lane (n, q) = (lane / 4, lane % 4) has row n's maximum (log2 domain) and its
// own share of the sum, and of O^T the rows 2 q, 2 q + 1 of channels 16 i + 2 n (o[i][0..1]) and + 1 (o[i][2..3]).
struct Rows {
    float m, l, o[8][4];
    __device__ __forceinline__ void clear() {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    }
    // moves the maximum; what the exponentials are taken against
    __device__ __forceinline__ float raise(float top, int q) {
        const float m1 = fmaxf(m, top), ref = m1 == -INFINITY ? 0.f : m1;
        if (__any_sync(~0u, m1 > m)) {
            const float f = tc_ex2(m - ref);   // 0 for the first keys
            const float f0 = __shfl_sync(~0u, f, 8 * q), f1 = __shfl_sync(~0u, f, 8 * q + 4);
            l *= f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i][0] *= f0;
                o[i][1] *= f1;
                o[i][2] *= f0;
                o[i][3] *= f1;
            }
            m = m1;
        }
        return ref;
    }
};

struct Smem {
    uint32_t ring, full, empty;   // shared addresses
    float *o;                     // [warp][8][kOStride]
    float2 *ml;                   // [warp][8]
    int *stop;
};

// One row group's part of one pair's units, for as many units as the segment has for this warp's ring.
template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) block_attend_kernel(const BlockDev D, const BlockAttendArgs a, int groups) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Smem S;
    S.ring = smem_u32(smem);
    S.o = reinterpret_cast<float *>(smem + kSlots * kHalf);
    S.ml = reinterpret_cast<float2 *>(S.o + kWarps * 8 * kOStride);
    S.full = smem_u32(S.ml + kWarps * 8);
    S.empty = S.full + kSlots * 8;
    int *flags = reinterpret_cast<int *>(smem + kSmemBytes - 64);   // [0] stop, [1] this CTA joins the pair
    S.stop = flags;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, q = lane & 3;
    const int streams = kWarps / groups, stream = warp % streams, group = warp / streams;
    const int slots = kSlots / streams, slot0 = stream * slots;
    const int R = a.n_q * D.G;
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            tc_mbar_init(S.full + 8 * i, 1);
            tc_mbar_init(S.empty + 8 * i, groups);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        flags[0] = 0;
    }
    // units of all pairs; sequences without any get their rows here
    int total = 0;   // fits: a handle has fewer than 2^30 blocks
    for (int b = lane; b < D.B; b += 32) total += units_of(blk_len(D, a.kv_len, b));
    for (int s = 16; s; s >>= 1) total += __shfl_xor_sync(~0u, total, s);
    total *= D.Hkv;
    for (int b = blockIdx.x; b < D.B; b += gridDim.x) {
        if (blk_len(D, a.kv_len, b) > 0) continue;
        for (int i = tid; i < a.n_q * D.Hq * kHeadDim / 8; i += kThreads)
            reinterpret_cast<uint4 *>(a.out + (int64_t)b * a.n_q * D.Hq * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
        for (int i = tid; i < a.n_q * D.Hq && a.lse; i += kThreads) a.lse[(int64_t)b * a.n_q * D.Hq + i] = -INFINITY;
    }
    const int ctas = min((int)gridDim.x, (total + kLeastUnits - 1) / kLeastUnits);
    if ((int)blockIdx.x >= ctas || total == 0) return;
    const int begin = (int)((int64_t)total * blockIdx.x / ctas), end = (int)((int64_t)total * (blockIdx.x + 1) / ctas);
    __syncthreads();

    // copies: the ring's first warp issues them, in the order in which the ring's units are worked
    Walk cw;
    int cat = begin + ((stream - begin) & (streams - 1));
    const uint8_t *csrc = nullptr;
    int cslot = 0, chalf = 0, cuse = 0;
    cw.start(D, a.kv_len);
    auto issue = [&]() {
        if (cat >= end || *(volatile int *)S.stop) return;
        if (chalf == 0) {
            cw.to(D, a.kv_len, cat);
            const int x = cat - cw.base, u = x % cw.n, nb = cw.len >> 6;
            const int64_t pair = (int64_t)cw.b * D.Hkv + x / cw.n;
            csrc = u < nb ? D.codes + blk_code_off(D, pair, u) : D.open + blk_open_off(pair, nb, (u - nb) * kOpenHalf);
        }
        const int s = slot0 + cslot;
        // every warp of the ring has read what the slot held
        if (groups > 1 && cuse > 0 && !tc_wait(S.empty + 8 * s, (cuse - 1) & 1, S.stop)) return;
        if (lane == 0) copy_half(S.ring + s * kHalf, csrc + chalf * kHalf, S.full + 8 * s);
        chalf ^= 1;
        if (chalf == 0) cat += streams;
        if (++cslot == slots) cslot = 0, ++cuse;
    };
    if (group == 0)
        for (int i = 0; i < slots; ++i) issue();

    int slot = 0, use = 0;   // of the next half to read
    bool ok = true;
    auto wait_half = [&]() {
        ok = ok && tc_wait(S.full + 8 * (slot0 + slot), use & 1, S.stop);
        __syncwarp();
        return S.ring + (slot0 + slot) * kHalf;
    };
    auto done_half = [&]() {
        __syncwarp();
        if (groups > 1 && lane == 0) tc_arrive(S.empty + 8 * (slot0 + slot));
        if (++slot == slots) slot = 0, ++use;
        if (group == 0) issue();
    };

    Walk w;
    w.start(D, a.kv_len);
    constexpr float kLog2e = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)
    const int row = 8 * group + n;                                        // this lane's row of the pair
    for (int at = begin; at < end;) {
        w.to(D, a.kv_len, at);
        const int h = (at - w.base) / w.n, b = w.b, len = w.len, nb = len >> 6, first = w.base + h * w.n;
        const int64_t pair = (int64_t)b * D.Hkv + h;
        const int u0 = at - first, u1 = min(w.n, end - first), skip = (stream - at) & (streams - 1);
        at = first + u1;
        // the row's query: channels 32 q .. 32 q + 31 as fp16 fragments, scaled by a power of two
        const __nv_bfloat16 *qrow =
            a.q + (((int64_t)b * a.n_q + min(row / D.G, a.n_q - 1)) * D.Hq + h * D.G + row % D.G) * kHeadDim + 32 * q;
        uint32_t qf[8][2];
        float scale;
        {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = row < R ? __ldg(reinterpret_cast<const uint4 *>(qrow) + i) : make_uint4(0, 0, 0, 0);
            uint32_t top = 0;
            const uint32_t *xw = &x[0].x;
#pragma unroll
            for (int i = 0; i < 16; ++i) top = __vmaxu2(top, xw[i] & 0x7fff7fffu);
            top = max(top & 0xffffu, top >> 16);
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            // the largest channel into [2^14, 2^15); an infinite or NaN row stays so
            const int e = top >= 0x7f80u ? 14 : min(max((int)(top >> 7) - 127, -112), 127);
            const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
            scale = __uint_as_float((uint32_t)(127 - 14 + e) << 23) * kLog2e;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                qf[i >> 1][i & 1] = bits(__floats2half2_rn(__uint_as_float(xw[i] << 16) * up,
                                                           __uint_as_float(xw[i] & 0xffff0000u) * up));
        }
        const int last = len - a.n_q + (row < R ? row / D.G : a.n_q - 1);   // the last token the row sees
        Rows r;
        r.clear();
        // this ring's units of the segment
        for (int u = u0 + skip; u < u1; u += streams) {
            if (u < nb) {
                const float2 sc = __ldg(D.scale + pair * D.NB + u);
                uint32_t base = wait_half();
                float x[8][2];
                const uint32_t k0 = base + n * kHeadDim + (((2 * q) ^ n) << 4), k1 = base + n * kHeadDim + (((2 * q + 1) ^ n) << 4);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const uint4 lo = lds128(k0 + t * 8 * kHeadDim), hi = lds128(k1 + t * 8 * kHeadDim);
                    const uint32_t kw[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mma<false>(c, qf[i][0], 0u, qf[i][1], 0u, bits(blk_half2<FMT>(kw[i])),
                                   bits(blk_half2<FMT, true>(kw[i])));
                    x[t][0] = c[0];
                    x[t][1] = c[1];
                }
                done_half();
                const float f = sc.x * scale;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    x[t][0] *= f;
                    x[t][1] *= f;
                }
                if (a.weights && row < R) {
                    float *g = a.logits + ((pair * D.NB + u) * R + row) * kBlk + 2 * q;
#pragma unroll
                    for (int t = 0; t < 8; ++t) *reinterpret_cast<float2 *>(g + 8 * t) = make_float2(x[t][0], x[t][1]);
                }
                if (u * kBlk + kBlk - 1 > len - a.n_q) {
#pragma unroll
                    for (int t = 0; t < 8; ++t)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (u * kBlk + 8 * t + 2 * q + j > last) x[t][j] = -INFINITY;
                }
                float top = x[0][0];
#pragma unroll
                for (int t = 0; t < 8; ++t) top = fmaxf(top, fmaxf(x[t][0], x[t][1]));
                const float ref = r.raise(quad_max(top), q);
                uint32_t p[8];
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float p0 = tc_ex2(x[t][0] - ref), p1 = tc_ex2(x[t][1] - ref);
                    r.l += p0 + p1;
                    p[t] = bits(__floats2half2_rn(p0, p1));   // against the running maximum: 2^-12 of a term
                }
                base = wait_half();
                const uint32_t v0 = base + lane * kHeadDim;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 va = ldsm_t(v0 + ((i ^ (lane & 7)) << 4));
                    const uint4 vb = ldsm_t(v0 + 32 * kHeadDim + ((i ^ (lane & 7)) << 4));
                    const uint32_t vw[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        uint32_t a0, a1, a2, a3;
                        pair_halves<FMT>(vw[2 * t], a0, a1);
                        pair_halves<FMT>(vw[2 * t + 1], a2, a3);
                        mma<false>(c, a0, a1, a2, a3, p[2 * t], p[2 * t + 1]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) r.o[i][j] = fmaf(c[j], sc.y, r.o[i][j]);
                }
                done_half();
            } else {
                // 32 bf16 rows of the open block
                const int t0 = nb * kBlk + (u - nb) * kOpenHalf;
                uint4 qx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    qx[i] = row < R ? __ldg(reinterpret_cast<const uint4 *>(qrow) + i) : make_uint4(0, 0, 0, 0);
                const uint32_t *qw = &qx[0].x;
                uint32_t base = wait_half();
                float x[4][2];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 k = lds128(base + blk_open_chunk(8 * t + n, 4 * q + i));
                        mma<true>(c, qw[4 * i], 0u, qw[4 * i + 1], 0u, k.x, k.y);
                        mma<true>(c, qw[4 * i + 2], 0u, qw[4 * i + 3], 0u, k.z, k.w);
                    }
                    x[t][0] = c[0] * kLog2e;
                    x[t][1] = c[1] * kLog2e;
                }
                done_half();
                if (a.weights && row < R) {
                    float *g = a.logits + ((pair * D.NB + nb) * R + row) * kBlk + (u - nb) * kOpenHalf + 2 * q;
#pragma unroll
                    for (int t = 0; t < 4; ++t) *reinterpret_cast<float2 *>(g + 8 * t) = make_float2(x[t][0], x[t][1]);
                }
                float top = -INFINITY;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (t0 + 8 * t + 2 * q + j > last) x[t][j] = -INFINITY;
                        top = fmaxf(top, x[t][j]);
                    }
                const float ref = r.raise(quad_max(top), q);
                uint32_t p[4], pl[4];   // each probability as two bf16 parts
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float p0 = tc_ex2(x[t][0] - ref), p1 = tc_ex2(x[t][1] - ref);
                    r.l += p0 + p1;
                    p[t] = pack_bf(p0, p1);
                    pl[t] = pack_bf(p0 - __uint_as_float(p[t] << 16), p1 - __uint_as_float(p[t] & 0xffff0000u));
                }
                base = wait_half();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 va = ldsm_t(base + blk_open_chunk(lane, 2 * i));
                    const uint4 vb = ldsm_t(base + blk_open_chunk(lane, 2 * i + 1));
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
                    mma<true>(c, va.x, vb.x, va.y, vb.y, p[0], p[1]);
                    mma<true>(c, va.z, vb.z, va.w, vb.w, p[2], p[3]);
                    mma<true>(c, va.x, vb.x, va.y, vb.y, pl[0], pl[1]);
                    mma<true>(c, va.z, vb.z, va.w, vb.w, pl[2], pl[3]);
                    // c: channels n and 8 + n of the 16; the accumulators hold 2 n and 2 n + 1
                    const int s0 = ((2 * n) & 7) * 4 + q, s1 = s0 + 4;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float lo0 = __shfl_sync(~0u, c[j], s0), hi0 = __shfl_sync(~0u, c[2 + j], s0);
                        const float lo1 = __shfl_sync(~0u, c[j], s1), hi1 = __shfl_sync(~0u, c[2 + j], s1);
                        r.o[i][j] += n < 4 ? lo0 : hi0;
                        r.o[i][2 + j] += n < 4 ? lo1 : hi1;
                    }
                }
                done_half();
            }
        }
        // the segment's warps meet: maxima and sums, then outputs relative to the common maximum
        r.l += __shfl_xor_sync(~0u, r.l, 1);
        r.l += __shfl_xor_sync(~0u, r.l, 2);
        if (q == 0) S.ml[warp * 8 + n] = make_float2(r.m, r.l);
        __syncthreads();
        {
            float m = -INFINITY;
            for (int i = 0; i < streams; ++i) m = fmaxf(m, S.ml[(group * streams + i) * 8 + n].x);
            const float f = r.m == -INFINITY ? 0.f : tc_ex2(r.m - m);
            const float f0 = __shfl_sync(~0u, f, 8 * q), f1 = __shfl_sync(~0u, f, 8 * q + 4);
            float *o = S.o + (warp * 8 + 2 * q) * kOStride + 2 * n;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                *reinterpret_cast<float2 *>(o + 16 * i) = make_float2(r.o[i][0] * f0, r.o[i][2] * f0);
                *reinterpret_cast<float2 *>(o + kOStride + 16 * i) = make_float2(r.o[i][1] * f1, r.o[i][3] * f1);
            }
        }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == w.n;
        float *part = a.part + ((int64_t)blockIdx.x * 2 + (u0 == 0 ? 1 : 0)) * kRows * kOStride;
        auto finish = [&](int rr, float m, float l, float4 o) {   // a thread's four channels of a joined row
            const int i = rr / D.G, head = h * D.G + rr % D.G, c4 = tid & 31;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const uint2 v = make_uint2(pack_bf(o.x * inv, o.y * inv), pack_bf(o.z * inv, o.w * inv));
            reinterpret_cast<uint2 *>(a.out + (((int64_t)b * a.n_q + i) * D.Hq + head) * kHeadDim)[c4] = v;
            if (c4 == 0) {
                const float lse = l == 0.f ? -INFINITY : m + log2f(l);
                if (a.lse) a.lse[((int64_t)b * D.Hq + head) * a.n_q + i] = lse * 0.6931471805599453f;
                if (a.weights) a.row_lse[pair * R + rr] = lse;
            }
        };
        for (int rr = tid >> 5; rr < R; rr += kWarps) {
            const int w0 = (rr >> 3) * streams;
            float m = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = 0; i < streams; ++i) m = fmaxf(m, S.ml[(w0 + i) * 8 + (rr & 7)].x);
            const float ref = m == -INFINITY ? 0.f : m;   // a row that sees nothing here: sums of 0
            for (int i = 0; i < streams; ++i) {
                const float2 ml = S.ml[(w0 + i) * 8 + (rr & 7)];
                l = fmaf(ml.y, tc_ex2(ml.x - ref), l);
                const float4 x = *reinterpret_cast<const float4 *>(S.o + ((w0 + i) * 8 + (rr & 7)) * kOStride + 4 * (tid & 31));
                o.x += x.x;
                o.y += x.y;
                o.z += x.z;
                o.w += x.w;
            }
            if (whole) {
                finish(rr, m, l, o);
            } else {
                *reinterpret_cast<float4 *>(part + rr * kOStride + 4 * (tid & 31)) = o;
                if ((tid & 31) == 0) *reinterpret_cast<float2 *>(part + rr * kOStride + kHeadDim) = make_float2(m, l);
            }
        }
        if (!whole) {
            const int c0 = (int)(((int64_t)(first + 1) * ctas - 1) / total);
            const int c1 = (int)(((int64_t)(first + w.n) * ctas - 1) / total);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const uint32_t seen = atomicAdd(a.count + pair, 1u);
                flags[1] = seen == (uint32_t)(c1 - c0);
                if (flags[1]) a.count[pair] = 0;
            }
            __syncthreads();
            if (flags[1]) {
                __threadfence();
                for (int rr = tid >> 5; rr < R; rr += kWarps) {
                    auto at_part = [&](int c) {
                        return a.part + (((int64_t)c * 2 + (c == c0 ? 1 : 0)) * kRows + rr) * kOStride;
                    };
                    float m = -INFINITY, l = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, __ldcg(at_part(c) + kHeadDim));
                    for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, s));
                    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 4
                    for (int c = c0; c <= c1; ++c) {
                        const float *p = at_part(c);
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p + kHeadDim));
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(p) + lane);
                        const float f = tc_ex2(ml.x - ref);   // 0 for a part whose keys the row does not see
                        l = fmaf(ml.y, f, l);
                        o.x = fmaf(x.x, f, o.x);
                        o.y = fmaf(x.y, f, o.y);
                        o.z = fmaf(x.z, f, o.z);
                        o.w = fmaf(x.w, f, o.w);
                    }
                    finish(rr, m, l, o);
                }
            }
        }
        __syncthreads();   // the segment's shared memory may be written again
    }
    ok = !__any_sync(~0u, !ok);
    if (!ok && lane == 0) blk_status(D, QEVICT_ERR_TIMEOUT, 0, blockIdx.x);
    // after a wait that ran out: copies still on their way are waited for before the CTA ends
    if (!ok && group == 0) {
        for (int i = 0; i < slots; ++i) {
            const int uses = cuse + (i < cslot ? 1 : 0);
            const long long t = clock64();
            while (uses > 0 && !tc_try_wait(S.full + 8 * (slot0 + i), (uses - 1) & 1) && clock64() - t < kDefaultWaitCycles) {
            }
        }
    }
}

// The tokens' weights from the logits that the attention left: one thread per token, four blocks to a CTA.
__global__ void __launch_bounds__(kThreads) block_weights_kernel(const BlockDev D, const BlockAttendArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the attention kernel has ended
    const int per = (D.NB + 3) / 4;
    const int64_t pair = blockIdx.x / per;
    const int pos = (int)(blockIdx.x % per) * kThreads + threadIdx.x, R = a.n_q * D.G;
    if (pos >= blk_len(D, a.kv_len, (int)(pair / D.Hkv))) return;
    const int64_t j = pos >> 6;
    const int len = blk_len(D, a.kv_len, (int)(pair / D.Hkv));
    float w = 0.f;
    for (int r = 0; r < R; ++r) {
        const float x = a.logits[((pair * D.NB + j) * R + r) * kBlk + (pos & 63)];
        if (pos <= len - a.n_q + r / D.G) w += tc_ex2(x - a.row_lse[pair * R + r]);
    }
    float *o = a.weights + pair * D.capacity + pos;
    w /= D.G;
    *o = a.accumulate ? *o + w : w;
}

}  // namespace

int64_t blk_part_floats(int, int, int, int) { return (int64_t)kMaxBlkCtas * 2 * kRows * kOStride; }

cudaError_t launch_block_attend(const BlockDev &D, int fmt, const BlockAttendArgs &a, int num_sms, cudaStream_t s) {
    auto kernel = fmt == QEVICT_BLOCK_INT8 ? block_attend_kernel<QEVICT_BLOCK_INT8> : block_attend_kernel<QEVICT_BLOCK_E4M3>;
    cudaError_t e = once_per_device(fmt, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    const int R = a.n_q * D.G, groups = R <= 8 ? 1 : R <= 16 ? 2 : R <= 32 ? 4 : 8;
    kernel<<<num_sms < kMaxBlkCtas ? num_sms : kMaxBlkCtas, kThreads, kSmemBytes, s>>>(D, a, groups);
    e = cudaGetLastError();
    if (e != cudaSuccess || !a.weights) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((int64_t)D.B * D.Hkv * ((D.NB + 3) / 4)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, block_weights_kernel, D, a);
}

}  // namespace qevict
