// Attention of the last positions over the cache in 8 bits.
//
// Query i of n_q sits at p = kv_len - n_q + i and sees the keys j <= p: softmax(q k / sqrt(d)) V, with
// k = code * s of its block, v likewise, and bf16 rows in the block that is not full. A row is a (query, query
// head); the rows of one KV head read the same bytes, so that 4 G n_q 128 operations meet 256 bytes a token:
// memory-bound for single tokens.
//
// A unit is what one pair of bulk copies brings: a block's codes, or 32 rows of an open block, 16 KiB either way. The
// units of all (sequence, KV head) pairs, in one row, are divided evenly over the device's warps, whatever the
// lengths: each warp takes a run of them through a ring of its own (no warps ever meet), and keeps a running
// maximum, sum and output for 8 rows:
//   S = Q K^T      m16n8k16, rows x tokens (8 of the 16 rows used): a key's row is the operand as it lies, each
//                  lane 32 consecutive channels of a token; the query's fragments follow that order of channels.
//   O^T += V^T P   m16n8k16, channels x rows: S's registers are P's operand; V comes transposed from ldmatrix
//                  (which moves pairs of channels; their bytes are put in order on the way to fp16).
// Codes become fp16 exactly (int8 and e4m3 alike). A query row is scaled by a power of two into fp16's range:
// exact down to 2^-28 of its largest channel. Scales of K go into the factor of the logits, scales of V into an
// FMA per output after a block's product. More than 8 rows: warps share a ring, 8 rows each.
// A second kernel, launched while the first runs, adds up the parts of pairs that lie in several runs.
// Measured: single tokens of 4 x 128K (1.07 GB) 155 us, 6.9 TB/s; of 16 x 5-16K 31 us, 5.5 TB/s, of which 25 under load.
#include "qevict_block.cuh"
#include "qevict_tc.cuh"

namespace qevict {
namespace {

constexpr int kThreads = 256, kWarps = 8;          // of the joining kernel
constexpr int kHalf = kBlkBytes / 2;               // what one copy brings: K or V of a unit
// Of kHalf bytes, 2 for each warp: 128 KiB on their way to an SM. With 3 for each the memory system serves the SMs less
// evenly (the slowest took 17 % longer than the median for as many bytes: 4 x 128K 175 us against 158), with 1 it idles (190).
// That is with a ring to a warp; six rings of 9 to 16 rows divide the slots to 2 each as well and leave 4 (96 KiB).
constexpr int kSlots = 16;
constexpr int kRec = kHeadDim + 4;                 // floats of a row of a partial result: output, maximum, sum
static_assert(kRec % 4 == 0, "rows of whole float4");
constexpr int kSmemBytes = kSlots * kHalf + 2 * kSlots * 8 + 16;

__device__ __forceinline__ int units_of(int len) { return (len >> 6) + (((len & (kBlk - 1)) + kOpenHalf - 1) / kOpenHalf); }

// The units of all pairs in a row: how many there are, and with `b` those before sequence b's. A whole warp.
__device__ __forceinline__ int count_units(const BlockDev &D, const int32_t *kv_len, int b, int *before) {
    int total = 0, ahead = 0;   // fit: a handle has fewer than 2^30 blocks
    for (int i = threadIdx.x & 31; i < D.B; i += 32) {
        const int n = units_of(blk_len(D, kv_len, i));
        total += n;
        if (i < b) ahead += n;
    }
    if (before) *before = (int)__reduce_add_sync(~0u, (unsigned)ahead) * D.Hkv;
    return (int)__reduce_add_sync(~0u, (unsigned)total) * D.Hkv;
}

// A unit: unit u of n of KV head h of sequence b
struct Unit {
    int b, h, u, len, n;
    // the unit at position `at` of the row; a whole warp
    __device__ __forceinline__ void find(const BlockDev &D, const int32_t *kv_len, int at) {
        const int lane = threadIdx.x & 31;
        int base = 0;
        for (int b0 = 0;; b0 += 32) {
            const int l = b0 + lane < D.B ? blk_len(D, kv_len, b0 + lane) : 0;
            const int mine = units_of(l) * D.Hkv;
            int sum = mine;
            for (int s = 1; s < 32; s <<= 1) {
                const int x = __shfl_up_sync(~0u, sum, s);
                if (lane >= s) sum += x;
            }
            const uint32_t behind = __ballot_sync(~0u, base + sum > at);
            if (behind) {
                const int j = __ffs(behind) - 1;
                b = b0 + j;
                len = __shfl_sync(~0u, l, j);
                n = units_of(len);
                const int x = at - base - __shfl_sync(~0u, sum - mine, j);
                h = x / n;
                u = x - h * n;
                return;
            }
            base += __shfl_sync(~0u, sum, 31);
            if (b0 + 32 >= D.B) return;   // not reached: `at` lies in the row
        }
    }
    // the next one; the caller knows that there is one
    __device__ __forceinline__ void next(const BlockDev &D, const int32_t *kv_len, int steps = 1) {
        u += steps;
        while (u >= n) {
            u -= n;
            if (++h == D.Hkv) {
                h = 0;
                do len = b + 1 < D.B ? blk_len(D, kv_len, ++b) : kBlk;
                while (len == 0);
                n = units_of(len);
            }
        }
    }
    __device__ __forceinline__ const uint8_t *source(const BlockDev &D) const {
        const int64_t pair = (int64_t)b * D.Hkv + h;
        const int nb = len >> 6;
        return u < nb ? D.codes + blk_code_off(D, pair, u) : D.open + blk_open_off(pair, nb, (u - nb) * kOpenHalf);
    }
};

// The cache is read once a call: its lines leave the L2 first (the logits of a call with weights, and the parts, stay
// in: 8 x 32K 83.7 -> 81.2 us, 5 queries of 4 x 8K with weights 48 -> 45).
__device__ __forceinline__ void copy_half(uint32_t dst, const uint8_t *src, uint32_t bar) {
    uint64_t first_out;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first_out));
    tc_expect_tx(bar, kHalf);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::
                     "r"(dst), "l"(src), "r"(kHalf), "r"(bar), "l"(first_out)
                 : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
// What a warp keeps of its 8 rows: lane (n, q) = (lane / 4, lane % 4) has the maximum (log2 domain) of row n and its own
// share of its sum, and of O^T rows 2 q, 2 q + 1 of channels 16 i + 2 n (o[i][0..1]) and 16 i + 2 n + 1 (o[i][2..3]).
// Sums and outputs are relative to the maximum, times 2^15 while no block's scale (or 32 bf16 rows' product) reaches 2^64,
// so that the smallest values keep their bits, and times 2^-40 from the first that does, so that no sum of up to 2^21
// finite values passes fp32.
struct Rows {
    static constexpr float kLarge = 0x1p64f, kLess = 0x1p-55f;
    float m, l, unit, o[8][4];   // unit: 2^-15 of that factor, 1 or kLess
    __device__ __forceinline__ void clear() {
        m = -INFINITY;
        l = 0.f;
        unit = 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    }
    // Powers of two that the probabilities carry into their product. In fp16 they reach up to 2^15, so that one keeps its
    // 11 bits down to 2^-29 of the largest; with bf16 rows, whose exponent is fp32's, up to 2^-8, so that 32 of them times
    // the largest values stay finite.
    static constexpr float kLift = 15.f, kDrop = 8.f;
    __device__ __forceinline__ float of_rows() const { return 0x1p23f * unit; }
    // what sums and outputs are relative to, log2 domain
    __device__ __forceinline__ float base() const { return m + (unit == 1.f ? -15.f : 40.f); }
    __device__ __forceinline__ void less() {
        if (unit != 1.f) return;
        unit = kLess;
        l *= kLess;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] *= kLess;
    }
    // moves the maximum; what the exponentials are taken against
    __device__ __forceinline__ float raise(float top, int q) {
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const float m1 = fmaxf(m, top), ref = m1 == -INFINITY ? 0.f : m1;
        if (__any_sync(~0u, m1 > m)) {
            const float f = tc_ex2(m - ref);   // 0 for the first keys; 1 for the rows that stay
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

// log-sum-exp of a row from its maximum and sum, log2 domain; a row that sees nothing has a sum of 0
__device__ __forceinline__ float row_lse(float m, float l) { return l == 0.f ? -INFINITY : m + log2f(l); }

template <int FMT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1) block_attend_kernel(const BlockDev D, const BlockAttendArgs a, int groups) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t ring = smem_u32(smem), full = ring + kSlots * kHalf, empty = full + kSlots * 8;
    volatile int *stop = reinterpret_cast<int *>(smem + kSlots * kHalf + 2 * kSlots * 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, q = lane & 3;
    const int streams = WARPS / groups, stream = warp % streams, group = warp / streams;
    const int slots = kSlots / streams, slot0 = stream * slots;
    const int R = a.n_q * D.G, room = 8 * groups;
    if (tid < kSlots) {
        tc_mbar_init(full + 8 * tid, 1);
        tc_mbar_init(empty + 8 * tid, groups);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) *stop = 0;
    // this ring's run of the row of units
    const int total = count_units(D, a.kv_len, 0, nullptr);
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int runs = min((int)gridDim.x * streams, total), run = stream * gridDim.x + blockIdx.x;
    if (run >= runs || group >= groups) return;
    const int begin = (int)((int64_t)total * run / runs), end = (int)((int64_t)total * (run + 1) / runs);
    Unit w;
    w.find(D, a.kv_len, begin);

    // copies: the ring's first warp issues them, at first one from each lane
    Unit cu = w;
    int left = 2 * (end - begin), chalf = 0, cslot = 0, cuse = 0;   // copies not issued yet
    if (group == 0) {
        if (lane < min(slots, left)) {
            cu.next(D, a.kv_len, lane >> 1);
            copy_half(ring + (slot0 + lane) * kHalf, cu.source(D) + (lane & 1) * kHalf, full + 8 * (slot0 + lane));
        }
        __syncwarp();
        cu = w;
        const int m = min(slots, left);
        left -= m;
        if (left > 0) cu.next(D, a.kv_len, m >> 1);
        chalf = m & 1;
        cslot = m == slots ? 0 : m;
        cuse = m == slots;
    }
    int slot = 0, use = 0;   // of the next half to read
    bool ok = true;
    auto wait_half = [&]() {
        ok = __all_sync(~0u, ok && tc_wait(full + 8 * (slot0 + slot), use & 1, stop));
        return ring + (slot0 + slot) * kHalf;
    };
    auto done_half = [&]() {
        __syncwarp();
        if (groups > 1 && lane == 0) tc_arrive(empty + 8 * (slot0 + slot));
        if (++slot == slots) slot = 0, ++use;
        if (group != 0 || left == 0 || !ok) return;
        const int s = slot0 + cslot;   // the slot just read; every warp of the ring has read it
        if (groups > 1) {
            ok = __all_sync(~0u, tc_wait(empty + 8 * s, (cuse - 1) & 1, stop));   // a warp gives up as one
            if (!ok) return;
        }
        if (lane == 0) copy_half(ring + s * kHalf, cu.source(D) + chalf * kHalf, full + 8 * s);
        chalf ^= 1;
        if (--left > 0 && chalf == 0) cu.next(D, a.kv_len);
        if (++cslot == slots) cslot = 0, ++cuse;
    };

    constexpr float kLog2e = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)
    const int row = 8 * group + n;   // this lane's row of a pair
    for (int at = begin; at < end;) {
        const int b = w.b, h = w.h, u0 = w.u, len = w.len, nb = len >> 6, u1 = min(w.n, u0 + end - at);
        const int64_t pair = (int64_t)b * D.Hkv + h;
        const bool whole = u0 == 0 && u1 == w.n;
        at += u1 - u0;
        // the row's query: channels 32 q .. 32 q + 31 as fp16 fragments, scaled by a power of two
        const int i_q = min(row / D.G, a.n_q - 1), last = len - a.n_q + i_q;   // last: the last token that the row sees
        const uint4 *qrow = reinterpret_cast<const uint4 *>(
            a.q + (((int64_t)b * a.n_q + i_q) * D.Hq + h * D.G + row % D.G) * kHeadDim + 32 * q);
        uint32_t qf[16];
        float scale;
        {
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint4 x = row < R ? __ldg(qrow + e) : make_uint4(0, 0, 0, 0);
                qf[4 * e] = x.x;
                qf[4 * e + 1] = x.y;
                qf[4 * e + 2] = x.z;
                qf[4 * e + 3] = x.w;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) top = __vmaxu2(top, qf[e] & 0x7fff7fffu);
            top = max(top & 0xffffu, top >> 16);
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            // the largest channel into [2^14, 2^15); an infinite or NaN row stays so
            const int e2 = top >= 0x7f80u ? 14 : min(max((int)(top >> 7) - 127, -112), 127);
            const float up = __uint_as_float((uint32_t)(127 + 14 - e2) << 23);
            scale = __uint_as_float((uint32_t)(127 - 14 + e2) << 23) * kLog2e;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                qf[e] = bits(__floats2half2_rn(__uint_as_float(qf[e] << 16) * up, __uint_as_float(qf[e] & 0xffff0000u) * up));
        }
        Rows r;
        r.clear();
        for (int u = u0; u < u1; ++u) {
            float *logits = a.weights && row < R ? a.logits + (pair * D.NB + min(u, nb)) * R * kBlk + row * 8 + 2 * q : nullptr;
            if (u < nb) {
                const float2 sc = __ldg(D.scale + pair * D.NB + u);
                uint32_t base = wait_half();
                float x[8][2];
                const uint32_t k0 = base + n * kHeadDim + (((2 * q) ^ n) << 4), k1 = base + n * kHeadDim + (((2 * q + 1) ^ n) << 4);
                // two tiles of 8 tokens at a time: their chains of products overlap
#pragma unroll
                for (int t = 0; t < 8; t += 2) {
                    float c[2][4] = {};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t ka = half ? k1 : k0;
                        const uint4 ta = lds128(ka + t * 8 * kHeadDim), tb = lds128(ka + (t + 1) * 8 * kHeadDim);
                        const uint32_t kw[2][4] = {{ta.x, ta.y, ta.z, ta.w}, {tb.x, tb.y, tb.z, tb.w}};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                mma<false>(c[e], qf[8 * half + 2 * i], 0u, qf[8 * half + 2 * i + 1], 0u,
                                           bits(blk_half2<FMT>(kw[e][i])), bits(blk_half2<FMT, true>(kw[e][i])));
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[t + e][0] = c[e][0];
                        x[t + e][1] = c[e][1];
                    }
                }
                done_half();
                const float f = sc.x * scale;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    x[t][0] *= f;
                    x[t][1] *= f;
                }
                if (logits) {
#pragma unroll
                    for (int t = 0; t < 8; ++t) *reinterpret_cast<float2 *>(logits + t * R * 8) = make_float2(x[t][0], x[t][1]);
                }
                if (u * kBlk + kBlk - 1 > len - a.n_q) {
#pragma unroll
                    for (int t = 0; t < 8; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (u * kBlk + 8 * t + 2 * q + e > last) x[t][e] = -INFINITY;
                }
                float top = x[0][0];
#pragma unroll
                for (int t = 0; t < 8; ++t) top = max3(top, x[t][0], x[t][1]);
                const float ref = r.raise(top, q) - Rows::kLift;
                if (sc.y >= Rows::kLarge) r.less();
                uint32_t p[8];
                float sum = 0.f;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float p0 = tc_ex2(x[t][0] - ref), p1 = tc_ex2(x[t][1] - ref);
                    sum += p0 + p1;
                    p[t] = bits(__floats2half2_rn(p0, p1));   // off by 2^-11 of a term
                }
                r.l = fmaf(sum, r.unit, r.l);
                const float vs = sc.y * r.unit;
                base = wait_half();
                const uint32_t v0 = base + lane * kHeadDim;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {   // two sets of 16 channels at a time
                    float c[2][4] = {};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {   // 32 tokens each
                        uint4 v[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) v[e] = ldsm_t(v0 + half * 32 * kHeadDim + (((i + e) ^ (lane & 7)) << 4));
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t a0, a1, a2, a3;
                                pair_halves<FMT>(t ? v[e].z : v[e].x, a0, a1);
                                pair_halves<FMT>(t ? v[e].w : v[e].y, a2, a3);
                                mma<false>(c[e], a0, a1, a2, a3, p[4 * half + 2 * t], p[4 * half + 2 * t + 1]);
                            }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int g = 0; g < 4; ++g) r.o[i + e][g] = fmaf(c[e][g], vs, r.o[i + e][g]);
                }
                done_half();
            } else {
                // 32 bf16 rows of the open block
                const int t0 = nb * kBlk + (u - nb) * kOpenHalf;
                uint32_t base = wait_half();
                float x[4][2];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 k = lds128(base + blk_open_chunk(8 * t + n, 4 * q + i));
                        const uint4 y = row < R ? __ldg(qrow + i) : make_uint4(0, 0, 0, 0);
                        mma<true>(c, y.x, 0u, y.y, 0u, k.x, k.y);
                        mma<true>(c, y.z, 0u, y.w, 0u, k.z, k.w);
                    }
                    x[t][0] = c[0] * kLog2e;
                    x[t][1] = c[1] * kLog2e;
                }
                done_half();
                if (logits) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        *reinterpret_cast<float2 *>(logits + ((u - nb) * 4 + t) * R * 8) = make_float2(x[t][0], x[t][1]);
                }
                float top = -INFINITY;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (t0 + 8 * t + 2 * q + e > last) x[t][e] = -INFINITY;
                        top = fmaxf(top, x[t][e]);
                    }
                const float ref = r.raise(top, q) + Rows::kDrop;
                uint32_t p[4], pl[4];   // each probability as two bf16 parts
                float sum = 0.f;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float p0 = tc_ex2(x[t][0] - ref), p1 = tc_ex2(x[t][1] - ref);
                    sum += p0 + p1;
                    p[t] = pack_bf(p0, p1);
                    pl[t] = pack_bf(p0 - __uint_as_float(p[t] << 16), p1 - __uint_as_float(p[t] & 0xffff0000u));
                }
                r.l = fmaf(sum, r.of_rows(), r.l);
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
                    const float top_c = max3(fmaxf(fabsf(c[0]), fabsf(c[1])), fabsf(c[2]), fabsf(c[3]));
                    if (__any_sync(~0u, top_c >= Rows::kLarge)) r.less();
                    const float back = r.of_rows();
                    // c: channels n and 8 + n of the 16; the accumulators hold 2 n and 2 n + 1
                    const int s0 = ((2 * n) & 7) * 4 + q, s1 = s0 + 4;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float lo0 = __shfl_sync(~0u, c[e], s0), hi0 = __shfl_sync(~0u, c[2 + e], s0);
                        const float lo1 = __shfl_sync(~0u, c[e], s1), hi1 = __shfl_sync(~0u, c[2 + e], s1);
                        r.o[i][e] = fmaf(n < 4 ? lo0 : hi0, back, r.o[i][e]);
                        r.o[i][2 + e] = fmaf(n < 4 ? lo1 : hi1, back, r.o[i][2 + e]);
                    }
                }
                done_half();
            }
        }
        // the run's part of the pair: its result, or one of the parts that the joining kernel adds up (a run has at
        // most two: of the pair that it begins inside of, and of the one that it ends inside of)
        float *part = a.part + ((int64_t)run * 2 + (u0 == 0 ? 1 : 0)) * room * kRec;
        float l = r.l + __shfl_xor_sync(~0u, r.l, 1);
        l += __shfl_xor_sync(~0u, l, 2);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (q == 0 && row < R) {
            if (whole) {
                const float lse = row_lse(r.base(), l);
                if (a.lse) a.lse[((int64_t)b * D.Hq + h * D.G + row % D.G) * a.n_q + i_q] = lse * 0.6931471805599453f;
                if (a.weights) a.row_lse[pair * R + row] = lse;
            } else {
                *reinterpret_cast<float2 *>(part + row * kRec + kHeadDim) = make_float2(r.base(), l);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float f = __shfl_sync(~0u, inv, 8 * q + 4 * e);
            const int rr = 8 * group + 2 * q + e;
            if (rr >= R) continue;
            if (whole) {
                __nv_bfloat16 *o = a.out + (((int64_t)b * a.n_q + rr / D.G) * D.Hq + h * D.G + rr % D.G) * kHeadDim + 2 * n;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint32_t *>(o + 16 * i) = pack_bf(r.o[i][e] * f, r.o[i][2 + e] * f);
            } else {
                float *o = part + rr * kRec + 2 * n;
#pragma unroll
                for (int i = 0; i < 8; ++i) *reinterpret_cast<float2 *>(o + 16 * i) = make_float2(r.o[i][e], r.o[i][2 + e]);
            }
        }
        if (at < end) w.next(D, a.kv_len, u1 - u0);
    }
    if (!ok && lane == 0) blk_status(D, QEVICT_ERR_TIMEOUT, 0, blockIdx.x);
    // after a wait that ran out: copies still on their way are waited for before the CTA ends
    if (!ok && group == 0) {
        for (int i = 0; i < slots; ++i) {
            const int uses = cuse + (i < cslot ? 1 : 0);
            const long long t = clock64();
            while (uses > 0 && !tc_try_wait(full + 8 * (slot0 + i), (uses - 1) & 1) && clock64() - t < kDefaultWaitCycles) {
            }
        }
    }
}

// Behind the attention: the first CTAs turn the logits that it left into the tokens' weights, `tiles` CTAs to a pair, each
// an equal share of its blocks; then pairs x rows CTAs add up the parts of the pairs that lie in several runs, one row each.
__global__ void __launch_bounds__(kThreads, 4) block_join_kernel(const BlockDev D, const BlockAttendArgs a, int max_runs, int room, int tiles) {
    __shared__ float4 red4[kWarps][kRec / 4];
    float (*red)[kRec] = reinterpret_cast<float (*)[kRec]>(red4);
    __shared__ float lse[kMaxBlkQueries * kMaxG];   // of the pair's rows, log2 domain
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, R = a.n_q * D.G;
    const int64_t pairs = (int64_t)D.B * D.Hkv;
    const bool join = blockIdx.x >= pairs * tiles;
    const int64_t x = join ? blockIdx.x - pairs * tiles : blockIdx.x, pair = join ? x / R : x / tiles;
    const int b = (int)(pair / D.Hkv), h = (int)(pair % D.Hkv), len = blk_len(D, a.kv_len, b), n = units_of(len);
    int before;
    const int total = count_units(D, a.kv_len, b, &before);
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the attention kernel has ended
    const int runs = min(max_runs, total), first = before + h * n;
    // the runs that the pair lies in
    const int c0 = total ? (int)(((int64_t)(first + 1) * runs - 1) / total) : 0;
    const int c1 = total ? (int)(((int64_t)(first + n) * runs - 1) / total) : 0;
    auto part = [&](int c, int row) { return a.part + (((int64_t)c * 2 + (c == c0 ? 1 : 0)) * room + row) * kRec; };
    if (join) {
        const int row = (int)(x % R), i = row / D.G, head = h * D.G + row % D.G;
        __nv_bfloat16 *out = a.out + (((int64_t)b * a.n_q + i) * D.Hq + head) * kHeadDim;
        float *out_lse = a.lse ? a.lse + ((int64_t)b * D.Hq + head) * a.n_q + i : nullptr;
        if (len == 0) {
            if (tid < kHeadDim) out[tid] = __float2bfloat16_rn(0.f);
            if (tid == 0 && out_lse) *out_lse = -INFINITY;
            return;
        }
        if (c0 == c1) return;   // its run has written the result
        // warp w adds up the parts w, w + 8, ..., four at a time, relative to their running maximum
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0 + warp; c <= c1; c += 4 * kWarps) {
            float2 ml[4];
            float4 y[4];
            float top = m;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = c + e * kWarps <= c1;
                const float *p = part(in ? c + e * kWarps : c, row);
                ml[e] = *reinterpret_cast<const float2 *>(p + kHeadDim);
                y[e] = *(reinterpret_cast<const float4 *>(p) + lane);
                if (!in) ml[e].x = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, ml[e].x);
            const float ref = top == -INFINITY ? 0.f : top, f0 = tc_ex2(m - ref);
            m = top;
            l *= f0;
            o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (c + e * kWarps > c1) break;
                const float f = tc_ex2(ml[e].x - ref);   // 0 for a part whose keys the row does not see
                l = fmaf(ml[e].y, f, l);
                o.x = fmaf(y[e].x, f, o.x);
                o.y = fmaf(y[e].y, f, o.y);
                o.z = fmaf(y[e].z, f, o.z);
                o.w = fmaf(y[e].w, f, o.w);
            }
        }
        red4[warp][lane] = o;
        if (lane == 0) {
            red[warp][kHeadDim] = m;
            red[warp][kHeadDim + 1] = l;
        }
        __syncthreads();
        if (tid >= kHeadDim) return;
        m = red[0][kHeadDim];
        for (int e = 1; e < kWarps; ++e) m = fmaxf(m, red[e][kHeadDim]);
        const float ref = m == -INFINITY ? 0.f : m;
        l = 0.f;
        float s = 0.f;
        for (int e = 0; e < kWarps; ++e) {
            const float f = tc_ex2(red[e][kHeadDim] - ref);
            l = fmaf(red[e][kHeadDim + 1], f, l);
            s = fmaf(red[e][tid], f, s);
        }
        out[tid] = __float2bfloat16_rn(l == 0.f ? 0.f : s * (1.f / l));
        if (tid == 0 && out_lse) *out_lse = row_lse(m, l) * 0.6931471805599453f;
        return;
    }
    constexpr int kEach = kThreads / 16;   // blocks at a time
    const int blocks = (len + kBlk - 1) / kBlk, even = (blocks + tiles - 1) / tiles;
    const int share = even <= kEach ? kEach : (even + 2 * kEach - 1) / (2 * kEach) * (2 * kEach);   // two at a time below
    const int j0 = (int)(x % tiles) * share, j1 = min(j0 + share, blocks);
    if (j0 >= blocks) return;
    // their log-sum-exps: half a warp to a row, a pass over its parts with a running maximum
    for (int row = tid >> 4; row < ((R + 1) & ~1); row += kThreads / 16) {   // both halves of a warp go round alike
        float m = -INFINITY, l = 0.f;
        if (c0 != c1 && row < R)
#pragma unroll 2
            for (int c = c0 + (tid & 15); c <= c1; c += 16) {
                const float2 ml = *reinterpret_cast<const float2 *>(part(c, row) + kHeadDim);
                const float top = fmaxf(m, ml.x), ref = top == -INFINITY ? 0.f : top;
                l = fmaf(ml.y, tc_ex2(ml.x - ref), l * tc_ex2(m - ref));
                m = top;
            }
        __syncwarp();
#pragma unroll
        for (int s = 8; s; s >>= 1) {
            const float m2 = __shfl_xor_sync(~0u, m, s), l2 = __shfl_xor_sync(~0u, l, s);
            const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.f : top;
            l = fmaf(l2, tc_ex2(m2 - ref), l * tc_ex2(m - ref));
            m = top;
        }
        if ((tid & 15) == 0 && row < R) lse[row] = c0 == c1 ? a.row_lse[pair * R + row] : row_lse(m, l);
    }
    __syncthreads();
    // four tokens of each of two blocks to a thread at a time, eight loads on their way
    const int t = 4 * (tid & 15);
    const float inv = 1.f / D.G;
    for (int j = j0 + (tid >> 4); j < j1; j += 2 * kEach) {
        const int pos[2] = {j * kBlk + t, j + kEach < j1 ? (j + kEach) * kBlk + t : len};
        if (pos[0] >= len) return;
        const float4 *g = reinterpret_cast<const float4 *>(a.logits + (pair * D.NB + j) * R * kBlk + (t >> 3) * R * 8 + (t & 7));
        float w[2][4] = {};
        for (int r0 = 0; r0 < R; r0 += 4) {
            float4 y[2][4];
#pragma unroll
            for (int b2 = 0; b2 < 2; ++b2)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r0 + i < R && pos[b2] < len) y[b2][i] = __ldcs(g + b2 * kEach * R * (kBlk / 4) + (r0 + i) * 2);
#pragma unroll
            for (int b2 = 0; b2 < 2; ++b2)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (r0 + i >= R || pos[b2] >= len) continue;
                    const float z[4] = {y[b2][i].x, y[b2][i].y, y[b2][i].z, y[b2][i].w}, ref = lse[r0 + i];
                    const int last = len - a.n_q + (r0 + i) / D.G;
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[b2][e] += pos[b2] + e <= last ? tc_ex2(z[e] - ref) : 0.f;
                }
        }
#pragma unroll
        for (int b2 = 0; b2 < 2; ++b2) {
            if (pos[b2] >= len) continue;
            float *o = a.weights + pair * D.capacity + pos[b2];
            if (pos[b2] + 4 <= len && !(reinterpret_cast<uintptr_t>(o) & 15)) {
                float4 *o4 = reinterpret_cast<float4 *>(o);
                const float4 y = a.accumulate ? *o4 : make_float4(0.f, 0.f, 0.f, 0.f);
                *o4 = make_float4(fmaf(w[b2][0], inv, y.x), fmaf(w[b2][1], inv, y.y), fmaf(w[b2][2], inv, y.z),
                                  fmaf(w[b2][3], inv, y.w));
            } else {
                for (int e = 0; e < 4; ++e)
                    if (pos[b2] + e < len) o[e] = fmaf(w[b2][e], inv, a.accumulate ? o[e] : 0.f);
            }
        }
    }
}

}  // namespace

// Warps of a CTA: 8 for up to 8 rows (the memory bounds them; 128 KiB are on their way either way). More rows share a
// ring, a warp for every 8, and there arithmetic bounds: 12 warps, what the registers allow (5 queries of 4 x 8K 41 us,
// 43.5 with 8 warps of 16 rows, which share the codes' way to fp16, 43 with 16 warps). Rows that do not divide 12 warps
// leave some idle: 33 to 40 rows two, 49 to 56 five, 57 to 64 four (4 x 8K with 64 rows 44 us, with weights 69).
constexpr int kFewWarps = 8, kManyWarps = 12;

int64_t blk_part_floats(int G, int num_sms) {
    // runs x rows of a part: a ring's runs times its warps' rows, at most 8 rows to a warp
    const int rows = kMaxBlkQueries * G > 8 ? 8 * kManyWarps : 8 * kFewWarps;
    return (int64_t)num_sms * 2 * rows * kRec;
}

template <int FMT, int WARPS>
static cudaError_t launch_attend(const BlockDev &D, const BlockAttendArgs &a, int grid, int groups, cudaStream_t s) {
    cudaError_t e = once_per_device(0, [&] {
        return cudaFuncSetAttribute(block_attend_kernel<FMT, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    block_attend_kernel<FMT, WARPS><<<grid, 32 * WARPS, kSmemBytes, s>>>(D, a, groups);
    return cudaGetLastError();
}

cudaError_t launch_block_attend(const BlockDev &D, int fmt, const BlockAttendArgs &a, int num_sms, cudaStream_t s) {
    const int R = a.n_q * D.G, groups = (R + 7) / 8, warps = groups == 1 ? kFewWarps : kManyWarps;
    constexpr int I = QEVICT_BLOCK_INT8, E = QEVICT_BLOCK_E4M3, F = kFewWarps, M = kManyWarps;
    const cudaError_t e = fmt == I ? (groups == 1 ? launch_attend<I, F>(D, a, num_sms, groups, s) : launch_attend<I, M>(D, a, num_sms, groups, s))
                                   : (groups == 1 ? launch_attend<E, F>(D, a, num_sms, groups, s) : launch_attend<E, M>(D, a, num_sms, groups, s));
    if (e != cudaSuccess) return e;
    // CTAs that write weights: about four to an SM whatever the capacity, none for fewer than 16 blocks
    const int64_t pairs = (int64_t)D.B * D.Hkv, many = (4 * (int64_t)num_sms + pairs - 1) / pairs, most = (D.NB + 15) / 16;
    const int tiles = a.weights ? (int)(many < most ? many : most) : 0;
    const int64_t ctas = pairs * R + pairs * tiles;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    // its launch overlaps the attention; it waits for that kernel's end before it reads what it left
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, block_join_kernel, D, a, num_sms * (warps / groups), 8 * groups, tiles);
}

}  // namespace qevict
