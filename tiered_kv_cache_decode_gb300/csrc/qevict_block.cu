// The cache in 8 bits: tokens in, tokens out, and eviction by accumulated weight.
//
// A block of 64 tokens of one KV head holds its keys as codes c with one scale s, its
// values likewise: x ~ c s, s = max |x| / Q (Q = 127 for int8, 448 for e4m3), c = x / s
// rounded to the nearest code. A block is quantised once, when its last token comes; until
// then its rows are bf16 in one of two slots that the blocks take in turn. The rows of the
// last full block stay in the other slot, so a sequence can be set back by up to a block
// (drafted tokens that are rejected) and go on exactly.
#include "qevict_block.cuh"
#include "qevict_tc.cuh"

namespace qevict {
namespace {

constexpr int kThreads = 256;   // 16 lanes to a token's row, 8 channels each; 16 rows at a time, 4 times

__device__ __forceinline__ uint32_t amax2(uint32_t m, const uint4 &x) {
    m = __vmaxu2(m, x.x & 0x7fff7fffu);
    m = __vmaxu2(m, x.y & 0x7fff7fffu);
    m = __vmaxu2(m, x.z & 0x7fff7fffu);
    return __vmaxu2(m, x.w & 0x7fff7fffu);
}
// non-finite bf16 become 0
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}
__device__ __forceinline__ uint4 finite8(const uint4 &x) {
    return make_uint4(finite2(x.x), finite2(x.y), finite2(x.z), finite2(x.w));
}
__device__ __forceinline__ void unpack8(const uint4 &x, uint64_t *y) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
// The largest word over the CTA, a non-negative fp32 number's bits, and the scale that follows from it, which the first
// warp computes for all. A call begins behind what the CTA's threads have read before.
struct ScaleRoom {
    uint32_t m[kThreads / 32], top;
    BlockScale q;
};
template <int FMT>
__device__ __forceinline__ uint32_t cta_scale(uint32_t m, ScaleRoom &sm, BlockScale &q) {
    m = __reduce_max_sync(~0u, m);
    if ((threadIdx.x & 31) == 0) sm.m[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = __reduce_max_sync(~0u, threadIdx.x < kThreads / 32 ? sm.m[threadIdx.x] : 0u);
        if (threadIdx.x == 0) {
            sm.top = m;
            sm.q = blk_scale<FMT>(__uint_as_float(m));
        }
    }
    __syncthreads();
    q = sm.q;
    return sm.top;
}
// what a CTA works on: the keys (0) or values (1) of block number j of KV head h of sequence b. Neighbouring CTAs have
// the heads of a block, so that they read whole tokens between them.
struct Place {
    int kv, h, j, b;
    int64_t pair;
    __device__ __forceinline__ explicit Place(const BlockDev &D)
        : kv(blockIdx.x & 1), h(blockIdx.x >> 1), j(blockIdx.y), b(blockIdx.z), pair((int64_t)b * D.Hkv + h) {}
};
inline dim3 places(const BlockDev &D, int blocks) { return dim3(2u * D.Hkv, (unsigned)blocks, (unsigned)D.B); }

// One CTA takes the keys or the values of one block of one (sequence, KV head). Thread: channels 8 c .. 8 c + 7 of rows
// r + 16 i. Memory-bound: every row is read once and its codes written once (keys and values in CTAs of their own, six
// to an SM; with both in one CTA 53 us). A 32K prompt of 8 KV heads takes 34 us, 5.9 TB/s.
template <int FMT>
__global__ void __launch_bounds__(kThreads) block_append_kernel(const BlockDev D, const BlockAppendArgs a) {
    __shared__ ScaleRoom sm;
    const Place x(D);
    const int b = x.b, tid = threadIdx.x, c = tid & 15, r = tid >> 4;
    const bool speaks = x.j == 0 && x.h == 0 && x.kv == 0 && tid == 0;
    const int s = a.start ? a.start[b] : 0;
    const int m = a.n_new ? min(max(a.n_new[b], 0), a.n) : a.n;
    if (m == 0) return;
    if (s < 0) {
        if (speaks) blk_status(D, QEVICT_ERR_INVALID_ARG, b, s);
        return;
    }
    if ((int64_t)s + m > D.capacity && speaks) blk_status(D, QEVICT_ERR_CAPACITY, b, s);
    const int e = (int)min((int64_t)s + m, (int64_t)D.capacity);
    const int jb = (s >> 6) + x.j;
    if (e <= s || jb * kBlk >= e) return;
    const int64_t stride = x.kv ? a.v_stride : a.k_stride;
    const __nv_bfloat16 *in = (x.kv ? a.v : a.k) + (int64_t)b * a.n * stride + x.h * kHeadDim + 8 * c;
    const int half = x.kv * (kBlkBytes / 2), p0 = jb * kBlk + r;
    if (a.weights && x.kv == 0 && tid < kBlk) {
        const int pos = jb * kBlk + tid;
        if (pos >= s && pos < e) a.weights[x.pair * D.capacity + pos] = 0.f;
    }
    const bool full = (jb + 1) * kBlk <= e;
    uint4 y[4];
    const __nv_bfloat16 *at = in + (int64_t)(p0 - s) * stride;   // row r's; where the block begins before the tokens, not read
    if (jb * kBlk >= s && full) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __ldcs(reinterpret_cast<const uint4 *>(at + 16 * i * stride));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = r + 16 * i, pos = p0 + 16 * i;
            y[i] = make_uint4(0, 0, 0, 0);
            if (pos >= s && pos < e) y[i] = __ldcs(reinterpret_cast<const uint4 *>(at + 16 * i * stride));
            else if (pos < s && full)
                y[i] = *reinterpret_cast<const uint4 *>(D.open + blk_open_off(x.pair, jb, t) + half + blk_open_chunk(t, c));
        }
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = amax2(top, y[i]);
    BlockScale q;
    const uint32_t amax = cta_scale<FMT>(max(top & 0xffffu, top >> 16) << 16, sm, q);   // all rows of the slot are read by now
    if (amax >= 0x7f800000u) {
        if (tid == 0) blk_status(D, QEVICT_ERR_DEVICE, b, jb);
        top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = finite8(y[i]);
            top = amax2(top, y[i]);
        }
        __syncthreads();
        cta_scale<FMT>(max(top & 0xffffu, top >> 16) << 16, sm, q);
    }
    if (full) {
        if (tid == 0) reinterpret_cast<float *>(D.scale + x.pair * D.NB + jb)[x.kv] = q.s;
        uint8_t *o = D.codes + blk_code_off(D, x.pair, jb) + half + 8 * (c & 1) + blk_chunk(r, c >> 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // rows 16 apart have their chunks at the same places
            uint64_t z[4];
            unpack8(y[i], z);
            *reinterpret_cast<uint2 *>(o + 16 * i * kHeadDim) = blk_codes<FMT>(z, q);
        }
    }
    // The new rows of the last full block and of the open one, into their slots. Where the
    // first block's CTA has read rows from a slot, it writes both itself, behind its reads.
    const int last = (e >> 6) - 1;
    const bool alone = (s & (kBlk - 1)) != 0;
    if (jb >= last && (x.j == 0 || !alone)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = r + 16 * i, pos = jb * kBlk + t;
            if (pos >= s && pos < e)
                *reinterpret_cast<uint4 *>(D.open + blk_open_off(x.pair, jb, t) + half + blk_open_chunk(t, c)) = y[i];
        }
    }
    if (x.j == 0 && alone) {
        for (int j = max(last, jb + 1); j * kBlk < e; ++j)
            for (int t = r; t < kBlk && j * kBlk + t < e; t += 16)
                *reinterpret_cast<uint4 *>(D.open + blk_open_off(x.pair, j, t) + half + blk_open_chunk(t, c)) =
                    finite8(*reinterpret_cast<const uint4 *>(in + (int64_t)(j * kBlk + t - s) * stride));
    }
}

// One CTA: the keys or the values that lie in one block of one (sequence, KV head). 32K tokens of 8 KV heads: 29 us, 6.8 TB/s.
template <int FMT>
__global__ void __launch_bounds__(kThreads) block_read_kernel(const BlockDev D, const BlockReadArgs a) {
    const Place x(D);
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
    const int len = blk_len(D, a.kv_len, x.b);
    const int64_t first = a.first ? a.first[x.b] : 0;
    const int64_t jb = max(first >> 6, (int64_t)0) + x.j;
    if (jb * kBlk >= len) return;
    const bool full = (jb + 1) * kBlk <= len;
    const int half = x.kv * (kBlkBytes / 2);
    const float s = full ? reinterpret_cast<const float *>(D.scale + x.pair * D.NB + jb)[x.kv] : 0.f;
    const uint8_t *in = D.codes + blk_code_off(D, x.pair, (int)jb) + half + 8 * (c & 1);
    __nv_bfloat16 *out = (x.kv ? a.v : a.k) + ((int64_t)x.b * a.n * D.Hkv + x.h) * kHeadDim + 8 * c;
    uint4 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = r + 16 * i;
        if (full) {
            const uint2 code = *reinterpret_cast<const uint2 *>(in + blk_chunk(t, c >> 1));
            y[i].x = code.x;
            y[i].y = code.y;
        } else {
            y[i] = *reinterpret_cast<const uint4 *>(D.open + blk_open_off(x.pair, (int)jb, t) + half + blk_open_chunk(t, c));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t pos = jb * kBlk + r + 16 * i, row = pos - first;
        if (row < 0 || row >= a.n || pos >= len) continue;
        if (full) {
            uint64_t z[4];
            blk_values<FMT>(make_uint2(y[i].x, y[i].y), s, z);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = f2_unpack(z[j]);
                const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
                w[j] = *reinterpret_cast<const uint32_t *>(&p);
            }
            y[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *reinterpret_cast<uint4 *>(out + row * D.Hkv * kHeadDim) = y[i];
    }
}

// ---- eviction ---------------------------------------------------------------
constexpr int kMoveCtas = 8;                // CTAs (a cluster) that move a pair's tokens in place
constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kSelCtas = 8;                 // CTAs (a cluster) that rank a pair's tokens, at most
constexpr int kSelTokens = 8192;            // tokens for which one more CTA is taken
constexpr int kSelBins = 2048, kSelReps = 4;   // copies of a CTA's histogram, against lanes that meet in a bin
constexpr int kSelKeys = 40960;             // keys of a CTA that are kept in shared memory, at most
constexpr int kSelFixed = (kSelReps + 2) * kSelBins * 4;   // bytes of shared memory before the keys

// a weight as an integer of the same order; NaN last, -0 as 0
__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0;
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// One cluster per (sequence, KV head): the `want`-th largest key of the candidates by passes over eleven, eleven and ten
// bits, the CTAs' histograms added in distributed shared memory; then each warp counts its run's keys above it and equal to
// it, and with the counts of all warps before it gives every kept token its rank. Bound by latency: one read of the weights
// (then kept in shared memory: CACHED), three passes of one cluster barrier each, one more for the counts. Caches with
// room for 8K tokens take a cluster of one CTA, whose barrier is the CTA's own, those with room for more up to eight; keys
// are kept where a CTA's share of the room fits (40,960). The capacity decides both, whatever the lengths. 2K tokens 7 us, 32 pairs of 32K 15, 8 of 128K 19.
template <bool CACHED>
__global__ void __launch_bounds__(kSelThreads) block_select_kernel(const BlockDev D, const BlockEvictArgs a, int ctas) {
    extern __shared__ __align__(16) uint32_t sel[];
    uint32_t *rep = sel, *hists = rep + kSelReps * kSelBins, *keys = hists + 2 * kSelBins;   // keys: CACHED, this CTA's
    __shared__ uint2 coarse[2][kSelBins / 64];   // sums of 32 bins, two at a time
    __shared__ uint2 count[kSelWarps];
    __shared__ uint32_t found[2];
    const int64_t pair = blockIdx.x / ctas;
    const int rank = blockIdx.x % ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = (int)(pair / D.Hkv);
    const int len = blk_len(D, a.kv_len, b), c = len & ~(kBlk - 1);
    int32_t *kept = a.kept + pair * a.keep;
    if (c <= a.keep) {   // nothing leaves
        for (int i = rank * kSelThreads + tid; i < a.keep; i += ctas * kSelThreads) kept[i] = i < c ? i : -1;
        return;
    }
    const float *w = a.weights + pair * D.capacity;
    const int cand = c - a.recent;
    // a run of tokens to each warp, in order, four at a time to a lane (c is a multiple of 64)
    const int run = ((c + ctas * kSelWarps - 1) / (ctas * kSelWarps) + 127) & ~127;
    const int lo = rank * kSelWarps * run, hi = min(lo + kSelWarps * run, c);
    auto load4 = [&](int i) {   // the recent tokens' keys are above all
        const float4 x = __ldg(reinterpret_cast<const float4 *>(w + i));
        return make_uint4(i < cand ? weight_key(x.x) : ~0u, i + 1 < cand ? weight_key(x.y) : ~0u,
                          i + 2 < cand ? weight_key(x.z) : ~0u, i + 3 < cand ? weight_key(x.w) : ~0u);
    };
    if (CACHED)
#pragma unroll 4
        for (int i = lo + 4 * tid; i < hi; i += 4 * kSelThreads) *reinterpret_cast<uint4 *>(keys + i - lo) = load4(i);
    auto keys4 = [&](int i) { return CACHED ? *reinterpret_cast<const uint4 *>(keys + i - lo) : load4(i); };
    uint32_t want = a.keep - a.recent;   // of the candidates
    uint32_t prefix = 0;
    if (want == 0) prefix = ~0u - 1;   // the recent ones' keys alone are above it, and none is equal to it
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        if (a.keep == a.recent) break;
        const int bits = pass < 2 ? 11 : 10, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        uint32_t *hist = hists + (pass & 1) * kSelBins;
        for (int i = tid; i < kSelReps * kSelBins / 4; i += kSelThreads)
            reinterpret_cast<uint4 *>(rep)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        for (int i = lo + 4 * tid; i < hi; i += 4 * kSelThreads) {
            const uint4 k4 = keys4(i);
            const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k[j] != ~0u && (pass == 0 || (k[j] >> (shift + bits)) == prefix))
                    atomicAdd(&rep[((k[j] >> shift) & ((1u << bits) - 1)) * kSelReps + lane % kSelReps], 1u);
        }
        __syncthreads();
        uint32_t *sums = reinterpret_cast<uint32_t *>(coarse[pass & 1]);
#pragma unroll
        for (int i = tid; i < kSelBins; i += kSelThreads) {
            const uint4 x = reinterpret_cast<const uint4 *>(rep)[i];
            const uint32_t n = x.x + x.y + x.z + x.w, sum = __reduce_add_sync(~0u, n);
            hist[i] = n;
            if (lane == 0) sums[i / 32] = sum;
        }
        __syncwarp();
        cl_sync();
        if (warp == 0) {
            // the 32 bins, from the top, in which the wanted key lies, then the bin: both from all CTAs' counts
            uint32_t n0 = 0, n1 = 0;   // coarse bins 2 lane and 2 lane + 1
#pragma unroll
            for (int i = 0; i < kSelCtas; ++i) {
                if (i >= ctas) continue;
                const uint2 x = cl_pair(&coarse[pass & 1][lane], i);
                n0 += x.x;
                n1 += x.y;
            }
            auto from_here = [&](uint32_t n) {   // sum over this lane and those behind it
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const uint32_t x = __shfl_down_sync(~0u, n, s);
                    if (lane + s < 32) n += x;
                }
                return n;
            };
            uint32_t above = from_here(n0 + n1) - n0 - n1;
            bool upper = above + n1 >= want;
            uint32_t rest = want - above - (upper ? 0 : n1);
            const int l = 31 - __clz(__ballot_sync(~0u, above < want && above + n0 + n1 >= want));
            const int group = __shfl_sync(~0u, 2 * lane + (upper ? 1 : 0), l);
            rest = __shfl_sync(~0u, rest, l);
            uint32_t n = 0;
#pragma unroll
            for (int i = 0; i < kSelCtas; ++i)
                if (i < ctas) n += (uint32_t)cl_ldi(cl_addr(smem_u32(hist + 32 * group + lane), i));
            above = from_here(n) - n;
            if (above < rest && above + n >= rest) {
                found[0] = 32 * group + lane;
                found[1] = rest - above;
            }
        }
        __syncthreads();
        prefix = prefix << bits | found[0];
        want = found[1];
    }
    __syncthreads();   // the keys, where no pass has met
    const int wlo = min(lo + warp * run, hi), whi = min(wlo + run, hi);
    uint32_t above = 0, equal = 0;
    for (int i = wlo + 4 * lane; i < whi; i += 128) {
        const uint4 k = keys4(i);
        above += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
        equal += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
    }
    above = __reduce_add_sync(~0u, above);
    equal = __reduce_add_sync(~0u, equal);
    if (lane == 0) count[warp] = make_uint2(above, equal);
    __syncwarp();
    cl_sync();
    above = equal = 0;
#pragma unroll
    for (int i = 0; i < kSelCtas; ++i) {   // of the warps before this one
        if (i > rank || (i == rank && lane >= warp)) continue;
        const uint2 x = cl_pair(&count[lane], i);
        above += x.x;
        equal += x.y;
    }
    above = __reduce_add_sync(~0u, above);
    equal = __reduce_add_sync(~0u, equal);
    for (int i0 = wlo; i0 < whi; i0 += 128) {
        const int i = i0 + 4 * lane;
        const uint4 k4 = i < whi ? keys4(i) : make_uint4(0, 0, 0, 0);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w}, lower = (1u << lane) - 1;
        uint32_t up = above, eq = equal;   // of the tokens before this lane's
        bool is_up[4], is_eq[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            is_up[j] = i < whi && k[j] > prefix;
            is_eq[j] = i < whi && k[j] == prefix;
            const uint32_t mu = __ballot_sync(~0u, is_up[j]), me = __ballot_sync(~0u, is_eq[j]);
            up += __popc(mu & lower);
            eq += __popc(me & lower);
            above += __popc(mu);
            equal += __popc(me);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (is_up[j] || (is_eq[j] && eq < want)) kept[up + min(eq, want)] = i + j;
            up += is_up[j];
            eq += is_eq[j];
        }
    }
    __syncwarp();
    cl_sync();   // no CTA leaves while others read its counts
}

// What a thread holds of a block's keys or values on their way: 16 channels (a chunk) of rows r and r + 32
struct Moved {
    uint4 code[2];
    float s[2];
    float w;   // threads 0 .. 63: the weight of row tid
};

__device__ __forceinline__ void load_moved(const BlockDev &D, int64_t pair, int kv, const int32_t *kept, int block, int c_len,
                                           const float *w, Moved &m) {
    const int tid = threadIdx.x, c = tid & 7;
    const uint8_t *in = D.codes + blk_code_off(D, pair, 0) + kv * (kBlkBytes / 2);
    const float *scale = reinterpret_cast<const float *>(D.scale + pair * D.NB) + kv;
    kept += block * kBlk;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int x = min(max(kept[(tid >> 3) + 32 * i], 0), c_len - 1);
        m.code[i] = *reinterpret_cast<const uint4 *>(in + (int64_t)(x >> 6) * kBlkBytes + blk_chunk(x & (kBlk - 1), c));
        m.s[i] = scale[2 * (x >> 6)];
    }
    m.w = w && tid < kBlk ? w[min(max(kept[tid], 0), c_len - 1)] : 0.f;
}

template <int FMT>
__device__ __forceinline__ void store_moved(const BlockDev &D, int64_t pair, int kv, int block, const Moved &m, float *w_out,
                                            ScaleRoom &sm) {
    const int tid = threadIdx.x;
    uint64_t x[2][8];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        blk_values<FMT>(make_uint2(m.code[i].x, m.code[i].y), m.s[i], x[i]);
        blk_values<FMT>(make_uint2(m.code[i].z, m.code[i].w), m.s[i], x[i] + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = f2_unpack(x[i][j]);
            top = max3(top, fabsf(f.x), fabsf(f.y));
        }
    }
    BlockScale q;
    cta_scale<FMT>(__float_as_uint(top), sm, q);
    if (tid == 0) reinterpret_cast<float *>(D.scale + pair * D.NB + block)[kv] = q.s;
    if (w_out && tid < kBlk) w_out[block * kBlk + tid] = m.w;
    uint8_t *o = D.codes + blk_code_off(D, pair, block) + kv * (kBlkBytes / 2) + blk_chunk(tid >> 3, tid & 7);
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // rows 32 apart have their chunks at the same places
        const uint2 lo = blk_codes<FMT>(x[i], q), hi = blk_codes<FMT>(x[i] + 4, q);
        *reinterpret_cast<uint4 *>(o + 32 * i * kHeadDim) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
}

// The open block's rows and weights, and the new length. Its slot follows its new place.
__device__ __forceinline__ void move_open(const BlockDev &D, const BlockDev &to, const BlockEvictArgs &a, int64_t pair,
                                          int len, int c, int kept) {
    const int tid = threadIdx.x, from = c >> 6, dst = kept >> 6;
    if (pair % D.Hkv == 0 && tid == 0) a.new_len[pair / D.Hkv] = kept + len - c;
    if (a.weights_out && tid < len - c)
        a.weights_out[pair * to.capacity + kept + tid] = a.weights[pair * D.capacity + c + tid];
    const uint4 *in = reinterpret_cast<const uint4 *>(D.open + blk_open_off(pair, from, 0));
    uint4 *out = reinterpret_cast<uint4 *>(to.open + blk_open_off(pair, dst, 0));
    if (in != out && len > c)
        for (int i = tid; i < 2 * kBlkBytes / 16; i += kThreads) out[i] = in[i];
}

// Into another cache: a CTA for the keys and one for the values of each new block, the last ones for the open block.
// 4 x 32K tokens of 8 KV heads to 6.5K: 28 us, 3.8 TB/s, bound by instructions (0.69 of the issue slots; 12.6 a code, of
// which the conversion takes 7 and a thread's fixed part, spread over 32 codes, the rest) and by the chain of a block:
// positions, codes, two barriers (with the next block's loads under it 35, a warp to a block 32 us).
template <int FMT>
__global__ void __launch_bounds__(kThreads, 6)
    block_move_kernel(const BlockDev D, const BlockDev to, const BlockEvictArgs a) {
    __shared__ ScaleRoom sm;
    const Place x(D);
    const int len = blk_len(D, a.kv_len, x.b), c = len & ~(kBlk - 1), kept = min(c, a.keep);
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the selection has ended
    if (x.j == gridDim.y - 1) {
        if (x.kv == 0) move_open(D, to, a, x.pair, len, c, kept);
    } else if (x.j * kBlk < kept) {
        const bool weights = a.weights_out && x.kv == 0;
        Moved m;
        load_moved(D, x.pair, x.kv, a.kept + x.pair * a.keep, x.j, c, weights ? a.weights + x.pair * D.capacity : nullptr, m);
        store_moved<FMT>(to, x.pair, x.kv, x.j, m, weights ? a.weights_out + x.pair * to.capacity : nullptr, sm);
    }
}

// In place: a cluster per (sequence, KV head), keys and values, goes over the new blocks in rounds of one per
// CTA. A token only ever moves towards the front, so what round n reads lies at or behind
// the blocks that it writes, and a barrier between a round's reads and its writes suffices. Bound by the chain of its
// rounds, 8 blocks each: whole evictions of 4 x 32K to 6.5K 56 us (into another cache 42), of 128K to 13K 74 (36).
template <int FMT>
__global__ void __cluster_dims__(kMoveCtas, 1, 1) __launch_bounds__(kThreads)
    block_compact_kernel(const BlockDev D, const BlockEvictArgs a) {
    __shared__ ScaleRoom sm;
    const int64_t pair = blockIdx.x / (2 * kMoveCtas);
    const int rank = blockIdx.x % kMoveCtas, kv = blockIdx.x / kMoveCtas & 1, b = (int)(pair / D.Hkv);
    const int len = blk_len(D, a.kv_len, b), c = len & ~(kBlk - 1), kept = min(c, a.keep);
    float *w = a.weights_out && kv == 0 ? a.weights_out + pair * D.capacity : nullptr;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the selection has ended
    if (c > kept) {
        for (int j0 = 0; j0 * kBlk < kept; j0 += kMoveCtas) {
            const int j = j0 + rank;
            Moved m;
            if (j * kBlk < kept)
                load_moved(D, pair, kv, a.kept + pair * a.keep, j, c, w ? a.weights + pair * D.capacity : nullptr, m);
            __syncwarp();
            cl_sync();   // also behind the last round's reads of `sm`
            if (j * kBlk < kept) store_moved<FMT>(D, pair, kv, j, m, w, sm);
        }
    }
    if (c <= kept && kv == 0 && a.weights_out && a.weights_out != a.weights)
        for (int i = rank * kThreads + threadIdx.x; i < c; i += kMoveCtas * kThreads)
            a.weights_out[pair * D.capacity + i] = a.weights[pair * D.capacity + i];
    // the last round's reads are behind a barrier: the open block's weights may go where they lay
    if (rank == 0 && kv == 0) move_open(D, D, a, pair, len, c, kept);
}

}  // namespace

#define BY_FORMAT(fmt, kernel) ((fmt) == QEVICT_BLOCK_INT8 ? kernel<QEVICT_BLOCK_INT8> : kernel<QEVICT_BLOCK_E4M3>)

cudaError_t launch_block_append(const BlockDev &D, int fmt, const BlockAppendArgs &a, cudaStream_t s) {
    const int blocks = a.n == 1 ? 1 : (a.n + kBlk - 2) / kBlk + 1;   // that n tokens can touch
    BY_FORMAT(fmt, block_append_kernel)<<<places(D, blocks), kThreads, 0, s>>>(D, a);
    return cudaGetLastError();
}

cudaError_t launch_block_read(const BlockDev &D, int fmt, const BlockReadArgs &a, cudaStream_t s) {
    BY_FORMAT(fmt, block_read_kernel)<<<places(D, min((a.n + kBlk - 2) / kBlk + 1, D.NB)), kThreads, 0, s>>>(D, a);
    return cudaGetLastError();
}

cudaError_t launch_block_evict(const BlockDev &D, const BlockDev &to, int fmt, const BlockEvictArgs &a,
                               cudaStream_t s) {
    const int64_t pairs = (int64_t)D.B * D.Hkv;
    // the selection's keys in shared memory where the longest run of tokens that the capacity allows fits
    int ctas = 1;
    while (ctas < kSelCtas && ctas * kSelTokens < D.capacity) ctas *= 2;
    const int run = ((D.capacity + ctas * kSelWarps - 1) / (ctas * kSelWarps) + 127) & ~127, keys = run * kSelWarps;
    const bool cached = keys <= kSelKeys;
    cudaError_t e = once_per_device(0, [&] {
        const cudaError_t r = cudaFuncSetAttribute(block_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kSelFixed + kSelKeys * 4);
        return r != cudaSuccess ? r : cudaFuncSetAttribute(block_select_kernel<false>,
                                                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSelFixed);
    });
    if (e != cudaSuccess) return e;
    {
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = ctas;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)(pairs * ctas));
        cfg.blockDim = dim3(kSelThreads);
        cfg.dynamicSmemBytes = kSelFixed + (cached ? keys * 4 : 0);
        cfg.stream = s;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, cached ? block_select_kernel<true> : block_select_kernel<false>, D, a, ctas);
        if (e != cudaSuccess) return e;
    }
    // the moving kernel's launch overlaps the selection, for whose end it waits
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (to.codes == D.codes) {
        cfg.gridDim = dim3((unsigned)(2 * pairs * kMoveCtas));
        return cudaLaunchKernelEx(&cfg, BY_FORMAT(fmt, block_compact_kernel), D, a);
    }
    cfg.gridDim = places(D, a.keep / kBlk + 1);
    return cudaLaunchKernelEx(&cfg, BY_FORMAT(fmt, block_move_kernel), D, to, a);
}

}  // namespace qevict
