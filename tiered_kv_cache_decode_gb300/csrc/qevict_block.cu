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
__device__ __forceinline__ void unpack8(const uint4 &x, float *y) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = __uint_as_float(w[i] << 16);
        y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// the largest of two words over the CTA; `sm` has room for 2 x 8, and a call ends with all threads past its reads
__device__ __forceinline__ uint2 cta_max(uint2 m, uint2 *sm) {
    m.x = __reduce_max_sync(~0u, m.x);
    m.y = __reduce_max_sync(~0u, m.y);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = m;
    __syncthreads();
    uint2 r = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        r.x = max(r.x, sm[i].x);
        r.y = max(r.y, sm[i].y);
    }
    __syncthreads();
    return r;
}

// One CTA takes one block of one (sequence, KV head): CTAs of the heads of a block are
// neighbours, so that they read whole tokens between them. Thread: channels 8 c .. 8 c + 7
// of rows r + 16 i.
template <int FMT>
__global__ void __launch_bounds__(kThreads) block_append_kernel(const BlockDev D, const BlockAppendArgs a, int nbx) {
    __shared__ uint2 sm[kThreads / 32];
    const int64_t u = blockIdx.x;
    const int h = (int)(u % D.Hkv), jx = (int)(u / D.Hkv % nbx), b = (int)(u / D.Hkv / nbx);
    const int64_t pair = (int64_t)b * D.Hkv + h;
    const int tid = threadIdx.x, c = tid & 15, r = tid >> 4;
    const int s = a.start ? a.start[b] : 0;
    const int m = a.n_new ? min(max(a.n_new[b], 0), a.n) : a.n;
    if (m == 0) return;
    if (s < 0) {
        if (jx == 0 && h == 0 && tid == 0) blk_status(D, QEVICT_ERR_INVALID_ARG, b, s);
        return;
    }
    if ((int64_t)s + m > D.capacity && jx == 0 && h == 0 && tid == 0)
        blk_status(D, QEVICT_ERR_CAPACITY, b, s);
    const int e = (int)min((int64_t)s + m, (int64_t)D.capacity);
    const int jb = (s >> 6) + jx;
    if (e <= s || jb * kBlk >= e) return;
    const __nv_bfloat16 *kin = a.k + (int64_t)b * a.n * a.k_stride + h * kHeadDim + 8 * c;
    const __nv_bfloat16 *vin = a.v + (int64_t)b * a.n * a.v_stride + h * kHeadDim + 8 * c;
    if (a.weights && tid < kBlk) {
        const int pos = jb * kBlk + tid;
        if (pos >= s && pos < e) a.weights[pair * D.capacity + pos] = 0.f;
    }
    const bool full = (jb + 1) * kBlk <= e;
    uint4 k[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = r + 16 * i, pos = jb * kBlk + t;
        k[i] = v[i] = make_uint4(0, 0, 0, 0);
        if (pos >= s && pos < e) {
            k[i] = *reinterpret_cast<const uint4 *>(kin + (pos - s) * a.k_stride);
            v[i] = *reinterpret_cast<const uint4 *>(vin + (pos - s) * a.v_stride);
        } else if (pos < s && full) {
            const uint8_t *o = D.open + blk_open_off(pair, jb, t) + blk_open_chunk(t, c);
            k[i] = *reinterpret_cast<const uint4 *>(o);
            v[i] = *reinterpret_cast<const uint4 *>(o + kBlkBytes / 2);
        }
    }
    uint2 top = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        top.x = amax2(top.x, k[i]);
        top.y = amax2(top.y, v[i]);
    }
    top.x = max(top.x & 0xffffu, top.x >> 16);
    top.y = max(top.y & 0xffffu, top.y >> 16);
    uint2 amax = cta_max(top, sm);   // all rows of the slot are read by now
    if (amax.x >= 0x7f80u || amax.y >= 0x7f80u) {
        if (tid == 0) blk_status(D, QEVICT_ERR_DEVICE, b, jb);
        top = make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k[i] = finite8(k[i]);
            v[i] = finite8(v[i]);
            top.x = amax2(top.x, k[i]);
            top.y = amax2(top.y, v[i]);
        }
        top.x = max(top.x & 0xffffu, top.x >> 16);
        top.y = max(top.y & 0xffffu, top.y >> 16);
        amax = cta_max(top, sm);
    }
    if (full) {
        const BlockScale qk = blk_scale<FMT>(__uint_as_float(amax.x << 16));
        const BlockScale qv = blk_scale<FMT>(__uint_as_float(amax.y << 16));
        if (tid == 0) D.scale[pair * D.NB + jb] = make_float2(qk.s, qv.s);
        uint8_t *o = D.codes + blk_code_off(D, pair, jb) + 8 * (c & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = r + 16 * i;
            float x[8];
            unpack8(k[i], x);
            *reinterpret_cast<uint2 *>(o + blk_chunk(t, c >> 1)) = blk_codes<FMT>(x, qk);
            unpack8(v[i], x);
            *reinterpret_cast<uint2 *>(o + kBlkBytes / 2 + blk_chunk(t, c >> 1)) = blk_codes<FMT>(x, qv);
        }
    }
    // The new rows of the last full block and of the open one, into their slots. Where the
    // first block's CTA has read rows from a slot, it writes both itself, behind its reads.
    const int last = (e >> 6) - 1;
    const bool alone = (s & (kBlk - 1)) != 0;
    if (jb >= last && (jx == 0 || !alone)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = r + 16 * i, pos = jb * kBlk + t;
            if (pos < s || pos >= e) continue;
            uint8_t *o = D.open + blk_open_off(pair, jb, t) + blk_open_chunk(t, c);
            *reinterpret_cast<uint4 *>(o) = k[i];
            *reinterpret_cast<uint4 *>(o + kBlkBytes / 2) = v[i];
        }
    }
    if (jx == 0 && alone) {
        for (int j = max(last, jb + 1); j * kBlk < e; ++j)
            for (int t = r; t < kBlk && j * kBlk + t < e; t += 16) {
                const int64_t i = j * kBlk + t - s;
                uint8_t *o = D.open + blk_open_off(pair, j, t) + blk_open_chunk(t, c);
                *reinterpret_cast<uint4 *>(o) = finite8(*reinterpret_cast<const uint4 *>(kin + i * a.k_stride));
                *reinterpret_cast<uint4 *>(o + kBlkBytes / 2) =
                    finite8(*reinterpret_cast<const uint4 *>(vin + i * a.v_stride));
            }
    }
}

// One CTA: the rows that lie in one block of one (sequence, KV head).
template <int FMT>
__global__ void __launch_bounds__(kThreads) block_read_kernel(const BlockDev D, const BlockReadArgs a, int nbx) {
    const int64_t u = blockIdx.x;
    const int h = (int)(u % D.Hkv), jx = (int)(u / D.Hkv % nbx), b = (int)(u / D.Hkv / nbx);
    const int64_t pair = (int64_t)b * D.Hkv + h;
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
    const int len = blk_len(D, a.kv_len, b);
    const int64_t first = a.first ? a.first[b] : 0;
    const int64_t jb = max(first >> 6, (int64_t)0) + jx;
    if (jb * kBlk >= len) return;
    const bool full = (jb + 1) * kBlk <= len;
    const float2 s = full ? D.scale[pair * D.NB + jb] : make_float2(0.f, 0.f);
    const uint8_t *in = D.codes + blk_code_off(D, pair, (int)jb) + 8 * (c & 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = r + 16 * i;
        const int64_t pos = jb * kBlk + t, row = pos - first;
        if (row < 0 || row >= a.n || pos >= len) continue;
        uint4 k, v;
        if (full) {
            float x[8];
            uint32_t w[4];
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint2 code = *reinterpret_cast<const uint2 *>(in + kv * (kBlkBytes / 2) + blk_chunk(t, c >> 1));
                blk_values<FMT>(code, kv ? s.y : s.x, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t *>(&p);
                }
                (kv ? v : k) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
            const uint8_t *o = D.open + blk_open_off(pair, (int)jb, t) + blk_open_chunk(t, c);
            k = *reinterpret_cast<const uint4 *>(o);
            v = *reinterpret_cast<const uint4 *>(o + kBlkBytes / 2);
        }
        const int64_t at = (((int64_t)b * a.n + row) * D.Hkv + h) * kHeadDim + 8 * c;
        *reinterpret_cast<uint4 *>(a.k + at) = k;
        *reinterpret_cast<uint4 *>(a.v + at) = v;
    }
}

// ---- eviction ---------------------------------------------------------------
constexpr int kSelCtas = 8;                           // CTAs (a cluster) that rank a pair's tokens
constexpr int kSelWarps = kSelCtas * kThreads / 32;   // each ranks a run of tokens of its own

// a weight as an integer of the same order; NaN last, -0 as 0
__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0;
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// One cluster per (sequence, KV head): the `want`-th largest key of the candidates by
// four passes over eight bits each, the CTAs' histograms added in distributed shared memory;
// then each warp counts its run's keys above it and equal to it, and with the counts of all
// warps before it gives every kept token its rank.
__global__ void __cluster_dims__(kSelCtas, 1, 1) __launch_bounds__(kThreads)
    block_select_kernel(const BlockDev D, const BlockEvictArgs a) {
    __shared__ uint32_t hist[2][256];
    __shared__ uint32_t sum[256], found[2];
    __shared__ uint2 count[kThreads / 32];
    const int64_t pair = blockIdx.x / kSelCtas;
    const int rank = blockIdx.x % kSelCtas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = (int)(pair / D.Hkv);
    const int len = blk_len(D, a.kv_len, b), c = len & ~(kBlk - 1);
    int32_t *kept = a.kept + pair * a.keep;
    if (c <= a.keep) {   // nothing leaves
        for (int i = rank * kThreads + tid; i < a.keep; i += kSelCtas * kThreads) kept[i] = i < c ? i : -1;
        return;
    }
    const float *w = a.weights + pair * D.capacity;
    const int cand = c - a.recent;
    uint32_t want = a.keep - a.recent;   // of the candidates
    uint32_t prefix = 0;
    if (want > 0) {
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            uint32_t *hs = hist[pass & 1];
            hs[tid] = 0;
            __syncthreads();
            for (int i = rank * kThreads + tid; i < cand; i += kSelCtas * kThreads) {
                const uint32_t key = weight_key(w[i]);
                if (pass == 0 || (key >> (shift + 8)) == prefix) atomicAdd(&hs[(key >> shift) & 255], 1u);
            }
            __syncwarp();
            cl_sync();
            uint32_t n = 0;
            for (int i = 0; i < kSelCtas; ++i)
                n += (uint32_t)cl_ldi(cl_addr(smem_u32(&hs[tid]), i));
            sum[tid] = n;
            __syncthreads();
            // the bin, from the top, in which the wanted key lies
            uint32_t above = 0;
            for (int i = tid + 1; i < 256; ++i) above += sum[i];
            if (above < want && above + n >= want) {
                found[0] = tid;
                found[1] = want - above;
            }
            __syncthreads();
            prefix = prefix << 8 | found[0];
            want = found[1];
        }
    } else {
        prefix = ~0u;   // no key is above it, and none of those equal to it is wanted
    }
    // runs of tokens, a warp each, in order
    const int run = ((c + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int lo = min((rank * (kThreads / 32) + warp) * run, c), hi = min(lo + run, c);
    uint32_t above = 0, equal = 0;
    for (int i = lo + lane; i < hi; i += 32) {
        const uint32_t key = i < cand ? weight_key(w[i]) : 0;
        if (i >= cand || key > prefix) ++above;
        else if (key == prefix) ++equal;
    }
    above = __reduce_add_sync(~0u, above);
    equal = __reduce_add_sync(~0u, equal);
    if (lane == 0) count[warp] = make_uint2(above, equal);
    __syncwarp();
    cl_sync();
    above = equal = 0;
    for (int i = lane; i < rank * (kThreads / 32) + warp; i += 32) {
        const uint32_t at = cl_addr(smem_u32(&count[i % (kThreads / 32)]), i / (kThreads / 32));
        above += (uint32_t)cl_ldi(at);
        equal += (uint32_t)cl_ldi(at + 4);
    }
    above = __reduce_add_sync(~0u, above);
    equal = __reduce_add_sync(~0u, equal);
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < cand ? weight_key(w[i]) : 0;
        const bool up = i < hi && (i >= cand || key > prefix), eq = i < hi && !up && key == prefix;
        const uint32_t mu = __ballot_sync(~0u, up), me = __ballot_sync(~0u, eq), below = (1u << lane) - 1;
        const uint32_t e = equal + __popc(me & below);
        if (up || (eq && e < want)) kept[above + __popc(mu & below) + min(e, want)] = i;
        above += __popc(mu);
        equal += __popc(me);
    }
    __syncwarp();
    cl_sync();   // no CTA leaves while others read its counts
}

// What a thread holds of a block on its way: channels 8 c .. + 7 of rows r + 16 i
struct Moved {
    uint2 k[4], v[4];
    float2 s[4];
    float w;   // threads 0 .. 63: the weight of row tid
};

__device__ __forceinline__ void load_moved(const BlockDev &D, int64_t pair, const int32_t *kept, int block, int c_len,
                                           const float *w, Moved &m) {
    const int tid = threadIdx.x, c = tid & 15, r = tid >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int idx = min(max(kept[block * kBlk + r + 16 * i], 0), c_len - 1), j = idx >> 6, t = idx & (kBlk - 1);
        const uint8_t *in = D.codes + blk_code_off(D, pair, j) + blk_chunk(t, c >> 1) + 8 * (c & 1);
        m.k[i] = *reinterpret_cast<const uint2 *>(in);
        m.v[i] = *reinterpret_cast<const uint2 *>(in + kBlkBytes / 2);
        m.s[i] = D.scale[pair * D.NB + j];
    }
    m.w = 0.f;
    if (w && tid < kBlk) m.w = w[min(max(kept[block * kBlk + tid], 0), c_len - 1)];
}

template <int FMT>
__device__ __forceinline__ void store_moved(const BlockDev &D, int64_t pair, int block, const Moved &m, float *w_out,
                                            uint2 *sm) {
    const int tid = threadIdx.x, c = tid & 15, r = tid >> 4;
    float x[8];
    uint2 top = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        blk_values<FMT>(m.k[i], m.s[i].x, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) top.x = max(top.x, __float_as_uint(fabsf(x[j])));
        blk_values<FMT>(m.v[i], m.s[i].y, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) top.y = max(top.y, __float_as_uint(fabsf(x[j])));
    }
    const uint2 amax = cta_max(top, sm);
    const BlockScale qk = blk_scale<FMT>(__uint_as_float(amax.x)), qv = blk_scale<FMT>(__uint_as_float(amax.y));
    if (tid == 0) D.scale[pair * D.NB + block] = make_float2(qk.s, qv.s);
    if (w_out && tid < kBlk) w_out[block * kBlk + tid] = m.w;
    uint8_t *o = D.codes + blk_code_off(D, pair, block) + 8 * (c & 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = r + 16 * i;
        blk_values<FMT>(m.k[i], m.s[i].x, x);
        *reinterpret_cast<uint2 *>(o + blk_chunk(t, c >> 1)) = blk_codes<FMT>(x, qk);
        blk_values<FMT>(m.v[i], m.s[i].y, x);
        *reinterpret_cast<uint2 *>(o + kBlkBytes / 2 + blk_chunk(t, c >> 1)) = blk_codes<FMT>(x, qv);
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

// Into another cache: one CTA per new block, the last one for the open block.
template <int FMT>
__global__ void __launch_bounds__(kThreads)
    block_move_kernel(const BlockDev D, const BlockDev to, const BlockEvictArgs a, int nbx) {
    __shared__ uint2 sm[kThreads / 32];
    const int64_t u = blockIdx.x;
    const int h = (int)(u % D.Hkv), j = (int)(u / D.Hkv % nbx), b = (int)(u / D.Hkv / nbx);
    const int64_t pair = (int64_t)b * D.Hkv + h;
    const int len = blk_len(D, a.kv_len, b), c = len & ~(kBlk - 1), kept = min(c, a.keep);
    if (j == nbx - 1) {
        move_open(D, to, a, pair, len, c, kept);
    } else if (j * kBlk < kept) {
        Moved m;
        load_moved(D, pair, a.kept + pair * a.keep, j, c, a.weights_out ? a.weights + pair * D.capacity : nullptr, m);
        store_moved<FMT>(to, pair, j, m, a.weights_out ? a.weights_out + pair * to.capacity : nullptr, sm);
    }
}

// In place: a cluster per (sequence, KV head) goes over the new blocks in rounds of one per
// CTA. A token only ever moves towards the front, so what round n reads lies at or behind
// the blocks that it writes, and a barrier between a round's reads and its writes suffices.
template <int FMT>
__global__ void __cluster_dims__(kSelCtas, 1, 1) __launch_bounds__(kThreads)
    block_compact_kernel(const BlockDev D, const BlockEvictArgs a) {
    __shared__ uint2 sm[kThreads / 32];
    const int64_t pair = blockIdx.x / kSelCtas;
    const int rank = blockIdx.x % kSelCtas, b = (int)(pair / D.Hkv);
    const int len = blk_len(D, a.kv_len, b), c = len & ~(kBlk - 1), kept = min(c, a.keep);
    float *w = a.weights_out ? a.weights_out + pair * D.capacity : nullptr;
    if (c > kept) {
        for (int j0 = 0; j0 * kBlk < kept; j0 += kSelCtas) {
            const int j = j0 + rank;
            Moved m;
            if (j * kBlk < kept) load_moved(D, pair, a.kept + pair * a.keep, j, c, w, m);
            __syncwarp();
            cl_sync();
            if (j * kBlk < kept) store_moved<FMT>(D, pair, j, m, w, sm);
        }
    }
    // the last round's reads are behind a barrier: the open block's weights may go where they lay
    if (rank == 0) move_open(D, D, a, pair, len, c, kept);
}

}  // namespace

#define BY_FORMAT(fmt, kernel) ((fmt) == QEVICT_BLOCK_INT8 ? kernel<QEVICT_BLOCK_INT8> : kernel<QEVICT_BLOCK_E4M3>)

cudaError_t launch_block_append(const BlockDev &D, int fmt, const BlockAppendArgs &a, cudaStream_t s) {
    const int nbx = a.n == 1 ? 1 : (a.n + kBlk - 2) / kBlk + 1;   // blocks that n tokens can touch
    const int64_t grid = (int64_t)D.B * D.Hkv * nbx;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    BY_FORMAT(fmt, block_append_kernel)<<<(unsigned)grid, kThreads, 0, s>>>(D, a, nbx);
    return cudaGetLastError();
}

cudaError_t launch_block_read(const BlockDev &D, int fmt, const BlockReadArgs &a, cudaStream_t s) {
    const int nbx = min((a.n + kBlk - 2) / kBlk + 1, D.NB);
    const int64_t grid = (int64_t)D.B * D.Hkv * nbx;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    BY_FORMAT(fmt, block_read_kernel)<<<(unsigned)grid, kThreads, 0, s>>>(D, a, nbx);
    return cudaGetLastError();
}

cudaError_t launch_block_evict(const BlockDev &D, const BlockDev &to, int fmt, const BlockEvictArgs &a,
                               cudaStream_t s) {
    const int64_t pairs = (int64_t)D.B * D.Hkv;
    const int nbx = a.keep / kBlk + 1;
    if (pairs * kSelCtas > 0x7fffffffll || pairs * nbx > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    block_select_kernel<<<(unsigned)(pairs * kSelCtas), kThreads, 0, s>>>(D, a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (to.codes == D.codes)
        BY_FORMAT(fmt, block_compact_kernel)<<<(unsigned)(pairs * kSelCtas), kThreads, 0, s>>>(D, a);
    else
        BY_FORMAT(fmt, block_move_kernel)<<<(unsigned)(pairs * nbx), kThreads, 0, s>>>(D, to, a, nbx);
    return cudaGetLastError();
}

}  // namespace qevict
