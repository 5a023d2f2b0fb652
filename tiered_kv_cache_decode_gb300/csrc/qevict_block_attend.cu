// Attention of the last positions over the cache in 8 bits.
//
// Query i of n_q sits at p = kv_len - n_q + i and sees the keys j <= p: softmax(q k / sqrt(d)) V, with
// k = code * s of its block, v likewise, and bf16 rows in the block that is not full. One pass over the keys:
// running maximum and sum per row, partial results of kParts parts of a (sequence, KV head) joined by a second
// kernel. The weight that a token receives is the sum over the queries and the mean over the query heads of its
// probabilities, from the logits that the first kernel leaves behind.
#include "qevict_block.cuh"
#include "qevict_tc.cuh"

namespace qevict {
namespace {

constexpr int kParts = 16;
constexpr int kRows = kMaxBlkQueries * kMaxG;
constexpr int kTile = 32;
constexpr int kRec = kHeadDim + 2;   // O, maximum, sum

template <int FMT>
__global__ void __launch_bounds__(128) block_attend_kernel(const BlockDev D, const BlockAttendArgs a) {
    extern __shared__ float sm[];
    float *q = sm, *o = q + kRows * kHeadDim, *k = o + kRows * kHeadDim, *v = k + kTile * (kHeadDim + 1),
          *x = v + kTile * kHeadDim, *st = x + kRows * kTile;   // st: [row] maximum, sum, factor
    const int64_t pair = blockIdx.x / kParts;
    const int part = blockIdx.x % kParts, b = (int)(pair / D.Hkv), h = (int)(pair % D.Hkv), tid = threadIdx.x;
    const int R = a.n_q * D.G, len = blk_len(D, a.kv_len, b), closed = len & ~(kBlk - 1);
    for (int i = tid; i < R * kHeadDim; i += 128) {
        const int r = i >> 7;
        q[i] = __bfloat162float(a.q[(((int64_t)b * a.n_q + r / D.G) * D.Hq + h * D.G + r % D.G) * kHeadDim + (i & 127)]);
        o[i] = 0.f;
    }
    if (tid < R) {
        st[tid] = -INFINITY;
        st[kRows + tid] = 0.f;
    }
    for (int t0 = part * kTile; t0 < len; t0 += kParts * kTile) {
        __syncthreads();
        for (int i = tid; i < kTile * 16; i += 128) {
            const int t = i >> 4, c = i & 15, pos = t0 + t;
            float kx[8] = {}, vx[8] = {};
            if (pos < closed) {
                const uint8_t *in = D.codes + blk_code_off(D, pair, pos >> 6) + blk_chunk(pos & 63, c >> 1) + 8 * (c & 1);
                const float2 s = D.scale[pair * D.NB + (pos >> 6)];
                blk_values<FMT>(*reinterpret_cast<const uint2 *>(in), s.x, kx);
                blk_values<FMT>(*reinterpret_cast<const uint2 *>(in + kBlkBytes / 2), s.y, vx);
            } else if (pos < len) {
                const uint8_t *in = D.open + blk_open_off(pair, pos >> 6, pos & 63) + blk_open_chunk(pos & 63, c);
                for (int e = 0; e < 8; ++e) {
                    kx[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(in)[e]);
                    vx[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(in + kBlkBytes / 2)[e]);
                }
            }
            for (int e = 0; e < 8; ++e) {
                k[t * (kHeadDim + 1) + 8 * c + e] = kx[e];
                v[t * kHeadDim + 8 * c + e] = vx[e];
            }
        }
        __syncthreads();
        for (int i = tid; i < R * kTile; i += 128) {
            const int r = i / kTile, t = i % kTile, pos = t0 + t;
            float s = 0.f;
            for (int e = 0; e < kHeadDim; ++e) s = fmaf(q[r * kHeadDim + e], k[t * (kHeadDim + 1) + e], s);
            x[i] = pos <= len - a.n_q + r / D.G ? s * (1.4426950408889634f * 0.08838834764831845f) : -INFINITY;
            if (a.weights) a.logits[((pair * D.NB + (pos >> 6)) * R + r) * kBlk + (pos & 63)] = x[i];
        }
        __syncthreads();
        if (tid < R) {
            float m = st[tid], l = 0.f;
            for (int t = 0; t < kTile; ++t) m = fmaxf(m, x[tid * kTile + t]);
            const float ref = m == -INFINITY ? 0.f : m, f = exp2f(st[tid] - ref);
            for (int t = 0; t < kTile; ++t) l += x[tid * kTile + t] = exp2f(x[tid * kTile + t] - ref);
            st[tid] = m;
            st[kRows + tid] = st[kRows + tid] * f + l;
            st[2 * kRows + tid] = f;
        }
        __syncthreads();
        for (int r = 0; r < R; ++r) {
            float s = o[r * kHeadDim + tid] * st[2 * kRows + r];
            for (int t = 0; t < kTile; ++t) s = fmaf(x[r * kTile + t], v[t * kHeadDim + tid], s);
            o[r * kHeadDim + tid] = s;
        }
    }
    __syncthreads();
    float *p = a.part + (int64_t)blockIdx.x * kRows * kRec;
    for (int r = 0; r < R; ++r) p[r * kRec + tid] = o[r * kHeadDim + tid];
    if (tid < R) {
        p[tid * kRec + kHeadDim] = st[tid];
        p[tid * kRec + kHeadDim + 1] = st[kRows + tid];
    }
}

// one CTA per (pair, row)
__global__ void __launch_bounds__(128) block_join_kernel(const BlockDev D, const BlockAttendArgs a) {
    const int R = a.n_q * D.G, r = blockIdx.x % R, tid = threadIdx.x;
    const int64_t pair = blockIdx.x / R;
    const float *p = a.part + (pair * kParts * kRows + r) * kRec;
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int i = 0; i < kParts; ++i) m = fmaxf(m, p[(int64_t)i * kRows * kRec + kHeadDim]);
    if (m > -INFINITY)
        for (int i = 0; i < kParts; ++i) {
            const float *pi = p + (int64_t)i * kRows * kRec, f = exp2f(pi[kHeadDim] - m);
            l += f * pi[kHeadDim + 1];
            o += f * pi[tid];
        }
    const int b = (int)(pair / D.Hkv), head = (int)(pair % D.Hkv) * D.G + r % D.G, i = r / D.G;
    a.out[(((int64_t)b * a.n_q + i) * D.Hq + head) * kHeadDim + tid] = __float2bfloat16_rn(l > 0.f ? o / l : 0.f);
    if (tid == 0) {
        const float lse = l > 0.f ? m + log2f(l) : -INFINITY;
        if (a.lse) a.lse[((int64_t)b * D.Hq + head) * a.n_q + i] = lse * 0.6931471805599453f;
        a.row_lse[pair * R + r] = lse;
    }
}

__global__ void __launch_bounds__(kBlk) block_weights_kernel(const BlockDev D, const BlockAttendArgs a) {
    const int64_t pair = blockIdx.x / D.NB;
    const int j = blockIdx.x % D.NB, R = a.n_q * D.G, t = threadIdx.x;
    const int len = blk_len(D, a.kv_len, (int)(pair / D.Hkv)), pos = j * kBlk + t;
    if (pos >= len) return;
    float w = 0.f;
    for (int r = 0; r < R; ++r) {
        const float lse = a.row_lse[pair * R + r];
        if (lse > -INFINITY) w += exp2f(a.logits[((pair * D.NB + j) * R + r) * kBlk + t] - lse);
    }
    float *o = a.weights + pair * D.capacity + pos;
    *o = (a.accumulate ? *o : 0.f) + w / D.G;
}

}  // namespace

int64_t blk_part_floats(int B, int Hkv, int, int) { return (int64_t)B * Hkv * kParts * kRows * kRec; }

cudaError_t launch_block_attend(const BlockDev &D, int fmt, const BlockAttendArgs &a, int, cudaStream_t s) {
    const int64_t pairs = (int64_t)D.B * D.Hkv;
    const int R = a.n_q * D.G;
    const int smem = (2 * kRows * kHeadDim + kTile * (2 * kHeadDim + 1) + kRows * kTile + 3 * kRows) * 4;
    auto kernel = fmt == QEVICT_BLOCK_INT8 ? block_attend_kernel<QEVICT_BLOCK_INT8> : block_attend_kernel<QEVICT_BLOCK_E4M3>;
    cudaError_t e = once_per_device(fmt, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(pairs * kParts), 128, smem, s>>>(D, a);
    block_join_kernel<<<(unsigned)(pairs * R), 128, 0, s>>>(D, a);
    if (a.weights) block_weights_kernel<<<(unsigned)(pairs * D.NB), kBlk, 0, s>>>(D, a);
    return cudaGetLastError();
}

}  // namespace qevict
