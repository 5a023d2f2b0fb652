// The cache in 8 bits: its layout, the quantiser of a block and the launch entry
// points of qevict_block.cu and qevict_block_attend.cu.
#pragma once

#include "qevict_internal.cuh"

namespace qevict {

constexpr int kBlk = QEVICT_BLOCK_TOKENS;      // tokens that share a scale
constexpr int kBlkBytes = 2 * kBlk * kHeadDim; // a block's codes of K, then of V
constexpr int kOpenHalf = 32;                  // tokens of half an open block: as many bytes as a block's codes
constexpr int kMaxBlkQueries = QEVICT_BLOCK_MAX_QUERIES;
constexpr int kMaxBlkTokens = 1 << 21;         // of a sequence, and of a call (blocks are a grid's second dimension)

// A layer's memory. "pair" = sequence * Hkv + KV head.
//  codes  [pair][NB][K, V][64 tokens][128 channels], a byte each. The eight
//         16-byte chunks of a token's row lie at chunk ^ (token & 7), so that
//         eight lanes that read one chunk of eight tokens, or two neighbouring
//         tokens' alternate chunks, meet no shared-memory bank twice.
//  scale  [pair][NB] (K, V)
//  open   [pair][block & 1][token >> 5][K, V][32 tokens][128] bf16: the rows of the
//         block that is not full, and of the one before it.
struct BlockDev {
    uint8_t *codes;
    float2 *scale;
    uint8_t *open;
    int B, Hq, Hkv, G, NB, capacity, layer;
    int32_t *status;   // [4] as CacheDev::status
};

__host__ __device__ inline int64_t blk_code_off(const BlockDev &D, int64_t pair, int block) {
    return (pair * D.NB + block) * kBlkBytes;
}
// byte of chunk c (16 channels) of token t of a block's K codes (V: kBlkBytes / 2 further)
__host__ __device__ inline int blk_chunk(int t, int c) { return t * kHeadDim + ((c ^ (t & 7)) << 4); }
__host__ __device__ inline int64_t blk_open_off(int64_t pair, int block, int t) {
    return ((pair * 2 + (block & 1)) * 2 + (t >> 5)) * kBlkBytes;
}
// byte of chunk c (8 channels) of token t & 31 of half an open block's K rows. Chunks c and
// c + 8 of a row, 128 bytes apart, differ in bit 1 of their place, for the same reason.
__host__ __device__ inline int blk_open_chunk(int t, int c) {
    return (t & 31) * (2 * kHeadDim) + (((c & 8) | ((c & 7) ^ (t & 7) ^ ((c >> 3) << 1))) << 4);
}

struct BlockAppendArgs {
    const __nv_bfloat16 *k, *v;      // token i of sequence b: (b * n + i) * stride elements on
    int64_t k_stride, v_stride;
    const int32_t *start, *n_new;    // [B] or NULL: 0, n
    int n;
    float *weights;                  // [pair][capacity] or NULL
};
struct BlockReadArgs {
    const int32_t *kv_len, *first;   // [B]; first NULL: 0
    int n;
    __nv_bfloat16 *k, *v;            // [B][n][Hkv][128]
};
struct BlockEvictArgs {
    const int32_t *kv_len;
    int keep, recent;
    const float *weights;            // [pair][capacity]
    float *weights_out;              // [pair][the other cache's capacity] or NULL
    int32_t *new_len, *kept;         // [B], [pair][keep]
};
struct BlockAttendArgs {
    const __nv_bfloat16 *q;          // [B][n_q][Hq][128]
    const int32_t *kv_len;
    int n_q;
    __nv_bfloat16 *out;
    float *lse;                      // [B][Hq][n_q] or NULL
    float *weights;                  // [pair][capacity] or NULL
    int accumulate;
    // scratch of the handle
    float *part;
    float *logits;                   // [pair][NB][8][rows][8 tokens] where weights are wanted
    float *row_lse;                  // [pair][rows], log2 domain
};

cudaError_t launch_block_append(const BlockDev &D, int fmt, const BlockAppendArgs &a, cudaStream_t s);
cudaError_t launch_block_read(const BlockDev &D, int fmt, const BlockReadArgs &a, cudaStream_t s);
cudaError_t launch_block_evict(const BlockDev &D, const BlockDev &to, int fmt, const BlockEvictArgs &a,
                               cudaStream_t s);
cudaError_t launch_block_attend(const BlockDev &D, int fmt, const BlockAttendArgs &a, int num_sms, cudaStream_t s);
int64_t blk_part_floats(int G, int num_sms);   // of `part`, for the calls of a handle with G query heads per KV head

__device__ __forceinline__ void blk_status(const BlockDev &D, int code, int b, int info) {
    if (atomicCAS(D.status, 0, code) == 0) {
        D.status[1] = D.layer;
        D.status[2] = b;
        D.status[3] = info;
    }
}

__device__ __forceinline__ int blk_len(const BlockDev &D, const int32_t *len, int b) {
    return min(max(len[b], 0), D.capacity);
}

// Two neighbouring codes (the low or high half of w) as two halves, exactly: an int8 code is
// held with 128 added, and 1024 + u is the half 0x6400 | u.
template <int FMT, bool HIGH = false>
__device__ __forceinline__ __half2 blk_half2(uint32_t w) {
    uint32_t x;
    if constexpr (FMT == QEVICT_BLOCK_INT8) {
        x = __byte_perm(w, 0x64646464u, HIGH ? 0x5342 : 0x5140);
        return __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x6480)));
    } else if constexpr (HIGH) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(x) : "r"(w));
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(x) : "r"(w));
    }
    return *reinterpret_cast<const __half2 *>(&x);
}

// The codes of a block's scale. s = fl32(amax / Q); code = round(fl32(x / s)), to the
// nearest, ties to even. The quotient comes from the reciprocal and two FMAs, which
// round it as the division does while nothing underflows; below 2^-60 (values of no
// model) both sides are first multiplied by 2^80, which changes no quotient, and the
// quotient is clamped (s is then rounded to few bits). amax is finite.
struct BlockScale {
    float s, up, d, r;   // up 1 or 2^80; d = s up, r its reciprocal (s = 0: 0)
};
template <int FMT>
__device__ __forceinline__ BlockScale blk_scale(float amax) {
    BlockScale q;
    q.s = __fdiv_rn(amax, FMT == QEVICT_BLOCK_INT8 ? 127.f : 448.f);
    q.up = q.s >= 0x1p-60f ? 1.f : 0x1p80f;
    q.d = q.s * q.up;
    q.r = q.s > 0.f ? __frcp_rn(q.d) : 0.f;
    return q;
}
// two fp32 operations in one instruction, each rounded as usual
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 f2_unpack(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// Eight codes of four pairs of values. The quotient is that of div_by_recip (qevict_div.cuh), two at a time.
template <int FMT>
__device__ __forceinline__ uint2 blk_codes(const uint64_t *x, const BlockScale &q) {
    constexpr float top = FMT == QEVICT_BLOCK_INT8 ? 127.f : 448.f;
    const uint64_t r2 = f2_pack(q.r, q.r), nd2 = f2_pack(-q.d, -q.d);
    uint64_t z[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = x[j];
    if (q.up != 1.f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = f2_mul(z[j], f2_pack(q.up, q.up));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint64_t q0 = f2_mul(z[j], r2);
        z[j] = f2_fma(f2_fma(q0, nd2, z[j]), r2, q0);
    }
    if (q.up != 1.f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 y = f2_unpack(z[j]);
            z[j] = f2_pack(fminf(fmaxf(y.x, -top), top), fminf(fmaxf(y.y, -top), top));
        }
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (FMT == QEVICT_BLOCK_INT8) {
            // 1.5 * 2^23 + 128 + y: rounded to an integer, code + 128 in the low byte
            const uint64_t magic = f2_pack(12583040.f, 12583040.f);
            const float2 a = f2_unpack(f2_add(z[2 * i], magic)), b = f2_unpack(f2_add(z[2 * i + 1], magic));
            w[i] = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                               __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
        } else {
            const float2 a = f2_unpack(z[2 * i]), b = f2_unpack(z[2 * i + 1]);
            asm("{\n\t.reg .b16 l, h;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
                "mov.b32 %0, {l, h};\n\t}"
                : "=r"(w[i])
                : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
        }
    }
    return make_uint2(w[0], w[1]);
}
// eight codes as four pairs of values fl32(code * s)
template <int FMT>
__device__ __forceinline__ void blk_values(uint2 c, float s, uint64_t *x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? c.x : c.y;
        uint64_t y;
        if constexpr (FMT == QEVICT_BLOCK_INT8) {
            // 2^23 + code + 128 has the held code in its low byte
            const uint32_t a = __byte_perm(w, 0x4B000000u, (i & 1) ? 0x7652 : 0x7650);
            const uint32_t b = __byte_perm(w, 0x4B000000u, (i & 1) ? 0x7653 : 0x7651);
            y = f2_add(f2_pack(__uint_as_float(a), __uint_as_float(b)), f2_pack(-8388736.f, -8388736.f));
        } else {
            const float2 f = __half22float2((i & 1) ? blk_half2<FMT, true>(w) : blk_half2<FMT>(w));
            y = f2_pack(f.x, f.y);
        }
        x[i] = f2_mul(y, f2_pack(s, s));
    }
}

}  // namespace qevict
