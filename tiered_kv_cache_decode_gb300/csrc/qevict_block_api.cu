// Host side of the calls on the cache in 8 bits: argument checks, allocations, launches.
#include <new>
#include <vector>

#include "qevict_block.cuh"
#include "qevict_host.h"

using namespace qevict;

struct qevict_block_cache {
    qevict_block_config cfg{};
    qevict_allocator alloc{};
    bool user_alloc = false;
    cudaStream_t stream = nullptr;
    int device = 0, num_sms = 1, G = 1, NB = 0, capacity = 0;
    int32_t *status = nullptr;
    float *part = nullptr, *logits = nullptr, *row_lse = nullptr;
    std::vector<BlockDev> layers;
    std::vector<void *> memory;
};

namespace {

void *take(qevict_block_cache *c, size_t bytes) {
    void *p = nullptr;
    if (c->user_alloc) {
        p = c->alloc.alloc(bytes, (void *)c->stream, c->alloc.ctx);
    } else if (cudaMalloc(&p, bytes) != cudaSuccess) {
        cudaGetLastError();
        p = nullptr;
    }
    if (p) c->memory.push_back(p);
    return p;
}

void release(qevict_block_cache *c) {
    for (void *p : c->memory) {
        if (c->user_alloc) c->alloc.free(p, (void *)c->stream, c->alloc.ctx);
        else cudaFree(p);
    }
    delete c;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

qevict_status check_config(const qevict_block_config &f) {
    if (f.batch < 1 || f.num_layers < 1 || f.num_kv_heads < 1 || f.num_q_heads < 1)
        return fail(QEVICT_ERR_INVALID_ARG, "batch, layers and head counts must be >= 1");
    if (f.num_q_heads % f.num_kv_heads != 0 || f.num_q_heads / f.num_kv_heads > kMaxG)
        return fail(QEVICT_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads, at most %d per KV head",
                    kMaxG);
    if (f.head_dim != kHeadDim) return fail(QEVICT_ERR_INVALID_ARG, "head_dim must be %d", kHeadDim);
    if (f.capacity < 1 || f.capacity > kMaxBlkTokens)
        return fail(QEVICT_ERR_INVALID_ARG, "capacity must be in [1, 2^21]");
    if (f.format != QEVICT_BLOCK_INT8 && f.format != QEVICT_BLOCK_E4M3)
        return fail(QEVICT_ERR_INVALID_ARG, "format must be QEVICT_BLOCK_INT8 or QEVICT_BLOCK_E4M3");
    if (f.score_queries < 0 || f.score_queries > kMaxBlkQueries)
        return fail(QEVICT_ERR_INVALID_ARG, "score_queries must be in [0, %d]", kMaxBlkQueries);
    if (f.batch > 65535 || (int64_t)f.batch * f.num_kv_heads > 1 << 20)
        return fail(QEVICT_ERR_INVALID_ARG, "batch must be at most 65535, batch x num_kv_heads at most 2^20");
    if ((int64_t)f.batch * f.num_kv_heads * ((f.capacity + kBlk - 1) / kBlk + 2) >= 1 << 30)
        return fail(QEVICT_ERR_INVALID_ARG, "batch x num_kv_heads x blocks must be below 2^30");
    return QEVICT_OK;
}

qevict_status check_call(const qevict_block_cache *c, int32_t layer) {
    if (!c) return fail(QEVICT_ERR_INVALID_ARG, "cache is NULL");
    if (layer < 0 || layer >= c->cfg.num_layers)
        return fail(QEVICT_ERR_INVALID_ARG, "layer %d out of range [0, %d)", layer, c->cfg.num_layers);
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "current device");
    if (dev != c->device)
        return fail(QEVICT_ERR_INVALID_ARG, "the cache is on device %d, the current device is %d", c->device, dev);
    return QEVICT_OK;
}

qevict_status check_align(uintptr_t p, int align, const char *what) {
    if (p & (uintptr_t)(align - 1)) return fail(QEVICT_ERR_INVALID_ARG, "%s must be %d-byte aligned", what, align);
    return QEVICT_OK;
}

}  // namespace

extern "C" {

qevict_status qevict_block_create(const qevict_block_config *config, const qevict_allocator *allocator, void *stream,
                                  qevict_block_cache **out) {
    if (!config || !out) return fail(QEVICT_ERR_INVALID_ARG, "config and out must not be NULL");
    *out = nullptr;
    const qevict_block_config f = *config;
    const qevict_status st = check_config(f);
    if (st) return st;
    if (allocator && (!allocator->alloc || !allocator->free))
        return fail(QEVICT_ERR_INVALID_ARG, "allocator needs both alloc and free");
    qevict_block_cache *c = new (std::nothrow) qevict_block_cache();
    if (!c) return fail(QEVICT_ERR_OUT_OF_MEMORY, "no host memory for the handle");
    c->cfg = f;
    if (allocator) {
        c->alloc = *allocator;
        c->user_alloc = true;
    }
    c->stream = (cudaStream_t)stream;
    cudaError_t e = cudaGetDevice(&c->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->device);
    if (e != cudaSuccess && !c->user_alloc) {
        release(c);
        return cuda_fail(e, "device query");
    }
    cudaGetLastError();
    c->G = f.num_q_heads / f.num_kv_heads;
    c->NB = (f.capacity + kBlk - 1) / kBlk;
    c->capacity = c->NB * kBlk;
    const size_t pairs = (size_t)f.batch * f.num_kv_heads;
    // every allocation first, so that a failing allocator leaves nothing behind
    const size_t o_lse = 256, o_part = o_lse + up256(pairs * kMaxBlkQueries * c->G * 4);
    const size_t base_bytes = o_part + (size_t)blk_part_floats(c->G, c->num_sms) * 4;
    const size_t logit_bytes = pairs * c->capacity * c->G * f.score_queries * 4;
    const size_t o_scale = up256(pairs * c->NB * (size_t)kBlkBytes), o_open = o_scale + up256(pairs * c->NB * 8);
    const size_t layer_bytes = o_open + pairs * 4 * (size_t)kBlkBytes;
    size_t failed = 0;
    try {
        c->memory.reserve((size_t)f.num_layers + 2);
        c->layers.reserve(f.num_layers);
    } catch (const std::bad_alloc &) {
        release(c);
        return fail(QEVICT_ERR_OUT_OF_MEMORY, "no host memory for %d layers", f.num_layers);
    }
    uint8_t *base = (uint8_t *)take(c, base_bytes);
    if (!base) failed = base_bytes;
    if (!failed && logit_bytes && !(c->logits = (float *)take(c, logit_bytes))) failed = logit_bytes;
    for (int l = 0; l < f.num_layers && !failed; ++l) {
        BlockDev D{};
        D.B = f.batch;
        D.Hq = f.num_q_heads;
        D.Hkv = f.num_kv_heads;
        D.G = c->G;
        D.NB = c->NB;
        D.capacity = c->capacity;
        D.layer = l;
        D.codes = (uint8_t *)take(c, layer_bytes);
        if (!D.codes) failed = layer_bytes;
        D.scale = (float2 *)(D.codes + o_scale);
        D.open = D.codes + o_open;
        D.status = (int32_t *)base;
        c->layers.push_back(D);
    }
    if (failed) {
        release(c);
        return fail(QEVICT_ERR_OUT_OF_MEMORY, "allocation of %zu B failed", failed);
    }
    c->status = (int32_t *)base;
    c->row_lse = (float *)(base + o_lse);
    c->part = (float *)(base + o_part);
    e = cudaMemsetAsync(base, 0, o_part, c->stream);
    for (const BlockDev &D : c->layers)
        if (e == cudaSuccess) e = cudaMemsetAsync(D.codes, 0, layer_bytes, c->stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(c->stream);
    if (e != cudaSuccess) {
        release(c);
        return cuda_fail(e, "cache initialisation");
    }
    *out = c;
    return QEVICT_OK;
}

qevict_status qevict_block_destroy(qevict_block_cache *c) {
    if (!c) return fail(QEVICT_ERR_INVALID_ARG, "cache is NULL");
    // Also while the thread captures another stream (a handle that goes at any time): a wait in the usual mode would end
    // that capture. The handle's own stream, where that is the one in capture, cannot be waited for.
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    const bool relaxed = cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess;
    cudaStreamCaptureStatus state = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(c->stream, &state);
    if (e == cudaSuccess && state == cudaStreamCaptureStatusNone) e = cudaStreamSynchronize(c->stream);
    if (e != cudaSuccess) cudaGetLastError();
    release(c);
    if (relaxed) cudaThreadExchangeStreamCaptureMode(&mode);
    return QEVICT_OK;
}

int32_t qevict_block_capacity(const qevict_block_cache *c) { return c ? c->capacity : -1; }

qevict_status qevict_block_append(qevict_block_cache *c, int32_t layer, const void *k, int64_t k_stride, const void *v,
                                  int64_t v_stride, int32_t n, const int32_t *start, const int32_t *n_new,
                                  float *weights, void *stream) {
    qevict_status st = check_call(c, layer);
    if (st) return st;
    if (!k || !v) return fail(QEVICT_ERR_INVALID_ARG, "k and v must not be NULL");
    if (n < 1 || n > kMaxBlkTokens) return fail(QEVICT_ERR_INVALID_ARG, "n (%d) must be in [1, 2^21]", n);
    const int64_t row = (int64_t)c->cfg.num_kv_heads * kHeadDim;
    for (const int64_t x : {k_stride, v_stride})
        if (x < row || x % 8 || x > (int64_t)1 << 32)
            return fail(QEVICT_ERR_INVALID_ARG, "a token stride of %lld elements: a multiple of 8, at least the token's "
                        "%d heads and at most 2^32", (long long)x, c->cfg.num_kv_heads);
    st = check_align((uintptr_t)k | (uintptr_t)v, 16, "k and v");
    if (!st) st = check_align((uintptr_t)start | (uintptr_t)n_new | (uintptr_t)weights, 4, "start, n_new and weights");
    if (st) return st;
    const int64_t B = c->cfg.batch, last = B * n - 1;
    const Extent x[4] = {{k, (last * k_stride + row) * 2, "k"}, {v, (last * v_stride + row) * 2, "v"},
                         {start, B * 4, "start"}, {n_new, B * 4, "n_new"}};
    st = check_apart({weights, B * c->cfg.num_kv_heads * (int64_t)c->capacity * 4, "weights"}, x, 4);
    if (st) return st;
    BlockAppendArgs a{};
    a.k = (const __nv_bfloat16 *)k;
    a.v = (const __nv_bfloat16 *)v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.n = n;
    a.start = start;
    a.n_new = n_new;
    a.weights = weights;
    const cudaError_t e = launch_block_append(c->layers[layer], c->cfg.format, a, (cudaStream_t)stream);
    return e == cudaSuccess ? QEVICT_OK : cuda_fail(e, "block append kernel");
}

qevict_status qevict_block_attention(qevict_block_cache *c, int32_t layer, const void *q, int32_t n_q,
                                     const int32_t *kv_len, void *out, float *lse, float *weights, int32_t accumulate,
                                     void *stream) {
    qevict_status st = check_call(c, layer);
    if (st) return st;
    if (!q || !kv_len || !out) return fail(QEVICT_ERR_INVALID_ARG, "q, kv_len and out must not be NULL");
    if (n_q < 1 || n_q > kMaxBlkQueries)
        return fail(QEVICT_ERR_INVALID_ARG, "n_q (%d) must be in [1, %d]", n_q, kMaxBlkQueries);
    if (weights && n_q > c->cfg.score_queries)
        return fail(QEVICT_ERR_INVALID_ARG, "weights of %d queries; the cache has scratch for %d (score_queries)", n_q,
                    c->cfg.score_queries);
    st = check_align((uintptr_t)q | (uintptr_t)out, 16, "q and out");
    if (!st) st = check_align((uintptr_t)kv_len | (uintptr_t)lse | (uintptr_t)weights, 4, "kv_len, lse and weights");
    if (st) return st;
    const int64_t B = c->cfg.batch, rows = B * n_q * c->cfg.num_q_heads;
    const Extent x[5] = {{q, rows * kHeadDim * 2, "q"}, {kv_len, B * 4, "kv_len"}, {out, rows * kHeadDim * 2, "out"},
                         {lse, rows * 4, "lse"},
                         {weights, B * c->cfg.num_kv_heads * (int64_t)c->capacity * 4, "weights"}};
    for (int i = 2; i < 5 && !st; ++i) st = check_apart(x[i], x, i);
    if (st) return st;
    BlockAttendArgs a{};
    a.q = (const __nv_bfloat16 *)q;
    a.kv_len = kv_len;
    a.n_q = n_q;
    a.out = (__nv_bfloat16 *)out;
    a.lse = lse;
    a.weights = weights;
    a.accumulate = accumulate;
    a.part = c->part;
    a.logits = c->logits;
    a.row_lse = c->row_lse;
    const cudaError_t e = launch_block_attend(c->layers[layer], c->cfg.format, a, c->num_sms, (cudaStream_t)stream);
    return e == cudaSuccess ? QEVICT_OK : cuda_fail(e, "block attention kernel");
}

qevict_status qevict_block_read(qevict_block_cache *c, int32_t layer, const int32_t *kv_len, const int32_t *first,
                                int32_t n, void *k, void *v, void *stream) {
    qevict_status st = check_call(c, layer);
    if (st) return st;
    if (!kv_len || !k || !v) return fail(QEVICT_ERR_INVALID_ARG, "kv_len, k and v must not be NULL");
    if (n < 1 || n > kMaxBlkTokens) return fail(QEVICT_ERR_INVALID_ARG, "n (%d) must be in [1, 2^21]", n);
    st = check_align((uintptr_t)k | (uintptr_t)v, 16, "k and v");
    if (!st) st = check_align((uintptr_t)kv_len | (uintptr_t)first, 4, "kv_len and first");
    if (st) return st;
    const int64_t B = c->cfg.batch, bytes = B * n * c->cfg.num_kv_heads * kHeadDim * 2;
    const Extent x[4] = {{kv_len, B * 4, "kv_len"}, {first, B * 4, "first"}, {k, bytes, "k"}, {v, bytes, "v"}};
    for (int i = 2; i < 4 && !st; ++i) st = check_apart(x[i], x, i);
    if (st) return st;
    BlockReadArgs a{};
    a.kv_len = kv_len;
    a.first = first;
    a.n = n;
    a.k = (__nv_bfloat16 *)k;
    a.v = (__nv_bfloat16 *)v;
    const cudaError_t e = launch_block_read(c->layers[layer], c->cfg.format, a, (cudaStream_t)stream);
    return e == cudaSuccess ? QEVICT_OK : cuda_fail(e, "block read kernel");
}

qevict_status qevict_block_evict(qevict_block_cache *c, int32_t layer, const int32_t *kv_len, int32_t keep,
                                 int32_t recent, const float *weights, qevict_block_cache *to, int32_t to_layer,
                                 float *weights_out, int32_t *new_len, int32_t *kept, void *stream) {
    qevict_status st = check_call(c, layer);
    if (!st) st = check_call(to, to_layer);
    if (st) return st;
    if (!kv_len || !weights || !new_len || !kept)
        return fail(QEVICT_ERR_INVALID_ARG, "kv_len, weights, new_len and kept must not be NULL");
    if (to->cfg.batch != c->cfg.batch || to->cfg.num_kv_heads != c->cfg.num_kv_heads ||
        to->cfg.format != c->cfg.format)
        return fail(QEVICT_ERR_INVALID_ARG, "the destination must have the same batch, KV heads and format");
    if (keep < kBlk || keep % kBlk || keep + kBlk > to->capacity)
        return fail(QEVICT_ERR_INVALID_ARG, "keep (%d) must be a multiple of %d, at least %d and at most %d (the "
                    "destination's capacity without the open block)", keep, kBlk, kBlk, to->capacity - kBlk);
    if (recent < 0 || recent > keep)
        return fail(QEVICT_ERR_INVALID_ARG, "recent (%d) must be in [0, keep]", recent);
    st = check_align((uintptr_t)weights, 16, "weights");
    if (!st)
        st = check_align((uintptr_t)kv_len | (uintptr_t)weights_out | (uintptr_t)new_len | (uintptr_t)kept, 4,
                         "kv_len, weights_out, new_len and kept");
    if (st) return st;
    const int64_t B = c->cfg.batch, pairs = B * c->cfg.num_kv_heads;
    const bool own = weights_out == weights && to == c && to_layer == layer;   // elsewhere tokens move in no order
    const Extent x[5] = {{kv_len, B * 4, "kv_len"}, {weights, pairs * (int64_t)c->capacity * 4, "weights"},
                         {own ? nullptr : weights_out, pairs * (int64_t)to->capacity * 4, "weights_out"},
                         {new_len, B * 4, "new_len"}, {kept, pairs * keep * 4, "kept"}};
    for (int i = 2; i < 5 && !st; ++i) st = check_apart(x[i], x, i);
    if (st) return st;
    BlockEvictArgs a{};
    a.kv_len = kv_len;
    a.keep = keep;
    a.recent = recent;
    a.weights = weights;
    a.weights_out = weights_out;
    a.new_len = new_len;
    a.kept = kept;
    const cudaError_t e =
        launch_block_evict(c->layers[layer], to->layers[to_layer], c->cfg.format, a, (cudaStream_t)stream);
    return e == cudaSuccess ? QEVICT_OK : cuda_fail(e, "block eviction kernels");
}

qevict_status qevict_block_view(const qevict_block_cache *c, int32_t layer, const void **codes, const float **scales) {
    if (!c) return fail(QEVICT_ERR_INVALID_ARG, "cache is NULL");
    if (layer < 0 || layer >= c->cfg.num_layers)
        return fail(QEVICT_ERR_INVALID_ARG, "layer %d out of range [0, %d)", layer, c->cfg.num_layers);
    if (!codes || !scales) return fail(QEVICT_ERR_INVALID_ARG, "codes and scales must not be NULL");
    *codes = c->layers[layer].codes;
    *scales = (const float *)c->layers[layer].scale;
    return QEVICT_OK;
}

qevict_status qevict_block_get_status(qevict_block_cache *c, void *stream) {
    if (!c) return fail(QEVICT_ERR_INVALID_ARG, "cache is NULL");
    cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "stream synchronise");
    int32_t s[4];
    e = cudaMemcpy(s, c->status, sizeof s, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "status copy");
    return s[0] ? fail((qevict_status)s[0], "device status %d at layer %d (sequence %d, item %d)", s[0], s[1], s[2], s[3])
                : QEVICT_OK;
}

qevict_status qevict_block_clear_status(qevict_block_cache *c, void *stream) {
    if (!c) return fail(QEVICT_ERR_INVALID_ARG, "cache is NULL");
    const cudaError_t e = cudaMemsetAsync(c->status, 0, 16, (cudaStream_t)stream);
    return e == cudaSuccess ? QEVICT_OK : cuda_fail(e, "status reset");
}

}  // extern "C"
