"""Plain 64-bit forms of the operators between a layer's projections and its
cache (head norms with rotation, span attention, window scores), in numpy."""
import numpy as np

D = 128


def norm_rope(x, weight, eps, pos, inv_freq, interleaved=False):
    """x [B][n][H][128] float64, pos [B][n], weight [128] or None."""
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * weight
    t = np.asarray(pos, np.float64)[:, :, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(t), np.sin(t)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :64], x[..., 64:])
    y = np.empty_like(x)
    u, v = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0::2], y[..., 1::2] = u, v
    else:
        y[..., :64], y[..., 64:] = u, v
    return y


def visible(n_q, n_kv, span, sinks):
    """bool [n_q][n_kv]: the queries are the last n_q of n_kv positions (earlier ones see nothing)."""
    p = n_kv - n_q + np.arange(n_q)[:, None]
    j = np.arange(n_kv)[None, :]
    return (j <= p) & ((j > p - (span or n_kv + n_q)) | (j < sinks))


def attention_head(q, k, v, seen):
    """(out [n_q][128], lse [n_q]) of one head in float64; a row that sees nothing gives 0 and -inf."""
    x = np.where(seen, q @ k.T / np.sqrt(D), -np.inf)
    m = np.max(x, -1, keepdims=True, initial=-np.inf)
    p = np.exp(x - np.where(np.isneginf(m), 0.0, m))
    p[~seen] = 0.0
    total = p.sum(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = np.log(total[:, 0]) + m[:, 0]
        out = np.where(total > 0, p @ np.where(seen.any(0)[:, None], v, 0.0) / total, 0.0)
    return out, lse


def attention(q, k, v, q_len, kv_len, span, sinks):
    """q [B][n_q][Hq][128], k, v [B][n_kv][Hkv][128] float64. Rows past q_len are NaN."""
    B, n_q, Hq, _ = q.shape
    G = Hq // k.shape[2]
    out = np.full(q.shape, np.nan)
    lse = np.full((B, Hq, n_q), np.nan)
    for b in range(B):
        nq, nk = q_len[b], kv_len[b]
        seen = visible(nq, nk, span, sinks)
        for h in range(Hq):
            o, s = attention_head(q[b, :nq, h], k[b, :nk, h // G], v[b, :nk, h // G], seen)
            out[b, :nq, h], lse[b, h, :nq] = o, s
    return out, lse


def scores(q, k, lse, q_len, kv_len, span, sinks, w, per_head=False):
    """Window scores [B][W] (or [B * Hkv][W]) in float64."""
    B, n_q, Hq, _ = q.shape
    Hkv, n_kv = k.shape[2], k.shape[1]
    G, W = Hq // Hkv, -(-n_kv // w)
    out = np.zeros((B, Hkv, W))
    for b in range(B):
        nq, nk = q_len[b], kv_len[b]
        seen = visible(nq, nk, span, sinks)
        for h in range(Hq):
            x = q[b, :nq, h] @ k[b, :nk, h // G].T / np.sqrt(D)
            with np.errstate(invalid="ignore", over="ignore"):
                mass = np.where(seen, np.exp(x - lse[b, h, :nq, None]), 0.0).sum(0)
            out[b, h // G] += np.pad(mass, (0, W * w - nk)).reshape(W, w).sum(1) / G
    return out.reshape(B * Hkv, W) if per_head else out.mean(1)
