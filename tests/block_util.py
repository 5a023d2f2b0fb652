"""Plain forms of the cache in 8 bits in numpy: the quantiser as it is defined (a scale and a quotient rounded to
fp32), attention and weights in 64 bits, eviction by a stable sort."""
import numpy as np
import torch

D, T = 128, 64
TOP = {"int8": 127.0, "e4m3": 448.0}


def quantise(x, fmt):
    """x [..., 64, 128] fp32: (codes as fp32 numbers, scales fp32 [...])."""
    x = np.asarray(x, np.float32)
    s = np.abs(x).max((-2, -1)) / np.float32(TOP[fmt])
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s[..., None, None] > 0, x / s[..., None, None], np.float32(0)).astype(np.float32)
    y = np.clip(y, -TOP[fmt], TOP[fmt])
    if fmt == "int8":
        return np.rint(y), s
    return torch.from_numpy(y).to(torch.float8_e4m3fn).float().numpy(), s


def held(x, fmt):
    """fp32 values that whole blocks x [..., n, 128] stand for."""
    code, s = quantise(x.reshape(*x.shape[:-2], -1, T, D), fmt)
    return (code * s[..., None, None]).astype(np.float32).reshape(x.shape)


class Cache:
    """Values [B][Hkv][n][128] fp32: of full blocks what their codes stand for, of the open block its bf16 rows."""

    def __init__(self, B, Hkv, capacity, fmt):
        self.fmt, self.cap = fmt, capacity
        self.raw = {x: np.zeros((B, Hkv, capacity, D), np.float32) for x in "kv"}

    def append(self, k, v, start, n_new):
        """k, v [B][n][Hkv][128] bf16 tensors"""
        for x, t in (("k", k), ("v", v)):
            t = t.detach().cpu().float().numpy()
            for b in range(t.shape[0]):
                e = min(start[b] + n_new[b], self.cap)
                self.raw[x][b, :, start[b]:e] = t[b, :e - start[b]].transpose(1, 0, 2)

    def values(self, x, b, length):
        r = self.raw[x][b, :, :length].copy()
        c = length // T * T
        r[:, :c] = held(r[:, :c], self.fmt)
        return r


def attention(q, k, v):
    """q [n_q][Hq][128], k, v [Hkv][n][128] in 64 bits: out [n_q][Hq][128], lse [Hq][n_q], weights [Hkv][n] and, for
    tolerances, sum p |v|, sum |v| relative to the largest probability, and the largest sum |q k| / sqrt(128)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n_q, Hq, _ = q.shape
    Hkv, n = k.shape[:2]
    G = Hq // Hkv
    out, mag, low = (np.zeros((n_q, Hq, D)) for _ in range(3))
    lse = np.full((Hq, n_q), -np.inf)
    w = np.zeros((Hkv, n))
    big = 0.0
    for i in range(n_q):
        e = n - n_q + i + 1
        if e <= 0:
            continue
        for h in range(Hq):
            x = k[h // G, :e] @ q[i, h] / np.sqrt(D)
            big = max(big, (np.abs(k[h // G, :e]) @ np.abs(q[i, h])).max() / np.sqrt(D))
            m = x.max()
            p = np.exp(x - m)
            lse[h, i] = m + np.log(p.sum())
            low[i, h] = np.abs(v[h // G, :e]).sum(0) / p.sum()
            p /= p.sum()
            out[i, h] = p @ v[h // G, :e]
            mag[i, h] = p @ np.abs(v[h // G, :e])
            w[h // G, :e] += p / G
    return out, lse, w, mag, low, big


def select(w, c, keep, recent):
    """Positions that stay of c tokens with weights w."""
    if c <= keep:
        return np.arange(c)
    w = w[:c - recent].astype(np.float64)
    nan = np.isnan(w)
    order = np.lexsort((np.arange(c - recent), -np.where(nan, 0.0, w), nan))   # NaN below every number, -inf too
    return np.concatenate([np.sort(order[:keep - recent]), np.arange(c - recent, c)])
