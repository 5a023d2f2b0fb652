"""The operators between a prompt's projections and its tiered cache, as a user's program calls them.

Three operators, in the order in which a layer runs them:

* rope: RMS norm of every query and key head, the rotation by position, and the
  values copied out of the fused projection, in one pass;
* attention: causal softmax attention of the last n_q positions over a layer's
  uncompressed keys, each query seeing the `span` latest positions (0: all)
  and the first `sinks` ones, with the log-sum-exp of every row;
* scores: the attention mass that each cache window receives from a set of
  queries (mean over the query heads, summed over the queries): the initial
  window scores on which a prompt's prefill routes.

`run` computes them in elementary torch operations (fp32, rounded once) where
`own` is false, and through the library where it is true.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head size
EPS = 1e-6       # of the norms
CHUNK = 1 << 28  # logits that the plain form holds at a time


def _case(name, op, B, Hq, Hkv, n_q, n_kv, ragged=0, span=0, sinks=0, window=64, norm=True, far=0):
    c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, n_q=n_q, n_kv=n_kv, ragged=ragged, span=span, sinks=sinks, window=window,
             norm=norm, far=far)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode step of a batch of 16 conversations (28 query, 4 KV heads), far into their contexts
        _case("rope step b16", "rope", 16, 28, 4, 1, 1, far=16384),
        # the next chunk of four prompts of odd length on a model without head norms (rotation only)
        _case("rope chunk b4", "rope", 4, 32, 8, 777, 777, norm=False, far=4096),
        # a 32K prompt (32 query, 8 KV heads) read in one go
        _case("rope prompt 32k", "rope", 1, 32, 8, 32768, 32768),
        # one token of 8 conversations of 32K over uncompressed keys: the step that the tiered cache replaces
        _case("attention step b8 32k", "attention", 8, 32, 8, 1, 32768, ragged=1001),
        # one token of 16 conversations on a sliding-window layer with four sink tokens
        _case("attention step b16 span 4k", "attention", 16, 28, 4, 1, 16384, ragged=333, span=4096, sinks=4),
        # a prompt of 32K, full causal attention: the largest
        _case("attention prompt 32k", "attention", 1, 32, 8, 32768, 32768),
        # four 8K prompts on a sliding-window layer
        _case("attention prompt span 4k", "attention", 4, 32, 8, 8192, 8192, span=4096, sinks=4),
        # a padded batch of three prompts of unlike, odd lengths
        _case("attention prompt ragged", "attention", 3, 28, 4, 2047, 2047, ragged=700),
        # a chunk of 512 tokens appended to two contexts of 16K
        _case("attention chunk 512", "attention", 2, 32, 8, 512, 16384, ragged=77),
        # window scores of 8 prompts of 32K from the last 64 queries
        _case("scores 64 of 32k", "scores", 8, 32, 8, 64, 32768, ragged=500),
        # window scores from every query of an 8K prompt
        _case("scores all of 8k", "scores", 1, 32, 8, 8192, 8192),
        # a small model's layer with a narrow span and small windows
        _case("scores tiny", "scores", 1, 8, 2, 250, 2048, span=512, sinks=16, window=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the ranges above, whose work does not pass the largest listed one's."""
    op = rng.choice(["rope", "attention", "scores"])
    Hkv = rng.choice([2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 7]) if Hkv == 4 else Hkv * rng.choice([1, 3, 4])
    if op == "rope":
        B = _log(rng, 1, 16)
        n = _log(rng, 1, 32768 // B)
        return _case("", op, B, Hq, Hkv, n, n, norm=rng.random() < 0.5, far=rng.choice([0, 1000, 100000]))
    n_kv = _log(rng, 128, 32768)
    B = _log(rng, 1, max(1, min(16, 131072 // n_kv)))
    form = rng.choice(["step", "chunk", "prompt"])
    n_q = 1 if form == "step" else _log(rng, 2, min(n_kv, 512)) if form == "chunk" else min(n_kv, 16384 // B)
    n_kv = n_q if form == "prompt" else n_kv
    span = rng.choice([0, 0, _log(rng, 16, 8192)])
    sinks = rng.choice([0, 4, 100]) if span else 0
    return _case("", op, B, Hq, Hkv, n_q, n_kv, ragged=rng.randrange(0, max(1, n_kv // B)), span=span, sinks=sinks,
                 window=rng.choice([16, 32, 64, 128]))


def _lengths(case):
    """Keys and queries of each sequence of a padded batch (the queries are the last positions)."""
    kv = [max(1, case["n_kv"] - b * case["ragged"]) for b in range(case["B"])]
    return kv, [min(case["n_q"], n) for n in kv]


def prepare(case, seed):
    B, Hq, Hkv, n_q, n_kv = (case[k] for k in ("B", "Hq", "Hkv", "n_q", "n_kv"))
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case)
    if own:
        from tiered_kv_cache_decode_gb300 import binding
        s["cache"] = binding.TieredCache(B, 1, Hq, Hkv, case["window"], max(n_kv, 1), fp_capacity=1, ledger_capacity=1)
    if case["op"] == "rope":
        # what a fused projection gives: the heads of q, k and v side by side for each token
        s["qkv"] = (normal(B, n_q, Hq + 2 * Hkv, D) * 2).bfloat16()
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = first + torch.arange(n_q, device="cuda")
        s["wq"], s["wk"] = ((1 + 0.2 * normal(D)).bfloat16() if case["norm"] else None for _ in range(2))
        return s
    s["q"], s["k"], s["v"] = normal(B, n_q, Hq, D), normal(B, n_kv, Hkv, D), normal(B, n_kv, Hkv, D)
    s["k"] *= torch.where(torch.rand(Hkv, D, generator=g, device="cuda") < 0.01, 4.0, 1.0)   # outlier channels
    for x in "qkv":
        s[x] = s[x].bfloat16()
    s["kv_host"], s["q_host"] = _lengths(case)
    s["kv_len"], s["q_len"] = (torch.tensor(s[x], dtype=torch.int32).cuda() for x in ("kv_host", "q_host"))
    # the caller's buffers; rows past a sequence's queries are left as they were
    s["out"] = torch.zeros(B, n_q, Hq, D, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros(B, Hq, n_q, device="cuda")
    s["scores"] = torch.zeros(B, -(-n_kv // case["window"]), device="cuda")
    if case["op"] == "scores":   # the rows' log-sum-exps, which the attention before it gave
        _plain_attention(s, False)
        del s["v"]
    return s


def _plain_rope(s):
    B, n, Hq, Hkv = s["B"], s["n_q"], s["Hq"], s["Hkv"]
    angle = s["pos"].double()[:, :, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()

    def rotated(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).bfloat16()

    q, k, v = s["qkv"].split([Hq, Hkv, Hkv], 2)
    return rotated(q, s["wq"]), rotated(k, s["wk"]), v.contiguous()


def _chunks(s):
    """Chunks of the queries with the keys that any of them sees, so that the logits fit in memory."""
    B, n_q, n_kv, span = s["B"], s["n_q"], s["n_kv"], s["span"] or s["n_kv"]
    step = max(1, min(n_q, CHUNK // (B * s["Hq"] * min(n_kv, span + max(1, n_q // 8)))))
    shift = [a - b for a, b in zip(s["kv_host"], s["q_host"])]
    for i in range(0, n_q, step):
        e = min(n_q, i + step)
        lo, hi = max(0, min(shift) + i - span + 1), min(n_kv, max(shift) + e)
        j = torch.arange(lo, hi, device="cuda")
        first = min(s["sinks"], lo)
        yield i, e, torch.cat([torch.arange(first, device="cuda"), j]) if first else j


def _logits(s, kT, i, e, j):
    """fp32 [B][Hkv][e - i][G][keys j], -inf where query and key do not see each other, and the rows in use."""
    B, Hkv, G = s["B"], s["Hkv"], s["Hq"] // s["Hkv"]
    rows = s["q"][:, i:e].float().view(B, e - i, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    at = torch.arange(i, e, device="cuda")
    used = at < s["q_len"][:, None]
    pos = ((s["kv_len"] - s["q_len"])[:, None] + at)[:, :, None]
    seen = (j <= pos) & ((pos - j < (s["span"] or s["n_kv"])) | (j < s["sinks"])) & used[:, :, None]
    x = torch.matmul(rows, kT[..., j] if len(j) < kT.shape[-1] else kT).mul_(D ** -0.5).view(B, Hkv, e - i, G, -1)
    return x.masked_fill_(~seen[:, None, :, None], -math.inf), used


def _plain_attention(s, values=True):
    B, Hq, Hkv = s["B"], s["Hq"], s["Hkv"]
    kT = s["k"].float().permute(0, 2, 3, 1).contiguous()
    v = s["v"].float().permute(0, 2, 1, 3).contiguous() if values else None
    for i, e, j in _chunks(s):
        x, used = _logits(s, kT, i, e, j)
        top = x.amax(-1, keepdim=True).clamp_min(-3e38)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        lse = (top + total.log())[..., 0].permute(0, 1, 3, 2).reshape(B, Hq, e - i)
        s["lse"][:, :, i:e] = torch.where(used[:, None], lse, s["lse"][:, :, i:e])
        if values:
            o = torch.matmul(p.view(B, Hkv, -1, len(j)), v[:, :, j] if len(j) < v.shape[2] else v)
            o = (o.view(B, Hkv, e - i, -1, D) / total.clamp_min(1e-38)).permute(0, 2, 1, 3, 4).reshape(B, e - i, Hq, D)
            s["out"][:, i:e] = torch.where(used[:, :, None, None], o.bfloat16(), s["out"][:, i:e])
    return s["out"], s["lse"]


def _plain_scores(s):
    B, Hq, Hkv, w, W = s["B"], s["Hq"], s["Hkv"], s["window"], s["scores"].shape[1]
    kT = s["k"].float().permute(0, 2, 3, 1).contiguous()
    mass = torch.zeros(B, W * w, device="cuda")
    for i, e, j in _chunks(s):
        x, used = _logits(s, kT, i, e, j)
        lse = s["lse"][:, :, i:e].reshape(B, Hkv, -1, e - i).transpose(2, 3)
        mass[:, j] += x.sub_(lse[..., None]).exp_().sum((1, 2, 3)) / Hq
    s["scores"].copy_(mass.view(B, W, w).sum(-1))
    return s["scores"]


def run(s):
    if own:
        c = s["cache"]
        if s["op"] == "rope":
            q, k, v = s["qkv"].split([s["Hq"], s["Hkv"], s["Hkv"]], 2)
            return c.qk_norm_rope(0, q, k, s["inv_freq"], v=v, positions=s["pos"], q_weight=s["wq"],
                                  k_weight=s["wk"], eps=EPS)
        if s["op"] == "attention":
            return c.span_attention(0, s["q"], s["k"], s["v"], span=s["span"], sinks=s["sinks"], q_len=s["q_len"],
                                    kv_len=s["kv_len"], out=s["out"], lse=s["lse"])
        return c.span_scores(0, s["q"], s["k"], s["lse"], span=s["span"], sinks=s["sinks"], q_len=s["q_len"],
                             kv_len=s["kv_len"], out=s["scores"])
    if s["op"] == "rope":
        return _plain_rope(s)
    if s["op"] == "attention":
        return _plain_attention(s)
    return _plain_scores(s)


def _pairs(case):
    """(visible query-key pairs, keys that some query sees) of one head, summed over the sequences."""
    pairs = keys = 0
    for kv, q in zip(*_lengths(case)):
        span = case["span"] or kv
        p = np.arange(kv - q, kv, dtype=np.int64)
        pairs += int((np.minimum(p + 1, span) + np.minimum(case["sinks"], np.maximum(p + 1 - span, 0))).sum())
        lo = max(0, kv - q - span + 1)
        keys += kv - lo + min(case["sinks"], lo)
    return pairs, keys


def work(case):
    B, Hq, Hkv, n = case["B"], case["Hq"], case["Hkv"], case["n_q"]
    if case["op"] == "rope":
        rows = B * n * (Hq + 2 * Hkv)
        return {"bytes": rows * D * 4 + B * n * 8 + D * 6, "flops": B * n * (Hq + Hkv) * D * 8}
    pairs, keys = _pairs(case)
    rows = sum(_lengths(case)[1]) * Hq
    if case["op"] == "attention":
        return {"bytes": keys * Hkv * D * 4 + rows * (D * 4 + 4), "flops": 4 * D * Hq * pairs}
    return {"bytes": keys * Hkv * D * 2 + rows * (D * 2 + 4) + B * -(-case["n_kv"] // case["window"]) * 4,
            "flops": 2 * D * Hq * pairs}


def exact(case, seed):
    """The definitions in 64 bits, one (sequence, query head) at a time."""
    if case["op"] != "rope" and case["B"] * case["Hq"] * case["n_q"] * case["n_kv"] > 1.2e10:
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        Hq, Hkv = case["Hq"], case["Hkv"]
        x = s["qkv"].double()
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["pos"].double().unsqueeze(-1) * s["inv_freq"].double()).unsqueeze(2)
        res = []
        for y, w in ((x[:, :, :Hq], s["wq"]), (x[:, :, Hq:Hq + Hkv], s["wk"])):
            if w is not None:
                y = y / (y.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
            z = torch.complex(y[..., :D // 2].contiguous(), y[..., D // 2:].contiguous()) * turn
            res.append(torch.cat([z.real, z.imag], -1))
        return res[0], res[1], x[:, :, Hq + Hkv:]
    q, k, G = s["q"].double(), s["k"].double(), case["Hq"] // case["Hkv"]
    out, lse, scores = s["out"].double(), s["lse"].double(), s["scores"].double()
    w, W = case["window"], s["scores"].shape[1]
    for b in range(case["B"]):
        nk, nq = s["kv_host"][b], s["q_host"][b]
        p = torch.arange(nk - nq, nk, device="cuda").unsqueeze(1)
        j = torch.arange(nk, device="cuda").unsqueeze(0)
        seen = j <= p
        if case["span"]:
            seen = seen & ((j > p - case["span"]) | (j < case["sinks"]))
        for h in range(case["Hq"]):
            x = q[b, :nq, h] @ k[b, :nk, h // G].T / math.sqrt(D)
            x = torch.where(seen, x, -math.inf)
            if case["op"] == "scores":
                mass = (x - s["lse"][b, h, :nq].double().unsqueeze(1)).exp().sum(0) / case["Hq"]
                scores[b] += torch.nn.functional.pad(mass, (0, W * w - nk)).view(W, w).sum(1)
            else:
                lse[b, h, :nq] = x.logsumexp(1)
                out[b, :nq, h] = x.softmax(1) @ s["v"][b, :nk, h // G].double()
    return scores if case["op"] == "scores" else (out, lse)
