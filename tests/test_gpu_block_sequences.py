"""Random runs of calls on the cache in 8 bits against a plain model, bit by bit: chunks of any sizes, sequences set back
as far as the header allows, evictions in place and into another layer, ragged batches in which some sequences rest."""
import random

import numpy as np
import pytest
import torch

import block_util as U
from tiered_kv_cache_decode_gb300 import binding

pytestmark = pytest.mark.gpu
D, T = 128, 64


class Sequence:
    """Rows of all KV heads, [Hkv][n][128] fp32: what full blocks stand for, the last full block's rows, the open ones."""

    def __init__(self, Hkv, fmt):
        self.fmt, self.least = fmt, 0
        self.closed, self.last, self.open = (np.zeros((Hkv, 0, D), np.float32) for _ in range(3))

    def __len__(self):
        return self.closed.shape[1] + self.open.shape[1]

    def lowest(self):
        """how far back it may be set: within the last full block, if its rows are there"""
        return max(self.least, self.closed.shape[1] - self.last.shape[1])

    def append(self, rows, start):
        c = self.closed.shape[1]
        if start < c:
            self.closed, self.open = self.closed[:, :c - T], self.last[:, :start - (c - T)]
            self.last = self.last[:, :0]
        else:
            self.open = self.open[:, :start - c]
        x = np.concatenate([self.open, rows], 1)
        full = x.shape[1] // T * T
        if full:
            self.closed = np.concatenate([self.closed, U.held(x[:, :full], self.fmt)], 1)
            self.last = x[:, full - T:full]
        self.open = x[:, full:]

    def evict(self, at):
        self.closed = U.held(np.stack([self.closed[h, a] for h, a in enumerate(at)]), self.fmt)
        self.last = self.last[:, :0]
        self.least = self.closed.shape[1]

    def values(self):
        return torch.from_numpy(np.concatenate([self.closed, self.open], 1)).bfloat16().transpose(0, 1)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("seed", range(5))
def test_random_calls(fmt, seed):
    rng = random.Random(100 * seed + len(fmt))
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, cap = rng.choice([1, 3, 5]), rng.choice([1, 2, 3]), 1024
    c = binding.BlockCache(B, 2, Hkv, Hkv, cap, fmt)
    layer, model = 0, {s: [Sequence(Hkv, fmt) for _ in range(B)] for s in "kv"}
    weights = torch.zeros(B, Hkv, cap, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()   # noqa: E731
    for step in range(60):
        lens = [len(s) for s in model["k"]]
        op = rng.choice(["append"] * 6 + ["back"] * 3 + ["evict", "evict into"])
        if op in ("append", "back"):
            start = [rng.randint(s.lowest(), len(s)) if op == "back" and rng.random() < 0.7 else len(s) for s in model["k"]]
            n = rng.choice([1, 1, 2, rng.randint(1, 70), rng.randint(60, 200)])
            n_new = [max(0, min(rng.choice([n, n, rng.randint(0, n)]), cap - s)) for s in start]
            k, v = (torch.randn(B, n, Hkv, D, generator=g, device="cuda").bfloat16() * 2.0 ** rng.randint(-3, 3) for _ in "kv")
            c.append(layer, k, v, start=ints(start), n_new=ints(n_new))
            for b in range(B):
                if n_new[b] == 0:
                    continue   # rests; also not set back
                for s, t in (("k", k), ("v", v)):
                    model[s][b].append(t[b, :n_new[b]].float().cpu().numpy().transpose(1, 0, 2), start[b])
        else:
            keep = T * rng.randint(1, 8)
            recent = rng.choice([0, keep, rng.randint(0, keep)])
            weights.copy_(torch.rand(weights.shape, generator=g, device="cuda").mul(50).round())
            w = weights.cpu().numpy()
            to = layer if op == "evict" else 1 - layer
            new_len, kept = c.evict(layer, ints(lens), keep, recent, weights, into=None if to == layer else c, into_layer=to)
            kept = kept.cpu().numpy()
            for b, L in enumerate(lens):
                full = L // T * T
                at = [U.select(w[b, h], full, keep, recent) for h in range(Hkv)]
                assert all(np.array_equal(kept[b, h, :len(a)], a) and np.all(kept[b, h, len(a):] == -1) for h, a in enumerate(at))
                assert int(new_len[b]) == len(at[0]) + L - full
                for s in "kv":
                    if to != layer or full > keep:
                        model[s][b].evict(at)
            layer = to
        lens = [len(s) for s in model["k"]]
        got = c.read(layer, ints(lens), max(max(lens), 1))
        for s, t in zip("kv", got):
            for b, L in enumerate(lens):
                assert torch.equal(t[b, :L].cpu(), model[s][b].values()), (step, op, s, b, L)
    assert c.status() == 0, c.last_error()
