"""Calls of the operators between projections and the cache that their documentation allows and that stand apart
from the usual ones: lengths outside their range, more queries than keys, no log-sum-exps, a layer other than the
first, one token without a token dimension, and a process whose first calls are captured into a graph. Against
the plain 64-bit forms, with the tolerances of the outputs' types (bf16 2^-8 once for the output and once for the
probabilities; fp32 sums 1e-5), or bit by bit against the same call in its usual form."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import span_util as U
from tiered_kv_cache_decode_gb300 import binding

pytestmark = pytest.mark.gpu
D = 128
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True, scope="module")
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tiered_kv_cache_decode_gb300 import build
    build.build()
    binding.load()


def cache_for(B, Hq, Hkv, w=64, layers=1, **kw):
    return binding.TieredCache(B, layers, Hq, Hkv, w, 4096, fp_capacity=1, ledger_capacity=1, **kw)


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def f64(t):
    return t.detach().cpu().double().numpy()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("B,Hq,Hkv,n", [(4, 8, 2, 300), (4, 20, 20, 700)])   # split, wide
def test_lengths_outside_their_range(B, Hq, Hkv, n):
    q, k, v = rand(1, B, n, Hq, D).cuda(), rand(2, B, n, Hkv, D).cuda(), rand(3, B, n, Hkv, D).cuda()
    cache = cache_for(B, Hq, Hkv)
    got = []
    for lens in (dict(q_len=ints(-5, n + 1, 2 ** 31 - 1, 7), kv_len=ints(n, 2 ** 31 - 1, n + 9, -2 ** 31)),
                 dict(q_len=ints(0, n, n, 7), kv_len=ints(n, n, n, 0))):
        out, lse = torch.zeros_like(q), torch.zeros(B, Hq, n, device="cuda")
        cache.span_attention(0, q, k, v, out=out, lse=lse, **lens)
        got.append((out, lse, cache.span_scores(0, q, k, lse, **lens)))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and cache.status() == 0
    assert torch.all(torch.isneginf(got[0][1][3, :, :7])) and torch.all(got[0][2][3] == 0)


@pytest.mark.parametrize("B,Hq,Hkv,n_q,n_kv,span,sinks", [
    (1, 8, 2, 500, 200, 0, 0), (2, 7, 1, 300, 1, 0, 0), (3, 28, 4, 1000, 900, 100, 3)])
def test_more_queries_than_keys(B, Hq, Hkv, n_q, n_kv, span, sinks):
    q, k, v = rand(1, B, n_q, Hq, D), rand(2, B, n_kv, Hkv, D), rand(3, B, n_kv, Hkv, D)
    cache = cache_for(B, Hq, Hkv)
    out, lse = cache.span_attention(0, q.cuda(), k.cuda(), v.cuda(), span=span, sinks=sinks)
    ref, rl = U.attention(f64(q), f64(k), f64(v), [n_q] * B, [n_kv] * B, span, sinks)
    mag, _ = U.attention(f64(q), f64(k), np.abs(f64(v)), [n_q] * B, [n_kv] * B, span, sinks)
    assert np.all(np.abs(f64(out) - ref) <= 2.0 ** -8 * (np.abs(ref) + mag) + 1e-5)
    seen = np.isfinite(rl)
    assert np.array_equal(seen, np.isfinite(f64(lse)))
    assert np.all(np.abs(f64(lse)[seen] - rl[seen]) <= 1e-5 + 1e-6 * np.abs(rl[seen]))
    got = cache.span_scores(0, q.cuda(), k.cuda(), lse, span=span, sinks=sinks)
    want = U.scores(f64(q), f64(k), f64(lse), [n_q] * B, [n_kv] * B, span, sinks, 64)
    assert np.all(np.abs(f64(got) - want) <= 1e-5 * want + 1e-9)
    assert cache.status() == 0, cache.last_error()


@pytest.mark.parametrize("B,Hq,Hkv,n", [(1, 8, 2, 300), (4, 20, 20, 700)])
def test_no_log_sum_exps_other_layers_and_one_token(B, Hq, Hkv, n):
    cache = cache_for(B, Hq, Hkv, layers=3)
    q, k, v = rand(1, B, n, Hq, D).cuda(), rand(2, B, n, Hkv, D).cuda(), rand(3, B, n, Hkv, D).cuda()
    out, lse = cache.span_attention(0, q, k, v)
    bare, none = cache.span_attention(2, q, k, v, want_lse=False)
    assert none is None and torch.equal(bare, out)
    assert torch.equal(cache.span_scores(2, q, k, lse), cache.span_scores(0, q, k, lse))
    last = q[:, -1].contiguous()
    one, l1 = cache.span_attention(1, last, k, v)
    same, l2 = cache.span_attention(1, last[:, None], k, v)
    assert one.shape == last.shape and torch.equal(one, same[:, 0]) and torch.equal(l1, l2)
    assert torch.equal(cache.span_scores(1, last, k, l1), cache.span_scores(1, last[:, None], k, l2))
    assert cache.status() == 0, cache.last_error()


FIRST = """
import torch
from tiered_kv_cache_decode_gb300 import binding
B, Hq, Hkv, n, D = %s
g = torch.Generator().manual_seed(1)
x = torch.randn(B, n, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
inv = (10000.0 ** (-torch.arange(0, D, 2) / D)).cuda()
cache = binding.TieredCache(B, 1, Hq, Hkv, 64, n, fp_capacity=1, ledger_capacity=1)
pos = torch.arange(n).expand(B, n).contiguous().cuda()

def layer():
    q, k, v = x.split([Hq, Hkv, Hkv], 2)
    q, k, v = cache.qk_norm_rope(0, q, k, inv, v=v, positions=pos)
    out, lse = cache.span_attention(0, q, k, v)
    return q, k, out, lse, cache.span_scores(0, q, k, lse)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = layer()
graph.replay()
torch.cuda.synchronize()
want = layer()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and cache.status() == 0
print("same bits")
"""


@pytest.mark.parametrize("sizes", [(1, 8, 2, 900, 128), (4, 20, 20, 700, 128)])
def test_first_calls_of_a_process_are_captured(sizes):
    r = subprocess.run([sys.executable, "-c", FIRST % (sizes,)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stdout + r.stderr
