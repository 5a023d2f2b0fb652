"""64-bit attention of one KV head over given values, on the GPU, for contexts that are long for numpy, and what an output
of the cache in 8 bits may be off by."""
import math

import torch

STEP = 2.0 ** -8        # half a step of a bf16 output, relative
HALF = 2.0 ** -11       # half a step of a probability in fp16, relative
LEAST = 2.0 ** -40      # what a probability below fp16's normal numbers is off by, of the largest
TINY = 2.0 ** -133      # the least step of bf16, which takes in what fp32 sums of subnormal numbers are off by


def head(q, k, v):
    """q [n_q][G][128], k, v [n][128] (any type): out [n_q][G][128], lse [n_q][G], weights [n], and what the tolerances
    need: sum p |v|, sum |v| relative to the largest probability, the largest sum |q k| / sqrt(128)."""
    q, k, v = (x.double().cuda() for x in (q, k, v))
    n_q, n = q.shape[0], k.shape[0]
    x = torch.einsum("igd,jd->igj", q, k) / math.sqrt(q.shape[2])
    hidden = torch.arange(n, device="cuda") > (n - n_q + torch.arange(n_q, device="cuda"))[:, None]
    x.masked_fill_(hidden[:, None], -math.inf)
    lse = x.logsumexp(-1)
    p = torch.where(torch.isneginf(lse)[..., None], 0.0, (x - lse[..., None]).exp())
    top = p.amax(-1, keepdim=True)
    low = torch.where(hidden[:, None], 0.0, torch.ones_like(x)) @ v.abs() * top
    big = (torch.einsum("igd,jd->igj", q.abs(), k.abs()).amax() / math.sqrt(q.shape[2])).item() if n else 0.0
    return p @ v, lse, p.mean(1).sum(0), p @ v.abs(), low, big


def check(q, k, v, out, lse, weights=None, sums=2.0 ** -13):
    """Hold one head's results to 64 bits. `sums`: what fp32 sums are off by, of sum p |v|: 2^-23 for each term of the
    longest chain of additions (64 tokens of a block, then the blocks of a run, then the parts of a warp), of the output
    and of the row's sum."""
    want, wl, ww, mag, low, big = head(q, k, v)
    out, lse = out.double(), lse.double()
    off = 2.0 ** -20 * big   # of a logit: 128 products added in fp32
    assert torch.isfinite(out).all()
    allowed = STEP * want.abs() + (HALF + 2 * off + sums) * mag + LEAST * low + TINY
    worst = ((out - want).abs() / allowed).max().item()
    assert worst <= 1, worst
    seen = torch.isfinite(wl)
    assert torch.equal(torch.isfinite(lse), seen) and torch.isneginf(lse[~seen]).all()
    slack = 1e-5 + 2.0 ** -22 * wl[seen].abs() + off
    assert torch.all((lse[seen] - wl[seen]).abs() <= slack)
    if weights is not None:
        rel = 2 * off + 2.0 ** -20 + 2.0 ** -22 * (wl[seen].abs().max().item() if seen.any() else 0.0) + 2e-5
        assert torch.all((weights.double() - ww).abs() <= rel * ww + 1e-30)
