"""A cache in 8 bits that goes while calls on a side stream are still waiting to run (its memory is not used again before
they have), or while another stream is captured."""
import pytest
import torch

from tiered_kv_cache_decode_gb300 import binding

pytestmark = pytest.mark.gpu
D = 128


def test_a_cache_that_goes_with_work_on_its_way():
    B, Hq, Hkv, n = 2, 8, 2, 4000
    g = torch.Generator().manual_seed(1)
    k, v, q = (torch.randn(B, m, h, D, generator=g).bfloat16().cuda() for m, h in ((n, Hkv), (n, Hkv), (1, Hq)))
    kv_len = torch.tensor([n, n - 77], dtype=torch.int32).cuda()
    results = []
    for side in (torch.cuda.current_stream(), torch.cuda.Stream()):
        c = binding.BlockCache(B, 1, Hq, Hkv, n)
        side.wait_stream(torch.cuda.current_stream())
        busy = torch.randn(4096, 4096, device="cuda")
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            for _ in range(40):   # some milliseconds before the calls
                busy = (busy @ busy).clamp(-1, 1)
        c.append(0, k, v, n_new=kv_len, stream=side)
        out, lse = c.attend(0, q, kv_len, stream=side)
        kr, vr = c.read(0, kv_len, n, stream=side)
        bytes_held = B * Hkv * 2 * (n + 63) // 64 * 64 * D
        del c
        # what the allocator gives out now may be the cache's memory
        others = [torch.full((bytes_held,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        results.append((out, lse, kr, vr))
        del others, busy
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("torch_allocator", [True, False])
def test_a_cache_may_go_while_another_stream_is_captured(torch_allocator):
    """Closing one in the middle of a capture does not end that."""
    old, c = (binding.BlockCache(1, 1, 4, 1, 256, torch_allocator=torch_allocator) for _ in range(2))
    k = torch.randn(1, 200, 1, D, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    lens = torch.tensor([200], dtype=torch.int32).cuda()
    k_out, v_out = (torch.zeros(1, 200, 1, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    old.append(0, k, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.append(0, k, k)
        old.close()
        c.read(0, lens, 200, k_out=k_out, v_out=v_out)
    graph.replay()
    torch.cuda.synchronize()
    assert k_out[:, 192:].equal(k[:, 192:]) and k_out.equal(v_out) and k_out[:, :192].any() and c.status() == 0


def test_a_cache_of_a_side_stream_may_go_while_another_is_captured():
    """The wait for the side stream joins nothing to the capture, and its memory is not used before its work is done."""
    n = 4000
    k = torch.randn(2, n, 2, D, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    lens = torch.full((2,), n, dtype=torch.int32).cuda()
    side, x = torch.cuda.Stream(), torch.zeros(8, device="cuda")
    want = None
    for closes in (False, True):
        c = binding.BlockCache(2, 1, 4, 2, n)
        busy = torch.randn(4096, 4096, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            for _ in range(40):
                busy = (busy @ busy).clamp(-1, 1)
        c.append(0, k, k, stream=side)
        got = c.read(0, lens, n, stream=side)
        if closes:
            with torch.cuda.graph(graph):
                x += 1
                c.close()
                x += 1
            graph.replay()
        others = [torch.full((c.B * c.Hkv * 2 * c.capacity * D,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del others
    assert torch.all(x == 2)
