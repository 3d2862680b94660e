"""Calls of the binding on a stream that is not torch's current one, while the
current one lags behind: what a call allocates and fills belongs to the call's
stream.  The lag is a timed device sleep."""
import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def dev():
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def lag():
    torch.cuda._sleep(100_000_000)  # (some 50 ms)


def append_problem(T=33, seed=1):
    g = torch.Generator().manual_seed(seed)
    k, v, q = (torch.randn(2, h, T, 64, generator=g).to(BF16).to(dev()) for h in (2, 2, 8))
    pos = torch.arange(T, dtype=torch.int32).repeat(2, 1)
    pos[1, T - 5:] = -1  # padding
    table = torch.randperm(10, generator=g).to(torch.int32).reshape(2, 5)
    pools = [torch.zeros(10, 2, 16, 64, dtype=BF16, device=dev()) for _ in range(2)]
    phases = blkattn.rope_phases(blkattn.rope_angles(64)[0])
    return (k, v, pos.to(dev()), table.to(dev()), *pools), dict(phases=phases, q=q)


def test_append_without_q_out():
    a, kw = append_problem()
    want = blkattn.paged_append(*a, **kw)
    assert bool((want[1, :, -5:] == 0).all()) and bool((want[0].abs().amax(-1) > 0).all())
    junk = torch.full_like(want, 7.0)  # (memory that the next allocation may take)
    del junk
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    lag()
    out = blkattn.paged_append(*a, stream=s, **kw)
    with torch.cuda.stream(s):
        early = out.clone()  # the call does not wait for the current stream
    s.synchronize()
    assert torch.equal(early, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want)  # and nothing lands in it afterwards
    assert blkattn.paged_append(*a, phases=kw["phases"], stream=s) is None
    torch.cuda.synchronize()
    again = torch.empty_like(want)
    assert blkattn.paged_append(*a, q_out=again, stream=s.cuda_stream, **kw) is again
