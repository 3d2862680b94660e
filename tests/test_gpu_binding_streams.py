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


def rope_call(seed=3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, 8, 100, 64, generator=g).to(dev())
    pos = torch.arange(100, dtype=torch.int32, device=dev()).repeat(2, 1)
    ph = blkattn.rope_phases(blkattn.rope_angles(64)[0])
    return lambda **kw: (blkattn.rope(x, pos, ph, **kw),)


def rope_backward_call(seed=4):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, 8, 100, 64, generator=g).to(dev())
    pos = torch.arange(100, dtype=torch.int32, device=dev()).repeat(2, 1)
    ph = blkattn.rope_phases(blkattn.rope_angles(64)[0])
    return lambda **kw: (blkattn.rope_backward(x, pos, ph, **kw),)


def paged_call(seed=5):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(2, 8, 30, 64, generator=g).to(dev())
    kp, vp = (torch.randn(20, 2, 16, 64, generator=g).to(dev()) for _ in range(2))
    table = torch.randperm(20, generator=g).to(torch.int32).reshape(2, 10).to(dev())
    lens = torch.full((2,), 150, dtype=torch.int32, device=dev())
    pos = torch.arange(120, 150, dtype=torch.int32, device=dev()).repeat(2, 1)
    return lambda **kw: blkattn.attention_paged(q, kp, vp, table, lens, pos, **kw)


def contiguous_call(seed=6):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(2, 8, 30, 64, generator=g).to(dev())
    k, v = (torch.randn(2, 2, 150, 64, generator=g).to(dev()) for _ in range(2))
    lens = torch.full((2,), 150, dtype=torch.int32, device=dev())
    pos = torch.arange(120, 150, dtype=torch.int32, device=dev()).repeat(2, 1)
    return lambda **kw: blkattn.attention(q, k, v, lens, pos, **kw)


def backward_call(seed=7):
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(1, 2, 130, 128, generator=g).to(BF16).to(dev()) for _ in range(4))
    lens = torch.full((1,), 130, dtype=torch.int32, device=dev())
    pos = torch.arange(130, dtype=torch.int32, device=dev()).repeat(1, 1)
    out, lse = blkattn.attention(q, k, v, lens, pos)
    return lambda **kw: blkattn.attention_backward(q, k, v, lens, pos, out, lse, do, **kw)


def sample_call(seed=8):
    g = torch.Generator().manual_seed(seed)
    p, q = (torch.softmax(torch.randn(4, n, 500, generator=g), -1).to(dev()) for n in (4, 3))
    draft = torch.randint(0, 500, (4, 3), generator=g).to(torch.int32).to(dev())
    ua = torch.rand(4, 3, generator=g).to(dev())
    us = torch.randint(-2 ** 31, 2 ** 31, (4,), generator=g).to(torch.int32).to(dev())
    return lambda **kw: blkattn.spec_sample(p, q, draft, ua, us, **kw)


CALLS = [rope_call, rope_backward_call, paged_call, contiguous_call, backward_call, sample_call]


@pytest.mark.parametrize("problem", CALLS)
def test_outputs_are_not_memory_that_the_current_stream_still_uses(problem):
    call = problem()
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy = [torch.empty_like(t) for t in want]
    lag()
    for t in busy:
        t.fill_(7.0)  # queued behind the lag
    del busy, t       # free for the current stream, not for another
    got = call(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("problem", CALLS)
def test_outputs_are_kept_for_the_current_stream_s_reads(problem):
    first, second = problem(), problem(seed=77)
    want = [t.clone() for t in first()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = first(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    lag()
    read = [t.clone() for t in got]  # queued behind the lag
    del got
    later = second(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want))
    assert all(torch.equal(a, b) for a, b in zip(later, second()))


@pytest.mark.parametrize("problem", CALLS)
def test_special_stream_handles(problem):
    call = problem()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for handle in (0, 1, side.cuda_stream):  # the default stream by both its handles, and the current one
            got = call(stream=handle)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        with pytest.raises(ValueError, match="per-thread"):  # no torch stream stands for it
            call(stream=2)
