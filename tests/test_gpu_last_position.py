"""Query rows at the largest position there is (2^31 - 1, a row that sees the
whole cache) on every forward kernel: the same bits as at len - 1."""
import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Tq,d,dtype", [(8, 1, 128, torch.bfloat16), (8, 5, 128, torch.bfloat16),
                                           (4, 3, 64, torch.bfloat16), (2, 100, 128, torch.bfloat16),
                                           (4, 2, 64, torch.float32)])
def test_largest_position_sees_the_cache(Hq, Tq, d, dtype):
    torch.cuda.set_device(0)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(s, generator=g).to(dtype).cuda() for s in ((2, Hq, Tq, d), (2, 2, 300, d), (2, 2, 300, d)))
    lens = torch.tensor([300, 77], dtype=torch.int32, device="cuda")
    last = (lens[:, None] - 1).expand(2, Tq).contiguous()
    far = torch.full((2, Tq), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    want, want_lse = blkattn.attention(q, k, v, lens, last)
    out, lse = blkattn.attention(q, k, v, lens, far)
    assert blkattn.check_device_error() == 0
    assert bool((want_lse > -float("inf")).all())
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
