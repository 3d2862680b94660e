"""A query row of NaN over the paged cache: its output and its lse are NaN
wherever its keys are cut and masked, and the other rows keep their bits."""
import math

import pytest
import torch

from exact_blocked_attention_gb300 import blkattn

from test_gpu_paged import BF16, F32, call, dev, make

pytestmark = pytest.mark.gpu


def nan_rows_stay_nan(a, rows):
    """rows: (sequence, head, row) one after another."""
    want, want_lse = call(a)
    for b, h, i in rows:
        keep = a["q"][b, h, i].clone()
        a["q"][b, h, i] = math.nan
        out, lse = call(a)
        assert blkattn.check_device_error() == 0
        assert bool(torch.isnan(out[b, h, i]).all()), (b, h, i, out[b, h, i])
        assert bool(torch.isnan(lse[b, h, i])), (b, h, i, lse[b, h, i])
        rest = torch.ones(out.shape[:3], dtype=torch.bool, device=out.device)
        rest[b, h, i] = False
        assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])
        a["q"][b, h, i] = keep


# rows whose keys lie in a partly masked key tile only, and rows that also see
# whole ones; whole items and (with a table much longer than the sequences)
# items in parts
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("Tq,lens,entries", [(100, [100], None), (100, [100], 190), (300, [300, 700], 190),
                                             (300, [900, 301], None), (70, [3000, 70], 200)])
def test_prompt_rows(Tq, lens, entries, window, d):
    a = make(len(lens), 4, 2, Tq, d, 16, lens, BF16, seed=7, entries=entries)
    a["window"] = window
    last = len(lens) - 1
    nan_rows_stay_nan(a, [(0, 1, 0), (0, 1, 5), (last, 2, Tq - 1), (last, 3, Tq // 2)])


# units that one CTA finishes, that their last CTA folds (26 or more of them)
# and that a second kernel joins
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("B,Hq,Hkv,Tq,lens", [(1, 4, 1, 1, [40]), (4, 32, 8, 1, [3000, 2000, 3000, 100]),
                                              (1, 8, 2, 3, [3000]), (4, 64, 8, 5, [2500] * 4)])
def test_decode_rows(B, Hq, Hkv, Tq, lens, d):
    a = make(B, Hq, Hkv, Tq, d, 16, lens, BF16, seed=11)
    nan_rows_stay_nan(a, [(0, 0, 0), (B - 1, Hq - 1, Tq - 1), (B - 1, 1, 0)])


# up to 8 rows a KV head and more of them; rows in one split and in several,
# that end inside a key tile, on its edge and behind it
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("Hq,Hkv,Tq", [(2, 2, 1), (4, 2, 3), (8, 2, 3), (2, 1, 20), (4, 1, 60)])
@pytest.mark.parametrize("n,entries", [(60, None), (64, None), (65, 300), (900, None), (3001, None)])
def test_f32_rows(Hq, Hkv, Tq, n, entries, window, d):
    a = make(2, Hq, Hkv, Tq, d, 16, [n, 60], F32, seed=13, entries=entries)
    a["window"] = window
    nan_rows_stay_nan(a, [(0, 0, 0), (0, Hq - 1, Tq - 1), (1, 1, Tq // 2)])


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("n", [9, 64, 1000])
def test_bf16_rows_without_alignment(n, d):
    a = make(1, 4, 2, 3, d, 16, [n], BF16, seed=17)
    q = torch.zeros(1, 4, 3, d + 3, dtype=BF16, device=dev())[..., 1:d + 1]
    q.copy_(a["q"])
    nan_rows_stay_nan(dict(a, q=q), [(0, 0, 0), (0, 3, 2)])
