"""The binding on a stream other than the current one, as far as the host
shows it.  No GPU."""
import torch

from exact_blocked_attention_gb300 import blkattn


class Recorder:
    """Stands in for the marshalling extension."""

    def __init__(self):
        self.args = None

    def append(self, *args):
        self.args = args
        return 0, args[10]


def test_append_leaves_its_missing_output_to_the_call_s_stream(monkeypatch):
    # a fill here would go to torch's current stream, which nothing orders
    # with the given one
    rec = Recorder()
    monkeypatch.setattr(blkattn, "_bind", rec)
    for name in ("zeros_like", "zeros", "empty_like", "empty"):
        monkeypatch.setattr(torch, name, lambda *a, **k: (_ for _ in ()).throw(AssertionError("allocated on the current stream")))
    x = torch.ones(1, 1, 1, 64)
    blkattn.paged_append(x, x, x, x, x, x, q=x, stream=12345)
    assert rec.args[9] is x and rec.args[10] is None and rec.args[11] == 12345
