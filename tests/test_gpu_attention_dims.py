"""Heads without channels are refused as any other size that is none of those taken."""
import pytest

from test_gpu_attention import BF16, ints, say, tq  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_heads_without_channels(tq):
    say("no channels")
    x = torch.empty((3, 2, 0), dtype=BF16, device="cuda")
    cache = torch.empty((4, 2, 16, 0), dtype=BF16, device="cuda")
    space = torch.empty(4096, dtype=torch.uint8, device="cuda")
    for kw in ({}, {"workspace": space}):
        with pytest.raises(tq.MoeError, match="head_dim 0"):
            tq.attention_prefill(x, x, x, ints([0, 3]), **kw)
        with pytest.raises(tq.MoeError):
            tq.attention_decode(x, cache, cache, ints([[0]] * 3), ints([1] * 3), **kw)
