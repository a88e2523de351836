"""Windows and sinks outside the ABI's 32 bits are not taken for others (no GPU needed)."""
import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from test_attention_abi import _Cuda


@pytest.mark.parametrize("n", [-(1 << 31), -(1 << 31) - 1, -(1 << 32) + 5, -(1 << 40) + 1024])
def test_below_32_bits(n, monkeypatch):
    """Taken modulo 2^32, -2^32 + 5 would be a window of 5."""
    assert binding._window(n, 0) == (-(1 << 31), 0) and binding._window(5, n) == (5, -(1 << 31))
    monkeypatch.setattr(binding, "_stream", lambda s=None: 0)
    q = _Cuda(torch.zeros((5, 4, 64), dtype=torch.bfloat16))
    off = _Cuda(torch.tensor([0, 5], dtype=torch.int32))
    for kw in (dict(window=n), dict(window=5, sinks=n)):
        with pytest.raises(binding.DsparkError) as e:
            binding.attn_prompt(q, q, q, off, ws=off, out=dict(out=q), **kw)
        assert e.value.code == -1


def test_inside_and_above():
    assert binding._window(7, 3) == (7, 3) and binding._window(1 << 31, 1 << 31) == (0x7FFFFFFF, 0x7FFFFFFF)
