"""Argument checks of attention with a window (no GPU needed)."""
import ctypes

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from test_attention_abi import OK, _batch, _cache


def _paged(c, b, q=OK, qs=256, heads=4, scale=0.125, window=8, sinks=1, out=OK, ws=OK, wsb=1 << 40):
    return binding.load().dspark_attn_paged_window(q, qs, c and ctypes.byref(c), b and ctypes.byref(b), heads, scale, window,
                                                   sinks, out, None, ws, wsb, None)


def _prompt(q=OK, k=OK, v=OK, qs=256, ks=128, vs=128, off=OK, B=2, T=5, heads=4, kv=2, dim=64, scale=0.125, window=8, sinks=1,
            out=OK, ws=OK, wsb=1 << 40):
    return binding.load().dspark_attn_prompt_window(q, k, v, qs, ks, vs, off, B, T, heads, kv, dim, scale, window, sinks, out,
                                                    None, ws, wsb, None)


def test_windows_and_sinks_are_checked():
    c, b = _cache(), _batch()
    for kw in (dict(window=0), dict(window=-1), dict(window=-2 ** 31), dict(sinks=-1), dict(sinks=-2 ** 31)):
        assert _paged(c, b, **kw) == -1 and _prompt(**kw) == -1, kw
        assert _paged(c, _batch(T=0), **kw) == -1 and _prompt(T=0, **kw) == -1, kw
    # more places than positions of a window can be told apart, unless it covers them all
    big = _batch(max_pages=(1 << 26) + 1)
    assert _paged(c, big, window=1 << 30) == -3
    assert _paged(c, big, window=2 ** 31 - 1) == -1                   # no device memory
    assert _paged(c, _batch(max_pages=1 << 26), window=5) == -1


def test_the_rest_is_checked_as_without_one():
    c, b = _cache(), _batch()
    assert _paged(None, b) == -1 and _paged(c, None) == -1
    assert _paged(_cache(dtype=7), b) == -2 and _paged(_cache(page=48), b) == -3 and _paged(c, _batch(R=0)) == -3
    for kw in (dict(q=None), dict(out=None), dict(q=OK + 8), dict(qs=260), dict(scale=float("nan"))):
        assert _paged(c, b, **kw) == -1, kw
        assert _prompt(**kw) == -1, kw
    for kw in (dict(heads=3), dict(heads=258, qs=1 << 20)):
        assert _paged(c, b, **kw) == -3 and _prompt(**kw) == -3, kw
    for kw in (dict(ws=None), dict(ws=OK + 16), dict(wsb=100)):
        assert _paged(c, b, **kw) == -8 and _prompt(**kw) == -8, kw
    assert _paged(c, _batch(T=0, q_off=None, kv_len=None, page_table=None)) == 0
    assert _prompt(T=0, q=None, k=None, v=None, off=None, out=None, ws=None) == 0
    assert _paged(c, b) == -1 and _prompt() == -1                     # no device memory


def test_binding():
    assert binding._window(None, 0) == () and binding._window(5, 0) == (5, 0)
    assert binding._window(1 << 40, 1 << 33) == (2 ** 31 - 1, 2 ** 31 - 1) and binding._window(-3, 2) == (-3, 2)
    with pytest.raises(ValueError, match="go with a window"):
        binding._window(None, 4)
    with pytest.raises(ValueError, match="go with a window"):
        q = torch.zeros((5, 4, 64), dtype=torch.bfloat16)
        from test_attention_abi import _Cuda
        off = torch.zeros(2, dtype=torch.int32)
        binding.attn_prompt(_Cuda(q), _Cuda(q[:, :2]), _Cuda(q[:, :2]), off, sinks=1, ws=_Cuda(off), out=dict(out=_Cuda(q)))
