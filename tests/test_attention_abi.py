"""Argument checks of the cache and attention entry points (no GPU needed):
every refusal comes before anything is enqueued."""
import ctypes

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding

OK = 1 << 20                  # 256-byte aligned, never dereferenced


def _cache(**kw):
    a = dict(k=OK, v=OK, k_scale=None, v_scale=None, dtype=binding.BF16, n_pages=4, page=16, n_kv_heads=2, head_dim=64)
    a.update(kw)
    return binding._Cache(*(a[n] for n, _ in binding._Cache._fields_))


def _batch(**kw):
    a = dict(q_off=OK, kv_len=OK, page_table=OK, R=2, max_pages=3, T=5)
    a.update(kw)
    return binding._Batch(*(a[n] for n, _ in binding._Batch._fields_))


def _write(c, b, K=OK, V=OK, ks=128, vs=128, ws=OK, wsb=1 << 30):
    return binding.load().dspark_kv_write(c and ctypes.byref(c), b and ctypes.byref(b), K, V, ks, vs, ws, wsb, None)


def _read(c, b, K=OK, V=OK, ws=OK, wsb=1 << 30):
    return binding.load().dspark_kv_read(c and ctypes.byref(c), b and ctypes.byref(b), K, V, ws, wsb, None)


def _paged(c, b, q=OK, qs=256, heads=4, scale=0.125, out=OK, ws=OK, wsb=1 << 40):
    return binding.load().dspark_attn_paged(q, qs, c and ctypes.byref(c), b and ctypes.byref(b), heads, scale, out,
                                            None, ws, wsb, None)


def _prompt(q=OK, k=OK, v=OK, qs=256, ks=128, vs=128, off=OK, B=2, T=5, heads=4, kv=2, dim=64, scale=0.125, out=OK,
            ws=OK, wsb=1 << 40):
    return binding.load().dspark_attn_prompt(q, k, v, qs, ks, vs, off, B, T, heads, kv, dim, scale, out, None, ws, wsb,
                                             None)


@pytest.mark.parametrize("call", [_write, _read, _paged])
def test_cache_and_batch_are_checked(call):
    assert call(None, _batch()) == -1
    assert call(_cache(), None) == -1
    assert call(_cache(dtype=binding.F32), _batch()) == -2
    assert call(_cache(dtype=7), _batch()) == -2
    for kw in (dict(head_dim=96), dict(head_dim=0), dict(n_pages=0), dict(page=8), dict(page=48), dict(page=512),
               dict(n_kv_heads=0), dict(n_kv_heads=4097)):
        assert call(_cache(**kw), _batch()) == -3, kw
    for kw in (dict(k=None), dict(v=None), dict(k=OK + 8), dict(v=OK + 2), dict(dtype=binding.E4M3),
               dict(dtype=binding.E4M3, k_scale=OK), dict(dtype=binding.E4M3, k_scale=OK, v_scale=OK + 4)):
        assert call(_cache(**kw), _batch()) == -1, kw
    for kw in (dict(R=0), dict(max_pages=0), dict(T=-1)):
        assert call(_cache(), _batch(**kw)) == -3, kw
    for kw in (dict(q_off=None), dict(page_table=None)):
        assert call(_cache(), _batch(**kw)) == -1, kw
    assert call(_cache(), _batch(T=0, q_off=None, kv_len=None, page_table=None)) == 0       # nothing to do
    for kw in (dict(ws=None), dict(ws=OK + 16), dict(wsb=255)):
        assert call(_cache(), _batch(), **kw) == -8, kw
    # an address that is no device memory of the current device
    assert call(_cache(), _batch()) == -1


def test_rows_strides_and_heads_are_checked():
    c, b = _cache(), _batch()
    for kw in (dict(K=None), dict(V=None), dict(K=OK + 4), dict(ks=120), dict(vs=132), dict(ks=-128)):
        assert _write(c, b, **kw) == -1, kw
    assert _write(c, _batch(kv_len=None)) == -1
    for kw in (dict(K=None), dict(V=OK + 8)):
        assert _read(c, b, **kw) == -1, kw
    for kw in (dict(q=None), dict(out=None), dict(q=OK + 8), dict(out=OK + 2), dict(qs=248), dict(qs=260),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _paged(c, b, **kw) == -1, kw
    assert _paged(c, _batch(kv_len=None)) == -1
    for heads in (0, 3, -2, 2 * 129):
        assert _paged(c, b, heads=heads, qs=1 << 20) == -3, heads
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(off=None), dict(out=None), dict(q=OK + 2), dict(k=OK + 8),
               dict(v=OK + 4), dict(qs=252), dict(ks=64), dict(vs=130), dict(scale=float("inf"))):
        assert _prompt(**kw) == -1, kw
    for kw in (dict(B=0), dict(T=-1), dict(heads=3), dict(kv=0), dict(dim=80), dict(heads=2 * 129)):
        assert _prompt(**kw) == -3, kw
    for kw in (dict(ws=None), dict(ws=OK + 8), dict(wsb=100)):
        assert _prompt(**kw) == -8, kw
    assert _prompt(T=0, q=None, k=None, v=None, off=None, out=None, ws=None) == 0
    assert _prompt() == -1                                            # no device memory


def test_workspace_sizes():
    L = binding.load()
    assert L.dspark_kv_workspace_size() == 256
    for size in (L.dspark_attn_paged_workspace_size, L.dspark_attn_prompt_workspace_size):
        assert size(4, 5, 8, 2, 128) >= 256
        for bad in ((0, 5, 8, 2, 128), (4, -1, 8, 2, 128), (4, 5, 7, 2, 128), (4, 5, 8, 0, 128), (4, 5, 8, 2, 96),
                    (4, 5, 258, 2, 64)):
            assert size(*bad) == 0, bad


def test_binding_checks_shapes_before_any_launch():
    bf = torch.bfloat16
    k = torch.zeros((4, 2, 16, 64), dtype=bf)
    with pytest.raises(TypeError, match="cache"):
        binding.KvCache(k.float(), k.float())
    with pytest.raises(ValueError, match="v must"):
        binding.KvCache(k, k[:3])
    with pytest.raises(ValueError, match="k_scale"):
        binding.KvCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn))
    with pytest.raises(ValueError, match="v_scale"):
        binding.KvCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn), torch.zeros(4, 2, 16), torch.zeros(4, 2, 8))
    with pytest.raises(ValueError, match="scale"):
        binding.KvCache(k, k, torch.zeros(4, 2, 16), torch.zeros(4, 2, 16))
    cache = binding.KvCache(k, k)
    i32 = torch.int32
    off, n, table = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros((2, 3), dtype=i32)
    q = torch.zeros((5, 4, 64), dtype=bf)
    with pytest.raises(ValueError, match="q_off"):
        binding.attn_paged(q, cache, off[:2], n, table)
    with pytest.raises(ValueError, match="kv_len"):
        binding.attn_paged(q, cache, off, n[:1], table)
    with pytest.raises(TypeError, match="page_table"):
        binding.attn_paged(q, cache, off, n, table.long())
    with pytest.raises(ValueError, match="CUDA"):
        binding.attn_paged(q, cache, off, n, table)
    with pytest.raises(TypeError, match="k must"):
        binding.attn_prompt(q.cuda() if torch.cuda.is_available() else _Cuda(q), q[:, :2].float(), q[:, :2],
                            _Cuda(off))
    with pytest.raises(ValueError, match="seq_off"):
        binding.attn_prompt(_Cuda(q), q[:, :2], q[:, :2], torch.zeros((2, 3), dtype=i32))


class _Cuda:
    """A CPU tensor that passes for a CUDA one up to the pointer marshalling."""

    def __init__(self, t):
        self._t = t

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)
