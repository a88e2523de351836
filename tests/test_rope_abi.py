"""Argument checks of the norm and rotation entry points (no GPU needed): every
refusal comes before anything is enqueued."""
import ctypes

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from test_attention_abi import OK, _batch, _cache, _Cuda


def _rope(rot=64, interleaved=0, n_axes=1, amplitude=1.0, axis=(), inv_freq=()):
    r = binding._Rope(rot, interleaved, n_axes, amplitude)
    for i, a in enumerate(axis):
        r.axis[i] = a
    for i, f in enumerate(inv_freq):
        r.inv_freq[i] = f
    return r


def _norm(q=OK, k=OK, dtype=binding.F32, eps=1e-6):
    return binding._HeadNorm(q, k, dtype, eps)


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _turn(q=OK, k=OK, qs=256, ks=128, pos=OK, T=5, heads=4, kv=2, dim=64, rope=None, norm=None, qo=OK, ko=OK, qos=256, kos=128):
    return binding.load().dspark_qk_rope(q, k, qs, ks, pos, T, heads, kv, dim, _ref(rope), _ref(norm), qo, ko, qos, kos, None)


def _write(c, b, q=OK, K=OK, V=OK, qs=256, ks=128, vs=128, heads=4, pos=None, rope=None, norm=None, qo=OK, ko=None, qos=256,
           kos=128, ws=OK, wsb=256):
    return binding.load().dspark_rope_write(_ref(c), _ref(b), q, K, V, qs, ks, vs, heads, pos, _ref(rope), _ref(norm), qo, ko,
                                            qos, kos, ws, wsb, None)


def test_rotations_and_norms_are_checked():
    calls = (lambda **kw: _turn(**kw), lambda **kw: _write(_cache(), _batch(), **kw))
    nan, inf = float("nan"), float("inf")
    for call in calls:
        for kw in (dict(rot=0), dict(rot=4), dict(rot=12), dict(rot=72), dict(rot=-8), dict(n_axes=0), dict(n_axes=5)):
            assert call(rope=_rope(**kw)) == -3, kw
        for kw in (dict(amplitude=nan), dict(amplitude=inf), dict(axis=[0] * 31 + [1]), dict(n_axes=2, axis=[2]),
                   dict(inv_freq=[nan]), dict(inv_freq=[0.0] * 31 + [inf])):
            assert call(rope=_rope(**kw)) == -1, kw
        # what stands behind rot / 2 does not count: the call gets as far as its addresses
        assert call(rope=_rope(rot=32, axis=[0] * 16 + [9], inv_freq=[0.0] * 16 + [nan])) == -1
        assert call(norm=_norm(dtype=binding.E4M3)) == -2
        for kw in (dict(eps=0.0), dict(eps=1e-31), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(q=OK + 8), dict(k=OK + 4)):
            assert call(norm=_norm(**kw)) == -1, kw
        assert call(rope=_rope(), norm=_norm()) == -1                 # no device memory


def test_rows_are_checked():
    for kw in (dict(dim=96), dict(dim=0), dict(heads=0), dict(heads=(1 << 19) + 1), dict(kv=-1), dict(kv=4097), dict(T=-1)):
        assert _turn(**kw) == -3, kw
    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(q=OK + 2), dict(k=OK + 8), dict(qo=OK + 4),
               dict(ko=OK + 8), dict(qs=248), dict(ks=132), dict(qos=-256), dict(kos=64), dict(qs=1 << 36),
               dict(pos=None, rope=_rope())):
        assert _turn(**kw) == -1, kw
    assert _turn(T=0, q=None, k=None, pos=None, qo=None, ko=None) == 0
    assert _turn(kv=0, k=None, ko=None) == -1                         # no device memory
    c, b = _cache(), _batch()
    for heads in (-1, (1 << 19) + 1):
        assert _write(c, b, heads=heads, qs=1 << 30, qos=1 << 30) == -3
    for kw in (dict(q=None), dict(K=None), dict(V=None), dict(qo=None), dict(q=OK + 8), dict(V=OK + 2), dict(ko=OK + 4),
               dict(qs=250), dict(ks=64), dict(vs=-128), dict(qos=8), dict(ko=OK, kos=100)):
        assert _write(c, b, **kw) == -1, kw
    for kw in (dict(ws=None), dict(ws=OK + 64), dict(wsb=255)):
        assert _write(c, b, **kw) == -8, kw
    assert _write(c, _batch(kv_len=None)) == -1
    assert _write(c, _batch(T=0, q_off=None, kv_len=None, page_table=None), q=None, K=None, V=None, qo=None, ws=None) == 0


@pytest.mark.parametrize("kw,code", [(dict(dtype=7), -2), (dict(page=24), -3), (dict(head_dim=80), -3), (dict(v=OK + 2), -1),
                                     (dict(dtype=binding.E4M3), -1)])
def test_the_cache_is_checked(kw, code):
    assert _write(_cache(**kw), _batch()) == code
    assert _write(None, _batch()) == -1
    assert _write(_cache(), None) == -1
    assert _write(_cache(), _batch(R=0)) == -3


def test_binding_checks_shapes_before_any_launch():
    bf = torch.bfloat16
    q, k = torch.zeros((5, 4, 64), dtype=bf), torch.zeros((5, 2, 64), dtype=bf)
    pos = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="frequencies"):
        binding.Rope([])
    with pytest.raises(ValueError, match="axis"):
        binding.Rope([1.0, 0.5], [0])
    with pytest.raises(ValueError, match="axis"):
        binding.Rope([1.0, 0.5], [0, 4])
    with pytest.raises(ValueError, match="queries, keys"):
        binding.HeadNorm()
    with pytest.raises(ValueError, match="one dtype"):
        binding.HeadNorm(torch.zeros(64), torch.zeros(64, dtype=bf))
    with pytest.raises(ValueError, match="CUDA"):
        binding.HeadNorm(torch.zeros(64))
    rope = binding.Rope.from_theta(64, 5e5, interleaved=True)
    assert rope.n_axes == 1 and rope._c.rot == 64 and rope._c.inv_freq[31] == 5e5 ** (-62 / 64)
    assert binding.Rope([1.0] * 4, [0, 2, 1, 0]).n_axes == 3 and binding.Rope([1.0] * 4, n_axes=2).n_axes == 2
    with pytest.raises(ValueError, match="takes positions"):
        binding.qk_rope(q, k, None, rope)
    with pytest.raises(ValueError, match="go with a rope"):
        binding.qk_rope(q, k, pos)
    with pytest.raises(ValueError, match="positions must"):
        binding.qk_rope(q, k, pos[:4], rope)
    with pytest.raises(TypeError, match="positions must"):
        binding.qk_rope(q, k, pos.long(), rope)
    with pytest.raises(ValueError, match="positions must"):
        binding.qk_rope(q, k, pos, binding.Rope([1.0] * 4, [0, 1, 2, 0]))
    with pytest.raises(ValueError, match="CUDA"):
        binding.qk_rope(q, k, pos, rope)
    with pytest.raises(ValueError, match="k must"):
        binding.qk_rope(_Cuda(q), k[:, 0], _Cuda(pos), rope, out=dict(q=_Cuda(q)))
    with pytest.raises(TypeError, match="q must"):
        binding.qk_rope(_Cuda(q.float()), None, _Cuda(pos), rope)
    with pytest.raises(ValueError, match="k must"):
        binding.qk_rope(_Cuda(q), _Cuda(k), _Cuda(pos), rope, out=dict(q=_Cuda(q), k=_Cuda(k[:4])))
