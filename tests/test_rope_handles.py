"""What HeadNorm and Rope hand to a call is what they hold at that call (no GPU
needed: the library's calls are recorded instead of made)."""
import ctypes

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from test_attention_abi import _Cuda

BF = torch.bfloat16


class _Recorder:
    """Stands for the loaded library: keeps the norm and the rope of each call."""

    def __init__(self):
        self.norm = self.rope = None

    @staticmethod
    def _copy(ref, kind):
        if ref is None:
            return None
        return kind.from_buffer_copy(bytes(ctypes.cast(ref, ctypes.POINTER(kind)).contents))

    def dspark_kv_workspace_size(self):
        return 256

    def dspark_qk_rope(self, q, k, qs, ks, pos, T, heads, kv, dim, rope, norm, *rest):
        self.rope, self.norm = self._copy(rope, binding._Rope), self._copy(norm, binding._HeadNorm)
        return 0

    def dspark_rope_write(self, c, b, q, K, V, qs, ks, vs, heads, pos, rope, norm, *rest):
        self.rope, self.norm = self._copy(rope, binding._Rope), self._copy(norm, binding._HeadNorm)
        return 0


@pytest.fixture
def lib(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(binding, "load", lambda *a: r)
    monkeypatch.setattr(binding, "_stream", lambda s=None: 0)
    return r


def _calls(rope, norm, positions=None, T=3):
    """qk_rope and rope_write of the same rows."""
    q, k = (_Cuda(torch.zeros((T, h, 64), dtype=BF)) for h in (4, 2))
    cache = binding.KvCache(*(_Cuda(torch.zeros((1, 2, 16, 64), dtype=BF)) for _ in range(2)))
    off, kv_len, table = (_Cuda(torch.tensor(x, dtype=torch.int32)) for x in ([0, T], [T], [[0]]))
    ws = _Cuda(torch.zeros(256, dtype=torch.uint8))
    yield lambda: binding.qk_rope(q, k, positions, rope, norm, out=dict(q=q, k=k))
    yield lambda: binding.rope_write(cache, q, k, k, off, kv_len, table, rope, norm, positions=positions, ws=ws, out=dict(q=q))


def test_a_norm_follows_its_weights(lib):
    wq, wk = torch.ones(64), torch.ones(64)
    norm = binding.HeadNorm(_Cuda(wq), _Cuda(wk), 1e-6)
    for call in _calls(None, norm):
        call()
        assert (lib.norm.q_w, lib.norm.k_w, lib.norm.w_dtype) == (wq.data_ptr(), wk.data_ptr(), binding.F32)
        # other storage under the same tensor, of another dtype, as a cast of a module leaves it
        old = wq.data, wk.data
        wq.data, wk.data = wq.to(BF), wk.to(BF)
        call()
        assert (lib.norm.q_w, lib.norm.k_w, lib.norm.w_dtype) == (wq.data_ptr(), wk.data_ptr(), binding.BF16)
        assert lib.norm.q_w != old[0].data_ptr()
        wq.data, wk.data = old
        # another tensor, another eps, a side without a norm
        other = torch.full((64,), 2.0)
        norm.q, norm.k, norm.eps = _Cuda(other), None, 0.25
        call()
        assert (lib.norm.q_w, lib.norm.k_w, lib.norm.eps) == (other.data_ptr(), None, 0.25)
        norm.q, norm.k, norm.eps = _Cuda(wq), _Cuda(wk), 1e-6


def test_a_norm_is_checked_at_the_call(lib):
    norm = binding.HeadNorm(_Cuda(torch.ones(64)), _Cuda(torch.ones(64)))
    good = norm.q
    for call in _calls(None, norm):
        call()
        for bad, error in ((_Cuda(torch.ones(63)), ValueError), (_Cuda(torch.ones(64, dtype=BF)), ValueError),
                           (_Cuda(torch.ones((64, 1))), ValueError), (torch.ones(64), ValueError),
                           (_Cuda(torch.ones(128)[::2]), ValueError)):
            lib.norm = None
            norm.q = bad
            with pytest.raises(error):
                call()
            assert lib.norm is None
        norm.q, norm.k = None, None
        with pytest.raises(ValueError, match="queries, keys"):
            call()
        norm.q = norm.k = _Cuda(torch.ones(64, dtype=torch.float16))
        with pytest.raises(TypeError):
            call()
        norm.q = norm.k = good


def test_positions_are_checked_against_what_the_kernel_reads(lib):
    """A rope's number of axes is the one that its struct holds: setting it apart from
    that would pass positions that the kernel reads past."""
    rope = binding.Rope([1.0, 0.5, 0.25, 0.1], [0, 1, 2, 0])
    with pytest.raises(AttributeError):
        rope.n_axes = 1
    assert rope.n_axes == rope._c.n_axes == 3
    for call in _calls(rope, None, _Cuda(torch.zeros((3, 3), dtype=torch.int32))):
        call()
        assert lib.rope.n_axes == 3
    for call in _calls(rope, None, _Cuda(torch.zeros((3,), dtype=torch.int32))):
        with pytest.raises(ValueError, match="positions must"):
            call()
