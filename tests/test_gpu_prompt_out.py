"""Prompt attention whose results go to memory other than the device's own: plain
stores take them there, to the bits that a device buffer gets."""
import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from test_gpu_attention import _off, _rand

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


# whole row tiles (128 / group tokens) and ends of sequences; a list of items and none
@pytest.mark.parametrize("lens", [[300], [64, 1, 128, 257], [40] * 60 + [700]])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (3, 1, 128), (2, 2, 128)])
@pytest.mark.parametrize("kw", [dict(), dict(window=90, sinks=5)])
def test_results_in_pinned_host_memory(lens, heads, kv_heads, dim, kw):
    g = torch.Generator().manual_seed(dim + heads + len(lens))
    T = sum(lens)
    q, k, v = (_rand(g, T, h, dim) for h in (heads, kv_heads, kv_heads))
    for mend in (False, True):
        if mend:                               # the CTAs that see it go over their items again
            v[T // 2, 0, 3] = float("nan")
        want = binding.attn_prompt(q, k, v, _off(lens), lse=True, **kw)
        # a row before and one behind, which stay as they were
        host = torch.full((T + 2, heads, dim), 7.0, dtype=BF).pin_memory()
        lse = torch.full((T + 2, heads), 7.0).pin_memory()
        binding.attn_prompt(q, k, v, _off(lens), out=dict(out=binding.host_view(host[1:T + 1], DEV),
                                                          lse=binding.host_view(lse[1:T + 1], DEV)), **kw)
        torch.cuda.synchronize()
        assert binding.workspace_status(want["ws"]) == 0
        assert torch.equal(host[1:T + 1].view(torch.int16), want["out"].cpu().view(torch.int16))
        assert torch.equal(lse[1:T + 1], want["lse"].cpu())
        for t in (host, lse):
            assert (t[0] == 7).all() and (t[-1] == 7).all()
