"""Prompt attention over many sequences of a few key tiles: its row tiles end
at different tiles, item by item, and a CTA takes many items."""
import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from test_gpu_attention import _check_prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 8, 128), (8, 8, 64), (16, 8, 64), (24, 8, 128), (7, 1, 64)])
@pytest.mark.parametrize("most", [60, 300, 700])
def test_many_short_sequences(heads, kv_heads, dim, most):
    g = torch.Generator().manual_seed(most + heads)
    lens = torch.randint(0, most, (90,), generator=g).tolist()
    lens[::7] = [most % 256 + 1] * len(lens[::7])
    q, k, v, first = _check_prompt(lens, heads, kv_heads, dim, seed=most)
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(q.device)
    for _ in range(20):
        r = binding.attn_prompt(q, k, v, off, scale=0.7 / dim ** 0.5, lse=True, ws=first["ws"])
        assert torch.equal(r["out"], first["out"]) and torch.equal(r["lse"], first["lse"])
    assert binding.workspace_status(first["ws"]) == 0
