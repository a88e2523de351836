"""Positions that begin off a 16-byte boundary: slices of longer ones."""
import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from test_gpu_attention import _i32, _rand

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
DEV = "cuda:0"


@pytest.mark.parametrize("axes", [1, 2, 3])
@pytest.mark.parametrize("first", [1, 2, 3])
def test_slices_of_positions(axes, first):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator().manual_seed(axes)
    T, heads, hk, dim = 21, 4, 2, 64
    q, k, v = (_rand(g, T, h, dim) for h in (heads, hk, hk))
    rope = binding.Rope([10000.0 ** (-i / 32) for i in range(32)], [i % axes for i in range(32)])
    long = torch.randint(0, 5000, (T + first, axes), generator=g, dtype=torch.int32).to(DEV)
    part, whole = long[first:], long[first:].clone()
    assert part.is_contiguous() and (part.data_ptr() % 16 != 0 or first * axes % 4 == 0)
    off, kv_len, table = _i32([0, T]), _i32([T]), _i32([[1, 0]])
    rows, caches = [], []
    for pos in (part, whole):
        a = binding.qk_rope(q, k, pos, rope)
        cache = binding.KvCache(*(torch.zeros((2, hk, 16, dim), dtype=BF, device=DEV) for _ in range(2)))
        b = binding.rope_write(cache, q, k, v, off, kv_len, table, rope, positions=pos, keep=True)
        assert binding.workspace_status(b["ws"]) == 0
        rows.append([a["q"], a["k"], b["q"], b["k"]])
        caches.append(cache.k)
    for x, y in zip(*rows):
        assert torch.equal(x, y)
    assert torch.equal(*caches) and torch.equal(rows[0][0], rows[0][2])
