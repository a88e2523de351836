"""Values that are not finite in many short prompts: each CTA goes over several items
again, one after another, and every one of them keeps its own."""
import math

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from _window import visible
from test_gpu_attention import _off, _rand

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


@pytest.mark.parametrize("heads,kv_heads,dim", [(31, 1, 64), (48, 8, 128), (4, 4, 64), (100, 1, 128), (16, 4, 64)])
@pytest.mark.parametrize("kw", [dict(window=3), dict(window=1), dict(window=140, sinks=9), dict(window=64, sinks=130), dict()])
def test_every_item_keeps_its_own(heads, kv_heads, dim, kw):
    g = torch.Generator().manual_seed(heads + kw.get("window", 0))
    lens = torch.randint(0, 400, (48,), generator=g).tolist() + [1, 2, 1, 2, 2]
    T = sum(lens)
    q, k, v = _rand(g, T, heads, dim), _rand(g, T, kv_heads, dim, size=1.5), _rand(g, T, kv_heads, dim)
    clean = binding.attn_prompt(q, k, v, _off(lens), **kw)["out"]
    spoilt = v.clone()
    for i in range(40):
        at = tuple(int(torch.randint(0, n, (), generator=g)) for n in (T, kv_heads, dim))
        spoilt[at] = (INF, -INF, NAN)[i % 3]
    # which rows see one of either sign (a NaN counts as both)
    signs = []
    for sign in (INF, -INF):
        x = (torch.isnan(spoilt.float()) | (spoilt.float() == sign)).double()
        rows, at = [], 0
        for n in lens:
            mask = visible(torch.arange(n), n, kw.get("window", T), kw.get("sinks", 0)).to(DEV).double()
            rows.append(torch.einsum("nm,mhd->nhd", mask, x[at:at + n]) > 0)
            at += n
        signs.append(torch.cat(rows).repeat_interleave(heads // kv_heads, 1))
    up, down = signs
    want = clean.float()
    want[up & ~down], want[down & ~up], want[up & down] = INF, -INF, NAN
    ws = None
    for _ in range(10):
        r = binding.attn_prompt(q, k, spoilt, _off(lens), ws=ws, **kw)
        ws = r["ws"]
        torch.cuda.synchronize()
        assert binding.workspace_status(ws) == 0
        assert torch.equal(torch.nan_to_num(r["out"].float(), 1e30, 2e30, -2e30), torch.nan_to_num(want, 1e30, 2e30, -2e30))
