"""Attention of values far from 1: tiny and zero rows of V, large scores, and
rows that pass the e4m3 split of q."""
import math

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from _attention import attend
from test_gpu_attention import Scene, _close

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def _off(lengths):
    return torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32).to(DEV)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _rand(g, *shape, size=1.0):
    return (torch.randn(shape, generator=g) * size).to(BF).to(DEV)


def _one_request(K, V, dtype, page=64):
    n, hk, dim = K.shape
    pages = -(-n // page)
    cache = binding.KvCache.empty(pages, hk, page, dim, dtype, DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    binding.kv_write(cache, K, V, _i32([0, n]), _i32([n]), table)
    return cache, table


@pytest.mark.parametrize("heads,dim,n", [(4, 128, 300), (16, 64, 1000), (40, 128, 77), (24, 128, 700)])
@pytest.mark.parametrize("sizes", [(1e-35,), (1e-35, 0.0), (1e-29, 1e-35), (1e-33, 0.0, 1.0), (0.0, 1e-20), (0.0,)])
def test_e4m3_rows_of_tiny_values(sizes, heads, dim, n):
    """V rows of these sizes in turn.  Rows whose scale is below 2^-100 count
    as zeros, so their mass is added to the bound."""
    g = torch.Generator().manual_seed(n)
    K, V = _rand(g, n, 1, dim), torch.randn((n, 1, dim), generator=g)
    V = (V * torch.tensor([sizes[i % len(sizes)] for i in range(n)])[:, None, None]).to(BF).to(DEV)
    cache, table = _one_request(K, V, F8)
    q = _rand(g, 2, heads, dim)
    r = binding.attn_paged(q, cache, _i32([0, 2]), _i32([n]), table, lse=True)
    k, v = Scene._stored(K), Scene._stored(V)
    seen = torch.tensor([n - 1, n])
    want, lse, bo, bl = attend(q, k, v, seen, dim ** -0.5)
    tiny = (v.abs().amax(-1, keepdim=True) < 448 * 2.0 ** -100) * v.abs()
    mass, _, _, _ = attend(q, k, tiny, seen, dim ** -0.5)
    _close(r["out"], want, bo + mass, "out")
    _close(r["lse"], lse, bl, "lse")


# ------------------------------------------------------------------ values that are not finite
@pytest.mark.parametrize("lens", [[700], [130, 60, 257], [5, 1, 40, 128], [257, 31] * 60])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (4, 4, 64), (3, 1, 128), (7, 1, 64), (32, 1, 128), (2, 2, 128), (8, 8, 128)])
def test_prompt_rows_that_do_not_see_a_value_are_free_of_it(heads, kv_heads, dim, lens):
    """NaN and infinities in K and V of single tokens: rows before them keep
    every bit, rows from them on are what the definition says (a NaN or both
    infinities give NaN, one infinity that infinity; a NaN key a row of NaN),
    and the other values of V's row and the other heads stay."""
    g = torch.Generator().manual_seed(heads * dim + len(lens))
    T, group = sum(lens), heads // kv_heads
    q, k, v = (_rand(g, T, h, dim) for h in (heads, kv_heads, kv_heads))
    off = _off(lens)
    clean = binding.attn_prompt(q, k, v, off, lse=True)
    inf, nan = math.inf, math.nan
    for trial in range(12):
        a = [sum(lens[:i]) for i in range(len(lens))]
        bad = torch.zeros((T, kv_heads, dim), dtype=torch.float64)
        n_bad = (1, 1, 2, 5, 30, 200)[trial % 6]
        for _ in range(n_bad):
            b = int(torch.randint(0, len(lens), (1,), generator=g))
            t = a[b] + int(torch.randint(0, lens[b], (1,), generator=g))
            h, d = int(torch.randint(0, kv_heads, (1,), generator=g)), int(torch.randint(0, dim, (1,), generator=g))
            bad[t, h, d] = (nan, inf, -inf)[int(torch.randint(0, 3, (1,), generator=g))]
        if trial == 11:                              # a garbage tail, as behind a padded prompt
            bad[a[0] + lens[0] // 2:a[0] + lens[0]] = nan
        at = (bad != 0).to(DEV)
        v2 = torch.where(at, bad.to(BF).to(DEV), v)
        r = binding.attn_prompt(q, k, v2, off, lse=True)
        assert torch.equal(r["lse"], clean["lse"])
        want = clean["out"].double()
        seen = torch.zeros_like(bad)
        for i, n in enumerate(lens):                 # sums of what is not finite, over the tokens so far
            seen[a[i]:a[i] + n] = bad[a[i]:a[i] + n].cumsum(0)
        want = want + seen.to(DEV).repeat_interleave(group, 1)
        got = r["out"].double()
        ok = (got == want) | (torch.isnan(got) & torch.isnan(want))
        # where the value itself was replaced, the rows that see it are infinite or NaN: nothing else differs
        assert ok.all(), f"trial {trial}: {(~ok).nonzero()[:5].tolist()}"
    t = lens[0] // 2
    k2 = k.clone()
    k2[t, kv_heads - 1, 3] = nan
    r = binding.attn_prompt(q, k2, v, off, lse=True)
    hit = torch.zeros((T, heads), dtype=torch.bool, device=DEV)
    hit[t:lens[0], (kv_heads - 1) * group:] = True
    assert torch.isnan(r["out"].double())[hit].all()
    assert torch.equal(r["out"][~hit], clean["out"][~hit]) and torch.equal(r["lse"][~hit], clean["lse"][~hit])
