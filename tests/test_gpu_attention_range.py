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
