"""Bit-for-bit claims of the attention calls: what a row's result must not
depend on -- other sequences' values, what earlier kernels left in shared
memory, and cached values past a request's end."""
import pytest
import torch

from speculative_decoding_drafting_gb300 import binding

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


def _same(a, b):
    return all(torch.equal(a[n], b[n]) for n in ("out", "lse"))


@pytest.mark.parametrize("heads,kv_heads,dim", [(3, 1, 128), (7, 1, 64), (14, 2, 128), (100, 1, 64), (5, 1, 128)])
def test_prompt_reruns_agree_whatever_ran_between(heads, kv_heads, dim):
    """Groups that leave rows of a tile unused, with a call in between that
    fills every row with large queries."""
    g = torch.Generator().manual_seed(heads)
    lens = [900, 17, 640]
    T = sum(lens)
    q, k, v = (_rand(g, T, h, dim) for h in (heads, kv_heads, kv_heads))
    first = binding.attn_prompt(q, k, v, _off(lens), lse=True)
    for size in (30.0, 0.0, 300.0):
        other = [_rand(g, 4096, h, dim, size=size) for h in (8, 2, 2)]
        binding.attn_prompt(*other, _i32([0, 4096]))
        assert _same(binding.attn_prompt(q, k, v, _off(lens), lse=True), first)


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (4, 4, 64), (7, 1, 128), (16, 1, 64)])
def test_prompt_rows_do_not_depend_on_the_next_sequence(heads, kv_heads, dim):
    """Large finite values in the sequence after (and before) do not change a
    bit, whatever their scores would be."""
    g = torch.Generator().manual_seed(dim + heads)
    lens = [301, 457, 260]
    T = sum(lens)
    q, k, v = (_rand(g, T, h, dim) for h in (heads, kv_heads, kv_heads))
    first = binding.attn_prompt(q, k, v, _off(lens), lse=True)
    for which, rest in ((1, (slice(0, 301), slice(758, T))), (0, (slice(301, T),)), (2, (slice(0, 758),))):
        a = sum(lens[:which])
        for size in (20.0, 400.0):
            x = [t.clone() for t in (q, k, v)]
            for t in x:
                t[a:a + lens[which]] *= size
            r = binding.attn_prompt(*x, _off(lens), lse=True)
            for s in rest:
                assert torch.equal(r["out"][s], first["out"][s]) and torch.equal(r["lse"][s], first["lse"][s])
