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


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("heads,kv_heads,dim,new", [(3, 1, 128, 1), (10, 2, 64, 3), (8, 2, 128, 6), (40, 1, 64, 1), (4, 4, 128, 1)])
def test_paged_values_past_the_end_do_not_matter(dtype, heads, kv_heads, dim, new):
    """Whatever codes and scales stand behind a request's last token, its bits
    are the same (enough requests that a CTA takes several tiles of one, the
    last of them cut)."""
    g = torch.Generator().manual_seed(heads + dim)
    kv, page = [600 + (i * 37) % 700 for i in range(300 // kv_heads)] + [65, 5], 64
    counts = [-(-n // page) for n in kv]
    table = torch.full((len(kv), max(counts)), -1, dtype=torch.int32)
    for r, c in enumerate(counts):
        table[r, :c] = torch.arange(sum(counts[:r]), sum(counts[:r]) + c)
    table = table.to(DEV)
    shape = (sum(counts), kv_heads, page, dim)
    K, V = (_rand(g, sum(kv), kv_heads, dim) for _ in range(2))
    q = _rand(g, len(kv) * new, heads, dim)
    first = None
    nan, inf = float("nan"), float("inf")
    for code, scale in ((0x00, 1.0), (0x7F, nan), (0x38, 1.0), (0x7E, 3e38), (0x7E, inf), (0xF0, -2.0), (0x01, 1e-40)):
        if dtype == BF:
            bits = torch.tensor([code * 256 + 0x80], dtype=torch.int32).to(torch.int16).view(BF).item() if scale == scale else nan
            if scale == inf:
                bits = inf
            cache = binding.KvCache(*(torch.full(shape, bits, dtype=BF, device=DEV) for _ in range(2)))
        else:
            cache = binding.KvCache(*(torch.full(shape, code, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)),
                                    *(torch.full(shape[:3], scale, device=DEV) for _ in range(2)))
        binding.kv_write(cache, K, V, _off(kv), _i32(kv), table)
        r = binding.attn_paged(q, cache, _off([new] * len(kv)), _i32(kv), table, lse=True)
        assert torch.isfinite(r["out"].float()).all()
        first = first or r
        assert _same(r, first), (code, scale)


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (4, 4, 64), (7, 1, 128), (16, 1, 64)])
def test_prompt_rows_do_not_depend_on_later_tokens(heads, kv_heads, dim):
    """Large values in the later tokens of the same sequence, infinities among
    them, do not change a bit of the rows before."""
    g = torch.Generator().manual_seed(dim + heads)
    lens = [700, 90, 333]
    T = sum(lens)
    q, k, v = (_rand(g, T, h, dim) for h in (heads, kv_heads, kv_heads))
    first = binding.attn_prompt(q, k, v, _off(lens), lse=True)
    for keep in ((600, 50, 1), (129, 1, 300), (640, 89, 332)):
        good = torch.zeros(T, dtype=torch.bool)
        for i, n in enumerate(keep):
            good[sum(lens[:i]):sum(lens[:i]) + n] = True
        good = good.to(DEV)
        for size in (20.0, 400.0, float("inf"), float("nan")):
            x = [t.clone() for t in (q, k, v)]
            for t in x:
                t[~good] *= size
            r = binding.attn_prompt(*x, _off(lens), lse=True)
            assert torch.equal(r["out"][good], first["out"][good]) and torch.equal(r["lse"][good], first["lse"][good])


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (4, 4, 64), (12, 2, 128), (3, 1, 64)])
def test_paged_rows_do_not_depend_on_later_tokens(dtype, heads, kv_heads, dim):
    """The same for the new tokens of a block: large queries, keys and values of
    the later ones leave the first ones' bits alone."""
    g = torch.Generator().manual_seed(dim + heads)
    kv, new, page = [300 + (i * 29) % 500 for i in range(240 // kv_heads)], 6, 16
    R = len(kv)
    counts = [-(-n // page) for n in kv]
    table = torch.full((R, max(counts)), -1, dtype=torch.int32)
    for r, c in enumerate(counts):
        table[r, :c] = torch.arange(sum(counts[:r]), sum(counts[:r]) + c)
    table = table.to(DEV)
    K, V = (_rand(g, sum(kv), kv_heads, dim) for _ in range(2))
    q = _rand(g, R * new, heads, dim)
    last = torch.tensor([n - 1 for n in torch.tensor(kv).cumsum(0).tolist()], device=DEV)
    good = torch.arange(R * new, device=DEV) % new < 3
    first = None
    for size in (1.0, 20.0, 300.0):
        k2, v2, q2 = K.clone(), V.clone(), q.clone()
        for back in range(3):
            k2[last - back] *= size
            v2[last - back] *= size
        q2[~good] *= size
        cache = binding.KvCache.empty(sum(counts), kv_heads, page, dim, dtype, DEV)
        binding.kv_write(cache, k2, v2, _off(kv), _i32(kv), table)
        r = binding.attn_paged(q2, cache, _off([new] * R), _i32(kv), table, lse=True)
        first = first or r
        assert torch.equal(r["out"][good], first["out"][good]) and torch.equal(r["lse"][good], first["lse"][good]), size
