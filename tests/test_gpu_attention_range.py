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


# ------------------------------------------------------------------ large scores
@pytest.mark.parametrize("dtype", [BF, F8, None])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_up_to_2_26(dtype, sign):
    """Scores a little below 2^26 in magnitude, 2^18 apart: the largest takes all
    the weight (ties share it), whichever tile it stands in.  (dtype None: the
    prompt form, whose last row sees every key.)  No ties with e4m3 caches: V's
    scale joins the exponent there, so that float32 rounds equal scores of rows
    of different scales differently, by up to 4 at this size."""
    g = torch.Generator().manual_seed(3)
    n, dim, heads = 600, 128, 4
    q = torch.zeros((1, heads, dim), dtype=BF, device=DEV)
    q[:, :, 0] = 2.0 ** 12
    for tops in ([0], [599], [300], [5, 130, 420, 590])[:3 if dtype == F8 else 4]:
        a = 1.0 - 2.0 ** -7 * torch.randint(1, 60, (n,), generator=g).double()
        a[tops] = 1.0
        if sign < 0:
            a = 2.0 - a
        K = torch.zeros((n, 1, dim), dtype=torch.float64)
        K[:, 0, 0] = sign * a * 2.0 ** 12.99
        K = K.to(BF).to(DEV)
        V = _rand(g, n, 1, dim)
        top = K[:, 0, 0].double().max()
        hit = (K[:, 0, 0].double() == top).nonzero()[:, 0]
        if dtype is None:
            qq = q.expand(n, -1, -1).contiguous()
            r = binding.attn_prompt(qq, K, V, _i32([0, n]), scale=2.0, lse=True)
            r = dict(out=r["out"][-1:], lse=r["lse"][-1:])
            v = V.double()
        else:
            cache, table = _one_request(K, V, dtype)
            r = binding.attn_paged(q, cache, _i32([0, 1]), _i32([n]), table, scale=2.0, lse=True)
            v = V.double() if dtype == BF else Scene._stored(V)
        want = v[hit, 0].mean(0).expand(1, heads, dim)
        mass = v[hit, 0].abs().mean(0).expand(1, heads, dim)
        _close(r["out"], want, 2.0 ** -8 * want.abs() + 2.0 ** -8 * mass, f"out ({tops})")
        lse = (2.0 ** 13 * top + math.log(len(hit))).expand(1, heads)
        _close(r["lse"], lse, 2.0 ** -21 * lse.abs(), f"lse ({tops})")


# ------------------------------------------------------------------ the precision of e4m3 caches
def test_e4m3_split_of_q():
    """q meets e4m3 keys as two e4m3 terms: exact for values of 2^-9 of their
    row's largest and more, off by at most 2^-17 of it below.  One key with one
    value of 1 per request reads a value of q out as its lse.  That adds six
    roundings of 2^-24 of the value (scale log2 e, the key's scale, the product,
    the sum, ln 2) and, in binary orders, the rounding of the reference with V's
    scale (2^-20 up to 32), two exponentials (2^-21), a logarithm (2^-22) and the
    sum of both (2^-20): 2^-21 of the value and 2^-18."""
    g = torch.Generator().manual_seed(8)
    dim, rows = 64, 200
    x = torch.exp2(torch.rand((rows, dim), generator=g) * -16) * (torch.randint(0, 2, (rows, dim), generator=g) * 2 - 1)
    x[:, 0] = torch.exp2(torch.randint(-3, 4, (rows,), generator=g).float()) * torch.where(torch.arange(rows) % 2 == 0, 1.0, 1.9)
    x[:, 1:] *= x[:, :1].abs()
    x = x.to(BF)
    K = torch.eye(dim)[:, None].to(BF).to(DEV)
    cache = binding.KvCache.empty(dim, 1, 16, dim, F8, DEV)
    each = torch.arange(dim + 1, dtype=torch.int32, device=DEV)
    binding.kv_write(cache, K, K, each, torch.ones(dim, dtype=torch.int32, device=DEV), each[:dim, None].contiguous())
    q = x.repeat_interleave(dim, 0)[:, None].contiguous().to(DEV)          # request (row, value)
    R = rows * dim
    r = binding.attn_paged(q, cache, torch.arange(R + 1, dtype=torch.int32, device=DEV), torch.ones(R, dtype=torch.int32, device=DEV),
                           each[:dim].repeat(rows)[:, None].contiguous(), scale=1.0, lse=True)
    x = x.double()
    big = x.abs().amax(1, keepdim=True)
    off = (r["lse"].double().cpu().view(rows, dim) - x).abs() - 2.0 ** -18 - 2.0 ** -21 * x.abs()
    assert (off <= torch.where(x.abs() < 2.0 ** -9 * big, 2.0 ** -17 * big, torch.zeros_like(x))).all()


def _two_keys(rows, dim):
    """Requests of two keys whose V rows are each other's negatives, and whose
    scores are single products a little apart: the output is a small difference
    of large terms, which its own rounding does not hide."""
    g = torch.Generator().manual_seed(dim)
    heads = 4
    q = torch.zeros((rows, heads, dim), dtype=BF)
    q[:, :, 5] = torch.tensor([1.0, 0.75, 1.5, -1.25])
    K = torch.zeros((rows, 2, 1, dim))
    K[:, 1, 0, 5] = 0.002 + 0.1 * torch.rand((rows,), generator=g)
    V = torch.randn((rows, 2, 1, dim), generator=g)
    V[:, 1] = -V[:, 0]
    return q, K.to(BF), V.to(BF)


def _two_keys_64(q, k, v):
    """out and its bound for float64 q [n, H, D], k and v [n, 2, 1, D]: the output's
    rounding, 2^-11 of each weight (11 bits), and a score of six roundings."""
    s = torch.einsum("nhd,njd->nhj", q, k[:, :, 0])
    p = torch.softmax(s, -1)
    out = torch.einsum("nhj,njd->nhd", p, v[:, :, 0])
    mass = torch.einsum("nhj,njd->nhd", p, v[:, :, 0].abs())
    ds = 6 * 2.0 ** -24 * s.abs().amax(-1, keepdim=True)
    return p, out, 2.0 ** -8 * out.abs() + (2.0 ** -11 + 2 * (4 * ds + 2.0 ** -20)) * mass


@pytest.mark.parametrize("dim", [64, 128])
def test_e4m3_weights_keep_11_bits(dim):
    rows = 512
    q, K, V = (x.to(DEV) for x in _two_keys(rows, dim))
    cache = binding.KvCache.empty(rows, 1, 16, dim, F8, DEV)
    table = torch.arange(rows, dtype=torch.int32, device=DEV)[:, None].contiguous()
    two = torch.full((rows,), 2, dtype=torch.int32, device=DEV)
    binding.kv_write(cache, K.flatten(0, 1), V.flatten(0, 1), _off([2] * rows), two, table)
    r = binding.attn_paged(q, cache, _off([1] * rows), two, table, scale=1.0)
    p, want, bound = _two_keys_64(q.double(), Scene._stored(K), Scene._stored(V))
    _close(r["out"], want, bound, "out")
    # weights of 8 bits would not pass
    w = (p / p.amax(-1, keepdim=True)).to(BF).double()
    coarse = torch.einsum("nhj,njd->nhd", w * p.amax(-1, keepdim=True), Scene._stored(V)[:, :, 0])
    assert ((coarse - want).abs() > bound).double().mean() > 0.05
