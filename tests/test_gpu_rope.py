"""Head norms and rotary positions, as rows and on the way into the paged cache,
against plain 64-bit forms."""
import ctypes

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from _rope import close, turned
from test_gpu_attention_memory import Arena

pytestmark = pytest.mark.gpu

BF, F8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
DEV = "cuda:0"
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _off(lengths):
    return torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32).to(DEV)


def _rand(g, *shape, size=2.0):
    return (torch.randn(shape, generator=g) * size).to(BF).to(DEV)


def _freq(rot, theta=1e4):
    return [theta ** (-2.0 * i / rot) for i in range(rot // 2)]


def _axes(half, kind):
    return {"one": None, "blocks": [0 if i < half // 4 else (1 if i < half // 2 else 2) for i in range(half)],
            "cycled": [i % 3 for i in range(half)]}[kind]


def _weights(g, dim, kind, dtype=F32):
    """(q's, k's) norm weights for "", "q", "k" or "qk"."""
    return tuple((1 + 0.3 * torch.randn(dim, generator=g)).to(dtype).to(DEV) if s in kind else None for s in "qk")


def _norm(w):
    return binding.HeadNorm(*w, EPS) if any(x is not None for x in w) else None


# ------------------------------------------------------------------ rows in and out
@pytest.mark.parametrize("T,heads,kv_heads,dim,rot,pairs,axes,norm,dtype", [
    (1, 32, 8, 128, 128, False, "one", "qk", BF), (1, 1, 0, 64, 64, True, "one", "", F32),
    (3, 28, 4, 128, 128, False, "blocks", "", F32), (17, 5, 3, 128, 64, False, "one", "q", F32),
    (33, 16, 4, 64, 32, True, "one", "k", BF), (300, 7, 1, 64, 48, False, "cycled", "qk", F32),
    (257, 17, 17, 128, 96, True, "cycled", "qk", BF), (40, 3, 2, 128, 8, False, "one", "", F32),
    (41, 3, 2, 64, 8, True, "one", "qk", F32), (19, 70, 33, 128, 0, False, "one", "qk", F32), (3001, 4, 2, 64, 64, False, "one", "qk", BF),
    (2600, 3, 1, 128, 128, False, "blocks", "q", BF), (64, 64, 8, 64, 64, False, "blocks", "", F32)])
def test_rows(T, heads, kv_heads, dim, rot, pairs, axes, norm, dtype):
    g = torch.Generator().manual_seed(T + heads)
    freq, axis = _freq(rot) if rot else [], _axes(rot // 2, axes)
    w = _weights(g, dim, norm, dtype)
    n_axes = 1 if axis is None else 3
    pos = torch.randint(0, 30000, (T, n_axes), generator=g).to(torch.int32)
    fused = _rand(g, T, heads + kv_heads + 1, dim)                 # slices of one projection
    q, k = fused[:, :heads], fused[:, heads:heads + kv_heads]
    rope = binding.Rope(freq, axis, interleaved=pairs, amplitude=1.25 if T == 17 else 1.0) if rot else None
    amplitude = 1.25 if T == 17 else 1.0
    r = binding.qk_rope(q, k if kv_heads else None, pos.to(DEV) if rot else None, rope, _norm(w))
    assert ("k" in r) == (kv_heads > 0)
    for name, x, wx in (("q", q, w[0]), ("k", k, w[1]))[:1 + (kv_heads > 0)]:
        want, early = turned(x, pos, freq, axis, pairs, amplitude, wx, EPS)
        close(r[name], want, early, name)
        if wx is None:                                             # what is not turned passes bit for bit
            assert torch.equal(r[name][..., rot:], x[..., rot:])
    # in place, and into a strided output
    f2 = fused.clone()
    out = dict(q=f2[:, :heads])
    if kv_heads:
        out["k"] = f2[:, heads:heads + kv_heads]
    binding.qk_rope(out["q"], out.get("k"), pos.to(DEV) if rot else None, rope, _norm(w), out=out)
    for name in r:
        assert torch.equal(out[name], r[name])
    assert torch.equal(f2[:, heads + kv_heads:], fused[:, heads + kv_heads:])


def test_far_and_negative_positions():
    """The angle's fraction of a turn is as good at the last position as at the first."""
    g = torch.Generator().manual_seed(3)
    pos = torch.tensor([0, 1, 2 ** 20 + 7, 2 ** 24 - 1, 2 ** 31 - 1, 123456789, -1, -2 ** 31, -77777])[:, None].to(torch.int32)
    for freq in (_freq(128, 1e6), [7.5, -1.0, 0.0, 6.283185307179586, -1e-9, 1e300, 3.0, 0.5] * 8):
        q = _rand(g, 9, 3, 128)
        r = binding.qk_rope(q, None, pos.to(DEV), binding.Rope(freq))
        # a frequency of 1e300 is a whole number of radians: 64 bits of its turns say
        # nothing at all, so its pairs are left out
        want, early = turned(q, pos, [0.0 if abs(f) > 1e15 else f for f in freq])
        # the library rounds inv_freq / 2 pi to 53 bits: 2^-53 of the angle
        far = pos.double().abs().to(DEV)[:, None] * torch.tensor([abs(f) for f in freq] * 2, device=DEV).clamp_max(1e9) * 2.0 ** -52
        keep = torch.tensor([abs(f) < 1e15 for f in freq] * 2, device=DEV)
        size = q.double().abs()
        early = early + (size + size.roll(64, -1)) * far[:, None]
        close(r["q"][..., keep], want[..., keep], early[..., keep], "far positions")


def test_rows_that_are_not_finite_stay_alone():
    g = torch.Generator().manual_seed(4)
    q = _rand(g, 6, 4, 64)
    pos = _i32(list(range(6)))
    norm = binding.HeadNorm(torch.ones(64, device=DEV), None)
    rope = binding.Rope(_freq(32))
    clean = {n: binding.qk_rope(q, None, pos, rope, x)["q"] for n, x in (("norm", norm), ("plain", None))}
    q[2, 1, 3], q[4, 0, 40], q[5, 3, 63] = float("nan"), float("inf"), float("-inf")
    r = binding.qk_rope(q, None, pos, rope, norm)["q"]
    ok = torch.ones((6, 4), dtype=torch.bool, device=DEV)
    ok[2, 1] = ok[4, 0] = ok[5, 3] = False
    assert torch.equal(r[ok], clean["norm"][ok]) and torch.isnan(r[2, 1]).all()
    # without a norm a value reaches its own pair alone, and one that is not turned nothing
    r = binding.qk_rope(q, None, pos, rope)["q"]
    want = clean["plain"].clone()
    assert torch.isnan(r[2, 1, [3, 19]]).all()
    want[2, 1, [3, 19]] = r[2, 1, [3, 19]]
    want[4, 0, 40], want[5, 3, 63] = float("inf"), float("-inf")
    assert torch.equal(torch.nan_to_num(r, 7.0, 8.0, 9.0), torch.nan_to_num(want, 7.0, 8.0, 9.0))


def test_large_and_small_heads_are_normed():
    g = torch.Generator().manual_seed(5)
    size = torch.exp2(torch.linspace(-40, 55, 96)).to(DEV)[:, None, None]
    q = (_rand(g, 96, 2, 128).float() * size).to(BF)
    q[7] = 0
    w = _weights(g, 128, "q")
    pos = torch.arange(96, dtype=torch.int32)[:, None]
    want, early = turned(q, pos, _freq(128), w=w[0], eps=EPS)
    r = binding.qk_rope(q, None, pos.to(DEV), binding.Rope(_freq(128)), _norm(w))
    close(r["q"], want, early, "q")
    assert (r["q"][7] == 0).all()


# ------------------------------------------------------------------ into the cache
class Paged:
    """An empty paged cache (NaN everywhere) with pages for the requests."""

    def __init__(self, kv, kv_heads, dim, page, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        counts = [-(-n // page) for n in kv]
        self.pages = sum(counts) + 2
        self.table = torch.full((len(kv), max(max(counts), 1)), -1, dtype=torch.int32)
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        for r, c in enumerate(counts):
            self.table[r, :c] = order[sum(counts[:r]):sum(counts[:r]) + c]
        self.table = self.table.to(DEV)
        self.shape, self.dtype = (self.pages, kv_heads, page, dim), dtype

    def empty(self):
        if self.dtype == BF:
            return binding.KvCache(*(torch.full(self.shape, float("nan"), dtype=BF, device=DEV) for _ in range(2)))
        k, v = (torch.full(self.shape, 0x7F, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
        return binding.KvCache(k, v, *(torch.full(self.shape[:3], float("nan"), device=DEV) for _ in range(2)))


def _bits(cache):
    parts = [cache.k.view(torch.uint8), cache.v.view(torch.uint8)]
    return parts + [x.view(torch.int32) for x in (cache.k_scale, cache.v_scale) if x is not None]


def _places(kv, q_len, page, table):
    """(page, slot) of every new token with a place."""
    pos = torch.cat([torch.arange(n - m, n) for n, m in zip(kv, q_len)]) if kv else torch.empty(0, dtype=torch.int64)
    r = torch.repeat_interleave(torch.arange(len(kv)), torch.tensor(q_len))
    at = table.cpu()[r, pos.clamp_min(0) // page].long()
    return pos, at.to(DEV), (pos.clamp_min(0) % page).to(DEV)


CASES = [(8, 2, 128, 16, 128, False, "one", "qk"), (4, 4, 64, 64, 32, True, "one", ""), (9, 3, 128, 256, 64, False, "cycled", "k"),
         (40, 5, 64, 32, 64, False, "blocks", "q"), (3, 1, 128, 128, 96, True, "blocks", "qk"), (0, 17, 64, 16, 64, False, "one", "k")]


@pytest.mark.parametrize("heads,kv_heads,dim,page,rot,pairs,axes,norm", CASES)
def test_append_is_the_rotation_and_the_write(heads, kv_heads, dim, page, rot, pairs, axes, norm):
    """bf16: the queries, the kept keys and every byte of the cache are those of the two calls."""
    kv, new = [1, 40, 0, 700, 129, page, 64], [1, 7, 0, 3, 129, 1, 64]
    g = torch.Generator().manual_seed(heads + page)
    T = sum(new)
    s = Paged(kv, kv_heads, dim, page, BF, seed=page)
    fused = _rand(g, T, heads + 2 * kv_heads, dim)
    q, K, V = fused[:, :heads], fused[:, heads:heads + kv_heads], fused[:, heads + kv_heads:]
    axis = _axes(rot // 2, axes)
    rope = binding.Rope(_freq(rot), axis, interleaved=pairs)
    nm = _norm(_weights(g, dim, norm))
    pos, _, _ = _places(kv, new, page, s.table)
    positions = None if axis is None else torch.stack([pos, pos // 3, pos % 5], 1).to(torch.int32).to(DEV)
    a, b = s.empty(), s.empty()
    args = (_off(new), _i32(kv), s.table)
    r = binding.rope_write(a, q if heads else None, K, V, *args, rope=rope, norm=nm, positions=positions, keep=True)
    flat = pos.to(torch.int32).to(DEV) if positions is None else positions
    rows = binding.qk_rope(q if heads else K, K, flat, rope, nm if heads or nm is None else binding.HeadNorm(k=nm.k, eps=EPS))
    binding.kv_write(b, rows["k"], V, *args)
    torch.cuda.synchronize()
    assert binding.workspace_status(r["ws"]) == 0
    if heads:
        assert torch.equal(r["q"], rows["q"])
    assert torch.equal(r["k"], rows["k"])
    for x, y in zip(_bits(a), _bits(b)):
        assert torch.equal(x, y)
    # without the kept keys the cache is the same
    c = s.empty()
    binding.rope_write(c, q if heads else None, K, V, *args, rope=rope, norm=nm, positions=positions)
    for x, y in zip(_bits(a), _bits(c)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("heads,kv_heads,dim,page,rot,pairs,axes,norm", CASES)
def test_append_to_an_e4m3_cache(heads, kv_heads, dim, page, rot, pairs, axes, norm):
    """Queries and kept keys as over bf16; values bit for bit as the write stores
    them; keys within half an e4m3 step (2^-4 of the value, 2^-10 below 2^-6) of
    the quotient, with the float32 row's own error, and nothing else written."""
    kv, new = [1, 40, 0, 700, 129, page, 64], [1, 7, 0, 3, 129, 1, 64]
    g = torch.Generator().manual_seed(heads + page + 1)
    T = sum(new)
    s, plain = Paged(kv, kv_heads, dim, page, F8, seed=page), Paged(kv, kv_heads, dim, page, BF, seed=page)
    q, K, V = _rand(g, T, max(heads, 1), dim), _rand(g, T, kv_heads, dim), _rand(g, T, kv_heads, dim)
    K[0] = 0
    V[T // 2] = 0
    axis, freq = _axes(rot // 2, axes), _freq(rot)
    rope, w = binding.Rope(freq, axis, interleaved=pairs), _weights(g, dim, norm)
    pos, at, slot = _places(kv, new, page, s.table)
    positions = None if axis is None else torch.stack([pos, pos // 3, pos % 5], 1).to(torch.int32).to(DEV)
    a, b, c = s.empty(), plain.empty(), s.empty()
    args = (_off(new), _i32(kv), s.table)
    kw = dict(rope=rope, norm=_norm(w), positions=positions, keep=True)
    r = binding.rope_write(a, q if heads else None, K, V, *args, **kw)
    want = binding.rope_write(b, q if heads else None, K, V, *args, **kw)
    binding.kv_write(c, K, V, *args)
    torch.cuda.synchronize()
    assert binding.workspace_status(r["ws"]) == 0
    for name in ("q", "k"):
        assert (name in r) == (name in want) and (name not in r or torch.equal(r[name], want[name]))
    assert torch.equal(_bits(a)[1], _bits(c)[1]) and torch.equal(_bits(a)[3], _bits(c)[3])
    z, early = turned(K, pos[:, None] if positions is None else positions, freq, axis, pairs, 1.0, w[1], EPS)
    big = z.abs().amax(-1)
    scale = a.k_scale[at, :, slot].double()
    assert ((scale - big / 448).abs() <= (early.amax(-1) / 448) + big / 448 * 2.0 ** -23).all()
    code = a.k.view(torch.uint8)[at, :, slot].view(F8).double()
    per = torch.where(big > 0, 448 / big.clamp_min(1e-300), torch.zeros_like(big))[..., None]
    ratio = z * per
    slack = early * per + 448 * per * early.amax(-1, keepdim=True) / 448 + ratio.abs() * 2.0 ** -22
    assert ((code - ratio).abs() <= (ratio.abs() * 2.0 ** -4).clamp_min(2.0 ** -10) + slack).all()
    untouched = torch.ones(s.shape[0], s.shape[2], dtype=torch.bool, device=DEV)
    untouched[at, slot] = False
    untouched = untouched[:, None].expand(-1, kv_heads, -1)
    assert (a.k.view(torch.uint8)[untouched] == 0x7F).all() and torch.isnan(a.k_scale[untouched]).all()


def test_keys_as_they_come_are_quantised_as_the_write_does():
    """No rope and no norm of keys: midpoints are decided as in exact arithmetic."""
    g = torch.Generator().manual_seed(6)
    n, dim = 96, 128
    x = torch.randint(-127, 128, (n, 2, dim), generator=g).float() / 128 * 1.75
    x[:, :, 0] = 1.75
    x = x * torch.exp2(torch.randint(-125, 60, (n, 2, 1), generator=g).float())
    x[5] = 0
    x[9, 1, 3] = float("inf")
    x = x.to(BF).to(DEV)
    s = Paged([n], 2, dim, 16, F8)
    a, b = s.empty(), s.empty()
    binding.rope_write(a, None, x, x.flip(0).contiguous(), _i32([0, n]), _i32([n]), s.table,
                       norm=binding.HeadNorm(q=torch.ones(dim, device=DEV)))
    binding.kv_write(b, x, x.flip(0).contiguous(), _i32([0, n]), _i32([n]), s.table)
    for u, v in zip(_bits(a), _bits(b)):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dim,rot,pairs,heads", [(128, 128, False, 3), (64, 64, True, 2), (128, 32, True, 1)])
def test_keys_turned_by_nothing_are_quantised_as_the_write_does(dim, rot, pairs, heads):
    """Positions of 0 turn by nothing: codes and scales are the write's, bit for bit,
    midpoints of two codes among them; at other positions that holds for what lies
    behind the turned values, where the row's largest value lies there too."""
    g = torch.Generator().manual_seed(dim + rot)
    n = 200
    # rows of +-m c / 2^s with the largest 7 m: quotients 64 c / 2^s, midpoints for odd c
    # of 5 bits, and 64 / m is inexact
    m = torch.tensor([3, 5, 7, 9, 11, 13])[torch.arange(n) % 6][:, None, None]
    c = torch.randint(8, 16, (n, heads, dim), generator=g) * 2 + 1
    c = torch.where(c * m > 255, torch.full((), 17), c) * torch.randint(0, 2, c.shape, generator=g).mul(2).sub(1)
    x = (m * c).float() * torch.exp2(-torch.randint(3, 9, c.shape, generator=g).float())
    x[:, :, -1:] = 7.0 * m
    x[n // 2:] *= 2.0 ** -105                                 # below 2^-100 the rows are scaled up first
    K = x.to(BF).to(DEV)
    V = torch.zeros_like(K)
    s = Paged([n], heads, dim, 16, F8, seed=1)
    args = (_off([n]), _i32([n]), s.table)
    a, b, c = s.empty(), s.empty(), s.empty()
    rope = binding.Rope(_freq(rot), interleaved=pairs)
    binding.kv_write(b, K, V, *args)
    binding.rope_write(a, None, K, V, *args, rope=rope, positions=torch.zeros(n, dtype=torch.int32, device=DEV))
    for x, y in zip(_bits(a), _bits(b)):
        assert torch.equal(x, y)
    if rot < dim:
        # (a pair of values up to 31 m / 8 turns to 5.5 m at most)
        binding.rope_write(c, None, K, V, *args, rope=rope)
        codes, _, scale, _ = _bits(c)
        want, _, ours, _ = _bits(b)
        assert torch.equal(scale, ours) and torch.equal(codes[..., rot:], want[..., rot:])


def test_tiny_keys_keep_their_precision():
    """Turned rows far below 1 (their reciprocals would overflow float32)."""
    g = torch.Generator().manual_seed(7)
    n, dim = 64, 64
    size = torch.exp2(torch.linspace(-118, -90, n))[:, None, None]
    K = (torch.randn((n, 1, dim), generator=g) * size).to(BF).to(DEV)
    s = Paged([n], 1, dim, 16, F8)
    a = s.empty()
    binding.rope_write(a, None, K, K, _i32([0, n]), _i32([n]), s.table, rope=binding.Rope(_freq(dim)))
    pos, at, slot = _places([n], [n], 16, s.table)
    z, early = turned(K, pos[:, None], _freq(dim))
    big = z.abs().amax(-1, keepdim=True)
    code = a.k.view(torch.uint8)[at, :, slot].view(F8).double()
    ratio = z * 448 / big
    slack = (early + early.amax(-1, keepdim=True)) * 448 / big + ratio.abs() * 2.0 ** -22
    assert ((code - ratio).abs() <= (ratio.abs() * 2.0 ** -4).clamp_min(2.0 ** -10) + slack).all()


def test_tokens_without_a_place_or_a_request():
    g = torch.Generator().manual_seed(8)
    dim, page, hk = 64, 16, 2
    q, K, V = _rand(g, 12, 3, dim), _rand(g, 12, hk, dim), _rand(g, 12, hk, dim)
    rope = binding.Rope(_freq(dim))
    for dtype in (BF, F8):
        # request 0: 4 new tokens of 2 cached ones; rows 0 and 10, 11 belong to nobody
        cache = binding.KvCache.empty(2, hk, page, dim, dtype, DEV)
        cache.k.view(torch.uint8).fill_(0)
        out = dict(q=torch.full((12, 3, dim), 7.0, dtype=BF, device=DEV), k=torch.full((12, hk, dim), 7.0, dtype=BF, device=DEV))
        r = binding.rope_write(cache, q, K, V, _i32([1, 5, 10]), _i32([2, 7]), _i32([[1], [0]]), rope=rope, out=out)
        assert binding.workspace_status(r["ws"]) == 0
        pos = _i32([0, -2, -1, 0, 1, 2, 3, 4, 5, 6, 0, 0])
        want = binding.qk_rope(q, K, pos, rope)
        for name in ("q", "k"):
            assert torch.equal(out[name][1:10], want[name][1:10])
            assert (out[name][[0, 10, 11]] == 7).all()
        back = binding.kv_read(cache, _i32([0, 2]), _i32([[1]]), 2)
        if dtype == BF:
            assert torch.equal(back["K"], want["k"][3:5])
        assert (cache.k.view(torch.uint8)[1, :, 2:] == 0).all() and (cache.k.view(torch.uint8)[0, :, :2] == 0).all()
        # pages out of range: recorded, not written; the rows come out all the same
        before = [x.clone() for x in _bits(cache)]
        for bad in (-1, 2, 2 ** 31 - 1):
            r = binding.rope_write(cache, q, K, V, _i32([0, 12]), _i32([12]), _i32([[bad]]), rope=rope, keep=True)
            assert binding.workspace_status(r["ws"]) == -9
            same = binding.qk_rope(q, K, _i32(list(range(12))), rope)
            assert torch.equal(r["q"], same["q"]) and torch.equal(r["k"], same["k"])
            assert all(torch.equal(x, y) for x, y in zip(before, _bits(cache)))
        for off, kv in (([0, 13], [12]), ([-1, 12], [12]), ([0, 12], [17]), ([0, 12], [-3])):
            r = binding.rope_write(cache, q, K, V, _i32(off), _i32(kv), _i32([[0]]), rope=rope)
            assert binding.workspace_status(r["ws"]) == -9


def test_no_tokens_at_all():
    q, k = torch.empty((0, 4, 64), dtype=BF, device=DEV), torch.empty((0, 2, 64), dtype=BF, device=DEV)
    rope = binding.Rope(_freq(64))
    assert binding.qk_rope(q, k, torch.empty(0, dtype=torch.int32, device=DEV), rope)["k"].shape == (0, 2, 64)
    cache = binding.KvCache.empty(1, 2, 16, 64, BF, DEV)
    assert binding.rope_write(cache, q, k, k, _i32([0, 0]), _i32([0]), _i32([[0]]), rope=rope)["q"].shape == (0, 4, 64)


def test_streams_and_graphs():
    g = torch.Generator().manual_seed(9)
    dim, page, hk, heads = 128, 16, 2, 8
    kv, new = [90, 7, 33], [6, 1, 4]
    s = Paged([100] * 3, hk, dim, page, F8)
    q, K, V = _rand(g, 11, heads, dim), _rand(g, 11, hk, dim), _rand(g, 11, hk, dim)
    w = _weights(g, dim, "qk")                       # device memory that the graph reads: kept
    rope, norm = binding.Rope(_freq(dim)), _norm(w)
    off, kv_len = _off(new), _i32(kv)
    a, b = s.empty(), s.empty()
    first = binding.rope_write(a, q, K, V, off, kv_len, s.table, rope=rope, norm=norm, keep=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = binding.rope_write(b, q, K, V, off, kv_len, s.table, rope=rope, norm=norm, keep=True, stream=side,
                               ws=torch.zeros_like(first["ws"]), out=dict(q=torch.empty_like(q), k=torch.empty_like(K)))
    side.synchronize()
    assert torch.equal(first["q"], other["q"]) and torch.equal(first["k"], other["k"])
    assert all(torch.equal(x, y) for x, y in zip(_bits(a), _bits(b)))
    c = s.empty()
    out, ws = dict(q=torch.empty_like(q), k=torch.empty_like(K)), torch.zeros_like(first["ws"])
    pos, rows = _i32([0] * 11), dict(q=torch.empty_like(q), k=torch.empty_like(K))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.rope_write(c, q, K, V, off, kv_len, s.table, rope=rope, norm=norm, keep=True, ws=ws, out=out)
        binding.qk_rope(q, K, pos, rope, norm, out=rows)
    del rope, norm                                   # the structs were read when the calls were made
    for lens in ([10, 20, 30], kv):
        kv_len.copy_(torch.tensor(lens))
        pos.copy_(torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]))
        graph.replay()
        assert torch.equal(out["q"], rows["q"]) and torch.equal(out["k"], rows["k"])
    assert torch.equal(out["q"], first["q"])


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 1, 64, 16), (5, 3, 128, 64), (33, 9, 64, 256), (17, 17, 128, 16)])
def test_calls_write_their_buffers_only(dtype, heads, kv_heads, dim, page):
    kv, new = [1, 40, 0, 700, 129, 64], [1, 7, 0, 3, 129, 2]
    g = torch.Generator().manual_seed(heads + page)
    T = sum(new)
    s = Paged(kv, kv_heads, dim, page, dtype)
    mem = Arena(4 * s.pages * kv_heads * page * dim * 2 + T * (heads + kv_heads) * dim * 8 + (24 << 20))
    cache = binding.KvCache(mem.take(s.shape, dtype), mem.take(s.shape, dtype),
                            *((mem.take(s.shape[:3], F32) for _ in range(2)) if dtype == F8 else ()))
    ws = mem.workspace(binding.load().dspark_kv_workspace_size())
    q, K, V = _rand(g, T, heads, dim), _rand(g, T, kv_heads, dim), _rand(g, T, kv_heads, dim)
    rope, norm = binding.Rope(_freq(dim // 2)), _norm(_weights(g, dim, "qk"))
    out = dict(q=mem.take((T, heads, dim), BF), k=mem.take((T, kv_heads, dim), BF))
    binding.rope_write(cache, q, K, V, _off(new), _i32(kv), s.table, rope=rope, norm=norm, ws=ws, out=out)
    mem.check()
    assert binding.workspace_status(ws) == 0
    rows = dict(q=mem.take((T, heads, dim), BF), k=mem.take((T, kv_heads, dim), BF))
    binding.qk_rope(q, K, torch.arange(T, dtype=torch.int32, device=DEV), rope, norm, out=rows)
    mem.check()


def test_cache_past_32_bit_offsets():
    dim, hk, page = 128, 8, 16
    n_pages = (1 << 31) // (hk * page * dim) + 700
    g = torch.Generator().manual_seed(4)
    n = 50
    K, V = _rand(g, n, hk, dim), _rand(g, n, hk, dim)
    table = (n_pages - 1 - torch.arange(4, dtype=torch.int32, device=DEV))[None]
    rope = binding.Rope(_freq(dim))
    for dtype in (BF, F8):
        cache = binding.KvCache.empty(n_pages, hk, page, dim, dtype, DEV)
        r = binding.rope_write(cache, None, K, V, _i32([0, n]), _i32([n]), table, rope=rope, keep=True)
        back = binding.kv_read(cache, _i32([0, n]), table, n)
        assert binding.workspace_status(r["ws"]) == 0
        if dtype == BF:
            assert torch.equal(back["K"], r["k"]) and torch.equal(back["V"], V)
        else:
            # half an e4m3 step of the row's largest, 2^-4, and two bf16 roundings
            big = r["k"].double().abs().amax(-1, keepdim=True)
            assert ((back["K"].double() - r["k"].double()).abs() <= big * (2.0 ** -4 + 2.0 ** -7)).all()
        del cache


def test_rows_that_are_not_device_memory_are_refused():
    L = binding.load()
    T, heads, hk, dim = 3, 4, 2, 64
    cache = binding.KvCache.empty(2, hk, 16, dim, BF, DEV)
    b = binding._batch(_i32([0, T]), _i32([T]), _i32([[0, 1]]), T)
    c, b = ctypes.byref(cache._struct()), ctypes.byref(b)
    shapes = dict(q=heads, K=hk, V=hk, qo=heads, ko=hk)
    dev = {n: torch.zeros((T, h, dim), dtype=BF, device=DEV) for n, h in shapes.items()}
    host = {n: torch.zeros((T, h, dim), dtype=BF).pin_memory() for n, h in shapes.items()}
    ws, pos, rope = binding._workspace(256, DEV), _i32([0, 1, 2]), binding.Rope(_freq(dim))
    torch.cuda.synchronize()

    def at(name, moved):
        return (host if name == moved else dev)[name].data_ptr()

    places = [pos, torch.zeros(3, dtype=torch.int32).pin_memory()]
    weights = [torch.ones(dim, device=DEV), torch.ones(dim).pin_memory()]

    def norm(m):
        return ctypes.byref(binding._HeadNorm(weights[m == "wq"].data_ptr(), weights[m == "wk"].data_ptr(), 0, EPS))

    def write(m):
        return L.dspark_rope_write(c, b, at("q", m), at("K", m), at("V", m), 256, 128, 128, heads, places[m == "pos"].data_ptr(),
                                   rope._ref, norm(m), at("qo", m), at("ko", m), 256, 128, ws.data_ptr(), 256, None)

    def turn(m):
        return L.dspark_qk_rope(at("q", m), at("K", m), 256, 128, places[m == "pos"].data_ptr(), T, heads, hk, dim, rope._ref,
                                norm(m), at("qo", m), at("ko", m), 256, 128, None)

    for call, names in ((write, "q K V qo ko pos wq wk"), (turn, "q K qo ko pos wq wk")):
        assert call(None) == 0
        for name in names.split():
            assert call(name) == -1, name
    torch.cuda.synchronize()
