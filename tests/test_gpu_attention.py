"""Paged cache, paged attention and prompt attention against plain 64-bit forms."""
import math

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from _attention import attend, quantise

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


class Scene:
    """A paged cache filled with the requests' tokens; every place that no
    token holds is NaN (and its scale too)."""

    def __init__(self, kv, heads, kv_heads, dim, page, dtype, seed=0, extra=3, size=1.5):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.heads, self.kv_heads, self.dim, self.page, self.dtype = kv, heads, kv_heads, dim, page, dtype
        counts = [-(-n // page) for n in kv]
        self.n_pages = sum(counts) + extra
        most = max(max(counts), 1)
        order = torch.randperm(self.n_pages, generator=g)
        self.table = torch.full((len(kv), most), -1, dtype=torch.int32)
        at = 0
        for r, c in enumerate(counts):
            self.table[r, :c] = order[at:at + c].to(torch.int32)
            at += c
        self.K = [_rand(g, n, kv_heads, dim, size=size) for n in kv]
        self.V = [_rand(g, n, kv_heads, dim, size=size) for n in kv]
        shape = (self.n_pages, kv_heads, page, dim)
        nan = float("nan")
        if dtype == BF:
            self.cache = binding.KvCache(torch.full(shape, nan, dtype=BF, device=DEV),
                                         torch.full(shape, nan, dtype=BF, device=DEV))
        else:
            junk = torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV).view(F8)
            self.cache = binding.KvCache(junk, junk.clone(), torch.full(shape[:3], nan, device=DEV),
                                         torch.full(shape[:3], nan, device=DEV))
        self.g = g
        self.page_table = self.table.to(DEV)
        if sum(kv):
            ws = binding.kv_write(self.cache, torch.cat(self.K), torch.cat(self.V), _off(kv), _i32(kv), self.page_table)
            torch.cuda.synchronize()
            assert binding.workspace_status(ws) == 0
        if dtype == F8:      # what the cache stands for
            self.K = [self._stored(x) for x in self.K]
            self.V = [self._stored(x) for x in self.V]

    @staticmethod
    def _stored(x):
        y, s = quantise(x)
        return y * s.float().double()[..., None]

    def check(self, q_len, q=None, scale=None, **kw):
        T = sum(q_len)
        scale = 0.7 / math.sqrt(self.dim) if scale is None else scale
        if q is None:
            q = _rand(self.g, T, self.heads, self.dim)
        r = binding.attn_paged(q, self.cache, _off(q_len), _i32(self.kv), self.page_table, scale=scale, lse=True, **kw)
        torch.cuda.synchronize()
        assert binding.workspace_status(r["ws"]) == 0
        at = 0
        for i, (n, m) in enumerate(zip(self.kv, q_len)):
            seen = torch.arange(m) + (n - m + 1)
            want, lse, bo, bl = attend(q[at:at + m], self.K[i], self.V[i], seen, scale)
            _close(r["out"][at:at + m], want, bo, f"out of request {i} (kv {n}, q {m})")
            _close(r["lse"][at:at + m], lse, bl, f"lse of request {i} (kv {n}, q {m})")
            at += m
        return q, r


def _close(got, want, bound, what):
    got = got.double()
    assert torch.equal(torch.isinf(got), torch.isinf(want)), what
    assert not torch.isnan(got).any(), what
    d = torch.where(torch.isinf(want), torch.zeros_like(want), got - want).abs()
    over = d - bound
    assert d.numel() == 0 or over.max().item() <= 0, f"{what}: off by {d.max().item():.3e}, over by {over.max().item():.3e}"


# ------------------------------------------------------------------ the cache
@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("dim,page,kv_heads", [(64, 16, 1), (128, 64, 3), (128, 256, 8), (64, 128, 5)])
def test_write_and_read(dtype, dim, page, kv_heads):
    kv = [1, 0, page, page + 1, 300, 17]
    s = Scene(kv, kv_heads, kv_heads, dim, page, dtype, seed=dim + page)
    r = binding.kv_read(s.cache, _off(kv), s.page_table, sum(kv))
    torch.cuda.synchronize()
    assert binding.workspace_status(r["ws"]) == 0
    for name, rows in (("K", s.K), ("V", s.V)):
        want = torch.cat([x.double() for x in rows])
        assert torch.equal(r[name].double(), want.to(torch.float32).to(BF).double() if dtype == F8 else want)
    # nothing but the tokens' places was written
    used = torch.zeros((s.n_pages, page), dtype=torch.bool)
    for i, n in enumerate(kv):
        for j in range(n):
            used[s.table[i, j // page], j % page] = True
    free = ~used.to(DEV)[:, None, :].expand(-1, kv_heads, -1)
    if dtype == BF:
        assert torch.isnan(s.cache.k[free]).all() and torch.isnan(s.cache.v[free]).all()
    else:
        assert (s.cache.k.view(torch.uint8)[free] == 0x7F).all() and torch.isnan(s.cache.v_scale[free]).all()


def test_quantised_codes_are_the_nearest_ones():
    """Every code against the 64-bit definition: ordinary rows, rows whose
    quotients are midpoints, zero, tiny, huge and subnormal rows."""
    g = torch.Generator().manual_seed(5)
    dim, n = 128, 512
    x = torch.randn((n, 1, dim), generator=g) * torch.exp2(torch.randint(-130, 120, (n, 1, 1), generator=g).float())
    for i in range(0, n, 4):                     # largest value 7 2^k: quotients m 2^j hit midpoints
        top = [1.75, 1.0, 1.25, 1.5, 448.0, 3.5][(i // 4) % 6]
        x[i] = torch.randint(-127, 128, (1, dim), generator=g).float() / 128 * top
        x[i, 0, 0] = top
    x[7] = 0
    x[11] = 1e-39
    x[13] = 3.3e38
    x = x.to(BF).to(DEV)
    page = 16
    cache = binding.KvCache.empty(n // page, 1, page, dim, F8, DEV)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None]
    binding.kv_write(cache, x, x.flip(0).contiguous(), _i32([0, n]), _i32([n]), table)
    code, scale = quantise(x)
    got = cache.k.view(torch.uint8).transpose(1, 2).reshape(n, 1, dim).view(F8).double()
    assert torch.equal(got, code)
    assert torch.equal(cache.k_scale.transpose(1, 2).reshape(n, 1), scale.float())
    assert torch.equal(cache.v.view(torch.uint8).transpose(1, 2).reshape(n, 1, dim).flip(0).view(F8).double(), code)


def test_a_row_that_is_not_finite_reads_back_as_nan_and_alone():
    dim, page = 64, 16
    x = torch.ones((3, 2, dim), dtype=BF, device=DEV)
    x[1, 0, 5] = float("inf")
    x[2, 1, 63] = float("nan")
    for dtype in (F8,):
        cache = binding.KvCache.empty(1, 2, page, dim, dtype, DEV)
        table = _i32([[0]])
        binding.kv_write(cache, x, x, _i32([0, 3]), _i32([3]), table)
        r = binding.kv_read(cache, _i32([0, 3]), table, 3)
        bad = torch.zeros((3, 2), dtype=torch.bool, device=DEV)
        bad[1, 0] = bad[2, 1] = True
        for name in ("K", "V"):
            assert torch.isnan(r[name][bad]).all()
            assert (r[name][~bad] == 1).all()


def test_writes_of_strided_rows_and_of_tokens_without_a_place():
    """K and V as slices of one projection; a request whose cache is shorter
    than its block writes only the tokens that have a position."""
    g = torch.Generator().manual_seed(2)
    hk, dim, page = 2, 64, 16
    fused = _rand(g, 9, 2 * hk + 3, dim)
    K, V = fused[:, :hk], fused[:, hk:2 * hk]
    for dtype in (BF, F8):
        cache = binding.KvCache.empty(2, hk, page, dim, dtype, DEV)
        cache.k.view(torch.uint8).zero_()
        # request 0: 4 new tokens of 2 cached ones: the first two have no place
        binding.kv_write(cache, K, V, _i32([0, 4, 9]), _i32([2, 7]), _i32([[1], [0]]))
        r = binding.kv_read(cache, _i32([0, 2]), _i32([[1]]), 2)
        want = K[2:4].double()
        if dtype == F8:
            want = Scene._stored(K[2:4]).float().to(BF).double()
        assert torch.equal(r["K"].double(), want)
        r = binding.kv_read(cache, _i32([0, 7]), _i32([[0]]), 7)
        got = r["K"][2:].double()
        want = K[4:9].double() if dtype == BF else Scene._stored(K[4:9]).float().to(BF).double()
        assert torch.equal(got, want)
        assert (cache.k.view(torch.uint8)[1, :, 2:] == 0).all()


# ------------------------------------------------------------------ paged attention
@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [
    (8, 2, 128, 16), (4, 4, 64, 32), (6, 2, 128, 64), (8, 1, 64, 128), (5, 1, 128, 256), (24, 2, 64, 16)])
def test_paged_lengths(dtype, heads, kv_heads, dim, page):
    """Lengths from none to several tiles, odd ones, blocks longer than the
    cache (tokens without keys) and requests without tokens."""
    kv = [1, 0, 15, 16, 17, 127, 128, 129, 300, 5, 2, 257, 0, 640]
    q = [1, 1, 3, 1, 0, 6, 5, 2, 1, 5, 4, 17, 0, 1]
    Scene(kv, heads, kv_heads, dim, page, dtype, seed=heads).check(q)


@pytest.mark.parametrize("dtype", [BF, F8])
def test_paged_one_request_split_over_the_device(dtype):
    Scene([20011], 8, 2, 128, 16, dtype, seed=1).check([3])
    Scene([9000], 4, 1, 64, 64, dtype, seed=2).check([1])


@pytest.mark.parametrize("heads,kv_heads", [(128, 1), (100, 1), (48, 3), (17, 17)])
def test_paged_many_rows(heads, kv_heads):
    """Row counts that fill several row tiles, with groups up to 128."""
    Scene([200, 33], heads, kv_heads, 64, 32, BF, seed=3).check([7, 33])
    Scene([140], heads, kv_heads, 128, 16, F8, seed=4).check([40])


def test_paged_many_requests():
    g = torch.Generator().manual_seed(9)
    kv = torch.randint(0, 400, (300,), generator=g).tolist()
    q = [min(n, 1 + i % 6) for i, n in enumerate(kv)]
    s = Scene(kv, 8, 2, 64, 16, BF, seed=5)
    s.check(q)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("heads,kv_heads,dim,most", [(24, 4, 64, 700), (16, 4, 128, 300), (32, 8, 64, 1500)])
def test_paged_row_tiles_of_changing_shape(dtype, heads, kv_heads, dim, most):
    """Several segments to a worker whose row tiles change between few and many
    rows, with one key tile or several, and lengths of zero in between."""
    g = torch.Generator().manual_seed(most)
    n = 330
    kv = torch.randint(0, most, (n,), generator=g).tolist()
    q = torch.randint(0, 18, (n,), generator=g).tolist()
    for i in range(0, n, 9):                     # long quiet runs of one shape, then a change
        if i % 27:
            q[i:i + 9] = [1] * len(q[i:i + 9])
    s = Scene(kv, heads, kv_heads, dim, 16, dtype, seed=most)
    _, first = s.check(q)
    _, second = s.check(q[::-1])
    assert not torch.equal(first["out"], second["out"])


@pytest.mark.parametrize("dtype", [BF, F8])
def test_paged_sharp_and_flat_scores(dtype):
    """Scores far apart (one key takes all the weight, the maximum moves late)
    and all equal."""
    s = Scene([700], 4, 2, 128, 16, dtype, seed=6, size=8.0)
    s.check([4], scale=1.0)
    s.check([4], scale=0.0)
    s.check([4], scale=-0.3)


def test_paged_rerun_streams_strides_and_graph():
    s = Scene([3000, 70, 513], 8, 2, 128, 16, F8, seed=7)
    q_len = [6, 1, 4]
    q, first = s.check(q_len)
    args = (s.cache, _off(q_len), _i32(s.kv), s.page_table)
    scale = 0.7 / math.sqrt(128)
    again = binding.attn_paged(q, *args, scale=scale, lse=True, ws=first["ws"])
    assert torch.equal(again["out"], first["out"]) and torch.equal(again["lse"], first["lse"])
    # a strided q (a slice of a fused projection) on a side stream
    fused = torch.full((11, 12, 128), float("nan"), dtype=BF, device=DEV)
    fused[:, :8] = q
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = binding.attn_paged(fused[:, :8], *args, scale=scale, lse=True, stream=side,
                               ws=torch.zeros_like(first["ws"]))
    side.synchronize()
    assert torch.equal(other["out"], first["out"]) and torch.equal(other["lse"], first["lse"])
    # captured once, replayed at other lengths
    kv_len = _i32(s.kv)
    out = dict(out=torch.zeros_like(first["out"]), lse=torch.zeros_like(first["lse"]))
    ws = torch.zeros_like(first["ws"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.attn_paged(q, s.cache, args[1], kv_len, s.page_table, scale=scale, ws=ws, out=out)
    for kv in ([2990, 70, 512], [9, 3, 4], s.kv):
        kv_len.copy_(torch.tensor(kv))
        graph.replay()
        want = binding.attn_paged(q, s.cache, args[1], kv_len, s.page_table, scale=scale, lse=True)
        assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])


def test_paged_rows_of_no_request_stay():
    s = Scene([40], 4, 2, 64, 16, BF, seed=8)
    q = _rand(s.g, 5, 4, 64)
    out = dict(out=torch.full((5, 4, 64), 7.0, dtype=BF, device=DEV), lse=torch.full((5, 4), 7.0, device=DEV))
    binding.attn_paged(q, s.cache, _i32([1, 3]), _i32([40]), s.page_table, out=out)
    stay = torch.tensor([True, False, False, True, True], device=DEV)
    assert (out["out"][stay] == 7).all() and (out["lse"][stay] == 7).all()
    want, _, bo, _ = attend(q[1:3], s.K[0], s.V[0], torch.tensor([39, 40]), 1 / 8)
    _close(out["out"][1:3], want, bo, "the request's rows")


def test_paged_cache_past_32_bit_offsets():
    """A cache of more than 2^31 values, the tokens in its last pages."""
    dim, hk, page = 128, 8, 16
    n_pages = (1 << 31) // (hk * page * dim) + 700
    for dtype in (BF, F8):
        cache = binding.KvCache.empty(n_pages, hk, page, dim, dtype, DEV)
        g = torch.Generator().manual_seed(4)
        n = 333
        K, V = _rand(g, n, hk, dim), _rand(g, n, hk, dim)
        table = (n_pages - 1 - torch.arange(21, dtype=torch.int32, device=DEV))[None]
        ws = binding.kv_write(cache, K, V, _i32([0, n]), _i32([n]), table)
        q = _rand(g, 2, 16, dim)
        r = binding.attn_paged(q, cache, _i32([0, 2]), _i32([n]), table, lse=True)
        back = binding.kv_read(cache, _i32([0, n]), table, n)
        assert binding.workspace_status(ws) == 0 and binding.workspace_status(r["ws"]) == 0
        k, v = (K, V) if dtype == BF else (Scene._stored(K), Scene._stored(V))
        assert torch.equal(back["K"].double(), k.float().to(BF).double())
        want, lse, bo, bl = attend(q, k, v, torch.tensor([n - 1, n]), dim ** -0.5)
        _close(r["out"], want, bo, "out")
        _close(r["lse"], lse, bl, "lse")
        del cache


# ------------------------------------------------------------------ prompts
def _check_prompt(lens, heads, kv_heads, dim, seed=0, scale=None, size=1.5, q=None, k=None, v=None):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    q = _rand(g, T, heads, dim) if q is None else q
    k = _rand(g, T, kv_heads, dim, size=size) if k is None else k
    v = _rand(g, T, kv_heads, dim, size=size) if v is None else v
    scale = 0.7 / math.sqrt(dim) if scale is None else scale
    r = binding.attn_prompt(q, k, v, _off(lens), scale=scale, lse=True)
    torch.cuda.synchronize()
    assert binding.workspace_status(r["ws"]) == 0
    a = 0
    for i, n in enumerate(lens):
        want, lse, bo, bl = attend(q[a:a + n], k[a:a + n], v[a:a + n], torch.arange(1, n + 1), scale)
        _close(r["out"][a:a + n], want, bo, f"out of sequence {i} ({n} tokens)")
        _close(r["lse"][a:a + n], lse, bl, f"lse of sequence {i} ({n} tokens)")
        a += n
    return q, k, v, r


@pytest.mark.parametrize("heads,kv_heads,dim", [
    (4, 4, 64), (4, 4, 128), (8, 2, 128), (6, 2, 64), (3, 1, 128), (16, 1, 64), (7, 1, 128), (128, 1, 64), (100, 1, 128)])
def test_prompt_lengths(heads, kv_heads, dim):
    _check_prompt([1, 5, 0, 63, 64, 65, 127, 128, 129, 0, 300, 2], heads, kv_heads, dim, seed=heads)


def test_prompt_one_long_sequence():
    _check_prompt([2500], 4, 2, 128, seed=1)
    _check_prompt([2049], 4, 1, 64, seed=2)


def test_prompt_sharp_and_flat_scores():
    for scale in (1.0, 0.0, -0.3):
        _check_prompt([400, 77], 4, 2, 128, seed=3, scale=scale, size=6.0)


def test_prompt_many_sequences():
    g = torch.Generator().manual_seed(1)
    _check_prompt(torch.randint(0, 90, (200,), generator=g).tolist(), 4, 2, 64, seed=4)


def test_prompt_sequences_do_not_mix():
    """A sequence of NaN and infinities between two others leaves them alone."""
    g = torch.Generator().manual_seed(6)
    lens = [70, 50, 201]
    q, k, v = (_rand(g, 321, h, 128) for h in (8, 2, 2))
    clean = binding.attn_prompt(q, k, v, _off(lens), lse=True)
    for x, value in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        x[70:120] = value
    r = binding.attn_prompt(q, k, v, _off(lens), lse=True)
    for name in ("out", "lse"):
        assert torch.equal(r[name][:70], clean[name][:70])
        assert torch.equal(r[name][120:], clean[name][120:])


def test_prompt_strides_streams_and_graph():
    g = torch.Generator().manual_seed(7)
    lens = [130, 1, 77]
    fused = _rand(g, 208, 8 + 2 + 2, 64)
    q, k, v = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    _, _, _, r = _check_prompt(lens, 8, 2, 64, q=q, k=k, v=v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = binding.attn_prompt(q, k, v, _off(lens), scale=0.7 / 8, lse=True, stream=side, ws=torch.zeros_like(r["ws"]))
    side.synchronize()
    assert torch.equal(other["out"], r["out"]) and torch.equal(other["lse"], r["lse"])
    off = _off(lens)
    out = dict(out=torch.zeros_like(r["out"]), lse=torch.zeros_like(r["lse"]))
    ws = torch.zeros_like(r["ws"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.attn_prompt(q, k, v, off, ws=ws, out=out)
    for lengths in ([208, 0, 0], [1, 2, 205], lens):
        off.copy_(_off(lengths))
        graph.replay()
        want = binding.attn_prompt(q, k, v, _off(lengths), lse=True)
        assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])


def test_prompt_rows_of_no_sequence_stay():
    g = torch.Generator().manual_seed(8)
    q, k, v = (_rand(g, 20, h, 64) for h in (4, 2, 2))
    out = dict(out=torch.full((20, 4, 64), 7.0, dtype=BF, device=DEV), lse=torch.full((20, 4), 7.0, device=DEV))
    binding.attn_prompt(q, k, v, _i32([3, 9, 15]), out=out)
    for rows in (slice(0, 3), slice(15, 20)):
        assert (out["out"][rows] == 7).all() and (out["lse"][rows] == 7).all()
    want, _, bo, _ = attend(q[9:15], k[9:15], v[9:15], torch.arange(1, 7), 1 / 8)
    _close(out["out"][9:15], want, bo, "second sequence")


def test_prompt_agrees_with_the_paged_form():
    """The whole prompt as one block over a cache that holds it."""
    g = torch.Generator().manual_seed(10)
    n, heads, hk, dim = 333, 8, 2, 128
    s = Scene([n], heads, hk, dim, 32, BF, seed=11)
    q = _rand(g, n, heads, dim)
    s.check([n], q=q)
    _check_prompt([n], heads, hk, dim, q=q, k=s.K[0], v=s.V[0])


# ------------------------------------------------------------------ values out of range on the device
def test_bad_pages_lengths_and_offsets_are_recorded_and_stay_in_range():
    s = Scene([40, 50, 33], 4, 2, 64, 16, BF, seed=12)
    q = _rand(s.g, 3, 4, 64)
    good = binding.attn_paged(q, s.cache, _i32([0, 1, 2, 3]), _i32(s.kv), s.page_table, lse=True)
    ws = good["ws"]
    assert binding.workspace_status(ws) == 0
    for bad_id in (-5, s.n_pages, 2 ** 31 - 1):
        table = s.page_table.clone()
        table[1, 1] = bad_id
        r = binding.attn_paged(q, s.cache, _i32([0, 1, 2, 3]), _i32(s.kv), table, lse=True, ws=ws)
        assert binding.workspace_status(ws) == -9
        for i in (0, 2):
            assert torch.equal(r["out"][i], good["out"][i])
        k, v = s.K[1].clone(), s.V[1].clone()
        k[16:32] = 0
        v[16:32] = 0
        want, _, bo, _ = attend(q[1:2], k, v, torch.tensor([50]), 1 / 8)
        _close(r["out"][1:2], want, bo, "the missing page reads as zeros")
        back = binding.kv_read(s.cache, _i32([0, 40, 90, 123]), table, 123, ws=ws)
        assert binding.workspace_status(ws) == -9
        assert (back["K"][56:72] == 0).all() and torch.equal(back["K"][:40], s.K[0])
        before = s.cache.k.clone()
        binding.kv_write(s.cache, s.K[1][16:32], s.V[1][16:32], _i32([0, 0, 16, 16]), _i32([0, 32, 0]), table, ws=ws)
        assert binding.workspace_status(ws) == -9
        assert torch.equal(before.view(torch.int16), s.cache.k.view(torch.int16))
    for off, kv in (([0, 1, 2, 9], s.kv), ([-3, 1, 2, 3], s.kv), ([0, 2, 1, 3], s.kv), ([0, 1, 2, 3], [40, -1, 33]),
                    ([0, 1, 2, 3], [40, 2 ** 31 - 1, 33])):
        binding.attn_paged(q, s.cache, _i32(off), _i32(kv), torch.zeros_like(s.page_table), lse=True, ws=ws)
        assert binding.workspace_status(ws) == -9
    k = _rand(s.g, 3, 2, 64)
    for off in ([0, 9], [-1, 3], [2, 1]):
        r = binding.attn_prompt(q, k, k, _i32(off), ws=None)
        assert binding.workspace_status(r["ws"]) == -9
    assert binding.workspace_status(ws) == 0


def test_no_tokens_at_all():
    cache = binding.KvCache.empty(1, 2, 16, 64, BF, DEV)
    q, k = torch.empty((0, 4, 64), dtype=BF, device=DEV), torch.empty((0, 2, 64), dtype=BF, device=DEV)
    table = _i32([[0]])
    assert binding.attn_paged(q, cache, _i32([0, 0]), _i32([5]), table, lse=True)["out"].shape == (0, 4, 64)
    assert binding.attn_prompt(q, k, k, _i32([0, 0]), lse=True)["lse"].shape == (0, 4)
    binding.kv_write(cache, k, k, _i32([0, 0]), _i32([0]), table)
    assert binding.kv_read(cache, _i32([0, 0]), table, 0)["K"].shape == (0, 2, 64)
