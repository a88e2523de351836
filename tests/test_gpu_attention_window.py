"""Attention with a sliding window and sinks, over pages and over prompts, against
plain 64-bit forms."""
import math

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from _window import attend_masked, visible
from test_gpu_attention import Scene, _close, _i32, _off, _rand
from test_gpu_attention_memory import Arena

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def _spoil(s, q_len, window, sinks):
    """Pages and places that no new token of their request sees: ids out of range
    and places of NaN (pages are not shared).  Returns the table."""
    table = s.page_table.clone()
    for r, (n, m) in enumerate(zip(s.kv, q_len)):
        if m == 0 or n == 0:
            continue
        seen = visible(torch.arange(n - m, n), n, window, sinks).any(0)
        for j in range(-(-n // s.page)):
            own = seen[j * s.page:(j + 1) * s.page]
            page = int(s.table[r, j])
            if not own.any():
                table[r, j] = (-1, s.n_pages, 2 ** 31 - 1)[j % 3]
            for x in (s.cache.k, s.cache.v):
                gone = (~own).nonzero()[:, 0].to(DEV)
                if s.dtype == BF:
                    x[page, :, gone] = float("nan")
                else:
                    x.view(torch.uint8)[page, :, gone] = 0x7F
            if s.dtype == F8:
                for x in (s.cache.k_scale, s.cache.v_scale):
                    x[page, :, (~own).nonzero()[:, 0].to(DEV)] = float("nan")
    return table


def _check(s, q_len, window, sinks, spoil=True, scale=None, **kw):
    T = sum(q_len)
    scale = 0.7 / math.sqrt(s.dim) if scale is None else scale
    q = _rand(s.g, T, s.heads, s.dim)
    table = _spoil(s, q_len, window, sinks) if spoil else s.page_table
    r = binding.attn_paged(q, s.cache, _off(q_len), _i32(s.kv), table, scale=scale, lse=True, window=window, sinks=sinks, **kw)
    torch.cuda.synchronize()
    assert binding.workspace_status(r["ws"]) == 0
    at = 0
    for i, (n, m) in enumerate(zip(s.kv, q_len)):
        mask = visible(torch.arange(n - m, n), n, window, sinks).to(DEV)
        want, lse, bo, bl = attend_masked(q[at:at + m], s.K[i], s.V[i], mask, scale)
        _close(r["out"][at:at + m], want, bo, f"out of request {i} (kv {n}, q {m}, window {window}, sinks {sinks})")
        _close(r["lse"][at:at + m], lse, bl, f"lse of request {i} (kv {n}, q {m}, window {window}, sinks {sinks})")
        at += m
    return q, table, r


# ------------------------------------------------------------------ paged
KV = [1, 0, 15, 16, 17, 127, 128, 129, 300, 5, 2, 257, 0, 640, 1500]
Q = [1, 1, 3, 1, 0, 6, 5, 2, 1, 5, 4, 17, 0, 1, 9]


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 2, 128, 16), (4, 4, 64, 32), (6, 2, 128, 64), (8, 1, 64, 128), (5, 1, 128, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (17, 4), (128, 0), (129, 16), (100, 130), (300, 300), (640, 4), (4000, 3)])
def test_paged_lengths(dtype, heads, kv_heads, dim, page, window, sinks):
    _check(Scene(KV, heads, kv_heads, dim, page, dtype, seed=heads + window), Q, window, sinks)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [
    (8, 2, 128, 16), (4, 4, 64, 32), (24, 2, 128, 64), (20, 1, 64, 128), (40, 1, 128, 16), (64, 1, 64, 256), (100, 1, 64, 16)])
def test_paged_single_tokens(dtype, heads, kv_heads, dim, page):
    """One new token each, for every way that rows of a token are laid out; and as
    many tokens as requests that are not one each."""
    for window, sinks in ((1, 0), (16, 3), (128, 0), (130, 17), (300, 200), (1000, 4)):
        _check(Scene(KV, heads, kv_heads, dim, page, dtype, seed=heads + window), [min(n, 1) for n in KV], window, sinks)
        _check(Scene(KV, heads, kv_heads, dim, page, dtype, seed=heads), [1] + [1 - (n == 0) for n in KV[1:-1]] + [3],
               window, sinks)
    one = [n for n in KV if n]
    _check(Scene(one, heads, kv_heads, dim, page, dtype, seed=1), [1] * len(one), 140, 5)
    _check(Scene(one, heads, kv_heads, dim, page, dtype, seed=2), [1] * (len(one) - 3) + [0, 0, 3], 140, 5)


@pytest.mark.parametrize("dtype", [BF, F8])
def test_paged_single_tokens_sharp_and_flat_scores(dtype):
    for scale in (1.0, 0.0, -0.3):
        for heads, kv_heads in ((8, 1), (48, 1)):
            _check(Scene([700, 130], heads, kv_heads, 128, 16, dtype, seed=6, size=8.0), [1, 1], 200, 3, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F8])
def test_paged_one_request_split_over_the_device(dtype):
    for window, sinks in ((1024, 4), (9000, 1000), (20000, 1), (130, 5000), (1 << 40, 7)):
        _check(Scene([20011], 8, 2, 128, 16, dtype, seed=1), [3], window, sinks)
    _check(Scene([9000], 4, 1, 64, 64, dtype, seed=2), [1], 4096, 128)


@pytest.mark.parametrize("heads,kv_heads", [(128, 1), (100, 1), (48, 3), (17, 17)])
def test_paged_many_rows(heads, kv_heads):
    """Row counts that fill several row tiles, each with a window of its own."""
    _check(Scene([900, 333], heads, kv_heads, 64, 32, BF, seed=3), [200, 33], 70, 4)
    _check(Scene([740], heads, kv_heads, 128, 16, F8, seed=4), [140], 33, 0)
    _check(Scene([1400], heads, kv_heads, 128, 16, BF, seed=5), [600], 129, 140)


@pytest.mark.parametrize("dtype", [BF, F8])
def test_paged_many_requests(dtype):
    g = torch.Generator().manual_seed(9)
    kv = torch.randint(0, 900, (300,), generator=g).tolist()
    q = [min(n, (i * 7) % 18) for i, n in enumerate(kv)]
    _check(Scene(kv, 8, 2, 64, 16, dtype, seed=5), q, 140, 4)
    _check(Scene(kv, 24, 4, 128, 16, dtype, seed=6), q, 30, 0)


@pytest.mark.parametrize("dtype", [BF, F8])
def test_paged_sharp_and_flat_scores(dtype):
    for scale in (1.0, 0.0, -0.3):
        _check(Scene([700], 4, 2, 128, 16, dtype, seed=6, size=8.0), [4], 200, 3, scale=scale)


def test_paged_window_of_everything_is_none():
    s = Scene([300, 40], 8, 2, 128, 16, BF, seed=7)
    q = _rand(s.g, 5, 8, 128)
    args = (q, s.cache, _i32([0, 4, 5]), _i32(s.kv), s.page_table)
    want = binding.attn_paged(*args, lse=True)
    for window in (s.page_table.shape[1] * 16, 1 << 33):
        got = binding.attn_paged(*args, lse=True, window=window, sinks=2)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


@pytest.mark.parametrize("dtype", [BF, F8])
def test_paged_rerun_streams_and_graph(dtype):
    s = Scene([3000, 70, 513], 8, 2, 128, 16, dtype, seed=7)
    q_len = [6, 1, 4]
    q, _, first = _check(s, q_len, 500, 4, spoil=False)
    args = (s.cache, _off(q_len), _i32(s.kv), s.page_table)
    kw = dict(scale=0.7 / math.sqrt(128), lse=True, window=500, sinks=4)
    again = binding.attn_paged(q, *args, ws=first["ws"], **kw)
    assert torch.equal(again["out"], first["out"]) and torch.equal(again["lse"], first["lse"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = binding.attn_paged(q, *args, stream=side, ws=torch.zeros_like(first["ws"]), **kw)
    side.synchronize()
    assert torch.equal(other["out"], first["out"]) and torch.equal(other["lse"], first["lse"])
    kv_len = _i32(s.kv)
    out = dict(out=torch.zeros_like(first["out"]), lse=torch.zeros_like(first["lse"]))
    ws = torch.zeros_like(first["ws"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.attn_paged(q, s.cache, args[1], kv_len, s.page_table, ws=ws, out=out, **kw)
    for kv in ([2990, 70, 512], [9, 3, 4], s.kv):
        kv_len.copy_(torch.tensor(kv))
        graph.replay()
        want = binding.attn_paged(q, s.cache, args[1], kv_len, s.page_table, **kw)
        assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])


@pytest.mark.parametrize("dtype", [BF, F8])
def test_paged_bad_pages_that_are_seen_are_recorded(dtype):
    s = Scene([400], 4, 2, 64, 16, dtype, seed=8)
    q = _rand(s.g, 1, 4, 64)
    args = (_i32([0, 1]), _i32([400]))
    kw = dict(window=100, sinks=20)
    for j, want in ((0, -9), (1, -9), (2, 0), (10, 0), (17, 0), (18, -9), (24, -9)):
        table = s.page_table.clone()
        table[0, j] = s.n_pages
        r = binding.attn_paged(q, s.cache, *args, table, **kw)
        assert binding.workspace_status(r["ws"]) == want, j
    for off, kv in (([0, 2], [400]), ([-1, 1], [400]), ([0, 1], [-3]), ([0, 1], [401]), ([0, 1], [2 ** 31 - 1])):
        r = binding.attn_paged(q, s.cache, _i32(off), _i32(kv), s.page_table, **kw)
        assert binding.workspace_status(r["ws"]) == -9


def test_paged_cache_past_32_bit_offsets():
    dim, hk, page = 128, 8, 16
    n_pages = (1 << 31) // (hk * page * dim) + 700
    for dtype in (BF, F8):
        cache = binding.KvCache.empty(n_pages, hk, page, dim, dtype, DEV)
        g = torch.Generator().manual_seed(4)
        n = 333
        K, V = _rand(g, n, hk, dim), _rand(g, n, hk, dim)
        table = (n_pages - 1 - torch.arange(21, dtype=torch.int32, device=DEV))[None]
        binding.kv_write(cache, K, V, _i32([0, n]), _i32([n]), table)
        q = _rand(g, 2, 16, dim)
        r = binding.attn_paged(q, cache, _i32([0, 2]), _i32([n]), table, lse=True, window=100, sinks=4)
        assert binding.workspace_status(r["ws"]) == 0
        k, v = (K, V) if dtype == BF else (Scene._stored(K), Scene._stored(V))
        want, lse, bo, bl = attend_masked(q, k, v, visible(torch.tensor([n - 2, n - 1]), n, 100, 4).to(DEV), dim ** -0.5)
        _close(r["out"], want, bo, "out")
        _close(r["lse"], lse, bl, "lse")
        del cache


# ------------------------------------------------------------------ prompts
def _prompt(lens, heads, kv_heads, dim, window, sinks, seed=0, scale=None, size=1.5, q=None, k=None, v=None):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    q = _rand(g, T, heads, dim) if q is None else q
    k = _rand(g, T, kv_heads, dim, size=size) if k is None else k
    v = _rand(g, T, kv_heads, dim, size=size) if v is None else v
    scale = 0.7 / math.sqrt(dim) if scale is None else scale
    r = binding.attn_prompt(q, k, v, _off(lens), scale=scale, lse=True, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert binding.workspace_status(r["ws"]) == 0
    a = 0
    for i, n in enumerate(lens):
        mask = visible(torch.arange(n), n, window, sinks).to(DEV)
        want, lse, bo, bl = attend_masked(q[a:a + n], k[a:a + n], v[a:a + n], mask, scale)
        _close(r["out"][a:a + n], want, bo, f"out of sequence {i} ({n} tokens, window {window}, sinks {sinks})")
        _close(r["lse"][a:a + n], lse, bl, f"lse of sequence {i} ({n} tokens, window {window}, sinks {sinks})")
        a += n
    return q, k, v, r


@pytest.mark.parametrize("heads,kv_heads,dim", [
    (4, 4, 64), (2, 2, 128), (8, 2, 128), (6, 2, 64), (3, 1, 128), (16, 1, 64), (7, 1, 128), (128, 1, 64), (100, 1, 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 1), (64, 4), (128, 0), (129, 130), (200, 4), (100, 300), (1000, 5)])
def test_prompt_lengths(heads, kv_heads, dim, window, sinks):
    _prompt([1, 5, 0, 63, 64, 65, 127, 128, 129, 0, 300, 2, 700], heads, kv_heads, dim, window, sinks, seed=heads)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (127, 4), (128, 0), (129, 0), (257, 128), (512, 1), (1000, 256), (60, 1300)])
def test_prompt_long_sequences(window, sinks):
    _prompt([2500], 4, 2, 128, window, sinks, seed=1)
    _prompt([2049, 1], 2, 2, 64, window, sinks, seed=2)
    _prompt([1700], 8, 1, 64, window, sinks, seed=3)


def test_prompt_sharp_and_flat_scores():
    for scale in (1.0, 0.0, -0.3):
        _prompt([700, 77], 4, 2, 128, 150, 3, seed=3, scale=scale, size=6.0)


def test_prompt_many_sequences():
    g = torch.Generator().manual_seed(1)
    _prompt(torch.randint(0, 90, (200,), generator=g).tolist(), 4, 2, 64, 20, 2, seed=4)
    _prompt(torch.randint(0, 500, (90,), generator=g).tolist(), 2, 2, 128, 130, 0, seed=5)


def test_prompt_window_of_everything_is_none():
    g = torch.Generator().manual_seed(2)
    q, k, v = (_rand(g, 300, h, 64) for h in (4, 2, 2))
    want = binding.attn_prompt(q, k, v, _i32([0, 100, 300]), lse=True)
    for window in (300, 1 << 40):
        got = binding.attn_prompt(q, k, v, _i32([0, 100, 300]), lse=True, window=window)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 128), (3, 3, 64), (16, 2, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 3), (128, 0), (200, 150), (300, 2)])
def test_prompt_values_that_are_not_finite_reach_their_rows_alone(heads, kv_heads, dim, window, sinks):
    g = torch.Generator().manual_seed(window + heads)
    lens = [90, 1200, 64]
    T, first = sum(lens), 90
    q, k, v = (_rand(g, T, h, dim) for h in (heads, kv_heads, kv_heads))
    bad = {0: float("nan"), 1: float("inf"), 2: float("-inf"), 139: float("inf"), 300: float("inf"), 301: float("-inf"),
           512: float("nan"), 640: float("-inf"), 767: float("inf"), 1199: float("inf")}
    clean = v.clone()
    for at, x in bad.items():
        d = (at * 7) % (dim - 1)
        v[first + at, at % kv_heads, d], clean[first + at, at % kv_heads, d] = x, 0.0
    args = (_off(lens),)
    kw = dict(lse=True, window=window, sinks=sinks, scale=0.05)
    want = binding.attn_prompt(q, k, clean, *args, **kw)
    r = binding.attn_prompt(q, k, v, *args, **kw)
    torch.cuda.synchronize()
    assert binding.workspace_status(r["ws"]) == 0
    assert torch.equal(r["lse"], want["lse"])
    mask = visible(torch.arange(lens[1]), lens[1], window, sinks)
    expect = want["out"].float().clone()
    for at, x in bad.items():
        rows = first + mask[:, at].nonzero()[:, 0].to(DEV)
        group = heads // kv_heads
        c = at % kv_heads
        expect[rows, c * group:(c + 1) * group, (at * 7) % (dim - 1)] += x
    got = r["out"].float()
    assert torch.equal(torch.isnan(got), torch.isnan(expect))
    assert torch.equal(torch.nan_to_num(got, 0.0, 1e30, -1e30), torch.nan_to_num(expect, 0.0, 1e30, -1e30))


def test_prompt_keys_and_values_that_nobody_sees():
    """Sequences of NaN between others, and hidden keys of infinities, leave the rest alone."""
    g = torch.Generator().manual_seed(6)
    lens = [370, 50, 401]
    q, k, v = (_rand(g, sum(lens), h, 128) for h in (8, 2, 2))
    kw = dict(lse=True, window=30, sinks=0)
    clean = binding.attn_prompt(q, k, v, _off(lens), **kw)
    for x, value in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        x[370:420] = value
    k[100], v[100] = float("nan"), float("inf")
    r = binding.attn_prompt(q, k, v, _off(lens), **kw)
    for name in ("out", "lse"):
        for rows in (slice(0, 100), slice(130, 370), slice(420, 821)):
            assert torch.equal(r[name][rows], clean[name][rows])


def test_prompt_strides_streams_and_graph():
    g = torch.Generator().manual_seed(7)
    lens = [530, 1, 277]
    fused = _rand(g, sum(lens), 8 + 2 + 2, 64)
    q, k, v = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    _, _, _, r = _prompt(lens, 8, 2, 64, 100, 4, q=q, k=k, v=v)
    kw = dict(scale=0.7 / 8, lse=True, window=100, sinks=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = binding.attn_prompt(q, k, v, _off(lens), stream=side, ws=torch.zeros_like(r["ws"]), **kw)
    side.synchronize()
    assert torch.equal(other["out"], r["out"]) and torch.equal(other["lse"], r["lse"])
    off = _off(lens)
    out = dict(out=torch.zeros_like(r["out"]), lse=torch.zeros_like(r["lse"]))
    ws = torch.zeros_like(r["ws"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.attn_prompt(q, k, v, off, ws=ws, out=out, **kw)
    for lengths in ([808, 0, 0], [1, 2, 805], lens):
        off.copy_(_off(lengths))
        graph.replay()
        want = binding.attn_prompt(q, k, v, _off(lengths), **kw)
        assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])


def test_prompt_agrees_with_the_paged_form():
    g = torch.Generator().manual_seed(10)
    n, heads, hk, dim = 733, 8, 2, 128
    s = Scene([n], heads, hk, dim, 32, BF, seed=11)
    q = _rand(g, n, heads, dim)
    r = binding.attn_paged(q, s.cache, _i32([0, n]), _i32([n]), s.page_table, lse=True, window=150, sinks=5)
    mask = visible(torch.arange(n), n, 150, 5).to(DEV)
    want, lse, bo, bl = attend_masked(q, s.K[0], s.V[0], mask, dim ** -0.5)
    _close(r["out"], want, bo, "paged")
    _prompt([n], heads, hk, dim, 150, 5, q=q, k=s.K[0], v=s.V[0], scale=dim ** -0.5)


# ------------------------------------------------------------------ memory
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 1, 64), (4, 2, 128), (7, 1, 128)])
def test_calls_write_their_buffers_only(heads, kv_heads, dim):
    g = torch.Generator().manual_seed(heads)
    lens = [130, 1, 2, 0, 700, 16, 33]
    T = sum(lens)
    q, k, v = (_rand(g, T, h, dim) for h in (heads, kv_heads, kv_heads))
    v[200, 0, 3] = float("inf")
    L = binding.load()
    mem = Arena(2 * T * heads * (dim * 2 + 4) + (48 << 20))
    ws = mem.workspace(L.dspark_attn_prompt_workspace_size(len(lens), T, heads, kv_heads, dim))
    out = dict(out=mem.take((T, heads, dim), BF), lse=mem.take((T, heads), torch.float32))
    binding.attn_prompt(q, k, v, _off(lens), ws=ws, out=out, window=90, sinks=3)
    mem.check()
    s = Scene(lens, heads, kv_heads, dim, 16, F8, seed=3)
    new = [min(n, 5) for n in lens]
    Tq = sum(new)
    ws = mem.workspace(L.dspark_attn_paged_workspace_size(len(lens), Tq, heads, kv_heads, dim))
    out = dict(out=mem.take((Tq, heads, dim), BF), lse=mem.take((Tq, heads), torch.float32))
    binding.attn_paged(q[:Tq], s.cache, _off(new), _i32(lens), s.page_table, ws=ws, out=out, window=90, sinks=3)
    mem.check()
    assert binding.workspace_status(ws) == 0


def test_rows_of_no_request_and_no_sequence_stay():
    s = Scene([340], 4, 2, 64, 16, BF, seed=8)
    q = _rand(s.g, 5, 4, 64)
    out = dict(out=torch.full((5, 4, 64), 7.0, dtype=BF, device=DEV), lse=torch.full((5, 4), 7.0, device=DEV))
    binding.attn_paged(q, s.cache, _i32([1, 3]), _i32([340]), s.page_table, out=out, window=20, sinks=1)
    stay = torch.tensor([True, False, False, True, True], device=DEV)
    assert (out["out"][stay] == 7).all() and (out["lse"][stay] == 7).all()
    g = torch.Generator().manual_seed(8)
    q, k, v = (_rand(g, 20, h, 64) for h in (4, 2, 2))
    out = dict(out=torch.full((20, 4, 64), 7.0, dtype=BF, device=DEV), lse=torch.full((20, 4), 7.0, device=DEV))
    binding.attn_prompt(q, k, v, _i32([3, 9, 15]), out=out, window=2, sinks=1)
    for rows in (slice(0, 3), slice(15, 20)):
        assert (out["out"][rows] == 7).all() and (out["lse"][rows] == 7).all()
