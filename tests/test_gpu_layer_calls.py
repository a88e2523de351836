"""The calls around a layer's attention in the ways that a server makes them: on two
streams at once, captured together, on the same workspace one after another, with
batches and sizes at the ends of their ranges."""
import math

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from _window import attend_masked, visible
from test_gpu_attention import Scene, _close, _i32, _off, _rand

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def _layer(g, cache, fused, heads, hk, off, kv_len, table, rope, ws, out, window, sinks, stream=None):
    q, K, V = fused[:, :heads], fused[:, heads:heads + hk], fused[:, heads + hk:]
    binding.rope_write(cache, q, K, V, off, kv_len, table, rope=rope, ws=ws[0], out=out["rows"], stream=stream)
    binding.attn_paged(out["rows"]["q"], cache, off, kv_len, table, ws=ws[1], out=out["attn"], window=window, sinks=sinks,
                       stream=stream)


def _buffers(T, heads, dim, R, hk):
    L = binding.load()
    return dict(rows=dict(q=torch.zeros((T, heads, dim), dtype=BF, device=DEV)),
                attn=dict(out=torch.zeros((T, heads, dim), dtype=BF, device=DEV), lse=torch.zeros((T, heads), device=DEV))), \
        (binding._workspace(256, DEV), binding._workspace(L.dspark_attn_paged_workspace_size(R, T, heads, hk, dim), DEV))


@pytest.mark.parametrize("dtype", [BF, F8])
def test_two_layers_on_two_streams_and_in_one_graph(dtype):
    """Two layers' calls at once on streams of their own, and captured as one chain
    replayed at growing lengths, give what each gives alone."""
    g = torch.Generator().manual_seed(1)
    heads, hk, dim, page, R = 8, 2, 128, 16, 5
    new, kv = [6, 1, 3, 6, 2], [700, 33, 3, 1200, 64]
    off, T = _off(new), sum(new)
    rope = binding.Rope.from_theta(dim)
    counts = [-(-(n + 40) // page) for n in kv]
    table = torch.arange(sum(counts), dtype=torch.int32)
    full = torch.full((R, max(counts)), -1, dtype=torch.int32)
    for r, c in enumerate(counts):
        full[r, :c] = table[sum(counts[:r]):sum(counts[:r]) + c]
    full = full.to(DEV)
    fused = [_rand(g, T, heads + 2 * hk, dim) for _ in range(2)]
    windows = ((100, 4), (300, 0))

    def caches():
        out = []
        for i in range(2):
            gen = torch.Generator(DEV).manual_seed(i)
            shape = (sum(counts), hk, page, dim)
            k, v = (torch.randn(shape, generator=gen, device=DEV).to(BF) for _ in range(2))
            if dtype == F8:
                out.append(binding.KvCache(k.to(F8), v.to(F8), *(torch.ones(shape[:3], device=DEV) for _ in range(2))))
            else:
                out.append(binding.KvCache(k, v))
        return out

    def run(lens, streams=None):
        cs = caches()
        kv_len = _i32(lens)
        res = []
        for i in range(2):
            out, ws = _buffers(T, heads, dim, R, hk)
            res.append((out, ws))
        torch.cuda.synchronize()
        for i in range(2):
            _layer(g, cs[i], fused[i], heads, hk, off, kv_len, full, rope, res[i][1], res[i][0], *windows[i],
                   stream=None if streams is None else streams[i])
        torch.cuda.synchronize()
        assert all(binding.workspace_status(w) == 0 for _, ws in res for w in ws)
        return [o["attn"] for o, _ in res]

    alone = run(kv)
    both = run(kv, [torch.cuda.Stream(), torch.cuda.Stream()])
    for a, b in zip(alone, both):
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    # one graph of both layers, on one pair of workspaces
    cs = caches()
    kv_len = _i32(kv)
    bufs = [_buffers(T, heads, dim, R, hk) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(2):
            _layer(g, cs[i], fused[i], heads, hk, off, kv_len, full, rope, bufs[0][1], bufs[i][0], *windows[i])
    for step in range(3):
        lens = [n + step * 6 for n in kv]
        kv_len.copy_(torch.tensor(lens))
        graph.replay()
    torch.cuda.synchronize()
    assert all(binding.workspace_status(w) == 0 for w in bufs[0][1])
    # the same three steps, call by call
    cs = caches()
    for step in range(3):
        kv_len = _i32([n + step * 6 for n in kv])
        for i in range(2):
            out, ws = _buffers(T, heads, dim, R, hk)
            _layer(g, cs[i], fused[i], heads, hk, off, kv_len, full, rope, ws, out, *windows[i])
            if step == 2:
                assert torch.equal(out["attn"]["out"], bufs[i][0]["attn"]["out"])
                assert torch.equal(out["attn"]["lse"], bufs[i][0]["attn"]["lse"])


@pytest.mark.parametrize("dtype", [BF, F8])
def test_shared_pages_and_repeated_requests(dtype):
    """Two requests whose tables name the same pages (a shared prefix) read them alike."""
    s = Scene([500, 260], 8, 2, 128, 16, dtype, seed=3)
    table = s.page_table.clone()
    table[1] = -1
    table[1, :17] = table[0, :17]                    # request 1's first 260 tokens are request 0's
    q = _rand(s.g, 2, 8, 128)
    q[1] = q[0]
    r = binding.attn_paged(q, s.cache, _i32([0, 1, 2]), _i32([260, 260]), table, lse=True, window=70, sinks=5)
    assert binding.workspace_status(r["ws"]) == 0
    mask = visible(torch.tensor([259]), 260, 70, 5).to(DEV)
    for i in range(2):
        want, lse, bo, bl = attend_masked(q[i:i + 1], s.K[0][:260], s.V[0][:260], mask, 128 ** -0.5)
        _close(r["out"][i:i + 1], want, bo, "out")
        _close(r["lse"][i:i + 1], lse, bl, "lse")


def test_a_long_prompt_of_many_heads():
    """Rows enough for every worker to have several items, checked against the paged
    form on the same data (both bounds together)."""
    g = torch.Generator().manual_seed(5)
    n, heads, hk, dim, window, sinks = 6000, 16, 4, 64, 700, 9
    s = Scene([n], heads, hk, dim, 64, BF, seed=6)
    q = _rand(g, n, heads, dim)
    a = binding.attn_prompt(q, s.K[0], s.V[0], _i32([0, n]), lse=True, window=window, sinks=sinks)
    b = binding.attn_paged(q, s.cache, _i32([0, n]), _i32([n]), s.page_table, lse=True, window=window, sinks=sinks)
    assert binding.workspace_status(a["ws"]) == 0 and binding.workspace_status(b["ws"]) == 0
    for at in range(0, n, 1000):
        rows = slice(at, at + 1000)
        low = max(0, at - window)
        keys = torch.cat([torch.arange(min(sinks, low)), torch.arange(low, min(n, at + 1000))])
        p = torch.arange(at, min(n, at + 1000))
        mask = ((keys[None] <= p[:, None]) & ((p[:, None] - keys[None] < window) | (keys[None] < sinks))).to(DEV)
        want, lse, bo, bl = attend_masked(q[rows], s.K[0][keys.to(DEV)], s.V[0][keys.to(DEV)], mask, dim ** -0.5)
        for r in (a, b):
            _close(r["out"][rows], want, bo, f"out from {at}")
            _close(r["lse"][rows], lse, bl, f"lse from {at}")


@pytest.mark.parametrize("heads,kv_heads", [(3, 1), (12, 4), (5, 5)])
def test_prompts_rerun_to_the_same_bits(heads, kv_heads):
    g = torch.Generator().manual_seed(heads)
    lens = torch.randint(1, 900, (40,), generator=g).tolist()
    q, k, v = (_rand(g, sum(lens), h, 128) for h in (heads, kv_heads, kv_heads))
    for kw in (dict(), dict(window=150, sinks=3)):
        first = binding.attn_prompt(q, k, v, _off(lens), lse=True, **kw)
        ws = first["ws"]
        for _ in range(4):
            r = binding.attn_prompt(q, k, v, _off(lens), lse=True, ws=ws, **kw)
            assert torch.equal(r["out"], first["out"]) and torch.equal(r["lse"], first["lse"])
        assert binding.workspace_status(ws) == 0


def test_outputs_that_begin_off_a_sector():
    """out 16-byte aligned, but not to 32 bytes."""
    g = torch.Generator().manual_seed(9)
    lens = [130, 7, 300]
    T = sum(lens)
    q, k, v = (_rand(g, T, h, 64) for h in (4, 2, 2))
    buf = torch.zeros(T * 4 * 64 + 8, dtype=BF, device=DEV)
    for kw in (dict(), dict(window=60, sinks=2)):
        want = binding.attn_prompt(q, k, v, _off(lens), **kw)
        out = buf[8:].view(T, 4, 64)
        assert out.data_ptr() % 32 == 16
        binding.attn_prompt(q, k, v, _off(lens), out=dict(out=out), **kw)
        assert torch.equal(out, want["out"])
        assert (buf[:8] == 0).all()


def test_scales_of_either_sign_and_none():
    g = torch.Generator().manual_seed(11)
    n = 333
    q, k, v = (_rand(g, n, h, 128) for h in (4, 2, 2))
    for scale in (0.3, -0.3, 0.0, 1e-30, -1e-30):
        mask = visible(torch.arange(n), n, 90, 2).to(DEV)
        r = binding.attn_prompt(q, k, v, _i32([0, n]), scale=scale, lse=True, window=90, sinks=2)
        want, lse, bo, bl = attend_masked(q, k, v, mask, scale)
        _close(r["out"], want, bo, f"out at {scale}")
        _close(r["lse"], lse, bl, f"lse at {scale}")
    # a negated query at the negated scale is the same query
    a = binding.attn_prompt(q, k, v, _i32([0, n]), scale=0.2, lse=True)
    b = binding.attn_prompt(-q, k, v, _i32([0, n]), scale=-0.2, lse=True)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
