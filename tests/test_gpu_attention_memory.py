"""What the cache and attention calls leave alone: the bytes around every
buffer that they write, with workspaces of exactly the stated size."""
import ctypes

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda:0"
GUARD, FILL = 1 << 16, 0x5A


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


class Arena:
    """Buffers with GUARD bytes of a known pattern around each."""

    def __init__(self, size=1 << 24):
        self.bytes = torch.full((size,), FILL, dtype=torch.uint8, device=DEV)
        self.inside = torch.zeros(size, dtype=torch.bool, device=DEV)
        self.at = GUARD

    def take(self, shape, dtype):
        n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        a, self.at = self.at, (self.at + n + 255) // 256 * 256 + GUARD
        assert self.at <= self.bytes.numel()
        self.inside[a:a + n] = True
        return self.bytes[a:a + n].view(dtype).view(shape)

    def workspace(self, nbytes):
        assert nbytes >= 256
        ws = self.take((nbytes,), torch.uint8)
        ws[:256] = 0
        return ws

    def check(self):
        torch.cuda.synchronize()
        bad = ((self.bytes != FILL) & ~self.inside).nonzero()
        assert bad.numel() == 0, f"{bad.numel()} bytes outside the buffers changed, from {bad[0].item()} on"


def _off(lengths):
    return torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32).to(DEV)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _rand(g, *shape):
    return torch.randn(shape, generator=g).to(BF).to(DEV)


@pytest.mark.parametrize("lens", [[1], [100], [333], [130, 1, 2, 15, 16, 17, 200], [30] * 8, [700, 0, 900], [40] * 90])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 1, 64), (4, 2, 128), (3, 3, 64), (16, 4, 64), (7, 1, 128), (128, 1, 128)])
def test_prompt_writes_its_buffers_only(lens, heads, kv_heads, dim):
    g = torch.Generator().manual_seed(sum(lens) + heads)
    T = sum(lens)
    q, k, v = (_rand(g, T, h, dim) for h in (heads, kv_heads, kv_heads))
    off = _off(lens)
    want = binding.attn_prompt(q, k, v, off, lse=True)
    mem = Arena(T * heads * (dim * 2 + 4) + (1 << 20))
    ws = mem.workspace(binding.load().dspark_attn_prompt_workspace_size(len(lens), T, heads, kv_heads, dim))
    out = dict(out=mem.take((T, heads, dim), BF), lse=mem.take((T, heads), torch.float32))
    for _ in range(2):
        binding.attn_prompt(q, k, v, off, ws=ws, out=out)
        mem.check()
    assert binding.workspace_status(ws) == 0
    assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 1, 64, 16), (4, 2, 128, 64), (9, 3, 128, 16), (4, 4, 64, 256)])
def test_cache_calls_write_their_buffers_only(dtype, heads, kv_heads, dim, page):
    kv, new = [1, 40, 0, 700, 129, 64], [1, 7, 0, 3, 129, 2]
    g = torch.Generator().manual_seed(heads + page)
    counts = [-(-n // page) for n in kv]
    pages, most = sum(counts) + 2, max(counts)
    table = torch.full((len(kv), most), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    for r, c in enumerate(counts):
        table[r, :c] = order[sum(counts[:r]):sum(counts[:r]) + c]
    table = table.to(DEV)
    T, Tq = sum(kv), sum(new)
    L = binding.load()
    mem = Arena(4 * pages * kv_heads * page * dim * 2 + T * kv_heads * dim * 4 + (24 << 20))
    shape = (pages, kv_heads, page, dim)
    cache = binding.KvCache(mem.take(shape, dtype), mem.take(shape, dtype),
                            *((mem.take(shape[:3], torch.float32) for _ in range(2)) if dtype == F8 else ()))
    small = mem.workspace(L.dspark_kv_workspace_size())
    K, V = _rand(g, T, kv_heads, dim), _rand(g, T, kv_heads, dim)
    binding.kv_write(cache, K, V, _off(kv), _i32(kv), table, ws=small)
    mem.check()
    back = dict(K=mem.take((T, kv_heads, dim), BF), V=mem.take((T, kv_heads, dim), BF))
    binding.kv_read(cache, _off(kv), table, T, ws=small, out=back)
    mem.check()
    if dtype == BF:
        assert torch.equal(back["K"], K) and torch.equal(back["V"], V)
    q = _rand(g, Tq, heads, dim)
    want = binding.attn_paged(q, cache, _off(new), _i32(kv), table, lse=True)
    ws = mem.workspace(L.dspark_attn_paged_workspace_size(len(kv), Tq, heads, kv_heads, dim))
    out = dict(out=mem.take((Tq, heads, dim), BF), lse=mem.take((Tq, heads), torch.float32))
    binding.attn_paged(q, cache, _off(new), _i32(kv), table, ws=ws, out=out)
    mem.check()
    assert binding.workspace_status(ws) == 0 and binding.workspace_status(small) == 0
    assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])


def test_rows_that_are_not_device_memory_are_refused():
    """Pinned host memory (which a kernel could read) in the place of each input:
    the same refusal in all the calls that take rows, before anything is enqueued."""
    L = binding.load()
    T, heads, kv_heads, dim = 3, 4, 2, 64
    cache = binding.KvCache.empty(2, kv_heads, 16, dim, BF, DEV)
    b = binding._batch(_i32([0, T]), _i32([T]), _i32([[0, 1]]), T)
    c, b = ctypes.byref(cache._struct()), ctypes.byref(b)
    dev = {n: torch.zeros((T, h, dim), dtype=BF, device=DEV) for n, h in (("q", heads), ("K", kv_heads), ("V", kv_heads), ("out", heads))}
    host = {n: torch.zeros(t.shape, dtype=BF).pin_memory() for n, t in dev.items()}
    ws = binding._workspace(1 << 24, DEV)
    off = _i32([0, T])
    torch.cuda.synchronize()

    def at(name, moved):
        return (host if name == moved else dev)[name].data_ptr()

    calls = {
        "write": (("K", "V"), lambda m: L.dspark_kv_write(c, b, at("K", m), at("V", m), 128, 128, ws.data_ptr(), 256, None)),
        "paged": (("q",), lambda m: L.dspark_attn_paged(at("q", m), 256, c, b, heads, 0.125, at("out", m), None,
                                                              ws.data_ptr(), 1 << 24, None)),
        "prompt": (("q", "K", "V"), lambda m: L.dspark_attn_prompt(
            at("q", m), at("K", m), at("V", m), 256, 128, 128, off.data_ptr(), 1, T, heads, kv_heads, dim, 0.125,
            at("out", m), None, ws.data_ptr(), 1 << 24, None))}
    for name, (arrays, call) in calls.items():
        assert call(None) == 0, name
        for moved in arrays:
            assert call(moved) == -1, (name, moved)
    torch.cuda.synchronize()
