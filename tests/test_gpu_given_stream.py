"""Calls given a stream while the current one is still busy: what a call allocates
and clears for itself belongs to its own stream."""
import types

import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from test_gpu_attention import _i32, _rand

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
DEV = "cuda:0"
T, HEADS, HK, DIM = 40, 4, 2, 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def _busy():
    torch.cuda._sleep(100_000_000)                     # about 50 ms of the current stream


def _calls():
    """Calls that make their outputs and workspaces: name, function(stream, table)."""
    g = torch.Generator().manual_seed(3)
    q, k, v = (_rand(g, T, h, DIM) for h in (HEADS, HK, HK))
    k_, v_ = (torch.randn((4, HK, 16, DIM), generator=g).to(BF).to(DEV) for _ in range(2))
    off, kv_len, pos = _i32([0, T]), _i32([T]), _i32(list(range(T)))
    rope = binding.Rope.from_theta(DIM)

    def cache():
        return binding.KvCache(k_, v_)

    return dict(
        qk_rope=lambda s, t: binding.qk_rope(q, k, pos, rope, stream=s),
        rope_write=lambda s, t: binding.rope_write(cache(), q, k, v, off, kv_len, t, rope, keep=True, stream=s),
        attn_paged=lambda s, t: binding.attn_paged(q, cache(), off, kv_len, t, lse=True, stream=s),
        attn_local=lambda s, t: binding.attn_paged(q, cache(), off, kv_len, t, lse=True, stream=s, window=20, sinks=2),
        attn_prompt=lambda s, t: binding.attn_prompt(q, k, v, off, lse=True, stream=s),
        prompt_local=lambda s, t: binding.attn_prompt(q, k, v, off, lse=True, stream=s, window=20, sinks=2),
        kv_read=lambda s, t: binding.kv_read(cache(), off, t, T, stream=s))


@pytest.mark.parametrize("name", ["qk_rope", "rope_write", "attn_paged", "attn_local", "attn_prompt", "prompt_local", "kv_read"])
def test_outputs_are_not_the_memory_of_pending_work(name):
    call = _calls()[name]
    table = _i32([[2, 0, 3]])
    want = call(None, table)                           # its outputs' sizes
    torch.cuda.synchronize()
    keep = {n: t.clone() for n, t in want.items() if n != "ws"}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy()
    # freed with work on it still queued: the current stream may use it again at once, no other
    for t in want.values():
        t.fill_(1)
    del want, t
    got = call(side, table)
    torch.cuda.synchronize()
    for n, t in keep.items():
        assert torch.equal(got[n].view(torch.uint8), t.view(torch.uint8)), n
    if "ws" in got:
        assert binding.workspace_status(got["ws"]) == 0


@pytest.mark.parametrize("name", ["rope_write", "attn_paged", "attn_local", "kv_read"])
@pytest.mark.parametrize("wrapped", [False, True])
def test_a_status_is_not_cleared_by_the_busy_stream(name, wrapped):
    """A page outside the cache is recorded, and stays so."""
    call = _calls()[name]
    table = _i32([[2, 7, 3]])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy()
    # (the handle is all that a call needs of a stream)
    r = call(types.SimpleNamespace(cuda_stream=side.cuda_stream) if wrapped else side, table)
    torch.cuda.synchronize()
    assert binding.workspace_status(r["ws"]) == -9


@pytest.mark.parametrize("name", ["qk_rope", "rope_write", "attn_paged", "attn_local", "attn_prompt", "prompt_local", "kv_read"])
def test_captured_on_a_stream_beside_the_capturing_one(name):
    """A call on a forked stream makes its buffers in the graph's pool; replays agree."""
    call = _calls()[name]
    table = _i32([[2, 0, 3]])
    want = call(None, table)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side, table)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for n, t in got.items():
            if n != "ws":
                t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for n, t in want.items():
            if n != "ws":
                assert torch.equal(got[n].view(torch.uint8), t.view(torch.uint8)), n
