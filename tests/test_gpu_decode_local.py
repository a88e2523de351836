"""The decoding loop with head norms, rotary positions and a window: every step's
queries, cached keys and attention against 64-bit forms."""
import pytest
import torch

from speculative_decoding_drafting_gb300 import binding, decode_example
from _rope import close, turned
from _window import attend_masked, visible
from test_gpu_attention import _close
from test_gpu_decode_steps import _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,dim,page,window,sinks", [
    (torch.bfloat16, 64, 16, 40, 4), (torch.bfloat16, 128, 32, 17, 0), (torch.float8_e4m3fn, 128, 16, 64, 3),
    (torch.float8_e4m3fn, 64, 64, 1, 1), (torch.bfloat16, 128, 16, None, 0)])
def test_each_step_of_a_local_layer(monkeypatch, dtype, dim, page, window, sinks):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    dev = torch.device("cuda", 0)
    vocab, rank, gamma, cycles, heads, hk = 512, 64, 5, 4, 4, 2
    g = torch.Generator().manual_seed(dim + page)
    prompts = [torch.randint(0, vocab, (n,), generator=g).tolist() for n in (231, 1, 2, 15, 16, 17, 64)]
    W1 = (torch.randn((vocab, rank), generator=g) * 0.02).to(torch.bfloat16).to(dev)
    W2 = (torch.randn((rank, vocab), generator=g) * 0.02).to(torch.bfloat16).to(dev)
    target = decode_example.Target(vocab, heads, hk, dim, dev, rotary=True, window=window, sinks=sinks)
    freq = [10000.0 ** (-2.0 * i / dim) for i in range(dim // 2)]
    write, attn = binding.rope_write, binding.attn_paged
    seen = dict(window=window or 10 ** 6, sinks=sinks)
    calls = dict(write=0, attn=0)

    def checked_write(cache, q, K, V, q_off, kv_len, table, **kw):
        r = write(cache, q, K, V, q_off, kv_len, table, **kw)
        off, n = q_off.tolist(), kv_len.tolist()
        pos = torch.cat([torch.arange(m - (b - a), m) for a, b, m in zip(off, off[1:], n)])[:, None]
        want, early = turned(q, pos, freq, w=target.norm.q, eps=target.norm.eps)
        close(r["q"], want, early, "queries")
        want, early = turned(K, pos, freq, w=target.norm.k, eps=target.norm.eps)
        if kw.get("keep"):
            close(r["k"], want, early, "kept keys")
        for i, m in enumerate(n):
            k, v = _rows(cache, table[i][:-(-m // page)].long(), m)
            a, b = off[i], off[i + 1]
            # e4m3: half a step, 2^-4, of values down to 2^-6 of 448th parts of the row's largest
            low = want[a:b].abs().amax(-1, keepdim=True) / 448 * 2.0 ** -10
            if dtype == torch.bfloat16:
                close(k[m - (b - a):], want[a:b], early[a:b], "cached keys")
                assert torch.equal(v[m - (b - a):], V[a:b].double())
            else:
                close(k[m - (b - a):], want[a:b], early[a:b] * 2 + low * 1.01 + want[a:b].abs() * 2.0 ** -20, "cached keys", 2.0 ** -4)
        calls["write"] += 1
        return r

    def checked_attn(q, cache, q_off, kv_len, table, **kw):
        assert kw.get("window") == window and kw.get("sinks", 0) == sinks
        r = attn(q, cache, q_off, kv_len, table, **kw)
        off, n = q_off.tolist(), kv_len.tolist()
        for i, m in enumerate(n):
            k, v = _rows(cache, table[i][:-(-m // page)].long(), m)
            a, b = off[i], off[i + 1]
            mask = visible(torch.arange(m - (b - a), m, device=dev), m, **seen)
            want, _, bo, _ = attend_masked(q[a:b], k, v, mask, dim ** -0.5)
            _close(r["out"][a:b], want, bo, f"step {calls['attn']}, request {i}")
        calls["attn"] += 1
        return r

    monkeypatch.setattr(binding, "rope_write", checked_write)
    monkeypatch.setattr(binding, "attn_paged", checked_attn)
    r = decode_example.decode(prompts, target, W1, W2, gamma=gamma, cycles=cycles, page=page, cache_dtype=dtype, device=dev)
    assert calls == dict(write=1 + cycles, attn=cycles)
    assert all(len(s) - len(p) >= 1 + cycles for s, p in zip(r["sequences"], prompts))
    assert torch.isfinite(r["gap"]).all()
    if dtype == torch.bfloat16:
        assert float((r["gap"] == 0).double().mean()) > 0.9
        assert torch.equal(r["K"][:231], r["prompt_K"]) and torch.equal(r["V"][:231], r["prompt_V"])


def test_the_command_runs(capsys):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    decode_example.main(["--requests", "3", "--cycles", "2", "--rotary", "--window", "50", "--sinks", "2"])
    assert "drafts accepted" in capsys.readouterr().out
