"""Every step of the decoding loop against 64-bit forms: the attention of each
block over what the cache holds, and the tokens that verification emits."""
import pytest
import torch

from speculative_decoding_drafting_gb300 import binding, decode_example
from _attention import attend
from test_gpu_attention import _close

pytestmark = pytest.mark.gpu


def _rows(cache, table, n):
    """The first n tokens of a request, as the cache's values stand for them."""
    def one(x, scale):
        y = x.view(torch.uint8)[table].view(x.dtype).double() if scale is not None else x[table].double()
        if scale is not None:
            y = y * scale[table].double()[..., None]
        return y.transpose(1, 2).reshape(-1, cache.n_kv_heads, cache.head_dim)[:n]
    return one(cache.k, cache.k_scale), one(cache.v, cache.v_scale)


@pytest.mark.parametrize("dtype,dim,page", [(torch.bfloat16, 64, 16), (torch.bfloat16, 128, 32),
                                            (torch.float8_e4m3fn, 128, 16), (torch.float8_e4m3fn, 64, 64)])
def test_each_step_of_the_loop(monkeypatch, dtype, dim, page):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    dev = torch.device("cuda", 0)
    vocab, rank, gamma, cycles = 512, 64, 5, 5
    g = torch.Generator().manual_seed(dim + page)
    prompts = [torch.randint(0, vocab, (n,), generator=g).tolist() for n in (131, 1, 2, 15, 16, 17, 64)]
    W1 = (torch.randn((vocab, rank), generator=g) * 0.02).to(torch.bfloat16).to(dev)
    W2 = (torch.randn((rank, vocab), generator=g) * 0.02).to(torch.bfloat16).to(dev)
    held = torch.tensor([len(p) for p in prompts])           # tokens that count
    emitted = [[] for _ in prompts]
    attn, verify = binding.attn_paged, binding.verify
    steps = []

    def checked_attn(q, cache, q_off, kv_len, table, **kw):
        r = attn(q, cache, q_off, kv_len, table, **kw)
        off, n = q_off.tolist(), kv_len.tolist()
        assert n == (held + gamma + 1).tolist()
        for i in range(len(prompts)):
            k, v = _rows(cache, table[i][:-(-n[i] // page)].long(), n[i])
            a, b = off[i], off[i + 1]
            want, _, bo, _ = attend(q[a:b], k, v, torch.arange(a - b, 0) + n[i] + 1, dim ** -0.5)
            _close(r["out"][a:b], want, bo, f"step {len(steps)}, request {i}")
        return r

    def checked_verify(P, U, W, draft, *args, **kw):
        r = verify(P, U, W, draft, *args, **kw)
        best, out, n_out = P.amax(-1), r["out_tokens"].long(), r["n_out"].tolist()
        for i, n in enumerate(n_out):
            tokens = out[i, :n]
            # each token is its row's best, all but the last are the drafts, and
            # the draft in the last one's place is not the best
            assert torch.equal(P[i, torch.arange(n), tokens], best[i, :n])
            assert torch.equal(tokens[:-1], draft["tokens"][i, :n - 1].long())
            assert n == gamma + 1 or draft["tokens"][i, n - 1] != tokens[-1]
            emitted[i].extend(tokens.tolist())
        held.add_(torch.tensor(n_out))
        steps.append(n_out)
        return r

    monkeypatch.setattr(binding, "attn_paged", checked_attn)
    monkeypatch.setattr(binding, "verify", checked_verify)
    target = decode_example.Target(vocab, 4, 2, dim, dev)
    r = decode_example.decode(prompts, target, W1, W2, gamma=gamma, cycles=cycles, page=page, cache_dtype=dtype, device=dev)
    assert len(steps) == cycles and max(max(s) for s in steps) > 1
    for i, p in enumerate(prompts):
        assert r["sequences"][i][:len(p)] == p and r["sequences"][i][len(p) + 1:] == emitted[i]
