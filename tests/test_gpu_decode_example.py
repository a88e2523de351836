"""The decoding loop: its tokens are the target's own, its cache holds their keys and values."""
import pytest
import torch

from speculative_decoding_drafting_gb300 import binding
from speculative_decoding_drafting_gb300.decode_example import Target, decode
from _attention import quantise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,dim,page", [(torch.bfloat16, 64, 16), (torch.bfloat16, 128, 32),
                                            (torch.float8_e4m3fn, 128, 16)])
def test_decoding_with_the_cache_gives_the_targets_own_tokens(dtype, dim, page):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    dev = torch.device("cuda", 0)
    vocab, rank = 512, 64
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, vocab, (n,), generator=g).tolist() for n in (130, 1, 2, 15, 16, 17, 200)]
    W1 = (torch.randn((vocab, rank), generator=g) * 0.02).to(torch.bfloat16).to(dev)
    W2 = (torch.randn((rank, vocab), generator=g) * 0.02).to(torch.bfloat16).to(dev)
    target = Target(vocab, 4, 2, dim, dev)
    r = decode(prompts, target, W1, W2, gamma=5, cycles=6, page=page, cache_dtype=dtype, device=dev)
    assert all(len(s) - len(p) >= 1 + 6 for s, p in zip(r["sequences"], prompts))
    assert r["accepted"] > 0
    # bf16 cache: an output is within 2^-8 |o| + 2.1 2^-8 max |v| of the exact one
    # (rounded output, rounded weights), in both calls; a logit sums the
    # differences over a column of the output weights, and a token's gap takes
    # two logits.  e4m3: K and V themselves are off by 2^-4 of each value, which
    # changes what plain decoding is; the outputs stay finite and the cache right.
    if dtype == torch.bfloat16:
        step = 2 * 3.1 * 2.0 ** -8 * float(r["values"].abs().max())
        assert float(r["gap"].max()) <= 2 * step * float(target.out.float().abs().sum(0).max())
        assert float((r["gap"] == 0).double().mean()) > 0.9
        assert torch.equal(r["K"][:130], r["prompt_K"]) and torch.equal(r["V"][:130], r["prompt_V"])
    else:
        assert torch.isfinite(r["gap"]).all()
        for name in ("K", "V"):
            code, scale = quantise(r["prompt_" + name])
            assert torch.equal(r[name][:130].double(), (code * scale.float().double()[..., None]).float().to(torch.bfloat16).double())
