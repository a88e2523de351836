"""A speculative decoding loop with the target's attention over the paged cache.

    python -m speculative_decoding_drafting_gb300.decode_example [--cache e4m3] [--cycles 8]

The target is one attention layer of random weights (tokens attend to what
stands before them; its projections are plain matrix products), the drafter a
Markov head on the anchor token's logits:

* the prompts run through ``attn_prompt``, their keys and values go into the
  cache with ``kv_write`` (slices of the fused projection, not copied);
* each cycle drafts gamma tokens (``draft_markov``), writes the block of the
  anchor and the drafts, attends it over the cache (``attn_paged``) and accepts
  the longest correct prefix (``verify``).  A rejected draft costs nothing to
  take back: the request's length does not count it, and the next block
  overwrites its place;
* at the end ``kv_read`` hands the first request's cache on as bf16.

A cycle never waits for the host.  With temperature 0 the tokens are the ones
that plain decoding would give, which the loop checks: the finished sequences
run through ``attn_prompt`` at once, and each token must be its own argmax but
for the two calls' rounding.
"""
import argparse
from typing import Dict, List

import torch

from . import binding


class Target:
    """One attention layer: logits of token t are out(x_t + o_t), float32."""

    def __init__(self, vocab: int, heads: int, kv_heads: int, dim: int, device, seed: int = 0):
        g = torch.Generator(device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        width = heads * dim

        def weights(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * rows ** -0.5).to(torch.bfloat16)

        self.embed = torch.randn((vocab, width), generator=g, device=device).to(torch.bfloat16)
        self.qkv = weights(width, (heads + 2 * kv_heads) * dim)
        self.out = weights(width, vocab)

    def project(self, tokens):
        """x [T, width], and q, k, v as slices of one projection."""
        x = self.embed[tokens.long()]
        h, hk = self.heads, self.kv_heads
        y = (x @ self.qkv).view(-1, h + 2 * hk, self.dim)
        return x, y[:, :h], y[:, h:h + hk], y[:, h + hk:]

    def logits(self, x, o):
        return (x.float() + o.reshape(x.shape).float()) @ self.out.float()


def _offsets(lengths, device):
    return torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32).to(device)


def decode(prompts: List[List[int]], target: Target, W1, W2, gamma: int = 5, cycles: int = 8, page: int = 16,
           cache_dtype=torch.bfloat16, device="cuda") -> Dict[str, object]:
    """Greedy speculative decoding.  Returns the sequences, the mean accepted
    length, the target's own check of them, the first request's cache and what
    its prompt put there."""
    R = len(prompts)
    lens = [len(p) for p in prompts]
    block = gamma + 1
    pages = -(-(max(lens) + cycles * block) // page)
    cache = binding.KvCache.empty(R * pages, target.kv_heads, page, target.dim, cache_dtype, device)
    # any order of pages will do
    g = torch.Generator().manual_seed(1)
    table = torch.randperm(R * pages, generator=g).to(torch.int32).view(R, pages).to(device)

    # prompts
    tokens = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device=device)
    off = _offsets(lens, device)
    cached = torch.tensor(lens, dtype=torch.int32, device=device)      # tokens that count
    x, q, k, v = target.project(tokens)
    prompt_k, prompt_v = k[:lens[0]], v[:lens[0]]
    o = binding.attn_prompt(q, k, v, off)
    kv_ws = binding.kv_write(cache, k, v, off, cached, table)
    last = (off[1:] - 1).long()
    anchor = target.logits(x[last], o["out"][last]).argmax(-1).to(torch.int32)

    # cycles
    block_off = torch.arange(0, (R + 1) * block, block, dtype=torch.int32, device=device)
    first, emitted, counts = anchor, [], []
    ws: Dict[str, object] = dict(draft=None, attn=None, verify=None)
    for step in range(cycles):
        base = target.embed[anchor.long()].float() @ target.out.float()
        U = base[:, None].expand(-1, gamma, -1).contiguous()
        d = binding.draft_markov(U, anchor, W1, W2, 0.0, step, ws=ws["draft"])
        ws["draft"] = d["ws"]
        x, q, k, v = target.project(torch.cat([anchor[:, None], d["tokens"]], 1).reshape(-1))
        kv_len = cached + block
        kv_ws = binding.kv_write(cache, k, v, block_off, kv_len, table, ws=kv_ws)
        o = binding.attn_paged(q, cache, block_off, kv_len, table, ws=ws["attn"])
        ws["attn"] = o["ws"]
        P = target.logits(x, o["out"]).view(R, block, -1)
        r = binding.verify(P, U, W2, d, 0.0, step, ws=ws["verify"])
        ws["verify"] = r["ws"]
        emitted.append(r["out_tokens"])
        counts.append(r["n_out"])
        cached = cached + r["n_out"]                                   # the anchor and the accepted drafts
        anchor = r["out_tokens"].gather(1, (r["n_out"] - 1).long()[:, None])[:, 0]

    # results
    n = torch.stack(counts).cpu()
    out = torch.stack(emitted).cpu()
    start = first.cpu()
    for w in (kv_ws, *ws.values()):
        status = binding.workspace_status(w)
        if status:
            raise binding.DsparkError("decode", status)
    sequences = [list(p) + [int(start[i])] + [int(t) for s in range(cycles) for t in out[s, i, :n[s, i]]]
                 for i, p in enumerate(prompts)]

    # every sequence at once: how far below its row's best each chosen token is
    tokens = torch.tensor([t for s in sequences for t in s[:-1]], dtype=torch.int32, device=device)
    off = _offsets([len(s) - 1 for s in sequences], device)
    x, q, k, v = target.project(tokens)
    o = binding.attn_prompt(q, k, v, off)
    logits = target.logits(x, o["out"])
    chosen = torch.tensor([t for s in sequences for t in s[1:]], device=device)
    gap = (logits.amax(-1) - logits.gather(1, chosen[:, None])[:, 0])
    new = torch.cat([torch.arange(len(s) - 1) >= len(p) - 1 for s, p in zip(sequences, prompts)]).to(device)

    held = int(cached[0])
    handed = binding.kv_read(cache, _offsets([held], device), table[:1], held)
    return dict(sequences=sequences, accepted=float(n.float().mean()) - 1.0, gap=gap[new], K=handed["K"], V=handed["V"],
                prompt_K=prompt_k, prompt_V=prompt_v, values=v)


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="bf16")
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--cycles", type=int, default=8)
    ap.add_argument("--gamma", type=int, default=5)
    a = ap.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    vocab, rank = 2048, 64
    g = torch.Generator().manual_seed(0)
    prompts = [torch.randint(0, vocab, (int(n),), generator=g).tolist()
               for n in torch.randint(1, 400, (a.requests,), generator=g)]
    target = Target(vocab, 8, 2, 128, dev)
    W1 = (torch.randn((vocab, rank), generator=g) * 0.02).to(torch.bfloat16).to(dev)
    W2 = (torch.randn((rank, vocab), generator=g) * 0.02).to(torch.bfloat16).to(dev)
    r = decode(prompts, target, W1, W2, a.gamma, a.cycles,
               cache_dtype=torch.bfloat16 if a.cache == "bf16" else torch.float8_e4m3fn, device=dev)
    new = sum(len(s) - len(p) for s, p in zip(r["sequences"], prompts))
    print(f"{a.requests} requests, {a.cycles} cycles: {new} tokens, {r['accepted']:.2f} drafts accepted per cycle, "
          f"chosen tokens at most {float(r['gap'].max()):.4f} below their row's best logit")


if __name__ == "__main__":
    main()
