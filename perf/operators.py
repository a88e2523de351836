"""The serving operators around one speculative-decoding cycle, as measured cases.

Four calls that share one paged key-value cache:

* ``write``  -- the new tokens' keys and values go into the cache's pages, as
  bf16 or quantised to e4m3 with one float32 scale per (token, head);
* ``read``   -- a request's tokens come back out of the pages, as bf16;
* ``paged``  -- attention of each request's newest tokens (one at plain
  decoding, up to gamma + 1 at verification) over its cached tokens;
* ``prompt`` -- causal attention over whole prompts, packed one after another.

``run`` computes a case in plain torch operations (``own`` false) or through
the library's entry points (``own`` true).
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user, one new token, a short chat: latency is all there is
        dict(name="paged-one", op="paged", R=1, q_max=1, ragged=False, kv_min=777, kv_max=777, heads=32, kv_heads=8,
             dim=128, page=16, cache="bf16"),
        # plain decoding of a middling batch over a quantised cache
        dict(name="paged-decode-e4m3", op="paged", R=64, q_max=1, ragged=False, kv_min=500, kv_max=8000, heads=64,
             kv_heads=8, dim=128, page=64, cache="e4m3"),
        # the headline cycle's verification: 256 requests, blocks of up to 5 drafts and the token before them
        dict(name="paged-verify", op="paged", R=256, q_max=6, ragged=True, kv_min=200, kv_max=4000, heads=32,
             kv_heads=8, dim=128, page=16, cache="bf16"),
        # verification of 16-token blocks with scheduled lengths, narrow heads, a group that is no power of two
        dict(name="paged-longblock", op="paged", R=64, q_max=17, ragged=True, kv_min=1000, kv_max=6001, heads=48,
             kv_heads=8, dim=64, page=32, cache="bf16"),
        # two requests with very long contexts: the work has to be split over the cache's length
        dict(name="paged-long-e4m3", op="paged", R=2, q_max=6, ragged=False, kv_min=150001, kv_max=260001, heads=32,
             kv_heads=4, dim=128, page=128, cache="e4m3"),
        # a few short questions arriving together
        dict(name="prompt-short", op="prompt", B=8, len_min=1, len_max=61, heads=16, kv_heads=4, dim=64),
        # a prefill batch of mixed lengths
        dict(name="prompt-packed", op="prompt", B=16, len_min=100, len_max=4000, heads=32, kv_heads=8, dim=128),
        # one long document
        dict(name="prompt-long", op="prompt", B=1, len_min=12001, len_max=12001, heads=32, kv_heads=8, dim=128),
        # the verification blocks' keys and values of one layer
        dict(name="write-step", op="write", R=256, q_max=6, ragged=True, kv_min=200, kv_max=700, kv_heads=8, dim=128,
             page=16, cache="bf16"),
        # whole prompts into a quantised cache
        dict(name="write-prompt-e4m3", op="write", R=30, q_max=0, ragged=False, kv_min=100, kv_max=2600, kv_heads=8,
             dim=128, page=64, cache="e4m3"),
        # a prefix of moderate size handed on in bf16
        dict(name="read-bf16", op="read", R=7, kv_min=1, kv_max=900, kv_heads=8, dim=64, page=16, cache="bf16"),
        # many requests' quantised caches unpacked, for a move to another layout
        dict(name="read-e4m3", op="read", R=40, kv_min=100, kv_max=6000, kv_heads=8, dim=128, page=64, cache="e4m3"),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["paged", "paged", "paged", "prompt", "prompt", "write", "read"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 6, 8, 8])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "paged":
        R = _between(rng, 1, 256)
        q_max = rng.choice([1, 1, 2, 5, 6, 9, 17])
        # no more cached values than the listed verification batch has
        longest = min(260000, 256 * 4000 // R * 8 // kv_heads, 256 * 4000 * 6 // (R * q_max))
        kv_max = _between(rng, 2 * q_max, longest)
        kv_min = rng.randint(q_max, kv_max) if rng.random() < 0.5 else min(kv_max, q_max + rng.randint(0, 40))
        return dict(op=op, R=R, q_max=q_max, ragged=q_max > 1 and rng.random() < 0.7, kv_min=kv_min, kv_max=kv_max,
                    heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, cache=cache)
    if op == "prompt":
        B = _between(rng, 1, 64)
        # tokens^2 x heads bounded by the listed long document's
        kv_heads = min(kv_heads, 32 // group) or 1
        longest = int(12001 * math.sqrt(min(1.0, 32.0 / (kv_heads * group)) / B))
        len_max = _between(rng, 1, longest)
        len_min = rng.randint(1, len_max)
        return dict(op=op, B=B, len_min=len_min, len_max=len_max, heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
    if op == "write":
        R = _between(rng, 1, 256)
        kv_max = _between(rng, 8, 78000 // R)
        q_max = rng.choice([0, 1, 6])
        return dict(op=op, R=R, q_max=q_max, ragged=q_max > 1, kv_min=rng.randint(max(1, q_max), kv_max), kv_max=kv_max,
                    kv_heads=kv_heads, dim=dim, page=page, cache=cache)
    R = _between(rng, 1, 64)
    kv_max = _between(rng, 1, 240000 // R)
    return dict(op=op, R=R, kv_min=rng.randint(1, kv_max), kv_max=kv_max, kv_heads=kv_heads, dim=dim, page=page,
                cache=cache)


def _lengths(case, seed):
    """(kv_len, q_len) of a case as Python lists, the same for prepare() and work() at any seed of the same case."""
    g = torch.Generator().manual_seed(int(seed))
    if case["op"] == "prompt":
        n = torch.randint(case["len_min"], case["len_max"] + 1, (case["B"],), generator=g)
        n[0] = case["len_max"]
        return n.tolist(), n.tolist()
    n = torch.randint(case["kv_min"], case["kv_max"] + 1, (case["R"],), generator=g)
    n[0] = case["kv_max"]
    if case["op"] == "read":
        return n.tolist(), n.tolist()
    if case["q_max"] == 0:                 # whole prompts: every cached token is new
        return n.tolist(), n.tolist()
    q = torch.full((case["R"],), case["q_max"], dtype=torch.int64)
    if case["ragged"]:
        q = torch.randint(1, case["q_max"] + 1, (case["R"],), generator=g)
        q[-1] = case["q_max"]
    return n.tolist(), torch.minimum(q, n).tolist()


# lengths are the case's, not the seed's: passes on other inputs cost the same
_LENGTH_SEED = 20


def work(case):
    kv, q = _lengths(case, _LENGTH_SEED)
    d = case["dim"]
    hk = case["kv_heads"]
    stored = 2 * d if case.get("cache") == "bf16" else d + 4      # bytes of one cached (token, head) row
    if case["op"] == "write":
        n = sum(q) * hk * 2
        return {"bytes": n * (2 * d + stored), "flops": 0 if case["cache"] == "bf16" else 3 * n * d}
    if case["op"] == "read":
        n = sum(kv) * hk * 2
        return {"bytes": n * (2 * d + stored), "flops": 0 if case["cache"] == "bf16" else n * d}
    h = case["heads"]
    if case["op"] == "prompt":
        pairs = sum(n * (n + 1) // 2 for n in kv)
        return {"bytes": sum(kv) * (2 * h + 2 * hk) * d * 2, "flops": 4 * pairs * h * d}
    pairs = sum(m * n - m * (m - 1) // 2 for n, m in zip(kv, q))
    return {"bytes": sum(kv) * hk * 2 * stored + sum(q) * h * d * 4, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1000 + int(seed))


def _rows(g, n, heads, dim, spread):
    """[n, heads, dim] bf16 rows; with `spread`, a few channels of each head run larger, as keys' do."""
    x = torch.randn((n, heads, dim), generator=g, device="cuda")
    if spread:
        loud = torch.rand((heads, dim), generator=g, device="cuda") < 0.04
        x = x * (1.0 + 3.0 * loud)
    return x.to(torch.bfloat16)


def _quantise(x):
    """e4m3 codes and float32 scales of bf16 rows (the last axis), for a cache that is already there."""
    big = x.float().abs().amax(-1)
    return (x.float() * E4M3_MAX / big.clamp_min(1e-30)[..., None]).to(torch.float8_e4m3fn), big / E4M3_MAX


def _offsets(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)


def prepare(case, seed):
    kv, q = _lengths(case, _LENGTH_SEED)
    g = _generator(seed)
    hk, d = case["kv_heads"], case["dim"]
    st = dict(case=case, scale=1.0 / math.sqrt(d))
    if case["op"] == "prompt":
        n = sum(kv)
        st["q"] = _rows(g, n, case["heads"], d, False) * 1.5
        st["k"] = _rows(g, n, hk, d, True)
        st["v"] = _rows(g, n, hk, d, False)
        st["seq_off"] = _offsets(kv)
        st["longest"] = max(kv)
        return st
    page = case["page"]
    R = case["R"]
    counts = [-(-n // page) for n in kv]
    pages = sum(counts) + 3
    # pages scattered over the cache, as they are after a while of serving; unused table entries are -1
    order = torch.randperm(pages, generator=g, device="cuda")[:sum(counts)].to(torch.int32)
    most = max(counts)
    table = torch.full((R, most), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(most, device="cuda")[None, :] < torch.tensor(counts, device="cuda")[:, None]
    table[used] = order
    st["page_table"] = table
    st["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    st["q_off"] = _offsets(q)
    st["kv_off"] = _offsets(kv)
    st["tokens"] = sum(q)
    st["kv_tokens"] = sum(kv)
    st["q_longest"] = max(q)
    st["k_scale"] = st["v_scale"] = None
    if case["op"] == "write":
        st["K"] = _rows(g, sum(q), hk, d, True)
        st["V"] = _rows(g, sum(q), hk, d, False)
        dtype = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
        st["k"] = torch.zeros((pages, hk, page, d), device="cuda").to(dtype)
        st["v"] = torch.zeros((pages, hk, page, d), device="cuda").to(dtype)
        if case["cache"] == "e4m3":
            st["k_scale"] = torch.zeros((pages, hk, page), device="cuda")
            st["v_scale"] = torch.zeros((pages, hk, page), device="cuda")
        return st
    st["k"] = _rows(g, pages * page, hk, d, True).view(pages, page, hk, d).transpose(1, 2).contiguous()
    st["v"] = _rows(g, pages * page, hk, d, False).view(pages, page, hk, d).transpose(1, 2).contiguous()
    if case["cache"] == "e4m3":
        st["k"], st["k_scale"] = _quantise(st["k"])
        st["v"], st["v_scale"] = _quantise(st["v"])
    if case["op"] == "paged":
        st["q"] = _rows(g, sum(q), case["heads"], d, False) * 1.5
    return st


# ------------------------------------------------------------------ plain forms
def _token_places(off, n):
    """For n packed tokens: the request each belongs to and its place in it."""
    t = torch.arange(n, device="cuda")
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    return r, t - off[r]


def _plain_write(st):
    case = st["case"]
    page = case["page"]
    q_off, kv_len = st["q_off"].long(), st["kv_len"].long()
    r, i = _token_places(q_off, st["tokens"])
    pos = kv_len[r] - (q_off[r + 1] - q_off[r]) + i
    at = st["page_table"][r, pos // page].long()
    slot = pos % page
    if case["cache"] == "bf16":
        st["k"][at, :, slot] = st["K"]
        st["v"][at, :, slot] = st["V"]
        return dict(k=st["k"], v=st["v"])
    x = torch.stack([st["K"], st["V"]]).float()
    big = x.abs().amax(-1, keepdim=True)
    codes = torch.where(big > 0, x * E4M3_MAX / big.clamp_min(1e-38), torch.zeros_like(x)).to(torch.float8_e4m3fn)
    scale = (big / E4M3_MAX)[..., 0]
    # index_put on the bytes: torch has none for 8-bit floats
    st["k"].view(torch.uint8)[at, :, slot] = codes[0].view(torch.uint8)
    st["v"].view(torch.uint8)[at, :, slot] = codes[1].view(torch.uint8)
    st["k_scale"][at, :, slot] = scale[0]
    st["v_scale"][at, :, slot] = scale[1]
    return dict(k=st["k"], v=st["v"], k_scale=st["k_scale"], v_scale=st["v_scale"])


def _plain_read(st):
    page = st["case"]["page"]
    r, pos = _token_places(st["kv_off"].long(), st["kv_tokens"])
    at, slot = st["page_table"][r, pos // page].long(), pos % page
    if st["k_scale"] is None:
        return dict(K=st["k"][at, :, slot], V=st["v"][at, :, slot])
    K = st["k"].view(torch.uint8)[at, :, slot].view(torch.float8_e4m3fn).float() * st["k_scale"][at, :, slot][..., None]
    V = st["v"].view(torch.uint8)[at, :, slot].view(torch.float8_e4m3fn).float() * st["v_scale"][at, :, slot][..., None]
    return dict(K=K.to(torch.bfloat16), V=V.to(torch.bfloat16))


def _softmax_product(s, v):
    """softmax(s) v and the log-sum-exp of s's rows; a row of -inf alone gives 0 and -inf.  s is used up."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    s = s.sub_(m).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (m + torch.log(total))[..., 0]


def _plain_paged(st):
    case = st["case"]
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    group = case["heads"] // hk
    R, Q = case["R"], st["q_longest"]
    table = st["page_table"].long().clamp_min(0)
    L = table.shape[1] * page

    def cached(x, scale):
        y = x.view(torch.uint8)[table].view(x.dtype) if scale is not None else x[table]
        y = y.float()
        if scale is not None:
            y = y * scale[table][..., None]
        return y.transpose(1, 2).reshape(R, hk, L, d)

    q_off, kv_len = st["q_off"].long(), st["kv_len"].long()
    q_len = q_off[1:] - q_off[:-1]
    i = torch.arange(Q, device="cuda")
    rows = st["q"][(q_off[:-1, None] + i).clamp_max(st["tokens"] - 1)].float()          # [R, Q, heads, d]
    rows = rows.view(R, Q, hk, group, d).permute(0, 2, 1, 3, 4).reshape(R, hk, Q * group, d)
    s = torch.matmul(rows, cached(st["k"], st["k_scale"]).transpose(2, 3)).mul_(st["scale"])
    seen = (kv_len - q_len)[:, None] + i + 1                                            # keys that row i sees
    hidden = torch.arange(L, device="cuda")[None, None, :] >= seen[:, :, None]           # [R, Q, L]
    s.view(R, hk, Q, group, L).masked_fill_(hidden[:, None, :, None, :], -math.inf)
    o, lse = _softmax_product(s, cached(st["v"], st["v_scale"]))
    r, at = _token_places(q_off, st["tokens"])
    o = o.view(R, hk, Q, group, d)[r, :, at].reshape(-1, case["heads"], d)
    lse = lse.view(R, hk, Q, group)[r, :, at].reshape(-1, case["heads"])
    return dict(out=o.to(torch.bfloat16), lse=lse)


def _plain_prompt(st):
    case = st["case"]
    hk, d = case["kv_heads"], case["dim"]
    group = case["heads"] // hk
    B, L = case["B"], st["longest"]
    off = st["seq_off"].long()
    n = st["q"].shape[0]
    at = (off[:-1, None] + torch.arange(L, device="cuda")).clamp_max(n - 1)
    q = st["q"][at].float().view(B, L, hk, group, d).permute(0, 2, 3, 1, 4)
    k = st["k"][at].float().permute(0, 2, 3, 1)[:, :, None]
    v = st["v"][at].float().permute(0, 2, 1, 3)[:, :, None]
    s = torch.matmul(q, k).mul_(st["scale"])                                            # [B, hk, group, L, L]
    late = torch.ones((L, L), dtype=torch.bool, device="cuda").triu_(1)
    s.masked_fill_(late, -math.inf)
    o, lse = _softmax_product(s, v)
    r, i = _token_places(off, n)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, L, hk * group, d)[r, i]
    lse = lse.permute(0, 3, 1, 2).reshape(B, L, hk * group)[r, i]
    return dict(out=o.to(torch.bfloat16), lse=lse)


# ------------------------------------------------------------------ one pass
def _own(st):
    from speculative_decoding_drafting_gb300 import binding
    case = st["case"]
    if case["op"] == "prompt":
        r = binding.attn_prompt(st["q"], st["k"], st["v"], st["seq_off"], scale=st["scale"], lse=True, ws=st.get("ws"))
        st["ws"] = r["ws"]                       # the workspace is kept, as a serving loop keeps it
        return dict(out=r["out"], lse=r["lse"])
    cache = binding.KvCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
    if case["op"] == "write":
        st["ws"] = binding.kv_write(cache, st["K"], st["V"], st["q_off"], st["kv_len"], st["page_table"],
                                    ws=st.get("ws"))
        out = dict(k=st["k"], v=st["v"])
        if case["cache"] == "e4m3":
            out.update(k_scale=st["k_scale"], v_scale=st["v_scale"])
        return out
    if case["op"] == "read":
        r = binding.kv_read(cache, st["kv_off"], st["page_table"], st["kv_tokens"], ws=st.get("ws"))
        st["ws"] = r["ws"]
        return dict(K=r["K"], V=r["V"])
    r = binding.attn_paged(st["q"], cache, st["q_off"], st["kv_len"], st["page_table"], scale=st["scale"], lse=True,
                           ws=st.get("ws"))
    st["ws"] = r["ws"]
    return dict(out=r["out"], lse=r["lse"])


def run(state):
    if own:
        return _own(state)
    plain = dict(write=_plain_write, read=_plain_read, paged=_plain_paged, prompt=_plain_prompt)
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _attend(q, k, v, scale, first):
    """One head's rows q [n, d] over k, v [m, d] in 64 bits: row i sees keys 0 .. first + i."""
    out, lse = torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    step = max(1, (1 << 26) // max(1, k.shape[0]))
    for a in range(0, q.shape[0], step):
        b = min(q.shape[0], a + step)
        last = min(k.shape[0], first + b)
        if last <= 0:
            continue
        s = q[a:b] @ k[:last].T * scale
        s += torch.where(torch.arange(last, device=q.device)[None] <= first + torch.arange(a, b, device=q.device)[:, None],
                         0.0, -math.inf)
        z = torch.logsumexp(s, 1)
        lse[a:b] = z
        p = torch.exp(s - torch.where(torch.isinf(z), torch.zeros_like(z), z)[:, None])
        out[a:b] = p @ v[:last]
    return out, lse


def exact(case, seed):
    flops = work(case)["flops"]
    if case["op"] in ("paged", "prompt") and flops > 4e12:
        return None
    st = prepare(case, seed)
    kv, q = _lengths(case, _LENGTH_SEED)
    if case["op"] == "prompt":
        group = case["heads"] // case["kv_heads"]
        n = sum(kv)
        out = torch.zeros((n, case["heads"], case["dim"]), dtype=torch.float64, device="cuda")
        lse = torch.zeros((n, case["heads"]), dtype=torch.float64, device="cuda")
        a = 0
        for m in kv:
            for h in range(case["heads"]):
                c = h // group
                out[a:a + m, h], lse[a:a + m, h] = _attend(st["q"][a:a + m, h].double(), st["k"][a:a + m, c].double(),
                                                           st["v"][a:a + m, c].double(), st["scale"], 0)
            a += m
        return dict(out=out, lse=lse)
    page = case["page"]
    table = st["page_table"].cpu().tolist()
    if case["op"] == "write":
        res = {"k": st["k"].double(), "v": st["v"].double()}
        scales = {"k": st["k_scale"], "v": st["v_scale"]}
        t = 0
        for r, (n, m) in enumerate(zip(kv, q)):
            pos = list(range(n - m, n))
            at = torch.tensor([table[r][p // page] for p in pos], device="cuda")
            slot = torch.tensor([p % page for p in pos], device="cuda")
            for name, src in (("k", st["K"]), ("v", st["V"])):
                x = src[t:t + m].double()
                if case["cache"] == "bf16":
                    res[name][at, :, slot] = x
                    continue
                big = x.abs().max(-1, keepdim=True).values
                y = torch.where(big > 0, x * 448.0 / torch.where(big > 0, big, torch.ones_like(big)), torch.zeros_like(x))
                # nearest value with 3 bits behind the leading one (steps of 2^-9 at least), ties to even
                step = torch.exp2(torch.frexp(y.abs().clamp_min(2.0 ** -6)).exponent.double() - 4.0)
                res[name][at, :, slot] = torch.round(y / step) * step
                if scales[name].dtype != torch.float64:
                    scales[name] = scales[name].double()
                scales[name][at, :, slot] = big[..., 0] / 448.0
            t += m
        if case["cache"] == "e4m3":
            res.update(k_scale=scales["k"], v_scale=scales["v"])
        return res
    outs, lses, Ks, Vs = [], [], [], []
    t = 0
    for r, (n, m) in enumerate(zip(kv, q)):
        at = torch.tensor(table[r][:-(-n // page)], device="cuda")
        if st["k_scale"] is None:
            K, V = st["k"][at].double(), st["v"][at].double()
        else:
            K = st["k"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * st["k_scale"][at].double()[..., None]
            V = st["v"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * st["v_scale"][at].double()[..., None]
        K = K.transpose(0, 1).reshape(case["kv_heads"], -1, case["dim"])[:, :n]
        V = V.transpose(0, 1).reshape(case["kv_heads"], -1, case["dim"])[:, :n]
        if case["op"] == "read":
            Ks.append(K.transpose(0, 1))
            Vs.append(V.transpose(0, 1))
            continue
        group = case["heads"] // case["kv_heads"]
        o = torch.zeros((m, case["heads"], case["dim"]), dtype=torch.float64, device="cuda")
        z = torch.zeros((m, case["heads"]), dtype=torch.float64, device="cuda")
        for h in range(case["heads"]):
            o[:, h], z[:, h] = _attend(st["q"][t:t + m, h].double(), K[h // group], V[h // group], st["scale"], n - m)
        outs.append(o)
        lses.append(z)
        t += m
    if case["op"] == "read":
        return dict(K=torch.cat(Ks), V=torch.cat(Vs))
    return dict(out=torch.cat(outs), lse=torch.cat(lses))
