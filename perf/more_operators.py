"""A layer's way from its projections to its attention, as measured cases.

Four calls of a model with rotary positions and local layers:

* ``rope``   -- the norm of every query and key head and the rotation by the
  tokens' positions (one axis, or several for images and video), in one pass;
* ``append`` -- the same on the way into a paged cache: queries come out, keys
  and values go into the pages as bf16 or as e4m3 with a scale per (token, head);
* ``paged``  -- attention of each request's newest tokens over its pages when a
  token sees only the last ``window`` tokens and the first ``sinks`` ones;
* ``prompt`` -- the same mask over whole prompts, packed one after another.

``run`` computes a case in plain torch operations (``own`` false) or through
the library's entry points (``own`` true).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's next token: queries and keys of one layer, latency is all there is
        dict(name="rope-one", op="rope", T=1, start=4321, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False,
             axes=1, cycled=False, theta=1e6, norm="bf16"),
        # a long video prompt: three axes, no norms
        dict(name="rope-video", op="rope", T=23457, start=117, heads=28, kv_heads=4, dim=128, rot=128, interleaved=False,
             axes=3, cycled=False, theta=1e6, norm=""),
        # verification of 256 requests, blocks of up to 5 drafts and the token before them
        dict(name="append-verify", op="append", R=256, q_max=6, ragged=True, kv_min=200, kv_max=4000, heads=32, kv_heads=8,
             dim=128, page=16, cache="bf16", rot=128, interleaved=False, axes=1, cycled=False, theta=1e6, norm="bf16",
             keep=False),
        # a batch of prompts into a quantised cache; their keys are also handed to the prompts' attention
        dict(name="append-prompt-e4m3", op="append", R=30, q_max=0, ragged=False, kv_min=100, kv_max=2600, heads=32,
             kv_heads=8, dim=128, page=64, cache="e4m3", rot=128, interleaved=False, axes=1, cycled=False, theta=5e5,
             norm="f32", keep=True),
        # narrow heads of which half is rotated, in neighbouring pairs: a batch of short questions
        dict(name="append-partial", op="append", R=40, q_max=0, ragged=False, kv_min=1, kv_max=300, heads=16, kv_heads=4,
             dim=64, page=32, cache="bf16", rot=32, interleaved=True, axes=1, cycled=False, theta=1e4, norm="",
             keep=False),
        # one user deep in a long document, a local layer
        dict(name="paged-window-one", op="paged", R=1, q_max=1, ragged=False, kv_min=98765, kv_max=98765, heads=32,
             kv_heads=8, dim=128, page=16, cache="bf16", window=1024, sinks=4),
        # plain decoding of a large batch through a local layer
        dict(name="paged-window-decode", op="paged", R=256, q_max=1, ragged=False, kv_min=200, kv_max=12000, heads=64,
             kv_heads=8, dim=64, page=32, cache="bf16", window=1024, sinks=4),
        # verification blocks over a quantised cache, a wide window
        dict(name="paged-window-e4m3", op="paged", R=128, q_max=6, ragged=True, kv_min=500, kv_max=20000, heads=32,
             kv_heads=8, dim=128, page=64, cache="e4m3", window=4096, sinks=16),
        # a few questions arriving together, a narrow window
        dict(name="prompt-window-short", op="prompt", B=6, len_min=20, len_max=500, heads=16, kv_heads=4, dim=64,
             window=128, sinks=0),
        # a prefill batch of mixed lengths
        dict(name="prompt-window-packed", op="prompt", B=16, len_min=100, len_max=6000, heads=32, kv_heads=8, dim=128,
             window=1024, sinks=4),
        # one long document
        dict(name="prompt-window-long", op="prompt", B=1, len_min=30001, len_max=30001, heads=32, kv_heads=8, dim=128,
             window=4096, sinks=128),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "paged", "paged", "paged", "prompt", "prompt"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 6, 8, 8])
    heads = kv_heads * group
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    turn = dict(rot=rng.choice([dim, dim, dim // 2, dim * 3 // 4]), interleaved=rng.random() < 0.3,
                axes=rng.choice([1, 1, 3]), cycled=rng.random() < 0.5, theta=rng.choice([1e4, 5e5, 1e6]),
                norm=rng.choice(["", "bf16", "f32"]))
    # values of one token against the listed video prompt's
    room = int(23457 * 32 * 128 / ((heads + kv_heads) * dim))
    if op == "rope":
        return dict(op=op, T=_between(rng, 1, min(room, 60000)), start=rng.randint(0, 200000), heads=heads,
                    kv_heads=kv_heads, dim=dim, **turn)
    if op == "append":
        R = _between(rng, 1, 256)
        q_max = rng.choice([0, 1, 6])
        kv_max = _between(rng, 8, max(8, min(78000, room) // R))
        return dict(op=op, R=R, q_max=q_max, ragged=q_max > 1, kv_min=rng.randint(max(1, min(q_max, kv_max)), kv_max),
                    kv_max=kv_max, heads=heads, kv_heads=kv_heads, dim=dim, page=page, cache=cache, keep=q_max == 0, **turn)
    window = _between(rng, 16, 8000)
    sinks = rng.choice([0, 0, 1, 4, 16, 130])
    if op == "paged":
        R = _between(rng, 1, 256)
        q_max = rng.choice([1, 1, 2, 5, 6, 9, 17])
        # no more visible values than the listed verification batch has
        window = min(window, max(16, 128 * 4096 * 8 // (R * kv_heads)), max(16, 128 * 4096 * 6 * 4 // (R * q_max * group)))
        kv_max = _between(rng, 2 * q_max, 1500000 // R)
        kv_min = rng.randint(q_max, kv_max) if rng.random() < 0.5 else min(kv_max, q_max + rng.randint(0, 40))
        return dict(op=op, R=R, q_max=q_max, ragged=q_max > 1 and rng.random() < 0.7, kv_min=kv_min, kv_max=kv_max,
                    heads=heads, kv_heads=kv_heads, dim=dim, page=page, cache=cache, window=window, sinks=sinks)
    B = _between(rng, 1, 64)
    kv_heads = min(kv_heads, 32 // group) or 1
    # tokens x window x heads bounded by the listed long document's
    most = 30001 * 4096 * 32 // (kv_heads * group)
    longest = int(min(60000, most // min(window + sinks, 30001)) // B)
    len_max = _between(rng, 1, max(1, longest))
    return dict(op=op, B=B, len_min=rng.randint(1, len_max), len_max=len_max, heads=kv_heads * group, kv_heads=kv_heads,
                dim=dim, window=window, sinks=sinks)


# lengths are the case's, not the seed's: passes on other inputs cost the same
_LENGTH_SEED = 21


def _lengths(case):
    """(kv_len, q_len) of a case as Python lists."""
    g = torch.Generator().manual_seed(_LENGTH_SEED)
    if case["op"] == "prompt":
        n = torch.randint(case["len_min"], case["len_max"] + 1, (case["B"],), generator=g)
        n[0] = case["len_max"]
        return n.tolist(), n.tolist()
    n = torch.randint(case["kv_min"], case["kv_max"] + 1, (case["R"],), generator=g)
    n[0] = case["kv_max"]
    if case["q_max"] == 0:                 # whole prompts: every cached token is new
        return n.tolist(), n.tolist()
    q = torch.full((case["R"],), case["q_max"], dtype=torch.int64)
    if case["ragged"]:
        q = torch.randint(1, case["q_max"] + 1, (case["R"],), generator=g)
        q[-1] = case["q_max"]
    return n.tolist(), torch.minimum(q, n).tolist()


def _pairs(first, count, window, sinks):
    """Keys seen in all by `count` tokens from position `first` on."""
    total = 0
    for p in range(first, first + count):
        low = max(0, p - window + 1)
        total += p + 1 - low + min(sinks, low)
    return total


def work(case):
    d, hk, h = case["dim"], case["kv_heads"], case["heads"]
    per_value = (4 if case.get("norm") else 0) + 3 * case.get("rot", 0) / d
    if case["op"] == "rope":
        values = case["T"] * (h + hk) * d
        return {"bytes": 4 * values + 4 * case["T"] * case["axes"], "flops": int(per_value * values)}
    kv, q = _lengths(case)
    if case["op"] == "append":
        n = sum(q)
        stored = 2 * d if case["cache"] == "bf16" else d + 4
        moved = n * h * 4 * d + n * hk * 2 * (2 * d + stored) + (n * hk * 2 * d if case["keep"] else 0)
        if case["axes"] > 1:
            moved += 4 * n * case["axes"]
        return {"bytes": moved, "flops": int(per_value * n * (h + hk) * d) + (0 if case["cache"] == "bf16" else 3 * n * hk * 2 * d)}
    W, S = case["window"], case["sinks"]
    if case["op"] == "prompt":
        pairs = sum(_pairs(0, n, W, S) for n in kv)
        return {"bytes": sum(kv) * (2 * h + 2 * hk) * d * 2, "flops": 4 * pairs * h * d}
    stored = 2 * d if case["cache"] == "bf16" else d + 4
    visible = 0
    for n, m in zip(kv, q):
        low = max(0, n - m - W + 1)
        visible += n - low + min(S, low)
    pairs = sum(_pairs(n - m, m, W, S) for n, m in zip(kv, q))
    return {"bytes": visible * hk * 2 * stored + sum(q) * h * d * 4, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1000 + int(seed))


def _rows(g, n, heads, dim, spread=0.0):
    """[n, heads, dim] bf16 rows; with `spread`, a few channels of each head run larger, as keys' do."""
    x = torch.randn((n, heads, dim), generator=g, device="cuda")
    if spread:
        loud = torch.rand((heads, dim), generator=g, device="cuda") < 0.04
        x = x * (1.0 + spread * loud)
    return x.to(torch.bfloat16)


def _quantise(x):
    """e4m3 codes and float32 scales of bf16 rows (the last axis), for a cache that is already there."""
    big = x.float().abs().amax(-1)
    return (x.float() * E4M3_MAX / big.clamp_min(1e-30)[..., None]).to(torch.float8_e4m3fn), big / E4M3_MAX


def _offsets(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)


def _axis_of(case):
    """The axis of each frequency: a quarter for time and the rest in halves, as blocks or in turn."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return [0] * half
    if case["cycled"]:
        return [i % 3 for i in range(half)]
    a, b = half // 4, half // 4 + (half - half // 4) // 2
    return [0 if i < a else (1 if i < b else 2) for i in range(half)]


def _grid_positions(n, start, axes):
    """[n, axes] positions: text counts on, an image or video patch has a time, a row and a column."""
    i = torch.arange(n, device="cuda")
    if axes == 1:
        return (start + i).to(torch.int32)[:, None].contiguous()
    return (start + torch.stack([i // 600, i // 30 % 20, i % 30], 1)).to(torch.int32)


def _turn_state(case, g, st):
    half = case["rot"] // 2
    st["inv_freq"] = [case["theta"] ** (-i / half) for i in range(half)]
    st["axis"] = _axis_of(case)
    st["q_w"] = st["k_w"] = None
    if case["norm"]:
        t = torch.bfloat16 if case["norm"] == "bf16" else torch.float32
        for name in ("q_w", "k_w"):
            st[name] = (1.0 + 0.2 * torch.randn((case["dim"],), generator=g, device="cuda")).to(t)


def prepare(case, seed):
    g = _generator(seed)
    hk, d, h = case["kv_heads"], case["dim"], case["heads"]
    st = dict(case=case, scale=1.0 / math.sqrt(d))
    if case["op"] == "rope":
        _turn_state(case, g, st)
        # slices of one projection, as a model has them
        y = _rows(g, case["T"], h + 2 * hk, d, 3.0)
        st["q"], st["k"] = y[:, :h], y[:, h:h + hk]
        st["positions"] = _grid_positions(case["T"], case["start"], case["axes"])
        return st
    kv, q = _lengths(case)
    if case["op"] == "prompt":
        n = sum(kv)
        st["lengths"] = kv
        st["q"] = _rows(g, n, h, d) * 1.5
        st["k"] = _rows(g, n, hk, d, 3.0)
        st["v"] = _rows(g, n, hk, d)
        st["seq_off"] = _offsets(kv)
        return st
    page, R = case["page"], case["R"]
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
    st["tokens"] = sum(q)
    st["q_longest"] = max(q)
    st["k_scale"] = st["v_scale"] = None
    if case["op"] == "append":
        _turn_state(case, g, st)
        y = _rows(g, sum(q), h + 2 * hk, d, 3.0)
        st["q"], st["K"], st["V"] = y[:, :h], y[:, h:h + hk], y[:, h + hk:]
        st["positions"] = None if case["axes"] == 1 else _grid_positions(sum(q), 0, case["axes"])
        dtype = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
        st["k"] = torch.zeros((pages, hk, page, d), device="cuda").to(dtype)
        st["v"] = torch.zeros((pages, hk, page, d), device="cuda").to(dtype)
        if case["cache"] == "e4m3":
            st["k_scale"] = torch.zeros((pages, hk, page), device="cuda")
            st["v_scale"] = torch.zeros((pages, hk, page), device="cuda")
        return st
    st["k"] = _rows(g, pages * page, hk, d, 3.0).view(pages, page, hk, d).transpose(1, 2).contiguous()
    st["v"] = _rows(g, pages * page, hk, d).view(pages, page, hk, d).transpose(1, 2).contiguous()
    if case["cache"] == "e4m3":
        st["k"], st["k_scale"] = _quantise(st["k"])
        st["v"], st["v_scale"] = _quantise(st["v"])
    st["q"] = _rows(g, sum(q), h, d) * 1.5
    return st


# ------------------------------------------------------------------ plain forms
def _token_places(off, n):
    """For n packed tokens: the request each belongs to and its place in it."""
    t = torch.arange(n, device="cuda")
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    return r, t - off[r]


def _plain_turn(st, x, w, cos, sin):
    """Norm and rotation of x [n, heads, dim] in 32 bits; cos and sin [n, 1, rot / 2]."""
    case = st["case"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    rot = case["rot"]
    z = y.clone()
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z[..., 0:rot:2] = a * cos - b * sin
        z[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z[..., :rot // 2] = a * cos - b * sin
        z[..., rot // 2:rot] = b * cos + a * sin
    return z


def _angles(st, positions):
    """cos and sin [n, 1, rot / 2] of positions [n, axes]; far positions need the angle in 64 bits."""
    axis = torch.tensor(st["axis"], device="cuda")
    t = positions[:, axis].double() * torch.tensor(st["inv_freq"], dtype=torch.float64, device="cuda")
    return t.cos().float()[:, None], t.sin().float()[:, None]


def _plain_rope(st):
    cos, sin = _angles(st, st["positions"])
    return dict(q=_plain_turn(st, st["q"], st["q_w"], cos, sin).to(torch.bfloat16),
                k=_plain_turn(st, st["k"], st["k_w"], cos, sin).to(torch.bfloat16))


def _plain_append(st):
    case = st["case"]
    page = case["page"]
    q_off, kv_len = st["q_off"].long(), st["kv_len"].long()
    r, i = _token_places(q_off, st["tokens"])
    pos = kv_len[r] - (q_off[r + 1] - q_off[r]) + i
    cos, sin = _angles(st, pos[:, None] if st["positions"] is None else st["positions"])
    K = _plain_turn(st, st["K"], st["k_w"], cos, sin)
    out = dict(q=_plain_turn(st, st["q"], st["q_w"], cos, sin).to(torch.bfloat16))
    if case["keep"]:
        out["kept"] = K.to(torch.bfloat16)
    at = st["page_table"][r, pos // page].long()
    slot = pos % page
    out.update(k=st["k"], v=st["v"])
    if case["cache"] == "bf16":
        st["k"][at, :, slot] = K.to(torch.bfloat16)
        st["v"][at, :, slot] = st["V"]
        return out
    x = torch.stack([K, st["V"].float()])
    big = x.abs().amax(-1, keepdim=True)
    codes = torch.where(big > 0, x * E4M3_MAX / big.clamp_min(1e-38), torch.zeros_like(x)).to(torch.float8_e4m3fn)
    scale = (big / E4M3_MAX)[..., 0]
    # index_put on the bytes: torch has none for 8-bit floats
    st["k"].view(torch.uint8)[at, :, slot] = codes[0].view(torch.uint8)
    st["v"].view(torch.uint8)[at, :, slot] = codes[1].view(torch.uint8)
    st["k_scale"][at, :, slot] = scale[0]
    st["v_scale"][at, :, slot] = scale[1]
    out.update(k_scale=st["k_scale"], v_scale=st["v_scale"])
    return out


def _softmax_product(s, v):
    """softmax(s) v and the log-sum-exp of s's rows; a row of -inf alone gives 0 and -inf.  s is used up."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    s = s.sub_(m).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (m + torch.log(total))[..., 0]


def _plain_paged(st):
    """Every request's first `sinks` keys and its last ones, gathered into one batch with a mask."""
    case = st["case"]
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    group = case["heads"] // hk
    R, Q, W, S = case["R"], st["q_longest"], case["window"], case["sinks"]
    q_off, kv_len = st["q_off"].long(), st["kv_len"].long()
    q_len = q_off[1:] - q_off[:-1]
    i = torch.arange(Q, device="cuda")
    at = kv_len - q_len                                                                  # the first new token's position
    low = (at - W + 1).clamp_min(0)
    span = min(W + Q, case["kv_max"])
    tail = low[:, None] + torch.arange(span, device="cuda")
    head = torch.arange(min(S, case["kv_max"]), device="cuda").expand(R, -1)
    pos = torch.cat([head, tail], 1)                                                     # [R, L]
    # a sink that the tail holds too counts there
    real = torch.cat([head < low[:, None], tail < kv_len[:, None]], 1)
    L = pos.shape[1]
    safe = torch.where(real, pos, torch.zeros_like(pos))
    pid, slot = st["page_table"].long().clamp_min(0).gather(1, safe // page), safe % page

    def cached(x, scale):
        y = x.view(torch.uint8)[pid, :, slot].view(x.dtype) if scale is not None else x[pid, :, slot]
        y = y.float()
        if scale is not None:
            y = y * scale[pid, :, slot][..., None]
        return y.transpose(1, 2)                                                         # [R, hk, L, d]

    rows = st["q"][(q_off[:-1, None] + i).clamp_max(st["tokens"] - 1)].float()          # [R, Q, heads, d]
    rows = rows.view(R, Q, hk, group, d).permute(0, 2, 1, 3, 4).reshape(R, hk, Q * group, d)
    s = torch.matmul(rows, cached(st["k"], st["k_scale"]).transpose(2, 3)).mul_(st["scale"])
    p = (at[:, None] + i)[:, :, None]
    seen = real[:, None] & (pos[:, None] <= p) & ((p - pos[:, None] < W) | (pos[:, None] < S))   # [R, Q, L]
    s.view(R, hk, Q, group, L).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    o, lse = _softmax_product(s, cached(st["v"], st["v_scale"]))
    r, k = _token_places(q_off, st["tokens"])
    o = o.view(R, hk, Q, group, d)[r, :, k].reshape(-1, case["heads"], d)
    lse = lse.view(R, hk, Q, group)[r, :, k].reshape(-1, case["heads"])
    return dict(out=o.to(torch.bfloat16), lse=lse)


def _plain_prompt(st):
    """Blocks of tokens over the keys that one of them sees."""
    case = st["case"]
    hk, d, W, S = case["kv_heads"], case["dim"], case["window"], case["sinks"]
    group = case["heads"] // hk
    outs, lses = [], []
    base = 0
    for n in st["lengths"]:
        step = max(64, min(n, W, 2048))
        for a in range(0, n, step):
            b = min(n, a + step)
            low = max(0, a - W + 1)
            pos = torch.cat([torch.arange(min(S, low), device="cuda"), torch.arange(low, b, device="cuda")])
            q = st["q"][base + a:base + b].float().view(b - a, hk, group, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
            k = st["k"][base + pos].float().permute(1, 2, 0)
            v = st["v"][base + pos].float().permute(1, 0, 2)
            s = torch.matmul(q, k).mul_(st["scale"])                                     # [hk, group * rows, keys]
            p = torch.arange(a, b, device="cuda")[:, None]
            hidden = (pos > p) | ((p - pos >= W) & (pos >= S))
            s.view(hk, group, b - a, -1).masked_fill_(hidden, -math.inf)
            o, lse = _softmax_product(s, v)
            outs.append(o.view(hk, group, b - a, d).permute(2, 0, 1, 3).reshape(b - a, hk * group, d).to(torch.bfloat16))
            lses.append(lse.view(hk * group, b - a).T)
        base += n
    return dict(out=torch.cat(outs), lse=torch.cat(lses))


# ------------------------------------------------------------------ one pass
def _own(st):
    from speculative_decoding_drafting_gb300 import binding
    case = st["case"]
    if case["op"] in ("rope", "append"):
        if "rope" not in st:                     # kept, as a model keeps them
            st["rope"] = binding.Rope(st["inv_freq"], st["axis"], interleaved=case["interleaved"])
            st["norm"] = binding.HeadNorm(st["q_w"], st["k_w"], EPS) if case["norm"] else None
        if case["op"] == "rope":
            r = binding.qk_rope(st["q"], st["k"], st["positions"], rope=st["rope"], norm=st["norm"])
            return dict(q=r["q"], k=r["k"])
        cache = binding.KvCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        r = binding.rope_write(cache, st["q"], st["K"], st["V"], st["q_off"], st["kv_len"], st["page_table"],
                               rope=st["rope"], norm=st["norm"], positions=st["positions"], keep=case["keep"],
                               ws=st.get("ws"))
        st["ws"] = r["ws"]
        out = dict(q=r["q"])
        if case["keep"]:
            out["kept"] = r["k"]
        out.update(k=st["k"], v=st["v"])
        if case["cache"] == "e4m3":
            out.update(k_scale=st["k_scale"], v_scale=st["v_scale"])
        return out
    if case["op"] == "prompt":
        r = binding.attn_prompt(st["q"], st["k"], st["v"], st["seq_off"], scale=st["scale"], lse=True, ws=st.get("ws"),
                                window=case["window"], sinks=case["sinks"])
    else:
        cache = binding.KvCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        r = binding.attn_paged(st["q"], cache, st["q_off"], st["kv_len"], st["page_table"], scale=st["scale"], lse=True,
                               ws=st.get("ws"), window=case["window"], sinks=case["sinks"])
    st["ws"] = r["ws"]                           # the workspace is kept, as a serving loop keeps it
    return dict(out=r["out"], lse=r["lse"])


def run(state):
    if own:
        return _own(state)
    plain = dict(rope=_plain_rope, append=_plain_append, paged=_plain_paged, prompt=_plain_prompt)
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _turned(st, x, w, positions):
    """x [n, heads, dim] normed and turned, pair by pair as complex numbers."""
    case = st["case"]
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS) * w.double()
    half = case["rot"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    angle = torch.stack([positions[:, a].double() * f for a, f in zip(st["axis"], st["inv_freq"])], 1)
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    y = y.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _nearest_e4m3(y):
    """The nearest value with 3 bits behind the leading one (steps of 2^-9 at least), ties to even."""
    step = torch.exp2(torch.frexp(y.abs().clamp_min(2.0 ** -6)).exponent.double() - 4.0)
    return torch.round(y / step) * step


def _weighted(q, k, v, seen, scale):
    """Rows q [heads, n, d] over k, v [kv heads, m, d] in 64 bits where seen [n, m] allows: out and log-sum-exp."""
    group = q.shape[0] // k.shape[0]
    s = torch.einsum("hgnd,hmd->hgnm", q.view(k.shape[0], group, *q.shape[1:]), k) * scale
    s = torch.where(seen, s, torch.full((), -math.inf, dtype=s.dtype, device=s.device))
    z = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
    return torch.einsum("hgnm,hmd->hgnd", p, v).reshape(q.shape), z.reshape(q.shape[:2])


def exact(case, seed):
    if case["op"] in ("paged", "prompt") and work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    if case["op"] == "rope":
        return dict(q=_turned(st, st["q"], st["q_w"], st["positions"]), k=_turned(st, st["k"], st["k_w"], st["positions"]))
    kv, q = _lengths(case)
    if case["op"] == "append":
        page = case["page"]
        table = st["page_table"].cpu()
        pos = [torch.arange(n - m, n) for n, m in zip(kv, q)]
        at = torch.cat([table[r][p // page] for r, p in enumerate(pos)]).long().cuda()
        pos = torch.cat(pos).cuda()
        slot = pos % page
        where = pos[:, None].expand(-1, case["axes"]) if st["positions"] is None else st["positions"]
        K = _turned(st, st["K"], st["k_w"], where)
        out = dict(q=_turned(st, st["q"], st["q_w"], where))
        if case["keep"]:
            out["kept"] = K
        for name, x in (("k", K), ("v", st["V"].double())):
            out[name] = st[name].double()
            if case["cache"] == "bf16":
                out[name][at, :, slot] = x
                continue
            big = x.abs().amax(-1)
            one = torch.ones_like(big)
            # the product is exact for bf16 values, so that their ties are ties
            y = _nearest_e4m3(x * 448.0 / torch.where(big > 0, big, one)[..., None])
            out[name][at, :, slot] = y
            out[name + "_scale"] = st[name + "_scale"].double()
            out[name + "_scale"][at, :, slot] = big / 448.0
        return out
    W, S = case["window"], case["sinks"]
    outs, lses = [], []
    if case["op"] == "prompt":
        base = 0
        for n in kv:
            rows = max(1, min(n, (1 << 28) // (case["heads"] * (W + S + 1)), 1024))
            for a in range(0, n, rows):
                p = torch.arange(a, min(n, a + rows), device="cuda")
                keys = torch.arange(0, int(p[-1]) + 1, device="cuda")
                keys = keys[(keys < S) | (keys > a - W)]
                seen = (keys[None] <= p[:, None]) & ((keys[None] > p[:, None] - W) | (keys[None] < S))
                o, z = _weighted(st["q"][base + p].double().transpose(0, 1).contiguous(),
                                 st["k"][base + keys].double().transpose(0, 1), st["v"][base + keys].double().transpose(0, 1),
                                 seen, st["scale"])
                outs.append(o.transpose(0, 1))
                lses.append(z.T)
            base += n
        return dict(out=torch.cat(outs), lse=torch.cat(lses))
    page = case["page"]
    table = st["page_table"].long()
    t = 0
    for r, (n, m) in enumerate(zip(kv, q)):
        keys = torch.arange(n, device="cuda")
        keys = keys[(keys < S) | (keys > n - m - W)]
        pid, slot = table[r][keys // page], keys % page
        if st["k_scale"] is None:
            K, V = st["k"][pid, :, slot].double(), st["v"][pid, :, slot].double()
        else:
            K, V = (st[c].view(torch.uint8)[pid, :, slot].view(torch.float8_e4m3fn).double()
                    * st[c + "_scale"][pid, :, slot].double()[..., None] for c in ("k", "v"))
        p = torch.arange(n - m, n, device="cuda")
        seen = (keys[None] <= p[:, None]) & ((keys[None] > p[:, None] - W) | (keys[None] < S))
        o, z = _weighted(st["q"][t:t + m].double().transpose(0, 1).contiguous(), K.transpose(0, 1), V.transpose(0, 1), seen,
                         st["scale"])
        outs.append(o.transpose(0, 1))
        lses.append(z.T)
        t += m
    return dict(out=torch.cat(outs), lse=torch.cat(lses))
