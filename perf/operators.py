"""Measured cases of the serving operators: rotary positions, appending to a
paged key/value cache, and attention of new tokens over that cache.

`listed()` names the cases, `draw()` gives more of the same ranges, `prepare()`
makes what a program holds before the call, `run()` makes one pass and
`work()` says what such a pass cannot do without.  With `own` false a pass is
the operator's formula in elementary torch operations (32 bits, rounded once);
with `own` true it is the library's call.  `exact()` is the formula in 64 bits.

Shapes: q [B, Hq, L, dqk], k [B, Hkv, L, dqk], v [B, Hkv, L, dv] in bf16;
caches [pages, Hkv, page, d] in bf16 or e4m3 (e4m3 holds x / scale[head]).
"""
import math

import torch

own = False

CUDA = "cuda"
E4M3_MAX = 448.0  # largest finite e4m3 value

# (Hq, Hkv, dqk, dv): the head layouts of the workloads and of the tests
HEADS = [(32, 8, 128, 128), (16, 8, 128, 128), (2, 2, 64, 64), (128, 128, 192, 128), (8, 1, 128, 128),
         (3, 1, 64, 64)]


def _heads(i):
    return dict(zip(("Hq", "Hkv", "dqk", "dv"), HEADS[i]))


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a training step's q and k before the dense causal GQA attention
        dict(name="rope_train", op="rope", B=2, L=4096, **_heads(0), rot=128, offset=0, interleaved=False, backward=False),
        # the gradient of the same step for 192-wide heads that rotate their last 64 dimensions
        dict(name="rope_grad_wide", op="rope", B=1, L=4096, **_heads(3), rot=64, offset=128, interleaved=True,
             backward=True),
        # a short odd sequence: latency
        dict(name="rope_short", op="rope", B=1, L=257, **_heads(2), rot=64, offset=0, interleaved=False, backward=False),
        # one request's next token: latency
        dict(name="append_one", op="append", B=1, L=1, start=1000, **_heads(0), page=16, cache="bf16", layout="heads",
             fused=True, packed=False, rot=128, offset=0, interleaved=False, k_out=False),
        # the next token of a large batch, 8-bit cache
        dict(name="append_step_e4m3", op="append", B=256, L=1, start=500, **_heads(1), page=64, cache="e4m3",
             layout="heads", fused=True, packed=False, rot=128, offset=0, interleaved=False, k_out=False),
        # packed prompts (documents of one 32768-token row), rotated keys kept for the prompt's attention
        dict(name="append_prompts", op="append", B=1, L=32768, start=0, **_heads(1), page=128, cache="bf16",
             layout="heads", fused=False, packed=True, rot=128, offset=0, interleaved=False, k_out=True),
        # one request early in its answer: latency
        dict(name="decode_one", op="decode", B=1, Lq=1, longest=300, ragged=False, **_heads(0), page=16, cache="bf16",
             layout="heads", window=-1, softcap=0.0),
        # an ordinary serving batch of mixed lengths
        dict(name="decode_batch", op="decode", B=64, Lq=1, longest=4096, ragged=True, **_heads(0), page=16,
             cache="bf16", layout="heads", window=-1, softcap=0.0),
        # long contexts through a local window with a soft cap
        dict(name="decode_window", op="decode", B=16, Lq=1, longest=65536, ragged=True, **_heads(0), page=64,
             cache="bf16", layout="heads", window=4095, softcap=30.0),
        # 128 heads of their own keys, 192 / 128 wide, token-major pages
        dict(name="decode_wide", op="decode", B=4, Lq=1, longest=4096, ragged=True, **_heads(3), page=64, cache="bf16",
             layout="tokens", window=-1, softcap=0.0),
        # many long requests, 8-bit cache
        dict(name="decode_long_e4m3", op="decode", B=64, Lq=1, longest=32768, ragged=True, **_heads(0), page=64,
             cache="e4m3", layout="heads", window=-1, softcap=0.0),
        # four draft tokens per request, checked at once
        dict(name="decode_draft", op="decode", B=8, Lq=4, longest=8191, ragged=True, **_heads(1), page=32,
             cache="bf16", layout="heads", window=-1, softcap=0.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "decode", "decode"))
    h = _heads(rng.randrange(len(HEADS)))
    wide = h["dqk"] == 192
    rot = 64 if wide or h["dqk"] == 64 else rng.choice((64, 128))
    pair = dict(rot=rot, offset=128 if wide else 0, interleaved=rng.random() < 0.5)
    page = rng.choice((16, 32, 64, 128))
    paged = dict(page=page, cache=rng.choice(("bf16", "e4m3")), layout=rng.choice(("heads", "tokens")))
    per_token = h["Hq"] * h["dqk"] + h["Hkv"] * (h["dqk"] + h["dv"])
    if op == "rope":
        B = rng.randint(1, 4)
        L = _log(rng, 1, max(1, min(8192, 200_000_000 // (B * per_token))))
        return dict(op=op, B=B, L=L, **h, **pair, backward=rng.random() < 0.5)
    if op == "append":
        if rng.random() < 0.5:
            return dict(op=op, B=_log(rng, 1, 256), L=1, start=_log(rng, 1, 1000), **h, **paged, fused=rng.random() < 0.5,
                        packed=False, **pair, k_out=False)
        packed = rng.random() < 0.5
        B = 1 if packed else rng.randint(1, 4)
        L = _log(rng, 2, max(2, min(32768, 100_000_000 // (B * per_token))))
        return dict(op=op, B=B, L=L, start=0 if packed else _log(rng, 1, 1000), **h, **paged, fused=False, packed=packed,
                    **pair, k_out=rng.random() < 0.5)
    B = _log(rng, 1, 64)
    width = h["Hkv"] * (h["dqk"] + h["dv"])
    longest = _log(rng, 1, max(1, min(65536, 1_000_000_000 // (B * width))))
    windowed = rng.random() < 0.25
    return dict(op=op, B=B, Lq=rng.choice((1, 1, 1, 2, 4)), longest=longest, ragged=rng.random() < 0.75, **h, **paged,
                window=_log(rng, 1, 8192) if windowed else -1, softcap=30.0 if rng.random() < 0.25 else 0.0)


# ------------------------------------------------------------------ sizes that follow from a case
def _lengths(c):
    """Cache lengths of a decode case (before the seed shuffles them): evenly
    spread over 1 .. longest, or all the longest."""
    B, n = c["B"], c["longest"]
    return [max(1, (n * (i + 1)) // B) for i in range(B)] if c["ragged"] else [n] * B


def _documents(L):
    """Prompt lengths that fill a row of L tokens (spread over 64 .. 4096)."""
    out, n, i = [], L, 0
    while n > 0:
        out.append(min(n, 64 + (i * 1543) % 4033))
        n -= out[-1]
        i += 1
    return out


def work(c):
    Hq, Hkv, dqk, dv = c["Hq"], c["Hkv"], c["dqk"], c["dv"]
    if c["op"] == "rope":
        T = c["B"] * c["L"]
        n = T * (Hq + Hkv)
        return {"bytes": 2 * 2 * n * dqk + 4 * T + 4 * c["rot"] * c["L"], "flops": 3 * n * c["rot"]}
    size = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "append":
        T = c["B"] * c["L"]
        distinct = max(_documents(c["L"])) if c["packed"] else min(T, c["start"] + c["L"] if c["L"] == 1 else T)
        b = 2 * 2 * T * Hq * dqk + T * Hkv * (dqk + dv) * (2 + size) + 4 * T + 4 * c["rot"] * distinct
        return {"bytes": b + (2 * T * Hkv * dqk if c["k_out"] else 0), "flops": 3 * T * (Hq + Hkv) * c["rot"]}
    Lq, keys, pairs = c["Lq"], 0, 0
    for n in _lengths(c):
        w = c["window"]
        keys += n if w < 0 else min(n, w + Lq)
        for i in range(Lq):
            p = n - Lq + i
            pairs += 0 if p < 0 else (p + 1 if w < 0 else min(p + 1, w + 1))
    rows = c["B"] * Hq * Lq
    b = keys * Hkv * (dqk + dv) * size + 2 * rows * (dqk + dv) + 4 * rows + 4 * c["B"] + 4 * (keys // c["page"])
    return {"bytes": b, "flops": 2 * pairs * Hq * (dqk + dv)}


# ------------------------------------------------------------------ inputs
def _table(n, rot):
    """cos | sin of position * 10000^(-2i/rot), fp32 [n, rot], from 64-bit angles."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=CUDA) / rot)
    a = torch.arange(n, dtype=torch.float64, device=CUDA)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def _caches(c, g, pages):
    """Key and value caches [pages, Hkv, page, d] holding earlier tokens, and
    the scales of an 8-bit one."""
    Hkv, page = c["Hkv"], c["page"]
    scales = [None, None]
    if c["cache"] == "e4m3":
        scales = [0.01 * (0.75 + 0.5 * torch.rand(Hkv, generator=g, device=CUDA)) for _ in range(2)]
    made = []
    for d, s in ((c["dqk"], scales[0]), (c["dv"], scales[1])):
        shape = (pages, page, Hkv, d) if c["layout"] == "tokens" else (pages, Hkv, page, d)
        t = torch.empty(shape, dtype=torch.bfloat16 if s is None else torch.float8_e4m3fn, device=CUDA)
        for part in t.split(max(1, (1 << 28) // (page * Hkv * d))):
            x = torch.randn(part.shape, generator=g, device=CUDA)
            if s is not None:
                x = (x / (s[:, None] if c["layout"] == "tokens" else s[:, None, None])).clamp(-E4M3_MAX, E4M3_MAX)
            part.copy_(x)
        made.append(t.transpose(1, 2) if c["layout"] == "tokens" else t)
    return made, scales


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=CUDA).bfloat16()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=CUDA).manual_seed(seed)
    B, Hq, Hkv, dqk, dv = c["B"], c["Hq"], c["Hkv"], c["dqk"], c["dv"]
    s = dict(case=c)
    if c["op"] == "rope":
        s["q"], s["k"] = _normal(g, B, Hq, c["L"], dqk), _normal(g, B, Hkv, c["L"], dqk)
        s["table"] = _table(c["L"], c["rot"])
        s["positions"] = torch.arange(c["L"], dtype=torch.int32, device=CUDA).expand(B, -1).contiguous()
        return s
    if c["op"] == "append":
        L = c["L"]
        if c["fused"] and dqk == dv:  # views of one projection's output, token by token
            x = _normal(g, B, L, Hq + 2 * Hkv, dqk)
            s["q"], s["k"], s["v"] = (y.transpose(1, 2) for y in x.split((Hq, Hkv, Hkv), 2))
        else:
            s["q"], s["k"], s["v"] = _normal(g, B, Hq, L, dqk), _normal(g, B, Hkv, L, dqk), _normal(g, B, Hkv, L, dv)
        if c["packed"]:
            lens = _documents(L)
            n_seq, most = len(lens), max(lens)
            s["positions"] = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])[None].to(CUDA)
            s["seq_ids"] = torch.cat([torch.full((n,), i, dtype=torch.int32) for i, n in enumerate(lens)])[None].to(CUDA)
        else:
            n_seq, most = B, c["start"] + L
            first = torch.randint(0, c["start"], (B, 1), generator=g, device=CUDA)
            s["positions"] = (first + torch.arange(L, device=CUDA)).to(torch.int32)
            s["seq_ids"] = None
        s["table"] = _table(most, c["rot"])
        per = -(-most // c["page"])
        if L == 1:
            # every request's next token falls on a page of its own; the table's other entries are other pages
            pages = max(64, 2 * n_seq)
            order = torch.randperm(pages, generator=g, device=CUDA)
            bt = torch.randint(0, pages, (n_seq, per), generator=g, device=CUDA)
            bt.scatter_(1, (s["positions"] // c["page"]).long(), order[:n_seq, None])
        else:
            pages = n_seq * per
            bt = torch.randperm(pages, generator=g, device=CUDA).view(n_seq, per)
        s["block_table"] = bt.to(torch.int32).contiguous()
        (s["k_cache"], s["v_cache"]), (s["k_scale"], s["v_scale"]) = _caches(c, g, pages)
        s["q_out"] = torch.empty((B, Hq, L, dqk), dtype=torch.bfloat16, device=CUDA)
        s["k_out"] = torch.empty((B, Hkv, L, dqk), dtype=torch.bfloat16, device=CUDA) if c["k_out"] else None
        return s
    lens = torch.tensor(_lengths(c), device=CUDA)
    lens = lens[torch.randperm(B, generator=g, device=CUDA)]
    per = -(-c["longest"] // c["page"])
    need = (lens + c["page"] - 1) // c["page"]
    pages = sum(-(-n // c["page"]) for n in _lengths(c))
    order = torch.randperm(pages, generator=g, device=CUDA)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(per, device=CUDA)
    at = (first[:, None] + col).clamp(max=pages - 1)
    s["block_table"] = torch.where(col < need[:, None], order[at], -1).to(torch.int32)
    s["seq_lens"] = lens.to(torch.int32)
    s["q"] = _normal(g, B, Hq, c["Lq"], dqk)
    (s["k_cache"], s["v_cache"]), (s["k_scale"], s["v_scale"]) = _caches(c, g, pages)
    s["scale"] = 1.0 / math.sqrt(dqk)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        import block_sparse_flash_gb300 as splash
        if c["op"] == "rope":
            f = splash.rope_bwd if c["backward"] else splash.rope_fwd
            return f(s["q"], s["k"], s["positions"], s["table"], rot_offset=c["offset"], interleaved=c["interleaved"])
        if c["op"] == "append":
            splash.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["positions"], q=s["q"],
                                table=s["table"], rot_offset=c["offset"], interleaved=c["interleaved"],
                                seq_ids=s["seq_ids"], k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=s["q_out"],
                                k_out=s["k_out"])
            return _appended(s)
        return splash.paged_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], s["scale"],
                                   softcap=c["softcap"], window_left=c["window"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"])
    if c["op"] == "rope":
        return tuple(_rotate(s[x], s["positions"], s["table"], c, c["backward"]).bfloat16() for x in ("q", "k"))
    if c["op"] == "append":
        s["q_out"].copy_(_rotate(s["q"], s["positions"], s["table"], c, False))
        k = _rotate(s["k"], s["positions"], s["table"], c, False)
        if s["k_out"] is not None:
            s["k_out"].copy_(k)
        _store(s, s["k_cache"], k, s["k_scale"])
        _store(s, s["v_cache"], s["v"].float(), s["v_scale"])
        return _appended(s)
    return _attend(s)


def _appended(s):
    out = {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["k_out"] is not None:
        out["k"] = s["k_out"]
    return out


def _rotate(x, positions, table, c, inverse):
    """Pairs (a, b) of each row become (a cos - b sin, a sin + b cos); the
    gradient turns the other way."""
    cs = table[positions.long()][:, None]
    half, o = c["rot"] // 2, c["offset"]
    cos, sin = cs[..., :half], cs[..., half:]
    if inverse:
        sin = -sin
    y = x.float()
    r = y[..., o:o + c["rot"]]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((y[..., :o], r, y[..., o + c["rot"]:]), -1)


def _store(s, cache, x, scale):
    """x [B, Hkv, L, d] into the pages of its tokens."""
    page = s["case"]["page"]
    pos = s["positions"].long()
    seq = torch.arange(pos.shape[0], device=pos.device)[:, None].expand_as(pos) if s["seq_ids"] is None else s["seq_ids"].long()
    at = s["block_table"][seq, pos // page].long()
    x = x.transpose(1, 2)
    if scale is None:
        cache[at, :, pos % page] = x.to(cache.dtype)
    else:
        x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
        cache.view(torch.uint8)[at, :, pos % page] = x.view(torch.uint8)


def _gathered(cache, block_table, scale):
    """[B, Hkv, pages * page, d] in 32 bits."""
    at = block_table.long().clamp(min=0)
    x = cache[at] if scale is None else cache.view(torch.uint8)[at].view(cache.dtype)
    x = x.transpose(1, 2).float()
    x = x if scale is None else x * scale[:, None, None, None]
    return x.flatten(2, 3)


def _attend(s):
    c = s["case"]
    B, Lq, Hq, Hkv = c["B"], c["Lq"], c["Hq"], c["Hkv"]
    G = Hq // Hkv
    k = _gathered(s["k_cache"], s["block_table"], s["k_scale"])
    x = s["q"].float().view(B, Hkv, G * Lq, c["dqk"]) @ k.transpose(2, 3)
    x = x.view(B, Hkv, G, Lq, -1) * s["scale"]
    if c["softcap"] > 0:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    p = s["seq_lens"][:, None] - Lq + torch.arange(Lq, device=CUDA)
    p = p[:, None, None, :, None]
    j = torch.arange(x.shape[-1], device=CUDA)
    hide = j > p
    if c["window"] >= 0:
        hide = hide | (p - j > c["window"])
    x = x.masked_fill(hide, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    z = e.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["block_table"], s["v_scale"])
    o = (e.flatten(2, 3) @ v).view(B, Hkv, G, Lq, -1) / z.masked_fill(z == 0, 1.0)
    return o.bfloat16().view(B, Hq, Lq, -1), (m + torch.log(z)).view(B, Hq, Lq)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "decode":
        return _exact_attention(c, s)

    def turn(x, sign):
        y = x.double().clone()
        t = s["table"].double().index_select(0, s["positions"].reshape(-1).long()).view(*s["positions"].shape, -1)
        for i in range(c["rot"] // 2):
            m = c["offset"] + (2 * i if c["interleaved"] else i)
            n = m + 1 if c["interleaved"] else m + c["rot"] // 2
            z = torch.complex(x[..., m].double(), x[..., n].double())
            z = z * torch.complex(t[..., i], sign * t[..., c["rot"] // 2 + i])[:, None]
            y[..., m], y[..., n] = z.real, z.imag
        return y

    if c["op"] == "rope":
        return tuple(turn(s[x], -1.0 if c["backward"] else 1.0) for x in ("q", "k"))
    q, k = turn(s["q"], 1.0), turn(s["k"], 1.0)
    out = {"q": q, "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    if c["k_out"]:
        out["k"] = k
    Hkv, page, bt = c["Hkv"], c["page"], s["block_table"].tolist()
    own_row = [[b] * c["L"] for b in range(c["B"])]
    ids = own_row if s["seq_ids"] is None else s["seq_ids"].tolist()
    at, rows, cols, slots = [], [], [], []
    for b, line in enumerate(s["positions"].tolist()):
        for l, p in enumerate(line):
            rows.append(b)
            cols.append(l)
            slots.append(p % page)
            at.append(bt[ids[b][l]][p // page])
    at, rows, cols, slots = (torch.tensor(x, device=CUDA) for x in (at, rows, cols, slots))
    for name, x, scale in (("k_cache", k, s["k_scale"]), ("v_cache", s["v"].double(), s["v_scale"])):
        for h in range(Hkv):
            y = x[rows, h, cols]
            if scale is not None:
                y = (y / scale[h].double()).clamp(-E4M3_MAX, E4M3_MAX)
            out[name][at, h, slots] = y
    return out


def _exact_attention(c, s):
    B, Lq, Hq, Hkv, page = c["B"], c["Lq"], c["Hq"], c["Hkv"], c["page"]
    G = Hq // Hkv
    out = torch.zeros((B, Hq, Lq, c["dv"]), dtype=torch.float64, device=CUDA)
    lse = torch.full((B, Hq, Lq), -math.inf, dtype=torch.float64, device=CUDA)
    for b, n in enumerate(s["seq_lens"].tolist()):
        pages = s["block_table"][b, :-(-n // page)].long()
        kv = []
        for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
            raw = cache if scale is None else cache.view(torch.uint8)
            x = raw[pages].view(cache.dtype).double().permute(1, 0, 2, 3).reshape(Hkv, -1, cache.shape[3])[:, :n]
            kv.append(x if scale is None else x * scale.double().view(-1, 1, 1))
        for i in range(Lq):
            p = n - Lq + i
            if p < 0:
                continue
            lo = 0 if c["window"] < 0 else max(0, p - c["window"])
            k, v = kv[0][:, lo:p + 1], kv[1][:, lo:p + 1]
            q = s["q"][b, :, i].double().view(Hkv, G, -1)
            t = torch.einsum("hgd,hkd->hgk", q, k) * s["scale"]
            if c["softcap"] > 0:
                t = c["softcap"] * torch.tanh(t / c["softcap"])
            z = torch.logsumexp(t, -1)
            lse[b, :, i] = z.reshape(-1)
            out[b, :, i] = torch.einsum("hgk,hkd->hgd", (t - z[..., None]).exp(), v).reshape(Hq, -1)
    return out, lse
