"""Measured cases of serving with drafts, forks and several position axes:
attention of a tree of drafted tokens over the paged cache, rotary positions
with several axes (their gradient, and appending with them), and the upkeep of
a paged cache -- forking sequences and compacting them.

`listed()` names the cases, `draw()` gives more of the same ranges, `prepare()`
makes what a program holds before the call, `run()` makes one pass and
`work()` says what such a pass cannot do without.  With `own` false a pass is
the operator's formula in elementary torch operations (32 bits, rounded once);
with `own` true it is the library's call.  `exact()` is the definition in 64
bits, sequence by sequence.

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
        # one request's drafts early in its answer: latency
        dict(name="tree_one", op="tree", B=1, T=16, longest=300, ragged=False, **_heads(0), page=16, cache="bf16",
             layout="heads", window=-1, softcap=0.0, tree="random"),
        # an ordinary batch of mixed lengths, 32 drafts each
        dict(name="tree_batch", op="tree", B=32, T=32, longest=4096, ragged=True, **_heads(0), page=16, cache="bf16",
             layout="heads", window=-1, softcap=0.0, tree="random"),
        # 128 heads of their own keys, 192 / 128 wide, a local window and a soft cap, few drafts
        dict(name="tree_wide_window", op="tree", B=6, T=7, longest=6000, ragged=True, **_heads(3), page=64,
             cache="bf16", layout="tokens", window=1023, softcap=30.0, tree="beams"),
        # the largest trees over long contexts in 8 bits
        dict(name="tree_long_e4m3", op="tree", B=16, T=64, longest=32768, ragged=True, **_heads(0), page=64,
             cache="e4m3", layout="heads", window=-1, softcap=0.0, tree="random"),
        # q and k of a video's tokens before attention: time, height, width
        dict(name="rope_axes_video", op="rope", B=1, L=16384, **_heads(0), rot=128, sections="16 24 24", cycled=False,
             offset=0, interleaved=False, backward=False),
        # the gradient for 192-wide heads that rotate their last 64 dimensions, axes in turn from pair to pair
        dict(name="rope_axes_grad", op="rope", B=1, L=1111, **_heads(3), rot=64, sections="12 10 10", cycled=True,
             offset=128, interleaved=True, backward=True),
        # a batch's drafts into an 8-bit cache: slots in a row, rotations by depth
        dict(name="append_drafts_e4m3", op="append", B=32, L=16, **_heads(1), page=64, cache="e4m3", layout="heads",
             fused=True, rot=128, sections="64", cycled=False, offset=0, interleaved=False, k_out=False),
        # a prompt of images and text, rotated keys kept for its attention
        dict(name="append_video", op="append", B=1, L=8192, **_heads(0), page=128, cache="bf16", layout="heads",
             fused=False, rot=128, sections="16 24 24", cycled=False, offset=0, interleaved=False, k_out=True),
        # one request's accepted drafts: latency
        dict(name="compact_one", op="compact", B=1, span=16, moved=5, start=1000, **_heads(0), page=16, cache="bf16",
             layout="heads"),
        # half of the tokens of long sequences leave the cache
        dict(name="compact_evict", op="compact", B=8, span=16384, moved=8192, start=4, **_heads(0), page=16,
             cache="bf16", layout="heads"),
        # a beam search step: 16 requests of 4 beams
        dict(name="fork_beams", op="fork", groups=16, before=4, after=4, longest=2000, room=1, **_heads(0), page=16,
             cache="bf16", layout="heads"),
        # eight answers to each of 64 prompts
        dict(name="fork_samples", op="fork", groups=64, before=1, after=8, longest=4096, room=1, **_heads(0),
             page=128, cache="bf16", layout="heads"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "rope", "append", "compact", "fork"))
    h = _heads(rng.randrange(len(HEADS)))
    wide = h["dqk"] == 192
    width = h["Hkv"] * (h["dqk"] + h["dv"])
    paged = dict(page=rng.choice((16, 32, 64, 128)), cache=rng.choice(("bf16", "e4m3")),
                 layout=rng.choice(("heads", "tokens")))
    per_token = h["Hq"] * h["dqk"] + h["Hkv"] * (h["dqk"] + h["dv"])
    if op == "tree":
        B, T = _log(rng, 1, 32), _log(rng, 1, 64)
        windowed = rng.random() < 0.25
        # (keys x heads x widths of the cache, and pairs x heads x widths of the products)
        most = min(32768, 300_000_000 // (B * width), 140_000_000_000 // (B * T * h["Hq"] * (h["dqk"] + h["dv"])))
        return dict(op=op, B=B, T=T, longest=_log(rng, T, max(T, most)), ragged=rng.random() < 0.75, **h, **paged,
                    window=_log(rng, 1, 8192) if windowed else -1, softcap=30.0 if rng.random() < 0.25 else 0.0,
                    tree=rng.choice(("random", "beams", "chain")))
    if op in ("rope", "append"):
        rot = 64 if wide or h["dqk"] == 64 else rng.choice((64, 128))
        n = rng.randint(1, 4)
        cuts = sorted(rng.randint(1, rot // 2 - 1) for _ in range(n - 1))
        sections = tuple(b - a for a, b in zip([0] + cuts, cuts + [rot // 2]))
        if rng.random() < 0.5:  # (sections of whole groups of 8 pairs, as models have them)
            eight = rot // 16
            n = min(n, eight)
            sections = tuple(8 * (eight // n + (i < eight % n)) for i in range(n))
        turn = dict(rot=rot, sections=" ".join(map(str, sections)), cycled=rng.random() < 0.3, offset=128 if wide else 0,
                    interleaved=rng.random() < 0.5)
        B = rng.randint(1, 4)
        if op == "rope":
            L = _log(rng, 1, max(1, min(16384, 80_000_000 // (B * per_token))))
            return dict(op=op, B=B, L=L, **h, **turn, backward=rng.random() < 0.5)
        if rng.random() < 0.5:
            B, L = _log(rng, 1, 64), _log(rng, 1, 64)
        else:
            L = _log(rng, 2, 8192)
        L = max(1, min(L, 40_000_000 // (B * per_token)))
        return dict(op=op, B=B, L=L, **h, **paged, fused=rng.random() < 0.5, **turn, k_out=rng.random() < 0.5)
    if op == "compact":
        B = _log(rng, 1, 64)
        most = max(2, min(16384, 260_000_000 // (B * width)))
        span = _log(rng, 2, most)
        return dict(op=op, B=B, span=span, moved=_log(rng, 1, max(1, span // 2)), start=_log(rng, 1, min(2000, 4 * most)),
                    **h, **paged)
    after = rng.randint(1, 8)
    before, room = rng.choice((1, 1, 4, after)), _log(rng, 1, 64)
    # (the copied rows: at most a page for each new row; the pool: three or so)
    groups = _log(rng, 1, max(1, min(64, 250_000_000 // (after * paged["page"] * width))))
    longest = _log(rng, 1, max(1, min(8192, 600_000_000 // (groups * max(before, after) * width))))
    return dict(op=op, groups=groups, before=before, after=after, longest=longest, room=room, **h, **paged)


# ------------------------------------------------------------------ sizes that follow from a case
def _contexts(c):
    """Context lengths of a tree case (before the seed shuffles them): evenly
    spread up to longest - T, or all of that."""
    B, n = c["B"], c["longest"] - c["T"]
    return [(n * (i + 1)) // B for i in range(B)] if c["ragged"] else [n] * B


def _sections(c):
    """Pairs of each axis."""
    return [int(x) for x in c["sections"].split()]


def _axes(c):
    """The axis of each rotated pair: sections in a row, or taking turns until
    each is used up."""
    left, out = _sections(c), []
    if not c["cycled"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    while any(left):
        for a, n in enumerate(left):
            if n:
                left[a] -= 1
                out.append(a)
    return out


def _lengths(c):
    """Tokens of a fork case's rows."""
    n = c["longest"]
    return [max(1, (n * (g + 1)) // c["groups"]) for g in range(c["groups"])]


def work(c):
    Hq, Hkv, dqk, dv = c["Hq"], c["Hkv"], c["dqk"], c["dv"]
    size = 1 if c.get("cache") == "e4m3" else 2
    if c["op"] == "rope":
        T = c["B"] * c["L"]
        n = T * (Hq + Hkv)
        return {"bytes": 2 * 2 * n * dqk + 4 * T * len(_sections(c)), "flops": 3 * n * c["rot"]}
    if c["op"] == "append":
        T = c["B"] * c["L"]
        b = 2 * 2 * T * Hq * dqk + T * Hkv * (dqk + dv) * (2 + size) + 4 * T * (1 + len(_sections(c)))
        return {"bytes": b + (2 * T * Hkv * dqk if c["k_out"] else 0), "flops": 3 * T * (Hq + Hkv) * c["rot"]}
    if c["op"] == "compact":
        n = c["B"] * c["moved"]
        return {"bytes": 2 * n * Hkv * (dqk + dv) * size + 4 * n, "flops": 0}
    if c["op"] == "fork":
        page, rows, most = c["page"], 0, 0
        alone = c["before"] * (1 - (1 - 1 / c["before"]) ** c["after"])  # rows that some new row goes on from
        for n in _lengths(c):
            rows += (c["after"] - alone) * (n % page)  # (one of a row's heirs keeps its last page)
            most = max(most, -(-(n + c["room"]) // page))
        table = (c["before"] + c["after"]) * c["groups"] * most
        return {"bytes": int(2 * rows * Hkv * (dqk + dv) * size) + 4 * table + 8 * _pool(c), "flops": 0}
    T, w = c["T"], c["window"]
    keys, pairs = 0, 0
    for n in _contexts(c):
        keys += T + (n if w < 0 else min(n, w))
        pairs += T * (1 + (n if w < 0 else min(n, w)))  # (at the least: roots)
    rows = c["B"] * Hq * T
    b = keys * Hkv * (dqk + dv) * size + 2 * rows * (dqk + dv) + 4 * rows + 4 * c["B"] * (T + 1) + 4 * (keys // c["page"])
    return {"bytes": b, "flops": 2 * pairs * Hq * (dqk + dv)}


def _pool(c):
    """Pages of a fork case's cache: what both tables can hold, and some more."""
    page = c["page"]
    held = sum(c["before"] * -(-n // page) for n in _lengths(c))
    fresh = sum(c["after"] * (2 + -(-c["room"] // page)) for _ in _lengths(c))
    return held + fresh + 16


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


def _paging(c, g, lens):
    """A block table whose rows hold lens tokens in pages of no order, and its
    number of pages."""
    page = c["page"]
    need = torch.tensor([-(-n // page) for n in lens], device=CUDA)
    pages = max(1, sum(-(-n // page) for n in lens))
    order = torch.randperm(pages, generator=g, device=CUDA)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(max(1, -(-max(lens) // page)), device=CUDA)
    at = (first[:, None] + col).clamp(max=pages - 1)
    return torch.where(col < need[:, None], order[at], -1).to(torch.int32), pages


def _trees(c, g):
    """Parents of each sequence's drafts, int32 [B, T]: an earlier draft, -1
    for the context's last token, -2 for padding (trees of half to all of T)."""
    B, T = c["B"], c["T"]
    l = torch.arange(T, device=CUDA).expand(B, T)
    if c["tree"] == "chain":
        p = l - 1
    elif c["tree"] == "beams":  # four continuations side by side
        p = torch.where(l < 4, -1, l - 4)
    else:
        p = (torch.rand(B, T, generator=g, device=CUDA).sqrt() * (l + 1)).long().clamp(max=T - 1).minimum(l) - 1
    tokens = torch.randint((T + 1) // 2, T + 1, (B, 1), generator=g, device=CUDA)
    return torch.where(l < tokens, p, -2).to(torch.int32).contiguous()


def _video(n):
    """Positions of time, height and width: text, then frames of 16 x 24, then text."""
    i = torch.arange(n, device=CUDA)
    head = min(n, 37)
    j = (i - head).clamp(min=0)
    frames = max(0, (n - head - 11) // 384)
    film = (i >= head) & (j < frames * 384)
    t = head + j // 384
    after = head + max(frames, 24) + (i - head - frames * 384)
    out = [torch.where(film, x, torch.where(i < head, i, after)) for x in (t, head + j % 384 // 24, head + j % 24)]
    return torch.stack(out)


def _rotations(c, g):
    """Rotation positions int32 [axes, B, L] and a table that has them."""
    B, L, A = c["B"], c["L"], len(_sections(c))
    p = _video(L)[:, None].expand(3, B, L) + torch.randint(0, 64, (1, B, 1), generator=g, device=CUDA)
    p = p[torch.arange(A) % 3].to(torch.int32).contiguous()
    return p, _table(L + 256, c["rot"])


def prepare(case, seed):
    c = case
    g = torch.Generator(device=CUDA).manual_seed(seed)
    s = dict(case=c)
    Hq, Hkv, dqk, dv = c["Hq"], c["Hkv"], c["dqk"], c["dv"]
    if c["op"] == "tree":
        B, T = c["B"], c["T"]
        ctx = torch.tensor(_contexts(c))[torch.randperm(B, generator=torch.Generator().manual_seed(seed))].tolist()
        lens = [n + T for n in ctx]
        s["block_table"], pages = _paging(c, g, lens)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=CUDA)
        s["parents"] = _trees(c, g)
        s["q"] = _normal(g, B, Hq, T, dqk)
        (s["k_cache"], s["v_cache"]), (s["k_scale"], s["v_scale"]) = _caches(c, g, pages)
        s["scale"] = 1.0 / math.sqrt(dqk)
        return s
    if c["op"] in ("rope", "append"):
        B, L = c["B"], c["L"]
        if c.get("fused") and dqk == dv:  # views of one projection's output, token by token
            x = _normal(g, B, L, Hq + 2 * Hkv, dqk)
            s["q"], s["k"], s["v"] = (y.transpose(1, 2) for y in x.split((Hq, Hkv, Hkv), 2))
        else:
            s["q"], s["k"], s["v"] = _normal(g, B, Hq, L, dqk), _normal(g, B, Hkv, L, dqk), _normal(g, B, Hkv, L, dv)
        s["rot_positions"], s["table"] = _rotations(c, g)
        s["axes"] = bytes(_axes(c))  # laid out once
        if c["op"] == "rope":
            return s
        start = torch.randint(0, 200, (B, 1), generator=g, device=CUDA)
        s["positions"] = (start + torch.arange(L, device=CUDA)).to(torch.int32)
        s["block_table"], pages = _paging(c, g, [L + 200] * B)
        (s["k_cache"], s["v_cache"]), (s["k_scale"], s["v_scale"]) = _caches(c, g, pages)
        s["q_out"] = torch.empty((B, Hq, L, dqk), dtype=torch.bfloat16, device=CUDA)
        s["k_out"] = torch.empty((B, Hkv, L, dqk), dtype=torch.bfloat16, device=CUDA) if c["k_out"] else None
        return s
    if c["op"] == "compact":
        B, n = c["B"], c["start"] + c["span"]
        s["block_table"], pages = _paging(c, g, [n] * B)
        s["start"] = torch.full((B,), c["start"], dtype=torch.int32, device=CUDA)
        # `moved` of the span's tokens in order; the last sequence keeps fewer (a negative entry ends its list)
        keep = torch.rand(B, c["span"], generator=g, device=CUDA).argsort(1)[:, :c["moved"]].sort(1).values + c["start"]
        if B > 1:
            keep[-1, (c["moved"] + 1) // 2:] = -1
        s["src"] = keep.to(torch.int32)
        (s["k_cache"], s["v_cache"]), _ = _caches(c, g, pages)
        return s
    lens, before, after, page = _lengths(c), c["before"], c["after"], c["page"]
    most = -(-(max(lens) + c["room"]) // page)
    table = torch.full((c["groups"] * before, most), -1, dtype=torch.int32)
    pages = _pool(c)
    pool = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    refs = torch.zeros(pages, dtype=torch.int32)
    for i, n in enumerate(lens):  # a group's rows share their first half; each has its own rest
        cols, shared = -(-n // page), n // page // 2
        first = [pool.pop() for _ in range(shared)]
        for b in range(before):
            row = first + [pool.pop() for _ in range(cols - shared)]
            table[i * before + b, :cols] = torch.tensor(row, dtype=torch.int32)
            refs[row] += 1
    pick = torch.randint(0, before, (c["groups"], after), generator=torch.Generator().manual_seed(seed + 1))
    parents = (torch.arange(c["groups"])[:, None] * before + pick).flatten()
    keep = torch.tensor(lens).repeat_interleave(after)
    room = keep + c["room"]
    for name, x in (("block_table", table), ("refs", refs), ("parents", parents), ("keep", keep), ("room", room)):
        s[name] = x.to(torch.int32).to(CUDA)
    (s["k_cache"], s["v_cache"]), _ = _caches(c, g, pages)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        import block_sparse_flash_gb300 as splash
        if c["op"] == "tree":
            return splash.paged_tree_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                                            s["parents"], s["scale"], softcap=c["softcap"], window_left=c["window"],
                                            k_scale=s["k_scale"], v_scale=s["v_scale"])
        if c["op"] == "rope":
            f = splash.rope_axes_bwd if c["backward"] else splash.rope_axes_fwd
            return f(s["q"], s["k"], s["rot_positions"], s["table"], s["axes"], rot_offset=c["offset"],
                     interleaved=c["interleaved"])
        if c["op"] == "append":
            splash.paged_append_axes(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["positions"],
                                     s["rot_positions"], s["table"], s["axes"], q=s["q"], rot_offset=c["offset"],
                                     interleaved=c["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                     q_out=s["q_out"], k_out=s["k_out"])
            return _appended(s)
        if c["op"] == "compact":
            splash.paged_compact(s["k_cache"], s["v_cache"], s["block_table"], s["src"], s["start"])
            return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        table, refs, copies, short = splash.paged_remap(s["block_table"], s["parents"], s["keep"], s["room"], s["refs"],
                                                        c["page"])
        splash.paged_copy(s["k_cache"], s["v_cache"], copies)
        return {"table": table, "refs": refs, "copies": copies, "short": short, "k_cache": s["k_cache"],
                "v_cache": s["v_cache"]}
    if c["op"] == "tree":
        return _attend(s)
    if c["op"] == "rope":
        return tuple(_rotate(s[x], s, c["backward"]).bfloat16() for x in ("q", "k"))
    if c["op"] == "append":
        s["q_out"].copy_(_rotate(s["q"], s, False))
        k = _rotate(s["k"], s, False)
        if s["k_out"] is not None:
            s["k_out"].copy_(k)
        _store(s, s["k_cache"], k, s["k_scale"])
        _store(s, s["v_cache"], s["v"].float(), s["v_scale"])
        return _appended(s)
    if c["op"] == "compact":
        return _compact(s)
    return _fork(s)


def _appended(s):
    out = {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["k_out"] is not None:
        out["k"] = s["k_out"]
    return out


def _rotate(x, s, inverse):
    """Pairs (a, b) of each row become (a cos - b sin, a sin + b cos), each by
    the position of its own axis; the gradient turns the other way."""
    c, table = s["case"], s["table"]
    half, o = c["rot"] // 2, c["offset"]
    axis = torch.tensor(list(s["axes"]), device=x.device)
    pos = s["rot_positions"].long()[axis].permute(1, 2, 0)  # [B, L, half]
    pair = torch.arange(half, device=x.device)
    cos, sin = table[pos, pair][:, None], table[pos, half + pair][:, None]
    if inverse:
        sin = -sin
    y = x.float()
    r = y[..., o:o + c["rot"]]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((y[..., :o], r, y[..., o + c["rot"]:]), -1)


def _raw(cache):
    """A cache as its bits, for indexing."""
    return cache.view(torch.uint8) if cache.element_size() == 1 else cache


def _store(s, cache, x, scale):
    """x [B, Hkv, L, d] into the pages of its tokens."""
    page = s["case"]["page"]
    pos = s["positions"].long()
    at = s["block_table"].long().gather(1, pos // page)
    x = x.transpose(1, 2)
    if scale is not None:
        x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    _raw(cache)[at, :, pos % page] = _raw(x.to(cache.dtype))


def _compact(s):
    """Token src[b, m] becomes token start[b] + m, every read before any write."""
    page, bt = s["case"]["page"], s["block_table"].long()
    src = s["src"].long()
    ok = torch.cumsum(src < 0, 1) == 0
    dst = s["start"].long()[:, None] + torch.arange(src.shape[1], device=CUDA)
    src, dst = torch.where(ok, src, 0), torch.where(ok, dst, 0)
    b = torch.arange(src.shape[0], device=CUDA)[:, None].expand_as(src)
    b, src, dst = b[ok], src[ok], dst[ok]
    for name in ("k_cache", "v_cache"):
        raw = _raw(s[name])
        raw[bt[b, dst // page], :, dst % page] = raw[bt[b, src // page], :, src % page]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _count(pages, ok, n):
    return torch.zeros(n, dtype=torch.long, device=CUDA).index_add_(0, torch.where(ok, pages, 0).flatten(), ok.long().flatten())


def _fork(s):
    page, old, refs = s["case"]["page"], s["block_table"].long(), s["refs"].long()
    N, P, M = refs.shape[0], old.shape[1], s["parents"].shape[0]
    col = torch.arange(P, device=CUDA)
    row = torch.arange(M, device=CUDA)
    keep = s["keep"].long()
    room = torch.maximum(s["room"].long(), keep)
    kept = torch.where(col < ((keep + page - 1) // page)[:, None], old[s["parents"].long()], -1)
    uses = refs - _count(old, old >= 0, N) + _count(kept, kept >= 0, N)
    # a last page that holds other tokens too is the row's own only if nobody else has it
    part = keep % page != 0
    last = torch.where(part, kept.gather(1, (keep // page).clamp(max=P - 1)[:, None])[:, 0], 0)
    parts = _count(last, part, N)
    first = torch.full((N,), M, device=CUDA).scatter_reduce(0, last, torch.where(part, row, M), "amin")
    copy = part & ~((uses[last] == parts[last]) & (first[last] == row))
    held = (col * page < keep[:, None]) & ~(copy[:, None] & (col == (keep // page)[:, None]))
    need = (col * page < room[:, None]) & ~held
    order = torch.cumsum(need.flatten().long(), 0).view(M, P) - 1
    free = torch.cumsum((refs == 0).long(), 0)  # (the k-th free page, in ascending order)
    total = free[-1]
    kth = torch.full((N + 1,), -1, device=CUDA).scatter(0, torch.where(refs == 0, free - 1, N), torch.arange(N, device=CUDA))
    fresh = torch.where(need & (order < total), kth[order.clamp(min=0, max=N - 1)], -1)
    table = torch.where(need, fresh, torch.where(held, kept, -1))
    uses = uses - _count(last, copy, N) + _count(fresh, fresh >= 0, N)
    to = table.gather(1, (keep // page).clamp(max=P - 1)[:, None])[:, 0]
    copy = copy & (to >= 0)
    copies = torch.stack((torch.where(copy, last, -1), torch.where(copy, to, -1), torch.where(copy, keep % page, 0)), 1)
    short = (need.sum() - total).clamp(min=0)
    src, dst, n = copies[copy].unbind(1)
    slot = torch.arange(page, device=CUDA)
    i, t = (slot < n[:, None]).nonzero(as_tuple=True)
    for name in ("k_cache", "v_cache"):
        raw = _raw(s[name])
        raw[dst[i], :, t] = raw[src[i], :, t]
    return {"table": table.int(), "refs": uses.int(), "copies": copies.int(), "short": short.int().view(1),
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(cache, block_table, scale):
    """[B, Hkv, pages * page, d] in 32 bits."""
    x = _raw(cache)[block_table.long().clamp(min=0)].view(cache.dtype)
    x = x.transpose(1, 2).float()
    x = x if scale is None else x * scale[:, None, None, None]
    return x.flatten(2, 3)


def _attend(s):
    c = s["case"]
    B, T, Hq, Hkv, w = c["B"], c["T"], c["Hq"], c["Hkv"], c["window"]
    G = Hq // Hkv
    # each draft's ancestors, itself among them; none for padding
    parents = s["parents"].long()
    up = torch.zeros(B, T, T, dtype=torch.bool, device=CUDA)
    row = torch.arange(B, device=CUDA)
    for l in range(T):
        p = parents[:, l]
        above = up[row, p.clamp(min=0)]
        there = (p == -1) | ((p >= 0) & above.any(1))
        up[:, l] = above & (p >= 0)[:, None] & there[:, None]
        up[:, l, l] = there
    depth = up.sum(2) - 1
    k = _gathered(s["k_cache"], s["block_table"], s["k_scale"])
    x = s["q"].float().view(B, Hkv, G * T, c["dqk"]) @ k.transpose(2, 3)
    x = x.view(B, Hkv, G, T, -1) * s["scale"]
    if c["softcap"] > 0:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    ctx = (s["seq_lens"].long() - T)[:, None]
    j = torch.arange(x.shape[-1], device=CUDA)
    see = (j < ctx)[:, None] & (depth >= 0)[:, :, None]
    if w >= 0:
        see = see & ((ctx + depth)[:, :, None] - j <= w)
        up = up & (depth[:, :, None] - depth[:, None] <= w)
    slot = j - ctx  # [B, keys]
    see = see | (up.gather(2, slot.clamp(0, T - 1)[:, None].expand(B, T, -1)) & ((slot >= 0) & (slot < T))[:, None])
    x = x.masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    z = e.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["block_table"], s["v_scale"])
    o = (e.flatten(2, 3) @ v).view(B, Hkv, G, T, -1) / z.masked_fill(z == 0, 1.0)
    return o.bfloat16().view(B, Hq, T, -1), (m + torch.log(z)).view(B, Hq, T)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "tree":
        return _exact_tree(c, s)
    if c["op"] == "compact":
        return _exact_compact(c, s)
    if c["op"] == "fork":
        return _exact_fork(c, s)

    def turn(x, sign):
        y = x.double().clone()
        t = s["table"].double()
        for i, a in enumerate(s["axes"]):
            m = c["offset"] + (2 * i if c["interleaved"] else i)
            n = m + 1 if c["interleaved"] else m + c["rot"] // 2
            at = s["rot_positions"][a].long()
            z = torch.complex(x[..., m].double(), x[..., n].double())
            z = z * torch.complex(t[:, i][at], sign * t[:, c["rot"] // 2 + i][at])[:, None]
            y[..., m], y[..., n] = z.real, z.imag
        return y

    if c["op"] == "rope":
        return tuple(turn(s[x], -1.0 if c["backward"] else 1.0) for x in ("q", "k"))
    q, k = turn(s["q"], 1.0), turn(s["k"], 1.0)
    out = {"q": q, "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    if c["k_out"]:
        out["k"] = k
    page, bt = c["page"], s["block_table"].tolist()
    at, rows, cols, slots = [], [], [], []
    for b, line in enumerate(s["positions"].tolist()):
        for l, p in enumerate(line):
            rows.append(b)
            cols.append(l)
            slots.append(p % page)
            at.append(bt[b][p // page])
    at, rows, cols, slots = (torch.tensor(x, device=CUDA) for x in (at, rows, cols, slots))
    for name, x, scale in (("k_cache", k, s["k_scale"]), ("v_cache", s["v"].double(), s["v_scale"])):
        for h in range(c["Hkv"]):
            y = x[rows, h, cols]
            if scale is not None:
                y = (y / scale[h].double()).clamp(-E4M3_MAX, E4M3_MAX)
            out[name][at, h, slots] = y
    return out


def _exact_tree(c, s):
    B, T, Hq, Hkv, page, w = c["B"], c["T"], c["Hq"], c["Hkv"], c["page"], c["window"]
    G = Hq // Hkv
    out = torch.zeros((B, Hq, T, c["dv"]), dtype=torch.float64, device=CUDA)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=CUDA)
    trees = s["parents"].tolist()
    for b, n in enumerate(s["seq_lens"].tolist()):
        ctx = n - T
        see = torch.zeros(T, n, dtype=torch.bool)
        for l in range(T):
            path, at = [], l
            while at >= 0:
                path.append(at)
                at = trees[b][at]
            if at < -1:
                continue  # padding
            p = ctx + len(path) - 1
            see[l, (0 if w < 0 else max(0, p - w)):ctx] = True
            for up, i in enumerate(path):
                if w < 0 or up <= w:
                    see[l, ctx + i] = True
        see = see.to(CUDA)
        pages = s["block_table"][b, :-(-n // page)].long()
        some = see.any(1)
        for h in range(Hkv):
            kv = []
            for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
                x = _raw(cache)[pages, h].view(cache.dtype).double().reshape(-1, cache.shape[3])[:n]
                kv.append(x if scale is None else x * scale[h].double())
            q = s["q"][b, h * G:(h + 1) * G].double()
            t = torch.einsum("gld,kd->glk", q, kv[0]) * s["scale"]
            if c["softcap"] > 0:
                t = c["softcap"] * torch.tanh(t / c["softcap"])
            t = t.masked_fill(~see, -math.inf)[:, some]
            z = torch.logsumexp(t, -1)
            lse[b, h * G:(h + 1) * G, some] = z
            out[b, h * G:(h + 1) * G, some] = torch.einsum("glk,kd->gld", (t - z[..., None]).exp(), kv[1])
    return out, lse


def _exact_compact(c, s):
    page, bt, starts = c["page"], s["block_table"].tolist(), s["start"].tolist()
    a, i, b, j = [], [], [], []
    for r, line in enumerate(s["src"].tolist()):
        for m, p in enumerate(line):
            if p < 0:
                break
            d = starts[r] + m
            a.append(bt[r][p // page])
            i.append(p % page)
            b.append(bt[r][d // page])
            j.append(d % page)
    a, i, b, j = (torch.tensor(x, device=CUDA) for x in (a, i, b, j))
    out = {}
    for name in ("k_cache", "v_cache"):
        x = s[name].double()
        x[b, :, j] = x[a, :, i].clone()
        out[name] = x
    return out


def _exact_fork(c, s):
    page, old, refs = c["page"], s["block_table"].tolist(), s["refs"].tolist()
    parents, keep, room = (s[x].tolist() for x in ("parents", "keep", "room"))
    M, P = len(parents), len(old[0])
    free = [p for p, n in enumerate(refs) if n == 0]
    uses = list(refs)
    for line in old:
        for p in line:
            if p >= 0:
                uses[p] -= 1
    whole, part = {}, {}
    for i in range(M):
        for j in range(-(-keep[i] // page)):
            p = old[parents[i]][j]
            uses[p] += 1
            (whole if (j + 1) * page <= keep[i] else part).setdefault(p, []).append(i)
    table = [[-1] * P for _ in range(M)]
    copies = [[-1, -1, 0] for _ in range(M)]
    given = 0
    for i in range(M):
        for j in range(-(-max(keep[i], room[i]) // page)):
            p = old[parents[i]][j] if j * page < keep[i] else -1
            mine = p >= 0 and ((j + 1) * page <= keep[i] or (uses[p] == len(part[p]) and part[p][0] == i))
            if mine:
                table[i][j] = p
                continue
            table[i][j] = free[given] if given < len(free) else -1
            given += 1
            if p >= 0 and table[i][j] >= 0:
                copies[i] = [p, table[i][j], keep[i] % page]
    count = list(refs)
    for line, sign in [(x, -1) for x in old] + [(x, 1) for x in table]:
        for p in line:
            if p >= 0:
                count[p] += sign
    out = {name: torch.tensor(x, dtype=torch.int32, device=CUDA) for name, x in
           (("table", table), ("refs", count), ("copies", copies), ("short", [max(0, given - len(free))]))}
    for name in ("k_cache", "v_cache"):
        x = s[name].double()
        for a, b, n in copies:
            if n:
                x[b, :, :n] = x[a, :, :n].clone()
        out[name] = x
    return out
