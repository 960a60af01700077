"""paged_tree_decode on the GPU against the float64 reference.

Bounds, as for paged_decode: with A = sum_j p_j |v_j| and u what the
probabilities lose on their way to the second product (bf16 caches 2^-16, e4m3
2^-11 and fp16's smallest step, 2^-25, on each of n keys):
  |out - exact| <= (u + 2 e) A + 2^-8 |exact| + n 2^-25 max|v|
  |lse - exact| <= e + 2^-20 + 2^-22 |exact|
where e bounds a score's error: dqk products summed in fp32, (dqk + 8) 2^-23 of
the sum of their absolute values, and with a cap 2^-20 of it for tanh."""
import math

import numpy as np
import pytest
import torch

import workloads
from oracle import drafting_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def splash():
    from block_sparse_flash_gb300 import build as b
    b.build()
    import block_sparse_flash_gb300 as m
    return m


def host(t):
    return None if t is None else t.double().cpu().numpy()


def make_trees(B, T, shape, seed):
    """Parents int32 [B, T]: an earlier token, -1 or padding."""
    rng = np.random.default_rng(seed)
    p = np.zeros((B, T), dtype=np.int32)
    for b in range(B):
        tokens = int(rng.integers((T + 1) // 2, T + 1)) if shape == "ragged" else T
        for l in range(T):
            p[b, l] = l - 1 if shape == "chain" else -1 if shape == "roots" else l // 2 - 1 if shape == "binary" else \
                int(rng.integers(-1, l)) if l < tokens else int(rng.integers(-9, -1))
    return torch.from_numpy(p)


def make(lens, T, Hq, Hkv, dqk, dv, page, kind="bf16", layout="heads", shape="ragged", seed=0, spare=3, extra_cols=2):
    """Caches whose unused rows and pages are NaN, a shuffled block table whose
    unused entries point nowhere, queries and trees."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).tolist()
    bt = torch.full((B, max(need + [1]) + extra_cols), -(1 << 30), dtype=torch.int32)
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for c in range(need[b]):
            p = order.pop()
            bt[b, c] = p
            used[p, :min(page, n - c * page)] = True
    caches, scales = [], [None, None]
    for i, d in enumerate((dqk, dv)):
        x = workloads.normal_bf16((pages, Hkv, page, d), seed + 1 + i).float()
        if kind == "e4m3":
            s = torch.linspace(0.01, 0.02, Hkv) * (1 + i)
            scales[i] = s.cuda()
            x = (x / s[:, None, None]).clamp(-448, 448)
        x = x.masked_fill(~used[:, None, :, None], float("nan"))
        x = x.to(torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16).cuda()
        if layout == "tokens":
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        caches.append(x)
    q = workloads.normal_bf16((B, Hq, T, dqk), seed + 3).cuda()
    return dict(q=q, k_cache=caches[0], v_cache=caches[1], block_table=bt.cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32).cuda(), parents=make_trees(B, T, shape, seed).cuda(),
                scale=1 / math.sqrt(dqk), k_scale=scales[0], v_scale=scales[1])


def bounds(x, cap=0.0, window=-1):
    out, lse, A, reach = ref.tree_decode(host(x["q"]), host(x["k_cache"]), host(x["v_cache"]), x["block_table"].cpu().numpy(),
                                         x["seq_lens"].cpu().numpy(), x["parents"].cpu().numpy(), x["scale"], cap, window,
                                         host(x["k_scale"]), host(x["v_scale"]))
    e = (x["q"].shape[3] + 8) * 2.0 ** -23 * reach + (cap * 2.0 ** -20 if cap > 0 else 0)
    small, u = 0, 2.0 ** -16
    if x["k_scale"] is not None:
        u = 2.0 ** -11
        small = int(x["seq_lens"].max()) * 2.0 ** -25 * np.nanmax(np.abs(host(x["v_cache"]))) * host(x["v_scale"]).max()
    return out, lse, (u + 2 * e[..., None]) * A + 2.0 ** -8 * np.abs(out) + small, \
        e + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isinf(lse), 0, lse))


def check(got, want):
    out, lse, room_o, room_l = want
    o, l = host(got[0]), host(got[1])
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(l), empty) and (o[empty] == 0).all()
    assert np.isfinite(o).all() and np.isfinite(l[~empty]).all()
    assert (np.abs(o - out) <= room_o).all(), float((np.abs(o - out) - room_o).max())
    assert (np.abs(l[~empty] - lse[~empty]) <= room_l[~empty]).all()


CASES = [
    # lens, T, Hq, Hkv, dqk, dv, page, kind, layout, shape, window, cap
    ([1], 1, 1, 1, 64, 64, 16, "bf16", "heads", "chain", -1, 0.0),
    ([316], 16, 32, 8, 128, 128, 16, "bf16", "heads", "ragged", -1, 0.0),
    ([0, 5, 15, 16, 17, 63, 64, 65], 5, 4, 2, 128, 128, 16, "bf16", "tokens", "ragged", -1, 0.0),
    ([0, 9, 64, 65, 127, 128, 129], 9, 8, 2, 128, 128, 32, "e4m3", "heads", "ragged", -1, 0.0),
    ([5, 0, 2, 3, 200, 1], 4, 6, 2, 64, 64, 16, "bf16", "heads", "binary", -1, 0.0),
    ([64, 130, 77, 30], 64, 8, 2, 128, 128, 64, "bf16", "heads", "ragged", -1, 0.0),
    ([63, 130, 577], 63, 8, 1, 128, 128, 16, "bf16", "heads", "ragged", -1, 0.0),
    ([63, 130, 577], 33, 3, 1, 64, 64, 16, "e4m3", "tokens", "binary", -1, 0.0),
    ([900, 31], 32, 16, 8, 128, 128, 128, "e4m3", "heads", "ragged", -1, 30.0),
    ([513, 1000, 20], 7, 4, 4, 192, 128, 64, "bf16", "tokens", "ragged", -1, 0.0),
    ([513, 164, 20], 64, 8, 2, 192, 128, 16, "bf16", "heads", "ragged", -1, 0.0),
    ([513, 164, 20], 64, 8, 2, 192, 128, 16, "e4m3", "heads", "ragged", -1, 0.0),
    ([513, 64, 20], 17, 4, 4, 192, 128, 16, "e4m3", "heads", "roots", -1, 0.0),
    ([700, 100, 33, 5, 0], 10, 4, 1, 128, 128, 16, "bf16", "heads", "ragged", 40, 5.0),
    ([700, 100, 33, 5, 1], 30, 4, 1, 128, 128, 16, "bf16", "heads", "ragged", 0, 0.0),
    ([700, 128, 33, 2], 40, 8, 2, 64, 64, 16, "e4m3", "heads", "chain", 65, 0.0),
    ([700, 128, 330], 64, 8, 2, 64, 64, 16, "bf16", "heads", "chain", 20, 0.0),
    ([700, 61], 60, 4, 2, 64, 64, 1024, "bf16", "heads", "ragged", 10 ** 12, 0.0),
    ([150, 70], 50, 24, 2, 64, 64, 16, "bf16", "heads", "ragged", -1, 0.0),
    ([4000], 31, 2, 1, 128, 128, 16, "bf16", "heads", "ragged", -1, 0.0),
    ([2500], 64, 16, 1, 128, 128, 256, "e4m3", "heads", "ragged", -1, 0.0),
    ([300, 90], 64, 9, 1, 128, 128, 32, "bf16", "heads", "roots", -1, 2.0),
]


@pytest.mark.parametrize("long_rows", [False, True], ids=["short", "long"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_tree_decode_matches_the_reference(splash, case, long_rows):
    lens, T, Hq, Hkv, dqk, dv, page, kind, layout, shape, window, cap = case
    x = make(lens, T, Hq, Hkv, dqk, dv, page, kind, layout, shape, seed=100 + CASES.index(case),
             extra_cols=1 + 40000 // page if long_rows else 0)
    got = splash.paged_tree_decode(**x, softcap=cap, window_left=window)
    splash.check_device_error()
    check(got, bounds(x, cap, window))
    again = splash.paged_tree_decode(**x, softcap=cap, window_left=window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("T", [1, 4, 8, 15, 16, 31, 32, 33, 64])
@pytest.mark.parametrize("Hq, Hkv", [(1, 1), (4, 1), (8, 1), (10, 2)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_every_number_of_rows(splash, kind, Hq, Hkv, T):
    for dqk, dv in ((64, 64), (128, 128), (192, 128)):
        x = make([177, 350, T], T, Hq, Hkv, dqk, dv, 32, kind, seed=T + dqk)
        got = splash.paged_tree_decode(**x)
        splash.check_device_error()
        check(got, bounds(x))


@pytest.mark.parametrize("B", [1, 130, 300])
def test_many_sequences_of_mixed_lengths(splash, B):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 200, (B,), generator=g).tolist()
    lens[0] = 1500
    for T, Hq in ((3, 2), (20, 4)):
        x = make(lens, T, Hq, 1, 64, 64, 16, seed=7)
        got = splash.paged_tree_decode(**x)
        splash.check_device_error()
        check(got, bounds(x))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [2, 40])
def test_large_scores(splash, kind, T):
    """Scores of thousands: the running maximum moves by whole hundreds, and
    queries of very different sizes share a tile."""
    x = make([400, 90], T, 4, 2, 64, 64, 16, kind, seed=60)
    x["q"] *= torch.tensor([1e-30, 1.0, 60.0, 3000.0], device="cuda").bfloat16().view(1, 4, 1, 1)
    x["scale"] = 1.0
    got = splash.paged_tree_decode(**x)
    splash.check_device_error()
    check(got, bounds(x))


def test_a_chain_is_the_plain_decode(splash):
    for kind in ("bf16", "e4m3"):
        x = make([700, 100, 33], 16, 8, 2, 128, 128, 16, kind, shape="chain", seed=65)
        want = bounds(x, 0.0, 50)
        got = splash.paged_tree_decode(**x, window_left=50)
        x.pop("parents")
        plain = splash.paged_decode(**x, window_left=50)
        splash.check_device_error()
        assert (np.abs(host(got[0]) - host(plain[0])) <= 2 * want[2]).all()
        assert (np.abs(host(got[1]) - host(plain[1])) <= 2 * want[3]).all()


def test_rows_before_the_window_are_not_read(splash):
    """Pages that have left the window may be gone: their entries point
    nowhere, their rows hold NaN."""
    n, page, window, T = 500, 16, 100, 20
    x = make([n], T, 4, 2, 128, 128, page, shape="chain", seed=70, extra_cols=100)
    want = bounds(x, 0.0, window)
    kc, vc, bt = x["k_cache"], x["v_cache"], x["block_table"]
    lo = n - T - window  # first key of the shallowest token
    for c in range(lo // page):
        kc[bt[0, c].item()] = float("nan")
        vc[bt[0, c].item()] = float("inf")
        bt[0, c] = 1 << 30
    part = bt[0, lo // page].item()
    kc[part, :, :lo % page] = float("nan")
    vc[part, :, :lo % page] = float("nan")
    got = splash.paged_tree_decode(**x, window_left=window)
    splash.check_device_error()
    check(got, want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq, T, window", [(2, 4, -1), (8, 30, -1), (8, 30, 70), (16, 9, 3), (2, 64, 16)])
def test_values_that_only_some_tokens_see(splash, kind, Hq, T, window):
    """A token's key and value reach its descendants alone, NaN and infinities
    among them; so do keys before the window of some."""
    n, d = 250, 64
    x = make([n, 90], T, Hq, 1, d, d, 16, kind, shape="binary", seed=85)
    want = bounds(x, 0.0, window)
    kc, vc, bt, parents = x["k_cache"], x["v_cache"], x["block_table"], x["parents"].cpu().numpy()
    nan = torch.tensor(float("nan"), device="cuda").to(kc.dtype)
    hit = np.zeros((2, T), dtype=bool)   # the value is not finite
    lost = np.zeros((2, T), dtype=bool)  # the score is NaN
    for b, total in enumerate((n, 90)):
        keys = [set(k) for k, _ in ref.tree_keys(parents[b], total, window)]
        def spoil(key, what):
            cache, value = what
            cache[bt[b, key // 16], :, key % 16] = value
            for l in range(T):
                if key in keys[l]:
                    (lost if cache is kc else hit)[b, l] = True
        spoil(total - T + T // 2, (vc, nan if kind == "e4m3" else float("-inf")))
        spoil(total - 1, (kc, nan))
        if window >= 0 and total - T - window > 0:
            spoil(total - T - window, (vc, nan))  # the roots' alone
    got = splash.paged_tree_decode(**x, window_left=window)
    splash.check_device_error()
    o, l = host(got[0]), host(got[1])
    for b in range(2):
        for t in range(T):
            if lost[b, t]:
                assert np.isnan(o[b, :, t]).all() and np.isnan(l[b, :, t]).all()
                continue
            assert (np.abs(l - want[1]) <= want[3])[b, :, t].all()
            if hit[b, t]:
                assert not np.isfinite(o[b, :, t]).any()
            else:
                assert (np.abs(o - want[0]) <= want[2])[b, :, t].all()
    assert hit.any() and not (hit | lost).all()


def test_an_infinite_value_keeps_its_sign(splash):
    """One that every token sees, and one of a tree's token: infinity in both."""
    for T, Hq in ((5, 2), (40, 4)):
        x = make([200], T, Hq, 1, 64, 64, 16, shape="binary", seed=86)
        want = bounds(x)
        bt = x["block_table"]
        x["v_cache"][bt[0, 3], 0, 5, 7] = float("inf")
        at = 200 - T  # the first root
        x["v_cache"][bt[0, at // 16], 0, at % 16, 9] = float("-inf")
        got = splash.paged_tree_decode(**x)
        splash.check_device_error()
        o = host(got[0])
        below = np.array([at in k for k, _ in ref.tree_keys(x["parents"].cpu().numpy()[0], 200)])
        assert (o[0, :, :, 7] == np.inf).all() and (o[0][:, below, 9] == -np.inf).all() and below.any() and not below.all()
        others = [c for c in range(64) if c not in (7, 9)]
        assert (np.abs(o - want[0]) <= want[2])[..., others].all()
        assert (np.abs(o - want[0]) <= want[2])[0][:, ~below, 9].all()


def test_strided_queries_shared_trees_and_given_outputs(splash):
    lens, Hq, Hkv, d, T = [100, 100, 37], 8, 2, 128, 12
    x = make(lens, T, Hq, Hkv, d, d, 16, seed=80, extra_cols=2600)
    bt = x["block_table"]
    bt[1, :5] = bt[0, :5]  # a shared prefix
    x["parents"] = x["parents"][2].contiguous()  # one tree for all
    wide = torch.zeros(3, T, Hq + 5, d, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 2:2 + Hq] = x["q"].transpose(1, 2)
    x["q"] = wide[:, :, 2:2 + Hq].transpose(1, 2)
    kv = torch.stack((x["k_cache"], x["v_cache"]), 1)  # K and V of a page side by side
    x["k_cache"], x["v_cache"] = kv[:, 0], kv[:, 1]
    out = torch.full((3, Hq, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, Hq, T, device="cuda")
    size = splash.paged_tree_decode_workspace_size(x["q"], x["k_cache"], x["v_cache"], bt)
    ws = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    got = splash.paged_tree_decode(**x, out=out, lse=lse, workspace=ws[:size])
    assert got[0] is out and got[1] is lse
    splash.check_device_error()
    check(got, bounds({**x, "parents": x["parents"].expand(3, T)}))
    assert (ws[size:] == 0xA5).all()
    if size:
        with pytest.raises(splash.SplashError):
            splash.paged_tree_decode(**x, workspace=ws[:size - 16])


@pytest.mark.parametrize("T, Hq", [(3, 2), (40, 8)])
def test_what_is_wrong_is_reported(splash, T, Hq):
    x = make([140, 120, 133], T, Hq, 1, 64, 64, 16, shape="binary", seed=90, extra_cols=0)
    good = splash.paged_tree_decode(**x)
    assert splash.last_device_error() == 0

    def others(got):
        return all(torch.equal(got[k][i], good[k][i]) for k in (0, 1) for i in (0, 2))
    for entry in (-1, x["k_cache"].shape[0], 2 ** 31 - 1, -2 ** 31):
        bad = x["block_table"].clone()
        bad[1, 0] = entry
        got = splash.paged_tree_decode(**{**x, "block_table": bad})
        assert splash.last_device_error() == 7 and others(got) and torch.isfinite(got[0]).all()
    want = bounds(x)
    for length in (-3, 10 ** 6):
        lens = x["seq_lens"].clone()
        lens[1] = length
        got = splash.paged_tree_decode(**{**x, "seq_lens": lens})
        assert splash.last_device_error() == 7
        # (other lengths cut the list of steps elsewhere: the others' sums are rounded in another order)
        for i in (0, 2):
            assert (np.abs(host(got[0]) - want[0]) <= want[2])[i].all() and (np.abs(host(got[1]) - want[1]) <= want[3])[i].all()
        if length < 0:
            assert not got[0][1].any() and torch.isneginf(got[1][1]).all()
    for parent in (1, T - 1, T, 2 ** 31 - 1):
        p = x["parents"].clone()
        p[1, 1] = parent
        got = splash.paged_tree_decode(**{**x, "parents": p})
        assert splash.last_device_error() == 7 and others(got)
        assert not got[0][1][:, 1].any() and torch.isneginf(got[1][1][:, 1]).all() and torch.equal(got[0][1][:, 0], good[0][1][:, 0])


def test_offsets_past_32_bits(splash):
    """A cache of more than 2^31 elements (and 2^32 bytes): keys in its last pages."""
    pages, Hkv, page, d = 2100, 8, 1024, 128
    kc = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    at = [pages - 1, pages - 2]
    small = workloads.normal_bf16((2, 2, Hkv, page, d), 95).cuda()
    for i, p in enumerate(at):
        kc[p], vc[p] = small[0, i], small[1, i]
    bt = torch.tensor([at], dtype=torch.int32, device="cuda")
    n = torch.tensor([1500], dtype=torch.int32, device="cuda")
    parents = make_trees(1, 30, "ragged", 3).cuda()
    q = workloads.normal_bf16((1, Hkv, 30, d), 96).cuda()
    got = splash.paged_tree_decode(q, kc, vc, bt, n, parents, 0.1)
    near = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    want = splash.paged_tree_decode(q, small[0], small[1], near, n, parents, 0.1)
    splash.check_device_error()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T, Hq", [(7, 2), (50, 8)])
@pytest.mark.parametrize("extra", [0, 2600], ids=["short", "long"])
def test_outputs_at_any_16_bytes(splash, extra, T, Hq):
    """A result that begins 16 bytes past a multiple of 32, its neighbours untouched."""
    x = make([140, 420, 133], T, Hq, 1, 64, 64, 16, seed=120, extra_cols=extra)
    want = splash.paged_tree_decode(**x)
    n = 3 * Hq * T * 64
    room = torch.full((n + 24,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[8:8 + n].view(3, Hq, T, 64)
    assert out.data_ptr() % 32 == 16
    got = splash.paged_tree_decode(**x, out=out)
    splash.check_device_error()
    assert torch.equal(out, want[0]) and torch.equal(got[1], want[1])
    assert (room[:8] == 7).all() and (room[8 + n:] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T, Hq", [(7, 8), (50, 8)])
def test_heads_and_pages_that_are_one_in_memory(splash, kind, T, Hq):
    """Caches whose heads, or pages, repeat (stride 0); a pool of a single page."""
    heads, d, page = 2, 64, 64
    g = torch.Generator().manual_seed(5)
    for pages, one_head, one_page in ((9, True, False), (9, False, True), (9, True, True), (1, False, False), (1, True, False)):
        base = [torch.randn(1 if one_page else pages, 1 if one_head else heads, page, d, generator=g).bfloat16().cuda() for _ in range(2)]
        x = dict(q=workloads.normal_bf16((2, Hq, T, d), 7).cuda(), scale=0.125, k_scale=None, v_scale=None,
                 block_table=torch.tensor([[i % pages for i in range(4)], [(3 * i + 1) % pages for i in range(4)]], dtype=torch.int32).cuda(),
                 seq_lens=torch.tensor([250, 61], dtype=torch.int32).cuda(), parents=make_trees(2, T, "ragged", 3).cuda())
        if kind == "e4m3":
            base = [b.to(torch.float8_e4m3fn) for b in base]
            x["k_scale"], x["v_scale"] = torch.tensor([0.7, -1.3]).cuda(), torch.tensor([1.0, 0.5]).cuda()
        x["k_cache"], x["v_cache"] = (b.expand(pages, heads, page, d) for b in base)
        got = splash.paged_tree_decode(**x)
        splash.check_device_error()
        check(got, bounds(x))


def test_two_thousand_rows_of_a_head(splash):
    """All of 32 query heads on one KV head, 64 tokens each: eight groups of 256 rows."""
    for lens, extra in (([200, 64, 700], 0), ([1900], 2600)):
        x = make(lens, 64, 32, 1, 128, 128, 16, seed=130, extra_cols=extra)
        got = splash.paged_tree_decode(**x)
        splash.check_device_error()
        check(got, bounds(x))


def test_scales_at_the_ends_of_the_range(splash):
    """The scores' factor would leave fp32's range; keys of zero still score 0, and
    those next to its lower end next to 0."""
    for kind in ("bf16", "e4m3"):
        x = make([90, 30], 9, 4, 2, 64, 64, 16, kind, seed=140)
        want = {}
        x["k_cache"] = torch.zeros_like(x["k_cache"])
        for scale, cap in ((3.4e38, 0.0), (3e38, 1e-3), (1e-38, 0.0)):
            x["scale"] = 1.0  # (the keys are 0: any scale gives the same scores)
            want = bounds(x, cap)
            x["scale"] = scale
            got = splash.paged_tree_decode(**x, softcap=cap)
            splash.check_device_error()
            check(got, want)


FEW = [
    # lens, T, Hq, Hkv, dqk, dv, page, kind, layout, shape, window, cap
    ([0, 3, 15, 16, 17, 40, 300], 16, 2, 2, 128, 128, 16, "bf16", "heads", "ragged", -1, 0.0),
    ([0, 3, 15, 16, 17, 40, 300], 16, 1, 1, 64, 64, 16, "e4m3", "tokens", "binary", -1, 0.0),
    ([700, 100, 33, 5, 0], 10, 2, 2, 128, 128, 16, "bf16", "heads", "chain", 4, 0.0),
    ([700, 100, 33, 5, 0], 16, 2, 2, 64, 64, 32, "bf16", "tokens", "chain", 0, 5.0),
    ([700, 100, 33, 5, 0], 4, 12, 3, 192, 128, 64, "bf16", "heads", "ragged", 33, 0.0),
    ([700, 100, 33, 5, 0], 16, 4, 4, 192, 128, 64, "e4m3", "heads", "chain", 20, 3.0),
    ([700, 1000, 333], 2, 16, 2, 128, 128, 128, "e4m3", "heads", "roots", 500, 0.0),
    ([700, 1000, 333], 3, 10, 2, 128, 128, 16, "bf16", "heads", "ragged", 10 ** 12, 50.0),
    ([1900], 8, 1, 1, 128, 128, 16, "e4m3", "heads", "ragged", -1, 0.0),
    ([1900, 1], 1, 8, 1, 192, 128, 16, "bf16", "heads", "roots", -1, 0.0),
]


@pytest.mark.parametrize("long_rows", [False, True], ids=["short", "long"])
@pytest.mark.parametrize("case", FEW, ids=str)
def test_few_rows(splash, case, long_rows):
    lens, T, Hq, Hkv, dqk, dv, page, kind, layout, shape, window, cap = case
    x = make(lens, T, Hq, Hkv, dqk, dv, page, kind, layout, shape, seed=300 + FEW.index(case),
             extra_cols=1 + 40000 // page if long_rows else 0)
    got = splash.paged_tree_decode(**x, softcap=cap, window_left=window)
    splash.check_device_error()
    check(got, bounds(x, cap, window))
    again = splash.paged_tree_decode(**x, softcap=cap, window_left=window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("value", [2.0 ** 100, 2.0 ** 127, float("inf"), float("nan")])
@pytest.mark.parametrize("T, Hq, window", [(8, 1, -1), (4, 4, -1), (16, 1, 2), (8, 2, 5), (40, 1, -1)])
def test_large_values_stay_with_those_who_see_them(splash, value, T, Hq, window):
    """A token's value, and with a window a key's at its start, far above all others."""
    x = make([230], T, Hq, 1, 64, 64, 16, shape="binary" if window < 0 else "chain", seed=150)
    want = bounds(x, 0.0, window)
    bt, parents = x["block_table"], x["parents"].cpu().numpy()[0]
    at = [230 - T + T // 2] + ([230 - T - window] if window >= 0 else [])
    for key in at:
        x["v_cache"][bt[0, key // 16], :, key % 16] = value
    got = splash.paged_tree_decode(**x, window_left=window)
    splash.check_device_error()
    keys = [set(k) for k, _ in ref.tree_keys(parents, 230, window)]
    blind = np.array([not any(k in seen for k in at) for seen in keys])
    assert blind.any() and not blind.all()
    o, l = host(got[0]), host(got[1])
    assert (np.abs(o - want[0]) <= want[2])[:, :, blind].all() and (np.abs(l - want[1]) <= want[3]).all()
    # (a value of 2^100 and more has a probability of 2^-60 at the least here: far above the others)
    assert not (np.abs(np.nan_to_num(o[:, :, ~blind], nan=np.inf)) < 2.0 ** 30).any()


def test_scales_at_the_ends_of_the_range_few_rows(splash):
    for kind in ("bf16", "e4m3"):
        x = make([90, 30], 5, 4, 2, 64, 64, 16, kind, seed=141)
        x["k_cache"] = torch.zeros_like(x["k_cache"])
        for scale, cap in ((3.4e38, 0.0), (3e38, 1e-3), (1e-38, 0.0)):
            x["scale"] = 1.0  # (the keys are 0: any scale gives the same scores)
            want = bounds(x, cap)
            x["scale"] = scale
            got = splash.paged_tree_decode(**x, softcap=cap)
            splash.check_device_error()
            check(got, want)


@pytest.mark.parametrize("T, G", [(64, 1), (40, 4), (4, 1)])
@pytest.mark.parametrize("window", [2 ** 63 - 1, 2 ** 63 - 64])
def test_a_window_past_every_key_is_none(splash, window, T, G):
    """64 segments in one list: with the largest numbers it is cut as without a window."""
    x = make([200, 64, 130, 70, 0, 65, 500, 300], T, 8 * G, 8, 64, 64, 16, seed=160, extra_cols=2600)
    size = splash.paged_tree_decode_workspace_size(x["q"], x["k_cache"], x["v_cache"], x["block_table"])
    assert size > 0 and size == splash.paged_tree_decode_workspace_size(x["q"], x["k_cache"], x["v_cache"], x["block_table"], window)
    want = splash.paged_tree_decode(**x)
    ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = splash.paged_tree_decode(**x, window_left=window, workspace=ws[:size])
    splash.check_device_error()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (ws[size:] == 0xA5).all()
    check(got, bounds(x))


@pytest.mark.parametrize("kind, value", [("bf16", 1.0), ("bf16", 2.0 ** 60), ("bf16", 2.0 ** 63), ("bf16", 2.0 ** 64), ("e4m3", 448.0)])
@pytest.mark.parametrize("T, Hq, window", [(9, 1, -1), (4, 4, -1), (16, 1, -1), (16, 1, 2), (8, 2, 5), (3, 5, 0), (8, 1, -1), (40, 1, -1), (40, 4, 7)])
def test_nothing_of_a_hidden_value_is_left(splash, T, Hq, window, kind, value):
    """All that a token sees is 0: so is its result, to the last bit, whatever a
    sibling, padding or a key before its window holds."""
    x = make([230, 77], T, Hq, 1, 64, 64, 16, kind, shape="binary" if window < 0 else "chain", seed=151)
    x["parents"][1, T - 1] = -5
    v = x["v_cache"].float()
    v = v.masked_fill(~torch.isnan(v), 0.0)
    bt, parents = x["block_table"], x["parents"].cpu().numpy()
    at = [[230 - T + T // 2] + ([230 - T - window] if window >= 0 else []), [76]]  # (the second one's padding)
    for b in range(2):
        for key in at[b]:
            v[bt[b, key // 16], :, key % 16] = value
    x["v_cache"] = v.to(x["v_cache"].dtype)
    got = splash.paged_tree_decode(**x, window_left=window)
    splash.check_device_error()
    o = host(got[0])
    for b, n in enumerate((230, 77)):
        keys = [set(k) for k, _ in ref.tree_keys(parents[b], n, window)]
        blind = np.array([not any(k in seen for k in at[b]) for seen in keys])
        assert blind.all() if b else blind.any() and not blind.all()
        assert (o[b][:, blind] == 0).all() and (o[b][:, ~blind] > 0).all()


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("T, Hq", [(4, 4), (16, 1), (9, 4), (40, 8)])
def test_small_scales(splash, T, Hq, cap):
    """Factors of the scores below fp32's normal numbers.  They are rounded to multiples of
    2^-149, which with sums of products below 2^128 moves a score by 2^-22 at the most, so that
    the usual bounds hold; masked keys stay masked where a factor would be 0."""
    x = make([190, 70], T, Hq, 1, 64, 64, 16, seed=170)
    large = {**x, "q": x["q"] * 2.0 ** 118, "scale": 2.0 ** -127}  # scores of 0.02
    got = splash.paged_tree_decode(**large, softcap=cap)
    splash.check_device_error()
    check(got, bounds(large, cap))
    x["scale"] = 2.0 ** -149
    got = splash.paged_tree_decode(**x, softcap=cap)
    splash.check_device_error()
    check(got, bounds(x, cap))
    y = make([190, 70], T, Hq, 1, 64, 64, 16, "e4m3", seed=171)
    for k_scale in (2.0 ** -140, 2.0 ** -149):
        y["k_scale"] = torch.full_like(y["k_scale"], k_scale)
        got = splash.paged_tree_decode(**y, softcap=cap)
        splash.check_device_error()
        check(got, bounds(y, cap))


@pytest.mark.parametrize("window", [-1, 100])
def test_many_rows_over_long_block_tables(splash, window):
    """Room for 20 million tokens of each sequence, 512 rows of a KV head."""
    x = make([200, 64, 1, 0, 700, 129, 65, 1100], 64, 64, 8, 64, 64, 1024, seed=180, extra_cols=20000)
    got = splash.paged_tree_decode(**x, window_left=window)
    splash.check_device_error()
    check(got, bounds(x, 0.0, window))
