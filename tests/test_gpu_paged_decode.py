"""paged_decode on the GPU against the float64 reference.

Bounds.  With A = sum_j p_j |v_j| and u the rounding of the probabilities to
the tensor cores' input type (bf16: 2^-8, or 2^-16 with up to 8 rows per KV head,
whose remainder is rounded a second time; e4m3 caches use fp16: 2^-11, and its
smallest step 2^-25 on each of n keys):
  |out - exact| <= (u + 2 e) A + 2^-8 |exact| + n 2^-25 max|v|
  |lse - exact| <= e + 2^-20 + 2^-22 |exact|
where e bounds a score's error: dqk products summed in fp32, (dqk + 8) 2^-23
of the sum of their absolute values, and with a cap 2^-20 of it for tanh."""
import math

import numpy as np
import pytest
import torch

import workloads
from oracle import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def splash():
    from block_sparse_flash_gb300 import build as b
    b.build()
    import block_sparse_flash_gb300 as m
    return m


def make(lens, Lq, Hq, Hkv, dqk, dv, page, kind="bf16", layout="heads", seed=0, spare=3, extra_cols=2):
    """Caches whose unused rows and pages are NaN, a shuffled block table whose
    unused entries point nowhere, and queries."""
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
            x = (x / s[:, None, None]).clamp(-448, 448)  # as append stores it (torch's conversion gives NaN beyond)
        x = x.masked_fill(~used[:, None, :, None], float("nan"))
        x = x.to(torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16).cuda()
        if layout == "tokens":
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        caches.append(x)
    q = workloads.normal_bf16((B, Hq, Lq, dqk), seed + 3).cuda()
    return q, caches[0], caches[1], bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scales[0], scales[1]


def bounds(q, kc, vc, bt, lens, scale, cap=0.0, window=-1, ks=None, vs=None):
    n = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    out, lse, A, reach = ref.decode(n(q), n(kc), n(vc), bt.cpu().numpy(), lens.cpu().numpy(), scale, cap, window,
                                    n(ks), n(vs))
    e = (q.shape[3] + 8) * 2.0 ** -23 * reach + (cap * 2.0 ** -20 if cap > 0 else 0)
    rows = q.shape[1] // kc.shape[1] * q.shape[2]
    u = 2.0 ** -11 if ks is not None else 2.0 ** -16 if rows <= 8 else 2.0 ** -8
    vmax = np.nanmax(np.abs(n(vc))) * (1 if vs is None else n(vs).max())
    small = 0 if ks is None else int(lens.max()) * 2.0 ** -25 * vmax
    return out, lse, (u + 2 * e[..., None]) * A + 2.0 ** -8 * np.abs(out) + small, \
        e + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isinf(lse), 0, lse))


def check(got, want):
    out, lse, room_o, room_l = want
    o, l = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(l), empty) and (o[empty] == 0).all()
    assert np.isfinite(o).all() and np.isfinite(l[~empty]).all()
    assert (np.abs(o - out) <= room_o).all(), float((np.abs(o - out) - room_o).max())
    assert (np.abs(l[~empty] - lse[~empty]) <= room_l[~empty]).all()


CASES = [
    # lens, Lq, Hq, Hkv, dqk, dv, page, kind, layout, window, cap
    ([1], 1, 1, 1, 64, 64, 16, "bf16", "heads", -1, 0.0),
    ([300], 1, 32, 8, 128, 128, 16, "bf16", "heads", -1, 0.0),
    ([0, 1, 15, 16, 17, 63, 64, 65], 1, 4, 2, 128, 128, 16, "bf16", "tokens", -1, 0.0),
    ([0, 1, 15, 16, 17, 63, 64, 65, 129], 1, 8, 2, 128, 128, 32, "e4m3", "heads", -1, 0.0),
    ([5, 0, 2, 3, 200, 1], 4, 6, 2, 64, 64, 16, "bf16", "heads", -1, 0.0),
    ([3, 130, 77], 16, 8, 2, 128, 128, 64, "bf16", "heads", -1, 0.0),
    ([3, 130, 77], 5, 16, 2, 64, 64, 16, "e4m3", "tokens", -1, 0.0),
    ([900, 31], 1, 3, 1, 64, 64, 128, "e4m3", "heads", -1, 30.0),
    ([513, 1000, 20], 1, 4, 4, 192, 128, 64, "bf16", "tokens", -1, 0.0),
    ([513, 64, 20], 2, 4, 4, 192, 128, 16, "e4m3", "heads", -1, 0.0),
    ([700, 100, 33, 5, 0], 1, 4, 1, 128, 128, 16, "bf16", "heads", 40, 5.0),
    ([700, 100, 33, 5, 1], 3, 4, 1, 128, 128, 16, "bf16", "heads", 0, 0.0),
    ([700, 128, 33, 2], 4, 8, 2, 64, 64, 16, "e4m3", "heads", 65, 0.0),
    ([700, 1], 1, 4, 2, 64, 64, 1024, "bf16", "heads", 10 ** 12, 0.0),
    ([150, 70], 1, 48, 1, 64, 64, 16, "bf16", "heads", -1, 0.0),
    ([150, 70], 3, 40, 1, 128, 128, 16, "bf16", "heads", 64, 0.0),
    ([40, 90], 2, 24, 1, 192, 128, 16, "bf16", "heads", -1, 0.0),
    ([4000], 1, 2, 1, 128, 128, 16, "bf16", "heads", -1, 0.0),
    ([2500], 2, 16, 1, 128, 128, 256, "e4m3", "heads", -1, 0.0),
]


@pytest.mark.parametrize("long_rows", [False, True], ids=["short", "long"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_decode_matches_the_reference(splash, case, long_rows):
    """With rows of pages that hold little more than the lengths (a cluster per
    sequence and head), and with rows that allow 40000 keys (the keys are then
    split over the whole GPU)."""
    lens, Lq, Hq, Hkv, dqk, dv, page, kind, layout, window, cap = case
    x = make(lens, Lq, Hq, Hkv, dqk, dv, page, kind, layout, seed=100 + CASES.index(case),
             extra_cols=1 + 40000 // page if long_rows else 0)
    q, kc, vc, bt, n, ks, vs = x
    scale = 1 / math.sqrt(dqk)
    got = splash.paged_decode(q, kc, vc, bt, n, scale, softcap=cap, window_left=window, k_scale=ks, v_scale=vs)
    splash.check_device_error()
    check(got, bounds(q, kc, vc, bt, n, scale, cap, window, ks, vs))
    again = splash.paged_decode(q, kc, vc, bt, n, scale, softcap=cap, window_left=window, k_scale=ks, v_scale=vs)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("long_rows", [False, True], ids=["short", "long"])
@pytest.mark.parametrize("Lq", [1, 2])
@pytest.mark.parametrize("rows", [6, 14, 22, 40])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dqk, dv", [(64, 64), (128, 128), (192, 128)])
def test_every_tile_of_rows(splash, dqk, dv, kind, rows, Lq, long_rows):
    q, kc, vc, bt, n, ks, vs = make([77, 150, 3], Lq, 2 * rows // Lq, 2, dqk, dv, 32, kind, seed=rows + dqk,
                                    extra_cols=1300 if long_rows else 0)
    got = splash.paged_decode(q, kc, vc, bt, n, dqk ** -0.5, k_scale=ks, v_scale=vs)
    splash.check_device_error()
    check(got, bounds(q, kc, vc, bt, n, dqk ** -0.5, 0.0, -1, ks, vs))


@pytest.mark.parametrize("B", [1, 130, 300, 700])
def test_many_sequences_of_mixed_lengths(splash, B):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 200, (B,), generator=g).tolist()
    lens[0] = 1500
    q, kc, vc, bt, n, _, _ = make(lens, 1, 2, 1, 64, 64, 16, seed=7)
    got = splash.paged_decode(q, kc, vc, bt, n, 0.125)
    splash.check_device_error()
    check(got, bounds(q, kc, vc, bt, n, 0.125))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_large_scores(splash, kind):
    """Scores of thousands: the running maximum moves by whole hundreds, and
    queries of very different sizes share a tile."""
    q, kc, vc, bt, n, ks, vs = make([400, 90], 2, 4, 2, 64, 64, 16, kind, seed=60)
    q *= torch.tensor([1e-30, 1.0, 60.0, 3000.0], device="cuda").bfloat16().view(1, 4, 1, 1)
    got = splash.paged_decode(q, kc, vc, bt, n, 1.0, k_scale=ks, v_scale=vs)
    splash.check_device_error()
    check(got, bounds(q, kc, vc, bt, n, 1.0, 0.0, -1, ks, vs))


def test_rows_before_the_window_are_not_read(splash):
    """Pages that have left the window may be gone: their entries point
    nowhere, their rows hold NaN."""
    n, page, window = 500, 16, 100
    q, kc, vc, bt, lens, _, _ = make([n], 2, 4, 2, 128, 128, page, seed=70, extra_cols=100)
    want = bounds(q, kc, vc, bt, lens, 0.1, 0.0, window)
    lo = n - 2 - window  # first key of the earliest query
    for c in range(lo // page):
        kc[bt[0, c].item()] = float("nan")
        vc[bt[0, c].item()] = float("inf")
        bt[0, c] = 1 << 30
    part = bt[0, lo // page].item()
    kc[part, :, :lo % page] = float("nan")
    vc[part, :, :lo % page] = float("nan")
    got = splash.paged_decode(q, kc, vc, bt, lens, 0.1, window_left=window)
    splash.check_device_error()
    check(got, want)


@pytest.mark.parametrize("long_rows", [False, True], ids=["short", "long"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq, Lq, window", [(2, 4, -1), (8, 3, 70), (16, 5, 9), (2, 16, 16)])
def test_values_that_only_some_queries_see(splash, kind, Hq, Lq, window, long_rows):
    """Keys after a query, and keys before its window, do not reach it, NaN
    and infinities among them; a query that sees one has it in its result."""
    n, d = 150, 64
    q, kc, vc, bt, lens, ks, vs = make([n, 40], Lq, Hq, 1, d, d, 16, kind, seed=85,
                                       extra_cols=2600 if long_rows else 1)
    want = bounds(q, kc, vc, bt, lens, 0.125, 0.0, window, ks, vs)
    nan = torch.tensor(float("nan"), device="cuda").to(kc.dtype)
    for b, total in enumerate((n, 40)):  # the newest key: the last query's alone
        at = total - 1
        kc[bt[b, at // 16], :, at % 16] = nan
        vc[bt[b, at // 16], :, at % 16] = nan if kind == "e4m3" else float("-inf")
        if window >= 0 and total - Lq - window >= 0:  # the earliest: the first query's alone
            at = total - Lq - window
            vc[bt[b, at // 16], :, at % 16] = nan
    got = splash.paged_decode(q, kc, vc, bt, lens, 0.125, window_left=window, k_scale=ks, v_scale=vs)
    splash.check_device_error()
    o, l = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    for b, total in enumerate((n, 40)):
        first = 1 if window >= 0 and total - Lq - window >= 0 else 0
        clear = slice(first, Lq - 1)
        assert (np.abs(o - want[0]) <= want[2])[b, :, clear].all() and (np.abs(l - want[1]) <= want[3])[b, :, clear].all()
        assert np.isnan(o[b, :, Lq - 1]).all() and np.isnan(l[b, :, Lq - 1]).all()
        if first:
            assert np.isnan(o[b, :, 0]).all() and (np.abs(l - want[1]) <= want[3])[b, :, 0].all()


def test_strided_queries_shared_pages_and_given_outputs(splash):
    lens, Hq, Hkv, d = [100, 100, 37], 8, 2, 128
    q, kc, vc, bt, n, _, _ = make(lens, 1, Hq, Hkv, d, d, 16, seed=80, extra_cols=2600)
    bt[1, :6] = bt[0, :6]  # a shared prefix
    wide = torch.zeros(3, 1, Hq + 5, d, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 2:2 + Hq] = q.transpose(1, 2)
    view = wide[:, :, 2:2 + Hq].transpose(1, 2)
    kv = torch.stack((kc, vc), 1)  # K and V of a page side by side
    out = torch.full((3, Hq, 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, Hq, 1, device="cuda")
    size = splash.paged_decode_workspace_size(view, kc, vc, bt)
    ws = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    got = splash.paged_decode(view, kv[:, 0], kv[:, 1], bt, n, 0.1, out=out, lse=lse, workspace=ws[:size])
    assert got[0] is out and got[1] is lse
    splash.check_device_error()
    check(got, bounds(q, kc, vc, bt, n, 0.1))
    assert (ws[size:] == 0xA5).all()
    with pytest.raises(splash.SplashError):
        splash.paged_decode(view, kv[:, 0], kv[:, 1], bt, n, 0.1, workspace=ws[:size - 16])


def test_bad_pages_and_lengths_are_reported(splash):
    q, kc, vc, bt, n, _, _ = make([40, 20, 33], 1, 2, 1, 64, 64, 16, seed=90, extra_cols=0)
    good = splash.paged_decode(q, kc, vc, bt, n, 0.125)
    assert splash.last_device_error() == 0
    for entry in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        bad = bt.clone()
        bad[1, 0] = entry
        got = splash.paged_decode(q, kc, vc, bad, n, 0.125)
        assert splash.last_device_error() == 7
        for i in (0, 2):  # the other sequences are not touched by it
            assert torch.equal(got[0][i], good[0][i]) and torch.equal(got[1][i], good[1][i])
        assert torch.isfinite(got[0]).all()
    lens = n.clone()
    lens[1] = -3
    got = splash.paged_decode(q, kc, vc, bt, lens, 0.125)
    assert splash.last_device_error() == 7
    assert not got[0][1].any() and torch.isneginf(got[1][1]).all() and torch.equal(got[0][0], good[0][0])
    lens[1] = 49  # one past the 3 pages of a row; its third page does not exist either
    got = splash.paged_decode(q, kc, vc, bt, lens, 0.125)
    assert splash.last_device_error() == 7 and torch.equal(got[0][2], good[0][2])


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
    q = workloads.normal_bf16((1, Hkv, 1, d), 96).cuda()
    got = splash.paged_decode(q, kc, vc, bt, n, 0.1)
    near = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    want = splash.paged_decode(q, small[0], small[1], near, n, 0.1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k = workloads.normal_bf16((1, Hkv, 1, d), 97).cuda()
    splash.paged_append(k, k, kc, vc, bt, torch.full((1, 1), 1500, dtype=torch.int32, device="cuda"))
    splash.check_device_error()
    assert torch.equal(kc[at[1], :, 1500 - 1024], k[0, :, 0]) and torch.equal(vc[at[1], :, 1500 - 1024], k[0, :, 0])
