"""paged_decode on the GPU where the numbers are far from ordinary: soft caps
of any size, one key far above very many, infinite values; and that a result
carries no rounding but its own.  References in float64; the bounds are derived
at each test."""
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


def make(lens, Lq, Hq, Hkv, dqk, dv, page, kind="bf16", cols=0, seed=0):
    """Caches, a shuffled block table of at least `cols` columns, queries."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need), generator=g).tolist()
    bt = torch.full((len(lens), max(need + [cols, 1])), -1, dtype=torch.int32)
    for b, m in enumerate(need):
        for c in range(m):
            bt[b, c] = order.pop()
    caches, scales = [], [None, None]
    for i, d in enumerate((dqk, dv)):
        x = workloads.normal_bf16((max(1, sum(need)), Hkv, page, d), seed + 1 + i).float()
        if kind == "e4m3":
            s = torch.linspace(0.01, 0.02, Hkv) * (1 + i)
            scales[i] = s.cuda()
            x = (x / s[:, None, None]).clamp(-448, 448)
        caches.append(x.to(torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16).cuda())
    q = workloads.normal_bf16((len(lens), Hq, Lq, dqk), seed + 3).cuda()
    return q, caches[0], caches[1], bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scales[0], scales[1]


def reference(x, scale, cap=0.0, window=-1):
    q, kc, vc, bt, lens, ks, vs = (None if t is None else t.cpu() for t in x)
    n = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    return ref.decode(n(q), n(kc), n(vc), bt.numpy(), lens.numpy(), scale, cap, window, n(ks), n(vs))


@pytest.mark.parametrize("kind, Lq, Hq, Hkv, dqk, dv, cols", [
    ("bf16", 1, 4, 2, 64, 64, 0), ("bf16", 1, 4, 2, 128, 128, 2600), ("bf16", 3, 10, 2, 128, 128, 0),
    ("bf16", 2, 24, 2, 192, 128, 2600), ("e4m3", 1, 4, 2, 64, 64, 2600), ("e4m3", 4, 8, 2, 192, 128, 0),
    ("e4m3", 2, 24, 2, 128, 128, 0)])
@pytest.mark.parametrize("cap", [3.0, 50.0, 1e3, 1e4, 1e6])
def test_soft_caps_of_any_size(splash, cap, kind, Lq, Hq, Hkv, dqk, dv, cols):
    """The cap's own error is relative to the score, however large the cap.
    For |t| <= 1/4 the fit of tanh(t)/t is off by 4.8e-7 and four fp32
    operations by 4 * 2^-24; above it 1 - 2 / (1 + e^2t) is off by at most
    3e-7, which is 2^-19.6 of tanh(1/4): 2^-19 |s| bounds both.  The scores
    before it: dqk products summed in fp32, (dqk + 8) 2^-23 of the sum of their
    absolute values (`reach`), which bounds |s| too."""
    x = make([300, 41], Lq, Hq, Hkv, dqk, dv, 16, kind, cols, seed=500)
    scale = 2 / math.sqrt(dqk)
    out, lse, A, reach = reference(x, scale, cap)
    got = splash.paged_decode(*x[:5], scale, softcap=cap, k_scale=x[5], v_scale=x[6])
    splash.check_device_error()
    o, l = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    e = ((dqk + 8) * 2.0 ** -23 + 2.0 ** -19) * reach
    assert (np.abs(l - lse) <= e + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)).all(), np.abs(l - lse).max()
    rows = Hq // Hkv * Lq
    u = 2.0 ** -11 if kind == "e4m3" else 2.0 ** -16 if rows <= 8 else 2.0 ** -8
    assert (np.abs(o - out) <= (u + 2 * e[..., None]) * A + 2.0 ** -8 * np.abs(out) + 300 * 2.0 ** -25 * 12).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("cap", [1e20, 1e30, 2.4e38, 3.4e38])
def test_soft_caps_next_to_the_end_of_fp32(splash, cap, kind):
    """A cap that no score comes near is none: tanh(t) = t in fp32.  Both sides
    differ by the roundings of scale / cap and of cap log2 e, 2^-22 of a score
    below 16 together."""
    x = make([300, 41], 1, 4, 2, 64, 64, 16, kind, seed=520)
    got = splash.paged_decode(*x[:5], 0.125, softcap=cap, k_scale=x[5], v_scale=x[6])
    want = splash.paged_decode(*x[:5], 0.125, k_scale=x[5], v_scale=x[6])
    splash.check_device_error()
    assert (got[1] - want[1]).abs().max().item() <= 16 * 2.0 ** -22 + 2.0 ** -20
    assert (got[0].float() - want[0].float()).abs().max().item() <= 2.0 ** -7 * want[0].float().abs().max().item()


@pytest.mark.parametrize("Hq", [1, 12, 24])
def test_one_key_far_above_very_many(splash, Hq):
    """One key 2^26 times as probable as each of the 2^17 - 1 others of an e4m3
    cache, all in the same warp (as many sequences as the GPU has warps, all on
    the same pages): together the others carry 2^-9 of the result, and it is
    they that have a value.

    Probabilities are fp16 in the second product: 2^-11 of each, and at the
    bottom of its range half a step of 2^-32 of the largest key's, on each of
    n keys.  The scores are exact but for the rounding of ln 2 (2^-24 of 26).
    What remains are the fp32 sums of n terms, n 2^-24 of their value."""
    n, d, page = 1 << 17, 64, 1024
    B = 4 * 2 * torch.cuda.get_device_properties(0).multi_processor_count
    k = torch.zeros(n // page, 1, page, d)
    k[0, 0, 5, 0] = 26.0
    v = torch.zeros_like(k)
    v[..., 1] = 1.0
    v[..., 2] = torch.tensor([1.0, -0.5]).repeat(n // 2).view(-1, 1, page)
    v[0, 0, 5] = 0.0
    x = [t.to(torch.float8_e4m3fn).cuda() for t in (k, v)]
    q = torch.zeros(B, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    bt = torch.arange(n // page, dtype=torch.int32, device="cuda").expand(B, -1)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    out, lse = splash.paged_decode(q, x[0], x[1], bt, lens, math.log(2.0), k_scale=one, v_scale=one)
    splash.check_device_error()
    z = 1 + (n - 1) * 2.0 ** -26
    exact = torch.zeros(d, dtype=torch.float64)
    exact[1] = (n - 1) * 2.0 ** -26 / z
    exact[2] = (n / 2 * 0.5 - (-0.5 if 5 % 2 else 1.0)) * 2.0 ** -26 / z
    room = (2.0 ** -11 + 2.0 ** -8 + n * 2.0 ** -24 + 2.0 ** -18) * exact[1] + n * 2.0 ** -32
    assert (out.double().cpu() - exact).abs().max().item() <= room
    assert (lse.double().cpu() - (26 * math.log(2.0) + math.log(z))).abs().max().item() <= n * 2.0 ** -24 + 2.0 ** -18


@pytest.mark.filterwarnings("ignore:invalid value encountered")  # (the reference's infinity - infinity)
@pytest.mark.parametrize("cols", [0, 2600], ids=["short", "long"])
@pytest.mark.parametrize("Hq, Lq", [(1, 1), (8, 1), (2, 3), (4, 4), (12, 2), (40, 1)])
def test_infinite_values_reach_the_result_as_they_are(splash, Hq, Lq, cols):
    """An infinite value of a finite key: its column of every query that sees
    it is that infinity (every probability is positive), the others are as
    without it; both infinities in one column give NaN."""
    n, d = 150, 64
    x = make([n, 70], Lq, Hq, 1, d, d, 16, cols=cols, seed=600)
    q, kc, vc, bt, lens = x[:5]
    inf = float("inf")

    def put(j, col, value):
        for b in range(2):
            vc[bt[b, j // 16], 0, j % 16, col] = value
    plain = reference(x, 0.125)
    clean = splash.paged_decode(q, kc, vc, bt, lens, 0.125)
    for j in range(66):
        put(j, j % 32, inf if j % 3 else -inf)
    for b, total in enumerate((n, 70)):  # the newest key: the last query's alone
        at = total - 1
        vc[bt[b, at // 16], 0, at % 16, 63] = -inf
    got = splash.paged_decode(q, kc, vc, bt, lens, 0.125)
    splash.check_device_error()
    want = reference(x, 0.125)[0]
    o = got[0].double().cpu().numpy()
    assert np.array_equal(np.isnan(o), np.isnan(want))
    assert np.array_equal(np.isposinf(o), np.isposinf(want)) and np.array_equal(np.isneginf(o), np.isneginf(want))
    fine = np.isfinite(want)
    assert fine[..., 32:63].all() and not fine[..., :32].any()
    assert np.array_equal(o[fine], clean[0].double().cpu().numpy()[fine]) and torch.equal(got[1], clean[1])
    assert np.abs(clean[1].double().cpu().numpy() - plain[1]).max() <= 1e-4


@pytest.mark.parametrize("Hq", [1, 8, 16, 24])
def test_an_infinite_value_of_the_largest_key(splash, Hq):
    """The key whose probability is exactly 1 has infinite values."""
    d, n = 64, 40
    kc = torch.zeros(3, 1, 16, d, dtype=torch.bfloat16, device="cuda")
    vc = workloads.normal_bf16((3, 1, 16, d), 620).cuda()
    kc[1, 0, 4] = 1.0
    vc[1, 0, 4, 0], vc[1, 0, 4, 1] = float("inf"), float("-inf")
    q = torch.ones(1, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
    bt = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    for cols in (3, 2600):
        table = torch.nn.functional.pad(bt, (0, cols - 3), value=-1).contiguous()
        out, lse = splash.paged_decode(q, kc, vc, table, lens, 0.125)
        splash.check_device_error()
        assert torch.isposinf(out[..., 0]).all() and torch.isneginf(out[..., 1]).all()
        assert torch.isfinite(out[..., 2:]).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("cols", [0, 2600], ids=["short", "long"])
@pytest.mark.parametrize("dqk, dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("Lq", [1, 2])
@pytest.mark.parametrize("rows", [6, 14, 22, 40])
def test_every_tile_of_rows_rounds_its_result_once(splash, rows, Lq, dqk, dv, cols):
    """A bf16 cache: the probabilities reach the product to 2^-16 of each
    (cut off to bf16, and the rest in bf16), the result is rounded to bf16, 2^-8
    of it.  Scores as above."""
    x = make([700, 333], Lq, 2 * rows // Lq, 2, dqk, dv, 32, cols=cols // 2, seed=700 + rows + dqk)
    out, lse, A, reach = reference(x, dqk ** -0.5)
    o, l = splash.paged_decode(*x[:5], dqk ** -0.5)
    splash.check_device_error()
    e = (dqk + 8) * 2.0 ** -23 * reach
    off = np.abs(o.double().cpu().numpy() - out)
    assert (off <= (2.0 ** -16 + 2 * e[..., None]) * A + 2.0 ** -8 * np.abs(out)).all(), off.max()
    assert (np.abs(l.double().cpu().numpy() - lse) <= e + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)).all()


@pytest.mark.parametrize("cols", [0, 2600], ids=["short", "long"])
@pytest.mark.parametrize("kind, Hq, d", [("e4m3", 1, 64), ("e4m3", 8, 128), ("bf16", 1, 64), ("bf16", 8, 128), ("bf16", 16, 64),
                                         ("bf16", 40, 128)])
def test_probabilities_whose_errors_add_up(splash, kind, Hq, d, cols):
    """Three keys of probability 1/3 and value 1 for each one of probability 1
    and value -1 (over their sum): the result is nearly 0, and what rounding
    1/3 loses adds up over all keys.  It reaches the product as two parts, to
    2^-16 of it for a bf16 cache and 2^-22 for an e4m3 one.  The scores are one
    fp32 product, ln 3 rounded (2^-24 of it), and exp2 is off by 2^-22: 2^-20
    for all of them and the sums' rounding of n terms of like size, 2^-24 each
    at most and random, below 2^-20 too."""
    n = 700
    k = torch.zeros(44, 1, 16, d)
    v = torch.zeros_like(k)
    j = torch.arange(44 * 16).view(44, 16)
    k[:, 0, :, 0] = (j % 4 == 3).float()
    v[:, 0, :, 1] = torch.where(j % 4 == 3, -1.0, 1.0)
    dtype = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    one = torch.ones(1, device="cuda") if kind == "e4m3" else None
    q = torch.zeros(1, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    bt = torch.arange(44, dtype=torch.int32)[None]
    bt = torch.nn.functional.pad(bt, (0, max(0, cols - 44)), value=-1).cuda()
    scale = float(torch.tensor(math.log(3.0)))
    out, lse = splash.paged_decode(q, k.to(dtype).cuda(), v.to(dtype).cuda(), bt, torch.tensor([n], dtype=torch.int32, device="cuda"),
                                   scale, k_scale=one, v_scale=one)
    splash.check_device_error()
    p = math.exp(-scale)
    exact = (3 * p - 1) / (3 * p + 1)
    room = 2.0 ** -16 if kind == "bf16" else 2.0 ** -22
    o = out.double().cpu()
    assert (o[..., 1] - exact).abs().max().item() <= room + 2.0 ** -19 + 2.0 ** -8 * abs(exact)
    assert not o[..., 2:].any() and not o[..., 0].any()
    assert (lse.double().cpu() - (scale + math.log(n / 4 * (3 * p + 1)))).abs().max().item() <= 2.0 ** -19
