"""rope_axes_fwd / rope_axes_bwd and paged_append_axes on the GPU against the
float64 reference.  Bounds as for the calls with one axis: a rotated value is
rounded once (2^-8 of it at most) after two fp32 products and a sum of at most
|a| + |b|, off by less than 4 * 2^-24 (|a| + |b|); e4m3 by half a step of the
format, with 8 * 2^-24 of the value for a rounding border crossed before it."""
import numpy as np
import pytest
import torch

import workloads
from oracle import drafting_ref as ref
from oracle import serving_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def splash():
    from block_sparse_flash_gb300 import build as b
    b.build()
    import block_sparse_flash_gb300 as m
    return m


def host(t):
    return t.double().cpu().numpy()


def room(exact, x):
    """Of a rotated row: (|a| + |b|) is below twice the row's largest element."""
    return 2.0 ** -8 * np.abs(exact) + 8 * 2.0 ** -24 * np.abs(host(x)).max(-1, keepdims=True)


CASES = [  # B, Hq, Hkv, L, d, rot, offset, interleaved, sections, cycled
    (1, 1, 1, 1, 16, 16, 0, False, (8,), False),
    (2, 3, 1, 37, 64, 64, 0, False, (16, 8, 8), False),
    (2, 3, 1, 37, 64, 64, 0, True, (12, 10, 10), True),
    (1, 4, 4, 130, 128, 128, 0, True, (16, 24, 24), False),
    (1, 4, 4, 130, 128, 128, 0, False, (24, 20, 20), True),
    (2, 2, 2, 65, 192, 64, 128, True, (1, 30, 1), False),
    (1, 5, 2, 33, 192, 64, 120, False, (32, 0), False),
    (3, 2, 1, 7, 96, 32, 8, True, (4, 4, 4, 4), False),
    (1, 2, 2, 19, 512, 512, 0, False, (64, 64, 64, 64), True),
    (1, 33, 3, 3, 48, 48, 0, False, (5, 9, 3, 7), False),
    (2, 8, 2, 1000, 128, 64, 64, False, (11, 10, 11), False),
]


def make_positions(A, B, L, rows, seed):
    pos = torch.randint(-2, rows, (A, B, L), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    pos[:, 0, 0] = rows - 1
    return pos


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_axes_match_the_reference(splash, case, inverse):
    B, Hq, Hkv, L, d, rot, offset, inter, sections, cycled = case
    q, k = (workloads.normal_bf16((B, h, L, d), 1 + i).cuda() for i, h in enumerate((Hq, Hkv)))
    table, axes = splash.rope_table(2 * L + 3, rot), splash.rope_axis_map(sections, cycled)
    pos = make_positions(len(sections), B, L, 2 * L + 3, 3)
    f = splash.rope_axes_bwd if inverse else splash.rope_axes_fwd
    got = f(q, k, pos.cuda(), table, axes, offset, inter)
    splash.check_device_error()
    still = [*range(offset), *range(offset + rot, d)]
    for y, x in zip(got, (q, k)):
        exact = ref.rope_axes(host(x), pos.numpy(), host(table), axes, offset, inter, inverse)
        assert (np.abs(host(y) - exact) <= room(exact, x)).all()
        assert torch.equal(y[..., still], x[..., still])
        # pairs without a rotation are left as they are
        for i, a in enumerate(axes):
            m = offset + (2 * i if inter else i)
            for e in (m, m + (1 if inter else rot // 2)):
                off = (pos[a] < 0).cuda()[:, None].expand(B, x.shape[1], L)
                assert torch.equal(y[..., e][off], x[..., e][off])
    q1, none = f(q, None, pos.cuda(), table, axes, rot_offset=offset, interleaved=inter)
    assert none is None and torch.equal(q1, got[0])


def test_equal_axes_are_the_plain_rotation(splash):
    B, L, H, d = 2, 77, 4, 128
    q = workloads.normal_bf16((B, H, L, d), 4).cuda()
    table = splash.rope_table(200, d)
    pos = torch.randint(-1, 200, (B, L), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
    want, _ = splash.rope_fwd(q, None, pos, table)
    for sections, cycled in (((16, 24, 24), False), ((22, 21, 21), True), ((7, 7, 50), False)):
        axes = splash.rope_axis_map(sections, cycled)
        got, _ = splash.rope_axes_fwd(q, None, pos.expand(3, B, L), table, axes)  # (a stride of 0 between the axes)
        assert torch.equal(got, want)
    splash.check_device_error()


def test_strided_views_and_in_place(splash):
    B, L, Hq, Hkv, d = 2, 45, 6, 2, 128
    x = workloads.normal_bf16((B, L, Hq + 2 * Hkv, d), 6).cuda()
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
    table, axes = splash.rope_table(L, d), splash.rope_axis_map((16, 24, 24))
    pos = make_positions(3, B, L, L, 7).cuda()
    want = splash.rope_axes_fwd(q.contiguous(), k.contiguous(), pos, table, axes)
    wide = torch.zeros(B, 3, L + 5, dtype=torch.int32, device="cuda")  # positions as a view
    wide[:, :, 2:2 + L] = pos.transpose(0, 1)
    before = x.clone()
    got = splash.rope_axes_fwd(q, k, wide.transpose(0, 1)[:, :, 2:2 + L], table, axes, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(x[:, :, Hq + Hkv:], before[:, :, Hq + Hkv:])
    splash.check_device_error()


@pytest.mark.parametrize("sections, cycled", [((16, 8, 8), False), ((11, 11, 10), True)])
def test_positions_without_a_rotation_are_reported(splash, sections, cycled):
    q = workloads.normal_bf16((1, 2, 3, 64), 8).cuda()
    table, axes = splash.rope_table(8, 64), splash.rope_axis_map(sections, cycled)
    pos = torch.full((3, 1, 3), 3, dtype=torch.int32)
    good, _ = splash.rope_axes_fwd(q, None, pos.cuda(), table, axes)
    assert splash.last_device_error() == 0
    pos[1, 0, 1], pos[2, 0, 2] = 8, 2 ** 31 - 1
    got, _ = splash.rope_axes_fwd(q, None, pos.cuda(), table, axes)
    assert splash.last_device_error() == 7 and splash.last_device_error() == 0
    assert torch.equal(got[:, :, 0], good[:, :, 0])
    for token, axis in ((1, 1), (2, 2)):
        for i, a in enumerate(axes):
            for e in (i, i + 32):
                want = q if a == axis else good
                assert torch.equal(got[0, :, token, e], want[0, :, token, e])


def test_infinities_stay_in_their_pairs(splash):
    q = workloads.normal_bf16((1, 1, 2, 64), 9).cuda()
    table, axes = splash.rope_table(8, 64), splash.rope_axis_map((11, 11, 10), True)
    pos = torch.tensor([[[3, 3]], [[5, -1]], [[7, 7]]], dtype=torch.int32)
    good, _ = splash.rope_axes_fwd(q, None, pos.cuda(), table, axes)
    q[0, 0, :, 1] = float("inf")  # pair 1, of axis 1: the second token does not turn it
    got, _ = splash.rope_axes_fwd(q, None, pos.cuda(), table, axes)
    assert torch.isinf(got[0, 0, 1, 1]) and got[0, 0, 1, 33] == q[0, 0, 1, 33]
    others = [e for e in range(64) if e not in (1, 33)]
    assert torch.equal(got[..., others], good[..., others]) and not torch.isfinite(got[0, 0, 0, [1, 33]]).any()


@pytest.mark.parametrize("sections, cycled", [((16, 8, 8), False), ((11, 11, 10), True)])
def test_gradient_against_differences(splash, sections, cycled):
    """<g, R x> is linear in x: its difference along e is <R^T g, e>.  Both sides
    carry bf16 roundings of their results, 2^-8 of each product."""
    B, H, L, d = 1, 2, 9, 64
    table, axes = splash.rope_table(L, d), splash.rope_axis_map(sections, cycled)
    pos = make_positions(3, B, L, L, 10).cuda()
    g, e = (workloads.normal_bf16((B, H, L, d), s).cuda() for s in (11, 12))
    gx, _ = splash.rope_axes_bwd(g, None, pos, table, axes, 0, True)
    re, _ = splash.rope_axes_fwd(e, None, pos, table, axes, 0, True)
    a, b = g.double() * re.double(), gx.double() * e.double()
    assert abs((a.sum() - b.sum()).item()) <= 2.0 ** -8 * (a.abs().sum() + b.abs().sum()).item()


APPENDS = [  # B, L, Hq, Hkv, dqk, dv, page, kind, layout, rot, offset, interleaved, sections, cycled
    (1, 1, 4, 2, 128, 128, 16, "bf16", "heads", 128, 0, False, (64,), False),
    (5, 16, 8, 2, 128, 128, 16, "e4m3", "tokens", 64, 0, True, (12, 10, 10), True),
    (2, 37, 3, 1, 64, 64, 16, "bf16", "tokens", 64, 0, False, (16, 8, 8), False),
    (2, 70, 2, 2, 192, 128, 64, "e4m3", "heads", 64, 128, True, (8, 16, 8), False),
    (1, 33, 2, 2, 64, 96, 32, "bf16", "heads", 32, 16, True, (3, 4, 5, 4), False),
    (3, 9, 0, 4, 16, 16, 1024, "e4m3", "heads", 16, 0, False, (8,), False),
]


@pytest.mark.parametrize("case", APPENDS, ids=str)
def test_append_axes_match_the_reference(splash, case):
    B, L, Hq, Hkv, dqk, dv, page, kind, layout, rot, offset, inter, sections, cycled = case
    g = torch.Generator().manual_seed(21)
    per = -(-(L + 3 * page) // page)
    pages = 2 * B * per
    bt = torch.full((B, per + 1), -7, dtype=torch.int32)
    bt[:, :per] = torch.randperm(pages, generator=g)[:B * per].view(B, per)
    start = torch.randint(0, 3 * page - 1, (B, 1), generator=g)
    slots = (start + torch.arange(L)).to(torch.int32)
    if L > 4:
        slots[0, 2] = -1  # padding inside and at the end
        slots[-1, -2:] = -5
    rows = 40
    pos = make_positions(len(sections), B, L, rows, 22)
    k, v = (workloads.normal_bf16((B, Hkv, L, d), 23 + i).cuda() for i, d in enumerate((dqk, dv)))
    q = workloads.normal_bf16((B, Hq, L, dqk), 25).cuda() if Hq else None
    table, axes = splash.rope_table(rows, rot), splash.rope_axis_map(sections, cycled)
    caches = []
    for i, d in enumerate((dqk, dv)):
        t = workloads.normal_bf16((pages, page, Hkv, d) if layout == "tokens" else (pages, Hkv, page, d), 26 + i).cuda()
        t = t.to(torch.float8_e4m3fn) if kind == "e4m3" else t
        caches.append(t.transpose(1, 2) if layout == "tokens" else t)
    scales = [torch.linspace(a, b, Hkv, device="cuda") if kind == "e4m3" else None for a, b in ((0.011, 0.03), (0.02, 0.007))]
    old = [host(c) for c in caches]
    k_out = torch.empty_like(k)
    qo, ko = splash.paged_append_axes(k, v, *caches, bt.cuda(), slots.cuda(), pos.cuda(), table, axes, q=q,
                                      rot_offset=offset, interleaved=inter, k_scale=scales[0], v_scale=scales[1], k_out=k_out)
    splash.check_device_error()
    assert ko is k_out and (q is not None or qo is None)

    def turned(x):
        return ref.rope_axes(host(x), pos.numpy(), host(table), axes, offset, inter)
    for got, x in ((qo, q), (ko, k)):
        if x is not None:
            exact = turned(x)
            assert (np.abs(host(got) - exact) <= room(exact, x)).all()
    for cache, before, x, raw, scale in zip(caches, old, (turned(k), host(v)), (k, v), scales):
        s = None if scale is None else host(scale)
        exact, written = serving_ref.append(before, x, bt.numpy(), slots.numpy(), scale=s)
        got = host(cache).transpose(0, 2, 1, 3)
        assert np.array_equal(got[~written], before.transpose(0, 2, 1, 3)[~written])
        got, want = got[written], exact.transpose(0, 2, 1, 3)[written]
        slop = 8 * 2.0 ** -24 * np.abs(host(raw)).max() / (1 if s is None else s.min())
        half = 2.0 ** -8 * np.abs(want) if s is None else 0.5 * serving_ref.e4m3_step(np.abs(want) + slop)
        assert (np.abs(got - want) <= half + slop).all() and got.shape[0] == int((slots >= 0).sum())


def test_append_with_the_slots_as_rotations_is_the_plain_one(splash):
    B, L, Hq, Hkv, d, page = 2, 20, 4, 2, 128, 16
    x = workloads.normal_bf16((B, L, Hq + 2 * Hkv, d), 31).cuda()
    q, k, v = (y.transpose(1, 2) for y in x.split((Hq, Hkv, Hkv), 2))
    pos = (torch.tensor([[3], [14]]) + torch.arange(L)).to(torch.int32).cuda()
    bt = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    table = splash.rope_table(60, d)
    a, b = (torch.zeros(2, 6, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qa, _ = splash.paged_append(k, v, a[0], a[1], bt, pos, q=q, table=table)
    qb, _ = splash.paged_append_axes(k, v, b[0], b[1], bt, pos, pos[None], table, splash.rope_axis_map([d // 2]), q=q)
    assert torch.equal(qa, qb) and torch.equal(a, b)
    # packed sequences, and a rotation that the table does not have: reported, not stored
    seq = torch.tensor([[0] * 12 + [1] * 8], dtype=torch.int32, device="cuda")
    slots = torch.cat((torch.arange(12), torch.arange(8))).to(torch.int32)[None].cuda()
    turn = torch.full((1, 1, L), 5, dtype=torch.int32, device="cuda")
    turn[0, 0, 3] = 60
    b.zero_()
    splash.paged_append_axes(k[:1], v[:1], b[0], b[1], bt, slots, turn, table, splash.rope_axis_map([d // 2]), seq_ids=seq)
    assert splash.last_device_error() == 7
    for i in range(L):
        s, p = int(seq[0, i]), int(slots[0, i])
        stored = b[1][bt[s, p // page], :, p % page]
        assert torch.equal(stored, torch.zeros_like(stored) if i == 3 else v[0, :, i])
