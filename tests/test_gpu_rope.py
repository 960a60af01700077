"""rope_fwd / rope_bwd on the GPU against the float64 reference.

Bound: the result is rounded to bf16 once (half a step, 2^-8 of the value at
most); before that, two products and a sum in fp32 of at most |a| + |b| are
off by less than 4 * 2^-24 (|a| + |b|).  Rows and dimensions that are not
rotated are copied bit by bit."""
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


def check(got, x, positions, table, offset, interleaved, inverse):
    exact = ref.rope(x.double().cpu().numpy(), positions.cpu().numpy(), table.cpu().numpy(), offset, interleaved, inverse)
    a = np.abs(x.double().cpu().numpy())
    rot = table.shape[1]
    both = a.copy()  # |a| + |b| of each element's pair
    r = a[..., offset:offset + rot]
    if interleaved:
        both[..., offset:offset + rot] = np.repeat(r[..., 0::2] + r[..., 1::2], 2, -1)
    else:
        half = r[..., :rot // 2] + r[..., rot // 2:]
        both[..., offset:offset + rot] = np.concatenate((half, half), -1)
    err = np.abs(got.double().cpu().numpy() - exact)
    assert (err <= 2.0 ** -8 * np.abs(exact) + 4 * 2.0 ** -24 * both).all(), err.max()
    still = [*range(offset), *range(offset + rot, x.shape[3])]
    assert torch.equal(got[..., still], x[..., still])


CASES = [  # B, Hq, Hkv, L, d, rot, offset, interleaved
    (1, 1, 1, 1, 16, 16, 0, False),
    (2, 3, 1, 37, 64, 64, 0, False),
    (1, 4, 4, 130, 128, 128, 0, True),
    (2, 2, 2, 65, 192, 64, 128, True),
    (1, 5, 2, 33, 192, 64, 120, False),
    (3, 2, 1, 7, 96, 32, 8, True),
    (1, 2, 2, 19, 512, 256, 64, False),
    (1, 33, 3, 3, 48, 48, 0, False),
    (2, 8, 2, 1000, 128, 64, 64, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_the_reference(splash, case, inverse):
    B, Hq, Hkv, L, d, rot, offset, inter = case
    q = workloads.normal_bf16((B, Hq, L, d), 1).cuda()
    k = workloads.normal_bf16((B, Hkv, L, d), 2).cuda()
    table = splash.rope_table(2 * L + 3, rot)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-1, 2 * L + 3, (B, L), generator=g, dtype=torch.int32)
    pos[0, 0] = 2 * L + 2
    f = splash.rope_bwd if inverse else splash.rope_fwd
    qo, ko = f(q, k, pos.cuda(), table, offset, inter)
    splash.check_device_error()
    check(qo, q, pos, table, offset, inter, inverse)
    check(ko, k, pos, table, offset, inter, inverse)
    q1, none = f(q, None, pos.cuda(), table, rot_offset=offset, interleaved=inter)
    assert none is None and torch.equal(q1, qo)


def test_strided_views_shared_positions_and_in_place(splash):
    B, L, Hq, Hkv, d = 2, 45, 6, 2, 128
    x = workloads.normal_bf16((B, L, Hq + 2 * Hkv, d), 5).cuda()
    before = x.clone()
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
    table = splash.rope_table(L, d)
    pos = torch.arange(L, dtype=torch.int32, device="cuda")  # one row for the batch
    qo, ko = splash.rope_fwd(q, k, pos, table)
    both = pos.expand(B, L)
    check(qo, q.contiguous(), both, table, 0, False, False)
    check(ko, k.contiguous(), both, table, 0, False, False)
    got = splash.rope_fwd(q, k, both, table, q_out=q, k_out=k)  # (a batch stride of 0)
    assert got[0] is q and torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(x[:, :, Hq + Hkv:], before[:, :, Hq + Hkv:])
    one = before[:1, :, :1].transpose(1, 2).expand(3, 4, L, d)  # an input that repeats its rows
    out, _ = splash.rope_fwd(one, None, pos, table)
    assert torch.equal(out[2, 3], qo[0, 0])
    with pytest.raises(splash.SplashError):
        splash.rope_fwd(q, None, pos, table, q_out=one[:1, :1].expand(2, Hq, L, d))
    splash.check_device_error()


def test_far_positions_and_odd_values(splash):
    table = splash.rope_table(1 << 20, 64)
    q = workloads.normal_bf16((1, 1, 4, 64), 6).cuda()
    pos = torch.tensor([[(1 << 20) - 1, 524287, 0, -7]], dtype=torch.int32, device="cuda")
    out, _ = splash.rope_fwd(q, None, pos, table)
    check(out, q, pos, table, 0, False, False)
    assert torch.equal(out[:, :, 3], q[:, :, 3])
    # the table itself: 64-bit angles
    p, i = (1 << 20) - 1, 1
    exact = np.cos(p * 10000.0 ** (-2 * i / 64))
    assert abs(table[p, i].item() - exact) <= 2.0 ** -24 + 1e-9
    q[0, 0, 3, 5], q[0, 0, 3, 6] = float("nan"), float("-inf")
    out, _ = splash.rope_fwd(q, None, pos, table)
    assert torch.equal(out.view(torch.int16)[:, :, 3], q.view(torch.int16)[:, :, 3])


def test_a_position_without_a_rotation_is_reported_and_copied(splash):
    q = workloads.normal_bf16((1, 2, 3, 64), 7).cuda()
    table = splash.rope_table(8, 64)
    pos = torch.tensor([[7, 8, 1 << 30]], dtype=torch.int32, device="cuda")
    out, _ = splash.rope_fwd(q, None, pos, table)
    assert splash.last_device_error() == 7 and splash.last_device_error() == 0
    assert torch.equal(out[:, :, 1:], q[:, :, 1:]) and not torch.equal(out[:, :, 0], q[:, :, 0])


def test_gradient_against_differences(splash):
    """<g, R x> is linear in x: its difference along e is <R^T g, e>.  Both
    sides carry bf16 roundings of their results, 2^-8 of each product."""
    B, H, L, d = 1, 2, 9, 64
    table = splash.rope_table(L, 32)
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    x, g, e = (workloads.normal_bf16((B, H, L, d), s).cuda() for s in (8, 9, 10))
    gx, _ = splash.rope_bwd(g, None, pos, table, 16, True)
    re, _ = splash.rope_fwd(e, None, pos, table, 16, True)
    left = (g.double() * re.double()).sum().item()
    right = (gx.double() * e.double()).sum().item()
    room = 2.0 ** -8 * ((g.double() * re.double()).abs().sum() + (gx.double() * e.double()).abs().sum()).item()
    assert abs(left - right) <= room
    up, _ = splash.rope_fwd(x + e, None, pos, table, 16, True)
    down, _ = splash.rope_fwd(x - e, None, pos, table, 16, True)
    diff = (g.double() * (up.double() - down.double())).sum().item() / 2
    # (x + e) and (x - e) are rounded too
    room += 2.0 ** -8 * (g.double().abs() * (up.double().abs() + down.double().abs())).sum().item() * 2
    assert abs(diff - right) <= room
