"""paged_append on the GPU against the float64 reference: what it writes, what
it leaves, and what it reports.

Bounds: a rotated value as in test_gpu_rope (2^-8 relative for bf16, fp32
products before it).  e4m3: half a step of the format at the stored value,
plus the fp32 roundings of the rotation and the division, which can carry a
value across a rounding border by 8 * 2^-24 of it."""
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


def host(t):
    return t.double().cpu().numpy()


def make_cache(pages, Hkv, page, d, kind, layout, seed):
    shape = (pages, page, Hkv, d) if layout == "tokens" else (pages, Hkv, page, d)
    t = workloads.normal_bf16(shape, seed).cuda()
    if kind == "e4m3":
        t = t.to(torch.float8_e4m3fn)
    return t.transpose(1, 2) if layout == "tokens" else t


def bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16)


CASES = [
    # B, L, Hq, Hkv, dqk, dv, page, kind, layout, rot, offset, interleaved
    (1, 1, 4, 2, 128, 128, 16, "bf16", "heads", 128, 0, False),
    (5, 1, 8, 2, 128, 128, 16, "e4m3", "tokens", 64, 0, True),
    (2, 37, 3, 1, 64, 64, 16, "bf16", "tokens", 64, 0, False),
    (2, 70, 2, 2, 192, 128, 64, "e4m3", "heads", 64, 128, True),
    (1, 33, 2, 2, 64, 96, 32, "bf16", "heads", 32, 16, True),
    (3, 9, 0, 4, 16, 16, 1024, "e4m3", "heads", 16, 0, False),
    (2, 5, 0, 1, 128, 64, 128, "bf16", "heads", 0, 0, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_append_matches_the_reference(splash, case):
    B, L, Hq, Hkv, dqk, dv, page, kind, layout, rot, offset, inter = case
    g = torch.Generator().manual_seed(11)
    per = -(-(L + 3 * page) // page)
    pages = 2 * B * per
    bt = torch.full((B, per + 1), -7, dtype=torch.int32)  # the last column is never used
    bt[:, :per] = torch.randperm(pages, generator=g)[:B * per].view(B, per)
    start = torch.randint(0, 3 * page - 1, (B, 1), generator=g)
    pos = (start + torch.arange(L)).to(torch.int32)
    if L > 4:
        pos[0, 2] = -1  # padding inside and at the end
        pos[-1, -2:] = -5
    k = workloads.normal_bf16((B, Hkv, L, dqk), 12).cuda()
    v = workloads.normal_bf16((B, Hkv, L, dv), 13).cuda()
    k[0, 0, 0, 3] = 3000.0  # past e4m3's range under the scales below
    q = workloads.normal_bf16((B, Hq, L, dqk), 14).cuda() if Hq else None
    table = splash.rope_table(5 * page + L, rot) if rot else None
    kc, vc = (make_cache(pages, Hkv, page, d, kind, layout, 15 + i) for i, d in enumerate((dqk, dv)))
    scales = [None, None]
    if kind == "e4m3":
        scales = [torch.linspace(0.011, 0.03, Hkv, device="cuda"), torch.linspace(0.02, 0.007, Hkv, device="cuda")]
    k0, v0 = kc.clone(), vc.clone()
    k_out = torch.empty_like(k)
    qo, ko = splash.paged_append(k, v, kc, vc, bt.cuda(), pos.cuda(), q=q, table=table, rot_offset=offset,
                                 interleaved=inter, k_scale=scales[0], v_scale=scales[1], k_out=k_out)
    splash.check_device_error()
    assert ko is k_out
    if q is None:
        assert qo is None

    def turned(x):
        return ref.rope(host(x), pos.numpy(), table.cpu().numpy(), offset, inter) if rot else host(x)
    for got, x in ((qo, q), (ko, k)):
        if x is not None:
            exact = turned(x)
            big = np.abs(host(x)).max(-1, keepdims=True)
            assert (np.abs(host(got) - exact) <= 2.0 ** -8 * np.abs(exact) + 8 * 2.0 ** -24 * big).all()
            pad = pos < 0
            assert torch.equal(got.transpose(1, 2)[pad.cuda()], x.transpose(1, 2)[pad.cuda()])
    for cache, old, x, raw, scale in ((kc, k0, turned(k), k, scales[0]), (vc, v0, host(v), v, scales[1])):
        s = None if scale is None else scale.double().cpu().numpy()
        exact, written = ref.append(host(old), x, bt.numpy(), pos.numpy(), scale=s)
        w = torch.from_numpy(written).cuda()
        assert torch.equal(bits(cache.transpose(1, 2))[~w], bits(old.transpose(1, 2))[~w])  # everything else as it was
        got, want = host(cache).transpose(0, 2, 1, 3)[written], exact.transpose(0, 2, 1, 3)[written]
        slop = 8 * 2.0 ** -24 * np.abs(host(raw)).max() / (1 if s is None else s.min())
        half = 2.0 ** -8 * np.abs(want) if s is None else 0.5 * ref.e4m3_step(np.abs(want) + slop)
        if s is None and (cache is vc or not rot):
            assert np.array_equal(got, want)
        assert (np.abs(got - want) <= half + slop).all()
        assert got.shape[0] == int((pos >= 0).sum())


def test_packed_sequences(splash):
    """A row of documents appended at once equals each appended alone."""
    lens, page, Hkv, d = [5, 1, 40, 16], 16, 2, 64
    L = sum(lens)
    k, v = (workloads.normal_bf16((1, Hkv, L, d), s).cuda() for s in (21, 22))
    q = workloads.normal_bf16((1, 4, L, d), 23).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])[None].cuda()
    seq = torch.cat([torch.full((n,), i, dtype=torch.int32) for i, n in enumerate(lens)])[None].cuda()
    bt = torch.randperm(12, generator=torch.Generator().manual_seed(24)).view(4, 3).to(torch.int32).cuda()
    table = splash.rope_table(64, d)
    kc, vc = (torch.zeros(12, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k1, v1 = kc.clone(), vc.clone()
    qo, _ = splash.paged_append(k, v, kc, vc, bt, pos, q=q, table=table, seq_ids=seq)
    at = 0
    for i, n in enumerate(lens):
        s = slice(at, at + n)
        qi, _ = splash.paged_append(k[:, :, s], v[:, :, s], k1, v1, bt[i:i + 1], pos[:, s], q=q[:, :, s], table=table)
        assert torch.equal(qi, qo[:, :, s])
        at += n
    assert torch.equal(kc, k1) and torch.equal(vc, v1)
    splash.check_device_error()


def test_strided_inputs_and_in_place_rotation(splash):
    B, L, Hq, Hkv, d, page = 3, 1, 8, 2, 128, 16
    x = workloads.normal_bf16((B, L, Hq + 2 * Hkv, d), 31).cuda()
    q, k, v = (y.transpose(1, 2) for y in x.split((Hq, Hkv, Hkv), 2))
    pos = torch.tensor([[0], [15], [16]], dtype=torch.int32, device="cuda")
    bt = torch.tensor([[3, 1, -1], [2, 5, -1], [4, 0, -1]], dtype=torch.int32, device="cuda")[:, :2]  # a row stride of 3
    table = splash.rope_table(17, d)
    big = torch.zeros(6, 2, Hkv, page, d, dtype=torch.bfloat16, device="cuda")  # K and V of a page side by side
    other = torch.zeros(6, 2, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    want_q, _ = splash.paged_append(k.contiguous(), v.contiguous(), other[:, 0], other[:, 1], bt, pos,
                                    q=q.contiguous(), table=table)
    raw_k = k.clone()
    qo, ko = splash.paged_append(k, v, big[:, 0], big[:, 1], bt, pos, q=q, table=table, q_out=q, k_out=k)
    assert qo is q and ko is k and torch.equal(qo, want_q) and torch.equal(big, other)
    assert torch.equal(k[1, :, 0], big[2, 0, :, 15]) and not torch.equal(k[1], raw_k[1])
    splash.check_device_error()


def test_e4m3_values(splash):
    """Saturation, NaN, ties to even and subnormals of the stored format."""
    vals = [448.0, 464.0, 1e30, -1e30, float("inf"), float("-inf"), 0.0, -0.0, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10,
            3 * 2.0 ** -10, float("nan"), 17.0, 19.0]
    want = [448.0, 448.0, 448.0, -448.0, 448.0, -448.0, 0.0, -0.0, 1.0, 1.25, 2.0 ** -9, 0.0, 2.0 ** -8, float("nan"),
            16.0, 20.0]
    v = torch.tensor(vals).bfloat16().view(1, 1, 1, 16).cuda()
    kc, vc = (torch.zeros(1, 1, 16, 16, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    one = torch.ones(1, device="cuda")
    i0 = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    splash.paged_append(v, v, kc, vc, i0, i0, k_scale=one, v_scale=one)
    for c in (kc, vc):
        got = c[0, 0, 0].float().cpu()
        np.testing.assert_array_equal(got.numpy(), np.float32(want))
        assert torch.signbit(got[7])
    splash.check_device_error()


def test_bad_indices_are_reported_and_touch_nothing(splash):
    page, Hkv, d = 16, 1, 64
    table = splash.rope_table(40, d)
    k = workloads.normal_bf16((1, Hkv, 1, d), 41).cuda()
    kc, vc = (torch.zeros(4, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt = torch.tensor([[0, 1], [4, -1]], dtype=torch.int32, device="cuda")

    def i32(x):
        return torch.tensor([[x]], dtype=torch.int32, device="cuda")
    # (position, sequence): past the row of pages, a page outside the cache on
    # both sides, sequences outside the table, a position past the rotations
    for p, s in ((32, 0), (0, 1), (16, 1), (0, 2), (0, -1), (2 ** 31 - 1, 0), (-2 ** 31, 0)):
        ko = torch.empty_like(k)
        splash.paged_append(k, k, kc, vc, bt, i32(p), table=table, seq_ids=i32(s), k_out=ko)
        assert splash.last_device_error() == (7 if p >= 0 else 0), (p, s)
        assert not kc.any() and not vc.any()
        if 0 <= p < 40:
            assert torch.equal(ko, splash.rope_fwd(k, None, i32(p), table)[0])
        else:
            assert torch.equal(ko, k)
    short = splash.rope_table(8, d)
    splash.paged_append(k, k, kc, vc, bt, i32(8), table=short)
    assert splash.last_device_error() == 7 and not kc.any() and not vc.any()


def test_the_same_row_twice_keeps_one_of_the_two(splash):
    page, Hkv, d = 16, 2, 64
    k = workloads.normal_bf16((1, Hkv, 2, d), 51).cuda()
    kc, vc = (torch.zeros(2, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    pos = torch.full((1, 2), 3, dtype=torch.int32, device="cuda")
    splash.paged_append(k, k, kc, vc, bt, pos)
    splash.check_device_error()
    for c in (kc, vc):
        got = c[0, :, 3]
        assert ((got == k[0, :, 0]) | (got == k[0, :, 1])).all()
        assert not c[1].any() and not c[0, :, 4:].any()
