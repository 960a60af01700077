"""Serving step by step -- a prompt, then its answer token by token and several
at once -- with every step's results at the sharp bounds of each call."""
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


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq, Hkv, dqk, dv, rot, offset, page, cols", [
    (8, 2, 128, 128, 128, 0, 16, 8), (4, 4, 192, 128, 64, 128, 64, 2), (16, 1, 64, 64, 64, 0, 16, 3000)])
def test_every_step_of_an_answer(splash, Hq, Hkv, dqk, dv, rot, offset, page, cols, kind):
    """The cache holds the rotated keys and the values rounded once; a step's
    attention is that of its (rotated) queries over what the cache holds: the
    probabilities to 2^-16 of each (e4m3: 2^-11), the result rounded once,
    2^-8, the scores to (dqk + 8) 2^-23 of the sum of their products'
    absolute values."""
    B, prompt, steps = 2, [50, 33], [1] * 6 + [4, 16]
    total = max(prompt) + sum(steps)
    q, k, v = (workloads.normal_bf16((B, h, total, d), 900 + i).cuda() for i, (h, d) in
               enumerate(((Hq, dqk), (Hkv, dqk), (Hkv, dv))))
    table = splash.rope_table(total, rot)
    per = -(-total // page)
    bt = torch.full((B, max(per, cols)), -1, dtype=torch.int32)
    bt[:, :per] = torch.randperm(B * per, generator=torch.Generator().manual_seed(2)).view(B, per).to(torch.int32)
    bt = bt.cuda()
    dtype = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    kc, vc = (torch.zeros(B * per, Hkv, page, d, device="cuda").to(dtype) for d in (dqk, dv))
    ks, vs = (torch.linspace(a, 2 * a, Hkv, device="cuda") if kind == "e4m3" else None for a in (0.01, 0.02))
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    lens, scale = torch.tensor(prompt, dtype=torch.int32, device="cuda"), 1 / math.sqrt(dqk)
    first = torch.zeros_like(lens)
    u = 2.0 ** -16 if kind == "bf16" else 2.0 ** -11
    for n in [max(prompt)] + steps:
        pos = first[:, None] + torch.arange(n, dtype=torch.int32, device="cuda")
        if n == max(prompt):
            pos[pos >= lens[:, None]] = -1
        at = first.long()
        tok = [torch.stack([x[b, :, at[b]:at[b] + n] for b in range(B)]) for x in (q, k, v)]
        qr, _ = splash.paged_append(tok[1], tok[2], kc, vc, bt, pos, q=tok[0], table=table, rot_offset=offset,
                                    k_scale=ks, v_scale=vs)
        splash.check_device_error()
        p = pos.cpu().numpy()
        exact_k = ref.rope(f(tok[1]), p, f(table), offset)
        for cache, x, s in ((kc, exact_k, f(ks)), (vc, f(tok[2]), f(vs))):
            held = f(cache)
            for b in range(B):
                for i in np.flatnonzero(p[b] >= 0):
                    row = held[bt[b, p[b, i] // page].item(), :, p[b, i] % page]
                    want = x[b, :, i] if s is None else np.clip(x[b, :, i] / s[:, None], -448, 448)
                    room = 2.0 ** -8 * np.abs(want) if s is None else ref.e4m3_step(want) / 2
                    assert (np.abs(row - want) <= room * (1 + 2.0 ** -10) + 2.0 ** -20).all()
        if n <= 16:
            first = first + n
            lens = first
            o, l = splash.paged_decode(qr, kc, vc, bt, lens, scale, k_scale=ks, v_scale=vs)
            splash.check_device_error()
            out, lse, A, reach = ref.decode(f(qr), f(kc), f(vc), bt.cpu().numpy(), lens.cpu().numpy(), scale,
                                            k_scale=f(ks), v_scale=f(vs))
            e = (dqk + 8) * 2.0 ** -23 * reach
            assert (np.abs(f(o) - out) <= (u + 2 * e[..., None]) * A + 2.0 ** -8 * np.abs(out)).all()
            assert (np.abs(f(l) - lse) <= e + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)).all()
        else:
            first = lens
