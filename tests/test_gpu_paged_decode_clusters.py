"""paged_decode's largest clusters on the GPU: 16 CTAs per segment, for every
size of a CTA's shared memory (a cluster that has no room would fail to
launch)."""
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


@pytest.mark.parametrize("Lq", [1, 2])
@pytest.mark.parametrize("rows", [4, 16, 32])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dqk, dv", [(64, 64), (128, 128), (192, 128)])
def test_sixteen_ctas_per_segment(splash, dqk, dv, kind, rows, Lq):
    """One sequence of 2500 keys and one KV head.  Bounds: the probabilities to
    2^-11 of each, the result's rounding 2^-8 of it, the scores (dqk + 8) 2^-23
    of the sum of their products' absolute values."""
    n, page = 2500, 64
    pages = -(-n // page)
    Hq = rows // Lq
    caches = [workloads.normal_bf16((pages, 1, page, d), 800 + i).float() for i, d in enumerate((dqk, dv))]
    scales = [None, None]
    if kind == "e4m3":
        scales = [torch.tensor([0.02], device="cuda"), torch.tensor([0.03], device="cuda")]
        caches = [(x / float(s)).clamp(-448, 448) for x, s in zip(caches, scales)]
    caches = [x.to(torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16).cuda() for x in caches]
    q = workloads.normal_bf16((1, Hq, Lq, dqk), 802).cuda()
    bt = torch.randperm(pages, generator=torch.Generator().manual_seed(4)).to(torch.int32)[None].cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    assert splash.paged_decode_workspace_size(q, *caches, bt) == 0
    o, l = splash.paged_decode(q, *caches, bt, lens, 1 / math.sqrt(dqk), k_scale=scales[0], v_scale=scales[1])
    splash.check_device_error()
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    out, lse, A, reach = ref.decode(f(q), f(caches[0]), f(caches[1]), bt.cpu().numpy(), [n], 1 / math.sqrt(dqk),
                                    k_scale=f(scales[0]), v_scale=f(scales[1]))
    e = (dqk + 8) * 2.0 ** -23 * reach
    room = (2.0 ** -11 + 2 * e[..., None]) * A + 2.0 ** -8 * np.abs(out) + n * 2.0 ** -32 * 14
    assert (np.abs(f(o) - out) <= room).all()
    assert (np.abs(f(l) - lse) <= e + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)).all()
