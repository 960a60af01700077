"""The serving calls together and as a program uses them: a training step with
rotated q and k, a prompt and its answer over the paged cache, graph capture
and replay, other streams."""
import math

import numpy as np
import pytest
import torch

import oracle
import workloads
from oracle import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def splash():
    from block_sparse_flash_gb300 import build as b
    b.build()
    import block_sparse_flash_gb300 as m
    return m


def test_training_step_gradients(splash):
    """rope_fwd -> attention_fwd -> attention_bwd -> rope_bwd: the gradients of
    the unrotated q and k against the oracle's, turned back in 64 bits (limit
    as for the backward's own parity: 2e-2 of the norm)."""
    B, Hq, Hkv, L, d = 1, 4, 2, 384, 64
    q, k, v, g = (workloads.normal_bf16((B, h, L, d), 200 + i) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    table = splash.rope_table(L, d)
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    mi = splash.build_mask_info(splash.MaskSpec(True), L, L, 128, 128)
    qr, kr = splash.rope_fwd(q.cuda(), k.cuda(), pos, table)
    vd, gd = v.cuda(), g.cuda()
    out, lse = splash.attention_fwd(qr, kr, vd, mi, 0.125)
    dqr, dkr, dv = splash.attention_bwd(qr, kr, vd, out, lse, gd, mi, 0.125)
    dq, dk = splash.rope_bwd(dqr, dkr, pos, table)
    splash.check_device_error()
    want = oracle.attention_bwd(qr.cpu(), kr.cpu(), v, g, oracle.MaskSpec(True), 0.125, 0.0)
    p = np.arange(L)[None].repeat(B, 0)
    t = table.cpu().numpy()
    for got, grad in ((dq, want["dq"].reshape(B, Hq, L, d)), (dk, want["dk"].reshape(B, Hkv, L, d))):
        exact = ref.rope(grad, p, t, inverse=True)
        err = got.double().cpu().numpy() - exact
        assert np.linalg.norm(err) <= 2e-2 * np.linalg.norm(exact)
    mi.close()


@pytest.mark.parametrize("Hq, Hkv, dqk, dv, rot, offset, page", [(8, 2, 128, 128, 128, 0, 16), (4, 4, 192, 128, 64, 128, 64)])
def test_prompt_then_answer_equals_the_whole_sequence_at_once(splash, Hq, Hkv, dqk, dv, rot, offset, page):
    """Two prompts of different lengths through append + attention_fwd, then
    tokens one by one through append + decode: every answer row equals the
    one-pass attention over the whole sequence.  Both sides round p to bf16
    and the output once: 2 (2^-8 + 2^-8) of sum p |v| <= 4 * 2^-8 max|v|."""
    B, prompt, answer = 2, [50, 33], 20
    top = max(prompt)
    total = top + answer
    q, k, v = (workloads.normal_bf16((B, h, total, d), 300 + i).cuda() for i, (h, d) in
               enumerate(((Hq, dqk), (Hkv, dqk), (Hkv, dv))))
    table = splash.rope_table(total, rot)
    scale = 1 / math.sqrt(dqk)
    per = -(-total // page)
    bt = torch.randperm(B * per, generator=torch.Generator().manual_seed(1)).view(B, per).to(torch.int32).cuda()
    kc = torch.full((B * per, Hkv, page, dqk), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full((B * per, Hkv, page, dv), float("nan"), dtype=torch.bfloat16, device="cuda")
    # the whole sequences at once
    every = torch.arange(total, dtype=torch.int32, device="cuda")
    qr, kr = splash.rope_fwd(q, k, every, table, rot_offset=offset)
    mi = splash.build_mask_info(splash.MaskSpec(True), total, total, 128, 128)
    want, want_lse = splash.attention_fwd(qr, kr, v, mi, scale)
    mi.close()
    room = 4 * 2.0 ** -8 * v.float().abs().max().item()
    # the prompts, padded to the longer one
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    pos = every[:top].expand(B, top).clone()
    pos[pos >= lens[:, None]] = -1
    k_out = torch.empty(B, Hkv, top, dqk, dtype=torch.bfloat16, device="cuda")
    qp, kp = splash.paged_append(k[:, :, :top], v[:, :, :top], kc, vc, bt, pos, q=q[:, :, :top], table=table,
                                 rot_offset=offset, k_out=k_out)
    mi = splash.build_mask_info(splash.MaskSpec(True), top, top, 128, 128)
    out, lse = splash.attention_fwd(qp, kp, v[:, :, :top].contiguous(), mi, scale)
    mi.close()
    for b in range(B):
        n = prompt[b]
        assert torch.equal(qp[b, :, :n], qr[b, :, :n]) and torch.equal(kp[b, :, :n], kr[b, :, :n])
        assert (out[b, :, :n].float() - want[b, :, :n].float()).abs().max().item() <= room
    # the answers, one token at a time and then the last four at once
    for step in range(answer - 4):
        at = lens.long()
        tok = [torch.stack([x[b, :, at[b]] for b in range(B)])[:, :, None] for x in (q, k, v)]
        q1, _ = splash.paged_append(tok[1], tok[2], kc, vc, bt, lens[:, None], q=tok[0], table=table, rot_offset=offset)
        lens = lens + 1
        o, l = splash.paged_decode(q1, kc, vc, bt, lens, scale)
        for b in range(B):
            i = prompt[b] + step
            assert (o[b, :, 0].float() - want[b, :, i].float()).abs().max().item() <= room
            assert (l[b, :, 0] - want_lse[b, :, i]).abs().max().item() <= 1e-3
    at = lens.long()
    tok = [torch.stack([x[b, :, at[b]:at[b] + 4] for b in range(B)]) for x in (q, k, v)]
    p4 = lens[:, None] + torch.arange(4, dtype=torch.int32, device="cuda")
    q4, _ = splash.paged_append(tok[1], tok[2], kc, vc, bt, p4, q=tok[0], table=table, rot_offset=offset)
    o, l = splash.paged_decode(q4, kc, vc, bt, lens + 4, scale)
    splash.check_device_error()
    for b in range(B):
        i = prompt[b] + answer - 4
        assert (o[b].float() - want[b, :, i:i + 4].float()).abs().max().item() <= room
        assert (l[b] - want_lse[b, :, i:i + 4]).abs().max().item() <= 1e-3


def decode_state(B=3, page=16, per=12, Hq=8, Hkv=2, d=128, seed=400):
    kc, vc = (workloads.normal_bf16((B * per, Hkv, page, d), seed + i).cuda() for i in range(2))
    bt = torch.randperm(B * per, generator=torch.Generator().manual_seed(seed)).view(B, per).to(torch.int32).cuda()
    tok = [workloads.normal_bf16((B, h, 1, d), seed + 2 + i).cuda() for i, h in enumerate((Hq, Hkv, Hkv))]
    lens = torch.tensor([5, 100, 64][:B], dtype=torch.int32, device="cuda")
    return tok, kc, vc, bt, lens


def step(splash, tok, kc, vc, bt, lens, table, q_out, out, lse, ws):
    splash.paged_append(tok[1], tok[2], kc, vc, bt, lens[:, None], q=tok[0], table=table, q_out=q_out)
    lens += 1
    splash.paged_decode(q_out, kc, vc, bt, lens, 0.1, out=out, lse=lse, workspace=ws)


@pytest.mark.parametrize("per", [12, 2600], ids=["short rows of pages", "long rows of pages"])
def test_a_captured_step_replays_with_growing_lengths(splash, per):
    tok, kc, vc, bt, lens = decode_state(per=per)
    table = splash.rope_table(256, 128)
    B, Hq, Hkv, d = 3, 8, 2, 128
    q_out, out = torch.empty_like(tok[0]), torch.empty(B, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, Hq, 1, device="cuda")
    ws = torch.empty(splash.paged_decode_workspace_size(tok[0], kc, vc, bt), dtype=torch.uint8, device="cuda")
    eager = [kc.clone(), vc.clone(), bt, lens.clone()]
    eo, el, eq = torch.empty_like(out), torch.empty_like(lse), torch.empty_like(q_out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(splash, tok, kc.clone(), vc.clone(), bt, lens.clone(), table, q_out, out, lse, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(splash, tok, kc, vc, bt, lens, table, q_out, out, lse, ws)
    for _ in range(70):  # past a page and past a tile of keys
        for t in tok:
            t.copy_(-t.roll(1, -1))
        graph.replay()
        step(splash, tok, *eager, table, eq, eo, el, ws)
        assert torch.equal(out, eo) and torch.equal(lse, el)
    assert torch.equal(kc, eager[0]) and torch.equal(vc, eager[1]) and torch.equal(lens, eager[3])
    assert splash.last_device_error() == 0


def test_two_captured_steps_replayed_at_once(splash):
    """Two graphs, each with a cache and a workspace of its own, replayed on two
    streams at the same time: both paths of the decode, bit for bit."""
    table = splash.rope_table(256, 128)
    runs = []
    for i, per in enumerate((12, 2600, 2600)):
        tok, kc, vc, bt, lens = decode_state(per=per, seed=500 + 10 * i)
        runs.append([tok, kc, vc, bt, lens, torch.empty_like(tok[0]), torch.empty_like(tok[0]),
                     torch.empty(3, 8, 1, device="cuda"), torch.cuda.CUDAGraph(), torch.cuda.Stream()])
    def one(r):
        splash.paged_append(r[0][1], r[0][2], r[1], r[2], r[3], r[4][:, None], q=r[0][0], table=table, q_out=r[5])
        r[4] += 1
        splash.paged_decode(r[5], r[1], r[2], r[3], r[4], 0.1, out=r[6], lse=r[7])  # (its own workspace)
    want = []
    for r in runs:
        keep = [x.clone() for x in (r[1], r[2], r[4])]
        for _ in range(5):
            one(r)
        want.append([r[i].clone() for i in (1, 2, 4, 6, 7)])
        for x, y in zip((r[1], r[2], r[4]), keep):
            x.copy_(y)
    torch.cuda.synchronize()
    for r in runs:
        with torch.cuda.graph(r[8]):
            one(r)
    for _ in range(5):
        for r in runs:
            with torch.cuda.stream(r[9]):
                r[8].replay()
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        for i, x in zip((1, 2, 4, 6, 7), w):
            assert torch.equal(r[i], x)
    assert splash.last_device_error() == 0


def test_calls_on_another_stream_and_two_at_once(splash):
    tok, kc, vc, bt, lens = decode_state(per=2600)
    table = splash.rope_table(256, 128)
    pos = lens[:, None].contiguous()
    q1, _ = splash.paged_append(tok[1], tok[2], kc, vc, bt, pos, q=tok[0], table=table)
    want = splash.paged_decode(q1, kc, vc, bt, lens + 1, 0.1)
    more = lens + 1
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):  # each call takes its workspace from its own stream's memory
        for s in (a, b.cuda_stream):
            qs, _ = splash.rope_fwd(tok[0], None, pos, table, stream=s)
            got.append((qs, *splash.paged_decode(q1, kc, vc, bt, more, 0.1, stream=s)))
    with torch.cuda.stream(a):
        got.append((splash.rope_fwd(tok[0], None, pos, table)[0], *splash.paged_decode(q1, kc, vc, bt, more, 0.1)))
    torch.cuda.synchronize()
    for qs, o, l in got:
        assert torch.equal(qs, q1) and torch.equal(o, want[0]) and torch.equal(l, want[1])
    assert splash.last_device_error() == 0


def test_parts_of_a_cache_join_through_the_log_sum_exp(splash):
    """Attention over a shared prefix and over the rest, merged by
    attention_merge, equals attention over all (within two bf16 roundings of
    the parts and one of the result)."""
    tok, kc, vc, bt, _ = decode_state(B=1)
    n = torch.tensor([150], dtype=torch.int32, device="cuda")
    want, want_lse = splash.paged_decode(tok[0], kc, vc, bt, n, 0.1)
    cut = 64
    a = splash.paged_decode(tok[0], kc, vc, bt, torch.full_like(n, cut), 0.1)
    b = splash.paged_decode(tok[0], kc, vc, bt[:, cut // 16:], n - cut, 0.1)
    o, l = splash.attention_merge(torch.stack((a[0], b[0])).float(), torch.stack((a[1], b[1])))
    room = 4 * 2.0 ** -8 * vc.float().abs().max().item()
    assert (o.float() - want.float()).abs().max().item() <= room
    assert (l - want_lse).abs().max().item() <= 1e-4
    assert splash.last_device_error() == 0
