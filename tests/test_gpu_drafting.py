"""Serving with drafts and forks as a program does it: drafts stored, checked and
kept, sequences forked and continued, a training step with three position axes,
graph capture and replay, other streams."""
import math

import numpy as np
import pytest
import torch

import oracle
import workloads
from oracle import drafting_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def splash():
    from block_sparse_flash_gb300 import build as b
    b.build()
    import block_sparse_flash_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def host(t):
    return t.double().cpu().numpy()


def test_training_step_gradients_with_three_axes(splash):
    """rope_axes_fwd -> attention_fwd -> attention_bwd -> rope_axes_bwd: the
    gradients of the unrotated q and k against the oracle's, turned back in 64 bits
    (limit as for the backward's own parity: 2e-2 of the norm)."""
    B, Hq, Hkv, L, d = 1, 4, 2, 384, 64
    q, k, v, g = (workloads.normal_bf16((B, h, L, d), 200 + i) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    table = splash.rope_table(L, d)
    i = torch.arange(L)
    pos = torch.stack((i // 48, i % 48 // 8, i % 8))[:, None].expand(3, B, L).to(torch.int32).cuda()
    for sections, cycled in (((16, 8, 8), False), ((12, 10, 10), True)):
        axes = splash.rope_axis_map(sections, cycled)
        mi = splash.build_mask_info(splash.MaskSpec(True), L, L, 128, 128)
        qr, kr = splash.rope_axes_fwd(q.cuda(), k.cuda(), pos, table, axes)
        vd, gd = v.cuda(), g.cuda()
        out, lse = splash.attention_fwd(qr, kr, vd, mi, 0.125)
        dqr, dkr, _ = splash.attention_bwd(qr, kr, vd, out, lse, gd, mi, 0.125)
        dq, dk = splash.rope_axes_bwd(dqr, dkr, pos, table, axes)
        splash.check_device_error()
        want = oracle.attention_bwd(qr.cpu(), kr.cpu(), v, g, oracle.MaskSpec(True), 0.125, 0.0)
        for got, grad in ((dq, want["dq"].reshape(B, Hq, L, d)), (dk, want["dk"].reshape(B, Hkv, L, d))):
            exact = ref.rope_axes(grad, pos.cpu().numpy(), host(table), axes, inverse=True)
            assert np.linalg.norm(host(got) - exact) <= 2e-2 * np.linalg.norm(exact)
        mi.close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq, Hkv, dqk, dv, rot, offset, page, T", [
    (8, 2, 128, 128, 128, 0, 16, 12), (4, 4, 192, 128, 64, 128, 64, 5), (16, 2, 64, 64, 64, 0, 32, 40)])
def test_drafts_stored_checked_and_kept(splash, Hq, Hkv, dqk, dv, rot, offset, page, T, kind):
    """A tree of drafts is stored behind each context and attends; one branch is
    kept.  The cache is then, bit for bit, what storing the branch alone makes, and
    the branch's rows are what paged_decode gives for it."""
    B, ctx = 3, [50, 1, 133]
    g = np.random.default_rng(7)
    parents = np.array([[int(g.integers(-1, l)) for l in range(T)] for _ in range(B)], dtype=np.int32)
    depth = np.zeros((B, T), dtype=np.int32)
    for b in range(B):
        for l in range(T):
            depth[b, l] = 0 if parents[b, l] < 0 else depth[b, parents[b, l]] + 1
    per = -(-(max(ctx) + T) // page)
    bt = torch.randperm(B * per, generator=torch.Generator().manual_seed(8)).view(B, per).to(torch.int32).cuda()
    dtype = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    ks, vs = (torch.linspace(a, 2 * a, Hkv, device="cuda") if kind == "e4m3" else None for a in (0.01, 0.02))
    kc, vc = (torch.zeros(B * per, Hkv, page, d, device="cuda").to(dtype) for d in (dqk, dv))
    table, axes = splash.rope_table(max(ctx) + T, rot), splash.rope_axis_map([rot // 2])
    kw = dict(rot_offset=offset, k_scale=ks, v_scale=vs)
    # the contexts
    top = max(ctx)
    pos = torch.arange(top, dtype=torch.int32, device="cuda").expand(B, top).clone()
    pos[pos >= i32(ctx)[:, None]] = -1
    k0, v0 = (workloads.normal_bf16((B, Hkv, top, d), 10 + i).cuda() for i, d in enumerate((dqk, dv)))
    splash.paged_append(k0, v0, kc, vc, bt, pos, table=table, **kw)
    plain = [kc.clone(), vc.clone()]
    # the drafts: slots in a row, rotations by depth
    q, k, v = (workloads.normal_bf16((B, h, T, d), 20 + i).cuda() for i, (h, d) in enumerate(((Hq, dqk), (Hkv, dqk), (Hkv, dv))))
    slots = i32(ctx)[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")
    turn = (i32(ctx)[:, None] + torch.from_numpy(depth).cuda())[None]
    qr, _ = splash.paged_append_axes(k, v, kc, vc, bt, slots, turn, table, axes, q=q, **kw)
    lens = i32(ctx) + T
    scale = 1 / math.sqrt(dqk)
    out, lse = splash.paged_tree_decode(qr, kc, vc, bt, lens, torch.from_numpy(parents).cuda(), scale, k_scale=ks, v_scale=vs)
    # the deepest branch of each tree is kept
    branches = []
    for b in range(B):
        at, path = int(depth[b].argmax()), []
        while at >= 0:
            path.append(at)
            at = int(parents[b, at])
        branches.append(path[::-1])
    longest = max(map(len, branches))
    src = i32([[ctx[b] + l for l in path] + [-1] * (longest - len(path)) for b, path in enumerate(branches)])
    splash.paged_compact(kc, vc, bt, src, i32(ctx))
    splash.check_device_error()
    for b, path in enumerate(branches):
        n, pick = len(path), torch.tensor(path, device="cuda")
        at = (ctx[b] + torch.arange(n, dtype=torch.int32, device="cuda"))[None]
        kb, vb, qb = (x[b:b + 1, :, pick] for x in (k, v, q))
        q1, _ = splash.paged_append(kb, vb, *plain, bt[b:b + 1], at, q=qb, table=table, **kw)
        assert torch.equal(q1[0], qr[b][:, pick])
        for j in range(ctx[b] + n):
            for c, p in zip((kc, vc), plain):
                x, y = (z.view(torch.uint8)[bt[b, j // page].item(), :, j % page] for z in (c, p))
                assert torch.equal(x, y), (b, j)
        for i in range(0, n, 16):  # the branch as a chain, 16 tokens a call
            m = min(16, n - i)
            o, l = splash.paged_decode(q1[:, :, i:i + m], *plain, bt[b:b + 1], i32([ctx[b] + i + m]), scale, k_scale=ks, v_scale=vs)
            a, c = out[b][:, pick[i:i + m]].float(), o[0].float()
            # both round p (2^-16, e4m3 2^-11) and the result (2^-8) once, and their scores in another order
            big = vc.float().abs().nan_to_num().max() * (1 if vs is None else vs.max())
            assert (a - c).abs().max() <= 2.0 ** -7 * a.abs().max() + 2.0 ** -9 * big
            assert (lse[b][:, pick[i:i + m]] - l[0]).abs().max() <= 1e-4
    splash.check_device_error()


def test_forks_continue_on_their_own(splash):
    """Two layers' caches of two prompts fork into samples; each sample goes on
    with tokens of its own; every one attends as if its pages were nobody else's.
    Then all but one end, and what they held is free."""
    layers, Hq, Hkv, d, page, cols, pages = 2, 8, 2, 128, 16, 6, 40
    prompts, samples = [37, 48], 3
    caches = [[torch.zeros(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(layers)]
    refs = i32([0] * pages)
    table, refs, copies, short = splash.paged_remap(torch.empty(0, cols, dtype=torch.int32, device="cuda"), i32([-1, -1]),
                                                    i32([0, 0]), i32(prompts), refs, page)
    tokens = [[workloads.normal_bf16((2, Hkv, 48, d), 30 + 2 * y + i).cuda() for i in range(2)] for y in range(layers)]
    pos = torch.arange(48, dtype=torch.int32, device="cuda").expand(2, 48).clone()
    pos[pos >= i32(prompts)[:, None]] = -1
    for y in range(layers):
        splash.paged_append(*tokens[y], *caches[y], table, pos)
    parents = [0] * samples + [1] * samples
    keep = [prompts[p] for p in parents]
    lens = i32(keep)
    rest = [[[] for _ in parents] for _ in range(layers)]
    for step in range(20):
        # (the first step forks, the others make room)
        if step == 0:
            table, refs, copies, short = splash.paged_remap(table, i32(parents), lens, lens + 1, refs, page)
            assert int((copies[:, 2] > 0).sum()) == samples - 1  # 48 fills its pages, the first of the others keeps its own
            for y in range(layers):
                splash.paged_copy(*caches[y], copies)
        else:
            own = torch.arange(len(parents), dtype=torch.int32, device="cuda")
            table, refs, copies, short = splash.paged_remap(table, own, lens, lens + 1, refs, page)
            assert (copies == i32([-1, -1, 0])).all()
        assert short.item() == 0
        for y in range(layers):
            kv = [workloads.normal_bf16((len(parents), Hkv, 1, d), 100 + 10 * step + 2 * y + i).cuda() for i in range(2)]
            splash.paged_append(*kv, *caches[y], table, lens[:, None].contiguous())
            for i in range(len(parents)):
                rest[y][i].append([x[i] for x in kv])
        lens = lens + 1
    splash.check_device_error()
    held = table.cpu().numpy()
    counts = np.bincount(held[held >= 0], minlength=pages)
    assert refs.cpu().tolist() == counts.tolist()
    # each sample against a cache of its own
    q = workloads.normal_bf16((len(parents), Hq, 1, d), 90).cuda()
    for y in range(layers):
        got = splash.paged_decode(q, *caches[y], table, lens, 0.1)
        alone = [torch.zeros(len(parents) * cols, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        bt = torch.arange(len(parents) * cols, dtype=torch.int32, device="cuda").view(-1, cols)
        for i, p in enumerate(parents):
            n = prompts[p]
            whole = [torch.cat([tokens[y][x][p, :, :n]] + [r[x] for r in rest[y][i]], 1)[None] for x in range(2)]
            splash.paged_append(*whole, *alone, bt[i:i + 1], torch.arange(n + 20, dtype=torch.int32, device="cuda")[None])
        want = splash.paged_decode(q, *alone, bt, lens, 0.1)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # one goes on, rolled back to 30 tokens; the others end
    table, refs, copies, _ = splash.paged_remap(table, i32([4]), i32([30]), i32([30]), refs, page)
    assert table.cpu().tolist()[0][2:] == [-1] * 4 and int(refs.sum()) == 2 and copies.cpu().tolist() == [[-1, -1, 0]]
    splash.check_device_error()


def tree_state(per, T=10, B=3, Hq=8, Hkv=2, d=128, page=16, seed=400):
    kc, vc = (workloads.normal_bf16((B * 12, Hkv, page, d), seed + i).cuda() for i in range(2))
    bt = torch.zeros(B, per, dtype=torch.int32)
    bt[:, :12] = torch.randperm(B * 12, generator=torch.Generator().manual_seed(seed)).view(B, 12)
    tok = [workloads.normal_bf16((B, h, T, d), seed + 2 + i).cuda() for i, h in enumerate((Hq, Hkv, Hkv))]
    parents = i32([[l // 2 - 1 if l else -1 for l in range(T)], [l - 1 for l in range(T)], [-1] * T])
    depth = i32([[int(math.log2(l + 1)) if l else 0 for l in range(T)], list(range(T)), [0] * T])
    for l in range(T):  # (l // 2 - 1: token 1's parent is none, 2 and 3 have token 0)
        depth[0, l] = 0 if l < 2 else depth[0, l // 2 - 1] + 1
    return tok, kc, vc, bt.cuda(), i32([5, 100, 64][:B]), parents, depth


def draft_step(splash, tok, kc, vc, bt, ctx, parents, depth, table, q_out, out, lse, ws):
    T = tok[0].shape[2]
    slots = ctx[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")
    splash.paged_append_axes(tok[1], tok[2], kc, vc, bt, slots, (ctx[:, None] + depth)[None], table,
                             splash.rope_axis_map([64]), q=tok[0], q_out=q_out)
    splash.paged_tree_decode(q_out, kc, vc, bt, ctx + T, parents, 0.1, out=out, lse=lse, workspace=ws)
    # the tokens 0 and 2 (their slots ascend) stay
    splash.paged_compact(kc, vc, bt, ctx[:, None] + i32([0, 2]), ctx)
    ctx += 2


@pytest.mark.parametrize("T", [10, 33])
@pytest.mark.parametrize("per", [12, 2600], ids=["short rows of pages", "long rows of pages"])
def test_a_captured_draft_step_replays_with_growing_lengths(splash, per, T):
    tok, kc, vc, bt, ctx, parents, depth = tree_state(per, T)
    table = splash.rope_table(256, 128)
    B, Hq, d = 3, 8, 128
    new = lambda: (torch.empty_like(tok[0]), torch.empty(B, Hq, T, d, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                   torch.empty(B, Hq, T, device="cuda"))
    size = splash.paged_tree_decode_workspace_size(tok[0], kc, vc, bt)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    got, want = new(), new()
    eager = [kc.clone(), vc.clone(), bt, ctx.clone(), parents, depth]
    keep = [ctx.clone(), i32([0, 2])]
    draft_step(splash, tok, kc.clone(), vc.clone(), bt, keep[0], parents, depth, table, *want, ws)
    ar, pick = torch.arange(T, dtype=torch.int32, device="cuda"), i32([0, 2])

    def captured():
        splash.paged_append_axes(tok[1], tok[2], kc, vc, bt, ctx[:, None] + ar, (ctx[:, None] + depth)[None], table,
                                 splash.rope_axis_map([64]), q=tok[0], q_out=got[0])
        splash.paged_tree_decode(got[0], kc, vc, bt, ctx + T, parents, 0.1, out=got[1], lse=got[2], workspace=ws)
        splash.paged_compact(kc, vc, bt, ctx[:, None] + pick, ctx)
        ctx.add_(2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured()
    for n in range(25):  # past a page and past a step of keys
        for t in tok:
            t.copy_(-t.roll(1, -1))
        if n == 12:  # another tree
            parents.copy_(parents.roll(1, 0))
            depth.copy_(depth.roll(1, 0))
        graph.replay()
        draft_step(splash, tok, *eager, table, *want, ws)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert torch.equal(kc, eager[0]) and torch.equal(vc, eager[1]) and torch.equal(ctx, eager[3])
    assert splash.last_device_error() == 0


def test_a_captured_remap_replays(splash):
    refs = i32([1, 1, 1] + [0] * 20)
    table, lens = i32([[0, 1, -1, -1], [2, -1, -1, -1]]), i32([20, 7])
    parents, room = i32([0, 0, 1]), i32([21, 21, 40])
    kc, vc = (workloads.normal_bf16((23, 2, 16, 64), s).cuda() for s in (1, 2))
    keep = lens[parents.long()].contiguous()
    out = [torch.empty(3, 4, dtype=torch.int32, device="cuda"), torch.empty_like(refs),
           torch.empty(3, 3, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")]
    ws = torch.empty(splash.paged_remap_workspace_size(23, 3), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        splash.paged_remap(table, parents, keep, room, refs, 16, *out, workspace=ws)
        splash.paged_copy(kc, vc, out[2])
    for lengths, ps in (([20, 7], [0, 0, 1]), ([32, 3], [1, 0, 1]), ([1, 16], [-1, 1, 0])):
        parents.copy_(i32(ps))
        keep.copy_(i32([0 if p < 0 else lengths[p] for p in ps]))
        before = [kc.clone(), vc.clone()]
        graph.replay()
        new, counts, copies, short = ref.remap(table.tolist(), ps, keep.tolist(), room.tolist(), refs.tolist(), 16)
        assert [x.cpu().tolist() for x in out] == [new, counts, [list(c) for c in copies], [short]]
        for c, b in zip((kc, vc), before):
            assert np.array_equal(host(c), ref.copy(host(b), copies))
    assert splash.last_device_error() == 0


@pytest.mark.parametrize("T, Hq", [(6, 2), (40, 8)])
def test_calls_on_other_streams_and_two_at_once(splash, T, Hq):
    """Each call takes its workspace and outputs from its own stream's memory."""
    tok, kc, vc, bt, ctx, parents, depth = tree_state(2600, T, Hq=Hq)
    table, axes = splash.rope_table(256, 128), splash.rope_axis_map([64])
    turn = (ctx[:, None] + depth)[None].contiguous()
    qr, _ = splash.rope_axes_fwd(tok[0], None, turn, table, axes)
    lens = ctx + T
    want = splash.paged_tree_decode(qr, kc, vc, bt, lens, parents, 0.1)
    refs = i32([1] * 36 + [0] * 30)
    args = (bt[:, :12].contiguous(), i32([0, 0, 1, 2]), i32([37, 40, 50, 192]), i32([60, 41, 50, 192]), refs, 16)
    remapped = splash.paged_remap(*args)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        for s in (a, b.cuda_stream):
            got.append((splash.rope_axes_fwd(tok[0], None, turn, table, axes, stream=s)[0],
                        *splash.paged_tree_decode(qr, kc, vc, bt, lens, parents, 0.1, stream=s),
                        *splash.paged_remap(*args, stream=s)))
    with torch.cuda.stream(a):
        got.append((splash.rope_axes_fwd(tok[0], None, turn, table, axes)[0],
                    *splash.paged_tree_decode(qr, kc, vc, bt, lens, parents, 0.1), *splash.paged_remap(*args)))
    torch.cuda.synchronize()
    for x in got:
        for y, z in zip(x, (qr, *want, *remapped)):
            assert torch.equal(y, z)
    assert splash.last_device_error() == 0


@pytest.mark.parametrize("per", [12, 2600], ids=["short rows of pages", "long rows of pages"])
def test_two_captured_draft_steps(splash, per):
    """Two graphs with one workspace, replayed one after the other, and two with their own,
    replayed at the same time on two streams."""
    states = [tree_state(per, T, Hq=Hq, seed=500 + T) for T, Hq in ((10, 8), (33, 8))]
    sizes = [splash.paged_tree_decode_workspace_size(s[0][0], *s[1:4]) for s in states]
    shared = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    want = [splash.paged_tree_decode(s[0][0], *s[1:4], s[4] + s[0][0].shape[2], s[5], 0.1) for s in states]
    torch.cuda.synchronize()

    def capture(s, ws, out, lse):
        lens = s[4] + s[0][0].shape[2]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            splash.paged_tree_decode(s[0][0], *s[1:4], lens, s[5], 0.1, out=out, lse=lse, workspace=ws)
        return graph, lens
    results = [[torch.empty_like(y) for y in w] for w in want]
    graphs = [capture(s, shared, *r) for s, r in zip(states, results)]
    own = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    results_own = [[torch.empty_like(y) for y in w] for w in want]
    apart = [capture(s, ws, *r) for s, ws, r in zip(states, own, results_own)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(30):
        for r in results + results_own:
            for y in r:
                y.fill_(float("nan"))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (g, _), stream in zip(apart, streams):
            with torch.cuda.stream(stream):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for w, r, o in zip(want, results, results_own):
            assert all(torch.equal(a, b) for a, b in zip(w, r)) and all(torch.equal(a, b) for a, b in zip(w, o))
    assert splash.last_device_error() == 0
