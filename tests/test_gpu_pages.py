"""paged_remap, paged_copy and paged_compact on the GPU: whole numbers and bits,
equal to the reference's."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_cache(pages, Hkv, page, d, kind, layout, seed):
    """Random bits, NaN patterns among them: values move as they are."""
    size = 1 if kind == "e4m3" else 2
    shape = (pages, page, Hkv, d * size) if layout == "tokens" else (pages, Hkv, page, d * size)
    t = torch.randint(0, 256, shape, generator=torch.Generator().manual_seed(seed), dtype=torch.uint8).cuda()
    t = t.view(torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16)
    return t.transpose(1, 2) if layout == "tokens" else t


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy()


def remap(splash, table, parents, keep, room, refs, page, **kw):
    out = splash.paged_remap(i32(table), i32(parents), i32(keep), i32(room), i32(refs), page, **kw)
    return [x.cpu().tolist() for x in out]


def agrees(got, want):
    new, out, copies, short = want
    assert got[0] == new and got[1] == out and got[2] == [list(c) for c in copies] and got[3] == [short]


def random_pool(rng, rows, cols, page, spare, shared):
    """A table with prefixes in common, its lengths and counts, and pages held by others."""
    table, lens, pool = [], [], list(rng.permutation(rows * cols + spare))
    refs = [0] * len(pool)
    for r in range(rows):
        n = int(rng.integers(0, cols * page + 1))
        need = -(-n // page)
        row = []
        if r and rng.random() < shared:
            row = [p for p in table[int(rng.integers(0, r))][:need] if p >= 0]
            row = row[:int(rng.integers(0, len(row) + 1))]
        row += [int(pool.pop()) for _ in range(need - len(row))]
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (cols - need))
        lens.append(n)
    for p in rng.permutation(len(refs))[:len(refs) // 8]:
        refs[p] += 1  # somebody else's
    return table, lens, refs


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("rows, new_rows, cols, page, spare", [
    (1, 1, 1, 16, 3), (3, 7, 5, 16, 40), (1, 40, 33, 64, 300), (64, 64, 9, 32, 0), (70, 300, 3, 128, 900), (300, 5, 40, 16, 5)])
def test_remap_matches_the_reference(splash, rows, new_rows, cols, page, spare, seed):
    rng = np.random.default_rng(seed)
    table, lens, refs = random_pool(rng, rows, cols, page, spare, 0.5)
    parents = [int(x) for x in rng.integers(-1, rows, size=new_rows)]
    keep = [0 if p < 0 else int(rng.integers(0, lens[p] + 1)) if rng.random() < 0.5 else lens[p] for p in parents]
    room = [min(cols * page, k + int(rng.integers(-3, 2 * page))) for k in keep]
    want = ref.remap(table, parents, keep, room, refs, page)
    got = remap(splash, table, parents, keep, room, refs, page)
    splash.check_device_error()
    agrees(got, want)
    # into given tensors, the counts in place
    r = i32(refs)
    ws = torch.full((splash.paged_remap_workspace_size(len(refs), new_rows) + 16,), 0x5A, dtype=torch.uint8, device="cuda")
    given = [torch.full((new_rows, cols), 9, dtype=torch.int32, device="cuda"), r, i32([[7] * 3] * new_rows), i32([5])]
    out = splash.paged_remap(i32(table), i32(parents), i32(keep), i32(room), r, page, *given, workspace=ws[:-16])
    assert all(a is b for a, b in zip(out, given)) and (ws[-16:] == 0x5A).all()
    agrees([x.cpu().tolist() for x in out], want)


def test_remap_of_a_large_pool(splash):
    """More pages, rows and columns than one round of the cluster's threads."""
    rng = np.random.default_rng(50)
    table, lens, refs = random_pool(rng, 600, 90, 16, 30000, 0.3)
    parents = [int(x) for x in rng.integers(-1, 600, size=9000)]
    keep = [0 if p < 0 else lens[p] for p in parents]
    room = [k + 1 if k < 90 * 16 else k for k in keep]
    want = ref.remap(table, parents, keep, room, refs, 16)
    agrees(remap(splash, table, parents, keep, room, refs, 16), want)
    splash.check_device_error()


def test_remap_without_an_old_table(splash):
    refs = [1, 0, 0, 1, 0]
    got = splash.paged_remap(torch.empty(0, 2, dtype=torch.int32, device="cuda"), i32([-1, -1]), i32([0, 0]), i32([20, 3]),
                             i32(refs), 16)
    assert [x.cpu().tolist() for x in got] == [[[1, 2], [4, -1]], [1, 1, 1, 1, 1], [[-1, -1, 0]] * 2, [0]]
    splash.check_device_error()


def test_remap_short_of_pages(splash):
    want = ref.remap([[5, -1, -1, -1]], [0, 0, 0, 0], [9] * 4, [64] * 4, [0] * 5 + [1, 0, 0], 16)
    got = remap(splash, [[5, -1, -1, -1]], [0, 0, 0, 0], [9] * 4, [64] * 4, [0] * 5 + [1, 0, 0], 16)
    assert want[3] == 8
    agrees(got, want)
    splash.check_device_error()


def test_remap_reports_what_is_wrong(splash):
    table, refs, page = [[0, 1, -1], [2, -1, -1]], [1, 1, 1, 0, 0, 0, 0, 0], 16
    good = remap(splash, table, [0, 1], [20, 10], [20, 10], refs, page)
    assert splash.last_device_error() == 0
    for parents, keep, room, same in (([2, 1], [20, 10], [0, 10], 1), ([0, 1], [-1, 10], [0, 10], 1),
                                      ([0, 1], [49, 10], [0, 10], 1), ([0, 1], [20, 10], [20, 49], 0)):
        got = remap(splash, table, parents, keep, room, refs, page)
        assert splash.last_device_error() == 7
        assert got[0][same] == good[0][same]
        assert all(-1 <= p < 8 for row in got[0] for p in row) and len(set(sum(got[0], [])) - {-1}) == sum(p >= 0 for row in got[0] for p in row)
    got = remap(splash, [[0, 99, -1], [2, -1, -1]], [0, 1], [20, 10], [20, 10], refs, page)
    assert splash.last_device_error() == 7 and got[0] == [[0, -1, -1], [2, -1, -1]]
    got = remap(splash, table, [-1, -1], [0, 0], [0, 0], [1, 0, 1, 0, 0, 0, 0, 0], page)  # counted less than used
    assert splash.last_device_error() == 7 and got[1][0] == 0


@pytest.mark.parametrize("Hkv, dqk, dv, page, kind, layout", [
    (2, 64, 64, 16, "bf16", "heads"), (3, 192, 128, 64, "bf16", "tokens"), (1, 128, 128, 32, "e4m3", "heads"),
    (8, 128, 128, 128, "bf16", "heads"), (2, 16, 48, 16, "e4m3", "tokens"), (1, 512, 16, 1024, "bf16", "heads")])
def test_copy_matches_the_reference(splash, Hkv, dqk, dv, page, kind, layout):
    pages = 12
    kc, vc = (make_cache(pages, Hkv, page, d, kind, layout, 60 + i) for i, d in enumerate((dqk, dv)))
    copies = [[0, 5, page], [-1, -1, 0], [0, 6, 1], [3, 7, page - 1], [2, 8, 0], [4, -1, 3], [11, 9, page // 2]]
    want = [ref.copy(bits(c), copies) for c in (kc, vc)]
    splash.paged_copy(kc, vc, i32(copies))
    splash.check_device_error()
    assert all(np.array_equal(bits(c), w) for c, w in zip((kc, vc), want))
    for bad in ([0, pages, 3], [pages, 0, 3], [0, 1, page + 1], [2 ** 31 - 1, 1, 1]):
        splash.paged_copy(kc, vc, i32([bad, [1, 10, 2]]))
        assert splash.last_device_error() == 7
        want = [ref.copy(w, [[1, 10, 2]]) for w in want]
        assert all(np.array_equal(bits(c), w) for c, w in zip((kc, vc), want))


COMPACTS = [  # B, Hkv, dqk, dv, page, kind, layout, length, start, moved
    (1, 8, 128, 128, 16, "bf16", "heads", 40, 20, 5),
    (3, 2, 64, 64, 16, "bf16", "tokens", 70, 1, 1),
    (2, 1, 192, 128, 64, "e4m3", "heads", 500, 0, 300),
    (2, 3, 16, 48, 16, "e4m3", "tokens", 900, 7, 700),
    (1, 1, 512, 96, 1024, "bf16", "heads", 1500, 1020, 470),
    (5, 2, 128, 64, 32, "bf16", "heads", 1300, 4, 1296),
    (2, 2, 112, 80, 16, "bf16", "heads", 400, 3, 222),
]


@pytest.mark.parametrize("case", COMPACTS, ids=str)
def test_compact_matches_the_reference(splash, case):
    B, Hkv, dqk, dv, page, kind, layout, length, start, moved = case
    rng = np.random.default_rng(70)
    per = -(-length // page)
    bt = rng.permutation(B * per + 2)[:B * per].reshape(B, per).tolist()
    bt = [row + [-1] for row in bt]
    src, starts = [], []
    for b in range(B):
        starts.append(start)
        picked = sorted(rng.permutation(length - start)[:moved] + start)
        if b == B - 1 and moved > 2:
            picked = picked[:moved // 2] + [-1] + picked[moved // 2 + 1:]  # what follows is ignored
        src.append([int(x) for x in picked])
    kc, vc = (make_cache(B * per + 2, Hkv, page, d, kind, layout, 71 + i) for i, d in enumerate((dqk, dv)))
    want = [ref.compact(bits(c), bt, src, starts) for c in (kc, vc)]
    splash.paged_compact(kc, vc, i32(bt), i32(src), i32(starts))
    splash.check_device_error()
    assert all(np.array_equal(bits(c), w) for c, w in zip((kc, vc), want))


@pytest.mark.parametrize("moved", [3, 200])
def test_compact_ends_at_what_is_wrong(splash, moved):
    Hkv, d, page, per = 2, 64, 16, 40
    bt = np.random.default_rng(80).permutation(2 * per + 4)[:2 * per].reshape(2, per).tolist()
    line = list(range(30, 30 + 2 * moved, 2))
    at = moved - 1
    cases = [("src", 9), ("src", line[at - 1]), ("src", per * page), ("src", 2 ** 31 - 1), ("from", -1), ("from", 2 * per + 4),
             ("to", -5), ("start", -1)]
    for what, value in cases:
        src, table, start = [list(line), list(line)], [list(r) for r in bt], [10, 10]
        if what == "src":
            src[1][at] = value
        elif what == "start":
            start[1] = value
        else:
            table[1][(line[at] if what == "from" else 10 + at) // page] = value
        kc, vc = (make_cache(2 * per + 4, Hkv, page, d, "bf16", "heads", 81 + i) for i in range(2))
        before = [bits(c).copy() for c in (kc, vc)]
        splash.paged_compact(kc, vc, i32(table), i32(src), i32(start))
        assert splash.last_device_error() == 7, what
        # the other sequence moves, this one up to the first entry that is wrong
        stop = 0 if what == "start" else next(
            m for m in range(moved) if (what == "src" and m == at) or
            (what != "src" and value in (table[1][line[m] // page], table[1][(10 + m) // page])))
        lists = [list(line), list(line[:stop])]
        want = [ref.compact(c, bt, lists, [10, 10]) for c in before]
        assert all(np.array_equal(bits(c), w) for c, w in zip((kc, vc), want)), what
    # an entry behind the end of a list is not looked at
    src = [list(line), line[:1] + [-1] + [2 ** 31 - 1] * (moved - 2)]
    splash.paged_compact(kc, vc, i32(bt), i32(src), i32([10, 10]))
    assert splash.last_device_error() == 0


def test_compact_past_32_bits(splash):
    pages, Hkv, page, d = 2100, 8, 1024, 128
    kc = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    small = workloads.normal_bf16((2, Hkv, page, d), 90).cuda()
    kc[pages - 1], vc[pages - 1] = small[0], small[1]
    bt = i32([[pages - 2, pages - 1]])
    splash.paged_compact(kc, vc, bt, i32([[1030, 1100]]), i32([5]))
    splash.paged_copy(kc, vc, i32([[pages - 1, pages - 3, 700]]))
    splash.check_device_error()
    for c, s in ((kc, small[0]), (vc, small[1])):
        assert torch.equal(c[pages - 2, :, 5], s[:, 6]) and torch.equal(c[pages - 2, :, 6], s[:, 76])
        assert torch.equal(c[pages - 3, :, :700], s[:, :700])
