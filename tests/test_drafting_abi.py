"""Refusals of the calls for drafts, forks and several axes on the CPU: the C
entry points reject invalid arguments before touching the GPU, and the binding
rejects tensors that do not fit.  No call here reaches a launch: the C ones run
without a device only."""
import ctypes

import pytest
import torch

from test_serving_abi import (BAD_CACHE, BAD_SCALES, BAD_TOKENS, CUDA, F32, I32, I64, INVALID, OK_PTR, P, SHAPE, UNSUPPORTED,
                              AppendArgs, DecodeArgs, RopeArgs, View, append_args, bf16, decode_args, dense, e4m3, fields,
                              i32, rope_args)

no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device pointers: only where there is no device")


@pytest.fixture(scope="module")
def splash():
    from block_sparse_flash_gb300 import build as b
    b.build()
    import block_sparse_flash_gb300 as m
    return m


class RopeAxesArgs(ctypes.Structure):
    _fields_ = fields((RopeArgs, "rope"), (I64, "positions_stride_a"), (P, "axes"), (I32, "num_axes reserved"))


class AppendAxesArgs(ctypes.Structure):
    _fields_ = fields((AppendArgs, "append"), (P, "rot_positions"), (I64, "rot_positions_stride_a rot_positions_stride_b"),
                      (P, "axes"), (I32, "num_axes reserved"))


class TreeArgs(ctypes.Structure):
    _fields_ = fields((DecodeArgs, "decode"), (P, "parents"), (I64, "parents_stride_b"))


class CompactArgs(ctypes.Structure):
    _fields_ = fields((View, "k_cache v_cache"), (P, "block_table"), (I64, "block_table_stride"), (P, "src"),
                      (I64, "src_stride"), (P, "start"), (I64, "num_pages moves"),
                      (I32, "B Hkv dqk dv max_pages page_size cache_type reserved"))


class RemapArgs(ctypes.Structure):
    _fields_ = fields((P, "block_table"), (I64, "block_table_stride"), (P, "new_table"), (I64, "new_table_stride"),
                      (P, "parents keep room refs refs_out copies short_pages workspace"), (ctypes.c_uint64, "workspace_bytes"),
                      (I64, "num_pages"), (I32, "num_rows new_rows max_pages page_size"))


class CopyArgs(ctypes.Structure):
    _fields_ = fields((View, "k_cache v_cache"), (P, "copies"), (I64, "num_pages"),
                      (I32, "count Hkv dqk dv page_size cache_type"))


AXES = (ctypes.c_uint8 * 64)(*[i % 3 for i in range(64)])
AXES_PTR = ctypes.addressof(AXES)  # host memory: it is read


def sized(a):
    a.struct_bytes = ctypes.sizeof(a)
    return a


def apart(view):
    view.ptr += 1 << 20
    return view


def rope_axes_args():
    return sized(RopeAxesArgs(rope=rope_args(), positions_stride_a=16, axes=AXES_PTR, num_axes=3))


def append_axes_args():
    return sized(AppendAxesArgs(append=append_args(), rot_positions=OK_PTR, rot_positions_stride_a=16,
                                rot_positions_stride_b=8, axes=AXES_PTR, num_axes=3))


def tree_args(T=5):
    d = decode_args()
    d.Lq, d.q = T, dense(4, T, 128)
    return sized(TreeArgs(decode=d, parents=OK_PTR, parents_stride_b=T))


def compact_args():
    return sized(CompactArgs(k_cache=dense(2, 16, 128), v_cache=apart(dense(2, 16, 128)), block_table=OK_PTR, block_table_stride=4,
                             src=OK_PTR, src_stride=8, start=OK_PTR, num_pages=9, moves=8, B=2, Hkv=2, dqk=128, dv=128,
                             max_pages=4, page_size=16))


def remap_args():
    return sized(RemapArgs(block_table=OK_PTR, block_table_stride=4, new_table=OK_PTR + (1 << 20), new_table_stride=4, parents=OK_PTR,
                           keep=OK_PTR, room=OK_PTR, refs=OK_PTR, refs_out=OK_PTR, copies=OK_PTR, short_pages=OK_PTR,
                           workspace=OK_PTR, workspace_bytes=1 << 20, num_pages=100, num_rows=2, new_rows=3, max_pages=4,
                           page_size=16))


def copy_args():
    return sized(CopyArgs(k_cache=dense(2, 16, 128), v_cache=dense(2, 16, 128), copies=OK_PTR, num_pages=9, count=3, Hkv=2,
                          dqk=128, dv=128, page_size=16))


MAKE = {"splash_rope_axes": rope_axes_args, "splash_paged_append_axes": append_axes_args,
        "splash_paged_tree_decode": tree_args, "splash_paged_compact": compact_args, "splash_paged_remap": remap_args,
        "splash_paged_copy": copy_args}


def status(splash, name, a):
    f = getattr(splash.lib(), name)
    f.restype = ctypes.c_int
    return f(bytes(a), None)


def check(splash, name, changes):
    for member, value, want in changes:
        a = MAKE[name]()
        where = a
        *path, last = member.split(".")
        for x in path:
            where = getattr(where, x)
        setattr(where, last, value)
        assert status(splash, name, a) == want, (name, member, value)


@no_device
def test_valid_arguments_reach_the_device(splash):
    for name, make in MAKE.items():
        assert status(splash, name, make()) == CUDA, name
        assert getattr(splash.lib(), name)(None, None) == INVALID


BAD_AXES = [("struct_bytes", 8, INVALID), ("axes", None, INVALID), ("num_axes", 0, INVALID), ("num_axes", -1, INVALID),
            ("num_axes", 2, INVALID), ("num_axes", 5, UNSUPPORTED), ("reserved", 1, INVALID)]
BAD_PAIR = [("struct_bytes", 8, INVALID), ("Hkv", 0, INVALID), ("Hkv", 65536, UNSUPPORTED), ("dqk", 0, INVALID),
            ("dqk", 120, UNSUPPORTED), ("dv", 528, UNSUPPORTED), ("k_cache.ptr", None, INVALID),
            ("v_cache.ptr", OK_PTR + 8, INVALID), ("k_cache.c", 132, INVALID), ("v_cache.a", 0, INVALID),
            ("num_pages", 0, INVALID), ("num_pages", 1 << 31, UNSUPPORTED), ("page_size", 0, INVALID),
            ("page_size", 24, UNSUPPORTED), ("page_size", 2048, UNSUPPORTED), ("cache_type", 2, INVALID)]


@no_device
def test_axes_refusals(splash):
    check(splash, "splash_rope_axes", BAD_AXES + [
        ("positions_stride_a", -1, INVALID), ("rope.struct_bytes", 8, INVALID), ("rope.positions", None, INVALID),
        ("rope.positions", OK_PTR + 2, INVALID), ("rope.positions_stride_b", -8, INVALID), ("rope.rot_dim", 24, UNSUPPORTED),
        ("rope.rot_offset", 16, SHAPE), ("rope.table", None, INVALID), ("rope.inverse", 2, INVALID),
        ("rope.q_out.c", 64, INVALID), ("rope.L", 0, INVALID)])
    check(splash, "splash_paged_append_axes", BAD_AXES + [
        ("rot_positions", None, INVALID), ("rot_positions", OK_PTR + 1, INVALID), ("rot_positions_stride_a", -1, INVALID),
        ("rot_positions_stride_b", -1, INVALID), ("append.struct_bytes", 8, INVALID), ("append.table", None, INVALID),
        ("append.positions", None, INVALID), ("append.num_seqs", 1, SHAPE), ("append.page_size", 8, UNSUPPORTED),
        ("append.k_cache.a", 0, INVALID), ("append.rot_dim", 144, SHAPE)])


@no_device
def test_tree_refusals(splash):
    check(splash, "splash_paged_tree_decode", [
        ("struct_bytes", 8, INVALID), ("decode.struct_bytes", 8, INVALID), ("parents", None, INVALID),
        ("parents", OK_PTR + 2, INVALID), ("parents_stride_b", -1, INVALID), ("decode.Lq", 0, INVALID),
        ("decode.Lq", 65, UNSUPPORTED), ("decode.Hkv", 3, SHAPE), ("decode.dqk", 64, UNSUPPORTED),
        ("decode.seq_lens", None, INVALID), ("decode.out", OK_PTR + 8, INVALID), ("decode.lse", None, INVALID),
        ("decode.scale", 0.0, INVALID), ("decode.scale", float("nan"), INVALID), ("decode.softcap", float("inf"), INVALID),
        ("decode.window_left", -2, INVALID), ("decode.reserved", 1, INVALID), ("decode.q.b", 4, INVALID),
        ("decode.k_cache.ptr", None, INVALID), ("decode.cache_type", 1, INVALID), ("decode.page_size", 12, UNSUPPORTED),
        ("decode.block_table", None, INVALID), ("decode.B", 65536, UNSUPPORTED), ("decode.max_pages", 0, INVALID)])
    a = tree_args(64)
    assert status(splash, "splash_paged_tree_decode", a) == CUDA
    a = tree_args(17)  # more than a chain may have
    assert status(splash, "splash_paged_tree_decode", a) == CUDA
    # 2^31 steps and starts of segments: 65535 sequences x 4096 heads x (1 + 9)
    a = tree_args(1)
    a.decode.B, a.decode.Hq, a.decode.Hkv, a.decode.max_pages = 65535, 4096, 4096, 1
    assert status(splash, "splash_paged_tree_decode", a) == UNSUPPORTED
    a.decode.Hq = a.decode.Hkv = 3000
    a.decode.q, a.decode.k_cache, a.decode.v_cache = dense(3000, 1, 128), dense(3000, 16, 128), dense(3000, 16, 128)
    assert status(splash, "splash_paged_tree_decode", a) == CUDA


@no_device
def test_tree_strides(splash):
    check(splash, "splash_paged_tree_decode", [
        ("decode.k_cache.c", 0, UNSUPPORTED), ("decode.v_cache.c", 0, UNSUPPORTED), ("decode.k_cache.a", 1 << 39, UNSUPPORTED),
        ("decode.v_cache.b", 1 << 39, UNSUPPORTED), ("decode.v_cache.a", (1 << 39) - 8, CUDA), ("decode.k_cache.b", 0, CUDA),
        ("decode.k_cache.a", 0, CUDA)])


@no_device
def test_upkeep_refusals(splash):
    check(splash, "splash_paged_compact", BAD_PAIR + [
        ("B", 0, INVALID), ("moves", 0, INVALID), ("moves", 1 << 31, UNSUPPORTED), ("src", None, INVALID),
        ("src", OK_PTR + 2, INVALID), ("src_stride", -1, INVALID), ("start", None, INVALID), ("block_table", None, INVALID),
        ("block_table_stride", -1, INVALID), ("max_pages", 0, INVALID), ("max_pages", 1 << 28, UNSUPPORTED),
        ("reserved", 1, INVALID)])
    check(splash, "splash_paged_copy", BAD_PAIR + [("count", 0, INVALID), ("copies", None, INVALID),
                                                   ("copies", OK_PTR + 2, INVALID)])
    check(splash, "splash_paged_remap", [(n, None, INVALID) for n in (
        "block_table new_table parents keep room refs refs_out copies short_pages workspace").split()] + [
        (n, OK_PTR + 2, INVALID) for n in "block_table new_table parents keep room refs refs_out copies short_pages".split()] + [
        ("struct_bytes", 8, INVALID), ("workspace", OK_PTR + 8, INVALID), ("workspace_bytes", 100, INVALID),
        ("num_rows", -1, INVALID), ("new_rows", 0, INVALID), ("max_pages", 0, INVALID), ("num_pages", 0, INVALID),
        ("num_pages", 1 << 31, UNSUPPORTED), ("page_size", 24, UNSUPPORTED), ("num_rows", 1 << 30, UNSUPPORTED), ("new_table_stride", 3, INVALID), ("block_table_stride", -1, INVALID)])
    a = remap_args()
    a.max_pages = a.new_table_stride = 1 << 28
    assert status(splash, "splash_paged_remap", a) == UNSUPPORTED
    a = remap_args()  # no old table at all
    a.num_rows, a.block_table = 0, None
    assert status(splash, "splash_paged_remap", a) == CUDA


@no_device
def test_upkeep_refuses_what_overlaps(splash):
    a = compact_args()
    a.v_cache = a.k_cache
    assert status(splash, "splash_paged_compact", a) == INVALID
    rows, cols, MIB = 3, 4, 1 << 20
    # (the new table's place and stride in entries, behind the old one's, which is 2 rows of 4 every 4)
    for offset, stride, old_stride, new_rows, want in (
            (0, 4, 4, rows, INVALID), (7, 4, 4, rows, INVALID), (8, 4, 4, rows, CUDA), (-11, 4, 4, rows, INVALID), (-12, 4, 4, rows, CUDA),
            (4, 8, 8, rows, CUDA), (3, 8, 8, rows, INVALID), (5, 8, 8, rows, INVALID), (-4, 8, 8, rows, CUDA), (-3, 8, 8, rows, INVALID),
            (4, 9, 8, rows, INVALID), (4, 4, 8, 1, CUDA), (2, 4, 0, 1, INVALID), (4, 4, 0, 1, CUDA)):
        a = remap_args()
        a.new_table, a.new_table_stride, a.block_table_stride, a.new_rows = OK_PTR + 4 * offset, stride, old_stride, new_rows
        assert status(splash, "splash_paged_remap", a) == want, (offset, stride, old_stride, new_rows)
    check(splash, "splash_paged_remap", [("refs_out", OK_PTR + 4, INVALID), ("refs_out", OK_PTR - 4 * 99, INVALID),
                                         ("refs_out", OK_PTR + 400, CUDA), ("refs_out", OK_PTR + MIB, CUDA),
                                         ("new_table_stride", (1 << 29) + 1, UNSUPPORTED),
                                         ("block_table_stride", (1 << 29) + 1, UNSUPPORTED)])


def test_workspace_sizes(splash):
    n = ctypes.c_size_t(0)

    def tree(B=4, Hq=32, Hkv=8, T=20, dqk=128, dv=128, max_pages=8192, page=16, kind=0, window=-1):
        return splash.lib().splash_paged_tree_decode_workspace_size(B, Hq, Hkv, T, dqk, dv, max_pages, page, kind, window,
                                                                    ctypes.byref(n))
    assert tree() == 0 and tree(T=64) == 0 and tree(window=0) == 0 and tree(T=1, max_pages=1) == 0
    q = torch.zeros(4, 32, 20, 128)
    cache = torch.zeros(2, 8, 16, 128, dtype=torch.bfloat16)
    assert tree() == 0 and splash.paged_tree_decode_workspace_size(q, cache, cache, torch.zeros(4, 8192)) == n.value
    assert tree(B=0) == INVALID and tree(kind=2) == INVALID and tree(window=-2) == INVALID
    assert tree(Hkv=7) == SHAPE and tree(T=65) == UNSUPPORTED and tree(dqk=64) == UNSUPPORTED and tree(page=20) == UNSUPPORTED
    assert splash.lib().splash_paged_tree_decode_workspace_size(4, 32, 8, 1, 128, 128, 8192, 16, 0, -1, None) == INVALID
    size = splash.paged_remap_workspace_size(1000, 10)
    assert size >= 4 * 1000 and size % 16 == 0
    for pages, rows, want in ((0, 1, INVALID), (1, 0, INVALID), (1 << 31, 1, UNSUPPORTED)):
        assert splash.lib().splash_paged_remap_workspace_size(pages, rows, ctypes.byref(n)) == want


def test_a_window_past_every_key_is_none(splash):
    """Sizes and their limits do not overflow next to the end of int64."""
    n = ctypes.c_size_t(0)

    def tree(window, B=4, Hq=32, Hkv=8, T=20, max_pages=8192):
        n.value = 0
        status = splash.lib().splash_paged_tree_decode_workspace_size(B, Hq, Hkv, T, 128, 128, max_pages, 16, 0, window, ctypes.byref(n))
        return status, n.value
    for window in (2 ** 63 - 1, 2 ** 63 - 64, 2 ** 63 - 65, 2 ** 62, 8192 * 16, 8192 * 16 - 1):
        for T in (1, 4, 5, 20, 64):
            assert tree(window, T=T) == tree(-1, T=T) and tree(window, T=T)[0] == 0
        # 2^31 steps and starts of segments: 65535 sequences x 4095 heads x (1 + 9)
        for heads in (4095, 4096):
            assert tree(window, B=65535, Hq=heads, Hkv=heads, T=1, max_pages=1)[0] == UNSUPPORTED


def test_the_longest_lists(splash):
    """Each kernel's own limit: more than 16 rows of a KV head have 64-key steps and 256 rows a
    group, up to 16 rows also the 16-key steps of paged_decode."""
    n = ctypes.c_size_t(0)

    def size(name, T, max_pages, page, Hq=64, window=-1):
        return getattr(splash.lib(), f"splash_paged_{name}_workspace_size")(256, Hq, 8, T, 128, 128, max_pages, page, 0, window,
                                                                            ctypes.byref(n))
    # 8 rows x 64: (16 pages + 9) x 256 sequences x 8 heads x 2 groups
    assert size("tree_decode", 64, 65536, 16) == 0
    assert size("tree_decode", 64, 32767, 1024) == 0 and size("tree_decode", 64, 32768, 1024) == UNSUPPORTED
    # ... or (window + 64) / 64 + 3 steps
    assert size("tree_decode", 64, 65536, 1024, window=64 * 524274) == 0
    for window in (64 * 524275, 2 ** 63 - 1, -1):
        assert size("tree_decode", 64, 65536, 1024, window=window) == UNSUPPORTED
    # 17 rows: one group; 16 rows: (pages + 1) x 256 sequences x 8 heads
    assert size("tree_decode", 17, 1048575, 16, Hq=8) == 0
    for name in ("tree_decode", "decode"):
        assert size(name, 16, 1048574, 16, Hq=8) == 0 and size(name, 16, 1048575, 16, Hq=8) == UNSUPPORTED
        assert size(name, 16, 1048575, 16, Hq=8, window=16 * 1048571) == 0
        assert size(name, 16, 1048575, 16, Hq=8, window=16 * 1048572) == UNSUPPORTED


def test_axis_maps(splash):
    assert splash.rope_axis_map((2, 1, 3)) == bytes([0, 0, 1, 2, 2, 2])
    assert splash.rope_axis_map((2, 1, 3), cycled=True) == bytes([0, 1, 2, 0, 2, 2])
    assert splash.rope_axis_map([8]) == bytes(8)
    for bad in ((), (3, -1)):
        with pytest.raises(ValueError):
            splash.rope_axis_map(bad)


def rope_call():
    return dict(q=bf16(2, 4, 8, 64), k=bf16(2, 2, 8, 64), positions=i32(3, 2, 8), table=torch.zeros(8, 64), axes=bytes(32))


def append_call():
    return dict(k=bf16(2, 2, 8, 64), v=bf16(2, 2, 8, 64), k_cache=bf16(5, 2, 16, 64), v_cache=bf16(5, 2, 16, 64),
                block_table=i32(2, 3), positions=i32(2, 8), rot_positions=i32(3, 2, 8), table=torch.zeros(8, 64),
                axes=bytes(32), q=bf16(2, 4, 8, 64))


def tree_call():
    return dict(q=bf16(2, 4, 6, 64), k_cache=bf16(5, 2, 16, 64), v_cache=bf16(5, 2, 16, 64), block_table=i32(2, 3),
                seq_lens=i32(2), parents=i32(2, 6), scale=0.125)


def compact_call():
    return dict(k_cache=bf16(5, 2, 16, 64), v_cache=bf16(5, 2, 16, 64), block_table=i32(2, 3), src=i32(2, 4), start=i32(2))


def remap_call():
    return dict(block_table=i32(2, 3), parents=i32(4), keep=i32(4), room=i32(4), refs=i32(9), page_size=16)


def copy_call():
    return dict(k_cache=bf16(5, 2, 16, 64), v_cache=bf16(5, 2, 16, 64), copies=i32(4, 3))


def bad_axes(name):
    return [(name, i32(2, 8)), (name, i32(3, 2, 7)), (name, i32(3, 1, 8)), (name, i32(3, 2, 8).long()), (name, i32(0, 2, 8)),
            (name, i32(3, 2, 16)[..., ::2]), ("axes", [0] * 32), ("axes", bytes(31)), ("axes", None)]


TOKENS = [x for x in BAD_TOKENS if x[0] != "positions"]
PAIR = [x for x in BAD_CACHE if x[0] in ("k_cache", "v_cache")]
BINDING = [
    ("rope_axes_fwd", rope_call, TOKENS + bad_axes("positions")),
    ("paged_append_axes", append_call, BAD_TOKENS + BAD_CACHE + bad_axes("rot_positions") + [("table", None)]),
    ("paged_append_axes", lambda: e4m3(append_call), BAD_SCALES),
    ("paged_tree_decode", tree_call, BAD_CACHE + [
        ("q", bf16(2, 4, 6, 128)), ("q", bf16(2, 4, 64)), ("block_table", i32(3, 3)), ("seq_lens", i32(3)),
        ("parents", i32(2, 5)), ("parents", i32(3, 6)), ("parents", i32(2, 6).long()), ("parents", i32(6, 2).t()),
        ("parents", None), ("out", bf16(2, 4, 6, 32)), ("lse", torch.zeros(2, 4))]),
    ("paged_tree_decode", lambda: e4m3(tree_call), BAD_SCALES),
    ("paged_compact", compact_call, PAIR + [
        ("block_table", i32(3)), ("src", i32(3, 4)), ("src", i32(2, 4).long()), ("src", i32(2)), ("src", i32(4, 2).t()),
        ("start", i32(3)), ("start", i32(4)[::2]), ("start", i32(2).long())]),
    ("paged_remap", remap_call, [
        ("block_table", i32(3)), ("parents", i32(4, 1)), ("parents", i32(4).long()), ("keep", i32(3)), ("room", i32(8)[::2]),
        ("refs", i32(9, 1)), ("refs", i32(9).long()), ("new_table", i32(4, 2)), ("new_table", i32(3, 4).t()),
        ("refs_out", i32(8)), ("copies", i32(4, 2)), ("copies", i32(3, 3)), ("short", i32(2)),
        ("workspace", torch.zeros(64, 2, dtype=torch.uint8)[:, 0]), ("page_size", 1 << 40)]),
    ("paged_copy", copy_call, PAIR + [("copies", i32(4, 2)), ("copies", i32(3, 4).t()), ("copies", i32(12)),
                                      ("copies", i32(4, 3).long())]),
]


@pytest.mark.parametrize("name, make, bad", BINDING, ids=[f"{i}-{x[0]}" for i, x in enumerate(BINDING)])
def test_the_binding_refuses_wrong_tensors(splash, name, make, bad):
    f = getattr(splash, name)

    def error(x):
        with pytest.raises(ValueError) as e:
            f(**x)
        return str(e.value)
    assert "current CUDA device" in error(make())  # CPU tensors: all else is right
    for member, value in bad:
        x = {**make(), member: value}
        assert "current CUDA device" not in error(x), (member, error(x))
        assert error(x) == error({**x, "stream": 0}), member


def test_the_binding_refuses_outputs_without_inputs(splash):
    x = rope_call()
    with pytest.raises(ValueError, match="k_out without k"):
        splash.rope_axes_bwd(x["q"], None, x["positions"], x["table"], x["axes"], dk_out=x["k"])
    x = append_call()
    q = x.pop("q")
    with pytest.raises(ValueError, match="q_out without q"):
        splash.paged_append_axes(**x, q_out=q)
