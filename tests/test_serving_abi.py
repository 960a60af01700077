"""Refusals of the serving calls (rope, paged_append, paged_decode) on the CPU:
the C entry points reject invalid arguments before touching the GPU, and the
binding rejects tensors that do not fit.  No call here reaches a launch: there
is no device."""
import ctypes

import pytest
import torch

OK_PTR = 1 << 20  # 16-byte aligned, never read


@pytest.fixture(scope="module")
def splash():
    from block_sparse_flash_gb300 import build as b
    b.build()
    import block_sparse_flash_gb300 as m
    return m


class View(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p)] + [(n, ctypes.c_int64) for n in ("a", "b", "c")]


def fields(*groups):
    out = [("struct_bytes", ctypes.c_uint64)]
    for kind, names in groups:
        out += [(n, kind) for n in names.split()]
    return out


P, I64, I32, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class RopeArgs(ctypes.Structure):
    _fields_ = fields((View, "q q_out k k_out"), (P, "positions"), (I64, "positions_stride_b"), (P, "table"),
                      (I64, "table_rows L"), (I32, "B Hq Hkv d rot_dim rot_offset interleaved inverse"))


class AppendArgs(ctypes.Structure):
    _fields_ = fields((View, "q q_out k k_out v k_cache v_cache"), (P, "k_scale v_scale block_table"),
                      (I64, "block_table_stride"), (P, "positions"), (I64, "positions_stride_b"), (P, "seq_ids"),
                      (I64, "seq_ids_stride_b"), (P, "table"), (I64, "table_rows L num_pages"),
                      (I32, "B Hq Hkv dqk dv num_seqs max_pages page_size cache_type rot_dim rot_offset interleaved"))


class DecodeArgs(ctypes.Structure):
    _fields_ = fields((View, "q k_cache v_cache"), (P, "k_scale v_scale block_table"), (I64, "block_table_stride"),
                      (P, "seq_lens out lse workspace"), (ctypes.c_uint64, "workspace_bytes"),
                      (I64, "num_pages window_left"), (I32, "B Hq Hkv Lq dqk dv max_pages page_size cache_type"),
                      (F32, "scale softcap"), (I32, "reserved"))


def dense(H, L, d):
    return View(OK_PTR, H * L * d, L * d, d)


def rope_args():
    a = RopeArgs(q=dense(4, 8, 128), q_out=dense(4, 8, 128), k=dense(2, 8, 128), k_out=dense(2, 8, 128),
                 positions=OK_PTR, positions_stride_b=8, table=OK_PTR, table_rows=8, L=8, B=2, Hq=4, Hkv=2, d=128,
                 rot_dim=128)
    a.struct_bytes = ctypes.sizeof(a)
    return a


def append_args():
    a = AppendArgs(q=dense(4, 8, 128), q_out=dense(4, 8, 128), k=dense(2, 8, 128), v=dense(2, 8, 128),
                   k_cache=dense(2, 16, 128), v_cache=dense(2, 16, 128), block_table=OK_PTR, block_table_stride=4,
                   positions=OK_PTR, positions_stride_b=8, table=OK_PTR, table_rows=8, L=8, num_pages=9, B=2, Hq=4,
                   Hkv=2, dqk=128, dv=128, num_seqs=2, max_pages=4, page_size=16, rot_dim=128)
    a.struct_bytes = ctypes.sizeof(a)
    return a


def decode_args():
    a = DecodeArgs(q=dense(4, 1, 128), k_cache=dense(2, 16, 128), v_cache=dense(2, 16, 128), block_table=OK_PTR,
                   block_table_stride=4, seq_lens=OK_PTR, out=OK_PTR, lse=OK_PTR, workspace=OK_PTR,
                   workspace_bytes=1 << 40, num_pages=9, window_left=-1, B=2, Hq=4, Hkv=2, Lq=1, dqk=128, dv=128,
                   max_pages=4, page_size=16, scale=0.1)
    a.struct_bytes = ctypes.sizeof(a)
    return a


def with_pages(a, n):
    a.max_pages = n
    return a


def call(splash, name, a):
    return getattr(splash.lib(), name)(bytes(a), None)


def refused(splash, name, make, changes):
    """Each (member, value, status): applied alone to valid arguments."""
    for member, value, status in changes:
        a = make()
        where = a
        *path, last = member.split(".")
        for x in path:
            where = getattr(where, x)
        setattr(where, last, value)
        assert call(splash, name, a) == status, (name, member, value)


INVALID, SHAPE, UNSUPPORTED, CUDA = 1, 2, 3, 4


def test_valid_arguments_reach_the_device(splash):
    """The library compares struct_bytes with its own sizeof: valid arguments
    get past every check and fail only at the missing device."""
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for name, make in (("splash_rope", rope_args), ("splash_paged_append", append_args),
                       ("splash_paged_decode", decode_args)):
        assert call(splash, name, make()) == CUDA


def test_null_arguments(splash):
    for f in (splash.lib().splash_rope, splash.lib().splash_paged_append, splash.lib().splash_paged_decode):
        assert f(None, None) == INVALID


COMMON_TOKENS = [("struct_bytes", 8, INVALID), ("B", 0, INVALID), ("L", 0, INVALID), ("L", -1, INVALID),
                 ("L", 1 << 31, UNSUPPORTED), ("positions", None, INVALID), ("positions", OK_PTR + 2, INVALID),
                 ("positions_stride_b", -8, INVALID), ("rot_dim", 0, INVALID), ("rot_dim", 24, UNSUPPORTED),
                 ("rot_dim", 144, SHAPE), ("rot_offset", 16, SHAPE), ("rot_offset", -8, INVALID),
                 ("rot_offset", 4, UNSUPPORTED), ("interleaved", 2, INVALID), ("table", OK_PTR + 4, INVALID),
                 ("table_rows", 0, INVALID), ("q_out.ptr", None, INVALID), ("q_out.ptr", OK_PTR + 8, INVALID),
                 ("q.c", 132, INVALID), ("q.a", -8, INVALID), ("q_out.b", 0, INVALID), ("q_out.c", 64, INVALID),
                 ("q_out.c", 256, INVALID)]


def test_rope_refusals(splash):
    refused(splash, "splash_rope", rope_args, COMMON_TOKENS + [
        ("Hq", 0, INVALID), ("Hkv", 0, INVALID), ("d", 0, INVALID), ("d", 120, UNSUPPORTED), ("d", 528, UNSUPPORTED),
        ("q.ptr", None, INVALID), ("k_out.ptr", None, INVALID), ("table", None, INVALID), ("inverse", 2, INVALID),
        ("Hq", 65534, UNSUPPORTED)])


def test_append_refusals(splash):
    refused(splash, "splash_paged_append", append_args, COMMON_TOKENS + [
        ("Hkv", 0, INVALID), ("dqk", 0, INVALID), ("dv", 0, INVALID), ("dv", 72, UNSUPPORTED), ("Hq", 0, INVALID),
        ("q.ptr", None, INVALID), ("k.ptr", None, INVALID), ("v.ptr", None, INVALID), ("v.c", 4, INVALID),
        ("k_cache.ptr", None, INVALID), ("v_cache.ptr", OK_PTR + 8, INVALID), ("k_cache.c", 136 + 4, INVALID),
        ("k_cache.a", 0, INVALID), ("v_cache.b", 64, INVALID), ("page_size", 0, INVALID),
        ("page_size", 8, UNSUPPORTED), ("page_size", 24, UNSUPPORTED), ("page_size", 2048, UNSUPPORTED),
        ("num_pages", 0, INVALID), ("max_pages", 0, INVALID), ("max_pages", 1 << 28, UNSUPPORTED),
        ("num_seqs", 1, SHAPE), ("cache_type", 2, INVALID), ("cache_type", 1, INVALID), ("block_table", None, INVALID),
        ("block_table_stride", -1, INVALID), ("seq_ids", OK_PTR + 1, INVALID)])


def test_append_rows_that_would_overlap_are_refused(splash):
    a = append_args()  # token-major pages: the same tensor with head and token strides exchanged
    a.k_cache = View(OK_PTR, 2 * 16 * 128, 128, 2 * 128)
    if not torch.cuda.is_available():
        assert call(splash, "splash_paged_append", a) == CUDA  # past every check
    a = append_args()
    a.k_cache = View(OK_PTR, 2 * 16 * 128, 128, 128)
    assert call(splash, "splash_paged_append", a) == INVALID


def test_decode_refusals(splash):
    long = lambda: with_pages(decode_args(), 8192)  # noqa: E731  (a call that needs a workspace)
    refused(splash, "splash_paged_decode", long, [
        ("struct_bytes", 8, INVALID), ("B", 0, INVALID), ("B", 65536, UNSUPPORTED), ("Hkv", 3, SHAPE),
        ("Lq", 0, INVALID), ("Lq", 17, UNSUPPORTED), ("dqk", 64, UNSUPPORTED), ("dv", 96, UNSUPPORTED),
        ("seq_lens", None, INVALID), ("seq_lens", OK_PTR + 2, INVALID), ("out", None, INVALID),
        ("out", OK_PTR + 8, INVALID), ("lse", None, INVALID), ("workspace", None, INVALID),
        ("workspace", OK_PTR + 8, INVALID), ("workspace_bytes", 8, INVALID), ("scale", 0.0, INVALID),
        ("scale", float("nan"), INVALID), ("scale", float("inf"), INVALID), ("softcap", float("nan"), INVALID),
        ("softcap", float("inf"), INVALID), ("window_left", -2, INVALID), ("reserved", 1, INVALID),
        ("q.ptr", None, INVALID), ("q.b", 4, INVALID), ("k_cache.ptr", None, INVALID), ("v_cache.c", 4, INVALID),
        ("cache_type", 1, INVALID), ("cache_type", -1, INVALID), ("page_size", 12, UNSUPPORTED),
        ("num_pages", 0, INVALID), ("max_pages", 0, INVALID), ("block_table", None, INVALID)])


def test_decode_limit_of_steps(splash):
    """2^31 steps of 16 keys: 65535 sequences x 2 heads x 16384 pages, unless a
    window keeps each sequence's short."""
    a = decode_args()
    a.B, a.max_pages = 65535, 16384
    assert call(splash, "splash_paged_decode", a) == UNSUPPORTED
    if not torch.cuda.is_available():
        a.window_left = 1000
        assert call(splash, "splash_paged_decode", a) == CUDA  # past every check
        a.window_left, a.max_pages = -1, 16000
        assert call(splash, "splash_paged_decode", a) == CUDA


def test_decode_workspace_size(splash):
    n = ctypes.c_size_t(0)

    def size(B=4, Hq=32, Hkv=8, Lq=1, dqk=128, dv=128, max_pages=8192, page=16, kind=0, window=-1):
        return splash.lib().splash_paged_decode_workspace_size(B, Hq, Hkv, Lq, dqk, dv, max_pages, page, kind, window,
                                                               ctypes.byref(n))
    assert size() == 0 and n.value > 0
    q = torch.zeros(4, 32, 1, 128)
    cache = torch.zeros(2, 8, 16, 128, dtype=torch.bfloat16)
    assert splash.paged_decode_workspace_size(q, cache, cache, torch.zeros(4, 8192)) == n.value
    # few and short sequences need none; many, or longer ones, do
    assert size(max_pages=32) == 0 and n.value == 0
    assert size(window=100) == 0 and n.value == 0
    assert size(B=64, max_pages=4) == 0 and n.value > 0
    assert size(B=0) == INVALID and size(kind=2) == INVALID and size(window=-2) == INVALID and size(page=0) == INVALID
    assert size(Hkv=7) == SHAPE and size(Lq=17) == UNSUPPORTED and size(dqk=64) == UNSUPPORTED
    assert size(page=20) == UNSUPPORTED and size(max_pages=1 << 28) == UNSUPPORTED
    assert splash.lib().splash_paged_decode_workspace_size(4, 32, 8, 1, 128, 128, 8192, 16, 0, -1, None) == INVALID


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def rope_call():
    return dict(q=bf16(2, 4, 8, 64), k=bf16(2, 2, 8, 64), positions=i32(2, 8), table=torch.zeros(8, 64))


def append_call():
    return dict(k=bf16(2, 2, 8, 64), v=bf16(2, 2, 8, 64), k_cache=bf16(5, 2, 16, 64), v_cache=bf16(5, 2, 16, 64),
                block_table=i32(2, 3), positions=i32(2, 8), q=bf16(2, 4, 8, 64), table=torch.zeros(8, 64))


def decode_call():
    return dict(q=bf16(2, 4, 1, 64), k_cache=bf16(5, 2, 16, 64), v_cache=bf16(5, 2, 16, 64), block_table=i32(2, 3),
                seq_lens=i32(2), scale=0.125)


def e4m3(call):
    x = call()
    x.update({n: x[n].to(torch.float8_e4m3fn) for n in ("k_cache", "v_cache")})
    x.update(k_scale=torch.ones(2), v_scale=torch.ones(2))
    return x


BAD_TOKENS = [("q", bf16(2, 4, 8, 64).float()), ("q", bf16(2, 4, 8, 128)[..., ::2]), ("q", bf16(2, 4, 64)),
              ("k", bf16(2, 2, 9, 64)), ("k", bf16(2, 2, 64)), ("k", bf16(2, 2, 8, 64).half()),
              ("positions", i32(2, 8).long()), ("positions", i32(2, 7)), ("positions", i32(3, 8)),
              ("positions", i32(8, 2).t()), ("positions", i32(2, 16)[:, ::2]), ("positions", i32(1)),
              ("table", torch.zeros(8, 64).double()), ("table", torch.zeros(64, 8).t()), ("table", torch.zeros(64)),
              ("q_out", bf16(2, 4, 8, 32)), ("k_out", bf16(2, 4, 8, 64)), ("positions", None)]
BAD_CACHE = [("k_cache", bf16(5, 2, 16, 64).half()), ("k_cache", bf16(4, 2, 16, 64)), ("v_cache", bf16(5, 2, 16)),
             ("v_cache", bf16(5, 2, 16, 128)[..., ::2]), ("v_cache", bf16(5, 2, 16, 64).to(torch.float8_e4m3fn)),
             ("k_scale", torch.ones(2)), ("block_table", i32(2, 3).long()), ("block_table", i32(3)),
             ("block_table", i32(3, 2).t()), ("block_table", [0])]
BAD_SCALES = [("k_scale", None), ("v_scale", torch.ones(3)), ("k_scale", torch.ones(2).double()),
              ("v_scale", torch.ones(4)[::2])]
BINDING = [
    ("rope_fwd", rope_call, BAD_TOKENS),
    ("paged_append", append_call, BAD_TOKENS + BAD_CACHE + [("v", bf16(2, 2, 8, 32)), ("seq_ids", i32(2, 9))]),
    ("paged_append", lambda: e4m3(append_call), BAD_SCALES),
    ("paged_decode", decode_call, BAD_CACHE + [
        ("q", bf16(2, 4, 1, 128)), ("q", bf16(2, 4, 64)), ("block_table", i32(3, 3)), ("seq_lens", i32(3)),
        ("seq_lens", i32(2).long()), ("seq_lens", i32(4)[::2]), ("out", bf16(2, 4, 1, 32)),
        ("out", bf16(2, 4, 1, 64).float()), ("lse", torch.zeros(2, 4)), ("lse", bf16(2, 4, 1)),
        ("workspace", torch.zeros(64, 2, dtype=torch.uint8)[:, 0])]),
    ("paged_decode", lambda: e4m3(decode_call), BAD_SCALES),
]


@pytest.mark.parametrize("name, make, bad", BINDING, ids=[f"{i}-{x[0]}" for i, x in enumerate(BINDING)])
def test_the_binding_refuses_wrong_tensors(splash, name, make, bad):
    f = getattr(splash, name)
    with pytest.raises(ValueError, match="current CUDA device"):
        f(**make())  # CPU tensors: all else is right
    for member, value in bad:
        x = make()
        x[member] = value
        with pytest.raises(ValueError) as e:
            f(**x)
        assert "current CUDA device" not in str(e.value), (member, str(e.value))


def test_the_binding_refuses_outputs_without_inputs(splash):
    x = rope_call()
    with pytest.raises(ValueError, match="k_out without k"):
        splash.rope_bwd(x["q"], None, x["positions"], x["table"], dk_out=x["k"])
    x = append_call()
    q = x.pop("q")
    with pytest.raises(ValueError, match="q_out without q"):
        splash.paged_append(**x, q_out=q)
    with pytest.raises(TypeError):
        splash.paged_decode(**{**decode_call(), "scale": "large"})
    with pytest.raises(ValueError):
        splash.rope_fwd(**rope_call(), rot_offset=1 << 40)


def test_the_binding_fails_loudly_when_it_is_missing(splash, monkeypatch):
    from block_sparse_flash_gb300 import build
    monkeypatch.setattr(splash, "_binding", None)
    monkeypatch.setattr(build, "binding_path", lambda: "/nonexistent/_binding.so")
    with pytest.raises(splash.SplashLibraryMissing):
        splash.rope_fwd(**rope_call())


def test_rope_table():
    import block_sparse_flash_gb300 as m
    t = m.rope_table(1000, 16, base=500.0, device="cpu")
    assert t.shape == (1000, 16) and t.dtype == torch.float32
    a = 999 * 500.0 ** (-6 / 16)
    assert abs(float(t[999, 3]) - torch.tensor(a, dtype=torch.float64).cos().item()) < 1e-7
    assert abs(float(t[999, 11]) - torch.tensor(a, dtype=torch.float64).sin().item()) < 1e-7
