"""Refusals of the serving calls with a stream given: the same ValueError for
the same wrong tensors as without one, before anything is allocated."""
import pytest
import torch

from test_serving_abi import BINDING, append_call, decode_call, rope_call


@pytest.fixture(scope="module")
def splash():
    from block_sparse_flash_gb300 import build as b
    b.build()
    import block_sparse_flash_gb300 as m
    return m


def error(f, x):
    with pytest.raises(ValueError) as e:
        f(**x)
    return str(e.value)


@pytest.mark.parametrize("name, make, bad", BINDING, ids=[f"{i}-{x[0]}" for i, x in enumerate(BINDING)])
def test_refusals_do_not_depend_on_the_stream(splash, name, make, bad):
    f = getattr(splash, name)
    for member, value in [(None, None)] + bad:
        x = make()
        if member:
            x[member] = value
        assert error(f, x) == error(f, {**x, "stream": 0}), member


@pytest.mark.parametrize("name, make, changes", [
    ("rope_fwd", rope_call, {"q": None}), ("rope_bwd", lambda: {"d" + n if n in "qk" else n: t for n, t in rope_call().items()},
                                           {"dk": 3}),
    ("paged_append", append_call, {"q": torch.zeros(4)}), ("paged_append", append_call, {"k": None}),
    ("paged_decode", decode_call, {"q": torch.zeros(4)}), ("paged_decode", decode_call, {"v_cache": torch.zeros(2)}),
    ("paged_decode", decode_call, {"k_cache": torch.zeros(5, 2, 16, 64).half()}),
    ("paged_decode", decode_call, {"block_table": torch.zeros(3, dtype=torch.int32)})])
def test_tensors_of_no_shape_at_all(splash, name, make, changes):
    f, x = getattr(splash, name), {**make(), **changes}
    assert error(f, x) == error(f, {**x, "stream": 0})


def test_workspace_size_refuses_by_value(splash):
    x = decode_call()
    for member, value in (("q", torch.zeros(4)), ("k_cache", x["k_cache"].half()), ("v_cache", torch.zeros(2)),
                          ("block_table", torch.zeros(3, dtype=torch.int32))):
        y = {**{n: x[n] for n in ("q", "k_cache", "v_cache", "block_table")}, member: value}
        with pytest.raises(ValueError):
            splash.paged_decode_workspace_size(**y)
