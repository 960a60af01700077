"""The float64 references of the serving operators against what fixes them:
closed forms, the attention oracle over gathered keys, and differences."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import serving_ref as ref


def table(n, rot, base=10000.0):
    a = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate((np.cos(a), np.sin(a)), 1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot, offset, d", [(16, 0, 16), (32, 16, 64), (16, 8, 48)])
def test_rope_keeps_lengths_and_depends_on_distance_only(interleaved, rot, offset, d):
    rng = np.random.default_rng(1)
    t = table(64, rot)
    x, y = rng.normal(size=(2, 1, 1, 1, d))
    def at(v, p):
        return ref.rope(v, [[p]], t, offset, interleaved)[0, 0, 0]
    assert np.allclose(np.linalg.norm(at(x, 37)), np.linalg.norm(x), rtol=1e-14)
    # scores of rotated pairs depend on the distance of the positions
    assert np.isclose(at(x, 9) @ at(y, 4), at(x, 45) @ at(y, 40), rtol=1e-12)
    assert np.array_equal(at(x, 0), x[0, 0, 0]) and np.array_equal(at(x, -5), x[0, 0, 0])
    back = ref.rope(ref.rope(x, [[11]], t, offset, interleaved), [[11]], t, offset, interleaved, inverse=True)
    assert np.allclose(back, x, rtol=0, atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient_equals_differences(interleaved):
    rng = np.random.default_rng(2)
    t = table(10, 16)
    x, g = rng.normal(size=(2, 1, 2, 3, 32))
    pos = [[7, 0, 3]]
    grad = ref.rope(g, pos, t, 8, interleaved, inverse=True)
    for i in [(0, 0, 0, 9), (0, 1, 2, 17), (0, 1, 0, 31), (0, 0, 2, 8)]:
        e = np.zeros_like(x)
        e[i] = 0.5
        diff = np.sum(g * (ref.rope(x + e, pos, t, 8, interleaved) - ref.rope(x - e, pos, t, 8, interleaved)))
        assert np.isclose(diff, grad[i], rtol=1e-12, atol=1e-13)


def test_e4m3_steps():
    assert ref.e4m3_step(np.array([448.0, 1.0, 1.9, 2.0 ** -6, 2.0 ** -9, 0.0])).tolist() == \
        [32.0, 0.125, 0.125, 2.0 ** -9, 2.0 ** -9, 2.0 ** -9]


@pytest.mark.parametrize("window, cap", [(-1, 0.0), (5, 0.0), (0, 3.0)])
def test_decode_equals_the_attention_oracle_over_gathered_keys(window, cap):
    rng = np.random.default_rng(3)
    page, n, Lq, Hq, Hkv, d = 16, 37, 3, 4, 2, 64
    def bf16(*shape):
        return torch.from_numpy(rng.normal(size=shape)).bfloat16().double().numpy()
    kc, vc = bf16(8, Hkv, page, d), bf16(8, Hkv, page, d)
    q = bf16(1, Hq, n, d)
    bt = [[5, 2, 7]]
    k = kc[bt[0]].transpose(1, 0, 2, 3).reshape(1, Hkv, -1, d)[:, :, :n]
    v = vc[bt[0]].transpose(1, 0, 2, 3).reshape(1, Hkv, -1, d)[:, :, :n]
    O, L = oracle.attention(*(torch.from_numpy(np.ascontiguousarray(x)).bfloat16() for x in (q, k, v)),
                            oracle.MaskSpec(True, window, -1), 0.125, cap)
    out, lse, _, _ = ref.decode(q[:, :, n - Lq:], kc, vc, bt, [n], 0.125, cap, window)
    assert np.allclose(out, O.reshape(1, Hq, n, d)[:, :, n - Lq:], rtol=0, atol=1e-12)
    assert np.allclose(lse, L.reshape(1, Hq, n)[:, :, n - Lq:], rtol=0, atol=1e-12)


def test_decode_without_keys_and_append_of_padding():
    q = np.ones((1, 1, 2, 4))
    out, lse, _, _ = ref.decode(q, np.ones((1, 1, 16, 4)), np.ones((1, 1, 16, 4)), [[0]], [1], 1.0)
    assert not out[0, 0, 0].any() and math.isinf(lse[0, 0, 0]) and np.allclose(out[0, 0, 1], 1)
    cache, written = ref.append(np.zeros((2, 1, 16, 4)), np.ones((1, 1, 3, 4)), [[1]], [[3, -1, 4]])
    assert written.sum() == 2 and written[1, 3] and written[1, 4] and cache.sum() == 8
