"""Pins of the softmax-attention oracle to facts fixed by the mathematics (CPU)."""

import math

import numpy as np
import pytest

from oracle import attn_oracle as ora


def draw(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_rotary_keeps_norms_and_depends_on_distances():
    f, s = ora.rotary_freqs(16)
    assert s == 1.0 and f[0] == 1.0 and np.all(np.diff(f) < 0)
    x, y = draw(1, 1, 1, 16), draw(1, 1, 1, 16, seed=1)
    for il in (False, True):
        at = lambda v, p: ora.rotary(v, np.array([[p]]), f, interleaved=il)  # noqa: E731
        assert np.allclose(np.linalg.norm(at(x, 7)), np.linalg.norm(x))
        assert np.allclose((at(x, 11) * at(y, 4)).sum(), (at(x, 107) * at(y, 100)).sum())
        assert np.allclose(ora.rotary(at(x, 5), np.array([[5]]), f, interleaved=il, inverse=True), x)
    z = np.array([1.0, 0.0, 0.0, 0.0]).reshape(1, 1, 1, 4)
    out = ora.rotary(z, np.array([[1]]), np.array([math.pi / 2, 0.0]))
    assert np.allclose(out.ravel(), [0, 0, 1, 0])
    out = ora.rotary(z, np.array([[1]]), np.array([math.pi / 2, 0.0]), interleaved=True)
    assert np.allclose(out.ravel(), [0, 1, 0, 0])


def test_rotary_scalings():
    f, _ = ora.rotary_freqs(64)
    lin, _ = ora.rotary_freqs(64, scaling="linear", factor=4.0)
    assert np.allclose(lin, f / 4)
    ntk, _ = ora.rotary_freqs(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], f[-1] / 4)      # the slowest channel is interpolated by the factor
    y, s = ora.rotary_freqs(64, scaling="yarn", factor=4.0, trained=4096)
    assert np.isclose(y[0], f[0]) and np.isclose(y[-1], f[-1] / 4) and np.isclose(s, 0.1 * math.log(4) + 1)
    assert np.all(y <= f + 1e-15) and np.all(y >= f / 4 - 1e-15)


def test_attention_limits():
    v = draw(1, 5, 1, 4)
    q, k = np.zeros((1, 5, 1, 4)), np.zeros((1, 5, 1, 4))
    o, lse = ora.attn_forward(q, k, v, 1.0)
    assert np.allclose(o[0, :, 0], np.cumsum(v[0, :, 0], 0) / np.arange(1, 6)[:, None])   # equal scores: the running mean
    assert np.allclose(lse[0, 0], np.log(np.arange(1, 6)))
    o, _ = ora.attn_forward(q, k, v, 1.0, window=1)
    assert np.allclose(o, v)                                                             # each sees itself
    o, lse = ora.attn_forward(q, k[:, :2], v[:, :2], 1.0)
    assert np.all(o[0, :3] == 0) and np.all(lse[0, 0, :3] == -np.inf)                      # before the first key
    assert np.allclose(o[0, 3], v[0, 0])


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3)])
def test_attention_gradient_against_differences(causal, window):
    q, k, v, w = draw(1, 5, 4, 3), draw(1, 6, 2, 3, seed=1), draw(1, 6, 2, 3, seed=2), draw(1, 5, 4, 3, seed=3)
    kw = dict(causal=causal, window=window, q_len=[4], kv_len=[5])
    grads = ora.attn_backward(q, k, v, w, 0.7, **kw)
    loss = lambda: float((ora.attn_forward(q, k, v, 0.7, **kw)[0] * w).sum())  # noqa: E731
    for x, g in zip((q, k, v), grads):
        for i in range(0, x.size, 3):
            keep, h = x.flat[i], 1e-6
            x.flat[i] = keep + h
            up = loss()
            x.flat[i] = keep - h
            down = loss()
            x.flat[i] = keep
            assert abs((up - down) / (2 * h) - g.flat[i]) < 1e-7


def test_e4m3_values_and_rounding():
    v = ora.e4m3_value(np.arange(256))
    assert v[0x7e] == 448 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and np.isnan(v[0x7f]) and v[0xfe] == -448
    fin = v[np.isfinite(v)]
    assert np.array_equal(ora.e4m3(fin), fin)
    pos = np.sort(fin[fin >= 0])
    pos = np.unique(pos)
    mid = (pos[1:] + pos[:-1]) / 2
    even = np.where(np.arange(len(mid)) % 2 == 0, pos[:-1], pos[1:])     # a tie goes to the even mantissa
    assert np.array_equal(ora.e4m3(mid), even)
    assert np.array_equal(ora.e4m3(np.nextafter(mid, 1e9)), pos[1:])
    assert np.array_equal(ora.e4m3(np.array([460.0, 1e9, -np.inf])), [448, 448, -448])


def test_page_scales():
    s = lambda *x: ora.page_scale(np.array(x))  # noqa: E731
    assert s(448.0) == 1.0 and s(448.0001) == 2.0 and s(224.0) == 0.5 and s(1e-3, -3.5) == 2.0 ** -7
    assert s(0.0) == 2.0 ** -100 and s(np.inf, 448.0) == 1.0 and s(3e38) == 2.0 ** 120


def test_cache_round_trip_and_growth():
    K = ora.Cache(4, 1, 16, 4)
    table = np.array([[2, 0]])
    x = draw(1, 20, 1, 4)
    K.append(x[:, :3], table, [0])
    K.append(x[:, 3:4] * 1000, table, [3])                # the scale grows: the first tokens move to it
    K.append(x[:, 4:], table, [4])
    got, have = K.tokens(table[0], 20)
    want = x[0].copy()
    want[3] *= 1000
    assert have.all()
    s = np.where(np.arange(20) < 16, K.scale[2, 0], K.scale[0, 0])[:, None, None]
    assert np.all(np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4 * 1.01, s * 2.0 ** -10 * 2.01))


def test_step_equals_attention_over_the_cached_values():
    K, V = ora.Cache(6, 2, 16, 8), ora.Cache(6, 2, 16, 8)
    table = np.array([[4, 1, 3], [0, 5, 2]])
    k, v, q = draw(2, 40, 2, 8, seed=1), draw(2, 40, 2, 8, seed=2), draw(2, 3, 4, 8, seed=3)
    n = [40, 21]
    K.append(k, table, [0, 0], n)
    V.append(v, table, [0, 0], n)
    got = ora.attn_step(q, K, V, table, [37, 18], 0.3, window=9)
    for b in range(2):
        kk, vv = K.tokens(table[b], n[b])[0][None], V.tokens(table[b], n[b])[0][None]
        want, _ = ora.attn_forward(q[b:b + 1], kk, vv, 0.3, window=9)
        assert np.allclose(got[b], want[0])
