"""Pins of the fp64 oracle of the gradient operators (CPU): hand values, closed forms and
central differences of every gradient."""
import numpy as np
import pytest

from oracle import gradient_oracle as go


def _rng(seed):
    return np.random.default_rng(seed)


def test_e4m3_table():
    v = go.e4m3_values()
    assert v[0x01] == 2.0 ** -9 and v[0x07] == 7 * 2.0 ** -9      # subnormals
    assert v[0x08] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7e] == 448.0
    assert v[0xb8] == -1.0 and np.isnan(v[0x7f]) and np.isnan(v[0xff])
    assert np.all(np.diff(v[:127]) > 0)


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.0000001, 1), (224.0, -1), (1.0, -8),
                                   (1.75, -8), (1.7500001, -7), (0.0, -117), (1e-40, -117),
                                   (3.4e38, 119)])
def test_block_exponent(top, e):
    assert go.act_exponent(top) == e


def test_rounding_of_a_block():
    x = np.zeros((1, 33))
    # the block's largest is 448: e = 0 and the grid near 1 has steps of 1/8
    x[0, :6] = [448, 1.0625, 1.1875, -1.07, 2.0 ** -10, 3 * 2.0 ** -10]
    x[0, 32] = 5.0                                   # its own block: 5 = 320 * 2^-6
    v, s = go.act_round(x)
    # ties go to the even fraction: 1.0625 -> 1, 1.1875 -> 1.25; 2^-10 -> 0, 3 2^-10 -> 2^-8
    assert list(v[0, :6]) == [448, 1.0, 1.25, -1.125, 0.0, 2.0 ** -8]
    assert v[0, 32] == 5.0 and list(s[0]) == [127, 127 - 6]


def test_a_block_with_nan_reads_as_nan():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.nan, -np.inf
    v, s = go.act_round(x)
    assert np.all(np.isnan(v[0, :32])) and np.all(v[0, 32:] == 1) and s[0, 0] == 255
    assert np.all(np.isnan(v[1, 32:])) and np.all(v[1, :32] == 1) and s[1, 1] == 255


def test_rounded_values_are_within_half_a_step():
    x = _rng(1).standard_normal((40, 96)) * 10.0 ** _rng(2).integers(-20, 20, (40, 1))
    v, s = go.act_round(x)
    top = np.repeat(np.abs(x).reshape(40, 3, 32).max(2), 32, 1)
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -16 * top))
    q = np.zeros((40, 96), np.uint8)                 # bytes found by value give it back
    vals = go.e4m3_values()
    f = np.repeat(2.0 ** (s.astype(float) - 127), 32, 1)
    for i in range(40):
        for j in range(96):
            q[i, j] = int(np.flatnonzero(vals == v[i, j] / f[i, j])[0])
    assert np.array_equal(go.act_value(q, s, 96), v)


def test_norm_hand_values():
    x, y = np.array([[3.0, 1.0]]), np.array([[0.0, 2.0]])
    # rms(y) = 1 / sqrt(2) at eps = 0 in effect; z = post * y / sqrt(2)
    h, u = go.norm_forward(x, y, pre_gain=np.array([1.0, 2.0]), post_gain=np.array([1.0, 0.5]),
                           gate=np.array([1.0, 2.0]), residual_scale=0.5, eps=1e-300)
    assert np.allclose(h, [[3.0, 1.0 + 0.5 * 2 * 0.5 * 2 / np.sqrt(2)]], rtol=1e-15)
    r = 1 / np.sqrt((9 + h[0, 1] ** 2) / 2)
    assert np.allclose(u, [[3 * r, 2 * h[0, 1] * r]], rtol=1e-15)
    h, u = go.norm_forward(x, y, gate=np.array([2.0, 3.0]), residual_scale=2.0)
    assert np.array_equal(h, [[3.0, 13.0]])          # no post norm: x + s gate y


@pytest.mark.parametrize("post_norm", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_norm_gradients_against_differences(post_norm, gated):
    r = _rng(3)
    t, d = 3, 7
    p = {"x": r.standard_normal((t, d)), "y": r.standard_normal((t, d)),
         "pre_gain": r.standard_normal(d)}
    if post_norm:
        p["post_gain"] = r.standard_normal(d)
    if gated:
        p["gate"] = r.standard_normal(d)
    du, dh = r.standard_normal((t, d)), r.standard_normal((t, d))
    kw = dict(residual_scale=0.7, eps=1e-3, post_norm=post_norm)

    def loss(q):
        h, u = go.norm_forward(q["x"], q["y"], **{k: v for k, v in q.items() if k not in "xy"}, **kw)
        return np.sum(h * dh) + np.sum(u * du)

    h, _ = go.norm_forward(p["x"], p["y"], **{k: v for k, v in p.items() if k not in "xy"}, **kw)
    got = go.norm_backward(h, p["y"], du=du, dh=dh,
                           **{k: v for k, v in p.items() if k not in "xy"}, **kw)
    for name, v in p.items():
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            step = 1e-5
            hi = {**p, name: v.copy()}
            lo = {**p, name: v.copy()}
            hi[name][i] += step
            lo[name][i] -= step
            num[i] = (loss(hi) - loss(lo)) / (2 * step)
        assert np.allclose(got["d" + name], num, rtol=1e-6, atol=1e-7), name


def test_norm_gradient_is_orthogonal_to_its_row():
    """u does not change when h is scaled (eps negligible): <dx, h> = 0 without dh."""
    r = _rng(4)
    h, du = r.standard_normal((5, 9)), r.standard_normal((5, 9))
    dx = go.norm_backward(h, du=du, eps=1e-300)["dx"]
    assert np.all(np.abs(np.sum(dx * h, 1)) < 1e-12)


def test_embedding_and_its_gradient_are_adjoint():
    r = _rng(5)
    table, dout = r.standard_normal((6, 4)), r.standard_normal((9, 4))
    ids = np.array([5, 0, 0, -1, 6, 3, 0, 5, 2])
    out = go.embed_lookup(table, ids, 1.5)
    assert np.all(out[3] == 0) and np.all(out[4] == 0) and np.array_equal(out[0], 1.5 * table[5])
    g = go.embed_grad(ids, dout, 6, 1.5)
    assert np.isclose(np.sum(out * dout), np.sum(g * table))
    assert np.all(g[1] == 0) and np.all(g[4] == 0)
    assert np.allclose(g[0], 1.5 * (dout[1] + dout[2] + dout[6]))


def test_weight_gradient_against_differences():
    r = _rng(6)
    a, d, w = r.standard_normal((5, 3)), r.standard_normal((5, 4)), r.standard_normal((3, 4))
    g = go.weight_grad(a, d)
    assert np.array_equal(go.weight_grad(a, d, True), g.T)
    for i in np.ndindex(w.shape):
        hi, lo = w.copy(), w.copy()
        hi[i] += 1e-4
        lo[i] -= 1e-4
        assert np.isclose((np.sum(a @ hi * d) - np.sum(a @ lo * d)) / 2e-4, g[i])
