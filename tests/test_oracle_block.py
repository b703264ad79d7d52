"""Pins of oracle/block_oracle.py (CPU): gradients against central differences, states
that continue, hand-computed values, and the 8-bit rounding against torch's."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as O


def directional(f, args, grads, i, rng, step=1e-6):
    """(difference quotient, gradient) of scalar f along a random direction of argument i."""
    v = rng.standard_normal(args[i].shape)
    up, down = list(args), list(args)
    up[i], down[i] = args[i] + step * v, args[i] - step * v
    return (f(*up) - f(*down)) / (2 * step), (grads[i] * v).sum()


def check(f, args, grads, seed):
    rng = np.random.default_rng(seed)
    for i in range(len(args)):
        if grads[i] is None or args[i].size == 0:
            continue
        a, b = directional(f, args, grads, i, rng)
        assert abs(a - b) <= 1e-6 * max(1.0, abs(a), abs(b)), (i, a, b)


@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_norm_gradients(eps):
    rng = np.random.default_rng(1)
    x, w, dy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    dh, dw = O.rms_norm_bwd(x, w, dy, eps)
    check(lambda x, w: (O.rms_norm(x, w, eps) * dy).sum(), [x, w], [dh, dw.sum(0)], 2)


def test_norm_with_unit_weights_is_the_l2_norm():
    x = np.random.default_rng(3).standard_normal((5, 16))
    y = O.rms_norm(x, np.full(16, 1 / 4.0), 0.0)
    assert np.allclose(np.linalg.norm(y, axis=-1), 1.0)
    assert np.all(O.rms_norm(np.zeros((1, 4)), np.ones(4), 0.0) == 0)


def test_e4m3_rounding_is_torchs():
    v = np.concatenate([np.linspace(-448, 448, 40001), np.linspace(-0.05, 0.05, 20001)]).astype(np.float32)
    t = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(O.e4m3_round(v.astype(np.float64)), t)


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("T,K", [(1, 4), (2, 4), (9, 3), (5, 1), (0, 3)])
def test_conv_gradients(T, K, act):
    rng = np.random.default_rng(T * 10 + K)
    C = 3
    args = [rng.standard_normal(s) for s in ((T, C), (C, K), (C,), (K - 1, C))]
    dy, df = rng.standard_normal((T, C)), rng.standard_normal((K - 1, C))

    def f(*a):
        y, s = O.conv(*a, act)
        return (y * dy).sum() + (s * df).sum()
    check(f, args, O.conv_bwd(*args, act, dy, df), 4)


def test_conv_by_hand_and_in_two_pieces():
    x = np.array([[1.0], [2.0], [3.0]])
    y, s = O.conv(x, np.array([[10.0, 1.0]]), np.array([0.5]), np.array([[7.0]]), False)
    assert np.allclose(y[:, 0], [70 + 1 + 0.5, 10 + 2 + 0.5, 20 + 3 + 0.5]) and s[0, 0] == 3
    rng = np.random.default_rng(5)
    x, w, b, s0 = (rng.standard_normal(n) for n in ((11, 2), (2, 4), (2,), (3, 2)))
    y, s = O.conv(x, w, b, s0, True)
    y1, s1 = O.conv(x[:4], w, b, s0, True)
    y2, s2 = O.conv(x[4:], w, b, s1, True)
    assert np.allclose(np.concatenate([y1, y2]), y) and np.allclose(s2, s)


def scan_inputs(seed, T, C, N, gate):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal((T, C)), 0.3 * rng.random((T, C)), -rng.random((C, N)) * 3,
            rng.standard_normal((T, C, N)), rng.standard_normal((T, C, N)), rng.standard_normal(C),
            rng.standard_normal((T, C)) if gate else None, rng.standard_normal((C, N))]


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("T,N", [(1, 1), (7, 3), (12, 5)])
def test_scan_gradients(T, N, gate):
    a = scan_inputs(T + N, T, 2, N, gate)
    rng = np.random.default_rng(6)
    dy, df = rng.standard_normal(a[0].shape), rng.standard_normal(a[7].shape)
    g = O.scan_bwd(*a, dy, df)

    def f(*v):
        v = list(v)
        if not gate:
            v.insert(6, None)
        y, h, _ = O.scan(*v)
        return (y * dy).sum() + (h * df).sum()
    grads = [g[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dh0")]
    keep = [i for i in range(8) if gate or i != 6]
    check(f, [a[i] for i in keep], [grads[i] for i in keep], 7)


def test_scan_by_hand_and_in_two_pieces():
    x, dt = np.array([[2.0], [1.0]]), np.array([[0.5], [1.0]])
    A, B, C = np.array([[-1.0]]), np.array([[[3.0]], [[1.0]]]), np.array([[[1.0]], [[2.0]]])
    y, h, _ = O.scan(x, dt, A, B, C, np.array([0.25]), None, np.array([[4.0]]))
    h1 = 4 * np.exp(-0.5) + 3.0
    h2 = h1 * np.exp(-1.0) + 1.0
    assert np.allclose(y[:, 0], [h1 + 0.5, 2 * h2 + 0.25]) and np.allclose(h, h2)
    a = scan_inputs(8, 9, 3, 4, True)
    y, h, _ = O.scan(*a)
    cut = lambda lo, hi, h0: [v[lo:hi] if i in (0, 1, 3, 4, 6) else h0 if i == 7 else v for i, v in enumerate(a)]
    y1, h1, _ = O.scan(*cut(0, 5, a[7]))
    y2, h2, _ = O.scan(*cut(5, 9, h1))
    assert np.allclose(np.concatenate([y1, y2]), y) and np.allclose(h2, h)


def test_magnitudes_bound_the_values():
    a = scan_inputs(9, 10, 3, 4, True)
    dy, df = np.random.default_rng(1).standard_normal((10, 3)), np.ones((3, 4))
    for lo, hi in ((O.scan(*a), O.scan(*a, mag=True)),
                   (O.scan_bwd(*a, dy, df).values(), O.scan_bwd(*a, dy, df, mag=True).values())):
        for v, m in zip(lo, hi):
            assert np.all(np.abs(v) <= m * (1 + 1e-12))


def test_group_layouts():
    rng = np.random.default_rng(2)
    Bm = rng.standard_normal((2, 2, 5, 3))               # G = 2 groups of 4 heads' channels
    s = O.spread(Bm, 1, 1, 4, 4, 6)
    assert s.shape == (3, 24, 3) and np.array_equal(s[0, 7], Bm[1, 0, 1]) and np.array_equal(s[2, 23], Bm[1, 1, 3])
    d = rng.standard_normal((3, 24, 3))
    assert np.allclose(O.gather(d, 4, 2, 6)[1], d[:, 12:].sum(1))
