"""The plain references of the operators around the scan against things other than themselves:
library convolutions, hand-worked values and central differences (CPU only)."""
import numpy as np
import pytest

from . import block_ref as ref


def test_packed_conv_is_numpy_convolve_per_sequence():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((11, 3)), rng.standard_normal((3, 4))
    cu = [0, 4, 4, 11]
    out, _, _ = ref.packed_conv(x, w, None, cu, None, None, None, False)
    for lo, hi in ((0, 4), (4, 11)):
        for d in range(3):
            full = np.convolve(x[lo:hi, d], w[d, ::-1])[:hi - lo]
            np.testing.assert_allclose(out[lo:hi, d], full, rtol=1e-12, atol=1e-12)


def test_packed_conv_split_anywhere_continues_from_its_state():
    rng = np.random.default_rng(2)
    x, w, b = rng.standard_normal((9, 2)), rng.standard_normal((2, 4)), rng.standard_normal(2)
    whole, _, _ = ref.packed_conv(x, w, b, [0, 9], np.zeros((1, 3, 2)), None, [0], True)
    for cut in range(10):
        st = np.zeros((1, 3, 2))
        first, st1, _ = ref.packed_conv(x[:cut], w, b, [0, cut], st, None, [0], True)
        second, _, _ = ref.packed_conv(x[cut:], w, b, [0, 9 - cut], st1 if cut else st, None, [cut > 0], True)
        np.testing.assert_allclose(np.concatenate([first, second]), whole, rtol=1e-12)


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("shape", [(2, 5, 3, 4), (1, 2, 2, 4), (1, 1, 1, 1), (2, 7, 1, 2)])
def test_conv_gradient_formulas_against_differences(shape, act):
    bt, length, d, width = shape
    rng = np.random.default_rng(3)
    x, w, b = rng.standard_normal((bt, length, d)), rng.standard_normal((d, width)), rng.standard_normal(d)
    dout = rng.standard_normal((bt, length, d))
    grads, _ = ref.conv_backward(x, w, b, dout, act)
    loss = lambda: float((dout * ref.conv_forward(x, w, b, act)).sum())
    eps = 1e-5  # central differences of a smooth function: error about eps^2 |f'''| / 6
    for arr, g in zip((x, w, b), grads):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + eps
            up = loss()
            arr[i] = keep - eps
            down = loss()
            arr[i] = keep
            assert abs((up - down) / (2 * eps) - g[i]) <= 1e-7 * (1 + abs(g[i]))


def test_packed_scan_hand_worked():
    """One channel, one state, A = 0: the state is a running sum of step * B * x."""
    x = np.array([[1.0], [2.0], [3.0], [5.0]])
    delta = np.array([[1.0], [0.5], [2.0], [1.0]])
    B, C = np.array([[2.0], [4.0], [1.0], [1.0]]), np.array([[1.0], [1.0], [3.0], [2.0]])
    y, st = ref.packed_scan(x, delta, np.zeros((1, 1)), B, C, None, None, [0, 2, 4], np.array([[[10.0]], [[7.0]]]),
                            None, [False, True], None, False)
    np.testing.assert_array_equal(y[:, 0], [2.0, 6.0, 39.0, 36.0])
    np.testing.assert_array_equal(st[:, 0, 0], [6.0, 18.0])


def test_packed_scan_agrees_with_the_oracle(oracle_lib):
    """Each packed sequence is a dense scan of its own."""
    rng = np.random.default_rng(4)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    t, d, n, cu = 12, 3, 4, [0, 5, 5, 12]
    x, delta, z, A, B, C, D = f(t, d), np.abs(f(t, d)) * 0.3, f(t, d), -np.abs(f(d, n)), f(t, n), f(t, n), f(d)
    state = f(3, d, n)
    y, st = ref.packed_scan(x, delta, A, B, C, D, z, cu, state, [2, 1, 0], [True, True, False], None, False)
    for s, h0, slot in ((0, state[2:3], 2), (2, None, 0)):
        r = slice(cu[s], cu[s + 1])
        yo, ho = oracle_lib.selective_scan(x[None, r], delta[None, r], A, B[None, r], C[None, r], D, z[None, r], h0)
        np.testing.assert_allclose(y[r], np.asarray(yo)[0], rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(st[slot], np.asarray(ho)[0], rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(st[1], state[1].astype(np.float64))


def differences(loss, arrays, eps=1e-5):
    """Central differences of loss() in every entry of the arrays, which it reads."""
    res = []
    for arr in arrays:
        g = np.zeros_like(arr)
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + eps
            up = loss()
            arr[i] = keep - eps
            down = loss()
            arr[i] = keep
            g[i] = (up - down) / (2 * eps)
        res.append(g)
    return res


@pytest.mark.parametrize("norm_first", [False, True])
@pytest.mark.parametrize("group,with_z", [(6, True), (2, True), (3, False), (1, True)])
def test_gated_norm_gradient_formulas_against_differences(group, with_z, norm_first):
    rng = np.random.default_rng(5)
    x, w, dout = rng.standard_normal((3, 6)), rng.standard_normal(6), rng.standard_normal((3, 6))
    z = rng.standard_normal((3, 6)) if with_z else None
    eps = 0.1  # large, so that single-channel groups have a gradient
    loss = lambda: float((dout * ref.gated_norm(x, w, z, group, eps, norm_first)[0]).sum())
    g = ref.gated_norm_grad(dout, x, w, z, ref.gated_norm(x, w, z, group, eps, norm_first)[1], group, norm_first)
    names = ("dx", "dweight") + (("dz",) if with_z else ())
    for name, d in zip(names, differences(loss, (x, w) + ((z,) if with_z else ()))):
        np.testing.assert_allclose(g[name][0], d, rtol=1e-6, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("post,scaled,first", [(True, True, False), (True, False, False), (False, True, False),
                                               (False, False, False), (True, True, True)])
def test_residual_norm_gradient_formulas_against_differences(post, scaled, first):
    rng = np.random.default_rng(6)
    x, w, dout, dnew = (rng.standard_normal(s) for s in ((3, 5), 5, (3, 5), (3, 5)))
    h = None if first else rng.standard_normal((3, 5))
    wp = rng.standard_normal(5) if post else None
    scale = rng.standard_normal(5) if scaled else None
    fwd = lambda: ref.residual_norm(x, w, h, wp, scale, 0.7, 0.01)
    loss = lambda: float((dout * fwd()[0]).sum() + (dnew * fwd()[1]).sum())
    _, new, r, rp, _ = fwd()
    g = ref.residual_norm_grad(dout, dnew, x, w, new, r, wp, scale, rp, 0.7)
    given = {"dx": x, "dweight": w, "dresidual": h, "dpost_weight": wp, "dscale": scale}
    given = {k: v for k, v in given.items() if v is not None}
    for (name, _), d in zip(given.items(), differences(loss, given.values())):
        np.testing.assert_allclose(g[name][0], d, rtol=1e-6, atol=1e-7, err_msg=name)


def test_norms_of_hand_worked_rows():
    out, r = ref.gated_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), None, 2, 0.0, False)
    np.testing.assert_allclose(out, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    out, new, *_ = ref.residual_norm(np.array([[1.0, -1.0]]), np.ones(2), np.array([[2.0, 5.0]]), np.array([2.0, 2.0]),
                                     np.array([0.5, 1.0]), 1.0, 0.0)
    np.testing.assert_allclose(new, [[3.0, 3.0]])
    np.testing.assert_allclose(out, [[1.0, 1.0]])
