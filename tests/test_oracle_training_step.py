"""Pins of the fp64 oracle's training-step operators (layer norm, orthogonalised
update, substrate step): central differences, closed forms and invariants."""
import numpy as np

from oracle import ref


def test_layer_norm_backward_matches_differences():
    r = np.random.default_rng(1)
    s = r.standard_normal((5, 7)) * 3.0 + 1.0
    gamma, beta = r.standard_normal(7), r.standard_normal(7)
    dy, ds = r.standard_normal((5, 7)), r.standard_normal((5, 7))

    def loss(s_, g_, b_):
        return (dy * ref.layer_norm(s_, g_, b_)[0]).sum() + (ds * s_).sum()

    _, mean, rstd = ref.layer_norm(s, gamma, beta)
    grads = ref.layer_norm_backward(dy, s, gamma, mean, rstd, ds)
    args, h = [s, gamma, beta], 1e-5
    for k, g in enumerate(grads):
        for i in np.ndindex(args[k].shape):
            up, dn = [a.copy() for a in args], [a.copy() for a in args]
            up[k][i] += h
            dn[k][i] -= h
            # central difference: truncation h^2 |f'''| / 6 below 1e-8 here,
            # cancellation 1e-16 |f| / h below 1e-9
            assert abs((loss(*up) - loss(*dn)) / (2 * h) - g[i]) < 1e-6


def test_layer_norm_rows_are_normalised():
    s = np.random.default_rng(2).standard_normal((9, 33)) * 5 + 2
    y, mean, rstd = ref.layer_norm(s, eps=0.0)
    assert np.allclose(y.mean(axis=1), 0, atol=1e-14) and np.allclose((y * y).mean(axis=1), 1, atol=1e-13)
    assert np.allclose(mean, s.mean(axis=1)) and np.allclose(rstd, 1 / s.std(axis=1))


def test_orthogonalize_acts_on_singular_values():
    """O = U diag(p^5(sigma / |sigma|)) V^T with the scalar polynomial iterated."""
    r = np.random.default_rng(3)
    for shape in ((6, 11), (11, 6), (5, 5)):
        g = r.standard_normal(shape)
        u, sv, vt = np.linalg.svd(g, full_matrices=False)
        x = sv / np.linalg.norm(sv)
        a, b, c = ref.NS_COEFFS
        for _ in range(5):
            x = a * x + b * x ** 3 + c * x ** 5
        o, m = ref.orthogonalize(g)
        assert m is None and np.allclose(o, (u * x) @ vt, atol=1e-12)


def test_orthogonalize_momentum():
    r = np.random.default_rng(4)
    g, m = r.standard_normal((4, 6)), r.standard_normal((4, 6))
    o, m1 = ref.orthogonalize(g, m, mu=0.9, nesterov=True)
    assert np.allclose(m1, 0.9 * m + g) and np.allclose(o, ref.orthogonalize(g + 0.9 * m1)[0])
    assert np.allclose(ref.orthogonalize(g, m, mu=0.9, nesterov=False)[0], ref.orthogonalize(0.9 * m + g)[0])


def test_substrate_step_codes_are_nearest():
    """The code is the nearest of -1, 0, 1 to W' / scale."""
    w = np.random.default_rng(5).standard_normal((8, 32)).astype(np.float32)
    o = np.random.default_rng(6).standard_normal((8, 32))
    w1, codes, scale = ref.substrate_step(w, o, step=0.1, decay=0.01)
    assert w1.dtype == np.float32 and np.allclose(w1, 0.99 * w - 0.1 * o, atol=1e-6)
    d = np.abs(w1[..., None] / scale - np.array([-1.0, 0.0, 1.0]))
    assert (d.argmin(axis=-1) - 1 == codes).all() and abs(scale - np.abs(w1).mean()) < 1e-6
    assert (ref.substrate_step(np.zeros((2, 16), np.float32))[1] == 0).all()
    # a tie goes to 0: eight weights of magnitude 3 and eight of 1 have mean 2
    tie = np.array([[3.0] * 4 + [-3.0] * 4 + [1.0] * 4 + [-1.0] * 4], np.float32)
    assert list(ref.substrate_step(tie)[1][0]) == [1] * 4 + [-1] * 4 + [0] * 8
