"""Pins of the fp64 oracle's operators around a layer: closed forms, differences and
invariants."""
import numpy as np

from oracle import ref


def test_adamw_first_step_is_the_gradients_sign():
    """Without moments the first step's m / sqrt(v) is the gradient's sign."""
    g = np.array([3.0, -2e-3, 5e-9, 0.0])
    p, m, v = ref.adamw(np.ones(4), g, np.zeros(4), np.zeros(4), 1, 0.1, eps=0.0 + 1e-30)
    assert np.allclose(p, 1 - 0.1 * np.sign(g)) and np.allclose(m, 0.1 * g) and np.allclose(v, 1e-3 * g * g)
    assert np.allclose(ref.adamw(2 * np.ones(4), 0 * g, 0 * g, 0 * g, 1, 0.1, decay=0.5)[0], 1.9)


def test_adamw_code_values_round_to_themselves():
    """Every code's value has that code whatever the fraction, and the values grow with
    their codes by steps of a factor of 9/8 at most above the first octave."""
    exps = np.array([100], dtype=np.uint8)
    for top, codes in ((13, np.arange(0, 121)), (29, np.arange(0, 249))):
        x = ref.adamw_values(codes, exps, top)
        assert (np.diff(x) > 0).all() and (x[9:] / x[8:-1] <= 9 / 8).all() and x[0] == 0
        assert x[8 * top + 8] == 2.0 ** (100 - 127) and x[1] == 2.0 ** (100 - 127 - top - 3)
        for r in (0.0, 0.5, 1 - 2.0 ** -16):
            assert (ref.adamw_codes(x, exps, top, r) == codes).all()


def test_adamw_codes_keep_the_mean():
    """Rounding by fractions is unbiased: the mean over all 2^16 of them is the value."""
    exps = np.array([127], dtype=np.uint8)
    r = np.arange(65536) / 65536.0
    for top, xs in ((13, (0.7, 1.3, 1.9999, 3e-4, 2e-5)), (29, (0.7, 1.0627, 3e-6, 1e-9, 3e-10))):
        for x in xs:
            block = np.full(256, x)
            got = np.concatenate([ref.adamw_values(ref.adamw_codes(block, exps, top, r[i:i + 256]), exps, top) for i in range(0, 65536, 256)])
            assert abs(got.mean() - x) <= 2.0 ** -16 * max(x / 8, 2.0 ** (-top - 3))


def test_adamw_random_is_uniform():
    """Means and variances of both fractions, and their correlation with each other, the
    next value's and the next step's: within 5 standard deviations."""
    n = 1 << 16
    rows = [ref.adamw_random(n, t, i, s) for t, i, s in ((1, 0, 0), (2, 0, 0), (1, 1, 0), (1, 0, 1))]
    flat = [f for pair in rows for f in pair]
    for k, f in enumerate(flat):
        assert abs(f.mean() - 0.5) < 5 * np.sqrt(1 / 12 / n) and abs(f.var() - 1 / 12) < 5 * np.sqrt(1 / 180 / n)
        for h in flat[:k] + [np.roll(f, 1)]:
            assert abs(np.corrcoef(f, h)[0, 1]) < 5 / np.sqrt(n)


def test_block_norm_backward_matches_differences():
    r = np.random.default_rng(4)
    n, w, eps = 4, 6, 1e-3
    for kind in ("layer", "rms"):
        for post in (True, False):
            for gates in (None, r.standard_normal(w), r.standard_normal((n, w))):
                x = {"b": r.standard_normal((n, w)) + 1, "residual": r.standard_normal((n, w)), "gate": gates}
                x["gamma_post"], x["beta_post"] = (r.standard_normal(w), r.standard_normal(w) if kind == "layer" else None) if post else (None, None)
                x["gamma"], x["beta"] = r.standard_normal(w), r.standard_normal(w) if kind == "layer" else None
                dy, dsum = r.standard_normal((n, w)), r.standard_normal((n, w))

                def forward(x):
                    s, m1, r1 = ref.block_norm(x["b"], x["residual"], x["gate"], 0.7, 1.3, post, kind, x["gamma_post"], x["beta_post"], eps)
                    y, m2, r2 = ref.row_norm(s, kind, eps)
                    y = y * x["gamma"] + (0 if x["beta"] is None else x["beta"])
                    return s, y, np.stack([m1, r1, m2, r2], 1)

                def loss(x):
                    s, y, _ = forward(x)
                    return (dy * y).sum() + (dsum * s).sum()

                s, _, stats = forward(x)
                got = ref.block_norm_backward(dy, x["b"], s, stats, gates, 0.7, 1.3, post, kind, x["gamma_post"], x["beta_post"], x["gamma"], dsum)
                for name, a in x.items():
                    if a is None:
                        continue
                    for i in np.ndindex(a.shape):
                        up, dn = dict(x, **{name: a.copy()}), dict(x, **{name: a.copy()})
                        up[name][i] += 1e-5
                        dn[name][i] -= 1e-5
                        assert abs((loss(up) - loss(dn)) / 2e-5 - got[name][i]) < 1e-6, (kind, post, name)


def test_gated_ffn_backward_matches_differences():
    r = np.random.default_rng(6)
    for act in ("silu", "gelu"):
        args = [r.standard_normal((3, 4)), r.standard_normal((10, 4)), r.standard_normal((4, 5))]
        dy = r.standard_normal((3, 4))
        for k, grad in enumerate(ref.gated_ffn_backward(*args, dy, act)):
            for i in np.ndindex(args[k].shape):
                up, dn = [a.copy() for a in args], [a.copy() for a in args]
                up[k][i] += 1e-5
                dn[k][i] -= 1e-5
                diff = ((dy * ref.gated_ffn(*up, act)[0]).sum() - (dy * ref.gated_ffn(*dn, act)[0]).sum()) / 2e-5
                assert abs(diff - grad[i]) < 1e-7, (act, k)


def test_gated_activations():
    g = np.array([-40.0, -1.0, 0.0, 1.0, 40.0])
    a, s = ref.gated_act(g, "silu")
    assert np.allclose(a, [0, -0.2689414213699951, 0, 0.7310585786300049, 40]) and s[2] == 0.5 and np.isclose(s[4], 1)
    a, s = ref.gated_act(g, "gelu")
    assert np.allclose(a, [0, -0.15865525393145707, 0, 0.8413447460685429, 40]) and s[2] == 0.5 and np.isclose(s[4], 1)


def test_adamw_codes_of_finite_values_are_finite():
    """The largest exponent's codes stop below 2^128, whatever the fraction; one exponent lower
    they go on to 2^127."""
    x = np.array([2.0 ** 127 * 15 / 8, np.finfo(np.float32).max, 2.0 ** 127])
    for top in (13, 29):
        for r in (0.0, 0.5, 1 - 2.0 ** -16):
            codes = ref.adamw_codes(x, np.array([254], dtype=np.uint8), top, r)
            assert np.isfinite(ref.adamw_values(codes, np.array([254], dtype=np.uint8), top).astype(np.float32)).all()
            assert list(codes) == [8 * top + 15, 8 * top + 15, 8 * top + 8]
        assert ref.adamw_codes(x[1:2] / 2, np.array([253], dtype=np.uint8), top, 0.99)[0] == 8 * top + 16
