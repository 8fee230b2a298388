"""The plain reference of the residual-stream calls (oracle.residual): every
backward pass against central differences of its forward, in fp64 (CPU only).

A central difference with step h has an error of h^2/6 |f'''| + 2^-52 |f| / h:
with h = 1e-5 and values of order one, about 1e-10 of both; 1e-7 leaves room
for third derivatives up to a few thousand."""

import numpy as np
import pytest

from oracle import residual as R

H, TOL = 1e-5, 1e-7


def _diff(f, a, d_out):
    """sum(d_out * f) differentiated by every element of a"""
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + H
        up = (f() * d_out).sum()
        a[i] = keep - H
        down = (f() * d_out).sum()
        a[i] = keep
        g[i] = (up - down) / (2 * H)
    return g


def test_embed_grad_by_differences():
    rng = np.random.default_rng(1)
    E, tok = rng.standard_normal((7, 4)), np.array([[3, 0, 3], [6, 3, -1]])
    d_h = rng.standard_normal((6, 4))
    got, mag, cnt = R.embed_grad(tok, d_h, 7, scale=0.5)
    assert np.abs(got - _diff(lambda: R.embed(tok, E, 0.5), E, d_h)).max() < TOL
    assert cnt.tolist() == [1, 0, 0, 3, 0, 0, 1]
    assert (mag >= np.abs(got) - 1e-15).all()


@pytest.mark.parametrize("with_gain", [False, True])
def test_add_norm_grad_by_differences(with_gain):
    rng = np.random.default_rng(2)
    x, res = rng.standard_normal((3, 8)), rng.standard_normal((3, 8))
    gain = 1.0 + 0.1 * rng.standard_normal(8) if with_gain else None
    d_y, d_sum = rng.standard_normal((3, 8)), rng.standard_normal((3, 8))
    s, r, _ = R.add_norm(x, res, gain)
    d_x, d_gain = R.add_norm_grad(d_y, s, r, gain, d_sum)

    def both():
        s, _, y = R.add_norm(x, res, gain)
        return np.concatenate([s, y])
    d_both = np.concatenate([d_sum, d_y])
    assert np.abs(d_x - _diff(both, x, d_both)).max() < TOL
    assert np.abs(d_x - _diff(both, res, d_both)).max() < TOL
    if with_gain:
        assert np.abs(d_gain - _diff(both, gain, d_both)).max() < TOL


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_ffn_grad_by_differences(kind):
    rng = np.random.default_rng(3)
    n, d, f = 4, 6, 5
    x, Wgu, Wd = rng.standard_normal((n, d)), rng.standard_normal((2 * f, d)), rng.standard_normal((d, f))
    d_y = rng.standard_normal((n, d))
    _, gu = R.ffn(x, Wgu, Wd, kind)
    got = R.ffn_grad(d_y, x, gu, Wgu, Wd, kind)
    for g, a in zip(got, (x, Wgu, Wd)):
        assert np.abs(g - _diff(lambda: R.ffn(x, Wgu, Wd, kind)[0], a, d_y)).max() < TOL


def test_gelu_is_near_the_normal_distribution_form():
    """the tanh form is within 5e-4 of g * Phi(g) (Hendrycks and Gimpel, 2016)"""
    from math import erf
    g = np.linspace(-6, 6, 601)
    phi = np.array([0.5 * (1 + erf(v / 2 ** 0.5)) for v in g])
    assert np.abs(R.act(g, "gelu")[0] - g * phi).max() < 5e-4
