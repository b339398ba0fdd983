"""The oracle of the RMS norm and of the layer in 8-bit integers, pinned by closed forms, brute force
and differences (CPU)."""
import numpy as np
import pytest

import oracle
from oracle import q8_oracle as Q


@pytest.mark.parametrize("T", range(1, 17))
def test_planes_and_back(T):
    g = np.random.default_rng(T)
    v = g.standard_normal((3, 5, T))
    pl = Q.planes(v, T)
    ks, where = Q.frequencies(T)
    spectrum = np.fft.fft(v, axis=2)
    assert len(ks) == T // 2 + 1 and sorted(sum(where, [])) == list(range(T))
    for k, w in zip(ks, where):
        assert np.allclose(pl[w[0]], spectrum[..., k].real, atol=1e-12)
        assert np.allclose(pl[w[1]] if len(w) == 2 else 0.0, spectrum[..., k].imag, atol=1e-12)
    assert np.allclose(Q.values(pl, T), v, atol=1e-12)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 12])
def test_codes(T):
    g = np.random.default_rng(T)
    v = g.standard_normal((4, 7, T)).astype(np.float16)
    v[2] = 0.0
    pl = Q.planes(v, T)
    codes, scales = Q.encode(pl, T)
    assert np.abs(codes.astype(int)).max() == 127 and not codes[:, 2].any()
    assert (scales > 0).all()
    back = Q.decode(codes, scales, T)
    for f, w in enumerate(Q.frequencies(T)[1]):
        assert (np.abs(back[w] - pl[w]) <= 0.5001 * scales[:, f][:, None]).all()


@pytest.mark.parametrize("T", [1, 2, 4])
def test_codes_follow_the_group(T):
    """A cyclic shift of the group axis of whole numbers permutes and negates the codes, scales stay."""
    g = np.random.default_rng(7)
    v = g.integers(-500, 500, (3, 6, T)).astype(np.float64)
    there, scales = Q.encode(Q.planes(np.roll(v, 1, axis=2), T), T)
    here, same = Q.encode(Q.planes(v, T), T)
    assert np.array_equal(scales, same)
    assert np.allclose(Q.values(Q.decode(there, scales, T), T), np.roll(Q.values(Q.decode(here, scales, T), T), 1, axis=2))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8])
def test_layer_is_the_layer(T):
    g = np.random.default_rng(T)
    x, w = g.standard_normal((6, 5, T)), g.standard_normal((4, 5, T))
    assert np.allclose(Q.layer(x, w).reshape(6, -1), oracle.fwd(x.reshape(6, -1), w), atol=1e-12)


def test_rmsnorm_gradients_against_differences():
    g = np.random.default_rng(3)
    n, c, T, eps = 4, 5, 3, 1e-5
    s, gamma, dy = g.standard_normal((n, c * T)), 1 + 0.2 * g.standard_normal(c), g.standard_normal((n, c * T))
    dres = g.standard_normal((n, c * T))
    y, h, rstd = Q.rmsnorm(s, gamma, T, eps)
    assert np.allclose((y / np.repeat(gamma, T)) ** 2 @ np.ones(c * T) / (c * T), 1.0, atol=1e-4)
    dx, dgamma = Q.rmsnorm_bwd(dy, h, rstd, gamma, T, dres)
    loss = lambda s, gamma: (Q.rmsnorm(s, gamma, T, eps)[0] * dy).sum() + (s * dres).sum()  # noqa: E731
    step = 1e-6
    for _ in range(20):
        ds, dg = g.standard_normal(s.shape), g.standard_normal(c)
        along = (loss(s + step * ds, gamma + step * dg) - loss(s - step * ds, gamma - step * dg)) / (2 * step)
        assert abs(along - ((dx * ds).sum() + (dgamma * dg).sum())) < 1e-6 * max(1.0, abs(along))
