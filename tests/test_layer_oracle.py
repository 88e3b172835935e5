"""Pins of the float64 oracle of the operators around the attention (CPU):
gradients against differences, the recurrence and the shared prefix against
other forms of the same quantity."""
import numpy as np
import pytest

from oracle import layer_oracle as L
from oracle import taylor_oracle as T


def _differences(f, x, dy, step=1e-6):
    """d<dy, f>/dx entry by entry, central."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = step
        g[i] = (dy * (f(x + e) - f(x - e))).sum() / (2 * step)
    return g


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,eps", [(6, 6, 0.0), (5, 2, 0.3), (4, 0, 0.0)])
def test_norm_rope_gradient_is_that_of_differences(d, rot, eps, interleaved):
    rng = np.random.default_rng(d)
    x, w = rng.standard_normal((2, 3, 2, d)), 1 + 0.2 * rng.standard_normal(d)
    pos = np.array([[0, 1, 7], [100, 3, -4]])
    freqs = 10.0 ** -np.arange(rot // 2)
    dy = rng.standard_normal((2, 2, 3, d))
    dx, dw = L.norm_rope_grad(x, dy, freqs, pos, w, interleaved, eps)
    np.testing.assert_allclose(dx, _differences(lambda z: L.norm_rope(z, freqs, pos, w, interleaved, eps), x, dy),
                               rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(dw, _differences(lambda z: L.norm_rope(x, freqs, pos, z, interleaved, eps), w, dy),
                               rtol=1e-6, atol=1e-7)


def test_rotated_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((1, 1, 1, 8)), rng.standard_normal((1, 1, 1, 8))
    freqs = 100.0 ** (-np.arange(4) / 4)
    score = lambda p, r: (L.norm_rope(q, freqs, [[p]]) * L.norm_rope(k, freqs, [[r]])).sum()  # noqa: E731
    np.testing.assert_allclose(score(5, 3), score(1005, 1003), rtol=1e-12)
    np.testing.assert_allclose(np.linalg.norm(L.norm_rope(q, freqs, [[9]])), 1.0, rtol=1e-14)


@pytest.mark.parametrize("coupled", [False, True])
def test_gated_gradient_is_that_of_differences(coupled):
    rng = np.random.default_rng(3)
    gate, x, h0 = rng.standard_normal((2, 5, 3)), rng.standard_normal((2, 5, 3)), rng.standard_normal((2, 3))
    dh, dl = rng.standard_normal((2, 5, 3)), rng.standard_normal((2, 3))
    lengths = [5, 3]

    def loss_of(g, u, s):
        h, last = L.gated_scan(g, u, coupled, s, lengths)
        return np.concatenate([(dh * h).ravel(), (dl * last).ravel()])

    dgate, dx, dh0 = L.gated_scan_grad(gate, x, dh, coupled, h0, lengths, dl)
    np.testing.assert_allclose(dgate, _differences(lambda z: loss_of(z, x, h0), gate, 1.0), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dx, _differences(lambda z: loss_of(gate, z, h0), x, 1.0), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dh0, _differences(lambda z: loss_of(gate, x, z), h0, 1.0), rtol=1e-6, atol=1e-8)


def test_gated_scan_closed_form_and_continuation():
    """Equal gates: a geometric sum; and a scan in two parts is the scan of the whole."""
    gate, x = np.full((1, 40, 2), 0.7), np.ones((1, 40, 2))
    h, last = L.gated_scan(gate, x, coupled=True)
    a = 1 / (1 + np.exp(-0.7))
    np.testing.assert_allclose(h[0, :, 0], 1 - a ** np.arange(1, 41), rtol=1e-12)
    h1, s1 = L.gated_scan(gate[:, :13], x[:, :13])
    h2, s2 = L.gated_scan(gate[:, 13:], x[:, 13:], h0=s1)
    np.testing.assert_allclose(np.concatenate([h1, h2], 1), h, rtol=1e-13)
    np.testing.assert_allclose(s2, last, rtol=1e-13)


@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_shared_prefix_is_attention_over_the_whole_sequence(n):
    rng = np.random.default_rng(n)
    H, P, L_, d, dv, tau = 2, 20, 6, 3, 4, 1.5
    unit = lambda *s: (lambda z: z / np.linalg.norm(z, axis=-1, keepdims=True))(rng.standard_normal(s))  # noqa: E731
    kp, vp = unit(1, H, P, d), rng.standard_normal((1, H, P, dv))
    kc, vc = unit(2, H, L_, d), rng.standard_normal((2, H, L_, dv))
    q = unit(2, H, d)
    lengths = [0, L_ - 1]
    state = T.state_of(kp, vp, n)[0]
    k = np.stack([kc[b, :, lengths[b]] for b in range(2)])
    v = np.stack([vc[b, :, lengths[b]] for b in range(2)])
    out = L.shared_prefix_decode(q, k, v, state, kc, vc, lengths, n, tau)
    for b in range(2):
        keys = np.concatenate([kp[0], kc[b, :, :lengths[b] + 1]], 1)[None]
        values = np.concatenate([vp[0], vc[b, :, :lengths[b] + 1]], 1)[None]
        queries = np.repeat(q[b][None, :, None], keys.shape[2], 2)
        want = T.attention_direct(queries, keys, values, n, tau)[0, :, -1]
        np.testing.assert_allclose(out[b], want, rtol=1e-12)
