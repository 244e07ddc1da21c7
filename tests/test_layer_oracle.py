"""The 64-bit definitions of the linear-attention layer and its norms against
independent formulations: sums over all pairs of tokens, torch's own norms, and
central differences for every gradient."""
import numpy as np
import pytest
import torch

from oracle import layer


def _case(seed, T=7, H=4, G=2, dk=3, dv=5):
    r = np.random.RandomState(seed)
    return (r.randn(T, H, dk), r.randn(T, G, dk), r.randn(T, G, dv), np.log(r.uniform(0.2, 0.99, H)), 0.7,
            r.randn(H, dk, dv))


def test_recurrence_is_the_sum_over_pairs():
    q, k, v, g, a, s0 = _case(1)
    T, H, G = 7, 4, 2
    o, fin = layer.linattn(q, k, v, g, a, s0)
    for h in range(H):
        lam, j = np.exp(g[h]), h // (H // G)
        for t in range(T):
            want = a * lam ** (t + 1) * q[t, h] @ s0[h]
            for s in range(t + 1):
                want = want + a * lam ** (t - s) * (q[t, h] @ k[s, j]) * v[s, j]
            np.testing.assert_allclose(o[t, h], want, rtol=1e-12, atol=1e-12)
        want = lam ** T * s0[h] + sum(lam ** (T - 1 - s) * np.outer(k[s, j], v[s, j]) for s in range(T))
        np.testing.assert_allclose(fin[h], want, rtol=1e-12, atol=1e-12)


def test_recurrence_splits():
    q, k, v, g, a, s0 = _case(2)
    o, fin = layer.linattn(q, k, v, g, a, s0)
    o1, f1 = layer.linattn(q[:3], k[:3], v[:3], g, a, s0)
    o2, f2 = layer.linattn(q[3:], k[3:], v[3:], g, a, f1)
    np.testing.assert_allclose(np.concatenate([o1, o2]), o, rtol=1e-12)
    np.testing.assert_allclose(f2, fin, rtol=1e-12)


def _differences(f, x, grad, rng):
    """A random direction's central difference against the gradient's part along it."""
    d = rng.randn(*x.shape)
    e = 1e-5
    num = (f(x + e * d) - f(x - e * d)) / (2 * e)
    assert abs(num - np.sum(grad * d)) <= 1e-7 * max(1.0, abs(num))


def test_linattn_gradients_by_differences():
    q, k, v, g, a, s0 = _case(3)
    r = np.random.RandomState(9)
    do, df = r.randn(7, 4, 5), r.randn(4, 3, 5)

    def loss(q=q, k=k, v=v, s0=s0):
        o, f = layer.linattn(q, k, v, g, a, s0)
        return np.sum(o * do) + np.sum(f * df)
    dq, dk, dv, d0 = layer.linattn_bwd(q, k, v, g, a, do, s0, df)
    for name, x, gr in (("q", q, dq), ("k", k, dk), ("v", v, dv), ("s0", s0, d0)):
        _differences(lambda y: loss(**{name: y}), x, gr, r)


@pytest.mark.parametrize("first", [False, True])
def test_gated_norm_against_torch_and_differences(first):
    r = np.random.RandomState(4)
    x, z, w, dy = r.randn(5, 12), 3 * r.randn(5, 12), r.randn(12), r.randn(5, 12)
    tx, tz = torch.from_numpy(x), torch.nn.functional.silu(torch.from_numpy(z))
    a = (tx * tz if first else tx).view(5, 3, 4)
    want = (torch.nn.functional.rms_norm(a, (4,), eps=1e-3).view(5, 12) * torch.from_numpy(w)).numpy()
    np.testing.assert_allclose(layer.gated_norm(x, z, w, 3, 1e-3, first), want if first else want * tz.numpy(), rtol=1e-10)
    dx, dz, dw = layer.gated_norm_bwd(x, z, w, dy, 3, 1e-3, first)
    f = lambda x=x, z=z, w=w: np.sum(dy * layer.gated_norm(x, z, w, 3, 1e-3, first))  # noqa: E731
    for name, v, gr in (("x", x, dx), ("z", z, dz), ("w", w, dw)):
        _differences(lambda y: f(**{name: y}), v, gr, r)


def test_residual_norm_against_torch_and_differences():
    r = np.random.RandomState(5)
    x, res, w, c, dy, dr = (r.randn(6, 9), r.randn(6, 9), r.randn(9), r.randn(9), r.randn(6, 9), r.randn(6, 9))
    y, s = layer.residual_norm(x, res, w, c, 0.3, 1e-4)
    np.testing.assert_allclose(s, res + 0.3 * c * x, rtol=1e-12)
    want = torch.nn.functional.rms_norm(torch.from_numpy(s), (9,), eps=1e-4).numpy() * w
    np.testing.assert_allclose(y, want, rtol=1e-10)
    dx, dres, dw, dc = layer.residual_norm_bwd(s, w, dy, dr, x, c, 0.3, 1e-4)

    def f(x=x, res=res, w=w, c=c):
        y, s = layer.residual_norm(x, res, w, c, 0.3, 1e-4)
        return np.sum(dy * y) + np.sum(dr * s)
    for name, v, gr in (("x", x, dx), ("res", res, dres), ("w", w, dw), ("c", c, dc)):
        _differences(lambda u: f(**{name: u}), v, gr, r)
