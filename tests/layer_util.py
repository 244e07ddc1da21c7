"""Tolerances of the layer's GPU tests, from the roundings that the kernels make.

* A result stored in bf16 is off by at most half a step, 2^-8 of its value (fp32
  2^-24).
* The bf16 path of linear attention rounds the scores and, where a query reads
  it, the state to bf16: each term of a result's sum is off by at most 2^-8 of
  its size. The sum of the terms' sizes, `mag`, is the same operator run on the
  inputs' absolute values.
* Sums in fp32 of n terms: at most n 2^-24 of mag, and 2^-22 for the weights and
  products.
The root mean square of such errors is far smaller: a rounding's is at most
2^-8 / sqrt(3), and those of many terms are independent; two roundings in a row
give 3.2e-3, and 4e-3 bounds the relative 2-norm of bf16 results. For fp32 results
it is bounded by 2^-24 sqrt(n), doubled, and 4 2^-24 for the weights.
"""
import numpy as np


def check(got, want, mag, n, bf16, what, through_bf16=False):
    got = got.detach().cpu().double().numpy() if hasattr(got, "detach") else np.asarray(got)
    want, mag = np.asarray(want), np.asarray(mag)
    assert got.shape == want.shape, f"{what}: {got.shape} {want.shape}"
    assert np.isfinite(got).all(), f"{what}: not finite"
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    step = (2.0 ** -8 if through_bf16 else 0.0) + n * 2.0 ** -24 + 2.0 ** -22
    bound = (half * np.abs(want) + step * mag) * (1 + 2.0 ** -6) + 1e-30
    err = np.abs(got - want)
    assert (err <= bound).all(), f"{what}: error {err.max():.3e}, {np.max(err / bound):.2f} of its bound"
    norm = np.linalg.norm(want)
    if norm > 0 and want.size >= 64:
        rel = np.linalg.norm(got - want) / norm
        most = 4e-3 if bf16 else 2.0 ** -23 * np.sqrt(n) + 2.0 ** -22
        assert rel <= most, f"{what}: relative 2-norm {rel:.3e} over {most:.3e}"
