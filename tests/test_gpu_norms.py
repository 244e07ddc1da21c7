"""The gated norm and the residual norm on the GPU against their formulas in 64
bits (oracle/layer.py).

Tolerances: a result is rounded to its type (half a step of its value) and
formed by a few fp32 operations; sums over a group's W columns, or over the rows,
are off by at most their count times 2^-24 of the terms' sizes, which the same
formula's parts on absolute values bound. silu takes two MUFU operations
(2^-22 each, and 2^-22 |z| for the exponent's argument)."""
import numpy as np
import pytest
import torch

from oracle import layer
from selective_state_space_40_b200 import binding as mb

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert mb.mamba_device_check() == mb.MS_OK


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def near(got, want, mag, n, dtype, what):
    """mag: a bound of the sizes of what is added up to the result, n: how many."""
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    bound = (half * np.abs(want) + (n + 32) * 2.0 ** -24 * mag) * 1.01 + 1e-30
    err = np.abs(got - want)
    assert (err <= bound).all(), f"{what}: error {err.max():.3e}, {np.max(err / bound):.2f} of its bound"


def rand(seed, *shape, dtype=F32, mul=1.0):
    return (mul * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def check_gated(x, z, w, dy, groups, eps, first, dtype):
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    X, Z, W, DY = to(x), to(z), to(w), to(dy)
    y = mb.gated_norm_fwd(X, Z, W, groups, eps, first)
    g = mb.gated_norm_bwd(X, Z, W, DY, groups, eps, first)
    torch.cuda.synchronize()
    a = [f64(t) for t in (x, z, w, dy)]
    n = x.shape[1] // groups
    zz = 0.0 if z is None else np.abs(a[1])
    want = layer.gated_norm(*a[:3], groups, eps, first)
    near(y, want, np.abs(want) * (1 + zz), n, dtype, "y")
    dx, dz, dw = layer.gated_norm_bwd(*a, groups, eps, first)
    # the sizes: |da| <= inv (|g| + |hat| mean |g hat|)
    gate, slope = (1.0, 0.0) if z is None else layer._silu(a[1])
    ww = 1.0 if w is None else np.abs(a[2])
    hat, inv = layer._norm(a[0] * gate if first else a[0], groups, eps)
    up = np.abs(a[3] if first else a[3] * gate)
    m = np.mean((up * ww * np.abs(hat)).reshape(x.shape[0], groups, -1), 2, keepdims=True)
    m = np.broadcast_to(m, (x.shape[0], groups, n)).reshape(x.shape)
    da = inv * (up * ww + np.abs(hat) * m)
    lift = 1 + zz  # the gate's own error grows with |z|
    near(g["dx"], dx, (da * np.abs(gate) if first else da) * (lift + np.max(zz)), n, dtype, "dx")
    if z is None:
        assert g["dz"] is None
    else:
        sl = np.abs(slope) + 2.0  # 1 + z (1 - sig) cancels: its parts, not its value
        near(g["dz"], dz, (da * np.abs(a[0]) if first else np.abs(a[3] * hat) * ww) * sl * (lift + np.max(zz)), n, dtype, "dz")
    near(g["dweight"], dw, np.sum(up * np.abs(hat) * (lift + 1), axis=0), n + x.shape[0], F32, "dweight")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("rows,width,groups", [(1, 1, 1), (1, 64, 1), (5, 96, 3), (300, 128, 2), (7, 33, 3), (40, 1536, 24),
                                               (9, 2560, 1), (3, 5120, 1), (130, 200, 8), (2, 4097, 1), (700, 8, 8)])
def test_gated_norm(dtype, first, rows, width, groups):
    s = rows * 31 + width
    check_gated(rand(s, rows, width, dtype=dtype), rand(s + 1, rows, width, dtype=dtype, mul=2.0), 1 + 0.3 * rand(s + 2, width),
                rand(s + 3, rows, width, dtype=dtype), groups, 1e-5, first, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,width,groups", [(1500, 130, 1), (2100, 33 * 5, 5), (700, 1503, 1), (400, 4001, 1), (333, 7 * 90, 7)])
def test_gated_norm_many_rows_of_any_width(dtype, rows, width, groups):
    s = rows + width
    check_gated(rand(s, rows, width, dtype=dtype), rand(s + 1, rows, width, dtype=dtype, mul=2.0), 1 + 0.3 * rand(s + 2, width),
                rand(s + 3, rows, width, dtype=dtype), groups, 1e-5, groups == 1, dtype)


@pytest.mark.parametrize("width", [8191, 10001, 16383, 16384])
def test_gated_norm_widest(width):
    check_gated(rand(1, 3, width, dtype=BF), rand(2, 3, width, dtype=BF), None, rand(3, 3, width, dtype=BF), 1, 1e-5, True, BF)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gated_norm_without_gate_or_weight(dtype):
    check_gated(rand(1, 20, 64, dtype=dtype), None, 1 + 0.1 * rand(2, 64), rand(3, 20, 64, dtype=dtype), 2, 1e-5, False, dtype)
    check_gated(rand(1, 20, 64, dtype=dtype), None, None, rand(3, 20, 64, dtype=dtype), 1, 1e-5, True, dtype)


def test_gated_norm_tails_and_zero_rows():
    """Gates far into both tails of silu, groups of zeros (eps decides), tiny and large values."""
    x = rand(5, 64, 64)
    x[0] = 0.0
    x[1, :32] = 0.0
    x[2] *= 1e-12
    x[3] *= 1e6
    z = torch.linspace(-120, 120, 64 * 64).view(64, 64)
    check_gated(x, z, None, rand(6, 64, 64), 2, 1e-5, False, F32)
    check_gated(x, z, None, rand(6, 64, 64), 2, 1e-5, True, F32)


def test_gated_norm_strides():
    """x, z and dy as slices of wider rows (aligned and not); y into a slice; nothing beside it written."""
    for off in (0, 8, 1):
        wide = rand(7, 50, 400, dtype=BF).to(DEV)
        x, z, dy = (wide[:, off + 128 * i: off + 128 * i + 128] for i in range(3))
        out = torch.full((50, 200), 7.0, dtype=BF, device=DEV)
        y = mb.gated_norm_fwd(x, z, None, 2, y=out[:, off:off + 128])
        ref = mb.gated_norm_fwd(x.contiguous(), z.contiguous(), None, 2)
        near(y, f64(ref), np.abs(f64(ref)) * 4, 64, BF, "strided y")
        assert (out[:, :off] == 7.0).all() and (out[:, off + 128:] == 7.0).all()
        g = mb.gated_norm_bwd(x, z, None, dy, 2)
        r = mb.gated_norm_bwd(x.contiguous(), z.contiguous(), None, dy.contiguous(), 2)
        for n in ("dx", "dz", "dweight"):
            # another layout of threads adds the sums in another order: a bf16 value may round to the next one
            assert torch.allclose(g[n].float(), r[n].float(), rtol=2.0 ** -7, atol=2e-5), n


def test_no_rows():
    e = torch.empty(0, 64, device=DEV)
    assert mb.gated_norm_fwd(e, e).shape == (0, 64)
    assert (mb.gated_norm_bwd(e, e, None, e)["dweight"] == 0).all()
    y, r = mb.residual_norm_fwd(e, e)
    assert y.shape == r.shape == (0, 64)
    g = mb.residual_norm_bwd(e, None, e, x=e, channel_scale=torch.ones(64, device=DEV))
    assert (g["dweight"] == 0).all() and (g["dchannel_scale"] == 0).all()


def check_residual(x, res, w, c, dy, dr, scale, eps, dtype, rdtype):
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    y, r = mb.residual_norm_fwd(to(x), to(res), to(w), eps, scale, to(c), residual_dtype=rdtype)
    n = x.shape[1]
    wy, wr = layer.residual_norm(f64(x), f64(res), f64(w), f64(c), scale, eps)
    size = np.abs(scale * f64(x) * (1.0 if c is None else f64(c))) + (0.0 if res is None else np.abs(f64(res)))
    near(r, wr, size, 2, rdtype, "residual_out")
    inv = layer._norm(wr, 1, eps)[1]
    near(y, wy, (size * inv + np.abs(wy)) * (1.0 if w is None else 1 + np.abs(f64(w))), n, dtype, "y")
    # the gradients start from the stored sum
    g = mb.residual_norm_bwd(r, to(w), to(dy), to(dr), to(x) if c is not None else None, eps, scale, to(c))
    torch.cuda.synchronize()
    want = layer.residual_norm_bwd(f64(r), f64(w), f64(dy), f64(dr), f64(x), f64(c), scale, eps)
    hat, inv = layer._norm(f64(r), 1, eps)
    up = np.abs(f64(dy)) * (1.0 if w is None else np.abs(f64(w)))
    d = inv * (up + np.abs(hat) * np.mean(up * np.abs(hat), 1, keepdims=True)) + (0.0 if dr is None else np.abs(f64(dr)))
    near(g["dresidual"], want[1], d, n, rdtype, "dresidual")
    near(g["dx"], want[0], abs(scale) * d * (1.0 if c is None else np.abs(f64(c))), n, dtype, "dx")
    near(g["dweight"], want[2], np.sum(np.abs(f64(dy) * hat), 0), n + x.shape[0], F32, "dweight")
    if c is None:
        assert g["dchannel_scale"] is None
    else:
        near(g["dchannel_scale"], want[3], np.sum(abs(scale) * np.abs(f64(x)) * d, 0), n + x.shape[0], F32, "dchannel_scale")


@pytest.mark.parametrize("dtype,rdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 2560), (64, 2560), (33, 100), (5, 777), (300, 128), (3, 6000), (2, 16384), (2, 9001)])
def test_residual_norm(dtype, rdtype, rows, width):
    s = rows + 7 * width
    x, res = rand(s, rows, width, dtype=dtype), rand(s + 1, rows, width, dtype=rdtype, mul=2.0)
    check_residual(x, res, 1 + 0.2 * rand(s + 2, width), 0.5 + 0.2 * rand(s + 3, width), rand(s + 4, rows, width, dtype=dtype),
                   rand(s + 5, rows, width, dtype=rdtype), 0.7, 1e-5, dtype, rdtype)


@pytest.mark.parametrize("dtype,rdtype", [(BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,width", [(2000, 398), (900, 1503), (400, 2562), (1200, 61)])
def test_residual_norm_many_rows_of_any_width(dtype, rdtype, rows, width):
    test_residual_norm(dtype, rdtype, rows, width)


@pytest.mark.parametrize("dtype,rdtype", [(BF, F32), (F32, F32)])
def test_residual_norm_without_parts(dtype, rdtype):
    x, dy = rand(1, 20, 96, dtype=dtype), rand(2, 20, 96, dtype=dtype)
    check_residual(x, None, None, None, dy, None, 1.0, 1e-5, dtype, rdtype)
    check_residual(x, rand(3, 20, 96, dtype=rdtype), None, None, dy, None, -0.5, 1e-5, dtype, rdtype)


def test_residual_norm_in_place_and_strided():
    x, res = rand(4, 40, 160, dtype=BF).to(DEV)[:, 32:], rand(5, 40, 128).to(DEV)
    y0, r0 = mb.residual_norm_fwd(x.contiguous(), res, res_scale=0.3)
    y1, r1 = mb.residual_norm_fwd(x, res, res_scale=0.3, residual_out=res)
    assert r1 is res and torch.equal(r0, res) and torch.equal(y0, y1)


def test_same_bits_again_and_in_a_graph():
    x, z, dy = (rand(i, 3000, 256, dtype=BF).to(DEV) for i in range(3))
    w, c, res = rand(4, 256).to(DEV), rand(5, 256).to(DEV), rand(6, 3000, 256).to(DEV)

    def step():
        y = mb.gated_norm_fwd(x, z, w, 4)
        g = mb.gated_norm_bwd(x, z, w, dy, 4)
        y2, r = mb.residual_norm_fwd(y, res, w, channel_scale=c)
        h = mb.residual_norm_bwd(r, w, dy, x=y, channel_scale=c)
        return [y, *g.values(), y2, r, *h.values()]
    first, second = step(), step()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for t in held:
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, held))
