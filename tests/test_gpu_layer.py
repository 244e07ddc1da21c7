"""The layer's operators run together, as a block uses them: norm, linear attention, gated
norm, residual and norm, forward and backward, against the same chain in 64 bits
(oracle/layer.py). The projections between them are the caller's; here one matrix.

Tolerances: in fp32 every operator is off by a few 2^-24 sqrt(n) of its terms (see
layer_util), and the chain of six by no more than 64 times 2^-24 sqrt(width): 1e-4 bounds the
relative 2-norm with room for the norms' division by small groups. In bf16 each of the
chain's six stored tensors is rounded once (2^-8 / sqrt(3) of its 2-norm) and attention rounds
twice inside: 8 roundings in the root of their squares are 6.4e-3, doubled for what the
following operators make of them."""
import numpy as np
import pytest
import torch

from oracle import layer
from selective_state_space_40_b200 import binding as mb

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert mb.mamba_device_check() == mb.MS_OK


def f64(t):
    return t.detach().cpu().double().numpy()


def rel(a, b):
    return np.linalg.norm(f64(a) - b) / np.linalg.norm(b)


@pytest.mark.parametrize("dtype,most", [(torch.float32, 1e-4), (torch.bfloat16, 1.3e-2)])
@pytest.mark.parametrize("b,L,H,d", [(2, 200, 4, 64), (1, 33, 3, 16), (1, 1, 2, 64)])
def test_block_forward_and_backward(dtype, most, b, L, H, d):
    gen = torch.Generator().manual_seed(L + H)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    D, rows = H * d, b * L
    x, res, z = r(rows, D).to(dtype), r(rows, D), r(rows, D).to(dtype)
    w1, w2, w3, c = 1 + 0.1 * r(D), 1 + 0.1 * r(D), 1 + 0.1 * r(D), 0.5 + 0.1 * r(D)
    mats = [(r(D, D) / D ** 0.5).to(dtype) for _ in range(3)]
    g = -torch.rand(H, generator=gen) * 0.2
    dy = r(rows, D).to(dtype)
    to = lambda t: t.to(DEV)  # noqa: E731
    eps, s = 1e-5, 0.7

    # forward: r1 = res + s c x, u = norm(r1) w1; q, k, v = u M; o = attention; y = gated norm per head; r2, out
    u, r1 = mb.residual_norm_fwd(to(x), to(res), to(w1), eps, s, to(c))
    q, k, v = ((u.float() @ to(m).float()).to(dtype).view(b, L, H, d) for m in mats)
    o, _ = mb.linattn_fwd(q, k, v, to(g))
    y = mb.gated_norm_fwd(o.view(rows, D), to(z), to(w2), H, eps, gate_first=False)
    out, r2 = mb.residual_norm_fwd(y, r1, to(w3), eps, s)
    # the same in 64 bits
    M = [f64(m) for m in mats]
    U, R1 = layer.residual_norm(f64(x), f64(res), f64(w1), f64(c), s, eps)
    Q, K, V = ((U @ m).reshape(b, L, H, d) for m in M)
    a = d ** -0.5
    O = np.stack([layer.linattn(Q[i], K[i], V[i], f64(g), a)[0] for i in range(b)]).reshape(rows, D)
    Y = layer.gated_norm(O, f64(z), f64(w2), H, eps, False)
    OUT, R2 = layer.residual_norm(Y, R1, f64(w3), None, s, eps)
    for name, got, want in (("u", u, U), ("o", o.view(rows, D), O), ("y", y, Y), ("out", out, OUT), ("r2", r2, R2)):
        assert rel(got, want) <= most, (name, rel(got, want))

    # backward of sum(out dy)
    g2 = mb.residual_norm_bwd(r2, to(w3), to(dy), eps=eps, res_scale=s)
    gn = mb.gated_norm_bwd(o.view(rows, D), to(z), to(w2), g2["dx"], H, eps, gate_first=False)
    ga = mb.linattn_bwd(q, k, v, to(g), gn["dx"].view(b, L, H, d), want_dinitial=False)
    assert ga["dinitial_state"] is None
    du = sum(ga[n].reshape(rows, D).float() @ to(m).float().t() for n, m in zip(("dq", "dk", "dv"), mats)).to(dtype)
    g1 = mb.residual_norm_bwd(r1, to(w1), du, dresidual_out=g2["dresidual"], x=to(x), eps=eps, res_scale=s,
                              channel_scale=to(c))
    torch.cuda.synchronize()
    DY, DR2, DW3, _ = layer.residual_norm_bwd(R2, f64(w3), f64(dy), None, None, None, s, eps)
    DO, DZ, DW2 = layer.gated_norm_bwd(O, f64(z), f64(w2), DY, H, eps, False)
    parts = [layer.linattn_bwd(Q[i], K[i], V[i], f64(g), a, DO.reshape(b, L, H, d)[i]) for i in range(b)]
    DQ, DK, DV = (np.stack([p[j] for p in parts]).reshape(rows, D) for j in range(3))
    DU = DQ @ M[0].T + DK @ M[1].T + DV @ M[2].T
    DX, DRES, DW1, DC = layer.residual_norm_bwd(R1, f64(w1), DU, DR2, f64(x), f64(c), s, eps)
    for name, got, want in (("dy", g2["dx"], DY), ("dw3", g2["dweight"], DW3), ("do", gn["dx"], DO), ("dz", gn["dz"], DZ),
                            ("dw2", gn["dweight"], DW2), ("dx", g1["dx"], DX), ("dres", g1["dresidual"], DRES),
                            ("dw1", g1["dweight"], DW1), ("dc", g1["dchannel_scale"], DC)):
        assert rel(got, want) <= 4 * most, (name, rel(got, want))
