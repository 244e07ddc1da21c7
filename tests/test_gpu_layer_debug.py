"""Linear attention and the norms through the MS_DEBUG build of the library: its kernels test
what an item, a row or a column may touch against the arrays, and record MS_ERR_BOUNDS instead
of performing an access out of range. Every way that the work is cut reports none, and gives the
product build's bits."""
import pytest
import torch

from selective_state_space_40_b200 import binding as mb
from selective_state_space_40_b200 import build as mbuild

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def debug_path():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return mbuild.build_debug()


def both(path, run):
    """run(status) with the product library and with the debug one: no bounds failure, the same bits."""
    out = []
    for lib in (None, path):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        if lib is None:
            res = run(st)
        else:
            with mb.use_library(lib):
                assert mb.mamba_debug_build() == 1
                res = run(st)
        torch.cuda.synchronize()
        assert st.item() == 0
        out.append([t for t in res if t is not None])
    assert len(out[0]) == len(out[1]) and all(torch.equal(a, b) for a, b in zip(*out))


# whole sequences, segments handed on, segments' own states, the plain recurrence
@pytest.mark.parametrize("b,L,H,G,dk,dv,dtype", [(2, 300, 4, 2, 64, 64, BF), (8, 700, 24, 24, 16, 16, BF),
                                                (1, 4000, 3, 3, 64, 128, BF), (2, 1100, 2, 1, 128, 72, BF),
                                                (2, 90, 3, 3, 20, 12, F32)])
def test_linattn_clean(debug_path, b, L, H, G, dk, dv, dtype):
    gen = torch.Generator().manual_seed(L)
    r = lambda *s: torch.randn(*s, generator=gen).to(dtype).to(DEV)  # noqa: E731
    q, k, v, do = r(b, L, H, dk), r(b, L, G, dk), r(b, L, G, dv), r(b, L, H, dv)
    g = -0.1 * torch.rand(H, generator=gen).to(DEV)

    def run(st):
        o, fin = mb.linattn_fwd(q, k, v, g, dev_status=st)
        gr = mb.linattn_bwd(q, k, v, g, do, initial_state=fin, dev_status=st)
        o1 = mb.linattn_state_update(fin, q[:, 0], k[:, 0], v[:, 0], g, dev_status=st)
        return [o, fin, o1, *gr.values()]
    both(debug_path, run)


@pytest.mark.parametrize("starts", [[0, 1, 1, 130, 700], [5, 5, 2100], [0] + list(range(3, 600, 7))])
def test_packed_linattn_clean(debug_path, starts):
    gen = torch.Generator().manual_seed(len(starts))
    n = starts[-1] + 3
    q, k, v, do = (torch.randn(n, 2, 64, generator=gen).to(BF).to(DEV) for _ in range(4))
    g = -0.1 * torch.rand(2, generator=gen).to(DEV)
    at = torch.tensor(starts, dtype=torch.int32, device=DEV)

    def run(st):
        zeros = {m: torch.zeros_like(q) for m in ("dq", "dk", "dv")}
        o, fin = mb.linattn_fwd(q, k, v, g, seq_start=at, o=torch.zeros_like(q), dev_status=st)
        return [o, fin, *mb.linattn_bwd(q, k, v, g, do, seq_start=at, grads=zeros, dev_status=st).values()]
    both(debug_path, run)


@pytest.mark.parametrize("rows,width,groups", [(3, 80, 5), (700, 1024, 1), (2, 16384, 1), (65, 777, 7), (2000, 2048, 16)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norms_clean(debug_path, rows, width, groups, dtype):
    gen = torch.Generator().manual_seed(rows)
    r = lambda *s: torch.randn(*s, generator=gen).to(dtype).to(DEV)  # noqa: E731
    x, z, dy, res = (r(rows, width) for _ in range(4))
    w = torch.randn(width, generator=gen).to(DEV)

    def run(st):
        y = mb.gated_norm_fwd(x, z, w, groups, dev_status=st)
        gg = mb.gated_norm_bwd(x, z, w, dy, groups, gate_first=True, dev_status=st)
        y2, ro = mb.residual_norm_fwd(x, res, w, channel_scale=w, dev_status=st)
        gr = mb.residual_norm_bwd(ro, w, dy, res, x=x, channel_scale=w, dev_status=st)
        return [y, *gg.values(), y2, ro, *gr.values()]
    both(debug_path, run)
