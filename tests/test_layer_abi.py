"""Argument checks of the linear-attention layer's and the norms' entry points
(host only: nothing is launched), and of their torch conveniences."""
import pytest
import torch

from selective_state_space_40_b200 import binding as mb
from selective_state_space_40_b200 import build as mbuild

FAKE = 1 << 20  # never dereferenced: every call below fails its host checks


@pytest.fixture(scope="module", autouse=True)
def lib():
    mbuild.build()
    return mb.library()


def _dims(**kw):
    d = dict(batch=2, seqlen=16, total=32, nheads=4, kv_heads=2, dk=64, dv=64, q_sb=4096, q_sl=256, q_sh=64, k_sb=2048,
             k_sl=128, k_sh=64, v_sb=2048, v_sl=128, v_sh=64, o_sb=4096, o_sl=256, o_sh=64, dtype=mb.MS_BF16)
    d.update(kw)
    return mb.LinattnDims(**d)


def _fwd(dims, q=FAKE, g=FAKE, o=FAKE, fin=None, seq=None, ws=None, wb=0):
    return mb.mamba_linattn_fwd(q, FAKE, FAKE, g, 1.0, seq, None, o, fin, dims, ws, wb, None, None)


def _bwd(dims, dq=FAKE, dfinal=None, dinit=None, ws=None, wb=0, seq=None):
    return mb.mamba_linattn_bwd(FAKE, FAKE, FAKE, FAKE, 1.0, seq, None, FAKE, dfinal, dq, FAKE, FAKE, dinit, dims, ws, wb,
                                None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), mb.MS_ERR_DTYPE),
    (dict(batch=-1), mb.MS_ERR_SHAPE),
    (dict(seqlen=-1), mb.MS_ERR_SHAPE),
    (dict(kv_heads=3), mb.MS_ERR_SHAPE),
    (dict(kv_heads=0), mb.MS_ERR_SHAPE),
    (dict(nheads=0), mb.MS_ERR_SHAPE),
    (dict(dk=0), mb.MS_ERR_SHAPE),
    (dict(dk=129), mb.MS_ERR_SHAPE),
    (dict(dv=129), mb.MS_ERR_SHAPE),
    (dict(seqlen=1 << 40), mb.MS_ERR_SHAPE),
    (dict(q_sb=1 << 62), mb.MS_ERR_SHAPE),
    (dict(v_sl=-8), mb.MS_ERR_STRIDE),
])
def test_linattn_rejects_bad_dims(kw, code):
    assert _fwd(_dims(**kw)) == code
    assert _bwd(_dims(**kw)) == code


def test_linattn_rejects_null_and_misaligned():
    assert mb.library().mamba_linattn_fwd(FAKE, FAKE, FAKE, FAKE, 1.0, None, None, FAKE, None, None, None, 0, None,
                                          None) == mb.MS_ERR_NULL
    assert _fwd(_dims(), q=None) == mb.MS_ERR_NULL
    assert _fwd(_dims(), o=None) == mb.MS_ERR_NULL
    assert _fwd(_dims(), g=None) == mb.MS_ERR_NULL
    assert _fwd(_dims(), q=FAKE + 1) == mb.MS_ERR_ALIGN
    assert _fwd(_dims(), g=FAKE + 2) == mb.MS_ERR_ALIGN
    assert _fwd(_dims(), fin=FAKE + 2) == mb.MS_ERR_ALIGN
    assert _fwd(_dims(), seq=FAKE + 2) == mb.MS_ERR_ALIGN
    assert _bwd(_dims(), dq=None) == mb.MS_ERR_NULL
    assert _bwd(_dims(), dfinal=FAKE, dinit=FAKE) == mb.MS_ERR_SHAPE
    assert _fwd(_dims(batch=0)) == mb.MS_OK


def test_linattn_workspaces():
    # shared heads: 2 x 16 tokens x 4 heads of fp32 dk and dv rows
    d = _dims()
    need = mb.mamba_linattn_bwd_workspace_size(d, False)
    assert need >= 2 * 16 * 4 * (64 + 64) * 4
    assert mb.mamba_linattn_bwd_workspace_size(d, True) >= 32 * 4 * (64 + 64) * 4
    assert _bwd(d) == mb.MS_ERR_WORKSPACE
    assert _bwd(d, ws=FAKE, wb=need - 1) == mb.MS_ERR_WORKSPACE
    assert _bwd(d, ws=FAKE + 8, wb=need) == mb.MS_ERR_ALIGN
    assert mb.library().mamba_linattn_workspace_size(None, 0) == 0
    assert mb.library().mamba_linattn_bwd_workspace_size(None, 0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), mb.MS_ERR_DTYPE),
    (dict(dv=257), mb.MS_ERR_SHAPE),
    (dict(dk=0), mb.MS_ERR_SHAPE),
    (dict(kv_heads=3), mb.MS_ERR_SHAPE),
    (dict(k_sh=-1), mb.MS_ERR_STRIDE),
    (dict(state_sh=64 * 64 - 1), mb.MS_ERR_STRIDE),   # heads' states overlap
    (dict(state_sb=0), mb.MS_ERR_STRIDE),             # rows share a state
    (dict(state_sb=1 << 62), mb.MS_ERR_SHAPE),
])
def test_linattn_update_rejects(kw, code):
    d = dict(batch=3, nheads=4, kv_heads=2, dk=64, dv=64, q_sb=256, q_sh=64, k_sb=128, k_sh=64, v_sb=128, v_sh=64,
             o_sb=256, o_sh=64, state_sb=4 * 4096, state_sh=4096, dtype=mb.MS_F32)
    d.update(kw)
    args = lambda st=FAKE, q=FAKE: (st, q, FAKE, FAKE, FAKE, 1.0, FAKE)  # noqa: E731
    assert mb.mamba_linattn_state_update(*args(), mb.LinattnUpdateDims(**d), None, None) == code
    ok = dict(d, dtype=0, dv=64, dk=64, kv_heads=2, k_sh=64, state_sh=4096, state_sb=4 * 4096)
    assert mb.mamba_linattn_state_update(*args(None), mb.LinattnUpdateDims(**ok), None, None) == mb.MS_ERR_NULL
    assert mb.mamba_linattn_state_update(*args(FAKE, FAKE + 2), mb.LinattnUpdateDims(**ok), None, None) == mb.MS_ERR_ALIGN
    assert mb.mamba_linattn_state_update(*args(), mb.LinattnUpdateDims(**dict(ok, batch=0)), None, None) == mb.MS_OK


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), mb.MS_ERR_DTYPE),
    (dict(rows=-1), mb.MS_ERR_SHAPE),
    (dict(width=0), mb.MS_ERR_SHAPE),
    (dict(groups=5), mb.MS_ERR_SHAPE),
    (dict(width=16385, groups=1), mb.MS_ERR_SHAPE),
    (dict(eps=-1.0), mb.MS_ERR_SHAPE),
    (dict(eps=float("nan")), mb.MS_ERR_SHAPE),
    (dict(x_sr=-64), mb.MS_ERR_STRIDE),
])
def test_gated_norm_rejects(kw, code):
    d = dict(rows=4, width=64, groups=2, x_sr=64, z_sr=64, y_sr=64, eps=1e-5, dtype=mb.MS_BF16, gate_first=0)
    fwd = lambda dm, x=FAKE, y=FAKE: mb.mamba_gated_norm_fwd(x, FAKE, None, y, dm, None, None)  # noqa: E731
    bwd = lambda dm, z=FAKE, dz=FAKE, dw=FAKE, ws=None, wb=0: mb.mamba_gated_norm_bwd(  # noqa: E731
        FAKE, z, None, FAKE, FAKE, dz, dw, dm, ws, wb, None, None)
    bad, ok = mb.GatedNormDims(**dict(d, **kw)), mb.GatedNormDims(**d)
    assert fwd(bad) == code and bwd(bad) == code
    assert mb.mamba_gated_norm_bwd_workspace_size(bad) in (0, mb.mamba_gated_norm_bwd_workspace_size(bad))
    assert fwd(ok, x=None) == mb.MS_ERR_NULL and fwd(ok, y=FAKE + 1) == mb.MS_ERR_ALIGN
    assert bwd(ok, dz=None) == mb.MS_ERR_NULL and bwd(ok, z=None) == mb.MS_ERR_NULL
    need = mb.mamba_gated_norm_bwd_workspace_size(ok)
    assert need >= 64 * 4
    assert bwd(ok) == mb.MS_ERR_WORKSPACE and bwd(ok, ws=FAKE, wb=need - 1) == mb.MS_ERR_WORKSPACE
    assert bwd(ok, ws=FAKE + 4, wb=need) == mb.MS_ERR_ALIGN
    assert fwd(mb.GatedNormDims(**dict(d, rows=0))) == mb.MS_OK


@pytest.mark.parametrize("kw,code", [
    (dict(res_dtype=5), mb.MS_ERR_DTYPE),
    (dict(width=16385), mb.MS_ERR_SHAPE),
    (dict(eps=float("inf")), mb.MS_ERR_SHAPE),
    (dict(resout_sr=-1), mb.MS_ERR_STRIDE),
])
def test_residual_norm_rejects(kw, code):
    d = dict(rows=4, width=64, x_sr=64, res_sr=64, y_sr=64, resout_sr=64, eps=1e-5, res_scale=1.0, dtype=mb.MS_BF16,
             res_dtype=mb.MS_F32)
    fwd = lambda dm, x=FAKE, r=FAKE: mb.mamba_residual_norm_fwd(x, r, None, None, FAKE, r, dm, None, None)  # noqa: E731
    bwd = lambda dm, x=FAKE, cs=FAKE, dc=FAKE, ws=None, wb=0: mb.mamba_residual_norm_bwd(  # noqa: E731
        FAKE, None, FAKE, FAKE, x, cs, FAKE, FAKE, FAKE, dc, dm, ws, wb, None, None)
    bad, ok = mb.ResidualNormDims(**dict(d, **kw)), mb.ResidualNormDims(**d)
    assert fwd(bad) == code and bwd(bad) == code
    assert fwd(ok, x=None) == mb.MS_ERR_NULL and fwd(ok, r=FAKE + 2) == mb.MS_ERR_ALIGN
    assert bwd(ok, x=None) == mb.MS_ERR_NULL and bwd(ok, cs=None) == mb.MS_ERR_NULL
    need = mb.mamba_residual_norm_bwd_workspace_size(ok)
    assert need >= 2 * 64 * 4
    assert bwd(ok, ws=FAKE, wb=need - 1) == mb.MS_ERR_WORKSPACE
    assert fwd(mb.ResidualNormDims(**dict(d, rows=0))) == mb.MS_OK


def test_conveniences_refuse_on_the_host():
    q = torch.zeros(2, 8, 4, 16)
    g = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        mb.linattn_fwd(q, q, q, g)
    with pytest.raises(ValueError, match="k must be"):
        mb.linattn_fwd(q, q.bfloat16(), q, g)
    with pytest.raises(ValueError, match="log_decay"):
        mb.linattn_fwd(q, q, q, g[:3])
    with pytest.raises(ValueError, match="dimensions"):
        mb.linattn_fwd(q, q, q, g, seq_start=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="seq_start"):
        mb.linattn_fwd(q[0], q[0], q[0], g, seq_start=torch.zeros(3))
    with pytest.raises(ValueError, match="unit stride"):
        mb.linattn_fwd(q.transpose(2, 3), q, q, g)
    with pytest.raises(ValueError, match="dout"):
        mb.linattn_bwd(q, q, q, g, q[:, :7])
    with pytest.raises(ValueError, match="state must"):
        mb.linattn_state_update(torch.zeros(2, 4, 16, 15), q[:, 0], q[:, 0], q[:, 0], g)
    x = torch.zeros(3, 8)
    with pytest.raises(ValueError, match="CUDA"):
        mb.gated_norm_fwd(x, x)
    with pytest.raises(ValueError, match="z must be"):
        mb.gated_norm_fwd(x, x[:, :7])
    with pytest.raises(ValueError, match="weight"):
        mb.residual_norm_fwd(x, weight=torch.zeros(7))
    with pytest.raises(ValueError, match="CUDA"):
        mb.residual_norm_bwd(x, None, x)


@pytest.mark.parametrize("kw,fwd,bwd", [
    (dict(o_sb=0), mb.MS_ERR_STRIDE, None),                  # rows of o written twice
    (dict(o_sl=0), mb.MS_ERR_STRIDE, None),
    (dict(o_sh=63), mb.MS_ERR_STRIDE, None),                 # heads overlap by one
    (dict(q_sb=0), None, mb.MS_ERR_STRIDE),                  # broadcast inputs: not those of the gradients
    (dict(k_sh=0), None, mb.MS_ERR_STRIDE),
    (dict(v_sl=0), None, mb.MS_ERR_STRIDE),
    (dict(k_sl=64, k_sh=16 * 64), None, None),               # heads outside the tokens
    (dict(o_sb=64, o_sl=128, o_sh=16 * 128), None, None),    # batch inside the tokens
    (dict(batch=1, q_sb=0, o_sb=0), None, None),             # one row: its stride is not used
    (dict(kv_heads=1, k_sh=0, v_sh=0), None, None),
])
def test_written_arrays_hold_no_element_twice(kw, fwd, bwd):
    # the workspace check comes behind the strides' one: the calls end there at the latest
    d = _dims(**kw)
    assert _bwd(d) == (bwd or mb.MS_ERR_WORKSPACE)
    assert _fwd(d, o=FAKE + 1) == (fwd or mb.MS_ERR_ALIGN)


def test_outputs_that_are_inputs_are_refused():
    d = _dims(kv_heads=4, k_sb=4096, k_sl=256, v_sb=4096, v_sl=256)
    need = max(mb.mamba_linattn_bwd_workspace_size(d, False), mb.mamba_linattn_workspace_size(d, False))
    at = [FAKE + (i << 12) for i in range(12)]
    for o in at[:3]:
        assert mb.mamba_linattn_fwd(*at[:3], at[3], 1.0, None, None, o, None, d, at[9], need, None, None) == mb.MS_ERR_SHAPE
    back = lambda grads, s0=None, ds0=None: mb.mamba_linattn_bwd(  # noqa: E731
        *at[:3], at[3], 1.0, None, s0, at[4], None, *grads, ds0, d, at[9], need, None, None)
    for bad in (at[0], at[1], at[2], at[4]):
        assert back((bad, at[6], at[7])) == back((at[5], bad, at[7])) == back((at[5], at[6], bad)) == mb.MS_ERR_SHAPE
    assert back((at[5], at[5], at[7])) == back((at[5], at[6], at[6])) == back((at[5], at[6], at[5])) == mb.MS_ERR_SHAPE
    assert back(at[5:8], at[8], at[8]) == mb.MS_ERR_SHAPE


def test_norms_refuse_rows_written_twice():
    g = dict(rows=4, width=64, groups=2, x_sr=0, z_sr=0, y_sr=63, eps=1e-5, dtype=mb.MS_BF16, gate_first=0)
    assert mb.mamba_gated_norm_fwd(FAKE, FAKE, None, FAKE, mb.GatedNormDims(**g), None, None) == mb.MS_ERR_STRIDE
    r = dict(rows=4, width=64, x_sr=64, res_sr=64, y_sr=64, resout_sr=64, eps=1e-5, res_scale=1.0, dtype=mb.MS_BF16,
             res_dtype=mb.MS_F32)
    for kw in (dict(y_sr=0), dict(resout_sr=32), dict(resout_sr=128)):  # the last: in place with another stride
        d = mb.ResidualNormDims(**dict(r, **kw))
        assert mb.mamba_residual_norm_fwd(FAKE, FAKE, None, None, FAKE, FAKE, d, None, None) == mb.MS_ERR_STRIDE
    u = dict(batch=3, nheads=4, kv_heads=2, dk=64, dv=64, q_sb=256, q_sh=64, k_sb=128, k_sh=64, v_sb=128, v_sh=64,
             o_sb=256, o_sh=64, state_sb=4 * 4096, state_sh=4096, dtype=mb.MS_F32)
    for kw in (dict(o_sb=0), dict(o_sh=0), dict(state_sb=4096, state_sh=4096)):
        d = mb.LinattnUpdateDims(**dict(u, **kw))
        assert mb.mamba_linattn_state_update(FAKE, FAKE, FAKE, FAKE, FAKE, 1.0, FAKE, d, None, None) == mb.MS_ERR_STRIDE
