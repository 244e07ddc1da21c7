"""Linear attention with a decay per head on the GPU against its recurrence in
64 bits (oracle/layer.py): forward, gradients and single tokens."""
import numpy as np
import pytest
import torch

from oracle import layer
from selective_state_space_40_b200 import binding as mb
from layer_util import check

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


def make(rows, H, G, dk, dv, dtype, seed, n=1, state=True, decays=None):
    """Packed inputs of `rows` tokens and states for n sequences, on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = dict(q=r(rows, H, dk).to(dtype), k=r(rows, G, dk).to(dtype), v=r(rows, G, dv).to(dtype),
             do=r(rows, H, dv).to(dtype), s0=r(n, H, dk, dv) if state else None, ds=r(n, H, dk, dv) if state else None)
    # a head that forgets at once, slow ones, a head without decay
    x["g"] = torch.tensor(([-2.0, -0.03, -2.0 ** -12, 0.0, -0.3] * H)[:H] if decays is None else decays)
    x["scale"] = dk ** -0.5
    return x


def runs_in_chunks(dk, dv, dtype):
    return dtype == BF and dk % 8 == 0 and dv % 8 == 0


def check_fwd(x, starts, o, fin, dtype):
    """Every sequence against the recurrence; tolerances from the same recurrence on absolute values."""
    tc = runs_in_chunks(x["q"].shape[2], x["v"].shape[2], dtype)
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        q, k, v = (f64(x[n][a:b]) for n in ("q", "k", "v"))
        s0 = None if x["s0"] is None else f64(x["s0"][i])
        want, wf = layer.linattn(q, k, v, f64(x["g"]), x["scale"], s0)
        mag, mf = layer.linattn(abs(q), abs(k), abs(v), f64(x["g"]), x["scale"], None if s0 is None else abs(s0))
        n = b - a + q.shape[2] + 4
        check(o[a:b], want, mag, n, dtype == BF, f"o of sequence {i}", tc)
        if fin is not None:
            check(fin[i], wf, mf, n, False, f"final state of sequence {i}")


def check_bwd(x, starts, g, dtype):
    tc = runs_in_chunks(x["q"].shape[2], x["v"].shape[2], dtype)
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        t = [f64(x[n][a:b]) for n in ("q", "k", "v")]
        do = f64(x["do"][a:b])
        st = [None if x[n] is None else f64(x[n][i]) for n in ("s0", "ds")]
        ab = [None if s is None else abs(s) for s in st]
        want = layer.linattn_bwd(*t, f64(x["g"]), x["scale"], do, *st)
        mag = layer.linattn_bwd(*(abs(y) for y in t), f64(x["g"]), x["scale"], abs(do), *ab)
        n = b - a + 128 + 4 + x["q"].shape[1]
        for name, w, m in zip(("dq", "dk", "dv"), want, mag):
            check(g[name][a:b], w, m, n, dtype == BF, f"{name} of sequence {i}", tc)
        check(g["dinitial_state"][i], want[3], mag[3], n, False, f"dinitial_state of sequence {i}")


def dev(x, *names):
    return [None if x[n] is None else x[n].to(DEV) for n in names]


def run_packed(x, starts, dtype):
    """Forward and backward of packed sequences; checks that rows of no sequence keep what was there."""
    q, k, v, g, do, s0, ds = dev(x, "q", "k", "v", "g", "do", "s0", "ds")
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = torch.full((q.shape[0], q.shape[1], v.shape[2]), 7.0, dtype=dtype, device=DEV)
    o, fin = mb.linattn_fwd(q, k, v, g, x["scale"], seq_start=st, initial_state=s0, o=o, dev_status=status)
    grads = {n: torch.full_like(t, 7.0) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    gr = mb.linattn_bwd(q, k, v, g, do, x["scale"], seq_start=st, initial_state=s0, dfinal=ds, grads=grads,
                        dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    check_fwd(x, starts, o, fin, dtype)
    check_bwd(x, starts, gr, dtype)
    for t in (o, gr["dq"], gr["dk"], gr["dv"]):
        assert (t[:starts[0]] == 7.0).all() and (t[starts[-1]:] == 7.0).all()


def run_dense(x, b, L, dtype):
    q, k, v, g, do, s0, ds = dev(x, "q", "k", "v", "g", "do", "s0", "ds")
    shaped = lambda t: t.view(b, L, *t.shape[1:])  # noqa: E731
    o, fin = mb.linattn_fwd(shaped(q), shaped(k), shaped(v), g, x["scale"], initial_state=s0)
    gr = mb.linattn_bwd(shaped(q), shaped(k), shaped(v), g, shaped(do), x["scale"], initial_state=s0, dfinal=ds)
    torch.cuda.synchronize()
    starts = [i * L for i in range(b + 1)]
    check_fwd(x, starts, o.flatten(0, 1), fin, dtype)
    check_bwd(x, starts, {n: t if n == "dinitial_state" else t.flatten(0, 1) for n, t in gr.items()}, dtype)


@pytest.mark.parametrize("L", [1, 2, 127, 128, 129, 255, 300, 640])
def test_lengths(L):
    run_dense(make(2 * L, 3, 3, 64, 64, BF, L, n=2), 2, L, BF)


@pytest.mark.parametrize("dk,dv", [(8, 8), (16, 128), (128, 16), (40, 72), (64, 64), (80, 96), (128, 128), (72, 64), (64, 120)])
def test_head_sizes(dk, dv):
    run_dense(make(2 * 200, 4, 2, dk, dv, BF, dk + dv, n=2), 2, 200, BF)


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 64, 64), (F32, 5, 3), (F32, 128, 128), (BF, 12, 20), (BF, 7, 64)])
def test_plain_recurrence(dtype, dk, dv):
    run_dense(make(2 * 70, 4, 2, dk, dv, dtype, dk, n=2), 2, 70, dtype)


@pytest.mark.parametrize("G", [1, 2, 8])
def test_shared_heads(G):
    run_dense(make(2 * 260, 8, G, 64, 128, BF, 77 + G, n=2), 2, 260, BF)


@pytest.mark.parametrize("state", [False, True])
def test_without_states(state):
    run_dense(make(150, 2, 1, 64, 64, BF, 5, n=1, state=state), 1, 150, BF)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_sequences(dtype):
    """Empty sequences at both ends and between, one token, chunk borders, rows of no sequence on both sides."""
    lens = [0, 1, 128, 0, 0, 129, 3, 300, 64, 127, 0]
    starts = np.cumsum([5] + lens).tolist()
    run_packed(make(starts[-1] + 9, 4, 2, 64, 64, dtype, 11, n=len(lens)), starts, dtype)


def test_packed_rows_behind_hold_nothing_readable():
    """NaN and infinity in the rows next to a sequence (another's, or nobody's) never reach it."""
    starts = [130, 130 + 5, 130 + 5 + 131]
    x = make(500, 2, 2, 64, 64, BF, 21, n=2)
    for n in ("q", "k", "v", "do"):
        x[n][:130] = float("nan")
        x[n][starts[-1]:] = float("inf")
    run_packed(x, starts, BF)
    y = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in x.items()}
    for n in ("q", "k", "v", "do"):
        y[n][135:] = float("nan")  # the second sequence too: the first one stays clean
    y["s0"][1] = y["ds"][1] = float("nan")
    q, k, v, g, do, s0, ds = dev(y, "q", "k", "v", "g", "do", "s0", "ds")
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    o, fin = mb.linattn_fwd(q, k, v, g, x["scale"], seq_start=st, initial_state=s0)
    gr = mb.linattn_bwd(q, k, v, g, do, x["scale"], seq_start=st, initial_state=s0, dfinal=ds)
    check_fwd(x, starts[:2], o, fin, BF)
    check_bwd(x, starts[:2], gr, BF)


@pytest.mark.parametrize("H,L", [(1, 4100), (2, 1793), (5, 2048)])
def test_long_and_few_heads(H, L):
    """Few heads: the sequence is cut into segments that run side by side."""
    run_dense(make(L, H, 1, 64, 64, BF, L, n=1, decays=[-2.0 ** -11, -0.01, 0.0, -1.0, -0.002][:H]), 1, L, BF)


def test_segments_of_packed_sequences():
    starts = [0, 700, 700, 701, 2900, 4211]
    run_packed(make(4300, 2, 2, 128, 64, BF, 31, n=5, decays=[-2.0 ** -11, -0.02]), starts, BF)


@pytest.mark.parametrize("b,L,H,G,dk,dv", [(8, 700, 24, 24, 16, 16), (5, 530, 33, 11, 128, 8)])
def test_chains_that_do_not_divide_by_the_sms(b, L, H, G, dk, dv):
    """Sequences in several items, the state handed from one CTA to the next."""
    run_dense(make(b * L, H, G, dk, dv, BF, L, n=b), b, L, BF)


def test_many_short_packed_sequences():
    r = np.random.RandomState(3)
    lens = r.randint(0, 40, 150).tolist() + [300] + [0] * 40 + [7]
    starts = np.cumsum([0] + lens).tolist()
    run_packed(make(starts[-1] + 3, 4, 4, 16, 24, BF, 33, n=len(lens)), starts, BF)


def test_rows_beyond_32_bit_offsets():
    """Arrays of more than 2^32 elements: with nothing remembered, o_t = a (q_t . k_t) v_t, whole and at both ends."""
    L, H, d = 270000, 128, 128
    gen = torch.Generator(device=DEV).manual_seed(1)
    q = torch.empty(1, L, H, d, dtype=BF, device=DEV)
    assert q.numel() > 2 ** 32
    q.normal_(generator=gen)
    o, fin = mb.linattn_fwd(q, q, q, torch.full((H,), float("-inf"), device=DEV), scale=1.0)
    for sl in (slice(0, 300), slice(L - 300, L)):
        x = q[0, sl].double()
        want = x.square().sum(-1, keepdim=True) * x
        assert ((o[0, sl].double() - want).norm() / want.norm()).item() <= 4e-3
    x = q[0, -1].double()
    assert ((fin[0].double() - x[:, :, None] * x[:, None, :]).norm() / fin.double().norm()).item() <= 1e-6
    # and gradients through rows of a wide buffer, 2^32 elements behind its start
    wide = q.view(-1)
    n, tail = 200, q.view(-1).numel() - 200 * H * d
    t = wide[tail:].view(1, n, H, d)
    gr = mb.linattn_bwd(t, t, t, torch.full((H,), -0.5, device=DEV), t, scale=1.0)
    c = t.clone()
    ref = mb.linattn_bwd(c, c, c, torch.full((H,), -0.5, device=DEV), c, scale=1.0)
    assert all(torch.equal(gr[m], ref[m]) for m in ("dq", "dk", "dv", "dinitial_state"))


def test_two_streams_with_their_own_workspaces():
    """Two long calls at once, each with its own workspace: the results of one after the other."""
    xs = [make(4096, 2, 2, 64, 64, BF, 80 + i, n=1, decays=[-0.001, -0.02]) for i in range(2)]
    ins = [dev(x, "q", "k", "v", "g") for x in xs]
    want = [mb.linattn_fwd(q[None], k[None], v[None], g) for q, k, v, g in ins]
    need = mb.mamba_linattn_workspace_size(mb.linattn_dims_for(*(t[None] for t in ins[0][:3]), ins[0][0][None]), False)
    assert need > 0
    ws = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (q, k, v, g), w, st in zip(ins, ws, streams):
            with torch.cuda.stream(st):
                got.append(mb.linattn_fwd(q[None], k[None], v[None], g, workspace=w))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    with pytest.raises(mb.MambaScanError) as e:
        mb.linattn_fwd(*(t[None] for t in ins[0][:3]), ins[0][3], workspace=ws[0][:need - 1])
    assert e.value.code == mb.MS_ERR_WORKSPACE
    with pytest.raises(ValueError, match="tensors on"):
        mb.linattn_fwd(*(t[None] for t in ins[0][:3]), ins[0][3].cpu())


def test_decay_extremes():
    """exp(log_decay) = 0 (the token alone), subnormal steps of the powers, and no decay at all."""
    x = make(300, 5, 5, 64, 64, BF, 41, n=1, decays=[float("-inf"), -80.0, -5.0, 0.0, -2.0 ** -20])
    run_dense(x, 1, 300, BF)
    run_dense(make(40, 5, 5, 6, 6, F32, 42, n=1, decays=[float("-inf"), -80.0, -5.0, 0.0, -2.0 ** -20]), 1, 40, F32)


def test_strides_and_in_place_state():
    """Heads outside the tokens, slices of one projection, and the final state written over the initial one."""
    b, L, H, G, d = 2, 200, 4, 2, 64
    x = make(b * L, H, G, d, d, BF, 51, n=b)
    qkv = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1)], 1).to(DEV)
    q = qkv[:, :H * d].view(b, L, H, d)
    k = qkv[:, H * d:(H + G) * d].view(b, L, G, d)
    v = qkv[:, (H + G) * d:].view(b, L, G, d)
    s = x["s0"].to(DEV)
    o = torch.empty(b, H, L, d, dtype=BF, device=DEV).transpose(1, 2)
    o, fin = mb.linattn_fwd(q, k, v, x["g"].to(DEV), x["scale"], initial_state=s, o=o, final_state=s)
    assert fin is s
    check_fwd(x, [0, L, 2 * L], o.flatten(0, 1), fin, BF)
    # rows that do not start on 16 bytes run the plain recurrence
    wide = torch.zeros(b, L, H * d + 1, dtype=BF, device=DEV)
    wide[..., 1:] = q.flatten(2)
    o2, f2 = mb.linattn_fwd(wide[..., 1:].unflatten(2, (H, d)), k, v, x["g"].to(DEV), x["scale"],
                            initial_state=x["s0"].to(DEV))
    check_fwd(x, [0, L, 2 * L], o2.flatten(0, 1), f2, BF)


def test_in_place_state_of_a_long_sequence():
    x = make(4096, 1, 1, 64, 128, BF, 52, n=1, decays=[-0.001])
    q, k, v, g, s = dev(x, "q", "k", "v", "g", "s0")
    o, fin = mb.linattn_fwd(q[None], k[None], v[None], g, x["scale"], initial_state=s, final_state=s)
    check_fwd(x, [0, 4096], o[0], fin, BF)


def test_zero_length_passes_the_state_on():
    s = torch.randn(2, 3, 64, 64, device=DEV)
    e = torch.empty(2, 0, 3, 64, dtype=BF, device=DEV)
    g = torch.full((3,), -0.1, device=DEV)
    o, fin = mb.linattn_fwd(e, e, e, g, initial_state=s)
    assert o.shape == (2, 0, 3, 64) and torch.equal(fin, s)
    gr = mb.linattn_bwd(e, e, e, g, e, initial_state=s, dfinal=s)
    assert torch.equal(gr["dinitial_state"], s)
    o, fin = mb.linattn_fwd(e, e, e, g)
    assert (fin == 0).all()


@pytest.mark.parametrize("starts,good", [([-3, 10, 200, 390, 401], (1, 2)), ([10, 200, 150], (0,))])
def test_bad_sequence_offsets_are_left_out(starts, good):
    """Offsets before the first row, past the last one or running backwards: reported, nothing written for
    those sequences, the others computed."""
    n = len(starts) - 1
    x = make(400, 2, 2, 64, 64, BF, 61, n=n)
    q, k, v, g, do, s0, ds = dev(x, "q", "k", "v", "g", "do", "s0", "ds")
    status = torch.zeros(2, dtype=torch.int32, device=DEV)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    o = torch.full((400, 2, 64), 7.0, dtype=BF, device=DEV)
    fin = torch.full((n, 2, 64, 64), 7.0, device=DEV)
    mb.linattn_fwd(q, k, v, g, x["scale"], seq_start=st, initial_state=s0, o=o, final_state=fin, dev_status=status)
    grads = {m: torch.full_like(t, 7.0) for m, t in (("dq", q), ("dk", k), ("dv", v))}
    gr = mb.linattn_bwd(q, k, v, g, do, x["scale"], seq_start=st, initial_state=s0, dfinal=ds, grads=grads,
                        dev_status=status[1:])
    torch.cuda.synchronize()
    assert status.tolist() == [mb.MS_ERR_SHAPE, mb.MS_ERR_SHAPE]
    lo, hi = starts[good[0]], starts[good[-1] + 1]
    for t in (o, *grads.values()):
        assert (t[:lo] == 7.0).all() and (t[hi:] == 7.0).all()
    for i in range(n):
        if i not in good:
            assert (fin[i] == 7.0).all()
    sub = {m: (t[good[0]:good[-1] + 1] if m in ("s0", "ds") else t) for m, t in x.items()}
    at = [starts[i] for i in good] + [hi]
    sel = slice(good[0], good[-1] + 1)
    check_fwd(sub, at, o, fin[sel], BF)
    check_bwd(sub, at, {**gr, "dinitial_state": gr["dinitial_state"][sel]}, BF)


def test_same_bits_again_and_in_a_graph():
    """Results do not depend on the run; a captured call replays them from inputs changed in between."""
    x = make(2 * 500, 4, 2, 64, 64, BF, 71, n=2)
    q, k, v, g, do, s0, ds = dev(x, "q", "k", "v", "g", "do", "s0", "ds")
    q, k, v, do = (t.view(2, 500, *t.shape[1:]) for t in (q, k, v, do))

    def step():
        o, fin = mb.linattn_fwd(q, k, v, g, initial_state=s0)
        gr = mb.linattn_bwd(q, k, v, g, do, initial_state=s0, dfinal=ds)
        return [o, fin, gr["dq"], gr["dk"], gr["dv"], gr["dinitial_state"]]
    first, second = step(), step()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        third = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, third))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    saved = q.clone()
    q.mul_(2.0)
    graph.replay()
    doubled = [t.clone() for t in held]
    assert torch.equal(doubled[0], step()[0])
    q.copy_(saved)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, held))


@pytest.mark.parametrize("b,L,H,G,dk,dv", [(8, 700, 24, 24, 64, 64), (3, 1100, 20, 10, 128, 128), (1, 4000, 3, 3, 64, 128)])
def test_same_bits_over_many_runs(b, L, H, G, dk, dv):
    """Items that change hands between CTAs, roles that run ahead of one another: never another bit."""
    gen = torch.Generator(device=DEV).manual_seed(b * L)
    r = lambda n, d: torch.randn(b, L, n, d, device=DEV, generator=gen).to(BF)  # noqa: E731
    q, k, v, do = r(H, dk), r(G, dk), r(G, dv), r(H, dv)
    g = -torch.rand(H, device=DEV, generator=gen) * 0.05

    def step():
        o, fin = mb.linattn_fwd(q, k, v, g)
        gr = mb.linattn_bwd(q, k, v, g, do)
        return [o, fin, gr["dq"], gr["dk"], gr["dv"], gr["dinitial_state"]]
    first = step()
    for _ in range(15):
        assert all(torch.equal(a, c) for a, c in zip(first, step()))


# ------------------------------------------------------------- single tokens ----

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("b,H,G,dk,dv", [(1, 1, 1, 1, 1), (3, 4, 2, 64, 64), (2, 8, 1, 128, 64), (2, 3, 3, 40, 72),
                                         (2, 2, 1, 7, 5), (1, 2, 2, 300, 256), (5, 6, 3, 16, 128), (2, 2, 2, 128, 130),
                                         (1, 2, 1, 300, 4), (2, 1, 1, 700, 16), (1, 1, 1, 513, 1)])
def test_step(dtype, b, H, G, dk, dv):
    x = make(b, H, G, dk, dv, dtype, b * dk + dv, n=b)
    st = x["s0"].to(DEV)
    q, k, v, g = dev(x, "q", "k", "v", "g")
    o = mb.linattn_state_update(st, q, k, v, g, x["scale"])
    for i in range(b):
        one = [f64(x[n][i:i + 1]) for n in ("q", "k", "v")]
        want, wf = layer.linattn(*one, f64(x["g"]), x["scale"], f64(x["s0"][i]))
        mag, mf = layer.linattn(*(abs(t) for t in one), f64(x["g"]), x["scale"], abs(f64(x["s0"][i])))
        check(o[i], want[0], mag[0], dk + 4, dtype == BF, "o")
        check(st[i], wf, mf, 4, False, "state")


def test_step_strides_and_repeat():
    """A state inside a larger pool, strided tokens; many steps equal the forward over the same tokens."""
    b, H, d, T = 2, 3, 64, 40
    pool = torch.full((b, H + 2, d, d), 9.0, device=DEV)
    st = pool[:, 1:H + 1]
    x = make(b * T, H, H, d, d, F32, 3, n=b)
    st.copy_(x["s0"])
    q, k, v = (x[n].view(b, T, H, d).to(DEV) for n in ("q", "k", "v"))
    g = x["g"].to(DEV)
    outs = [mb.linattn_state_update(st, q[:, t], k[:, t], v[:, t], g) for t in range(T)]
    check_fwd(x, [0, T, 2 * T], torch.stack(outs, 1).flatten(0, 1), st, F32)
    assert (pool[:, 0] == 9.0).all() and (pool[:, -1] == 9.0).all()


def test_prompt_then_tokens_in_a_graph():
    """Forward over a prompt, then captured steps from its state: the forward over all tokens."""
    b, L, T, H, G, d = 2, 150, 6, 4, 2, 64
    x = make(b * (L + T), H, G, d, d, BF, 90, n=b)
    q, k, v = (x[n].view(b, L + T, -1, d).to(DEV) for n in ("q", "k", "v"))
    g = x["g"].to(DEV)
    o, st = mb.linattn_fwd(q[:, :L], k[:, :L], v[:, :L], g, initial_state=x["s0"].to(DEV))
    first = st.clone()
    tok = [t[:, L].clone() for t in (q, k, v)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mb.linattn_state_update(st, *tok, g)  # (loads the kernel before the capture)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        y = mb.linattn_state_update(st, *tok, g)
    st.copy_(first)
    outs = [o]
    for t in range(T):
        for a, full in zip(tok, (q, k, v)):
            a.copy_(full[:, L + t])
        graph.replay()
        outs.append(y[:, None].clone())
    check_fwd(x, [0, L + T, 2 * (L + T)], torch.cat(outs, 1).flatten(0, 1), st, BF)


def test_step_state_beyond_32_bit_offsets():
    """Two rows' states 2^32 elements apart in one pool."""
    H, dk, dv = 2, 64, 64
    pool = torch.zeros(2 ** 32 + H * dk * dv, device=DEV)
    st = pool.as_strided((2, H, dk, dv), (2 ** 32, dk * dv, dv, 1))
    x = make(2, H, H, dk, dv, F32, 5, n=2)
    st.copy_(x["s0"])
    q, k, v, g = dev(x, "q", "k", "v", "g")
    o = mb.linattn_state_update(st, q, k, v, g, x["scale"])
    dense = x["s0"].to(DEV)
    ref = mb.linattn_state_update(dense, q, k, v, g, x["scale"])
    assert torch.equal(o, ref) and torch.equal(st, dense)
    assert pool[H * dk * dv:H * dk * dv + 1000].abs().max() == 0


@pytest.mark.parametrize("starts,lo,hi", [([0, 90, 200, 230], 0, 200), ([-7, 30, 150, 200], 30, 200)])
def test_shared_heads_rows_of_bad_sequences_stay(starts, lo, hi):
    """The sum over shared heads leaves rows of a sequence that is left out as they were, too."""
    x = make(200, 4, 2, 64, 64, BF, 62, n=3)
    q, k, v, g, do = dev(x, "q", "k", "v", "g", "do")
    st = torch.tensor(starts, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    grads = {m: torch.full_like(t, 7.0) for m, t in (("dq", q), ("dk", k), ("dv", v))}
    mb.linattn_bwd(q, k, v, g, do, x["scale"], seq_start=st, grads=grads, dev_status=status)
    assert status.item() == mb.MS_ERR_SHAPE
    for t in grads.values():
        assert (t[:lo] == 7.0).all() and (t[hi:] == 7.0).all() and (t[lo:hi] != 7.0).float().mean() > 0.9


@pytest.mark.parametrize("dtype", [BF, F32])
def test_broadcast_inputs(dtype):
    """Keys, values and the gradient of o that rows or tokens share (stride 0) give what their copies give."""
    b, L, H, d = 2, 70, 3, 16
    x = make(L, H, H, d, d, dtype, 63)
    q, k, v, g, do = dev(x, "q", "k", "v", "g", "do")
    qb = torch.stack([q, -q])
    kb, vb = k[None].expand(b, L, H, d), v[:1, :1].expand(b, L, H, d)
    db = do[None].expand(b, L, H, d)
    o, fin = mb.linattn_fwd(qb, kb, vb, g)
    # (copies of bf16 run on the tensor cores, with its roundings)
    for i, sign in ((0, 1.0), (1, -1.0)):
        y = dict(x, q=sign * x["q"], v=x["v"][:1, :1].expand(L, H, d))
        want, fw = layer.linattn(f64(y["q"]), f64(y["k"]), f64(y["v"]), f64(x["g"]), d ** -0.5)
        mag, _ = layer.linattn(*(np.abs(f64(y[m])) for m in ("q", "k", "v")), f64(x["g"]), d ** -0.5)
        check(o[i], want, mag, 4 * L + d, dtype is BF, "o")
    # (of bf16, each way is within 4e-3 of the exact gradients, with roundings of its own: 4e-3 sqrt(2) apart)
    kc, vc = kb.contiguous(), vb.contiguous()
    gr, gc = (mb.linattn_bwd(qb, kc, vc, g, t) for t in (db, db.contiguous()))
    for m in ("dq", "dk", "dv"):
        a, c = gr[m].double(), gc[m].double()
        assert ((a - c).norm() / c.norm()).item() <= (6e-3 if dtype is BF else 1e-6)
    with pytest.raises(mb.MambaScanError):
        mb.linattn_bwd(qb, kb, vc, g, db)


def test_nan_decay_spoils_its_head_only():
    x = make(300, 2, 2, 64, 64, BF, 64)
    q, k, v, g = dev(x, "q", "k", "v", "g")
    g2 = g.clone()
    g2[1] = float("nan")
    (o, fin), (o2, fin2) = (mb.linattn_fwd(q[None], k[None], v[None], t) for t in (g, g2))
    assert torch.equal(o[:, :, 0], o2[:, :, 0]) and torch.equal(fin[:, 0], fin2[:, 0])
    assert o2[:, 1:, 1].isnan().all() and fin2[:, 1].isnan().all()


def test_conveniences_on_another_stream():
    """Given a stream, what a call allocates belongs to that stream: work queued on the current one may still
    use memory that was freed there."""
    x = make(600, 4, 2, 64, 64, BF, 65, n=1)
    q, k, v, g, do = dev(x, "q", "k", "v", "g", "do")
    want = mb.linattn_bwd(q[None], k[None], v[None], g, do[None])
    o, fin = mb.linattn_fwd(q[None], k[None], v[None], g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    junk = [torch.empty(1 << 24, device=DEV) for _ in range(4)]
    for t in junk:
        for _ in range(20):
            t.normal_()
    del junk, t
    got = mb.linattn_bwd(q[None], k[None], v[None], g, do[None], stream=side)
    o2, fin2 = mb.linattn_fwd(q[None], k[None], v[None], g, stream=side)
    o3 = mb.linattn_state_update(fin2, q[:1], k[:1], v[:1], g, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, o2)
    for m in ("dq", "dk", "dv", "dinitial_state"):
        assert torch.equal(want[m], got[m])
    assert torch.equal(o3, mb.linattn_state_update(fin, q[:1], k[:1], v[:1], g)) and torch.equal(fin, fin2)


@pytest.mark.parametrize("L", [3, 7, 8, 9, 12])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 40)])
def test_few_tokens(L, dk, dv):
    """On both sides of the number of tokens from which chunks are used: dense, packed, and shared heads."""
    run_dense(make(3 * L, 4, 2, dk, dv, BF, 70 + L, n=3), 3, L, BF)
    run_packed(make(L, 4, 2, dk, dv, BF, 80 + L, n=4), [0, 1, 1, 3, L], BF)
