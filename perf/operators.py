"""Cases of the linear-attention layer and of the norms around it, for timing.

Three operators, each in its forward and backward direction and the first also
for single tokens:

* linear attention with one decay per head. With S the [dk, dv] state of a head,
  lam = exp(log_decay[h]) and a the scale,
      S_t = lam S_{t-1} + k_t v_t^T        o_t = a q_t S_t
  over whole sequences (batches or packed ragged ones), its gradients, and one
  token from a stored state;
* the gated group norm behind the layer: norm(x) w silu(z), or norm(x silu(z)) w;
* the residual add and norm in front of the next layer:
      r' = r + s c x,   y = norm(r') w.

``own`` false: elementary torch operations in 32 bits. ``own`` true: the calls
of the package.
"""
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases ----

def listed():
    bf, f32 = "bf16", "f32"
    return [
        # a training or prefill batch of the 130M-class layer: inner width 1536 as 24 heads of 64
        dict(name="la_fwd_batch", op="la_fwd", batch=8, length=2048, heads=24, kv=24, dk=64, dv=64, ragged=0, state=0),
        # one long document, few heads: only the length gives the card work
        dict(name="la_fwd_long", op="la_fwd", batch=1, length=65536, heads=16, kv=16, dk=128, dv=128, ragged=0, state=1),
        # prompts of mixed lengths packed behind one another, keys and values shared by 4 heads each
        dict(name="la_fwd_ragged", op="la_fwd", batch=13, length=9001, heads=32, kv=8, dk=128, dv=128, ragged=1, state=1),
        # one short prompt: latency
        dict(name="la_fwd_short", op="la_fwd", batch=1, length=100, heads=24, kv=24, dk=64, dv=64, ragged=0, state=0),
        # gradients of a training batch at the 130M-class width
        dict(name="la_bwd_batch", op="la_bwd", batch=4, length=2048, heads=24, kv=24, dk=64, dv=64, ragged=0, state=0),
        # gradients with shared keys and values, carried states, odd lengths
        dict(name="la_bwd_shared", op="la_bwd", batch=2, length=4001, heads=16, kv=4, dk=128, dv=96, ragged=0, state=1),
        # generation for 64 sequences of the 2.7B-class layer: 80 heads, state 128 x 64
        dict(name="la_step_b64", op="la_step", batch=64, heads=80, kv=80, dk=128, dv=64, dtype=bf),
        # generation for one sequence: latency
        dict(name="la_step_b1", op="la_step", batch=1, heads=24, kv=24, dk=64, dv=64, dtype=f32),
        # per-head norm and gate behind the 130M-class layer's 24 heads
        dict(name="gnorm_fwd_heads", op="gnorm_fwd", rows=16384, width=1536, groups=24, first=0, dtype=bf),
        # gate first, one norm over the whole inner width of the 2.7B-class layer, training
        dict(name="gnorm_bwd_wide", op="gnorm_bwd", rows=8192, width=5120, groups=1, first=1, dtype=bf),
        # residual add and norm of one generation step (64 sequences, model width 2560)
        dict(name="rnorm_fwd_step", op="rnorm_fwd", rows=64, width=2560, dtype=bf, rdtype=f32, channel=0),
        # the same with a scale per channel, gradients of a training batch
        dict(name="rnorm_bwd_train", op="rnorm_bwd", rows=8192, width=2560, dtype=bf, rdtype=f32, channel=1),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_fwd", "la_bwd", "la_step", "gnorm_fwd", "gnorm_bwd", "rnorm_fwd", "rnorm_bwd"])
    if op in ("la_fwd", "la_bwd"):
        kv, share = _log(rng, 1, 32), rng.choice([1, 1, 2, 4])
        dk, dv = (rng.choice([16, 40, 64, 80, 128, 128]) for _ in range(2))
        batch = _log(rng, 1, 24)
        length = _log(rng, 1, 16384)
        ragged = rng.choice([0, 1])
        tokens = length if ragged else batch * length
        most = (1_000_000 if op == "la_fwd" else 300_000) // (kv * share)  # token-heads: no dearer than the largest above
        if tokens > most:
            length = max(1, most if ragged else most // batch)
        return dict(op=op, batch=batch, length=length, heads=kv * share, kv=kv, dk=dk, dv=dv, ragged=ragged, state=rng.choice([0, 1]))
    if op == "la_step":
        kv, share = _log(rng, 1, 40), rng.choice([1, 1, 2])
        return dict(op=op, batch=_log(rng, 1, 64), heads=kv * share, kv=kv, dk=rng.choice([16, 40, 64, 128]),
                    dv=rng.choice([8, 40, 64, 72, 128]), dtype=rng.choice(["bf16", "f32"]))
    rows, dtype = _log(rng, 1, 16384), rng.choice(["bf16", "bf16", "f32"])
    if op in ("gnorm_fwd", "gnorm_bwd"):
        groups = rng.choice([1, 1, 2, 8, 20])
        width = groups * (_log(rng, 100, 5120) if groups == 1 else rng.choice([32, 33, 64, 96, 128, 200]))
        return dict(op=op, rows=rows, width=width, groups=groups, first=rng.choice([0, 1]), dtype=dtype)
    return dict(op=op, rows=rows, width=_log(rng, 100, 5120), dtype=dtype, rdtype=rng.choice([dtype, "f32"]),
                channel=rng.choice([0, 1]))


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _starts(case):
    """Where each of the packed sequences begins, and the end of the last; the rows behind it belong to none."""
    n, total = case["batch"], case["length"]
    used = total - total // 50
    gen = torch.Generator().manual_seed(n * 1000003 + total)
    cuts = torch.sort(torch.randint(0, used + 1, (n - 1,), generator=gen)).values.tolist() if n > 1 else []
    return [0] + cuts + [used]


def work(case):
    op = case["op"]
    if op in ("la_fwd", "la_bwd"):
        h, kv, dk, dv = case["heads"], case["kv"], case["dk"], case["dv"]
        tokens = _starts(case)[-1] if case["ragged"] else case["batch"] * case["length"]
        q, k, v, o = (2 * tokens * n for n in (h * dk, kv * dk, kv * dv, h * dv))
        st = 4 * case["batch"] * h * dk * dv
        if op == "la_fwd":
            return {"bytes": q + k + v + o + st * (1 + case["state"]), "flops": 4.0 * tokens * h * dk * dv}
        return {"bytes": 2 * (q + k + v) + o + st * (1 + 2 * case["state"]), "flops": 10.0 * tokens * h * dk * dv}
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "la_step":
        b, h, kv, dk, dv = (case[n] for n in ("batch", "heads", "kv", "dk", "dv"))
        return {"bytes": 8 * b * h * dk * dv + es * b * (h + kv) * (dk + dv), "flops": 5.0 * b * h * dk * dv}
    n, w = case["rows"] * case["width"], 4 * case["width"]
    if op == "gnorm_fwd":
        return {"bytes": 3 * n * es + w, "flops": 8.0 * n}
    if op == "gnorm_bwd":
        return {"bytes": 5 * n * es + 2 * w, "flops": 20.0 * n}
    rs = 2 if case["rdtype"] == "bf16" else 4
    if op == "rnorm_fwd":
        return {"bytes": 2 * n * (es + rs) + w * (1 + case["channel"]), "flops": 6.0 * n}
    return {"bytes": n * (2 * es + 3 * rs + es * case["channel"]) + 2 * w * (1 + case["channel"]), "flops": 14.0 * n}


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape, dtype=torch.float32, mul=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * mul).to(dtype)

    op, s = case["op"], {"case": dict(case)}
    if op.startswith("la_"):
        h, kv, dk, dv, b = (case[n] for n in ("heads", "kv", "dk", "dv", "batch"))
        # decays 1 - 2^-5 (some 30 tokens are remembered) to 1 - 2^-12 over the heads
        steps = torch.linspace(5.0, 12.0, h, dtype=torch.float64)
        s["log_decay"] = torch.log1p(-torch.exp2(-steps)).float().to(DEV)
        s["scale"] = dk ** -0.5
        lead = (b,) if op == "la_step" else (case["length"],) if case["ragged"] else (b, case["length"])
        t = _type(case.get("dtype", "bf16"))
        s["q"], s["k"], s["v"] = rand(*lead, h, dk, dtype=t), rand(*lead, kv, dk, dtype=t), rand(*lead, kv, dv, dtype=t)
        if op == "la_step":
            s["state"] = rand(b, h, dk, dv)
            return s
        s["s0"] = rand(b, h, dk, dv) if case["state"] else None
        s["starts"] = torch.tensor(_starts(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
        if op == "la_bwd":
            s["do"] = rand(*lead, h, dv, dtype=t)
            s["ds"] = rand(b, h, dk, dv) if case["state"] else None
            outs = {"dq": s["q"], "dk": s["k"], "dv": s["v"]}
        else:
            outs = {"o": torch.empty(*lead, h, dv, dtype=t, device="meta")}
        # the rows of a packed buffer behind the last sequence stay as the caller left them
        s["out"] = {n: torch.zeros(x.shape, dtype=t, device=DEV) for n, x in outs.items()}
        if case["ragged"]:
            # the longest sequence, which a caller that packed them knows (the plain form pads to it)
            at = _starts(case)
            s["longest"] = max(max(y - x for x, y in zip(at, at[1:])), 1)
        return s
    rows, width, t = case["rows"], case["width"], _type(case["dtype"])
    s["x"] = rand(rows, width, dtype=t)
    s["w"] = 1.0 + 0.1 * rand(width)
    if op.startswith("gnorm"):
        s["z"] = rand(rows, width, dtype=t)
    else:
        s["r"] = rand(rows, width, dtype=_type(case["rdtype"]), mul=2.0)
        s["c"] = 0.5 + 0.1 * rand(width) if case["channel"] else None
        s["s"] = 0.7
    if op.endswith("bwd"):
        s["dy"] = rand(rows, width, dtype=t)
        if op == "rnorm_bwd":
            s["dr"] = rand(rows, width, dtype=_type(case["rdtype"]))
    return s


# ------------------------------------------------------------- plain forms ----

CHUNK = 64
EPS = 1e-5


def _powers(log_decay, n):
    """lam^n for whole numbers n, exponents in 64 bits; n broadcast behind the heads."""
    return torch.exp(log_decay.double().view(-1, *([1] * n.dim())) * n).float()


def _chunks(x):
    b, length = x.shape[:2]
    n = -(-length // CHUNK)
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * CHUNK - length))
    return x.reshape(b, n, CHUNK, *x.shape[2:])


def _mix(x, y, z, log_decay, s0, first):
    """sum_{s <= t} lam^(t-s) (x_t . y_s) z_s + lam^(t+first) x_t s0, chunk by chunk."""
    length = x.shape[1]
    xc, yc, zc = _chunks(x), _chunks(y), _chunks(z)
    n, dev = xc.shape[1], x.device
    t, c = torch.arange(CHUNK, device=dev), torch.arange(n, device=dev)
    within = torch.where(t[:, None] >= t, _powers(log_decay, (t[:, None] - t).clamp(min=0)), 0.0)
    scores = torch.einsum("bcthd,bcshd->bchts", xc, yc) * within
    o = torch.einsum("bchts,bcshe->bcthe", scores, zc)
    if n > 1:
        ends = torch.einsum("bcshd,hs,bcshe->bchde", yc, _powers(log_decay, CHUNK - 1 - t), zc)
        over = torch.where(c[:, None] > c, _powers(log_decay, (CHUNK * (c[:, None] - 1 - c)).clamp(min=0)), 0.0)
        enter = torch.einsum("hij,bjhde->bihde", over, ends)
        o = o + torch.einsum("bcthd,bchde->bcthe", xc, enter) * _powers(log_decay, t + 1).t()[None, None, :, :, None]
    o = o.reshape(o.shape[0], n * CHUNK, *o.shape[3:])[:, :length]
    if s0 is not None:
        carried = _powers(log_decay, torch.arange(length, device=dev) + first).t()[None, :, :, None]
        o = o + torch.einsum("bthd,bhde->bthe", x, s0) * carried
    return o


def _sum(y, z, log_decay, expo, keep, s0, ends):
    """sum_s lam^expo[b, s] y_s z_s^T over the tokens kept, plus lam^ends[b] s0."""
    w = torch.where(keep[:, None], torch.exp(log_decay.double()[:, None] * expo.clamp(min=0)[:, None]).float(), 0.0)
    wc = _chunks(w.transpose(1, 2)[..., None])[..., 0]
    st = torch.einsum("bcshd,bcsh,bcshe->bchde", _chunks(y), wc, _chunks(z)).sum(1)
    if s0 is not None:
        st = st + torch.exp(log_decay.double() * ends[:, None]).float()[:, :, None, None] * s0
    return st


def _padded(s, names):
    """The sequences side by side, [n, longest, heads, d] in 32 bits, with each one's length and where its tokens lie."""
    ref = s["q"]
    if s["starts"] is None:
        lens = torch.full((ref.shape[0],), ref.shape[1], device=ref.device)
        return [s[n].float() for n in names], lens, None
    st = s["starts"].long()
    lens = st[1:] - st[:-1]
    at = torch.arange(s["longest"], device=ref.device)
    inside = at < lens[:, None]
    where = torch.where(inside, st[:-1, None] + at, 0)
    return [torch.where(inside[..., None, None], s[n].float()[where], 0.0) for n in names], lens, (where, inside)


def _unpad(x, place, like, out):
    """Back into the caller's buffer, rounded to its type."""
    if place is None:
        return x.to(out.dtype)
    where, inside = place
    out[where[inside]] = x[inside].to(out.dtype)
    return out


def _spread(x, heads):
    return x.repeat_interleave(heads // x.shape[2], dim=2)


def _turned(x, lens):
    """Each sequence in the order of its tokens from the last to the first (padding stays behind)."""
    at = torch.arange(x.shape[1], device=x.device)
    idx = torch.where(at < lens[:, None], lens[:, None] - 1 - at, at)
    return torch.gather(x, 1, idx[:, :, None, None].expand_as(x))


def _plain_la_fwd(s):
    (q, k, v), lens, place = _padded(s, ("q", "k", "v"))
    g, h = s["log_decay"], q.shape[2]
    k, v = _spread(k, h), _spread(v, h)
    o = s["scale"] * _mix(q, k, v, g, s["s0"], 1)
    at = torch.arange(q.shape[1], device=q.device)
    fin = _sum(k, v, g, lens[:, None] - 1 - at, at < lens[:, None], s["s0"], lens)
    return {"o": _unpad(o, place, s["q"], s["out"]["o"]), "state": fin}


def _plain_la_bwd(s):
    (q, k, v, do), lens, place = _padded(s, ("q", "k", "v", "do"))
    g, h, a, kv = s["log_decay"], q.shape[2], s["scale"], k.shape[2]
    k, v = _spread(k, h), _spread(v, h)
    s0 = s["s0"].transpose(2, 3) if s["s0"] is not None else None
    dq = a * _mix(do, v, k, g, s0, 1)
    rq, rk, rv, rdo = (_turned(x, lens) for x in (a * q, k, v, do))
    dv = _turned(_mix(rk, rq, rdo, g, s["ds"], 0), lens)
    dk = _turned(_mix(rv, rdo, rq, g, s["ds"].transpose(2, 3) if s["ds"] is not None else None, 0), lens)
    dk, dv = (x.reshape(*x.shape[:2], kv, h // kv, x.shape[3]).sum(3) for x in (dk, dv))
    at = torch.arange(q.shape[1], device=q.device)
    d0 = _sum(a * q, do, g, at.expand(len(lens), -1) + 1, at < lens[:, None], s["ds"], lens)
    out = {n: _unpad(x, place, s["q"], s["out"][n]) for n, x in (("dq", dq), ("dk", dk), ("dv", dv))}
    return {**out, "dstate": d0}


def _plain_la_step(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    h = q.shape[1]
    k, v = (x.repeat_interleave(h // x.shape[1], dim=1) for x in (k, v))
    st = s["state"] * torch.exp(s["log_decay"])[:, None, None] + k[..., :, None] * v[..., None, :]
    s["state"].copy_(st)
    return {"o": (s["scale"] * (q[..., :, None] * st).sum(2)).to(s["q"].dtype), "state": s["state"]}


def _grouped(x, groups):
    return x.reshape(x.shape[0], groups, -1)


def _plain_gnorm_fwd(s):
    c = s["case"]
    x, z = s["x"].float(), s["z"].float()
    gate = z / (1.0 + torch.exp(-z))
    if c["first"]:
        x = x * gate
    xg = _grouped(x, c["groups"])
    y = (xg * torch.rsqrt(xg.square().mean(-1, keepdim=True) + EPS)).reshape(x.shape) * s["w"]
    return {"y": (y if c["first"] else y * gate).to(s["x"].dtype)}


def _plain_gnorm_bwd(s):
    c, t = s["case"], s["x"].dtype
    x, z, dy = s["x"].float(), s["z"].float(), s["dy"].float()
    sig = 1.0 / (1.0 + torch.exp(-z))
    gate, dgate = z * sig, sig * (1.0 + z * (1.0 - sig))
    a = x * gate if c["first"] else x
    ag = _grouped(a, c["groups"])
    r = torch.rsqrt(ag.square().mean(-1, keepdim=True) + EPS)
    hat = (ag * r).reshape(x.shape)
    dn = dy if c["first"] else dy * gate
    dw = (dn * hat).sum(0)
    dh, hg = _grouped(dn * s["w"], c["groups"]), _grouped(hat, c["groups"])
    da = (r * (dh - hg * (dh * hg).mean(-1, keepdim=True))).reshape(x.shape)
    dx, dz = (da * gate, da * x * dgate) if c["first"] else (da, dy * hat * s["w"] * dgate)
    return {"dx": dx.to(t), "dz": dz.to(t), "dw": dw}


def _plain_rnorm_fwd(s):
    x = s["s"] * s["x"].float()
    r = s["r"].float() + (x if s["c"] is None else x * s["c"])
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["w"]
    return {"y": y.to(s["x"].dtype), "r": r.to(s["r"].dtype)}


def _plain_rnorm_bwd(s):
    r, dy = s["r"].float(), s["dy"].float()
    rs = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    hat = r * rs
    dh = dy * s["w"]
    dr = s["dr"].float() + rs * (dh - hat * (dh * hat).mean(-1, keepdim=True))
    out = {"dr": dr.to(s["r"].dtype), "dw": (dy * hat).sum(0)}
    dx = s["s"] * dr
    if s["c"] is not None:
        out["dc"] = (dx * s["x"].float()).sum(0)
        dx = dx * s["c"]
    out["dx"] = dx.to(s["x"].dtype)
    return out


# ----------------------------------------------------------------- passes ----

def _own(s):
    from selective_state_space_40_b200 import binding as mb
    c = s["case"]
    op = c["op"]
    if op == "la_fwd":
        o, fin = mb.linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], seq_start=s["starts"],
                                initial_state=s["s0"], o=s["out"]["o"])
        return {"o": o, "state": fin}
    if op == "la_bwd":
        g = mb.linattn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"], seq_start=s["starts"],
                           initial_state=s["s0"], dfinal=s["ds"], grads=s["out"])
        return {"dq": g["dq"], "dk": g["dk"], "dv": g["dv"], "dstate": g["dinitial_state"]}
    if op == "la_step":
        o = mb.linattn_state_update(s["state"], s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if op == "gnorm_fwd":
        return {"y": mb.gated_norm_fwd(s["x"], s["z"], s["w"], groups=c["groups"], eps=EPS, gate_first=bool(c["first"]))}
    if op == "gnorm_bwd":
        g = mb.gated_norm_bwd(s["x"], s["z"], s["w"], s["dy"], groups=c["groups"], eps=EPS, gate_first=bool(c["first"]))
        return {"dx": g["dx"], "dz": g["dz"], "dw": g["dweight"]}
    if op == "rnorm_fwd":
        y, r = mb.residual_norm_fwd(s["x"], s["r"], s["w"], eps=EPS, res_scale=s["s"], channel_scale=s["c"])
        return {"y": y, "r": r}
    g = mb.residual_norm_bwd(s["r"], s["w"], s["dy"], dresidual_out=s["dr"], x=s["x"] if s["c"] is not None else None,
                             eps=EPS, res_scale=s["s"], channel_scale=s["c"])
    out = {"dr": g["dresidual"], "dw": g["dweight"], "dx": g["dx"]}
    if s["c"] is not None:
        out["dc"] = g["dchannel_scale"]
    return out


_PLAIN = {"la_fwd": _plain_la_fwd, "la_bwd": _plain_la_bwd, "la_step": _plain_la_step, "gnorm_fwd": _plain_gnorm_fwd,
          "gnorm_bwd": _plain_gnorm_bwd, "rnorm_fwd": _plain_rnorm_fwd, "rnorm_bwd": _plain_rnorm_bwd}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------- 64-bit definition ----

def _exact_la(s):
    """The recurrence token by token (and backwards for the gradients), sequences and heads side by side."""
    bwd = s["case"]["op"] == "la_bwd"
    h, kv, b = s["case"]["heads"], s["case"]["kv"], s["case"]["batch"]
    if s["starts"] is None:
        begin = [i * s["case"]["length"] for i in range(b)]
        lens = [s["case"]["length"]] * b
    else:
        at = s["starts"].tolist()
        begin, lens = at[:-1], [y - x for x, y in zip(at, at[1:])]
    most = max(lens)
    flat = {n: s[n].reshape(-1, *s[n].shape[-2:]).double() for n in ("q", "k", "v") + (("do",) if bwd else ())}
    flat = {n: x if x.shape[1] == h else x[:, :, None].expand(-1, -1, h // kv, -1).flatten(1, 2) for n, x in flat.items()}
    lam = torch.exp(s["log_decay"].double())
    dk, dv, a = s["case"]["dk"], s["case"]["dv"], s["scale"]

    def laid(x):  # [most, b * h, d], zeros behind a sequence's end
        p = torch.zeros(most, b, h, x.shape[-1], dtype=torch.float64, device=DEV)
        for i, (st, n) in enumerate(zip(begin, lens)):
            p[:n, i] = x[st:st + n]
        return p.view(most, b * h, -1)

    live = (torch.arange(most, device=DEV)[:, None] < torch.tensor(lens, device=DEV)).double()  # [most, b]
    decay = (1.0 + live[:, :, None] * (lam - 1.0)).reshape(most, b * h, 1, 1)
    q, k, v = (laid(flat[n]) for n in ("q", "k", "v"))

    def back(x, template, heads=h):  # into the layout of the inputs
        out = torch.zeros(template.reshape(-1, *template.shape[-2:]).shape, dtype=torch.float64, device=DEV)
        x = x.view(most, b, h, -1).unflatten(2, (heads, h // heads)).sum(3)
        for i, (st, n) in enumerate(zip(begin, lens)):
            out[st:st + n] = x[:n, i]
        return out.view(template.shape)

    def initial(x):
        return torch.zeros(b * h, dk, dv, dtype=torch.float64, device=DEV) if x is None else x.double().reshape(b * h, dk, dv).clone()

    st, rows = initial(s["s0"]), torch.empty(most, b * h, dk if bwd else dv, dtype=torch.float64, device=DEV)
    do = laid(flat["do"]) if bwd else None
    for t in range(most):
        st.mul_(decay[t])
        st.baddbmm_(k[t, :, :, None], v[t, :, None])
        if bwd:
            torch.bmm(st, do[t, :, :, None], out=rows[t, :, :, None])
        else:
            torch.bmm(q[t, :, None], st, out=rows[t, :, None])
    rows *= a
    if not bwd:
        return {"o": back(rows, s["out"]["o"]), "state": st.view(b, h, dk, dv)}
    dq, dks, dvs = back(rows, s["q"]), torch.empty_like(k), torch.empty_like(v)
    r = initial(s["ds"])
    for t in reversed(range(most)):
        r.baddbmm_(q[t, :, :, None], do[t, :, None], alpha=a)
        torch.bmm(r, v[t, :, :, None], out=dks[t, :, :, None])
        torch.bmm(k[t, :, None], r, out=dvs[t, :, None])
        r.mul_(decay[t])
    return {"dq": dq, "dk": back(dks, s["k"], kv), "dv": back(dvs, s["v"], kv), "dstate": r.view(b, h, dk, dv)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("la_fwd", "la_bwd"):
        return _exact_la(s)
    if op == "la_step":
        h, n = case["heads"], case["heads"] // case["kv"]
        st = s["state"].double()
        q = s["q"].double()
        for i in range(h):
            st[:, i] *= torch.exp(s["log_decay"][i].double())
            st[:, i] += torch.einsum("bd,be->bde", s["k"][:, i // n].double(), s["v"][:, i // n].double())
        return {"o": torch.einsum("bhd,bhde->bhe", q, st) * s["scale"], "state": st}
    if op.startswith("gnorm"):
        return _exact_gnorm(s, case)
    x = s["x"].double() * s["s"]
    c = torch.ones_like(s["w"], dtype=torch.float64) if s["c"] is None else s["c"].double()
    w, r = s["w"].double(), s["r"].double()
    if op == "rnorm_fwd":
        r = torch.addcmul(r, x, c)
        return {"y": r / (r.norm(dim=1, keepdim=True) ** 2 / case["width"] + EPS).sqrt() * w, "r": r}
    var = r.norm(dim=1, keepdim=True) ** 2 / case["width"] + EPS
    dy = s["dy"].double()
    # y_j = r_j w_j var^-1/2; dvar/dr_i = 2 r_i / width
    along = (dy * w * r).sum(1, keepdim=True)
    dr = s["dr"].double() + dy * w / var.sqrt() - r * along / (case["width"] * var.sqrt() ** 3)
    out = {"dr": dr, "dw": torch.einsum("rw,rw->w", dy, r / var.sqrt()), "dx": dr * c * s["s"]}
    if s["c"] is not None:
        out["dc"] = torch.einsum("rw,rw->w", dr, x)
    return out


def _exact_gnorm(s, case):
    x, z = s["x"].double(), s["z"].double()
    e = torch.exp(-z)
    gate = z / (1 + e)
    w, n = s["w"].double(), case["width"] // case["groups"]
    a = x * gate if case["first"] else x
    var = (a.view(-1, case["groups"], n).norm(dim=2) ** 2 / n + EPS).repeat_interleave(n, dim=1)
    if case["op"] == "gnorm_fwd":
        return {"y": a * w / var.sqrt() * (1.0 if case["first"] else gate)}
    slope = 1 / (1 + e) + z * e / (1 + e) ** 2
    dy = s["dy"].double()
    up = dy if case["first"] else dy * gate
    along = (up * w * a).view(-1, case["groups"], n).sum(2).repeat_interleave(n, dim=1)
    da = up * w / var.sqrt() - a * along / (n * var.sqrt() ** 3)
    dw = torch.einsum("rw,rw->w", up, a / var.sqrt())
    if case["first"]:
        return {"dx": da * gate, "dz": da * x * slope, "dw": dw}
    return {"dx": da, "dz": dy * a * w / var.sqrt() * slope, "dw": dw}
