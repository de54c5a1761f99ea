"""Operators for training a block around the frame-aligned attention: what is measured.

Three operators, in their plain form (elementary torch operations) and, where
``own`` is true, as calls of the framework:

* attention's backward pass, which recomputes the probabilities
  (``fas_backward``);
* the norm after a block, its gate and residual, and the norm before the next
  one, forward and backward (``fas_residual_norm``,
  ``fas_residual_norm_backward``);
* activation checkpoints in 8 bits: 32-element blocks of e4m3 codes under one
  power of two (``fas_checkpoint_pack``, ``fas_checkpoint_unpack``), written
  by the norm's forward and read by its backward.
"""
import math

import torch

own = False

EPS = 1e-6
#: Listed geometries: the super-resolution chunks (frames of 3600 tokens at
#: 720p, of 8160 at 1080p), the mid and tiny ones, and frames of unequal spans.
RAGGED = "3600,3520,3600,3680,3600,3440,3600"


def listed():
    return [
        # A smoke-sized chunk, every launch's latency in full view.
        dict(name="bwd_tiny", op="bwd", heads=2, dim=64, spans=",".join(["48"] * 9), ref=1, radius=1, layout="hnd", sharp=0),
        # One layer of a small model: all heads on one GPU.
        dict(name="bwd_mid", op="bwd", heads=16, dim=128, spans=",".join(["880"] * 17), ref=1, radius=2, layout="hnd", sharp=0),
        # Frames of unequal spans, token-major as a projection writes them.
        dict(name="bwd_ragged", op="bwd", heads=6, dim=128, spans=RAGGED, ref=1, radius=2, layout="nhd", sharp=1),
        # A 720p chunk's heads on one of four sequence-parallel ranks; one
        # head's logits are sharp.
        dict(name="bwd_720p", op="bwd", heads=6, dim=128, spans=",".join(["3600"] * 22), ref=1, radius=2, layout="hnd", sharp=1),
        # One token through the norms: the call's latency.
        dict(name="norm_token", op="norm", width=2048, spans="1", residual="bf16", gated=1),
        # One layer of a small model, gates per frame.
        dict(name="norm_mid", op="norm", width=2048, spans=",".join(["880"] * 17), residual="bf16", gated=1),
        # fp32 residual stream, frames of unequal spans, with checkpoints of
        # both inputs of the backward pass, which recomputation unpacks.
        dict(name="norm_ckpt", op="norm_ckpt", width=1536, spans=RAGGED, residual="fp32", gated=1),
        # A smoke-sized backward pass: latency.
        dict(name="norm_bwd_tiny", op="norm_bwd", width=128, spans=",".join(["48"] * 9), residual="bf16", gated=1, bits=16),
        dict(name="norm_bwd_mid", op="norm_bwd", width=2048, spans=",".join(["880"] * 17), residual="bf16", gated=1, bits=16),
        # A whole 720p chunk's backward from 8-bit checkpoints.
        dict(name="norm_bwd_8bit", op="norm_bwd", width=2048, spans=",".join(["3600"] * 22), residual="bf16", gated=1, bits=8),
        # A 720p chunk's hidden states into 8 bits, and one frame's out again.
        dict(name="pack_720p", op="pack", width=2048, rows=79200, residual="bf16"),
        dict(name="unpack_frame", op="unpack", width=2048, rows=880, residual="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bwd", "bwd", "norm", "norm_ckpt", "norm_bwd", "norm_bwd", "pack", "unpack"])
    if op == "bwd":
        while True:
            ref, frames = rng.choice([0, 1, 1, 2]), rng.randint(1, 22)
            base = 16 * _log(rng, 1, 510)
            if rng.random() < 0.5:
                spans = [base] * (ref + frames)
            else:
                spans = [16 * max(1, round(base / 16 * rng.uniform(0.5, 1.5))) for _ in range(ref + frames)]
            case = dict(op=op, heads=_log(rng, 1, 24), dim=rng.choice([64, 128]), spans=",".join(map(str, spans)), ref=ref,
                        radius=rng.randint(0, 5), layout=rng.choice(["hnd", "nhd"]), sharp=rng.choice([0, 1]))
            if work(case)["flops"] <= work(listed()[3])["flops"]:
                return case
    while True:
        rows = _log(rng, 1, 120000)
        width = 32 * _log(rng, 1, 256)
        residual = rng.choice(["bf16", "bf16", "fp32"])
        if op in ("pack", "unpack"):
            case = dict(op=op, width=width, rows=rows, residual=residual)
        else:
            n = min(rows, rng.randint(1, 22))
            cuts = sorted(rng.sample(range(1, rows), n - 1)) if rng.random() < 0.5 else [rows * i // n for i in range(1, n)]
            spans = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
            case = dict(op=op, width=width, spans=",".join(map(str, spans)), residual=residual, gated=rng.choice([1, 1, 0]))
            if op == "norm_bwd":
                case["bits"] = rng.choice([16, 8])
            elif op == "norm":
                case["width"] = width = width + 8 * rng.randint(0, 3)  # without checkpoints any multiple of 8 goes
        if rows * width <= 79200 * 2048 and work(case)["bytes"] <= work(listed()[9])["bytes"]:
            return case


def _spans(case):
    return [int(t) for t in case["spans"].split(",")]


def _visible(spans, ref, radius):
    """Per frame, the token ranges it sees: the reference frames see all; the
    others the reference frames and the frames at most `radius` away."""
    at = [0]
    for t in spans:
        at.append(at[-1] + t)
    seen = []
    for f in range(len(spans)):
        if f < ref:
            seen.append([(0, at[-1])])
            continue
        lo, hi = max(ref, f - radius), min(len(spans) - 1, f + radius)
        seen.append([(0, at[hi + 1])] if lo == ref else [(0, at[ref]), (at[lo], at[hi + 1])] if ref else [(at[lo], at[hi + 1])])
    return at, seen


def work(case):
    op = case["op"]
    if op == "bwd":
        spans = _spans(case)
        _, seen = _visible(spans, case["ref"], case["radius"])
        pairs = sum(t * sum(b - a for a, b in s) for t, s in zip(spans, seen)) * case["heads"]
        n = sum(spans) * case["heads"]
        return {"bytes": n * (case["dim"] * 2 * 8 + 4), "flops": 10 * case["dim"] * pairs}
    res = 2 if case["residual"] == "bf16" else 4
    if op in ("pack", "unpack"):
        n = case["rows"] * case["width"]
        return {"bytes": n * (res + 1 + 1 / 32), "flops": 4 * n}
    spans = _spans(case)
    rows, c = sum(spans), case["width"]
    n = rows * c
    small = 4 * c * (2 + len(spans) * case["gated"]) + 8 * rows
    if op == "norm":
        return {"bytes": n * (2 + res + res + 2) + small, "flops": 12 * n}
    if op == "norm_ckpt":  # and both checkpoints written, read once and given out in 16 bits
        return {"bytes": n * (2 + res + res + 2 + 4 * (1 + 1 / 32) + 4) + small, "flops": 24 * n}
    held = 2 + res if case["bits"] == 16 else 2 * (1 + 1 / 32)
    return {"bytes": n * (res + 2 + held + res + 2) + 2 * small, "flops": 24 * n}


# --- inputs -----------------------------------------------------------------


def _attention(q, k, v, case):
    """out (bf16) and lse (fp32) of head-major q, k, v: what the forward pass left."""
    at, seen = _visible(_spans(case), case["ref"], case["radius"])
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    kf, vf = k.float(), v.float()
    for f, ranges in enumerate(seen):
        rows = slice(at[f], at[f + 1])
        ks, vs = (torch.cat([t[:, a:b] for a, b in ranges], 1) for t in (kf, vf))
        s = q[:, rows].float() @ ks.transpose(1, 2)
        s /= math.sqrt(case["dim"])
        lse[:, rows] = torch.logsumexp(s, 2)
        s -= lse[:, rows, None]
        out[:, rows] = (s.exp_() @ vs).to(torch.bfloat16)
    return out, lse


def _pack_plain(x):
    """e4m3 codes and exponent bytes of 32-element blocks, in elementary operations."""
    b = x.float().reshape(*x.shape[:-1], -1, 32)
    a = torch.where(torch.isfinite(b), b.abs(), torch.zeros_like(b)).amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1): a <= 448 2^(e-9) exactly where m <= 0.875
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(a > 0, e.clamp_min(-127), torch.full_like(e, -127))
    y = torch.ldexp(b, -e[..., None])
    y = torch.where(torch.isfinite(b), y, torch.full_like(y, math.nan))
    return y.to(torch.float8_e4m3fn).reshape(x.shape), (e + 127).to(torch.uint8)


def _unpack_plain(codes, scales):
    b = codes.float().reshape(*codes.shape[:-1], -1, 32)
    return torch.ldexp(b, scales.int()[..., None] - 127).reshape(codes.shape)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + 17)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    op = case["op"]
    st = {"case": case}
    if op == "bwd":
        h, n, d = case["heads"], sum(_spans(case)), case["dim"]
        q, v, dout = rand(h, n, d), rand(h, n, d), rand(h, n, d)
        k = rand(h, n, d) + 3.0 * rand(h, 1, d)  # keys share a large common component
        if case["sharp"]:
            q[int(torch.randint(h, (1,), generator=gen, device=dev))] *= 8.0
        q, k, v, dout = (t.to(torch.bfloat16) for t in (q, k, v, dout))
        out, lse = _attention(q, k, v, case)
        if case["layout"] == "nhd":
            q, k, v, out, dout = (t.transpose(0, 1).contiguous() for t in (q, k, v, out, dout))
        frame = torch.repeat_interleave(torch.arange(len(_spans(case)), device=dev), torch.tensor(_spans(case), device=dev))
        return st | dict(q=q, k=k, v=v, out=out, dout=dout, lse=lse, frame=frame)
    res = torch.bfloat16 if case["residual"] == "bf16" else torch.float32
    if op in ("pack", "unpack"):
        # Hidden states: unit scale with a few strong channels.
        x = rand(case["rows"], case["width"]) * torch.exp(1.5 * rand(1, case["width"]))
        x = x.to(res)
        if op == "pack":
            return st | dict(x=x)
        codes, scales = _pack_plain(x)
        return st | dict(codes=codes, scales=scales, dtype=res)
    spans = _spans(case)
    n, c = sum(spans), case["width"]
    st |= dict(spans=spans if len(set(spans)) > 1 else spans[0], alpha=0.7, gate=0.5 * rand(len(spans), c) if case["gated"] else None,
               gamma_post=1.0 + 0.1 * rand(c), gamma_pre=1.0 + 0.1 * rand(c),
               frame=torch.repeat_interleave(torch.arange(len(spans), device=dev), torch.tensor(spans, device=dev)))
    channels = torch.exp(0.5 * rand(1, c))
    y = (rand(n, c) * channels).to(torch.bfloat16)
    x = (2.0 * rand(n, c) * channels).to(res)
    if op != "norm_bwd":
        return st | dict(y=y, x=x)
    rstd = torch.stack([torch.rsqrt(t.float().square().mean(1) + EPS) for t in (y, x)])
    dx_out, dh = rand(n, c).to(res), rand(n, c).to(torch.bfloat16)
    st |= dict(rstd=rstd, dx_out=dx_out, dh=dh)
    if case["bits"] == 8:
        return st | dict(y8=_pack_plain(y), x8=_pack_plain(x))
    return st | dict(y=y, x=x)


# --- plain forms ------------------------------------------------------------


def _bwd_plain(st):
    case = st["case"]
    q, k, v, out, dout, lse = (st[t] for t in ("q", "k", "v", "out", "dout", "lse"))
    if case["layout"] == "nhd":
        q, k, v, out, dout = (t.transpose(0, 1) for t in (q, k, v, out, dout))
    q, k, v, out, dout = (t.float() for t in (q, k, v, out, dout))
    scale = 1.0 / math.sqrt(case["dim"])
    delta = (dout * out).sum(2, keepdim=True)
    h, n, _ = q.shape
    if h * n * n <= 1 << 28:  # few tokens: all pairs at once, the hidden ones masked
        f = st["frame"]
        seen = (f[:, None] - f[None, :]).abs() <= case["radius"]
        seen |= (f[:, None] < case["ref"]) | (f[None, :] < case["ref"])
        p = torch.where(seen, torch.exp(q @ k.transpose(1, 2) * scale - lse[:, :, None]), 0.0)
        ds = p * (dout @ v.transpose(1, 2) - delta) * scale
        dq, dk, dv = ds @ k, ds.transpose(1, 2) @ q, p.transpose(1, 2) @ dout
    else:  # one frame's rows at a time over the tokens it sees
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
        at, seen = _visible(_spans(case), case["ref"], case["radius"])
        for i, ranges in enumerate(seen):
            rows = slice(at[i], at[i + 1])
            ks, vs = (torch.cat([t[:, a:b] for a, b in ranges], 1) for t in (k, v))
            p = torch.exp(q[:, rows] @ ks.transpose(1, 2) * scale - lse[:, rows, None])
            ds = p * (dout[:, rows] @ vs.transpose(1, 2) - delta[:, rows]) * scale
            dq[:, rows] = ds @ ks
            dks, dvs = ds.transpose(1, 2) @ q[:, rows], p.transpose(1, 2) @ dout[:, rows]
            o = 0
            for a, b in ranges:
                dk[:, a:b] += dks[:, o:o + b - a]
                dv[:, a:b] += dvs[:, o:o + b - a]
                o += b - a
    if case["layout"] == "nhd":
        dq, dk, dv = (t.transpose(0, 1) for t in (dq, dk, dv))
    return tuple(t.to(torch.bfloat16).contiguous() for t in (dq, dk, dv))


def _norm_plain(st):
    y, x = st["y"].float(), st["x"].float()
    ry = torch.rsqrt(y.square().mean(1) + EPS)
    u = y * ry[:, None] * st["gamma_post"] * st["alpha"]
    if st["gate"] is not None:
        u = u * st["gate"][st["frame"]]
    x = x + u
    rx = torch.rsqrt(x.square().mean(1) + EPS)
    return x.to(st["x"].dtype), (x * rx[:, None] * st["gamma_pre"]).to(torch.bfloat16), torch.stack([ry, rx])


def _norm_bwd_plain(st):
    case = st["case"]
    if case["bits"] == 8:
        y, x = _unpack_plain(*st["y8"]), _unpack_plain(*st["x8"])
    else:
        y, x = st["y"].float(), st["x"].float()
    yh, xh = y * st["rstd"][0][:, None], x * st["rstd"][1][:, None]
    dh = st["dh"].float()
    a = dh * st["gamma_pre"]
    g = st["dx_out"].float() + st["rstd"][1][:, None] * (a - xh * (a * xh).mean(1, keepdim=True))
    b = g * st["gamma_post"] * st["alpha"]
    if st["gate"] is not None:
        b = b * st["gate"][st["frame"]]
    dy = st["rstd"][0][:, None] * (b - yh * (b * yh).mean(1, keepdim=True))
    z = torch.stack([t.sum(0, dtype=torch.float64) for t in (yh * g).split(_spans(case))])
    gate = 1.0 if st["gate"] is None else st["gate"].double()
    dgamma_post = (z * gate).sum(0) * st["alpha"]
    dgamma_pre = (dh * xh).sum(0, dtype=torch.float64)
    dgate = None if st["gate"] is None else (z * st["gamma_post"] * st["alpha"]).float()
    return g.to(st["dx_out"].dtype), dy.to(torch.bfloat16), dgamma_post.float(), dgamma_pre.float(), dgate


# --- the framework's calls ---------------------------------------------------

_planned = None  # the attention geometry the library's plan is for; a program plans once per geometry


def _run_own(st):
    global _planned
    import frame_aligned_sparse_gb300 as fas
    case = st["case"]
    op = case["op"]
    if op == "bwd":
        geometry = (case["spans"], case["ref"], case["radius"], case["heads"], case["dim"], case["layout"])
        if _planned != geometry:
            spans = _spans(case)
            fas.fas_plan(spans[0] if len(set(spans)) == 1 else spans, len(spans) - case["ref"], case["ref"], case["radius"],
                         case["heads"], case["dim"])
            fas.fas_set_layout(case["layout"])
            _planned = geometry
        return fas.fas_backward(st["q"], st["k"], st["v"], st["out"], st["lse"], st["dout"])
    if op == "pack":
        return tuple(fas.fas_checkpoint_pack(st["x"]))
    if op == "unpack":
        return fas.fas_checkpoint_unpack((st["codes"], st["scales"]), dtype=st["dtype"])
    if op == "norm":
        return fas.fas_residual_norm(st["y"], st["x"], st["gamma_post"], st["gamma_pre"], gate=st["gate"], frame_tokens=st["spans"],
                                     alpha=st["alpha"], eps=EPS)
    if op == "norm_ckpt":
        x, h, rstd, y8, x8 = fas.fas_residual_norm(st["y"], st["x"], st["gamma_post"], st["gamma_pre"], gate=st["gate"],
                                                   frame_tokens=st["spans"], alpha=st["alpha"], eps=EPS, checkpoint=True)
        return x, h, rstd, fas.fas_checkpoint_unpack(y8), fas.fas_checkpoint_unpack(x8)
    y, x = (st["y8"], st["x8"]) if case["bits"] == 8 else (st["y"], st["x"])
    return fas.fas_residual_norm_backward(st["dx_out"], st["dh"], y, x, st["rstd"], st["gamma_post"], st["gamma_pre"], gate=st["gate"],
                                          frame_tokens=st["spans"], alpha=st["alpha"])


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "bwd":
        return _bwd_plain(state)
    if op == "pack":
        return _pack_plain(state["x"])
    if op == "unpack":
        return _unpack_plain(state["codes"], state["scales"]).to(state["dtype"])
    if op == "norm":
        return _norm_plain(state)
    if op == "norm_ckpt":
        x, h, rstd = _norm_plain(state)
        return x, h, rstd, _unpack_plain(*_pack_plain(state["y"])).bfloat16(), _unpack_plain(*_pack_plain(x)).bfloat16()
    return _norm_bwd_plain(state)


# --- the definition in 64 bits ------------------------------------------------


def _nearest_e4m3(t):
    """The nearest value of 3 mantissa bits, exponents from -6, ties to even (|t| <= 448)."""
    e = torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -60))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return torch.round(t / step) * step


def _held(x):
    """What an 8-bit checkpoint of x stands for, and its codes' values and exponents."""
    b = x.double().unflatten(-1, (-1, 32))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((a / 448).clamp_min(2.0 ** -127)))
    e = torch.where(torch.exp2(e - 1) * 448 >= a, e - 1, e)  # where the logarithm was rounded up
    e = torch.where(torch.exp2(e) * 448 < a, e + 1, e).clamp_min(-127)
    c = _nearest_e4m3(b / torch.exp2(e))
    return (c * torch.exp2(e)).flatten(-2), c.flatten(-2), (e.squeeze(-1) + 127)


def exact(case, seed):
    op = case["op"]
    if op == "bwd":
        spans = _spans(case)
        n, h, d = sum(spans), case["heads"], case["dim"]
        if 10.0 * d * h * n * n > 5e12:  # all pairs, at the rate of 64 bits
            return None
        st = prepare(case, seed)
        names = ("q", "k", "v", "out", "dout")
        q, k, v, out, dout = (st[t].transpose(0, 1) if case["layout"] == "nhd" else st[t] for t in names)
        f = st["frame"]
        grads = torch.zeros(3, h, n, d, dtype=torch.float64, device=q.device)
        step = max(1, min(n, (1 << 27) // n))
        for i in range(h):
            qi, ki, vi, oi, di = (t[i].double() for t in (q, k, v, out, dout))
            for r in range(0, n, step):
                s = slice(r, r + step)
                hidden = ((f[s, None] - f[None]).abs() > case["radius"]) & (f[s, None] >= case["ref"]) & (f[None] >= case["ref"])
                logits = torch.einsum("ic,jc->ij", qi[s], ki) / d ** 0.5
                p = torch.exp((logits - st["lse"][i, s, None].double()).masked_fill(hidden, -math.inf))
                ds = p * (torch.einsum("ic,jc->ij", di[s], vi) - torch.einsum("ic,ic->i", di[s], oi[s])[:, None]) / d ** 0.5
                grads[0, i, s] = torch.einsum("ij,jc->ic", ds, ki)
                grads[1, i] += torch.einsum("ij,ic->jc", ds, qi[s])
                grads[2, i] += torch.einsum("ij,ic->jc", p, di[s])
        return tuple((t.transpose(0, 1) if case["layout"] == "nhd" else t).contiguous() for t in grads)
    st = prepare(case, seed)
    if op == "pack":
        _, codes, _ = _held(st["x"])
        return codes, None
    if op == "unpack":
        e = st["scales"].double().repeat_interleave(32, 1) - 127
        return st["codes"].double() * torch.exp2(e)
    gate = torch.ones(1, 1, dtype=torch.float64, device=st["frame"].device) if st["gate"] is None else st["gate"].double()[st["frame"]]
    gate = gate * st["alpha"]
    c = case["width"]
    post, pre = st["gamma_post"].double(), st["gamma_pre"].double()
    if op in ("norm", "norm_ckpt"):
        y, x = st["y"].double(), st["x"].double()
        ry = (EPS + (y * y).sum(1) / c) ** -0.5
        new = x + torch.einsum("nc,n,c->nc", y, ry, post) * gate
        rx = (EPS + (new * new).sum(1) / c) ** -0.5
        got = (new, torch.einsum("nc,n,c->nc", new, rx, pre), torch.stack([ry, rx]))
        # What the checkpoint of the sum stands for hangs on roundings of the sum that lie on a border of its 8 bits: no value.
        return got if op == "norm" else got + (_held(st["y"])[0], None)
    ry, rx = st["rstd"].double()
    if case["bits"] == 8:
        y, x = ((t[0].double().unflatten(1, (-1, 32)) * torch.exp2(t[1].double() - 127)[:, :, None]).flatten(1) for t in (st["y8"], st["x8"]))
    else:
        y, x = st["y"].double(), st["x"].double()
    dh = st["dh"].double()
    along = torch.einsum("nc,c,nc,n->n", dh, pre, x, rx) / c
    g = st["dx_out"].double() + rx[:, None] * (dh * pre) - torch.einsum("nc,n->nc", x, rx * rx * along)
    b = g * gate * post
    dy = ry[:, None] * b - torch.einsum("nc,n->nc", y, ry ** 3 * torch.einsum("nc,nc->n", b, y) / c)
    z = torch.einsum("nc,n,nc->nc", y, ry, g)
    dgate = None
    if st["gate"] is not None:
        dgate = torch.zeros_like(st["gate"], dtype=torch.float64).index_add_(0, st["frame"], z) * post * st["alpha"]
    return g, dy, (z * gate).sum(0), torch.einsum("nc,nc,n->c", dh, x, rx), dgate
