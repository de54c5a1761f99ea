"""Training operators on the GPU against 64-bit references: the attention's
backward pass, the residual norms and the 8-bit checkpoints.

Each tolerance is the reference's own bound for the roundings the kernels
make (tests/training_reference.py), or derived in the test.
"""
import numpy as np
import pytest
import torch

import frame_aligned_sparse_gb300 as fas
import training_reference as ref
import workloads
from training_reference import U16, U32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from frame_aligned_sparse_gb300 import build
    build.build()
    yield fas.load()
    fas.fas_free()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


# --------------------------------------------------------------- attention

def plan(spans, R0, r, h, d, layout="hnd"):
    uniform = len(set(spans)) == 1
    fas.fas_plan(spans[0] if uniform else list(spans), len(spans) - R0, R0, r, h, d)
    fas.fas_set_layout(layout)


class Attention:
    """Inputs of the backward pass in both layouts; out and lse from the forward kernel."""

    def __init__(self, spans, R0, r, h, d, layout="hnd", seed=0, mean=3.0, sharp=False):
        rnd = gen(seed)
        n = sum(spans)
        q, k, v, dout = rnd(h, n, d), rnd(h, n, d) + mean * rnd(h, 1, d), rnd(h, n, d), rnd(h, n, d)
        if sharp:
            q[0] *= 8
        self.geo = (spans, R0, r)
        self.layout = layout
        self.set(*(t.to(torch.bfloat16) for t in (q, k, v, dout)))
        plan(spans, R0, r, h, d, layout)
        self.out, self.lse = fas.fas_forward(self.q, self.k, self.v, mode="online")

    def set(self, *hnd):
        self.q, self.k, self.v, self.dout = (self.lay(t) for t in hnd)

    def lay(self, t):
        return t.transpose(0, 1).contiguous() if self.layout == "nhd" else t

    def hnd(self, t):
        return t.transpose(0, 1) if self.layout == "nhd" else t

    def run(self, **kw):
        got = fas.fas_backward(self.q, self.k, self.v, self.out, self.lse, self.dout, **kw)
        assert fas.fas_status() == fas.FAS_OK
        return dict(zip(("dq", "dk", "dv"), (self.hnd(t) for t in got)))

    def check(self, got, rows=None):
        want = ref.attention_backward(*(self.hnd(t) for t in (self.q, self.k, self.v, self.out)), self.lse,
                                      self.hnd(self.dout), *self.geo, rows=rows)
        for name, (w, bound, sd) in want.items():
            g = got[name].double()
            if rows is not None:
                g = g[:, rows]
            err = (g - w).abs()
            assert torch.all(err <= bound + 1e-30), (name, float((err / (bound + 1e-30)).max()))
            # Over all elements the errors are many independent roundings:
            # their norm stays near its deviation (a quarter above, for the
            # sample mean the common key component is taken out with).
            e, s = float(err.norm()), float(sd.norm())
            assert e <= 1.25 * s + 1e-30, (name, "error norm / deviation", e / s)


GEOMETRIES = [
    # spans, R0, r, H, d, layout
    ([16], 0, 0, 1, 64, "hnd"),
    ([16], 0, 0, 1, 128, "nhd"),
    ([48] * 9, 1, 1, 2, 64, "hnd"),
    ([48] * 9, 1, 1, 2, 64, "nhd"),
    ([128] * 3, 0, 1, 2, 128, "hnd"),
    ([144] * 5, 2, 1, 3, 128, "nhd"),
    ([272] * 4, 1, 0, 2, 64, "hnd"),
    ([880] * 4, 1, 1, 2, 128, "hnd"),
    ([16, 48, 128, 144, 32, 400], 1, 1, 2, 128, "hnd"),
    ([16, 48, 128, 144, 32, 400], 0, 2, 2, 64, "nhd"),
    ([112, 240, 16, 64, 368, 96], 2, 0, 1, 128, "nhd"),
    ([256, 16, 16, 16, 640], 1, 9, 2, 64, "hnd"),
]


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("geo", GEOMETRIES, ids=lambda g: "%d_%s_R%d_r%d_H%d_d%d_%s" % (
    len(g[0]), "u" if len(set(g[0])) == 1 else "ragged", *g[1:]))
def test_attention_backward(geo, sharp):
    c = Attention(*geo, sharp=sharp)
    c.check(c.run())


def test_attention_backward_at_full_size():
    """The 720p geometry with 4 heads, in the launch a user makes: sampled
    rows (frame edges, last tiles, reference rows) of every head."""
    w = workloads.get("720p_h4")
    spans = [w.frame_tokens] * w.total_frames
    c = Attention(spans, w.ref_frames, w.window_radius, w.heads, w.head_dim, sharp=True)
    got = c.run()
    rows = sorted({f * 3600 + r for f in (0, 1, 2, 11, 20, 21) for r in (0, 127, 128, 1777, 3583, 3584, 3599)})
    for h in range(w.heads):
        one = Attention.__new__(Attention)
        one.geo, one.layout = c.geo, "hnd"
        one.q, one.k, one.v, one.out, one.dout, one.lse = (t[h:h + 1] for t in (c.q, c.k, c.v, c.out, c.dout, c.lse))
        one.check({n: t[h:h + 1] for n, t in got.items()}, rows=torch.tensor(rows, device="cuda"))
    again = c.run()
    for n in got:
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("geo", [([3600] * 4, 1, 1, 2, 64, "hnd"), ([880] * 9, 1, 2, 4, 64, "nhd"),
                                 ([1000 // 16 * 16, 16, 2064, 3600], 1, 1, 2, 64, "nhd")], ids=["3600", "880", "ragged"])
def test_attention_backward_of_long_frames_with_narrow_heads(geo):
    """Heads of 64 on frames of many blocks: sampled rows of every frame."""
    c = Attention(*geo, sharp=True)
    ends = np.cumsum([0] + geo[0])
    rows = sorted({int(min(a + r, b - 1)) for a, b in zip(ends, ends[1:]) for r in (0, 127, 128, 143, 144, 777, b - a - 1)})
    c.check(c.run(), rows=torch.tensor(rows, device="cuda"))


def test_attention_backward_matches_differences():
    """Along a random direction, the 64-bit loss's central difference against
    the kernel's gradients: off by at most the gradients' own bounds, plus
    what out's rounding (2^-8) does to delta."""
    spans, R0, r, h, d = [48, 32, 64], 1, 1, 2, 64
    c = Attention(spans, R0, r, h, d, mean=0.0)
    got = c.run()
    want = ref.attention_backward(c.q, c.k, c.v, c.out, c.lse, c.dout, spans, R0, r)
    q, k, v, dout = (t.double() for t in (c.q, c.k, c.v, c.dout))
    rnd = gen(5)
    f = ref.frame_ids(spans, "cuda")
    s = d ** -0.5
    p = torch.exp((q @ k.transpose(1, 2) * s).masked_fill(~ref.visible(f, f, R0, r), -np.inf) - c.lse.double()[..., None])
    ddelta = (U16 + 2.0 ** -12) * (dout * c.out.double()).abs().sum(2)[..., None] * p  # and the forward's own error
    slack = {"dq": s * ddelta @ k.abs(), "dk": s * ddelta.transpose(1, 2) @ q.abs(), "dv": 2.0 ** -12 * got["dv"].double().abs()}
    for i, name in enumerate(("dq", "dk", "dv")):
        u = rnd(h, sum(spans), d).double()
        ends = [(ref.attention(*(t + e * u if j == i else t for j, t in enumerate((q, k, v))), spans, R0, r)[0] * dout).sum()
                for e in (1e-5, -1e-5)]
        diff = (ends[0] - ends[1]) / 2e-5
        tol = ((want[name][1] + 4 * slack[name]) * u.abs()).sum()
        assert abs((got[name].double() * u).sum() - diff) <= tol, name


def test_attention_backward_hidden_values_do_not_matter():
    """NaN and infinities in frames that a frame's gradients do not touch
    leave those gradients as they were, bit for bit (frame 7 reaches the
    queries of frames 6 and 7 and, through them, the keys of frames 5 to 7)."""
    spans, r = [80] * 8, 1
    c = Attention(spans, 0, r, 2, 128)
    clean = c.run()
    for t in (c.q, c.k, c.v, c.dout):
        t[:, 7 * 80:] = float("nan")
        t[:, 7 * 80 + 5] = float("inf")
    got = c.run()
    assert torch.equal(got["dq"][:, :6 * 80], clean["dq"][:, :6 * 80])
    for n in ("dk", "dv"):
        assert torch.equal(got[n][:, :5 * 80], clean[n][:, :5 * 80]), n
    assert torch.isnan(got["dq"][:, 7 * 80:]).all()


def test_attention_backward_rows_with_infinite_lse_take_no_part():
    spans, R0, r = [80, 48, 144], 1, 1
    c = Attention(spans, R0, r, 2, 128)
    out_rows = torch.tensor([3, 81, 130, 271], device="cuda")
    c.lse[:, out_rows] = float("inf")
    got = c.run()
    assert bool((got["dq"][:, out_rows] == 0).all())
    # The rest as if those rows' gradient were zero.
    c.lse[:, out_rows] = 1.0
    c.dout[:, out_rows] = 0
    want = c.run()
    keep = torch.tensor([i for i in range(sum(spans)) if i not in out_rows.tolist()], device="cuda")
    assert torch.equal(got["dq"][:, keep], want["dq"][:, keep])
    # Zero weights and zero gradients add the same zeros in the same order.
    assert torch.equal(got["dv"], want["dv"]) and torch.equal(got["dk"], want["dk"])


def test_attention_backward_takes_no_out_of_rows_with_infinite_lse():
    spans, R0, r = [80, 48, 144], 1, 1
    for d, layout in ((128, "hnd"), (64, "nhd")):
        c = Attention(spans, R0, r, 2, d, layout)
        rows = torch.tensor([3, 81, 130, 271], device="cuda")
        c.lse[:, rows] = float("inf")
        want = c.run()
        assert all(bool(torch.isfinite(t).all()) for t in want.values())
        for value in (float("nan"), float("inf"), -float("inf")):
            c.hnd(c.out)[:, rows] = value
            got = c.run()
            assert all(torch.equal(got[n], want[n]) for n in want)


def test_launch_counts():
    c = Attention([48] * 3, 1, 1, 2, 64)
    c.run()
    n = Norm([4, 4], 64, torch.bfloat16, True)
    x, h, rstd = n.forward()
    assert fas.fas_last_launch_count() == 1
    fas.fas_residual_norm_backward(n.dx_out, n.dh, n.y, x, rstd, n.post, n.pre, **n.kw)
    assert fas.fas_last_launch_count() == 2
    fas.fas_backward(c.q, c.k, c.v, c.out, c.lse, c.dout)
    assert fas.fas_last_launch_count() == 2


def test_attention_backward_zero_gradient_and_every_row_written():
    c = Attention([48, 112, 32], 1, 1, 2, 128)
    c.dout.zero_()
    outs = [torch.full_like(c.q, float("nan")) for _ in range(3)]
    got = c.run(dq=outs[0], dk=outs[1], dv=outs[2])
    for n, o in zip(got, outs):
        assert got[n].data_ptr() == o.data_ptr() and bool((got[n] == 0).all()), n


def test_attention_backward_after_every_mode_and_prepass():
    """out and lse from the bounded softmax serve as well as the online one's."""
    c = Attention([96] * 6, 1, 1, 3, 128)
    fas.fas_prepass(c.q, c.k)
    c.out, c.lse = fas.fas_forward(c.q, c.k, c.v, mode="auto")
    c.check(c.run())


def test_attention_backward_streams_and_graphs():
    """Two captured graphs and an eager call on a third stream, replayed at
    once: nothing is shared but the plan."""
    spans = [144] * 6
    c = Attention(spans, 1, 1, 4, 128)
    want = {n: t.clone() for n, t in c.run().items()}
    graphs = []
    for _ in range(2):
        outs = [torch.empty_like(c.q) for _ in range(3)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fas.fas_backward(c.q, c.k, c.v, c.out, c.lse, c.dout, *outs)
        graphs.append((g, outs))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = fas.fas_backward(c.q, c.k, c.v, c.out, c.lse, c.dout, stream=streams[2])
        torch.cuda.synchronize()
        for outs in [o for _, o in graphs] + [eager]:
            for n, o in zip(("dq", "dk", "dv"), outs):
                assert torch.equal(o, want[n]), n


def test_attention_backward_refuses():
    c = Attention([48] * 3, 1, 1, 2, 64)
    with pytest.raises(fas.FasError, match="invalid argument"):
        c.run(dq=c.q)
    same = torch.empty_like(c.q)
    with pytest.raises(fas.FasError, match="invalid argument"):
        c.run(dk=same, dv=same)
    with pytest.raises(ValueError):
        fas.fas_backward(c.q, c.k, c.v, c.out, c.lse, c.dout[:, :48])
    with pytest.raises(ValueError):
        fas.fas_backward(c.q.transpose(1, 2), c.k, c.v, c.out, c.lse, c.dout)
    flat = torch.empty(c.q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fas.FasError, match="aligned"):
        c.run(dq=flat[1:1 + c.q.numel()].view(c.q.shape))


# ------------------------------------------------------------------- norms

class Norm:
    def __init__(self, spans, width, residual, gated, seed=0, alpha=0.7):
        rnd = gen(seed)
        n = sum(spans)
        self.y = (rnd(n, width) * torch.exp(0.5 * rnd(1, width))).to(torch.bfloat16)
        self.x = (2 * rnd(n, width)).to(residual)
        self.post, self.pre = 1 + 0.1 * rnd(width), 1 + 0.1 * rnd(width)
        self.gate = rnd(len(spans), width) if gated else None
        self.spans = spans if len(set(spans)) > 1 else spans[0]
        self.frame = ref.frame_ids(spans, "cuda")
        self.alpha = alpha
        self.kw = dict(gate=self.gate, frame_tokens=self.spans, alpha=alpha)
        self.dx_out, self.dh = rnd(n, width).to(residual), rnd(n, width).to(torch.bfloat16)
        self.u = U16 if residual == torch.bfloat16 else U32

    def forward(self, **kw):
        return fas.fas_residual_norm(self.y, self.x, self.post, self.pre, **self.kw, **kw)

    def check_forward(self, x, h, rstd):
        """Row sums: at most 8 V + 5 + 16 <= 53 fp32 roundings and an rsqrt of
        2 ulp, so 1/rms is off by e <= (53 / 2 + 4) 2^-24; x' by e and 5
        roundings of its added term, h by the same of x', r_x and the stored
        rounding (r_x's row sum weighs the errors of x' by their size)."""
        wx, wh, wr = ref.residual_norm(self.y, self.x, self.post, self.pre, self.gate, self.frame, self.alpha, fas.RMS_EPS)
        e = 31 * U32
        term = (wx - self.x.double()).abs()
        ex = (e + 5 * U32) * term + 2 * U32 * wx.abs()
        err = (x.double() - wx).abs()
        assert torch.all(err <= ex + self.u * wx.abs()), float((err - ex - self.u * wx.abs()).max())
        er = e + ex.norm(dim=1) / wx.norm(dim=1)
        assert torch.all((rstd.double() - wr).abs() <= torch.stack([torch.full_like(er, e), er]) * wr)
        eh = ex * (wr[1][:, None] * self.pre.double().abs()) + wh.abs() * (er[:, None] + 3 * U32)
        err = (h.double() - wh).abs()
        assert torch.all(err <= 1.01 * eh + U16 * wh.abs() + 1e-38)

    def check_backward(self, got, y, x, rstd):
        """fp32 steps: a row mean has at most 53 roundings of its terms'
        magnitudes and each element a dozen more."""
        want = ref.residual_norm_backward(self.dx_out, self.dh, y, x, rstd, self.post, self.pre, self.gate, self.frame, self.alpha)
        ry, rx = rstd.double()[:, :, None]
        yh, xh = y.double() * ry, x.double() * rx
        a = self.dh.double() * self.pre.double()
        k = 70 * U32
        eg = k * (self.dx_out.double().abs() + rx * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True)))
        coef = self.alpha * self.post.double() * (1.0 if self.gate is None else self.gate.double()[self.frame])
        eb = coef.abs() * eg
        b = coef * want[0]
        ey = ry * (eb + yh.abs() * (eb * yh.abs()).mean(1, keepdim=True) +
                   k * (b.abs() + yh.abs() * (b * yh).abs().mean(1, keepdim=True)))
        for name, g, w, tol in (("dx", got[0], want[0], eg + self.u * want[0].abs()),
                                ("dy", got[1], want[1], 1.01 * ey + U16 * want[1].abs())):
            err = (g.double() - w).abs()
            assert torch.all(err <= tol + 1e-38), (name, float((err / (tol + 1e-38)).max()))
        # Column sums: terms' own errors and n 2^-24 of their magnitudes.
        n = y.shape[0]
        terms = yh.abs() * (eg + (n + 12) * U32 * want[0].abs())
        c = self.alpha * (1.0 if self.gate is None else self.gate.double().abs()[self.frame])
        tols = [("dgamma_post", got[2], want[2], (c * terms).sum(0)),
                ("dgamma_pre", got[3], want[3], (n + 12) * U32 * (self.dh.double() * xh).abs().sum(0))]
        if self.gate is not None:
            t = torch.zeros_like(want[4]).index_add_(0, self.frame, terms) * self.alpha * self.post.double().abs()
            tols.append(("dgate", got[4], want[4], t))
        else:
            assert got[4] is None
        for name, g, w, tol in tols:
            assert g.dtype == torch.float32 and g.shape == w.shape
            err = (g.double() - w).abs()
            assert torch.all(err <= tol + 1e-30), (name, float((err / (tol + 1e-30)).max()))


NORM_SHAPES = [
    # spans, width
    ([1], 8), ([1], 2048), ([3], 40), ([1, 1, 1], 264), ([5, 1, 7], 256), ([48] * 9, 128), ([33, 100, 1, 20], 96),
    ([17] * 5, 1000), ([300], 1536), ([64, 63], 2056), ([700, 40, 900], 2048), ([9, 4], 4104), ([6] * 3, 8192), ([5, 2], 8200),
    ([3, 4], 16384), ([2000, 3], 64), ([90] * 3, 16), ([40, 9], 2824), ([21], 3576), ([50, 5], 4096), ([11], 5120),
    ([1] * 1024, 72), ([3, 2] * 300, 32),
]


@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("spans,width", NORM_SHAPES, ids=lambda v: str(v) if isinstance(v, int) else "x".join(map(str, v)))
def test_residual_norm_and_its_backward(spans, width, gated, residual):
    c = Norm(spans, width, residual, gated)
    x, h, rstd = c.forward()
    assert x.dtype == residual and h.dtype == torch.bfloat16
    c.check_forward(x, h, rstd)
    got = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, x, rstd, c.post, c.pre, **c.kw)
    c.check_backward(got, c.y, x, rstd)
    again = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, x, rstd, c.post, c.pre, **c.kw)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("spans,width", [([1], 32), ([5, 1, 7], 96), ([33, 100, 1, 20], 2048), ([64, 63], 2080), ([3, 4], 8224),
                                         ([70, 1], 32), ([9] * 20, 64), ([40, 3], 3328), ([12], 5120)],
                         ids=lambda v: str(v) if isinstance(v, int) else "x".join(map(str, v)))
def test_checkpoints_from_the_forward_and_in_the_backward(spans, width, residual):
    """The forward's checkpoints are exactly those of y and of the x' it
    stored, and the backward from them is the backward from the values they
    stand for."""
    c = Norm(spans, width, residual, True)
    x, h, rstd, y8, x8 = c.forward(checkpoint=True)
    plain = c.forward()
    assert all(torch.equal(a, b) for a, b in zip((x, h, rstd), plain))
    for t, c8 in ((c.y, y8), (x, x8)):
        codes, scales = ref.checkpoint_pack(t.double().cpu().numpy())
        assert np.array_equal(c8.codes.view(torch.uint8).cpu().numpy(), codes)
        assert np.array_equal(c8.scales.cpu().numpy(), scales)
    got = fas.fas_residual_norm_backward(c.dx_out, c.dh, y8, x8, rstd, c.post, c.pre, **c.kw)
    c.check_backward(got, fas.fas_checkpoint_unpack(y8, torch.float32), fas.fas_checkpoint_unpack(x8, torch.float32), rstd)


@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("spans,width", [([3, 3, 3], 6656), ([1] * 400, 4104), ([2, 9], 11264), ([700], 9216), ([40, 1], 14336),
                                         ([1], 16376), ([1000, 7], 4352), ([150] * 2, 2560)],
                         ids=lambda v: str(v) if isinstance(v, int) else f"{len(v)}x{v[0]}")
def test_rows_over_several_ctas(spans, width, residual):
    """Clusters of two to eight CTAs of two to four warps, more rows and more
    frames than the clusters that run at once."""
    c = Norm(spans, width, residual, True, seed=4)
    x, h, rstd = c.forward()
    c.check_forward(x, h, rstd)
    got = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, x, rstd, c.post, c.pre, **c.kw)
    c.check_backward(got, c.y, x, rstd)
    if width % 32 == 0:
        x2, h2, rstd2, y8, x8 = c.forward(checkpoint=True)
        assert torch.equal(x2, x) and torch.equal(h2, h) and torch.equal(rstd2, rstd)
        for t, c8 in ((c.y, y8), (x, x8)):
            want = fas.fas_checkpoint_pack(t)
            assert torch.equal(c8.codes.view(torch.uint8), want.codes.view(torch.uint8)) and torch.equal(c8.scales, want.scales)
        got = fas.fas_residual_norm_backward(c.dx_out, c.dh, y8, x8, rstd, c.post, c.pre, **c.kw)
        c.check_backward(got, fas.fas_checkpoint_unpack(y8, torch.float32), fas.fas_checkpoint_unpack(x8, torch.float32), rstd)


def test_residual_norm_takes_spans_of_any_integer_sequence():
    c = Norm([3, 9, 4], 64, torch.bfloat16, True)
    want = c.forward()
    for spans in ((3, 9, 4), np.array([3, 9, 4]), [np.int64(3), 9, np.int32(4)], torch.tensor([3, 9, 4])):
        got = fas.fas_residual_norm(c.y, c.x, c.post, c.pre, gate=c.gate, frame_tokens=spans, alpha=c.alpha)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for spans in ([2**32 + 3, 9, 4 - 2**32], [[3, 9, 4]], [-3, 15, 4], [3, 9], ()):
        with pytest.raises((ValueError, OverflowError)):
            fas.fas_residual_norm(c.y, c.x, c.post, c.pre, gate=c.gate, frame_tokens=spans, alpha=c.alpha)


def test_rows_over_several_ctas_on_several_streams():
    """Clusters of different sizes that share the SMs, eager and captured."""
    plan([48] * 3, 0, 1, 2, 128)
    cases, want, graphs = [], [], []
    for width in (4608, 8192, 16384):
        c = Norm([90, 211], width, torch.bfloat16, True, seed=width)
        x, h, rstd = c.forward()
        cases.append(c)
        want.append((x, h, rstd, *fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, x, rstd, c.post, c.pre, **c.kw)))
        graphs.append(torch.cuda.CUDAGraph())
    outs = []
    for c, gr in zip(cases, graphs):
        with torch.cuda.graph(gr):
            fw = c.forward()
            bw = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, fw[0], fw[2], c.post, c.pre, **c.kw)
        outs.append((*fw, *bw))
    streams = [torch.cuda.Stream() for _ in range(6)]
    torch.cuda.synchronize()
    for _ in range(5):
        eager = []
        for i, (c, gr) in enumerate(zip(cases, graphs)):
            with torch.cuda.stream(streams[i]):
                gr.replay()
            with torch.cuda.stream(streams[i + 3]):
                fw = c.forward()
                eager.append((*fw, *fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, fw[0], fw[2], c.post, c.pre, **c.kw)))
        torch.cuda.synchronize()
        for got in (outs, eager):
            assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    assert fas.fas_status() == fas.FAS_OK


def test_a_row_whose_ctas_do_not_reach_one_another_is_reported():
    """A CTA that stops taking part: the other one's sums become NaN after the
    limit, the kernel ends, the status says so once, and the next call is as
    before."""
    plan([48] * 3, 0, 1, 2, 128)
    c = Norm([5, 40], 8192, torch.float32, True)
    want = c.forward()
    assert fas.fas_status() == fas.FAS_OK
    for limit_us in (2000, 1):
        assert fas.fas_selftest_row_wait_timeout(limit_us) == fas.FAS_ERR_TIMEOUT
        assert fas.fas_status() == fas.FAS_ERR_TIMEOUT
        assert fas.fas_status() == fas.FAS_OK
    assert all(torch.equal(a, b) for a, b in zip(c.forward(), want))


def test_residual_norm_in_place_streams_and_graphs():
    c = Norm([200, 56, 300], 1536, torch.bfloat16, True)
    x, h, rstd = c.forward()
    g = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, x, rstd, c.post, c.pre, **c.kw)
    # In place: the stream x' over x, h over y; dx over dx_out, dy over dh.
    y2, x2 = c.y.clone(), c.x.clone()
    x3, h3, r3 = fas.fas_residual_norm(y2, x2, c.post, c.pre, **c.kw, x_out=x2, h=y2)
    assert x3.data_ptr() == x2.data_ptr() and torch.equal(x3, x) and torch.equal(h3, h) and torch.equal(r3, rstd)
    d1, d2 = c.dx_out.clone(), c.dh.clone()
    g3 = fas.fas_residual_norm_backward(d1, d2, c.y, x, rstd, c.post, c.pre, **c.kw, dx=d1, dy=d2)
    assert all(torch.equal(a, b) for a, b in zip(g, g3))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            fw = c.forward()
            bw = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, fw[0], fw[2], c.post, c.pre, **c.kw)
        graphs.append((gr, (*fw, *bw)))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for (gr, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        eager = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, x, rstd, c.post, c.pre, **c.kw, stream=streams[2])
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, (x, h, rstd, *g)))
        assert all(torch.equal(a, b) for a, b in zip(eager, g))


def test_residual_norm_keeps_rows_apart():
    """A row of NaN or infinities spoils its own row and nothing else; the
    column sums say so."""
    c = Norm([10, 6], 512, torch.bfloat16, True)
    x, h, rstd = c.forward()
    c.y[3, 7] = float("nan")
    c.x[12, 100] = float("inf")
    x2, h2, rstd2 = c.forward()
    keep = torch.tensor([i for i in range(16) if i not in (3, 12)], device="cuda")
    assert torch.equal(x2[keep], x[keep]) and torch.equal(h2[keep], h[keep]) and torch.equal(rstd2[:, keep], rstd[:, keep])
    assert torch.isnan(h2[3]).all() and not torch.isfinite(h2[12, 100])
    got = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, x, rstd, c.post, c.pre, **c.kw)
    assert torch.isfinite(got[0]).all()      # dx reads no y
    assert torch.isnan(got[4][0, 7]) and torch.isfinite(got[4][1]).all()


def test_residual_norm_zero_rows():
    """A block output of zeros leaves x' = x; zero rows everywhere stay finite."""
    c = Norm([4], 64, torch.float32, True)
    c.y.zero_()
    x, h, rstd = c.forward()
    assert torch.equal(x, c.x)
    c.x.zero_()
    x, h, rstd = c.forward()
    assert bool((h == 0).all()) and torch.isfinite(rstd).all()
    got = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, x, rstd, c.post, c.pre, **c.kw)
    c.check_backward(got, c.y, x, rstd)


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("held", [True, False], ids=["8bit", "tensors"])
def test_plain_calls_take_native_code_and_give_the_same(held, gated, monkeypatch):
    """A call without outputs or stream is made by native code, one with them
    step by step in Python: the same results, types and shapes."""
    c = Norm([5, 90, 31], 256, torch.float32, gated)
    native = []
    real = fas._native
    monkeypatch.setattr(fas, "_native", lambda call, *a: native.append((call, real(call, *a))) or native[-1][1])
    x, h, rstd, y8, x8 = c.forward(checkpoint=True)
    y, xo = (y8, x8) if held else (c.y, x)
    post, pre = torch.nn.Parameter(c.post), torch.nn.Parameter(c.pre)
    got = fas.fas_residual_norm_backward(c.dx_out, c.dh, y, xo, rstd, post, pre, **c.kw)
    p8 = fas.fas_checkpoint_pack(x)
    un = [fas.fas_checkpoint_unpack(p8, t) for t in (None, torch.bfloat16, torch.float32)]
    assert len(native) == 6 and all(r is not None for _, r in native)
    assert isinstance(p8, fas.Checkpoint) and isinstance(y8, fas.Checkpoint) and not got[2].requires_grad
    del native[:]
    e = torch.empty_like
    x2, h2, r2, y82, x82 = c.forward(checkpoint=True, x_out=e(c.x), h=e(c.y))
    want = fas.fas_residual_norm_backward(c.dx_out, c.dh, y, xo, rstd, c.post, c.pre, **c.kw, dx=e(c.dx_out), dy=e(c.dh))
    p82 = fas.fas_checkpoint_pack(x, out=fas.Checkpoint(e(p8.codes), e(p8.scales)))
    un2 = [fas.fas_checkpoint_unpack(p8, out=e(u)) for u in un]
    assert not native
    flat = lambda *ts: [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in ts if t is not None]
    for a, b in zip(flat(x, h, rstd, *y8, *x8, *got, *p8, *un), flat(x2, h2, r2, *y82, *x82, *want, *p82, *un2), strict=True):
        assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device and torch.equal(a, b)
    assert (got[4] is None) == (not gated)


def test_calls_without_the_native_binding_give_the_same(monkeypatch):
    c = Norm([5, 90, 31], 256, torch.float32, True)
    a = Attention([48] * 3, 1, 1, 2, 64)

    def step():
        x, h, rstd, y8, x8 = c.forward(checkpoint=True)
        got = [x, h, rstd, *y8, *x8, *fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, x, rstd, c.post, c.pre, **c.kw),
               *fas.fas_residual_norm_backward(c.dx_out, c.dh, y8, x8, rstd, c.post, c.pre, **c.kw)]
        got += [*fas.fas_checkpoint_pack(x), fas.fas_checkpoint_unpack(x8, torch.float32), *a.run().values()]
        return [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in got]
    want = step()
    monkeypatch.setattr(fas, "_HOST", False)
    assert all(torch.equal(x, y) and x.dtype == y.dtype for x, y in zip(step(), want, strict=True))


def test_native_calls_run_on_the_current_stream_and_in_several_threads():
    """Each thread's stream, and the memory of a call's own buffers."""
    import threading
    cases = [Norm([200 + i, 100], 1024, torch.bfloat16, True, seed=i) for i in range(4)]
    step = lambda c: (lambda f: (*f, *fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, f[0], f[2], c.post, c.pre, **c.kw)))(c.forward())
    want = [step(c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(c, w):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                got = step(c)
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, w)):
                    bad.append(c)
    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_calls_of_several_widths_in_several_threads():
    """Widths that share a kernel and take rings of different sizes (three and
    four warps, a CTA of five and six, clusters of CTAs of three and four): no
    thread's call changes what another's launch may use."""
    import threading
    pairs = [(1536, 2048), (2560, 3056), (4608, 8192)]
    for widths in pairs:
        cases = [Norm([7, 3], w, torch.bfloat16, True, seed=w) for w in widths]
        step = lambda c: (lambda f: (*f, *fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, f[0], f[2], c.post, c.pre, **c.kw)))(c.forward())
        want = [step(c) for c in cases]
        torch.cuda.synchronize()
        bad = []

        def work(c, w):
            try:
                with torch.cuda.stream(torch.cuda.Stream()):
                    for _ in range(1500):
                        got = step(c)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, w)):
                        bad.append((widths, "values"))
            except fas.FasError as e:
                bad.append((widths, str(e)))
        threads = [threading.Thread(target=work, args=a) for a in zip(cases * 2, want * 2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not bad


def test_calls_on_a_stream_leave_the_current_streams_memory():
    """A tensor that is freed while work that reads it is still queued on the
    current stream keeps its values until that work has run, whatever a call
    on another stream allocates meanwhile."""
    c = Norm([64, 192], 2048, torch.bfloat16, True)
    a = Attention([128] * 8, 1, 1, 4, 128)
    want = (*c.forward(checkpoint=True)[:3], *(t for t in a.run().values()))
    back = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, want[0], want[2], c.post, c.pre, **c.kw)
    packed = fas.fas_checkpoint_pack(c.x)
    s = torch.cuda.Stream()
    for sizes in ([c.x.numel() * 2] * 6, [c.x.numel()] * 6, [a.q.numel() * 2] * 6, [1 << 18] * 40):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        held = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in sizes]
        inputs = torch.cuda.current_stream().record_event()
        torch.cuda._sleep(20_000_000)  # about 10 ms
        copies = [t.clone() for t in held]
        freed = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in held]
        del held
        s.wait_event(inputs)
        got = (*fas.fas_residual_norm(c.y, c.x, c.post, c.pre, **c.kw, checkpoint=True, stream=s)[:3],
               *fas.fas_backward(a.q, a.k, a.v, a.out, a.lse, a.dout, stream=s))
        gb = fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, want[0], want[2], c.post, c.pre, **c.kw, stream=s)
        p8 = fas.fas_checkpoint_pack(c.x, stream=s.cuda_stream)
        assert not any(lo <= t.data_ptr() < hi for t in (*got, *gb, *p8) for lo, hi in freed)
        torch.cuda.synchronize()
        assert all(bool((t == 77).all()) for t in copies)
        assert all(torch.equal(x, y) for x, y in zip((*got, *gb), (*want, *back)))
        assert torch.equal(p8.codes.view(torch.uint8), packed.codes.view(torch.uint8)) and torch.equal(p8.scales, packed.scales)
    # Handle 0 is the default stream.
    p8 = fas.fas_checkpoint_pack(c.x, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(p8.scales, packed.scales)


CAPTURED_FIRST = """
import torch
import frame_aligned_sparse_gb300 as fas

def run(width, residual):
    g = torch.Generator(device="cuda").manual_seed(width)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dx = rnd(37, width).to(residual), rnd(37, width).to(residual)
    y, dh = rnd(37, width).bfloat16(), rnd(37, width).bfloat16()
    post, pre, gate = rnd(width), rnd(width), rnd(1, width)

    def step():
        xo, h, rstd, y8, x8 = fas.fas_residual_norm(y, x, post, pre, gate=gate, checkpoint=True)
        a = fas.fas_residual_norm_backward(dx, dh, y, xo, rstd, post, pre, gate=gate)
        b = fas.fas_residual_norm_backward(dx, dh, y8, x8, rstd, post, pre, gate=gate)
        return (xo, h, rstd, *a, *b, fas.fas_checkpoint_unpack(fas.fas_checkpoint_pack(xo)))
    return step

q, k, v, out, dout = (torch.randn(2, 96, 64, device="cuda").bfloat16() for _ in range(5))
lse = torch.ones(2, 96, device="cuda") * 9
fas.fas_plan(48, 2, 0, 1, 2, 64)
steps = [run(w, r) for w in (128, 2048, 2560, 8192) for r in (torch.bfloat16, torch.float32)]
steps.append(lambda: fas.fas_backward(q, k, v, out, lse, dout))
torch.cuda.synchronize()
for step in steps:
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step(), strict=True))
assert fas.fas_status() == fas.FAS_OK
"""


def test_calls_captured_before_any_other():
    """A process whose first call of each kernel and shape is a captured one."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(fas.__file__)))
    res = subprocess.run([sys.executable, "-c", CAPTURED_FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-4000:]


def test_calls_captured_on_a_branch_of_the_capture():
    """stream= a stream that was forked from the capturing one: the branch's
    buffers and the other branch's are the graph's own at every replay."""
    c = Norm([64, 192], 2048, torch.bfloat16, True)
    a = Attention([128] * 8, 1, 1, 4, 128)
    x, h, rstd = c.forward()
    norm = lambda **kw: fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, x, rstd, c.post, c.pre, **c.kw, **kw)
    back = lambda **kw: fas.fas_backward(a.q, a.k, a.v, a.out, a.lse, a.dout, **kw)
    want = (*norm(), *back())
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        branch, here = [], []
        for _ in range(3):
            branch.append((*norm(stream=side), *back(stream=side)))
            here.append((*norm(), *back()))
        main.wait_stream(side)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for got in branch + here:
            assert all(torch.equal(x, y) for x, y in zip(got, want, strict=True))
            for t in got:
                t.zero_()


def test_attention_backward_native_and_with_outputs():
    c = Attention([48, 64, 16], 1, 1, 2, 64)
    got = c.run()
    want = c.run(dq=torch.empty_like(c.q), dk=torch.empty_like(c.q), dv=torch.empty_like(c.q))
    assert all(torch.equal(got[name], want[name]) for name in want)
    with pytest.raises(ValueError):
        c.run(dq=torch.empty_like(c.q)[:1])


def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 elements: their last rows as if alone."""
    n, c = 1_100_000, 2048
    small = Norm([7], c, torch.bfloat16, False)
    big = {}
    for name in ("y", "x", "dx_out", "dh"):
        t = torch.zeros(n, c, dtype=torch.bfloat16, device="cuda")
        t[-7:] = getattr(small, name)
        big[name] = t
    want = fas.fas_residual_norm(small.y, small.x, small.post, small.pre, alpha=0.7, checkpoint=True)
    got = fas.fas_residual_norm(big["y"], big["x"], small.post, small.pre, alpha=0.7, checkpoint=True)
    assert torch.equal(got[0][-7:], want[0]) and torch.equal(got[1][-7:], want[1]) and torch.equal(got[2][:, -7:], want[2])
    for a, b in zip(got[3:], want[3:]):
        assert torch.equal(a.codes[-7:].view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scales[-7:], b.scales)
    packed = fas.fas_checkpoint_pack(got[0])
    assert torch.equal(packed.codes[-7:].view(torch.uint8), want[4].codes.view(torch.uint8))
    back = fas.fas_checkpoint_unpack(packed)
    assert torch.equal(back[-7:], fas.fas_checkpoint_unpack(want[4])) and not back[:-7].any()
    del packed, back
    for held in ((got[3], got[4]), (big["y"], got[0])):
        alone = (want[3], want[4]) if held[0] is got[3] else (small.y, want[0])
        a = fas.fas_residual_norm_backward(big["dx_out"], big["dh"], *held, got[2], small.post, small.pre, alpha=0.7)
        b = fas.fas_residual_norm_backward(small.dx_out, small.dh, *alone, want[2], small.post, small.pre, alpha=0.7)
        assert torch.equal(a[0][-7:], b[0]) and torch.equal(a[1][-7:], b[1])
        for x, y in zip(a[2:4], b[2:4]):  # the zero rows add nothing, in another order
            assert float((x - y).norm() / y.norm()) <= 1e-6


def test_attention_backward_offsets_beyond_32_bits():
    """200 heads of 89,600 tokens (2.3 G elements a tensor): the last head's
    gradients, in both layouts, as that head's alone."""
    spans, h, d = [128] * 700, 200, 128
    one = Attention(spans, 0, 0, 1, d)
    want = one.run()
    for layout in ("hnd", "nhd"):
        plan(spans, 0, 0, h, d, layout)
        shape = (h, sum(spans), d) if layout == "hnd" else (sum(spans), h, d)
        at = (slice(-1, None),) if layout == "hnd" else (slice(None), slice(-1, None))
        big = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(5)]
        for t, src in zip(big, (one.q, one.k, one.v, one.out, one.dout)):
            t[at] = src if layout == "hnd" else src.transpose(0, 1)
        lse = torch.zeros(h, sum(spans), device="cuda")
        lse[-1] = one.lse[0]
        got = fas.fas_backward(*big[:4], lse, big[4])
        assert fas.fas_status() == fas.FAS_OK
        for n, g in zip(("dq", "dk", "dv"), got):
            g = g[at] if layout == "hnd" else g[at].transpose(0, 1)
            assert torch.equal(g, want[n]), (layout, n)
        del big, got, lse
        torch.cuda.empty_cache()


def test_norm_binding_refuses():
    c = Norm([4, 4], 64, torch.bfloat16, True)
    call = lambda **kw: fas.fas_residual_norm(c.y, c.x, c.post, c.pre, **{**c.kw, **kw})
    for kw, exc in ((dict(gate=c.gate[:, :32]), ValueError), (dict(gate=[1.0]), TypeError), (dict(gate=c.gate[0]), ValueError),
                    (dict(gate=c.gate.cpu()), TypeError), (dict(gate=c.gate.half()), TypeError), (dict(frame_tokens=3), ValueError),
                    (dict(frame_tokens=[4, 3]), ValueError), (dict(frame_tokens=[8]), ValueError), (dict(x_out=c.x[:4]), ValueError),
                    (dict(h=c.x.float()), TypeError), (dict(frame_tokens=[8, 0]), fas.FasError), (dict(eps=-1.0), fas.FasError)):
        with pytest.raises(exc):
            call(**kw)
    with pytest.raises(ValueError):
        fas.fas_residual_norm(c.y.T, c.x.T, c.post, c.pre)
    with pytest.raises(fas.FasError):
        fas.fas_residual_norm(c.y[:0], c.x[:0], c.post, c.pre)
    with pytest.raises(fas.FasError, match="invalid argument"):
        call(x_out=c.x, h=c.x)
    need = fas._norm_workspace(8, 64, None, 2, 0)
    p = [t.data_ptr() for t in (c.dx_out, c.dh, c.y, c.x)]
    o = [torch.empty_like(t) for t in (c.x, c.y, c.gate, c.post, c.pre)]
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    rstd = torch.ones(2, 8, device="cuda")
    assert fas.load().fas_residual_norm_backward(
        *p, 0, None, None, None, None, rstd.data_ptr(), c.gate.data_ptr(), c.post.data_ptr(), c.pre.data_ptr(), 1.0, 8, 64, None, 2,
        *(t.data_ptr() for t in o), ws.data_ptr(), need - 1, None) == fas.FAS_ERR_SCRATCH
    c2 = Norm([4, 4], 72, torch.bfloat16, True)
    with pytest.raises(ValueError):
        c2.forward(checkpoint=True)
    x, h, rstd = c.forward()
    with pytest.raises(TypeError, match="both"):
        fas.fas_residual_norm_backward(c.dx_out, c.dh, c.y, fas.fas_checkpoint_pack(x), rstd, c.post, c.pre, **c.kw)


# ------------------------------------------------------------- checkpoints

def special_values():
    """Blocks at every border of the format: zeros of both signs, scales at
    and next to 448 2^k, ties, subnormals, the largest values, NaN, inf."""
    rows = [np.zeros(32), -np.zeros(32)]
    for k in (-126, -60, -9, 0, 5, 100, 118):
        for m in (1.0, 1.75, 1.7578125, 1.9921875):
            row = np.linspace(-1, 1, 32) * m * 2.0 ** k
            row[7] = m * 2.0 ** k
            rows.append(row)
    ties = np.array([(8 + i + 0.5) * 2.0 ** e for e in (-3, 0, 4) for i in range(8)] + [448.0] + [0.5 * 2.0 ** -9, 1.5 * 2.0 ** -9, 2.5 * 2.0 ** -9,
                                                                                 7.5 * 2.0 ** -9, 2.0 ** -30, -2.0 ** -6, 3.0])
    rows += [ties, -ties]
    for bad in (np.nan, np.inf, -np.inf):
        row = np.linspace(0.1, 3, 32)
        row[3] = bad
        rows += [row, np.full(32, bad)]
    rows.append(np.full(32, 2.0 ** -133))
    rows.append(np.full(32, 3.3895313892515355e38))
    return np.stack(rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_checkpoint_is_exact_at_the_formats_borders(dtype):
    x = torch.from_numpy(special_values().astype(np.float32)).to(dtype).cuda()
    if dtype == torch.float32:
        x[-1] = torch.finfo(torch.float32).max
        x[-2] = 2.0 ** -149
    c = fas.fas_checkpoint_pack(x)
    codes, scales = ref.checkpoint_pack(x.double().cpu().numpy())
    got = c.codes.view(torch.uint8).cpu().numpy()
    nan = (codes & 127) == 127
    assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], codes[~nan])
    assert np.array_equal(c.scales.cpu().numpy(), scales)
    back = fas.fas_checkpoint_unpack(c, dtype)
    want = torch.from_numpy(ref.checkpoint_unpack(codes, scales)).to(dtype)  # exact but for subnormal results
    assert torch.equal(back.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(32,), (1, 96), (7, 64), (3, 5, 32), (1000, 2080), (4096, 4096)], ids=str)
def test_checkpoint_round_trip(shape, dtype):
    x = (gen(2)(*shape) * 3).to(dtype)
    c = fas.fas_checkpoint_pack(x)
    assert c.codes.shape == x.shape and c.scales.shape == (*shape[:-1], shape[-1] // 32)
    back = fas.fas_checkpoint_unpack(c, dtype)
    s = torch.exp2(c.scales.double() - 127).repeat_interleave(32, -1)
    err = (back.double() - x.double()).abs()
    assert torch.all(err <= torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * s))
    if x.numel() < 1 << 20:
        codes, scales = ref.checkpoint_pack(x.double().cpu().numpy())
        assert np.array_equal(c.codes.view(torch.uint8).cpu().numpy(), codes) and np.array_equal(c.scales.cpu().numpy(), scales)
    # A checkpoint of what a checkpoint stands for is itself.
    c2 = fas.fas_checkpoint_pack(back)
    assert torch.equal(fas.fas_checkpoint_unpack(c2, dtype), back)


def test_checkpoint_unpack_of_every_code():
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(8, 1)
    scales = torch.tensor([0, 1, 60, 120, 127, 128, 200, 247], dtype=torch.uint8, device="cuda")[:, None].repeat(1, 8)
    got = fas.fas_checkpoint_unpack((codes.view(torch.float8_e4m3fn), scales), torch.float32).cpu().numpy()
    with np.errstate(over="ignore"):  # code 448 under 2^120 is beyond fp32: infinite on both sides
        want = ref.checkpoint_unpack(codes.cpu().numpy(), scales.cpu().numpy()).astype(np.float32)
    assert np.array_equal(got, want, equal_nan=True)


def test_checkpoint_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    c = fas.fas_checkpoint_pack(x)
    for bad in (x[:, :48].contiguous(), x[:0]):
        with pytest.raises(ValueError):
            fas.fas_checkpoint_pack(bad)
    with pytest.raises(ValueError):
        fas.fas_checkpoint_pack(x[:, ::2])
    with pytest.raises(ValueError):
        fas.fas_checkpoint_unpack((c.codes, c.scales[:2]))
    with pytest.raises(TypeError):
        fas.fas_checkpoint_unpack((c.codes.view(torch.uint8), c.scales))
    with pytest.raises(TypeError):
        fas.fas_checkpoint_unpack(c, torch.float16)


# -------------------------------------------------------- a block's training

def test_a_block_trained_from_8_bit_checkpoints():
    """A block as it is trained: prologue, attention, output projection, the
    norms and gate around it with 8-bit checkpoints, then backward: the norms
    from the checkpoints, the projection, the attention recomputed from a
    checkpoint of the hidden states.  Every step against its 64-bit reference
    on the inputs it had."""
    w = workloads.get("tiny")
    T, nf, H, d = w.frame_tokens, w.total_frames, w.heads, w.head_dim
    N, C = w.tokens, H * d
    p = workloads.prologue_inputs(w)
    dev = lambda b: torch.from_numpy(b.view(np.int16)).view(torch.bfloat16).cuda()
    x, wt = dev(p["x"]), dev(p["w"])
    cos, sin = torch.from_numpy(p["cos"]).cuda(), torch.from_numpy(p["sin"]).cuda()
    fold = fas.fas_prologue_fold_weights(wt, torch.from_numpy(p["gamma"]).cuda())
    rnd = gen(9)
    wo = (rnd(C, C) / C ** 0.5).to(torch.bfloat16)
    post, pre, gate = 1 + 0.1 * rnd(C), 1 + 0.1 * rnd(C), rnd(nf, C)

    def attend(hidden):
        q, k, v = fas.fas_prologue(hidden, fold, cos, sin, H, d, layout="nhd")
        fas.fas_prepass(q, k)
        return (q, k, v, *fas.fas_forward(q, k, v))

    fas.fas_plan(T, w.n_frames, w.ref_frames, w.window_radius, H, d)
    fas.fas_set_layout("nhd")
    kept = fas.fas_checkpoint_pack(x)  # the block's input, in 8 bits
    held = fas.fas_checkpoint_unpack(kept)
    q, k, v, out, lse = attend(held)
    y = out.reshape(N, C) @ wo
    x_out, h, rstd, y8, x8 = fas.fas_residual_norm(y, held, post, pre, gate=gate, frame_tokens=T, checkpoint=True)
    dx_out, dh = rnd(N, C).to(torch.bfloat16), rnd(N, C).to(torch.bfloat16)

    dx, dy, dpost, dpre, dgate = fas.fas_residual_norm_backward(dx_out, dh, y8, x8, rstd, post, pre, gate=gate, frame_tokens=T)
    dout = (dy @ wo.T).reshape(N, H, d).contiguous()
    q2, k2, v2, out2, lse2 = attend(fas.fas_checkpoint_unpack(kept))  # recomputed: the same bits
    assert all(torch.equal(a, b) for a, b in zip((q, k, v, out, lse), (q2, k2, v2, out2, lse2)))
    dq, dk, dv = fas.fas_backward(q2, k2, v2, out2, lse2, dout)
    assert fas.fas_status() == fas.FAS_OK

    spans = [T] * nf
    f = ref.frame_ids(spans, "cuda")
    wants = ref.residual_norm_backward(dx_out, dh, fas.fas_checkpoint_unpack(y8), fas.fas_checkpoint_unpack(x8), rstd, post, pre,
                                       gate, f, 1.0)
    for g, wv, t in zip((dx, dy, dpost, dpre, dgate), wants, (U16, U16, 1e-5, 1e-5, 1e-5)):
        assert float((g.double() - wv).norm() / wv.norm()) <= t
    t = lambda z: z.transpose(0, 1)
    res = ref.attention_backward(t(q), t(k), t(v), t(out), lse, t(dout), spans, w.ref_frames, w.window_radius)
    for g, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        want, bound, _ = res[n]
        assert torch.all((t(g).double() - want).abs() <= bound)
    # And the whole against the loss of the un-checkpointed block: 8-bit
    # checkpoints move its gradients by their own error, at most 2^-4 a value.
    full = ref.residual_norm_backward(dx_out, dh, y, x_out, rstd, post, pre, gate, f, 1.0)
    for g, wv in zip((dx, dy), full):
        assert float((g.double() - wv).norm() / wv.norm()) <= 2.0 ** -4
