"""The block's operators on the GPU against 64-bit references: the gated
feed-forward block, rotary positions with several axes, and the gradients'
norm and clipping.

Tolerances are the references' own bounds (tests/block_reference.py) or
derived in the test.
"""
import math
import time

import numpy as np
import pytest
import torch

import block_reference as ref
import frame_aligned_sparse_gb300 as fas
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


BF16 = torch.bfloat16


# ------------------------------------------------------------- feed-forward

class Block:
    def __init__(self, n, c, f, seed=0):
        rnd = gen(seed)
        self.x = (rnd(n, c) * torch.exp(0.5 * rnd(1, c))).to(BF16)
        self.w_in, self.w_out = (rnd(2 * f, c) / c ** 0.5).to(BF16), (rnd(c, f) / f ** 0.5).to(BF16)
        self.dy = rnd(n, c).to(BF16)
        self.weights = (self.w_in, self.w_out)

    def forward(self, act="silu", **kw):
        return fas.fas_feed_forward(self.x, *self.weights, activation=act, **kw)

    def backward(self, kept=None, act="silu", **kw):
        return fas.fas_feed_forward_backward(self.dy, self.x, *self.weights, kept=kept, activation=act, **kw)

    def check(self, act="silu"):
        # A rounding lies within sqrt(3) of its deviation (uniform within half a
        # step).  Where fewer than 16 tokens, columns or inner features meet, one
        # of them can carry a whole norm, which may then lie as far out: the
        # bounds alone are compared.
        norm = min(*self.x.shape, self.w_out.shape[1]) >= 16
        y, kept = self.forward(act, keep=True)
        want = ref.feed_forward(self.x, *self.weights, act)
        ref.check(y, want["y"], "y", norm)
        ref.check(kept, want["kept"], "kept", norm)
        assert torch.equal(self.forward(act), y)
        # From what was kept, and computed again from x, where g and u are held more exactly.
        for held in (kept, None):
            want = ref.feed_forward_backward(self.dy, self.x, *self.weights, held, act)
            for name, g in zip(want, self.backward(held, act)):
                ref.check(g, want[name], name, norm)


SHAPES = [(1, 8, 8), (1, 64, 64), (1, 2048, 344), (2, 128, 264), (3, 72, 24), (17, 1000, 136), (64, 64, 64), (127, 128, 128),
          (128, 256, 192), (129, 136, 200), (255, 64, 520), (256, 256, 256), (257, 264, 248), (300, 2048, 1024), (432, 128, 344),
          (1000, 520, 1032), (2049, 320, 648), (130, 8, 4096), (130, 4096, 8), (5000, 512, 256), (8, 200, 72), (9, 264, 520), (16, 72, 1000),
          (24, 1032, 40), (31, 264, 520), (32, 264, 520), (33, 264, 520), (7, 8, 16), (640, 1544, 72), (40, 16384, 8), (40, 8, 16384), (3, 16384, 16)]


@pytest.mark.parametrize("act", list(fas.ACTIVATIONS))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_feed_forward_and_its_backward(shape, act):
    Block(*shape).check(act)


@pytest.mark.parametrize("shape", [(17, 64, 4104), (31, 2048, 5504), (12, 104, 8200), (20, 4104, 64), (16, 264, 16384), (8, 72, 16384),
                                   (30, 264, 4096)], ids=lambda s: "x".join(map(str, s)))
def test_feed_forward_of_few_tokens_by_either_form(shape):
    Block(*shape).check("gelu_tanh")


@pytest.mark.parametrize("shape", [(14960, 2048, 1376), (20000, 1000, 2728)], ids=lambda s: "x".join(map(str, s)))
def test_feed_forward_of_many_tiles(shape):
    Block(*shape).check()


@pytest.mark.parametrize("act", list(fas.ACTIVATIONS))
@pytest.mark.parametrize("shape", [(9000, 104, 1032), (6001, 72, 5000), (23374, 104, 136), (3000, 8, 9336), (20000, 256, 1024)],
                         ids=lambda s: "x".join(map(str, s)))
def test_feed_forward_of_narrow_widths_and_many_tokens(shape, act):
    """Sums of one to four steps of 64 over many tiles, some left over after
    whole rounds, in the forms of both single CTAs and pairs."""
    Block(*shape).check(act)


@pytest.mark.parametrize("shape", [(700, 200, 328), (4, 96, 64)], ids=str)
def test_feed_forward_matches_differences(shape):
    """Along a random direction, the 64-bit loss's central difference against
    the kernel's gradients, off by at most their own bounds and what the kept
    projections' rounding (2^-8 of each) does."""
    c = Block(*shape, seed=3)
    kept = c.forward(keep=True)[1]
    got = dict(zip(("x", "w_in", "w_out"), c.backward(kept)))
    want = dict(zip(("x", "w_in", "w_out"), ref.feed_forward_backward(c.dy, c.x, *c.weights, kept, "silu").values()))
    exact = ref.feed_forward_backward(c.dy, c.x, *c.weights, ref.projections(c.x, c.w_in)[0], "silu")
    exact = dict(zip(("x", "w_in", "w_out"), exact.values()))
    args = {"x": c.x.double(), "w_in": c.w_in.double(), "w_out": c.w_out.double()}

    def loss(x, w_in, w_out):
        g, u = (x @ w_in.T).chunk(2, 1)
        return ((ref.activation(g, "silu")[0] * u) @ w_out.T * c.dy.double()).sum()

    rnd = gen(4)
    for name, g in got.items():
        d = rnd(*g.shape).double()
        diff = (loss(**{**args, name: args[name] + 1e-5 * d}) - loss(**{**args, name: args[name] - 1e-5 * d})) / 2e-5
        assert abs((exact[name][0] * d).sum() - diff) <= 1e-6 * (exact[name][0] * d).abs().sum(), name  # the formula
        moved = ((want[name][0] - exact[name][0]) * d).sum().abs()  # by the kept projections' rounding
        assert abs((g.double() * d).sum() - diff) <= (want[name][1] * d.abs()).sum() + moved + 1e-6 * (g.double() * d).abs().sum(), name


def test_feed_forward_saturated_gates():
    """Gates far on both sides, where a sigmoid is 0 or 1 and its derivative none."""
    n, c, f = 64, 64, 64
    b = Block(n, c, f)
    b.x.zero_()
    b.x[:, 0] = torch.linspace(-3000, 3000, n, device="cuda").to(BF16)
    b.x[:, 1] = 1
    b.w_in.zero_()
    b.w_in[:f, 0] = torch.linspace(0.5, 100, f, device="cuda").to(BF16)
    b.w_in[f:, 1] = 1
    for act in fas.ACTIVATIONS:
        y, kept = b.forward(act, keep=True)
        ref.check(y, ref.feed_forward(b.x, *b.weights, act)["y"], "y", norm=False)
        for held in (kept, None):
            want = ref.feed_forward_backward(b.dy, b.x, *b.weights, held, act)
            for name, g in zip(want, b.backward(held, act)):
                ref.check(g, want[name], name, norm=False)


def test_feed_forward_keeps_rows_apart():
    """A row of NaN or infinities stays its own: in y, dx and the kept projections."""
    b = Block(300, 136, 200)
    y, kept = b.forward(keep=True)
    dx = b.backward(kept)[0]
    b.x[77] = float("nan")
    b.x[131] = float("inf")
    b.dy[200] = float("nan")
    y2, kept2 = b.forward(keep=True)
    dx2 = b.backward(kept2)[0]
    rows = [i for i in range(300) if i not in (77, 131)]
    assert torch.equal(y[rows], y2[rows]) and torch.equal(kept[rows], kept2[rows])
    rows.remove(200)
    assert torch.equal(dx[rows], dx2[rows])
    assert y2[77].isnan().all() and y2[131].isnan().any() and dx2[200].isnan().all()


@pytest.mark.parametrize("act", list(fas.ACTIVATIONS))
def test_feed_forward_backward_keeps_nan(act):
    """A gate or an up value that is NaN makes the gradients that depend on it NaN."""
    b = Block(200, 64, 72)
    kept = b.forward(act, keep=True)[1]
    kept[50, 3] = float("nan")  # a gate
    kept[60, 72 + 9] = float("nan")  # an up value
    dx, dw_in, dw_out = b.backward(kept, act)
    assert dx[50].isnan().all() and dx[60].isnan().all() and int(dx.isnan().any(1).sum()) == 2
    assert dw_in[3].isnan().all() and dw_in[72 + 3].isnan().all() and dw_in[9].isnan().all() and not dw_in[72 + 9].isnan().any()
    assert dw_out[:, [3, 9]].isnan().all() and int(dw_out.isnan().any(0).sum()) == 2


def test_feed_forward_writes_its_outputs_and_nothing_else():
    """Outputs given, with a guard on both sides of each."""
    n, c, f = 333, 72, 136
    b = Block(n, c, f)
    want_y, kept = b.forward(keep=True)
    want = b.backward(kept)

    def guarded(rows, cols):
        t = torch.full(((rows + 4) * cols,), float("nan"), device="cuda", dtype=BF16)
        return t, t[2 * cols:(rows + 2) * cols].view(rows, cols)

    outs = [guarded(*s) for s in ((n, c), (n, c), (2 * f, c), (c, f))]
    y = b.forward(y=outs[0][1])
    got = b.backward(kept, dx=outs[1][1], dw_in=outs[2][1], dw_out=outs[3][1])
    for (base, view), g, w in zip(outs, (y, *got), (want_y, *want)):
        assert g.data_ptr() == view.data_ptr() and torch.equal(g, w)
        cols = view.shape[1]
        assert base[:2 * cols].isnan().all() and base[-2 * cols:].isnan().all()


def test_feed_forward_offsets_beyond_32_bits():
    """2.2 G elements of kept projections: first and last rows against the reference."""
    n, c, f = 136000, 64, 8192
    b = Block(n, c, f)
    y, kept = b.forward(keep=True)
    dx, dw_in, dw_out = b.backward(kept)
    rows = torch.tensor([0, 1, 131071, 131072, n - 130, n - 1], device="cuda")
    want = ref.feed_forward(b.x[rows], *b.weights, "silu")
    ref.check(y[rows], want["y"], "y")
    ref.check(kept[rows], want["kept"], "kept")
    back = ref.feed_forward_backward(b.dy[rows], b.x[rows], *b.weights, kept[rows], "silu")
    ref.check(dx[rows], back["dx"], "dx")
    del dx
    # The weights' gradients of a few inner features, over all rows.
    cols = torch.tensor([0, 63, 4097, f - 1], device="cuda")
    both = torch.cat([cols, cols + f])
    back = ref.feed_forward_backward(b.dy, b.x, b.w_in[both], b.w_out[:, cols], kept[:, both], "silu")
    ref.check(dw_in[both], back["dw_in"], "dw_in")
    ref.check(dw_out[:, cols], back["dw_out"], "dw_out")


def test_feed_forward_streams_and_graphs():
    """Two captured graphs and an eager call on a third stream, replayed at once."""
    b = Block(700, 264, 520)
    want = (*b.forward(keep=True),)
    want += tuple(b.backward(want[1]))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, kept = b.forward(keep=True)
            out = (y, kept, *b.backward(kept))
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, out), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for t in out:
                    t.zero_()
                g.replay()
        y, kept = b.forward(keep=True, stream=streams[2])
        eager = (y, kept, *b.backward(kept, stream=streams[2]))
        torch.cuda.synchronize()
        for out in (graphs[0][1], graphs[1][1], eager):
            assert all(torch.equal(a, w) for a, w in zip(out, want))


def test_feed_forward_is_reproducible():
    for shape in ((1, 512, 1024), (3000, 256, 2048), (40, 1024, 1024)):
        b = Block(*shape)
        y, kept = b.forward(keep=True)
        first = b.backward(kept)
        for _ in range(3):
            assert torch.equal(b.forward(), y)
            assert all(torch.equal(p, q) for p, q in zip(b.backward(kept), first))


def test_feed_forward_reports_nothing_to_fas_status():
    fas.fas_plan(48, 3, 1, 1, 2, 64)
    Block(100, 64, 64).check()
    assert fas.fas_status() == fas.FAS_OK


@pytest.mark.parametrize("shape", [(300, 8200, 520), (6000, 72, 5000), (25000, 264, 136), (25000, 1032, 72), (14960, 2048, 1376)],
                         ids=lambda s: "x".join(map(str, s)))
def test_feed_forward_pairs_of_ctas_end(shape):
    """Shapes whose products take pairs of CTAs, with fewer and more steps of 64
    than there are stages, several tiles a pair and none left over: CTAs wait
    for every arrival under way to them before they end, and no such wait runs
    out (half a second each, then fas_status tells).  Calls one behind the
    other: a CTA's shared memory is the next kernel's at once."""
    fas.fas_plan(48, 3, 1, 1, 2, 64)
    b = Block(*shape)
    b.check()
    y, kept = b.forward(keep=True)
    grads = b.backward(kept)
    torch.cuda.synchronize()
    start = time.monotonic()
    for _ in range(20):
        again = b.forward(), *b.backward(kept)
    torch.cuda.synchronize()
    assert time.monotonic() - start < 0.4  # 20 calls of at most 3 ms
    assert all(torch.equal(p, q) for p, q in zip(again, (y, *grads)))
    assert fas.fas_status() == fas.FAS_OK


def test_feed_forward_waits_that_run_out():
    """A product whose waits run out ends, frees what it holds and is reported
    once; the products after it are as before."""
    fas.fas_plan(48, 3, 1, 1, 2, 64)
    b = Block(300, 8200, 520)
    y, kept = b.forward(keep=True)
    grads = b.backward(kept)
    for limit_us in (1, 2000, 5000):
        assert fas.fas_selftest_product_wait_timeout(limit_us) == fas.FAS_ERR_TIMEOUT
        assert fas.fas_status() == fas.FAS_ERR_TIMEOUT
        assert fas.fas_status() == fas.FAS_OK
        assert all(torch.equal(p, q) for p, q in zip((b.forward(), *b.backward(kept)), (y, *grads)))
    assert fas.fas_status() == fas.FAS_OK


def test_lost_waits_are_reported_without_a_plan():
    """A process that only trains has no plan: fas_status is out of order there,
    fas_training_status tells, on whatever stream, and both clear the same words."""
    fas.fas_free()
    b = Block(300, 264, 520)
    b.check()
    assert fas.fas_training_status() == fas.FAS_OK
    for lose in (fas.fas_selftest_product_wait_timeout, fas.fas_selftest_row_wait_timeout):
        assert lose(1000) == fas.FAS_ERR_TIMEOUT
        with pytest.raises(fas.FasError) as e:
            fas.fas_status()
        assert e.value.code == fas.FAS_ERR_STATE
        assert fas.fas_training_status(torch.cuda.Stream()) == fas.FAS_ERR_TIMEOUT
        assert fas.fas_training_status() == fas.FAS_OK
        fas.fas_plan(48, 3, 1, 1, 2, 64)
        assert lose(1000) == fas.FAS_ERR_TIMEOUT
        assert fas.fas_training_status() == fas.FAS_ERR_TIMEOUT
        assert fas.fas_status() == fas.FAS_OK
        fas.fas_free()


def test_feed_forward_refuses():
    b = Block(16, 64, 72)
    with pytest.raises(ValueError, match="activation"):
        fas.fas_feed_forward(b.x, *b.weights, activation="relu")
    with pytest.raises(TypeError, match="x must"):
        fas.fas_feed_forward(b.x.float(), *b.weights)
    with pytest.raises(ValueError, match="w_in"):
        fas.fas_feed_forward(b.x, b.w_in[:72], b.w_out)
    with pytest.raises(ValueError, match="contiguous"):
        fas.fas_feed_forward(b.x, b.w_in, b.w_out.T.contiguous().T)
    with pytest.raises(fas.FasError):  # 60 columns
        fas.fas_feed_forward(b.x[:, :60].contiguous(), b.w_in[:, :60].contiguous(), b.w_out[:60].contiguous())
    with pytest.raises(fas.FasError):  # no tokens
        fas.fas_feed_forward(b.x[:0], *b.weights)
    with pytest.raises(fas.FasError):  # in place
        fas.fas_feed_forward(b.x, *b.weights, y=b.x)
    with pytest.raises(ValueError, match="kept"):
        fas.fas_feed_forward_backward(b.dy, b.x, *b.weights, kept=b.x)
    with pytest.raises(ValueError, match="dy"):
        fas.fas_feed_forward_backward(b.dy[:8], b.x, *b.weights)
    with pytest.raises(TypeError, match="CUDA"):
        fas.fas_feed_forward(b.x.cpu(), *b.weights)
    with pytest.raises(fas.FasError) as e:  # not on a 16-byte boundary
        fas.fas_feed_forward(torch.zeros(16 * 64 + 1, device="cuda", dtype=BF16)[1:].view(16, 64), *b.weights)
    assert e.value.code == fas.FAS_ERR_ALIGN


@pytest.mark.parametrize("n", [5, 200])
def test_feed_forward_backward_computed_again_at_the_edges(n):
    """Projections of zero, of the smallest and of large values, and infinite
    ones: what bf16 and eight more bits hold of them."""
    b = Block(n, 64, 72)
    b.x[0] = 0
    b.x[1] *= 2.0 ** -120
    b.x[2] *= 2.0 ** 40
    b.dy[2] *= 2.0 ** -60
    got = b.backward()[0]
    want = ref.feed_forward_backward(b.dy, b.x, *b.weights, None, "silu")["dx"]
    assert torch.all((got.double() - want[0]).abs() <= want[1] + 1e-36)
    b.x[3] = float("inf")
    rows = [i for i in range(n) if i != 3]
    again = b.backward()[0]
    assert torch.equal(again[rows], got[rows]) and not torch.isfinite(again[3]).any()


def test_feed_forward_few_tokens_match_many():
    """The pass for few tokens and the tiles: the same sums up to the order of
    fp32 additions, so results on the same rows differ by two roundings at most."""
    b = Block(64, 520, 1032)
    many = b.forward(keep=True)
    for n in (1, 5, 8, 12, 16, 20, 31):
        y, kept = fas.fas_feed_forward(b.x[:n], *b.weights, keep=True)
        for got, want in ((y, many[0][:n]), (kept, many[1][:n])):
            d = (got.double() - want.double()).abs()
            assert torch.all(d <= 2.0 ** -7 * want.double().abs() + 2.0 ** -7 * float(want.double().abs().mean()))


# ------------------------------------------------------------------- rotary

def positions(frames, rows, cols):
    j = torch.arange(frames * rows * cols, device="cuda")
    return torch.stack([j // (rows * cols), j // cols % rows, j % cols], 1).float()


def lay(t, layout):
    """[H, N, d] in the layout."""
    return t if layout == "hnd" else t.transpose(0, 1).contiguous()


ROTARY = [  # H, d, (frames, rows, cols), pairs, theta
    (1, 64, (1, 1, 1), (32,), 10000.0), (2, 64, (9, 6, 8), (8, 12, 12), 10000.0), (3, 128, (2, 5, 7), (16, 24, 24), 10000.0),
    (16, 128, (3, 22, 40), (16, 24, 24), 256.0), (24, 128, (1, 45, 80), (16, 20, 20), (100.0, 10000.0, 500.0)),
    (5, 64, (1, 1, 33), (0, 7, 0), 10000.0), (40, 128, (1, 1, 1), (64, 0, 0), 1e6), (7, 128, (1, 1, 31), (1, 2, 3, 4), 10.0),
]


@pytest.mark.parametrize("pairing", list(fas.PAIRINGS))
@pytest.mark.parametrize("layout", list(fas.LAYOUTS))
@pytest.mark.parametrize("case", ROTARY, ids=lambda c: f"{c[0]}x{c[1]}_{'x'.join(map(str, c[2]))}")
def test_rotary_pack_unpack_and_turn(case, layout, pairing):
    H, d, grid, pairs, theta = case
    pos = positions(*grid)
    axes = len(pairs)
    pos = torch.cat([pos, 0.5 * pos[:, :1]], 1)[:, :axes].contiguous()
    N = pos.shape[0]
    rnd = gen(1)
    qkv = rnd(N, 3 * H * d).to(BF16)
    kw = dict(pairs=pairs, theta=theta, layout=layout, pairing=pairing)
    got = fas.fas_rotary_pack(qkv, pos, H, d, **kw)
    assert fas.fas_last_launch_count() == 1
    parts = qkv.view(N, 3, H, d).permute(1, 2, 0, 3)
    for i, g in enumerate(got):
        assert g.is_contiguous() and g.shape == lay(parts[i], layout).shape
        if i == 2:
            assert torch.equal(g, lay(parts[2], layout))
            continue
        want, bound = ref.rotary(parts[i], pos, pairs, theta, pairing)
        assert torch.all((g.double() - lay(want, layout)).abs() <= lay(bound, layout)), i
        assert torch.equal(fas.fas_rotary(lay(parts[i].contiguous(), layout), pos, **kw), g)
    # The way back, of other values.
    grads = [lay(rnd(H, N, d).to(BF16), layout) for _ in range(3)]
    dqkv = fas.fas_rotary_unpack(*grads, pos, **kw)
    assert dqkv.shape == (N, 3 * H * d)
    for i, g in enumerate(dqkv.view(N, 3, H, d).permute(1, 2, 0, 3)):
        src = lay(grads[i], layout)
        if i == 2:
            assert torch.equal(g, src)
            continue
        want, bound = ref.rotary(src, pos, pairs, theta, pairing, inverse=True)
        assert torch.all((g.double() - want).abs() <= bound), i


def test_rotary_matches_the_prologues_tables():
    """The same turn as the prologue's from the workload's tables."""
    w = workloads.get("tiny")
    cos, sin = (torch.from_numpy(t).cuda().double() for t in workloads.rotary_tables(w))
    gw = workloads.GRID_W[w.name]
    j = torch.arange(w.tokens, device="cuda")
    pos = torch.stack([j // w.frame_tokens, j % w.frame_tokens // gw, j % w.frame_tokens % gw], 1).float()
    d = w.head_dim
    n_t, n_y = d // 8, (d // 2 - d // 8) // 2
    x = gen(0)(w.heads, w.tokens, d).to(BF16)
    got = fas.fas_rotary(x, pos, pairs=(n_t, n_y, d // 2 - n_t - n_y))
    a, b = x.double().chunk(2, 2)
    want = torch.cat([a * cos - b * sin, a * sin + b * cos], 2)
    # The tables are rounded to fp32, the angles here off by 2^-22: both within 2^-21 of |a| + |b|.
    assert torch.all((got.double() - want).abs() <= U16 * want.abs() + 2.0 ** -20 * (a.abs() + b.abs()).repeat(1, 1, 2))


def test_rotary_at_the_largest_positions_and_frequencies():
    """Frequencies up to almost 2^32 at positions of +-2^90: a turn and its
    opposite give the tensor back.  Each rounds once (2^-8 of an element): the
    first error, at most 2^-8 of the pair's length r, is turned, the second adds
    2^-8 of the element, so an element is off by 2 x 2^-8 r and a little."""
    rnd = gen(5)
    x = rnd(2, 9, 64).to(BF16)
    positions = torch.tensor([0.0, 1.0, -1.0, 2.0 ** 24 + 2, 2.0 ** 60, -2.0 ** 60, 2.0 ** 90, -2.0 ** 90, 2.0 ** -90], device="cuda")[:, None]
    turned = fas.fas_rotary(x, positions, (32,), 2.0 ** -33)
    back = fas.fas_rotary(turned, positions, (32,), 2.0 ** -33, inverse=True)
    r = (x.double()[..., :32].square() + x.double()[..., 32:].square()).sqrt().repeat(1, 1, 2)
    assert bool(((back.double() - x.double()).abs() <= 2.05 * 2.0 ** -8 * r).all())
    assert torch.equal(turned[:, 0], x[:, 0])


def test_rotary_far_and_fractional_positions():
    """Angles of up to 2^21 radians, negative and fractional positions."""
    n, d = 400, 64
    rnd = gen(2)
    pos = torch.stack([torch.exp2(torch.linspace(0, 21, n, device="cuda")), -1000 * rnd(n)], 1).float()
    x = rnd(2, n, d).to(BF16)
    want, bound = ref.rotary(x, pos, (16, 16), 10000.0, "half")
    got = fas.fas_rotary(x, pos, pairs=(16, 16))
    assert torch.all((got.double() - want).abs() <= bound)


def test_rotary_in_place_zero_positions_and_round_trip():
    x = gen(3)(3, 50, 128).to(BF16)
    pos = torch.zeros(50, 2, device="cuda")
    assert torch.equal(fas.fas_rotary(x, pos, pairs=(32, 32)), x)
    pos = positions(1, 5, 10)[:, 1:].contiguous()
    want = fas.fas_rotary(x, pos, pairs=(32, 32))
    y = x.clone()
    assert fas.fas_rotary(y, pos, pairs=(32, 32), out=y).data_ptr() == y.data_ptr()
    assert torch.equal(y, want)
    # There and back: two roundings of each element of a pair.
    back = fas.fas_rotary(y, pos, pairs=(32, 32), inverse=True)
    a, b = x.double().abs().chunk(2, 2)
    assert torch.all((back.double() - x.double()).abs() <= (2.5 * U16 * (a + b)).repeat(1, 1, 2))


@pytest.mark.parametrize("pairing", list(fas.PAIRINGS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("count", [0, 1, 2, 3, 5, 7, 8, 9, 12, 15, 16, 31])
def test_rotary_copies_the_pairs_that_do_not_turn(count, d, pairing):
    """Bit by bit: next to infinities, NaN with their own bits, zeros of either
    sign, and at positions that are infinite or NaN, as padding may be."""
    rnd = gen(30 + count)
    bits = torch.tensor([0x7F80, -0x80, 0x7FC1, -0x3F, -0x8000, 0x0001, 0x3F80], device="cuda", dtype=torch.int16)
    for layout in fas.LAYOUTS:
        x = lay(rnd(3, 41, d).to(BF16), layout)
        where = torch.rand(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(count)) < 0.2
        some = bits[torch.randint(0, len(bits), x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1))]
        x = torch.where(where, some, x.view(torch.int16)).view(BF16)
        pos = positions(1, 1, 41)[:, :2].contiguous()
        pos[3], pos[4, 0], pos[5, 1] = math.inf, math.nan, -math.inf
        pair = torch.arange(d, device="cuda") % (d // 2) if pairing == "half" else torch.arange(d, device="cuda") // 2
        still = pair >= count
        for inverse in (False, True):
            got = fas.fas_rotary(x, pos, pairs=(count - count // 2, count // 2), layout=layout, pairing=pairing, inverse=inverse)
            assert torch.equal(got[..., still].view(torch.int16), x[..., still].view(torch.int16))
            assert count == 0 or not torch.equal(got[..., ~still].view(torch.int16), x[..., ~still].view(torch.int16))


def test_rotary_of_rows_further_apart():
    """The projection's output and its gradient as columns of wider matrices."""
    H, d, n = 3, 64, 37
    wide = gen(4)(n, 3 * H * d + 40).to(BF16)
    pos = positions(1, 1, n)
    view = wide[:, 8:8 + 3 * H * d]
    kw = dict(pairs=(8, 12, 12))
    got = fas.fas_rotary_pack(view, pos, H, d, **kw)
    want = fas.fas_rotary_pack(view.contiguous(), pos, H, d, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    before = wide.clone()
    fas.fas_rotary_unpack(*got, pos, dqkv=view, **kw)
    assert torch.equal(view, fas.fas_rotary_unpack(*got, pos, **kw))
    assert torch.equal(wide[:, :8], before[:, :8]) and torch.equal(wide[:, 8 + 3 * H * d:], before[:, 8 + 3 * H * d:])


def test_rotary_of_many_heads():
    H, d, n = 4096, 64, 3
    pos = positions(1, 1, n)
    qkv = gen(12)(n, 3 * H * d).to(BF16)
    got = fas.fas_rotary_pack(qkv, pos, H, d, pairs=(4, 4, 24))
    parts = qkv.view(n, 3, H, d).permute(1, 2, 0, 3)
    want, bound = ref.rotary(parts[1], pos, (4, 4, 24), 10000.0, "half")
    assert torch.all((got[1].double() - want).abs() <= bound) and torch.equal(got[2], parts[2])


def test_rotary_offsets_beyond_32_bits():
    H, d, n = 24, 128, 240000  # 2.2 G elements
    qkv = torch.empty(n, 3 * H * d, device="cuda", dtype=BF16)
    rows = torch.tensor([0, 31, 32, 116508, 116509, 233016, 233017, n - 1], device="cuda")
    qkv[rows] = gen(5)(len(rows), 3 * H * d).to(BF16)
    pos = torch.arange(n, device="cuda")[:, None].float()
    q, k, v = fas.fas_rotary_pack(qkv, pos, H, d, pairs=(64,))
    parts = qkv[rows].view(-1, 3, H, d).permute(1, 2, 0, 3)
    for i, g in enumerate((q, k)):
        want, bound = ref.rotary(parts[i], pos[rows], (64,), 10000.0, "half")
        assert torch.all((g[:, rows].double() - want).abs() <= bound)
    assert torch.equal(v[:, rows], parts[2])
    del qkv
    back = fas.fas_rotary_unpack(q, k, v, pos, pairs=(64,))
    want, bound = ref.rotary(k[:, rows], pos[rows], (64,), 10000.0, "half", inverse=True)
    assert torch.all((back[rows].view(-1, 3, H, d)[:, 1].transpose(0, 1).double() - want).abs() <= bound)


def test_rotary_streams_and_graphs():
    H, d = 4, 128
    pos = positions(3, 20, 30)
    qkv = gen(6)(pos.shape[0], 3 * H * d).to(BF16)
    kw = dict(pairs=(16, 24, 24))
    want = fas.fas_rotary_pack(qkv, pos, H, d, **kw)
    back = fas.fas_rotary_unpack(*want, pos, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fas.fas_rotary_pack(qkv, pos, H, d, **kw)
        dqkv = fas.fas_rotary_unpack(*out, pos, **kw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            dqkv.zero_()
            g.replay()
        mine = fas.fas_rotary_pack(qkv, pos, H, d, stream=torch.cuda.current_stream(), **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip((*out, dqkv, *mine), (*want, back, *want)))


def test_rotary_refuses():
    qkv, pos = torch.zeros(10, 3 * 2 * 64, device="cuda", dtype=BF16), positions(1, 2, 5)
    ok = dict(pairs=(8, 12, 12))
    for match, call in (("positions", lambda: fas.fas_rotary_pack(qkv, pos[:, :2].contiguous(), 2, 64, **ok)),
                        ("positions", lambda: fas.fas_rotary_pack(qkv, pos[:9], 2, 64, **ok)),
                        ("qkv", lambda: fas.fas_rotary_pack(qkv, pos, 3, 64, **ok)),
                        ("more than", lambda: fas.fas_rotary_pack(qkv, pos, 2, 64, pairs=(20, 20, 20))),
                        ("pairs", lambda: fas.fas_rotary_pack(qkv, pos, 2, 64, pairs=(-1, 2, 3))),
                        ("pairs", lambda: fas.fas_rotary_pack(qkv, pos, 2, 64, pairs=(8, 12, 12), theta=(1.0, 2.0))),
                        ("layout", lambda: fas.fas_rotary_pack(qkv, pos, 2, 64, layout="dnh", **ok)),
                        ("pairing", lambda: fas.fas_rotary_pack(qkv, pos, 2, 64, pairing="quarter", **ok)),
                        ("strides", lambda: fas.fas_rotary_pack(qkv.T.contiguous().T, pos, 2, 64, **ok))):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(TypeError, match="positions"):
        fas.fas_rotary_pack(qkv, pos.double(), 2, 64, **ok)
    with pytest.raises(fas.FasError):  # heads of 32
        fas.fas_rotary_pack(qkv, pos, 4, 32, pairs=(4, 6, 6))
    q = torch.zeros(2, 10, 64, device="cuda", dtype=BF16)
    with pytest.raises(fas.FasError):  # two outputs at one address
        fas.fas_rotary_pack(qkv, pos, 2, 64, q=q, k=q, **ok)
    with pytest.raises(fas.FasError):  # no tokens
        fas.fas_rotary_pack(qkv[:0], pos[:0], 2, 64, **ok)


# ----------------------------------------------------- gradients' norm, clipping

def norm64(grads):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in grads))


def check_norm(got, grads):
    """Sums of 32 squares in fp32 (35 roundings of 2^-24 at most), the rest in
    64 bits; a square root halves that; the result rounded once."""
    want = norm64(grads)
    assert got.shape == () and got.dtype == torch.float32
    assert abs(float(got) - want) <= (18 * U32 + U32) * want, (float(got), want)
    return want


def check_clipped(out, grads, norm, max_norm, eps=1e-6):
    f = min(1.0, max_norm / (norm + eps))
    for o, g in zip(out, grads):
        want = g.double() * f
        u = torch.finfo(g.dtype).eps / 2
        tiny = torch.finfo(g.dtype).smallest_normal * torch.finfo(g.dtype).eps  # a step of the smallest values
        assert o.dtype == g.dtype and torch.all((o.double() - want).abs() <= (u + 24 * U32) * want.abs() + tiny)


SETS = {
    "one": [(1,)], "odd": [(333,), (7, 11), (8191,), (8193,), (3, 5, 7)], "aligned": [(8192,), (16384, 2), (64, 64)],
    "empty": [(0,), (5,), (0, 3), (17,), (0,)], "none": [(0,)], "many": [(i % 37,) for i in range(200)],
    "most": [(1 + i % 5,) for i in range(1000)], "exactly 960": [(2,)] * 960, "exactly 64": [(3,)] * 64, "two launches": [(9,)] * 1921,
    "big": [(4096, 2048), (2048,), (1000, 1001)],
}


@pytest.mark.parametrize("kind", ["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("name", list(SETS))
def test_gradient_norm_and_clipping(name, kind):
    rnd = gen(7)
    types = {"bf16": [BF16], "fp32": [torch.float32], "mixed": [BF16, torch.float32]}[kind]
    grads = [(rnd(*s) * 10.0 ** ((i % 7) - 4)).to(types[i % len(types)]) for i, s in enumerate(SETS[name])]
    norm = check_norm(fas.fas_gradient_norm(grads), grads)
    for max_norm in (0.3 * norm, 3 * norm + 1, 0.0):
        out = [torch.full_like(t, float("nan")) for t in grads]
        check_norm(fas.fas_clip_gradients(grads, max_norm, out=out), grads)
        check_clipped(out, grads, norm, max_norm)
        mine = [t.clone() for t in grads]
        fas.fas_clip_gradients(mine, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(mine, out))
    assert fas.fas_gradient_norm(tuple(grads)) == fas.fas_gradient_norm(iter(grads))


def test_gradient_norm_of_views():
    """Any alignment, transposed matrices, and outputs aligned otherwise."""
    rnd = gen(8)
    base = rnd(40000).to(BF16), rnd(40000)
    grads = [b[i:i + 9000 + 13 * i] for b in base for i in (0, 1, 2, 3, 5, 7, 8)]
    grads += [rnd(33, 65).t(), rnd(4, 6, 8).to(BF16).permute(2, 0, 1), rnd(1, 9).t()]
    norm = check_norm(fas.fas_gradient_norm(grads), grads)
    outs = []
    for i, g in enumerate(grads[:14]):
        outs.append(torch.empty(g.numel() + 8, dtype=g.dtype, device="cuda")[(i * 3) % 8:][:g.numel()])
    outs += [torch.empty_like(g) for g in grads[14:]]
    fas.fas_clip_gradients(grads, 0.5 * norm, out=outs)
    check_clipped(outs, grads, norm, 0.5 * norm)


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e15, 1e20, 1e30, 3e38])
def test_gradient_norm_beyond_the_range_of_squares(scale):
    """Values whose squares leave fp32's range, alone and among ordinary ones."""
    rnd = gen(9)
    for dtype in (BF16, torch.float32):
        grads = [(rnd(20000).clamp(-1, 1) * scale).to(dtype), torch.zeros(9000, dtype=dtype, device="cuda")]
        want = norm64(grads)
        got = fas.fas_gradient_norm(grads)
        if want < 3.4e38:
            assert abs(float(got) - want) <= 20 * U32 * want + 2.0 ** -149
        else:
            assert float(got) == math.inf
        if 1e-30 < want < 1e38:
            out = [torch.empty_like(t) for t in grads]
            fas.fas_clip_gradients(grads, 0.25 * want, eps=0.0, out=out)
            check_clipped(out, grads, want, float(np.float32(0.25 * want)), eps=0.0)
        mixed = [grads[0], rnd(30000).to(dtype)]
        check = norm64(mixed)
        if check < 3.4e38:
            check_norm(fas.fas_gradient_norm(mixed), mixed)


@pytest.mark.parametrize("scale,max_norm", [(1e37, 1.0), (3e38, 1.0), (3e38, 1e-6), (3e38, 1e-30), (1e30, 1e-12)])
def test_clipping_by_factors_below_fp32(scale, max_norm):
    """Huge gradients clipped to small norms: the factor is below fp32's normal
    numbers, the results need not be.  The norm itself may be beyond fp32."""
    rnd = gen(21)
    max_norm = float(np.float32(max_norm))
    for dtype in (BF16, torch.float32):
        grads = [(rnd(1_000_000).clamp(-1, 1) * scale).to(dtype), (rnd(8193)[1:] * 1e30).to(dtype), torch.ones(9, dtype=dtype, device="cuda")]
        norm = norm64(grads)
        assert max_norm / norm < 2.0 ** -126
        out = [torch.empty_like(t) for t in grads]
        got = float(fas.fas_clip_gradients(grads, max_norm, eps=0.0, out=out))
        assert got == math.inf if norm > 3.41e38 else abs(got - norm) <= 20 * U32 * norm
        check_clipped(out, grads, norm, max_norm, eps=0.0)
        fas.fas_clip_gradients(grads, max_norm, eps=0.0)
        assert all(torch.equal(a, b) for a, b in zip(grads, out))
    grads = [torch.full((100,), 3e38, device="cuda")]
    fas.fas_clip_gradients(grads, 0.0)
    assert bool((grads[0] == 0).all())
    grads = [torch.full((100,), 3e38, device="cuda")]
    fas.fas_clip_gradients(grads, math.inf)
    assert bool((grads[0] == 3e38).all())


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_gradient_norm_of_zeros(dtype):
    """Gradients of zero (rows that no token took) are read once like any
    others: they take no longer.  Zeros of both signs, and one value among them."""
    n = 300_000_000 if dtype == BF16 else 150_000_000  # 600 MB, several times L2
    dense, zeros = torch.ones(n, device="cuda", dtype=dtype), torch.zeros(n, device="cuda", dtype=dtype)
    zeros[1::2] = -0.0
    assert float(fas.fas_gradient_norm([zeros])) == 0.0

    def once(t):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(4):
            fas.fas_gradient_norm([t])
        end.record()
        end.synchronize()
        return start.elapsed_time(end)

    times = [(once(dense), once(zeros)) for _ in range(12)][2:]
    took = [sorted(t)[len(t) // 2] for t in zip(*times)]
    assert took[1] <= 1.25 * took[0], took
    for i, x in ((0, 3.0), (n // 2 + 1, 1e-30), (n - 1, -2e30)):
        zeros[i] = x
        check_norm(fas.fas_gradient_norm([zeros, zeros[:7]]), [zeros[i:i + 1], zeros[:7]])
        zeros[i] = 0


def test_gradient_norm_not_finite():
    x = [torch.ones(100, device="cuda"), torch.ones(50, device="cuda", dtype=BF16)]
    x[1][7] = float("inf")
    out = [torch.empty_like(t) for t in x]
    assert float(fas.fas_clip_gradients(x, 1.0, out=out)) == math.inf
    assert bool((out[0] == 0).all()) and bool(out[1][7].isnan()) and int(out[1].isnan().sum()) == 1
    x[0][3] = float("nan")
    assert math.isnan(float(fas.fas_clip_gradients(x, 1.0, out=out)))
    assert all(bool(t.isnan().all()) for t in out)


def test_gradients_that_need_no_clipping_stay():
    x = [torch.randn(5000, device="cuda").to(BF16), torch.zeros(10, device="cuda")]
    before = [t.clone() for t in x]
    fas.fas_clip_gradients(x, float("inf"))
    fas.fas_clip_gradients(x, 2 * norm64(x))
    assert all(torch.equal(a, b) for a, b in zip(x, before))
    zero = [torch.zeros(10, device="cuda")]
    assert float(fas.fas_clip_gradients(zero, 0.0, eps=0.0)) == 0.0 and bool((zero[0] == 0).all())
    assert float(fas.fas_gradient_norm([])) == 0.0 and float(fas.fas_clip_gradients([], 1.0)) == 0.0


def test_gradient_norm_streams_and_graphs():
    rnd = gen(10)
    grads = [rnd(1000, 301).to(BF16), rnd(77), rnd(4096, 64)]
    norm = norm64(grads)
    out = [torch.empty_like(t) for t in grads]
    want_norm = fas.fas_clip_gradients(grads, 0.1 * norm, out=out)
    want = [t.clone() for t in out]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fas.fas_clip_gradients(grads, 0.1 * norm, out=out)
    s = torch.cuda.Stream()
    other = [torch.empty_like(t) for t in grads]
    torch.cuda.synchronize()
    for _ in range(3):
        for t in (*out, *other, got):
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        mine = fas.fas_clip_gradients(grads, 0.1 * norm, out=other, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert float(got) == float(want_norm) == float(mine)
        assert all(torch.equal(a, w) and torch.equal(b, w) for a, b, w in zip(out, other, want))


def test_gradient_norm_offsets_beyond_32_bits():
    t = torch.zeros((1 << 31) + 5000, device="cuda", dtype=BF16)
    t[-3:] = 2.0
    t[17] = 1.0
    assert float(fas.fas_clip_gradients([t], 0.5, eps=0.0)) == float(np.float32(math.sqrt(13.0)))
    f = 0.5 / math.sqrt(13.0)
    assert abs(float(t[-1]) - 2 * f) <= 2 * f * 2 * U16 and abs(float(t[17]) - f) <= f * 2 * U16 and float(t[-4]) == 0.0


def test_gradient_norm_refuses():
    a, b = torch.zeros(100, device="cuda"), torch.zeros(100, device="cuda", dtype=BF16)
    with pytest.raises(fas.FasError):  # the same tensor twice would be scaled twice
        fas.fas_clip_gradients([a, a], 1.0)
    with pytest.raises(fas.FasError):
        fas.fas_clip_gradients([a[:60], a[50:]], 1.0)
    with pytest.raises(fas.FasError):
        fas.fas_clip_gradients([a, torch.zeros_like(a)], 1.0, out=[torch.zeros_like(a), a])
    assert float(fas.fas_gradient_norm([a, a])) == 0.0
    for bad in (-1.0, float("nan")):
        with pytest.raises(fas.FasError):
            fas.fas_clip_gradients([a], bad)
        with pytest.raises(fas.FasError):
            fas.fas_clip_gradients([a], 1.0, eps=bad)
    with pytest.raises(TypeError):
        fas.fas_gradient_norm([a.double()])
    with pytest.raises(TypeError):
        fas.fas_gradient_norm([a.cpu()])
    with pytest.raises(ValueError, match="contiguous"):
        fas.fas_gradient_norm([a[::2]])
    with pytest.raises(ValueError, match="out must hold"):
        fas.fas_clip_gradients([a, b], 1.0, out=[a])
    with pytest.raises(ValueError, match="type"):
        fas.fas_clip_gradients([a], 1.0, out=[b])


# ------------------------------------------------------- all of them, as called

class Step:
    """Every call once, on inputs of its own."""

    def __init__(self, seed=0, n=300):
        self.b = Block(n, 136, 200, seed=seed)
        rnd = gen(seed + 100)
        self.pos = positions(1, 1, n)
        self.qkv = rnd(n, 3 * 2 * 64).to(BF16)
        self.grads = [rnd(1000, 33).to(BF16), rnd(17), rnd(5000)]
        self.out = [torch.empty_like(t) for t in self.grads]

    def __call__(self, **kw):
        y, kept = self.b.forward(keep=True, **kw)
        pairs = dict(pairs=(8, 12, 12), **kw)
        q, k, v = fas.fas_rotary_pack(self.qkv, self.pos, 2, 64, **pairs)
        dqkv = fas.fas_rotary_unpack(q, k, v, self.pos, **pairs)
        out = [torch.empty_like(t) for t in self.grads] if not kw else self.out
        norm = fas.fas_clip_gradients(self.grads, 1.0, out=out, **kw)
        return (y, kept, *self.b.backward(kept, **kw), *self.b.backward(None, **kw), q, k, v, dqkv,
                fas.fas_rotary(q, self.pos, **pairs), fas.fas_gradient_norm(self.grads, **kw), norm, *out)


def test_plain_calls_take_native_code_and_give_the_same(monkeypatch):
    s = Step()
    native = []
    real = fas._native
    monkeypatch.setattr(fas, "_native", lambda call, *a: native.append((call, real(call, *a))) or native[-1][1])
    got = s()
    assert len(native) == 7 and all(r is not None for _, r in native)  # all but fas_rotary, which has no native form
    monkeypatch.setattr(fas, "_HOST", False)
    want = s()
    for a, b in zip(got, want, strict=True):
        assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device and torch.equal(a, b)
    p = torch.nn.Parameter(s.b.w_in)
    monkeypatch.setattr(fas, "_HOST", None)
    assert not fas.fas_feed_forward(s.b.x, p, s.b.w_out).requires_grad


def test_calls_in_several_threads():
    import threading
    cases = [Step(seed=i, n=n) for i, n in enumerate((300, 20, 4000, 129))]
    want = [c() for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(c, w):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                got = c()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, w, strict=True)):
                    bad.append(c)
    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_calls_on_a_stream_leave_the_current_streams_memory():
    """A tensor that is freed while work that reads it is still queued on the
    current stream keeps its values, whatever a call on another stream allocates."""
    c = Step(n=2000)
    want = [t.clone() for t in c()]
    s = torch.cuda.Stream()
    for size in (1 << 16, 1 << 18, 1 << 20):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        held = [torch.full((size,), 77, dtype=torch.uint8, device="cuda") for _ in range(30)]
        inputs = torch.cuda.current_stream().record_event()
        torch.cuda._sleep(20_000_000)  # about 10 ms
        copies = [t.clone() for t in held]
        del held
        s.wait_event(inputs)
        got = c(stream=s)
        torch.cuda.synchronize()
        assert all(bool((t == 77).all()) for t in copies)
        assert all(torch.equal(x, y) for x, y in zip(got, want, strict=True))


CAPTURED_FIRST = """
import torch
import frame_aligned_sparse_gb300 as fas
rnd = lambda *s: torch.randn(*s, device="cuda")
steps = []
for n, c, f in ((1, 64, 128), (12, 72, 64), (20, 64, 64), (100, 136, 200), (6000, 1024, 2048)):
    x, dy, w_in, w_out = (t.bfloat16() for t in (rnd(n, c), rnd(n, c), rnd(2 * f, c) / c ** 0.5, rnd(c, f) / f ** 0.5))
    def step(x=x, dy=dy, w_in=w_in, w_out=w_out):
        y, kept = fas.fas_feed_forward(x, w_in, w_out, keep=True)
        return (y, kept, *fas.fas_feed_forward_backward(dy, x, w_in, w_out, kept), *fas.fas_feed_forward_backward(dy, x, w_in, w_out))
    steps.append(step)
pos, qkv = torch.arange(50, device="cuda").float()[:, None], rnd(50, 3 * 2 * 64).bfloat16()
def turn():
    q, k, v = fas.fas_rotary_pack(qkv, pos, 2, 64, pairs=(32,), pairing="interleaved")
    return (q, k, v, fas.fas_rotary_unpack(q, k, v, pos, pairs=(32,)))
grads = [rnd(1000), rnd(10, 30).bfloat16()] * 1 + [rnd(3) for _ in range(70)]
out = [torch.empty_like(t) for t in grads]
def clip():
    return (fas.fas_gradient_norm(grads), fas.fas_clip_gradients(grads, 1.0, out=out), *[t.clone() for t in out])
steps += [turn, clip]
torch.cuda.synchronize()
for step in steps:
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step(), strict=True))
fas.fas_plan(48, 2, 0, 1, 2, 64)
assert fas.fas_status() == fas.FAS_OK
"""


def test_calls_captured_before_any_other():
    """A process whose first call of each kernel is a captured one."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(fas.__file__)))
    res = subprocess.run([sys.executable, "-c", CAPTURED_FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-4000:]


def test_calls_captured_on_a_branch_of_the_capture():
    """stream= a stream that was forked from the capturing one."""
    c = Step(n=700)
    want = [t.clone() for t in c()]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        branch, here = [], []
        for _ in range(2):
            branch.append(c(stream=side)[:-3])  # (the clipped gradients are one buffer for all)
            here.append(c())
        main.wait_stream(side)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for got in branch + here:
            assert all(torch.equal(x, y) for x, y in zip(got, want))
            for t in got:
                t.zero_()


def test_launch_counts():
    b = Block(300, 64, 128)
    y, kept = b.forward(keep=True)
    n = fas.fas_last_launch_count()
    assert n in (2, 3)  # a product split along k takes one more
    b.backward(kept)
    assert fas.fas_last_launch_count() in (3, 4, 5)
    fas.fas_feed_forward(b.x[:4], *b.weights)
    assert fas.fas_last_launch_count() == 2
    fas.fas_gradient_norm([b.x])
    assert fas.fas_last_launch_count() == 2
    fas.fas_clip_gradients([b.x.clone() for _ in range(961)], 1.0)
    assert fas.fas_last_launch_count() == 4


def test_a_training_step_of_a_block():
    """A block's step with the library's calls - projection split and turned,
    attention, norms with gates, feed-forward, their backward passes, clipping
    - against the same step in 64 bits by automatic differentiation.  About ten
    roundings to bf16 of at most 2^-8 each lie on a gradient's way:
    independent, they add up to at most sqrt(10) 2^-8 < 2^-6 of its norm."""
    w = workloads.get("tiny")
    T, nf, H, d = w.frame_tokens, w.total_frames, w.heads, w.head_dim
    N, C, F = w.tokens, H * d, 344
    rnd = gen(11)
    bf = lambda *s, scale=1.0: (rnd(*s) * scale).to(BF16)
    x, wqkv, wo = bf(N, C), bf(3 * C, C, scale=C ** -0.5), bf(C, C, scale=C ** -0.5)
    w_in, w_out = bf(2 * F, C, scale=C ** -0.5), bf(C, F, scale=F ** -0.5)
    post1, pre1, post2, pre2 = (1 + 0.1 * rnd(C) for _ in range(4))
    gate1, gate2 = 0.5 + 0.2 * rnd(nf, C), 0.5 + 0.2 * rnd(nf, C)
    dx2, dh2 = bf(N, C), bf(N, C)
    pos = positions(nf, 6, T // 6)
    pairs = (d // 8, 12, d // 2 - d // 8 - 12)
    fas.fas_plan(T, w.n_frames, w.ref_frames, w.window_radius, H, d)
    fas.fas_set_layout("nhd")

    # Forward.
    q, k, v = fas.fas_rotary_pack(x @ wqkv.T, pos, H, d, pairs=pairs, layout="nhd")
    fas.fas_prepass(q, k)
    out, lse = fas.fas_forward(q, k, v)
    y1 = out.reshape(N, C) @ wo.T
    x1, h1, r1 = fas.fas_residual_norm(y1, x, post1, pre1, gate=gate1, frame_tokens=T)
    y2, kept = fas.fas_feed_forward(h1, w_in, w_out, keep=True)
    x2, h2, r2 = fas.fas_residual_norm(y2, x1, post2, pre2, gate=gate2, frame_tokens=T)
    # Backward.
    dx1, dy2, dpost2, dpre2, dgate2 = fas.fas_residual_norm_backward(dx2, dh2, y2, x2, r2, post2, pre2, gate=gate2, frame_tokens=T)
    dh1, dw_in, dw_out = fas.fas_feed_forward_backward(dy2, h1, w_in, w_out, kept)
    dx, dy1, dpost1, dpre1, dgate1 = fas.fas_residual_norm_backward(dx1, dh1, y1, x1, r1, post1, pre1, gate=gate1, frame_tokens=T)
    dwo = dy1.T @ out.reshape(N, C)
    dq, dk, dv = fas.fas_backward(q, k, v, out, lse, (dy1 @ wo).reshape(N, H, d).contiguous())
    dqkv = fas.fas_rotary_unpack(dq, dk, dv, pos, pairs=pairs, layout="nhd")
    dwqkv = dqkv.T @ x
    dx = dx + dqkv @ wqkv
    grads = [dwqkv, dwo, dw_in, dw_out, dpost1, dpre1, dgate1, dpost2, dpre2, dgate2]
    before = [t.clone() for t in grads]
    norm = fas.fas_clip_gradients(grads, 1.0)
    assert fas.fas_status() == fas.FAS_OK

    # The same in 64 bits.
    leaves = [t.double().requires_grad_() for t in (wqkv, wo, w_in, w_out, post1, pre1, gate1, post2, pre2, gate2, x)]
    Wqkv, Wo, Win, Wout, p1, e1, g1, p2, e2, g2, X = leaves
    f = torch.arange(N, device="cuda") // T
    f64, axis = (t.cuda() for t in ref.frequencies(pairs, 10000.0, d))
    angle = pos.double()[:, axis] * f64
    turn = lambda t: torch.cat([t[..., :d // 2] * angle.cos() - t[..., d // 2:] * angle.sin(),
                                t[..., :d // 2] * angle.sin() + t[..., d // 2:] * angle.cos()], -1)
    Q, K, V = (X @ Wqkv.T).view(N, 3, H, d).permute(1, 2, 0, 3)
    fi, fj = f[:, None], f[None]
    see = (fi < w.ref_frames) | (fj < w.ref_frames) | ((fi - fj).abs() <= w.window_radius)
    A = (turn(Q) @ turn(K).transpose(1, 2) / d ** 0.5).masked_fill(~see, -math.inf).softmax(2) @ V
    rms = lambda t: t / torch.sqrt((t * t).mean(1, keepdim=True) + fas.RMS_EPS)
    X1 = X + g1[f] * rms(A.transpose(0, 1).reshape(N, C) @ Wo.T) * p1
    g, u = ((rms(X1) * e1) @ Win.T).chunk(2, 1)
    X2 = X1 + g2[f] * rms((g * torch.sigmoid(g) * u) @ Wout.T) * p2
    ((X2 * dx2.double()).sum() + (rms(X2) * e2 * dh2.double()).sum()).backward()
    names = ("wqkv", "wo", "w_in", "w_out", "post1", "pre1", "gate1", "post2", "pre2", "gate2", "x")
    for name, got, leaf in zip(names, (*before, dx), leaves):
        off = float((got.double() - leaf.grad).norm() / leaf.grad.norm())
        assert off <= 2.0 ** -6, (name, off)
    total = norm64(before)
    check_norm(norm, before)
    check_clipped(grads, before, total, 1.0)
