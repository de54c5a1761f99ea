"""The block's operators, host side (no GPU): the references agree with
differences and with each other, and bad arguments are refused before any
device work."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import block_reference as ref
import frame_aligned_sparse_gb300 as fas


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from frame_aligned_sparse_gb300 import build
    build.build()
    return fas.load()


# ------------------------------------------------------------- references

@pytest.mark.parametrize("act", list(fas.ACTIVATIONS))
def test_feed_forward_reference_matches_differences(act):
    """Central differences in 64 bits, step 1e-5: truncation 1e-10 and cancellation 1e-11 relative."""
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    n, c, f = 5, 16, 24
    args = {"x": rnd(n, c), "w_in": rnd(2 * f, c) / 4, "w_out": rnd(c, f) / 4}
    dy = rnd(n, c)

    def loss(x, w_in, w_out):
        gate, up = (x @ w_in.T).chunk(2, 1)
        return ((ref.activation(gate, act)[0] * up) @ w_out.T * dy).sum()

    kept = ref.projections(args["x"], args["w_in"])[0]
    got = ref.feed_forward_backward(dy, *args.values(), kept, act)
    for name, res in zip(args, got.values()):
        d = rnd(*res[0].shape)
        diff = (loss(**{**args, name: args[name] + 1e-5 * d}) - loss(**{**args, name: args[name] - 1e-5 * d})) / 2e-5
        assert abs((res[0] * d).sum() - diff) <= 1e-6 * (res[0] * d).abs().sum(), name
    y = ref.feed_forward(*args.values(), act)["y"][0]
    assert abs((y * dy).sum() - loss(**args)) <= 1e-12 * (y * dy).abs().sum()


def test_feed_forward_bounds_hold_for_rounded_arithmetic():
    """The forward and backward passes done in fp32 with the kernels'
    roundings to bf16 stay within the references' bounds and deviations."""
    g = torch.Generator().manual_seed(1)
    n, c, f = 60, 128, 96
    x, dy = (torch.randn(n, c, generator=g).bfloat16() for _ in range(2))
    w_in, w_out = (torch.randn(2 * f, c, generator=g) / 11).bfloat16(), (torch.randn(c, f, generator=g) / 10).bfloat16()
    for act in fas.ACTIVATIONS:
        gu = x.float() @ w_in.float().T
        gate, up = gu.chunk(2, 1)
        h = (ref.activation(gate, act)[0] * up).bfloat16()
        want = ref.feed_forward(x, w_in, w_out, act)
        ref.check((h.float() @ w_out.float().T).bfloat16(), want["y"], "y")
        ref.check(gu.bfloat16(), want["kept"], "kept")
        kept = gu.bfloat16()
        gate, up = kept.float().chunk(2, 1)
        a, da = ref.activation(gate, act)
        dh = dy.float() @ w_out.float()
        dgu = torch.cat([dh * up * da, dh * a], 1).bfloat16().float()
        want = ref.feed_forward_backward(dy, x, w_in, w_out, kept, act)
        ref.check((dgu @ w_in.float()).bfloat16(), want["dx"], "dx")
        ref.check((dgu.T @ x.float()).bfloat16(), want["dw_in"], "dw_in")
        ref.check((dy.float().T @ (a * up).bfloat16().float()).bfloat16(), want["dw_out"], "dw_out")


@pytest.mark.parametrize("pairing", list(fas.PAIRINGS))
def test_rotary_reference_is_a_rotation(pairing):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(3, 10, 64, generator=g, dtype=torch.float64)
    pos = torch.randn(10, 2, generator=g) * 50
    y, _ = ref.rotary(x, pos, (10, 20), (100.0, 1000.0), pairing)
    back, _ = ref.rotary(y, pos, (10, 20), (100.0, 1000.0), pairing, inverse=True)
    assert torch.allclose(back, x, rtol=0, atol=1e-12) and torch.allclose(y.norm(dim=2), x.norm(dim=2), rtol=1e-12)
    # The gradient's way back is the opposite turn: <turn x, z> = <x, turn back z>.
    z = torch.randn(3, 10, 64, generator=g, dtype=torch.float64)
    assert torch.allclose((y * z).sum(), (x * ref.rotary(z, pos, (10, 20), (100.0, 1000.0), pairing, inverse=True)[0]).sum())
    # Pair 0 of the first axis turns by its position; pairs beyond the 30 given stay.
    i, j = (0, 32) if pairing == "half" else (0, 1)
    p = pos[:, 0].double()
    assert torch.allclose(y[..., i], x[..., i] * p.cos() - x[..., j] * p.sin(), rtol=0, atol=1e-12)
    rest = [30, 31, 62, 63] if pairing == "half" else [60, 61, 62, 63]
    assert torch.equal(y[..., rest], x[..., rest])


def test_turns_are_the_frequencies():
    t = fas._turns_of([3, 0, 5], [10.0, 2.0, 100.0], 64)
    assert t.axes == 3 and t.pairs == 8 and list(t.axis) == [0] * 3 + [2] * 5
    assert np.allclose(list(t.frequencies), [10.0 ** (-i / 3) for i in range(3)] + [100.0 ** (-i / 5) for i in range(5)], rtol=1e-15)
    assert fas._turns_of((3, 0, 5), (10.0, 2.0, 100.0), 64) is t  # made once
    for pairs, theta in (((), 10.0), ((20, 20), 10.0), ((-1,), 10.0), ((1.5,), 10.0), ((4, 4), (10.0,)), ((4,), 0.0), ((4,), -1.0), ((4,), math.nan)):
        with pytest.raises(ValueError):
            fas._turns_of(pairs, theta, 64)


# --------------------------------------------------------------- refusals

A = 0x1000  # an aligned address; never dereferenced by a refused call


def ff_call(**kw):
    a = dict(x=A, w_in=2 * A, w_out=3 * A, act=0, tokens=4, width=64, inner=72, y=4 * A, kept=None, ws=6 * A, wsb=1 << 40)
    a.update(kw)
    return fas.load().fas_feed_forward(*a.values(), None)


def ff_bwd_call(**kw):
    a = dict(dy=A, x=2 * A, w_in=3 * A, w_out=4 * A, kept=5 * A, act=0, tokens=4, width=64, inner=72, dx=6 * A, dwi=7 * A,
             dwo=8 * A, ws=9 * A, wsb=1 << 40)
    a.update(kw)
    return fas.load().fas_feed_forward_backward(*a.values(), None)


SHAPE_REFUSALS = [(dict(tokens=0), fas.FAS_ERR_ARG), (dict(tokens=-5), fas.FAS_ERR_ARG), (dict(tokens=1 << 31), fas.FAS_ERR_ARG),
                  (dict(width=60), fas.FAS_ERR_ARG), (dict(inner=0), fas.FAS_ERR_ARG), (dict(inner=-8), fas.FAS_ERR_ARG),
                  (dict(width=1 << 25), fas.FAS_ERR_UNSUPPORTED), (dict(inner=1 << 25), fas.FAS_ERR_UNSUPPORTED),
                  (dict(act=2), fas.FAS_ERR_ARG), (dict(act=-1), fas.FAS_ERR_ARG), (dict(x=None), fas.FAS_ERR_ARG),
                  (dict(ws=None), fas.FAS_ERR_ARG), (dict(x=2 * A + 8), fas.FAS_ERR_ALIGN)]


@pytest.mark.parametrize("kw,code", SHAPE_REFUSALS + [(dict(y=A), fas.FAS_ERR_ARG), (dict(kept=4 * A), fas.FAS_ERR_ARG),
                                                      (dict(ws=3 * A), fas.FAS_ERR_ARG), (dict(y=4 * A + 2), fas.FAS_ERR_ALIGN),
                                                      (dict(kept=5 * A + 4), fas.FAS_ERR_ALIGN), (dict(y=None), fas.FAS_ERR_ARG)])
def test_feed_forward_refuses(kw, code):
    assert ff_call(**kw) == code


@pytest.mark.parametrize("kw,code", SHAPE_REFUSALS + [(dict(dx=A), fas.FAS_ERR_ARG), (dict(dwi=3 * A), fas.FAS_ERR_ARG),
                                                      (dict(dwo=7 * A), fas.FAS_ERR_ARG), (dict(dx=5 * A), fas.FAS_ERR_ARG),
                                                      (dict(dwo=None), fas.FAS_ERR_ARG), (dict(kept=5 * A + 2), fas.FAS_ERR_ALIGN),
                                                      (dict(dwo=8 * A + 8), fas.FAS_ERR_ALIGN), (dict(dy=None), fas.FAS_ERR_ARG)])
def test_feed_forward_backward_refuses(kw, code):
    assert ff_bwd_call(**kw) == code


def test_feed_forward_workspace_refuses():
    n = ctypes.c_int64()
    lib = fas.load()
    for args in ((0, 64, 64), (4, 4, 64), (4, 64, 12)):
        assert lib.fas_feed_forward_workspace(*args, 0, 0, ctypes.byref(n)) == fas.FAS_ERR_ARG
    assert lib.fas_feed_forward_workspace(4, 64, 64, 0, 0, None) == fas.FAS_ERR_ARG


def test_product_wait_selftest_refuses():
    for limit_us in (0, 5001):
        assert fas.load().fas_selftest_product_wait_timeout(limit_us, None) == fas.FAS_ERR_ARG


SPREADS = r"""
#include "feed_forward_plan.h"

#include <cstdio>
#include <random>

using namespace fas::feed_forward;

static int bad(const char* what, Machine m, long n, long c, long f) {
  std::printf("%s: %d CTAs, %d pairs, %ld x %ld x %ld\n", what, m.ctas, m.pairs, n, c, f);
  return 1;
}

int main() {
  std::mt19937 rng(7);
  auto size = [&](double most) { return (long)std::exp(std::uniform_real_distribution<double>(0, std::log(most))(rng)); };
  const Machine machines[] = {{152, 76}, {152, 70}, {152, 75}, {148, 1}, {152, 0}, {1, 0}, {2, 1}};
  for (int i = 0; i < 20000; ++i) {
    const long n = size(300000), c = 8 * size(2048), f = 8 * size(4096);
    for (const Machine& m : machines) {
      struct {
        Epilogue e;
        long rows, cols, rows2, k;
        const Spread s;
        const Workspace* ws;
      } const products[] = {
          {kGateUp, n, 2 * f, 0, c, spread(kGateUp, n, 2 * f, c, m), nullptr},
          {kInner, n, f, 0, c, spread(kInner, n, f, c, m), nullptr},
          {kPlain, n, c, 0, f, spread(kPlain, n, c, f, m), nullptr},
          {kPlain, n, c, 0, 2 * f, spread(kPlain, n, c, 2 * f, m), nullptr},
          {kPlain, 2 * f, c, c, n, spread_weights(n, c, f, m), nullptr},
      };
      const Workspace forward(n, (int)c, (int)f, false, true, m), kept(n, (int)c, (int)f, true, true, m),
          again(n, (int)c, (int)f, true, false, m);
      const Workspace* const room[][2] = {{}, {}, {&forward, &forward}, {&kept, &again}, {&kept, &again}};
      for (int j = 0; j < 5; ++j) {
        const auto& p = products[j];
        const Spread& s = p.s;
        const Form& form = kForms[s.form];
        const long units = form.G == 1 ? m.ctas : m.pairs;
        if (units < 1) return bad("a form that cannot run", m, n, c, f);
        if (p.e != kPlain && (s.form == 2 || s.parts)) return bad("an epilogue in parts", m, n, c, f);
        const long tiles = form.tiles(p.rows, p.cols) + (p.rows2 ? form.tiles(p.rows2, f) : 0), steps = (p.k + 63) / 64;
        const long per = (steps + s.splits - 1) / s.splits;
        if (s.whole + s.parts / s.splits != tiles || s.parts % s.splits) return bad("tiles", m, n, c, f);
        if (s.parts && (s.whole % units || s.splits < 2 || s.parts / s.splits >= units)) return bad("rounds", m, n, c, f);
        if (s.parts && (s.splits - 1) * per >= steps) return bad("a part without a step", m, n, c, f);
        if (!s.parts && s.splits != 1) return bad("splits of nothing", m, n, c, f);
        for (const Workspace* w : room[j])
          if (w && (j != 2 || n > kFewTokens) && w->bytes - w->parts < s.parts * form.rows() * form.cols * 4)
            return bad("workspace", m, n, c, f);
      }
    }
  }
  return 0;
}
"""


def test_feed_forward_products_are_spread_over_what_runs(tmp_path):
    """Tiles, rounds, parts and workspace go by the CTAs and pairs that run at
    once, which need not be all SMs' worth of pairs."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    csrc = os.path.join(os.path.dirname(fas.__file__), "csrc")
    (tmp_path / "spreads.cpp").write_text("#include <cmath>\n" + SPREADS)
    exe = str(tmp_path / "spreads")
    subprocess.run([gxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + csrc, str(tmp_path / "spreads.cpp"), "-o", exe], check=True)
    got = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert got.returncode == 0, got.stdout


# Width, inner, tokens; us of a forward pass with both products over the weights
# in one pass, with the gate-up product only, with the other only, and with
# tiles for both (medians, weights in HBM).
FEW = [(64, 64, 31, 4.9, 5.7, 6.1, 7.2), (256, 1024, 24, 6.7, 10.8, 8.4, 12.8), (1024, 2728, 12, 10.9, 15.4, 14.5, 18.9),
       (1024, 2728, 31, 16.0, 18.1, 17.1, 19.1), (2048, 5504, 1, 15.8, 22.1, 22.7, 29.0), (2048, 5504, 16, 19.5, 23.2, 22.4, 26.1),
       (2048, 5504, 17, 26.9, 28.0, 25.1, 26.2), (2048, 5504, 24, 27.7, 28.3, 25.3, 25.9), (2048, 5504, 31, 28.4, 29.3, 25.7, 26.2),
       (4096, 11008, 16, 56.1, 59.8, 69.0, 71.7), (4096, 11008, 24, 80.6, 77.3, 75.9, 72.1), (8192, 1024, 8, 22.6, 25.4, 46.3, 49.2),
       (8192, 1024, 24, 46.2, 44.1, 51.2, 49.4), (1024, 16384, 12, 36.2, 33.4, 37.4, 35.3), (1024, 16384, 24, 54.3, 41.9, 44.5, 33.2),
       (104, 9336, 12, 18.8, 18.0, 21.2, 19.9), (104, 9336, 24, 28.6, 21.8, 27.5, 20.2)]


def test_few_tokens_take_the_form_that_was_measured_faster(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    calls = "".join(f'  std::printf("%d %d\\n", few_gate_up({n}, {f}), few_out({n}, {c}, {f}));\n' for c, f, n, *_ in FEW)
    (tmp_path / "few.cpp").write_text('#include "feed_forward_plan.h"\n#include <cstdio>\nusing namespace fas::feed_forward;\n'
                                      "int main() {\n" + calls + "}\n")
    exe = str(tmp_path / "few")
    csrc = os.path.join(os.path.dirname(fas.__file__), "csrc")
    subprocess.run([gxx, "-std=c++17", "-I" + csrc, str(tmp_path / "few.cpp"), "-o", exe], check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True, timeout=60).stdout.split("\n")
    for (c, f, n, *us), line in zip(FEW, got):
        gate_up, out = (bool(int(v)) for v in line.split())
        chosen = us[(0 if gate_up else 2) + (0 if out else 1)]
        assert chosen <= 1.04 * min(us), (c, f, n, gate_up, out)  # the measurements' own spread


def rotary_call(**kw):
    a = dict(ins=[A, 2 * A, 3 * A], in_strides=[384, 64] * 3, outs=[4 * A, 5 * A, 6 * A], out_strides=[64, 640] * 3, turned=[1, 1, 0],
             n=3, positions=7 * A, axes=2, freq=[1.0, 0.5, 0.25], axis=[0, 1, 1], pairs=3, pairing=0, inverse=0, tokens=10, heads=2,
             head_dim=64)
    a.update(kw)
    arr = lambda t, v: None if v is None else (t * len(v))(*v)
    return fas.load().fas_rotary(arr(ctypes.c_void_p, a["ins"]), arr(ctypes.c_int64, a["in_strides"]), arr(ctypes.c_void_p, a["outs"]),
                                 arr(ctypes.c_int64, a["out_strides"]), arr(ctypes.c_int32, a["turned"]), a["n"], a["positions"],
                                 a["axes"], arr(ctypes.c_double, a["freq"]), arr(ctypes.c_int32, a["axis"]), a["pairs"], a["pairing"],
                                 a["inverse"], a["tokens"], a["heads"], a["head_dim"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), fas.FAS_ERR_ARG), (dict(n=4), fas.FAS_ERR_ARG), (dict(ins=None), fas.FAS_ERR_ARG), (dict(turned=None), fas.FAS_ERR_ARG),
    (dict(positions=None), fas.FAS_ERR_ARG), (dict(axes=0), fas.FAS_ERR_ARG), (dict(axes=5), fas.FAS_ERR_ARG),
    (dict(axis=[0, 2, 1]), fas.FAS_ERR_ARG), (dict(axis=[0, -1, 1]), fas.FAS_ERR_ARG), (dict(pairs=33), fas.FAS_ERR_ARG),
    (dict(pairs=-1), fas.FAS_ERR_ARG), (dict(freq=None), fas.FAS_ERR_ARG), (dict(freq=[1.0, math.inf, 1.0]), fas.FAS_ERR_ARG),
    (dict(freq=[1.0, math.nan, 1.0]), fas.FAS_ERR_ARG), (dict(freq=[1.0, -2.0 ** 33, 1.0]), fas.FAS_ERR_ARG), (dict(pairing=2), fas.FAS_ERR_ARG), (dict(tokens=0), fas.FAS_ERR_ARG),
    (dict(tokens=1 << 31), fas.FAS_ERR_ARG), (dict(heads=0), fas.FAS_ERR_ARG), (dict(heads=4097), fas.FAS_ERR_ARG),
    (dict(head_dim=32), fas.FAS_ERR_ARG), (dict(head_dim=256), fas.FAS_ERR_ARG), (dict(ins=[A, None, 3 * A]), fas.FAS_ERR_ARG),
    (dict(outs=[4 * A, 4 * A, 6 * A]), fas.FAS_ERR_ARG), (dict(outs=[4 * A, A, 6 * A]), fas.FAS_ERR_ARG),
    (dict(outs=[A, 5 * A, 6 * A]), fas.FAS_ERR_ARG),  # in place with other strides
    (dict(in_strides=[384, 60] * 3), fas.FAS_ERR_ALIGN), (dict(out_strides=[68, 640] * 3), fas.FAS_ERR_ALIGN),
    (dict(ins=[A + 8, 2 * A, 3 * A]), fas.FAS_ERR_ALIGN), (dict(positions=7 * A + 2), fas.FAS_ERR_ALIGN),
])
def test_rotary_refuses(kw, code):
    assert rotary_call(**kw) == code


def clip_call(**kw):
    a = dict(grads=[A, 2 * A], outs=None, elements=[100, 50], dtypes=[0, 1], n=2, max_norm=1.0, eps=1e-6, norm=4 * A, ws=5 * A)
    a.update(kw)
    arr = lambda t, v: None if v is None else (t * len(v))(*v)
    lists = (arr(ctypes.c_void_p, a["grads"]), arr(ctypes.c_void_p, a["outs"]), arr(ctypes.c_int64, a["elements"]),
             arr(ctypes.c_int32, a["dtypes"]))
    clip = fas.load().fas_clip_gradients(*lists, a["n"], a["max_norm"], a["eps"], a["norm"], a["ws"], None)
    only = {k for k in kw} & {"outs", "max_norm", "eps"}
    if not only and "overlap" not in kw:
        assert fas.load().fas_gradient_norm(lists[0], *lists[2:], a["n"], a["norm"], a["ws"], None) == clip
    return clip


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), fas.FAS_ERR_ARG), (dict(grads=None), fas.FAS_ERR_ARG), (dict(elements=None), fas.FAS_ERR_ARG),
    (dict(dtypes=None), fas.FAS_ERR_ARG), (dict(grads=[A, None]), fas.FAS_ERR_ARG), (dict(elements=[-1, 4]), fas.FAS_ERR_ARG),
    (dict(dtypes=[0, 2]), fas.FAS_ERR_ARG), (dict(ws=None), fas.FAS_ERR_ARG), (dict(ws=5 * A + 8), fas.FAS_ERR_ALIGN),
    (dict(grads=[A + 1, 2 * A]), fas.FAS_ERR_ALIGN), (dict(grads=[A, 2 * A + 2]), fas.FAS_ERR_ALIGN),
    (dict(max_norm=-1.0), fas.FAS_ERR_ARG), (dict(max_norm=math.nan), fas.FAS_ERR_ARG), (dict(eps=-1.0), fas.FAS_ERR_ARG),
    (dict(outs=[A, None]), fas.FAS_ERR_ARG), (dict(outs=[A, 2 * A + 2]), fas.FAS_ERR_ALIGN),
    (dict(outs=[2 * A, A]), fas.FAS_ERR_ARG), (dict(outs=[A + 198, 2 * A]), fas.FAS_ERR_ARG), (dict(outs=[3 * A, 3 * A + 196]), fas.FAS_ERR_ARG),
    (dict(grads=[A, A], overlap=1), fas.FAS_ERR_ARG), (dict(grads=[A, A + 196], overlap=1), fas.FAS_ERR_ARG),
])
def test_clip_gradients_refuses(kw, code):
    assert clip_call(**kw) == code
