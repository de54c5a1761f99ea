"""Training operators, host side (no GPU): the references agree with
differences and with each other, and bad arguments are refused before any
device work."""
import ctypes

import numpy as np
import pytest
import torch

import frame_aligned_sparse_gb300 as fas
import training_reference as ref


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from frame_aligned_sparse_gb300 import build
    build.build()
    return fas.load()


@pytest.mark.parametrize("spans,R0,r", [([16, 32, 16, 48], 1, 1), ([16, 16, 32], 0, 0), ([16, 48], 2, 1)])
def test_attention_backward_reference_matches_differences(spans, R0, r):
    """The gradient formulas against central differences of the forward in 64
    bits: step 1e-5, so truncation 1e-10 and cancellation 1e-11 relative."""
    g = torch.Generator().manual_seed(0)
    h, n, d = 2, sum(spans), 64
    x = [torch.randn(h, n, d, generator=g, dtype=torch.float64) for _ in range(4)]
    q, k, v, dout = x
    out, lse = ref.attention(q, k, v, spans, R0, r)
    res = ref.attention_backward(q, k, v, out, lse, dout, spans, R0, r)
    for name, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        u = torch.randn(h, n, d, generator=g, dtype=torch.float64)
        ends = []
        for step in (1e-5, -1e-5):
            y = [t + step * u if j == i else t for j, t in enumerate(x[:3])]
            ends.append((ref.attention(*y, spans, R0, r)[0] * dout).sum())
        diff = (ends[0] - ends[1]) / 2e-5
        got = (res[name][0] * u).sum()
        assert abs(got - diff) <= 1e-6 * (res[name][0] * u).abs().sum(), name


@pytest.mark.parametrize("gated", [True, False])
def test_residual_norm_backward_reference_matches_differences(gated):
    g = torch.Generator().manual_seed(1)
    spans, c = [3, 1, 4], 24
    f = ref.frame_ids(spans)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    args = {"y": rnd(8, c), "x": rnd(8, c), "gamma_post": rnd(c), "gamma_pre": rnd(c), "gate": rnd(3, c) if gated else None}
    dx_out, dh = rnd(8, c), rnd(8, c)
    loss = lambda a: sum((o * w).sum() for o, w in zip(ref.residual_norm(**a, frame=f, alpha=0.7, eps=1e-6), (dx_out, dh)))
    xn, _, rstd = ref.residual_norm(**args, frame=f, alpha=0.7, eps=1e-6)
    dx, dy, dpost, dpre, dgate = ref.residual_norm_backward(dx_out, dh, args["y"], xn, rstd, args["gamma_post"],
                                                            args["gamma_pre"], args["gate"], f, 0.7)
    for name, grad in (("x", dx), ("y", dy), ("gamma_post", dpost), ("gamma_pre", dpre), ("gate", dgate)):
        if grad is None:
            continue
        u = rnd(*grad.shape)
        diff = (loss({**args, name: args[name] + 1e-5 * u}) - loss({**args, name: args[name] - 1e-5 * u})) / 2e-5
        assert abs((grad * u).sum() - diff) <= 1e-6 * (grad * u).abs().sum(), name


@pytest.mark.parametrize("geo", [(48, 2, 1, 1), (16, 4, 0, 0), (32, 3, 2, 1)], ids=str)
def test_oracle_attention_backward_matches_the_reference(geo):
    """The oracle's row-by-row backward (NumPy, bf16 bits) against this
    directory's batched one: the same numbers to 64-bit rounding."""
    import oracle
    T, F, R0, r = geo
    g = torch.Generator().manual_seed(2)
    h, n, d = 2, (F + R0) * T, 64
    q, k, v, dout = (torch.randn(h, n, d, generator=g).bfloat16() for _ in range(4))
    out, lse = ref.attention(q, k, v, [T] * (F + R0), R0, r)
    out = out.bfloat16()
    bits = lambda t: t.view(torch.int16).numpy().view(np.uint16)
    got = oracle.attention_backward(bits(q), bits(k), bits(v), bits(out), lse.numpy(), bits(dout), T, R0, r)
    want = ref.attention_backward(q, k, v, out, lse, dout, [T] * (F + R0), R0, r)
    for name in ("dq", "dk", "dv"):
        assert np.allclose(got[name], want[name][0].numpy(), rtol=1e-11, atol=1e-12), name


def test_checkpoint_reference_is_nearest():
    """The search-based packing reference against torch's e4m3 conversion on
    scaled values, and its error bound: half a step, 2^-4 of the value or
    2^-10 of the scale."""
    x = np.random.default_rng(0).standard_normal((64, 96)).astype(np.float32) * 3
    codes, scales = ref.checkpoint_pack(x)
    s = 2.0 ** (scales.astype(np.float64).repeat(32, -1) - 127)
    want = torch.from_numpy(x / s.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)
    err = np.abs(ref.checkpoint_unpack(codes, scales) - x)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))


P = ctypes.c_void_p
A = 0x1000  # an aligned address; never dereferenced by a refused call


def test_backward_refuses_without_plan():
    lib = fas.load()
    lib.fas_free()
    assert lib.fas_backward(*[P(A * (i + 1)) for i in range(10)], None) == fas.FAS_ERR_STATE


def norm_call(**kw):
    a = dict(y=A, x=2 * A, residual=0, gate=None, gp=3 * A, gq=4 * A, alpha=1.0, eps=1e-6, tokens=4, width=64, spans=None,
             frames=1, x_out=5 * A, h=6 * A, rstd=7 * A, yc=None, ys=None, xc=None, xs=None)
    a.update(kw)
    if isinstance(a["spans"], list):
        keep = np.array(a["spans"], dtype=np.int32)
        a["spans"] = keep.ctypes.data
    return fas.load().fas_residual_norm(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0), fas.FAS_ERR_ARG), (dict(width=0), fas.FAS_ERR_ARG), (dict(width=12), fas.FAS_ERR_ARG),
    (dict(width=16392), fas.FAS_ERR_UNSUPPORTED), (dict(residual=2), fas.FAS_ERR_ARG), (dict(eps=-1.0), fas.FAS_ERR_ARG),
    (dict(eps=float("nan")), fas.FAS_ERR_ARG), (dict(y=None), fas.FAS_ERR_ARG), (dict(rstd=None), fas.FAS_ERR_ARG),
    (dict(x=2 * A + 8), fas.FAS_ERR_ALIGN), (dict(yc=A), fas.FAS_ERR_ARG), (dict(h=5 * A), fas.FAS_ERR_ARG),
    (dict(yc=A, ys=A, xc=A, xs=A, width=72), fas.FAS_ERR_ARG),
    (dict(gate=A, frames=0), fas.FAS_ERR_ARG), (dict(gate=A, frames=3), fas.FAS_ERR_ARG),
    (dict(gate=A, frames=2, spans=[1, 2]), fas.FAS_ERR_ARG), (dict(gate=A, frames=2, spans=[4, 0]), fas.FAS_ERR_ARG),
    (dict(gate=A, frames=2, spans=[5, -1]), fas.FAS_ERR_ARG),
    (dict(gate=A, frames=1025, tokens=1025, spans=[1] * 1025), fas.FAS_ERR_UNSUPPORTED),
])
def test_residual_norm_refuses(kw, code):
    assert norm_call(**kw) == code


def norm_bwd_call(**kw):
    a = dict(dx_out=A, dh=2 * A, y=3 * A, x_out=4 * A, residual=0, yc=None, ys=None, xc=None, xs=None, rstd=5 * A, gate=None,
             gp=6 * A, gq=7 * A, alpha=1.0, tokens=4, width=64, spans=None, frames=1, dx=8 * A, dy=9 * A, dgate=None,
             dgp=10 * A, dgq=11 * A, ws=12 * A, wsb=1 << 30)
    a.update(kw)
    return fas.load().fas_residual_norm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0), fas.FAS_ERR_ARG), (dict(width=20), fas.FAS_ERR_ARG), (dict(width=1 << 15), fas.FAS_ERR_UNSUPPORTED),
    (dict(gate=A), fas.FAS_ERR_ARG), (dict(dgate=A), fas.FAS_ERR_ARG), (dict(y=None), fas.FAS_ERR_ARG),
    (dict(yc=A, ys=A, xc=A, xs=A), fas.FAS_ERR_ARG), (dict(y=None, x_out=None, yc=A, ys=A, xc=A), fas.FAS_ERR_ARG),
    (dict(y=None, x_out=None, yc=A, ys=A, xc=A, xs=A, width=72), fas.FAS_ERR_ARG),
    (dict(ws=None), fas.FAS_ERR_ARG), (dict(dy=8 * A), fas.FAS_ERR_ARG), (dict(ws=12 * A + 8), fas.FAS_ERR_ALIGN), (dict(dgp=None), fas.FAS_ERR_ARG),
])
def test_residual_norm_backward_refuses(kw, code):
    assert norm_bwd_call(**kw) == code


@pytest.mark.parametrize("args,code", [
    ((None, 0, A, A, 32), fas.FAS_ERR_ARG), ((A, 0, A, A, 0), fas.FAS_ERR_ARG), ((A, 0, A, A, 48), fas.FAS_ERR_ARG),
    ((A, 2, A, A, 32), fas.FAS_ERR_ARG), ((A + 4, 0, A, A, 32), fas.FAS_ERR_ALIGN), ((A, 0, A + 8, A, 32), fas.FAS_ERR_ALIGN),
    ((A, 0, A, A, -32), fas.FAS_ERR_ARG),
])
def test_checkpoint_calls_refuse(args, code):
    lib = fas.load()
    x, dtype, codes, scales, n = args
    assert lib.fas_checkpoint_pack(x, dtype, codes, scales, n, None) == code
    assert lib.fas_checkpoint_unpack(codes, scales, x, dtype, n, None) == code


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    g = torch.zeros(64)
    with pytest.raises(TypeError, match="CUDA"):
        fas.fas_residual_norm(x, x, g, g)
    with pytest.raises(TypeError, match="CUDA"):
        fas.fas_residual_norm_backward(x, x, x, x, torch.zeros(2, 4), g, g)
    with pytest.raises(TypeError):
        fas.fas_residual_norm(x, x.half(), g, g)
    with pytest.raises(TypeError, match="CUDA"):
        fas.fas_checkpoint_pack(x)
    with pytest.raises(TypeError):
        fas.fas_checkpoint_pack(x.half())
    with pytest.raises(TypeError):
        fas.fas_checkpoint_unpack(x)


@pytest.mark.parametrize("spans", [
    [3.9, 9.0, 4.0], np.array([3.2, 9.7, 4.9]), np.array([2**32 + 3, 9, 4]), torch.tensor([3, 9, 2**32 + 4]),
    np.array([2**64 - 1, 9, 8], dtype=np.uint64), [float("nan"), 9, 4], [[3, 9, 4]], [np.float32(3.5), 9, 4], [True, 2.5, 13], (), [3, 9], "3"],
    ids=str)
def test_frames_of_a_norm_are_whole_numbers(spans):
    """Spans that are no whole numbers, or no 32-bit ones, are not cut to some."""
    with pytest.raises((ValueError, TypeError, OverflowError)):
        fas._norm_frames(16, 8, torch.zeros(3, 8), spans, -1)


@pytest.mark.parametrize("tokens,spans", [(16, 5.5), (15, 5.4), (15, np.float32(5.0001)), (15, float("inf")), (15, 2**32 + 5),
                                          (15, np.array([5]))], ids=str)
def test_one_span_for_all_frames_is_a_whole_number(tokens, spans):
    with pytest.raises((ValueError, TypeError, OverflowError)):
        fas._norm_frames(tokens, 8, torch.zeros(3, 8), spans, -1)


@pytest.mark.parametrize("spans", [[3, 9, 4], (3, 9, 4), np.array([3, 9, 4]), np.array([3.0, 9.0, 4.0]), torch.tensor([3, 9, 4]),
                                   [np.int64(3), 9, np.int32(4)]], ids=str)
def test_frames_of_a_norm_in_every_kind_of_sequence(spans):
    _, got, n = fas._norm_frames(16, 8, torch.zeros(3, 8), spans, -1)
    assert n == 3 and list(got) == [3, 9, 4]
    for one in (5, np.int32(5), 5.0, torch.tensor(5), np.array(5)):
        assert fas._norm_frames(15, 8, torch.zeros(3, 8), one, -1)[1:] == (None, 3)


class FakeStream:
    cuda_stream = 7


class FakeLibrary:
    """Every call succeeds and writes nothing."""

    def __getattr__(self, name):
        return lambda *args: 0


STREAM_CALLS = {
    "backward": lambda t, s: fas.fas_backward(t.q, t.q, t.q, t.q, t.lse, t.q, stream=s),
    "norm": lambda t, s: fas.fas_residual_norm(t.x, t.x, t.g, t.g, gate=t.gate, checkpoint=True, stream=s),
    "norm_backward": lambda t, s: fas.fas_residual_norm_backward(t.x, t.x, t.x, t.x, t.rstd, t.g, t.g, gate=t.gate, stream=s),
    "pack": lambda t, s: fas.fas_checkpoint_pack(t.x, stream=s),
    "unpack": lambda t, s: fas.fas_checkpoint_unpack((t.codes, t.scales), stream=s),
    "forward": lambda t, s: fas.fas_forward(t.q, t.q, t.q, stream=s),
    "ablation": lambda t, s: fas.fas_forward_ablation(t.q, t.q, t.q, stream=s),
    "fold": lambda t, s: fas.fas_prologue_fold_weights(t.x, t.g, stream=s),
    "prologue": lambda t, s: fas.fas_prologue_with_key_sums(t.hidden, t.w, t.angles, t.angles, 2, 64, stream=s),
}
BUFFERS = {"backward": 4, "norm": 7, "norm_backward": 6, "pack": 2, "unpack": 1, "forward": 2, "ablation": 2, "fold": 1, "prologue": 4}


@pytest.mark.parametrize("given", [FakeStream(), None], ids=["stream", "current"])
@pytest.mark.parametrize("name", STREAM_CALLS)
def test_buffers_of_a_call_are_of_the_stream_it_runs_on(name, given, monkeypatch):
    """What a call allocates comes from the pool of the stream that writes it:
    memory of the current stream may have been freed with work still queued on
    it.  (The library and the streams are stand-ins: no kernel runs.)"""
    import contextlib
    import types
    bf16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    t = types.SimpleNamespace(q=bf16(2, 32, 64), lse=torch.zeros(2, 32), x=bf16(6, 64), g=torch.zeros(64), gate=torch.zeros(2, 64),
                              rstd=torch.zeros(2, 6), codes=torch.zeros(4, 64).to(torch.float8_e4m3fn),
                              scales=torch.zeros(4, 2, dtype=torch.uint8), hidden=bf16(32, 64), w=bf16(384, 64),
                              angles=torch.zeros(32, 32))
    active, made, kept = ["current"], [], []

    @contextlib.contextmanager
    def on(stream):
        active.append(stream)
        yield
        active.pop()

    def counted(real):
        def make(*args, **kw):
            got = real(*args, **kw)
            made.append((got.data_ptr(), active[-1]))
            return got
        return make
    for f in ("empty", "empty_like"):
        monkeypatch.setattr(torch, f, counted(getattr(torch, f)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "current")
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: kept.append((self.data_ptr(), s)))
    monkeypatch.setattr(fas, "load", FakeLibrary)
    monkeypatch.setattr(fas, "_current", lambda *a: (-1, 0))
    monkeypatch.setattr(fas, "_current_device_stream", lambda *a: (-1, 0))
    monkeypatch.setattr(fas, "_check_tensor", lambda *a: None)
    monkeypatch.setattr(fas, "_norm_workspace", lambda *a: 256)
    monkeypatch.setattr(fas, "_PLAN", dict(heads=2, tokens=32, head_dim=64))
    STREAM_CALLS[name](t, given)
    where = given or "current"
    assert len(made) == BUFFERS[name] and all(s is where for _, s in made), made
    # The caller goes on with the results on the current stream.
    if given:
        assert all((p, "current") in kept for p, _ in made)


def test_build_without_torch_headers(tmp_path, monkeypatch, capsys):
    """Where _host.so does not compile, libfas.so is built all the same, once,
    and no _host.so of another build stays."""
    from frame_aligned_sparse_gb300 import build
    source = tmp_path / "unit.cpp"
    source.write_text('extern "C" int answer() { return 42; }\n')
    (tmp_path / "torch").mkdir()
    monkeypatch.setattr(build, "_sources", lambda: [str(source)])
    monkeypatch.setattr(build, "_torch", lambda: str(tmp_path / "torch"))
    for name, file in (("OUT", "libfas.so"), ("HOST_OUT", "_host.so"), ("BUILD", "_build")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    (tmp_path / "_host.so").write_text("stale")
    assert build.build() == str(tmp_path / "libfas.so")
    assert ctypes.CDLL(build.OUT).answer() == 42
    assert not (tmp_path / "_host.so").exists()
    assert "without _host.so" in capsys.readouterr().err
    when = (tmp_path / "libfas.so").stat().st_mtime_ns
    build.build()
    assert (tmp_path / "libfas.so").stat().st_mtime_ns == when
    monkeypatch.setattr(build, "_torch", lambda: None)
    build.build()
    source.write_text("no C++")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()


@pytest.mark.parametrize("there", [False, True], ids=["missing", "unloadable"])
def test_calls_without_the_native_binding(there, tmp_path, monkeypatch):
    """Without a _host.so that loads, a call is left to Python, with one warning."""
    import types
    import warnings
    fas._host()
    if there:
        (tmp_path / "_host.so").write_text("not a library")
    monkeypatch.setattr(fas, "library_path", lambda: str(tmp_path / "libfas.so"))
    monkeypatch.setattr(fas, "_HOST", None)
    x = types.SimpleNamespace(is_cuda=True)
    with pytest.warns(RuntimeWarning, match="without the native binding"):
        assert fas._native("checkpoint_pack", x, x) is None
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert fas._native("checkpoint_pack", x, x) is None


def test_row_wait_selftest_refuses():
    assert fas.load().fas_selftest_row_wait_timeout(0, None) == fas.FAS_ERR_ARG
    assert fas.load().fas_selftest_row_wait_timeout(1000001, None) == fas.FAS_ERR_ARG


def test_native_calls_load_without_a_gpu():
    host = fas._host()
    assert all(callable(getattr(host, f"{n}")) for n in (
        "backward", "residual_norm", "residual_norm_backward", "checkpoint_pack", "checkpoint_unpack"))
    with pytest.raises(TypeError):
        host.bind(1, 2)
