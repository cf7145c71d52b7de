"""The gated operators refuse what they cannot take, without a GPU: the binding's checks of
tensors, its warnings, the C entry points' checks before any HIP call."""
import ctypes
import os
import re
import warnings

import pytest

torch = pytest.importorskip("torch")

import fp4_communication_compression_amd as fp4q
from fp4_communication_compression_amd import gated, linear

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3, E5M2, BF16, F32 = torch.float8_e4m3fn, torch.float8_e5m2, torch.bfloat16, torch.float32


def status(status):
    return pytest.raises(fp4q.Fp4qError, match=r"\(status %d\)" % status)


def test_header_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp4q_gated.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fp4q_[a-z0-9_]+)\s*\(", text)))
    assert names == ["fp4q_gated4", "fp4q_gated8", "fp4q_gated8_backward", "fp4q_gated8_workspace", "fp4q_gemv4",
                     "fp4q_gemv4_workspace"]
    for n in names:
        assert hasattr(fp4q.lib(), n), n
    for i, name in enumerate(("FP4Q_ACT_SILU", "FP4Q_ACT_GELU", "FP4Q_ACT_GELU_TANH", "FP4Q_ACT_RELU")):
        assert re.search(r"%s = %d\b" % (name, i), text)
        assert getattr(fp4q, name) == getattr(gated, name) == i


# ------------------------------------------------------------------- binding
def operands(n=300, k=256):
    r = (n + 127) // 128 * 128 + n
    return (torch.zeros(4, k, dtype=E4M3), torch.ones((k + 127) // 128, 4), torch.zeros(r, k, dtype=E4M3),
            torch.ones((k + 127) // 128, (r + 127) // 128))


def test_gated8_arguments():
    a, sa, w, sw = operands()
    with pytest.raises(ValueError, match="activation"):
        fp4q.fp4q_gated8(a, sa, w, sw, "tanh")
    with pytest.raises(TypeError, match="float8"):
        fp4q.fp4q_gated8(a.view(torch.uint8), sa, w, sw)
    with pytest.raises(TypeError, match="gate_up must be float8"):
        fp4q.fp4q_gated8(a, sa, w.float(), sw)
    with pytest.raises(ValueError, match="columns"):
        fp4q.fp4q_gated8(a, sa, w[:, :128], sw)
    for rows in (100, 128, 600):      # an odd number of blocks of 128 rows
        with pytest.raises(ValueError, match="rows of the gate"):
            fp4q.fp4q_gated8(a, sa, w[:rows].contiguous(), sw)
    with pytest.raises(ValueError, match="gate_up's scales"):
        fp4q.fp4q_gated8(a, sa, w[:500].contiguous(), sw)
    with pytest.raises(ValueError, match="a's scales"):
        fp4q.fp4q_gated8(a, sa.t().contiguous(), w, sw)
    with pytest.raises(ValueError, match="gate_up's scales"):
        fp4q.fp4q_gated8(a, sa, w, torch.ones(2, w.shape[0]))
    with pytest.raises(TypeError, match="gate_up's scales"):
        fp4q.fp4q_gated8(a, sa, w, sw.double())
    with pytest.raises(ValueError, match="GPU"):
        fp4q.fp4q_gated8(a, sa, w, sw)


@pytest.mark.parametrize("n", [1, 127, 128, 129, 300, 11008, 2752])
def test_the_joined_rows_say_how_many_outputs_there_are(n, monkeypatch):
    a, sa, w, sw = operands(n, 128)
    seen = {}

    class Library:
        def fp4q_gated8(self, *args):
            seen["n"] = args[9]
            return 0

    monkeypatch.setattr(gated, "_bound", Library())
    monkeypatch.setattr(gated, "_gpu", lambda *t: 0)
    monkeypatch.setattr(gated, "_current_gpu", lambda: 0)
    monkeypatch.setattr(gated, "_launch_stream", lambda *s: None)
    monkeypatch.setattr(linear, "_workspace", lambda *s: 0)
    out = fp4q.fp4q_gated8(a, sa, w, sw, want_pre=True)
    assert seen["n"] == n and all(t.shape == (4, n) and t.dtype == BF16 for t in out)


def test_gated8_backward_arguments():
    x = torch.zeros(4, 256, dtype=BF16)
    with pytest.raises(ValueError, match="activation"):
        fp4q.fp4q_gated8_backward(x, x, x, "swish")
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        fp4q.fp4q_gated8_backward(x.half(), x.half(), x.half())
    with pytest.raises(TypeError, match="gate must"):
        fp4q.fp4q_gated8_backward(x, x.float(), x)
    with pytest.raises(ValueError, match="up must"):
        fp4q.fp4q_gated8_backward(x, x, x[:3])
    with pytest.raises(ValueError, match="contiguous"):
        fp4q.fp4q_gated8_backward(x, x, torch.zeros(256, 4, dtype=BF16).t())
    with pytest.raises(TypeError, match="float8"):
        fp4q.fp4q_gated8_backward(x, x, x, dtype=BF16)
    with pytest.raises(ValueError, match="ask for"):
        fp4q.fp4q_gated8_backward(x, x, x, straight=False, transposed=False)
    with status(fp4q.FP4Q_ERR_SHAPE):
        fp4q.fp4q_gated8_backward(*(x[:, :0].contiguous() for _ in range(3)))
    with pytest.raises(ValueError, match="GPU"):
        fp4q.fp4q_gated8_backward(x, x, x)


def payload(n=6, k=512):
    return (torch.zeros(n, k // 2, dtype=torch.uint8), torch.zeros(n, k // 16, dtype=torch.uint8), torch.ones(n, k // 256))


@pytest.mark.parametrize("call", [lambda x, w, **k: fp4q.fp4q_gemv4(x, w, **k),
                                  lambda x, w, **k: fp4q.fp4q_gated4(x, payload(), w, **k),
                                  lambda x, w, **k: fp4q.fp4q_gated4(x, w, payload(), **k)])
def test_4_bit_arguments(call):
    x, w = torch.zeros(3, 512, dtype=BF16), payload()
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        call(x.half(), w)
    with pytest.raises(ValueError, match="contiguous"):
        call(x[:, ::2], w)
    with status(fp4q.FP4Q_ERR_SHAPE):
        call(x[:, :500].contiguous(), w)
    with pytest.raises(TypeError, match="payload"):
        call(x, w[:2])
    with pytest.raises(TypeError, match="payload"):
        call(x, None)
    with pytest.raises(TypeError, match="codes"):
        call(x, (None,) + w[1:])
    with pytest.raises(ValueError, match="codes"):
        call(x[:, :256].contiguous(), w)
    with pytest.raises(TypeError, match="codes must be"):
        call(x, (w[0].to(torch.int8),) + w[1:])
    with pytest.raises(ValueError, match="micro-scales"):
        call(x, (w[0], w[1][:5], w[2]))
    with pytest.raises(TypeError, match="block scales"):
        call(x, w[:2] + (w[2].double(),))
    with pytest.raises(ValueError, match="contiguous"):
        call(x, (w[0].t().contiguous().t(),) + w[1:])
    with pytest.raises(ValueError, match="flags"):
        call(x, w, flags=2)
    with pytest.raises(ValueError, match="out must"):
        call(x, w, out=torch.zeros(3, 5))
    with pytest.raises(TypeError, match="out_dtype"):
        call(x, w, out=torch.zeros(3, 6), out_dtype=BF16)
    with pytest.raises(TypeError, match="out must"):
        call(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        call(x, w)


def test_gated4_arguments():
    x = torch.zeros(3, 512, dtype=BF16)
    with pytest.raises(ValueError, match="activation"):
        fp4q.fp4q_gated4(x, payload(), payload(), None)
    with pytest.raises(ValueError, match="gate has 6 rows"):
        fp4q.fp4q_gated4(x, payload(), payload(7))


# ------------------------------------------------------- warnings, other GPUs
def bf(grad):
    return torch.zeros(4, 512, dtype=BF16, requires_grad=grad)


def graded(payload_, grad):
    return payload_[:2] + (payload_[2].requires_grad_(grad),)


CALLS = {
    "fp4q_gated8 scales": lambda g: fp4q.fp4q_gated8(operands()[0], operands()[1].requires_grad_(g), *operands()[2:]),
    "fp4q_gated8_backward up": lambda g: fp4q.fp4q_gated8_backward(bf(False), bf(False), bf(g)),
    "fp4q_gemv4 x": lambda g: fp4q.fp4q_gemv4(bf(g), payload()),
    "fp4q_gemv4 scales": lambda g: fp4q.fp4q_gemv4(bf(False), graded(payload(), g)),
    "fp4q_gated4 x": lambda g: fp4q.fp4q_gated4(bf(g), payload(), payload()),
    "fp4q_gated4 up": lambda g: fp4q.fp4q_gated4(bf(False), payload(), graded(payload(), g)),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_gradient_that_ends_here_is_said(name):
    with pytest.warns(UserWarning, match="autograd does not record %s:" % name.split()[0]):
        with pytest.raises(ValueError, match="GPU"):
            CALLS[name](True)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="GPU"):
            CALLS[name](False)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            CALLS[name](True)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("tensors", [0, 1])
def test_the_tensors_gpu_is_current_for_the_launch(name, tensors, monkeypatch):
    state = {"current": 0, "launched": []}

    class device:
        def __init__(self, which):
            self.which = which

        def __enter__(self):
            self.before, state["current"] = state["current"], self.which

        def __exit__(self, *_):
            state["current"] = self.before

    class Library:
        def __getattr__(self, entry):
            return lambda *args: state["launched"].append((entry, state["current"])) or 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(gated, "_bound", Library())
    monkeypatch.setattr(gated, "_gpu", lambda *t: tensors)
    monkeypatch.setattr(gated, "_current_gpu", lambda: state["current"])
    monkeypatch.setattr(gated, "_launch_stream", lambda stream, index: index)
    monkeypatch.setattr(linear, "_workspace", lambda *s: 64)
    CALLS[name](False)
    assert state["launched"] == [(name.split()[0], tensors)] and state["current"] == 0


# --------------------------------------------------------------------- C ABI
# Fake device addresses: only where no GPU is visible, as a kernel would then fault on them.
fake_addresses = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake device addresses: CPU-only host")
G = 1 << 30   # buffers 1 GiB apart
OK, NULL, SHAPE, ALIGN, ARG = (fp4q.FP4Q_OK, fp4q.FP4Q_ERR_NULL, fp4q.FP4Q_ERR_SHAPE, fp4q.FP4Q_ERR_ALIGN,
                               fp4q.FP4Q_ERR_ARG)


def gated8(a=G, a_pitch=256, fa=0, sa=2 * G, w=3 * G, w_pitch=256, fw=0, sw=4 * G, m=4, n=300, k=256, act=0, y=5 * G,
           gate=6 * G, up=7 * G, space=8 * G, size=1 << 30):
    return gated._lib().fp4q_gated8(a, a_pitch, fa, sa, w, w_pitch, fw, sw, m, n, k, act, y, gate, up, space, size, None)


@fake_addresses
@pytest.mark.parametrize("change,want", [
    ({"m": -1}, SHAPE), ({"n": -1}, SHAPE), ({"k": -1}, SHAPE), ({"m": 1 << 27}, SHAPE), ({"n": 1 << 27}, SHAPE),
    ({"k": 1 << 27}, SHAPE), ({"a_pitch": 240}, SHAPE), ({"w_pitch": 1 << 23}, SHAPE), ({"act": -1}, ARG), ({"act": 4}, ARG),
    ({"fa": 2}, ARG), ({"fw": -1}, ARG), ({"m": 0, "a": None}, OK), ({"n": 0, "w": None}, OK), ({"a": None}, NULL),
    ({"w": None}, NULL), ({"sa": None}, NULL), ({"sw": None}, NULL), ({"y": None}, NULL), ({"gate": None}, NULL),
    ({"up": None}, NULL), ({"m": 100, "n": 100, "k": 2000, "a_pitch": 2000, "w_pitch": 2000, "space": None}, NULL),
    ({"m": 100, "n": 100, "k": 2000, "a_pitch": 2000, "w_pitch": 2000, "size": 100}, SHAPE),
    ({"a": G + 8}, ALIGN), ({"w_pitch": 264}, ALIGN), ({"y": 5 * G + 8}, ALIGN), ({"up": 7 * G + 2}, ALIGN),
    ({"sa": 2 * G + 2}, ALIGN), ({"space": 8 * G + 4}, ALIGN), ({"y": 3 * G}, ARG), ({"gate": 5 * G + 2384}, ARG),
    ({"up": 6 * G}, ARG), ({"y": 3 * G + 683 * 256}, ARG), ({"gate": 4 * G + 16}, ARG)])
def test_gated8_refuses(change, want):
    assert gated8(**change) == want


def grad(dy=G, gate=2 * G, up=3 * G, rows=4, cols=200, dtype=1, act=0, fmt=1, codes=4 * G, pitch=464, scales=5 * G,
         codes_t=6 * G, pitch_t=16, scales_t=7 * G, y=8 * G, y_pitch=16, y_scales=9 * G):
    return gated._lib().fp4q_gated8_backward(dy, gate, up, rows, cols, dtype, act, fmt, codes, pitch, scales, codes_t, pitch_t,
                                             scales_t, y, y_pitch, y_scales, None)


@fake_addresses
@pytest.mark.parametrize("change,want", [
    ({"rows": -1}, SHAPE), ({"cols": 0}, SHAPE), ({"cols": 1 << 23}, SHAPE), ({"rows": 1 << 23}, SHAPE), ({"pitch": 448}, SHAPE),
    ({"pitch": 1 << 25}, SHAPE), ({"pitch_t": 1 << 25}, SHAPE), ({"y_pitch": 1 << 25}, SHAPE),
    ({"pitch_t": 0}, SHAPE), ({"y_pitch": 0}, SHAPE), ({"dtype": 2}, ARG), ({"act": 4}, ARG), ({"fmt": 2}, ARG),
    ({"rows": 0, "dy": None}, OK), ({"dy": None}, NULL), ({"gate": None}, NULL), ({"up": None}, NULL), ({"scales": None}, NULL),
    ({"scales_t": None}, NULL), ({"y_scales": None}, NULL),
    ({"codes": None, "scales": None, "codes_t": None, "scales_t": None, "y": None, "y_scales": None}, NULL),
    ({"codes": None}, ARG), ({"codes_t": None}, ARG), ({"y": None}, ARG), ({"dy": G + 2}, ALIGN), ({"pitch": 472}, ALIGN),
    ({"pitch_t": 24}, ALIGN), ({"y_pitch": 40}, ALIGN), ({"codes_t": 6 * G + 8}, ALIGN), ({"y_scales": 9 * G + 1}, ALIGN),
    ({"codes": G}, ARG), ({"codes_t": 4 * G + 448}, ARG), ({"y": 6 * G + 16 * 455}, ARG), ({"y_scales": 5 * G}, ARG),
    ({"scales_t": 3 * G + 16}, ARG)])
def test_gated8_backward_refuses(change, want):
    assert grad(**change) == want


def gemv4(x=G, dtype=1, m=3, codes=2 * G, micro=3 * G, block=4 * G, n=6, k=512, out=5 * G, out_dtype=1, flags=0, space=6 * G,
          size=1 << 30):
    return gated._lib().fp4q_gemv4(x, dtype, m, codes, micro, block, n, k, out, out_dtype, flags, space, size, None)


def gated4(x=G, dtype=1, m=3, codes=2 * G, micro=3 * G, block=4 * G, n=6, k=512, out=5 * G, out_dtype=1, flags=0, space=6 * G,
           size=1 << 30, act=0, up_codes=7 * G, up_micro=8 * G, up_block=9 * G):
    return gated._lib().fp4q_gated4(x, dtype, m, codes, micro, block, up_codes, up_micro, up_block, n, k, act, out, out_dtype,
                                    flags, space, size, None)


BOTH = [({"m": -1}, SHAPE), ({"n": -1}, SHAPE), ({"k": 0}, SHAPE), ({"k": 300}, SHAPE), ({"k": 1 << 24}, SHAPE),
        ({"m": 1 << 19}, SHAPE), ({"n": 1 << 27}, SHAPE), ({"flags": 2}, ARG), ({"dtype": 2}, ARG), ({"out_dtype": -1}, ARG),
        ({"m": 0, "x": None}, OK), ({"n": 0, "codes": None}, OK), ({"x": None}, NULL), ({"codes": None}, NULL),
        ({"micro": None}, NULL), ({"block": None}, NULL), ({"out": None}, NULL), ({"m": 100, "space": None}, NULL),
        ({"m": 100, "size": 1000}, SHAPE), ({"x": G + 8}, ALIGN), ({"codes": 2 * G + 8}, ALIGN), ({"micro": 3 * G + 4}, ALIGN),
        ({"block": 4 * G + 2}, ALIGN), ({"out": 5 * G + 8}, ALIGN), ({"space": 6 * G + 8}, ALIGN), ({"out": 2 * G + 1520}, ARG),
        ({"out": 3 * G}, ARG), ({"out": 4 * G}, ARG), ({"out": G}, ARG), ({"m": 100, "space": G}, ARG),
        ({"m": 100, "space": 5 * G}, ARG)]


@fake_addresses
@pytest.mark.parametrize("change,want", BOTH)
def test_gemv4_refuses(change, want):
    assert gemv4(**change) == want


@fake_addresses
@pytest.mark.parametrize("change,want", BOTH + [
    ({"act": 4}, ARG), ({"up_codes": None}, NULL), ({"up_micro": None}, NULL), ({"up_block": None}, NULL),
    ({"up_codes": 7 * G + 8}, ALIGN), ({"up_micro": 8 * G + 8}, ALIGN), ({"up_block": 9 * G + 1}, ALIGN),
    ({"out": 7 * G}, ARG), ({"out": 9 * G}, ARG)])
def test_gated4_refuses(change, want):
    assert gated4(**change) == want


def test_workspace_sizes():
    L, size = gated._lib(), ctypes.c_size_t()
    assert L.fp4q_gated8_workspace(-1, 4, 4, ctypes.byref(size)) == SHAPE
    assert L.fp4q_gated8_workspace(4, 4, 4, None) == NULL
    assert L.fp4q_gated8_workspace(0, 4, 4, ctypes.byref(size)) == OK and size.value == 0
    assert L.fp4q_gated8_workspace(1 << 26, 1 << 26, 1, ctypes.byref(size)) == SHAPE
    assert L.fp4q_gemv4_workspace(4, 300, 1, 0, ctypes.byref(size)) == SHAPE
    assert L.fp4q_gemv4_workspace(4, 512, 2, 0, ctypes.byref(size)) == ARG
    assert L.fp4q_gemv4_workspace(4, 512, 1, 2, ctypes.byref(size)) == ARG
    assert L.fp4q_gemv4_workspace(4, 512, 1, 0, None) == NULL
    assert L.fp4q_gemv4_workspace(1, 4096, 1, 1, ctypes.byref(size)) == OK and size.value == 0
    # x in two parts and a factor for each block of 256
    assert L.fp4q_gemv4_workspace(100, 512, 0, 1, ctypes.byref(size)) == OK and size.value == 100 * 2 * (1024 + 8)
