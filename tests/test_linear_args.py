"""The 8-bit linear-layer operators refuse what they cannot take, without a GPU: the
binding's checks of tensors, and the C entry points' checks before any HIP call."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

import fp4_communication_compression_amd as fp4q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3, E5M2, BF16, F32 = torch.float8_e4m3fn, torch.float8_e5m2, torch.bfloat16, torch.float32


def status(status):
    return pytest.raises(fp4q.Fp4qError, match=r"\(status %d\)" % status)


def test_header_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp4q_linear.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fp4q_[a-z0-9_]+)\s*\(", text)))
    assert names == ["fp4q_gemm8", "fp4q_gemm8_workspace", "fp4q_quantize8", "fp4q_rmsnorm",
                     "fp4q_rmsnorm_backward", "fp4q_rmsnorm_backward_workspace"]
    for n in names:
        assert hasattr(fp4q.lib(), n), n
    from fp4_communication_compression_amd import linear
    for name, value in (("FP4Q_GROUP8", 128), ("FP4Q_E4M3", 0), ("FP4Q_E5M2", 1), ("FP4Q_FLAG_TILES", 2),
                        ("FP4Q_FLAG_ACCUMULATE", 4)):
        assert getattr(fp4q, name) == getattr(linear, name) == value
    with pytest.raises(AttributeError):
        fp4q.fp4q_no_such_thing


# ------------------------------------------------------------------- binding
def test_rmsnorm_arguments():
    x, w = torch.zeros(4, 256, dtype=BF16), torch.ones(256, dtype=BF16)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        fp4q.fp4q_rmsnorm(x.half(), w.half(), 1e-6)
    with pytest.raises(TypeError, match="torch tensor"):
        fp4q.fp4q_rmsnorm([[1.0]], w, 1e-6)
    with pytest.raises(ValueError, match="2-D"):
        fp4q.fp4q_rmsnorm(x[0], w, 1e-6)
    with pytest.raises(ValueError, match="contiguous"):
        fp4q.fp4q_rmsnorm(x.t(), w, 1e-6)
    with pytest.raises(TypeError, match="weight"):
        fp4q.fp4q_rmsnorm(x, w.float(), 1e-6)
    with pytest.raises(ValueError, match="weight"):
        fp4q.fp4q_rmsnorm(x, w[:255], 1e-6)
    with pytest.raises(ValueError, match="residual"):
        fp4q.fp4q_rmsnorm(x, w, 1e-6, residual=x[:3])
    with pytest.raises(ValueError, match="h is an output"):
        fp4q.fp4q_rmsnorm(x, w, 1e-6, h=x)
    with pytest.raises(ValueError, match="h must"):
        fp4q.fp4q_rmsnorm(x, w, 1e-6, residual=x, h=x[:2])
    with pytest.raises(ValueError, match="ask for"):
        fp4q.fp4q_rmsnorm(x, w, 1e-6, want_y=False)
    with status(fp4q.FP4Q_ERR_SHAPE):
        fp4q.fp4q_rmsnorm(x[:, :0].contiguous(), w[:0], 1e-6)
    with pytest.raises(ValueError, match="GPU"):
        fp4q.fp4q_rmsnorm(x, w, 1e-6)


def test_rmsnorm_backward_arguments():
    x, w, r = torch.zeros(4, 256, dtype=BF16), torch.ones(256, dtype=BF16), torch.ones(4)
    with pytest.raises(TypeError, match="h must"):
        fp4q.fp4q_rmsnorm_backward(x, x.float(), w, r)
    with pytest.raises(ValueError, match="rstd"):
        fp4q.fp4q_rmsnorm_backward(x, x, w, r[:3])
    with pytest.raises(TypeError, match="rstd"):
        fp4q.fp4q_rmsnorm_backward(x, x, w, r.to(BF16))
    with pytest.raises(ValueError, match="dh"):
        fp4q.fp4q_rmsnorm_backward(x, x, w, r, dh=x[:1])
    with pytest.raises(ValueError, match="GPU"):
        fp4q.fp4q_rmsnorm_backward(x, x, w, r, dh=x)


def test_quantize_arguments():
    x = torch.zeros(4, 256, dtype=BF16)
    with pytest.raises(TypeError, match="float8"):
        fp4q.fp4q_quantize8(x, torch.uint8)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        fp4q.fp4q_quantize8(x.half())
    with pytest.raises(ValueError, match="ask for"):
        fp4q.fp4q_quantize8(x, straight=False)
    with pytest.raises(ValueError, match="contiguous"):
        fp4q.fp4q_quantize8(x[:, ::2])
    with pytest.raises(ValueError, match="GPU"):
        fp4q.fp4q_quantize8(x)


def test_gemm_arguments():
    a, b = torch.zeros(4, 256, dtype=E4M3), torch.zeros(300, 256, dtype=E4M3)
    sa, sb, st = torch.ones(2, 4), torch.ones(2, 300), torch.ones(2, 3)
    with pytest.raises(TypeError, match="float8"):
        fp4q.fp4q_gemm8(a.view(torch.uint8), sa, b, sb)
    with pytest.raises(ValueError, match="columns"):
        fp4q.fp4q_gemm8(a, sa, b[:, :128], sb)
    with pytest.raises(ValueError, match="a's scales"):
        fp4q.fp4q_gemm8(a, sa.t().contiguous(), b, sb)
    with pytest.raises(ValueError, match="b's scales"):
        fp4q.fp4q_gemm8(a, sa, b, torch.ones(2, 4))
    with pytest.raises(TypeError, match="b's scales"):
        fp4q.fp4q_gemm8(a, sa, b, st.double())
    with pytest.raises(ValueError, match="multiples of 16"):
        fp4q.fp4q_gemm8(torch.zeros(4, 250, dtype=E4M3), sa, torch.zeros(300, 250, dtype=E4M3), sb)
    with pytest.raises(ValueError, match="multiples of 16"):
        fp4q.fp4q_gemm8(a[:1].expand(4, 256), sa, b, sb)
    with pytest.raises(ValueError, match="contiguous"):
        fp4q.fp4q_gemm8(torch.zeros(256, 4, dtype=E4M3).t(), sa, b, sb)
    with pytest.raises(ValueError, match="readable"):   # the last row ends inside its last 16 bytes
        room = torch.zeros(3 * 256 + 250, dtype=torch.uint8).view(E4M3)
        fp4q.fp4q_gemm8(room.as_strided((4, 250), (256, 1)), sa, b[:, :250], sb)
    with pytest.raises(ValueError, match="out must"):
        fp4q.fp4q_gemm8(a, sa, b, sb, out=torch.zeros(4, 299))
    with pytest.raises(TypeError, match="out_dtype"):
        fp4q.fp4q_gemm8(a, sa, b, sb, out=torch.zeros(4, 300), out_dtype=BF16)
    with pytest.raises(TypeError, match="out must"):
        fp4q.fp4q_gemm8(a, sa, b, sb, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="out must be float32"):
        fp4q.fp4q_gemm8(a, sa, b, sb, out=torch.zeros(4, 300, dtype=BF16), accumulate=True)
    with pytest.raises(ValueError, match="needs out"):
        fp4q.fp4q_gemm8(a, sa, b, sb, accumulate=True)
    for scales in (sb, st):
        with pytest.raises(ValueError, match="GPU"):
            fp4q.fp4q_gemm8(a, sa, b, scales)


# --------------------------------------------------------------------- C ABI
# Fake device addresses: only where no GPU is visible, as a kernel would then fault on them.
def _gpu_visible():
    return torch.cuda.device_count() > 0


fake_addresses = pytest.mark.skipif(_gpu_visible(), reason="fake device addresses: CPU-only host")
G = 1 << 30   # buffers 1 GiB apart
OK, NULL, SHAPE, ALIGN, ARG = (fp4q.FP4Q_OK, fp4q.FP4Q_ERR_NULL, fp4q.FP4Q_ERR_SHAPE, fp4q.FP4Q_ERR_ALIGN,
                               fp4q.FP4Q_ERR_ARG)


def library():
    from fp4_communication_compression_amd import linear
    return linear._lib()


def norm(x=G, residual=2 * G, weight=3 * G, eps=1e-6, rows=4, cols=256, dtype=1, h=4 * G, y=5 * G, codes=6 * G,
         pitch=256, scales=7 * G, rstd=8 * G):
    return library().fp4q_rmsnorm(x, residual, weight, eps, rows, cols, dtype, h, y, codes, pitch, scales, rstd, None)


@fake_addresses
@pytest.mark.parametrize("change,want", [
    ({"rows": -1}, SHAPE), ({"cols": 0}, SHAPE), ({"cols": 1 << 28}, SHAPE), ({"rows": 1 << 28}, SHAPE),
    ({"pitch": 255}, SHAPE), ({"dtype": 2}, ARG), ({"eps": 0.0}, ARG), ({"eps": -1.0}, ARG),
    ({"eps": float("nan")}, ARG), ({"eps": float("inf")}, ARG), ({"rows": 0, "x": None}, OK),
    ({"x": None}, NULL), ({"weight": None}, NULL), ({"h": None}, NULL), ({"y": None, "codes": None}, NULL),
    ({"scales": None}, NULL), ({"residual": None}, ARG), ({"codes": None}, ARG), ({"x": G + 8}, ALIGN),
    ({"y": 5 * G + 2}, ALIGN), ({"pitch": 264}, ALIGN), ({"scales": 7 * G + 2}, ALIGN), ({"rstd": 8 * G + 1}, ALIGN),
    ({"y": G}, ARG), ({"h": G}, ARG), ({"h": 2 * G + 16}, ARG), ({"codes": 5 * G + 512}, ARG),
    ({"rstd": 3 * G + 16}, ARG)])
def test_rmsnorm_refuses(change, want):
    assert norm(**change) == want


def norm_grad(dy=G, h=2 * G, weight=3 * G, rstd=4 * G, dh=5 * G, rows=4, cols=256, dtype=1, dx=6 * G, dw=7 * G,
              space=8 * G, size=1 << 20):
    return library().fp4q_rmsnorm_backward(dy, h, weight, rstd, dh, rows, cols, dtype, dx, dw, space, size, None)


@fake_addresses
@pytest.mark.parametrize("change,want", [
    ({"rows": -1}, SHAPE), ({"cols": 0}, SHAPE), ({"dtype": -1}, ARG), ({"dy": None}, NULL), ({"h": None}, NULL),
    ({"weight": None}, NULL), ({"rstd": None}, NULL), ({"dx": None}, NULL), ({"dw": None}, NULL),
    ({"rows": 0, "dw": None}, NULL), ({"space": None}, NULL), ({"size": 256 * 4 - 1}, SHAPE),
    ({"dx": 6 * G + 4}, ALIGN), ({"dw": 7 * G + 2}, ALIGN), ({"space": 8 * G + 8}, ALIGN), ({"dx": G}, ARG),
    ({"dx": 5 * G}, ARG), ({"dw": 3 * G}, ARG), ({"space": 6 * G + 64}, ARG)])
def test_rmsnorm_backward_refuses(change, want):
    assert norm_grad(**change) == want


def quant(x=G, rows=4, cols=256, dtype=1, fmt=0, codes=2 * G, pitch=256, scales=3 * G, codes_t=4 * G, pitch_t=16,
          scales_t=5 * G, flags=0):
    return library().fp4q_quantize8(x, rows, cols, dtype, fmt, codes, pitch, scales, codes_t, pitch_t, scales_t,
                                    flags, None)


@fake_addresses
@pytest.mark.parametrize("change,want", [
    ({"rows": -1}, SHAPE), ({"cols": 0}, SHAPE), ({"pitch": 240}, SHAPE), ({"pitch_t": 0}, SHAPE),
    ({"flags": 1}, ARG), ({"flags": 4}, ARG), ({"dtype": 3}, ARG), ({"fmt": 2}, ARG), ({"rows": 0, "x": None}, OK),
    ({"x": None}, NULL), ({"codes": None, "scales": None, "codes_t": None, "scales_t": None}, NULL),
    ({"scales": None}, NULL), ({"scales_t": None}, NULL), ({"codes": None}, ARG), ({"codes_t": None}, ARG),
    ({"x": G + 2}, ALIGN), ({"pitch": 260}, ALIGN), ({"pitch_t": 24}, ALIGN), ({"codes_t": 4 * G + 8}, ALIGN),
    ({"scales": 3 * G + 1}, ALIGN), ({"codes": G}, ARG), ({"codes_t": 2 * G + 512}, ARG),
    ({"scales_t": 3 * G}, ARG)])
def test_quantize_refuses(change, want):
    assert quant(**change) == want


def gemm(a=G, a_pitch=256, fa=0, sa=2 * G, b=3 * G, b_pitch=256, fb=0, sb=4 * G, m=4, n=300, k=256, out=5 * G,
         dtype=1, flags=0, space=6 * G, size=1 << 30):
    return library().fp4q_gemm8(a, a_pitch, fa, sa, b, b_pitch, fb, sb, m, n, k, out, dtype, flags, space, size, None)


@fake_addresses
@pytest.mark.parametrize("change,want", [
    ({"m": -1}, SHAPE), ({"n": -1}, SHAPE), ({"k": -1}, SHAPE), ({"m": 1 << 28}, SHAPE), ({"a_pitch": 240}, SHAPE),
    ({"b_pitch": 1 << 23}, SHAPE), ({"flags": 1}, ARG), ({"flags": 8}, ARG), ({"dtype": 2}, ARG),
    ({"flags": 4}, ARG), ({"fa": 2}, ARG), ({"fb": -1}, ARG), ({"m": 0, "a": None}, OK), ({"n": 0, "b": None}, OK),
    ({"a": None}, NULL), ({"b": None}, NULL), ({"sa": None}, NULL), ({"sb": None}, NULL), ({"out": None}, NULL),
    ({"a": G + 8}, ALIGN), ({"b_pitch": 264}, ALIGN), ({"out": 5 * G + 8}, ALIGN), ({"sa": 2 * G + 2}, ALIGN),
    ({"space": 6 * G + 4}, ALIGN), ({"out": 3 * G}, ARG), ({"out": 4 * G + 16}, ARG), ({"out": G - 16}, ARG)])
def test_gemm_refuses(change, want):
    assert gemm(**change) == want


@fake_addresses
def test_launches_past_32_bits_are_refused():
    """More threads than a launch can count, found before any HIP call."""
    far = 1 << 50
    assert norm(x=far, residual=None, h=None, weight=2 * far, y=3 * far, codes=None, scales=None, rstd=None,
                rows=1 << 27, cols=20000) == SHAPE
    assert gemm(a=far, sa=2 * far, b=3 * far, sb=4 * far, out=5 * far, m=1, n=(1 << 28) - 1, k=128, a_pitch=128,
                b_pitch=128, space=None, size=0) == SHAPE


def test_workspace_sizes():
    L, size = library(), ctypes.c_size_t()
    assert L.fp4q_rmsnorm_backward_workspace(4, 0, ctypes.byref(size)) == SHAPE
    assert L.fp4q_rmsnorm_backward_workspace(4, 8, None) == NULL
    assert L.fp4q_rmsnorm_backward_workspace(0, 8, ctypes.byref(size)) == OK and size.value == 0
    assert L.fp4q_gemm8_workspace(4, 4, 4, 1, 8, ctypes.byref(size)) == ARG
    assert L.fp4q_gemm8_workspace(4, 4, 4, 2, 0, ctypes.byref(size)) == ARG
    assert L.fp4q_gemm8_workspace(4, 4, 4, 1, 4, ctypes.byref(size)) == ARG
    assert L.fp4q_gemm8_workspace(-1, 4, 4, 1, 0, ctypes.byref(size)) == SHAPE
    assert L.fp4q_gemm8_workspace(4, 4, 4, 1, 0, None) == NULL
    assert L.fp4q_gemm8_workspace(0, 4, 4, 1, 0, ctypes.byref(size)) == OK and size.value == 0
    assert L.fp4q_gemm8_workspace(1 << 27, 1 << 27, 1, 1, 0, ctypes.byref(size)) == SHAPE
