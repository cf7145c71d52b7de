"""The 8-bit linear-layer functions say that autograd does not record them, where inputs that
require gradients meet them with gradients recorded, and nowhere else.  CPU only: the warning
comes before the tensors' place is looked at."""
import warnings

import pytest

torch = pytest.importorskip("torch")

import fp4_communication_compression_amd as fp4q

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def x(grad=False):
    return torch.zeros(4, 256, dtype=BF16, requires_grad=grad)


def w(grad=False):
    return torch.ones(256, dtype=BF16, requires_grad=grad)


def operand():
    return torch.zeros(4, 256, dtype=E4M3)


CALLS = {
    "fp4q_rmsnorm x": lambda g: fp4q.fp4q_rmsnorm(x(g), w(), 1e-6),
    "fp4q_rmsnorm weight": lambda g: fp4q.fp4q_rmsnorm(x(), w(g), 1e-6, residual=x()),
    "fp4q_rmsnorm residual": lambda g: fp4q.fp4q_rmsnorm(x(), w(), 1e-6, residual=x(g)),
    "fp4q_rmsnorm_backward dy": lambda g: fp4q.fp4q_rmsnorm_backward(x(g), x(), w(), torch.ones(4)),
    "fp4q_rmsnorm_backward dh": lambda g: fp4q.fp4q_rmsnorm_backward(x(), x(), w(), torch.ones(4), dh=x(g)),
    "fp4q_quantize8 x": lambda g: fp4q.fp4q_quantize8(x(g)),
    "fp4q_gemm8 scales": lambda g: fp4q.fp4q_gemm8(operand(), torch.ones(2, 4, requires_grad=g), operand(),
                                                   torch.ones(2, 4)),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_gradient_that_ends_here_is_said(name):
    call = CALLS[name]
    with pytest.warns(UserWarning, match="autograd does not record %s:" % name.split()[0]):
        with pytest.raises(ValueError, match="GPU"):
            call(True)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="GPU"):
            call(False)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            call(True)


def test_inside_an_autograd_function_nothing_is_said():
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight):
            return fp4q.fp4q_rmsnorm(x, weight, 1e-6).y

    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="GPU"):
            Norm.apply(x(True), w(True))
