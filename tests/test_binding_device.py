"""A call whose tensors lie on a GPU that is not the current one makes it current for the
launch: a default stream has no GPU of its own and would start the kernel on the current one,
with another GPU's addresses.  CPU only: the GPUs, the library and the tensors' places are
stand-ins."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

import fp4_communication_compression_amd as fp4q
from fp4_communication_compression_amd import linear

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture
def gpus(monkeypatch):
    """Two GPUs, the first one current, all tensors on number `tensors`, and a library that
    notes the GPU that is current when it is called."""
    state = types.SimpleNamespace(current=0, tensors=0, launched=[], status=0)

    @contextlib.contextmanager
    def device(which):
        before, state.current = state.current, getattr(which, "index", which)
        try:
            yield
        finally:
            state.current = before

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                state.launched.append((name, state.current))
                return state.status
            return entry

    library = Library()
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state.current)
    monkeypatch.setattr(fp4q, "lib", lambda: library)
    monkeypatch.setattr(fp4q, "_stream", lambda stream, device: None)
    monkeypatch.setattr(fp4q, "_on_gpu", lambda *tensors: torch.device("cuda", state.tensors))
    monkeypatch.setattr(linear, "_bound", library)
    monkeypatch.setattr(linear, "_current_gpu", lambda: state.current, raising=False)
    monkeypatch.setattr(linear, "_gpu", lambda *tensors: state.tensors)
    monkeypatch.setattr(linear, "_launch_stream", lambda stream, index: None)
    monkeypatch.setattr(linear, "_workspace", lambda *sizes: 64)
    return state


def payload():
    return (torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1))


X = torch.zeros(4, 256, dtype=BF16)
W = torch.ones(256, dtype=BF16)
A, S = torch.zeros(4, 256, dtype=E4M3), torch.ones(2, 4)
CALLS = {
    "fp4q_compress": lambda: fp4q.fp4q_compress(X),
    "fp4q_decompress": lambda: fp4q.fp4q_decompress(*payload()),
    "fp4q_decompress_accumulate": lambda: fp4q.fp4q_decompress_accumulate([payload()]),
    "fp4q_reduce_requantize": lambda: fp4q.fp4q_reduce_requantize([payload()], local=X),
    "fp4q_compress_mx": lambda: fp4q.fp4q_compress_mx(X),
    "fp4q_decompress_mx": lambda: fp4q.fp4q_decompress_mx(torch.zeros(4, 128, dtype=torch.uint8),
                                                          torch.zeros(4, 8, dtype=torch.uint8)),
    "fp4q_rmsnorm": lambda: fp4q.fp4q_rmsnorm(X, W, 1e-6, residual=X, want_codes=True),
    "fp4q_rmsnorm_backward": lambda: fp4q.fp4q_rmsnorm_backward(X, X, W, torch.ones(4), dh=X),
    "fp4q_quantize8": lambda: fp4q.fp4q_quantize8(X, transposed=True),
    "fp4q_gemm8": lambda: fp4q.fp4q_gemm8(A, S, A, S, out_dtype=torch.float32),
}


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_gpu_is_current_for_the_launch(gpus, name, index):
    gpus.tensors = index
    CALLS[name]()
    assert len(gpus.launched) == 1 and gpus.launched[0][0].startswith(name)
    assert gpus.launched[0][1] == index and gpus.current == 0
    gpus.status = fp4q.FP4Q_ERR_SHAPE
    with pytest.MonkeyPatch.context() as m, pytest.raises(fp4q.Fp4qError):
        m.setattr(fp4q, "fp4q_status_str", str)
        CALLS[name]()
    assert gpus.launched[1][1] == index and gpus.current == 0
