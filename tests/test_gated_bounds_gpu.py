"""The gated operators write what they say and nothing else, and calls do not meet: memory around
the outputs, a padded batch, calls on two streams at once, the same tensor given twice."""
import pytest

torch = pytest.importorskip("torch")

from tests import gated_shapes
from tests import linear_ref as ref
from tests.test_gated_gpu import ACTS, BF16, DEV, E5M2, F32, grad_inputs, operands, rows, weight
from tests.test_linear_gpu import fp4q  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu
MARK = 0x5A


def room(count, dtype):
    """`count` elements of marked bytes, with 256 bytes more on either side, and the whole."""
    size = torch.empty((), dtype=dtype).element_size()
    whole = torch.full((512 + count * size,), MARK, dtype=torch.uint8, device=DEV)
    return whole[256:256 + count * size].view(dtype), whole


def untouched(whole):
    return bool((whole[:256] == MARK).all()) and bool((whole[-256:] == MARK).all())


@pytest.mark.parametrize("shape", [s[:3] for s in gated_shapes.SHAPES] + [(1, 1, 1), (17, 5, 17), (129, 127, 15), (3, 333, 129)])
def test_gated8_leaves_the_rest(fp4q, shape):
    """Through the C ABI, at the outputs' own sizes: the bytes before and behind y, gate, up and
    the workspace stay."""
    from fp4_communication_compression_amd import gated, linear
    print(shape, flush=True)
    m, n, k = shape
    a, sa, w, sw = operands(*shape)
    want = fp4q.fp4q_gated8(a, sa, w, sw, "gelu", want_pre=True)
    need = linear._workspace("fp4q_gated8_workspace", m, n, k)
    outs = [room(m * n, BF16) for _ in range(3)]
    space, around = room(need, torch.uint8)
    status = gated._lib().fp4q_gated8(
        a.data_ptr(), a.stride(0) if m > 1 else (k + 15) // 16 * 16, linear._FORMATS[a.dtype], sa.data_ptr(),
        w.data_ptr(), w.stride(0), linear._FORMATS[w.dtype], sw.data_ptr(), m, n, k, fp4q.FP4Q_ACT_GELU,
        *(t.data_ptr() for t, _ in outs), space.data_ptr() if need else None, need,
        torch.cuda.current_stream().cuda_stream)
    assert status == 0
    for (t, whole), b in zip(outs, (want.y, want.gate, want.up)):
        assert torch.equal(t.view(m, n), b) and untouched(whole)
    assert untouched(around)


@pytest.mark.parametrize("shape", [(1, 1), (5, 7), (129, 127), (128, 256), (333, 203), (16, 1000), (127, 129)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward_leaves_the_rest(fp4q, shape, dtype):
    """Through the C ABI, with pitches wider than the rows: the columns past a row's end, and the
    bytes before and behind, stay."""
    from fp4_communication_compression_amd import gated, linear
    print(shape, dtype, flush=True)
    m, n = shape
    dy, gate, u = (t.to(DEV) for t in grad_inputs(shape, dtype)[:3])
    r = ref.groups(n) * 128 + n
    want = fp4q.fp4q_gated8_backward(dy, gate, u, "silu", E5M2, want_y=True)
    pitch = {c: (c + 15) // 16 * 16 + 32 for c in (r, m)}
    codes = [room((rows_ - 1) * pitch[cols] + cols, torch.uint8) + (rows_, cols) for rows_, cols in ((m, r), (r, m), (n, m))]
    scales = [room(t.numel(), F32) for t in (want.scales, want.scales_t, want.y_scales_t)]
    args = []
    for (c, _, _, cols), (s, _) in zip(codes, scales):
        args += [c.data_ptr(), pitch[cols], s.data_ptr()]
    status = gated._lib().fp4q_gated8_backward(dy.data_ptr(), gate.data_ptr(), u.data_ptr(), m, n,
                                               linear._TYPES[dtype], fp4q.FP4Q_ACT_SILU, linear._FORMATS[E5M2], *args,
                                               torch.cuda.current_stream().cuda_stream)
    assert status == 0
    for (c, whole, rows_, cols), b in zip(codes, (want.codes, want.codes_t, want.y_codes_t)):
        got = torch.as_strided(c, (rows_, cols), (pitch[cols], 1))
        assert torch.equal(got, b.view(torch.uint8)) and untouched(whole)
        if rows_ > 1:
            assert bool((torch.as_strided(c, (rows_ - 1, pitch[cols] - cols), (pitch[cols], 1), c.storage_offset() + cols) == MARK).all())
    for (s, whole), b in zip(scales, (want.scales, want.scales_t, want.y_scales_t)):
        assert torch.equal(s.view(b.shape), b) and untouched(whole)


@pytest.mark.parametrize("m,n,k", [(1, 1, 256), (1, 333, 11008), (3, 257, 512), (9, 5003, 1024), (17, 100, 4096), (40, 48, 4352)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("plain", [True, False])
def test_few_rows_of_a_padded_batch(fp4q, m, n, k, dtype, plain):
    """The first rows of a longer batch, whose others are NaN, into the first rows of a longer out."""
    print(m, n, k, dtype, plain, flush=True)
    flags = fp4q.FP4Q_FLAG_NO_FWHT if plain else 0
    w, v = weight(fp4q, n, k, flags), weight(fp4q, n, k, flags, 1)
    x = rows(m, k, dtype).to(DEV)
    batch = torch.full((m + 20, k), float("nan"), dtype=dtype, device=DEV)
    batch[:m] = x
    for call in (lambda x, **kw: fp4q.fp4q_gemv4(x, w, flags, **kw),
                 lambda x, **kw: fp4q.fp4q_gated4(x, w, v, "gelu", flags, **kw)):
        out, whole = room((m + 20) * n, dtype)
        got = call(batch[:m], out=out.view(m + 20, n)[:m])
        assert torch.equal(got, call(x)) and bool(torch.isfinite(got).all())
        size = x.element_size()
        assert bool((whole[256 + m * n * size:] == MARK).all()) and untouched(whole)


@pytest.mark.parametrize("tokens", [1, 24])
def test_two_streams_at_once(fp4q, tokens):
    """Two requests' calls, under way on two streams at the same time, with work in front of both
    so that they are issued together; each has its own workspace."""
    flags, n, k = 0, 1500, 4096
    w, v = weight(fp4q, n, k, flags), weight(fp4q, n, k, flags, 1)
    ops = [operands(tokens * 40, 300, 4096, seed=i) for i in range(2)]
    xs = [rows(tokens, k, BF16, i).to(DEV) for i in range(2)]
    grads = [[t.to(DEV) for t in grad_inputs((tokens * 40, 300), BF16, i)[:3]] for i in range(2)]

    def run(i, stream=None):
        h = fp4q.fp4q_gated8(*ops[i], "silu", stream=stream).y
        g = fp4q.fp4q_gated8_backward(*grads[i], stream=stream, want_y=True)
        return [h, *(t.view(torch.uint8) for t in g), fp4q.fp4q_gemv4(xs[i], w, flags, stream=stream),
                fp4q.fp4q_gated4(xs[i], w, v, flags=flags, stream=stream)]

    def same(got, want):
        return all(torch.equal(a, b) for a, b in zip(got, want))

    want = [run(i) for i in range(2)]
    sides = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(3):
        torch.cuda._sleep(2000000)
        for s in sides:
            s.wait_stream(torch.cuda.current_stream())
        got = [run(i, s) for i, s in enumerate(sides)] + [run(i, s) for i, s in enumerate(reversed(sides))]
        torch.cuda.synchronize()
        assert all(same(g, want[i % 2]) for i, g in enumerate(got)), turn


@pytest.mark.parametrize("act", ACTS)
def test_the_same_tensor_twice(fp4q, act):
    """dy, gate and up as one tensor, and one payload for the gate and the up projection."""
    t = grad_inputs((130, 300), BF16)[1].to(DEV)
    got = fp4q.fp4q_gated8_backward(t, t, t, act, want_y=True)
    want = fp4q.fp4q_gated8_backward(t, t.clone(), t.clone(), act, want_y=True)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    w = weight(fp4q, 100, 512, 0)
    x = rows(2, 512, F32).to(DEV)
    assert torch.equal(fp4q.fp4q_gated4(x, w, w, act), fp4q.fp4q_gated4(x, w, tuple(p.clone() for p in w), act))


def test_two_graphs_at_once(fp4q):
    """Two graphs with workspaces of their own, captured one after the other and replayed on two
    streams at the same time."""
    flags = fp4q.FP4Q_FLAG_NO_FWHT
    w = weight(fp4q, 700, 4096, flags)
    xs = [rows(24, 4096, BF16, i).to(DEV) for i in range(2)]
    ops = [operands(300, 200, 4096, seed=i) for i in range(2)]
    run = lambda i: [fp4q.fp4q_gemv4(xs[i], w, flags), fp4q.fp4q_gated8(*ops[i]).y]  # noqa: E731
    want = [run(i) for i in range(2)]
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    torch.cuda.synchronize()
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            held.append(run(i))
    sides = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(4):
        for out in held:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for h, v in zip(held, want) for a, b in zip(h, v)), turn
        run(turn % 2)
