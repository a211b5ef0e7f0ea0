"""Captured calls that use a handle's buffers, replayed after larger calls on the same handle have
outgrown them: the buffers a graph holds are kept. Also first calls of a handle inside a capture."""
import pytest
import torch

from ff_util import TYPES, matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    return g


def weights(K, N, t, seed, pad=0):
    return matrix(K, N, t, seed, "col", pad, scale=K ** -0.5)


def epilogue_backward(h, n, dtype="bf16"):
    t = TYPES[dtype]
    x, w = matrix(n, 136, t, 1), weights(136, 264, t, 2)
    dy, z = matrix(n, 264, t, 3), matrix(n, 264, t, 4)
    return [x, dy, z], lambda: h.matmul_epilogue_backward(dy, x, w, pre=z, activation="silu")


def gated_backward(h, n, dtype="bf16"):
    t = TYPES[dtype]
    x, wg, wu = matrix(n, 136, t, 1), weights(136, 264, t, 2), weights(136, 264, t, 3)
    dh, gate, up = [matrix(n, 264, t, s) for s in (4, 5, 6)]
    return [x, dh, gate, up], lambda: h.gated_backward(dh, x, wg, wu, gate, up)


def norm_backward(h, n, N=1000, grad=torch.bfloat16):
    x, dy = matrix(n, N, torch.bfloat16, 1), matrix(n, N, grad, 2)
    w = matrix(1, N, torch.float32, 3)[0]
    mean, rstd = matrix(1, n, torch.float32, 4)[0], matrix(1, n, torch.float32, 5)[0].abs()
    return [x, dy], lambda: h.layer_norm_backward(dy, x, w, mean, rstd)


def unfused_epilogue(h, n):
    x, w = matrix(n, 200, torch.float32, 1), weights(200, 520, torch.float32, 2)
    return [x], lambda: [h.matmul_epilogue(x, w, activation="gelu", precision="tf32", out_dtype="bf16")]


def unfused_gated(h, n):
    x, wg, wu = [matrix(n, 200, torch.float32, 1)] + [weights(200, 520, torch.float32, s) for s in (2, 3)]
    return [x], lambda: [h.gated(x, wg, wu, precision="tf32")]


def staged_epilogue(h, n):
    x, w = matrix(n, 133, torch.bfloat16, 1, pad=2), weights(133, 264, torch.bfloat16, 2, pad=2)
    return [x], lambda: [h.matmul_epilogue(x, w, activation="silu")]


def split_epilogue(h, n):  # (n: columns) K split over CTA pairs
    h.set_option("cta_pair", 2)
    h.set_option("stream_k", 2)
    x, w = matrix(300, 1024, torch.bfloat16, 1), weights(1024, n, torch.bfloat16, 2)
    return [x], lambda: [h.matmul_epilogue(x, w, activation="silu")]


def split_product(h, n):  # 128-wide tiles, whose partials the 256-wide ones outgrow
    h.set_option("cta_pair", 2)
    h.set_option("stream_k", 2)
    h.set_option("block_n", 128 if n < 1000 else 256)
    x, w = matrix(300, 1024, torch.bfloat16, 1), weights(1024, n, torch.bfloat16, 2)
    return [x], lambda: [h.matmul(x, w)]


def exact_product(h, n):
    x, w = matrix(n, 600, torch.float32, 1), weights(600, 300, torch.float32, 2)
    return [x], lambda: [h.matmul(x, w)]


def strided_product(h, n):
    x, w = matrix(n, 400, torch.bfloat16, 1), matrix(400, 300, torch.bfloat16, 2)
    return [x], lambda: [h.matmul(x[:, ::2], w[::2, ::3])]


CALLS = {
    "epilogue_backward": (epilogue_backward, 300, 5000),
    "epilogue_backward_f32": (lambda h, n: epilogue_backward(h, n, "f32"), 300, 5000),
    "gated_backward": (gated_backward, 300, 5000),
    "gated_backward_f32": (lambda h, n: gated_backward(h, n, "f32"), 300, 5000),
    "norm_backward": (norm_backward, 70, 70000),
    "norm_backward_other_type": (lambda h, n: norm_backward(h, n, 1000, torch.float32), 70, 20000),
    "norm_backward_long_rows": (lambda h, n: norm_backward(h, n, 9000), 70, 2000),
    "unfused_epilogue": (unfused_epilogue, 300, 5000),
    "unfused_gated": (unfused_gated, 300, 5000),
    "staged_epilogue": (staged_epilogue, 300, 5000),
    "split_epilogue": (split_epilogue, 264, 1032),
    "split_product": (split_product, 264, 1032),
    "exact_product": (exact_product, 300, 5000),
    "strided_product": (strided_product, 300, 5000),
}


@pytest.mark.parametrize("cold", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_replays_after_a_larger_call(g, name, cold):
    make, small, large = CALLS[name]
    other = g.Gemm(0)  # loads the kernels, and gives the values to compare with
    _, eager = make(other, small)
    eager()
    h = g.Gemm(0)
    inputs, call = make(h, small)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    if not cold:
        with torch.cuda.stream(s):
            call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = call()
    for seed in (50, 60):
        make(h, large)[1]()  # outgrows the captured call's buffer
        if name == "split_product":
            make(h, small)  # (the options back)
        torch.cuda.synchronize()
        poison = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]
        theirs, eager = make(other, small)
        for i, (x, y) in enumerate(zip(inputs, theirs)):
            x.copy_(matrix(*x.shape, x.dtype, seed + i))
            y.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, eager()):
            assert torch.isfinite(q).all() and torch.equal(p, q)
        # calls and replays take turns on the buffers
        for p, q in zip(call(), eager()):
            assert torch.equal(p, q)
        del poison
    assert h.status() == 0 and other.status() == 0
    del graph
    h.close()
    other.close()


def test_many_captures_of_growing_calls(g):
    """Every graph keeps its own buffer."""
    h, other = g.Gemm(0), g.Gemm(0)
    s = torch.cuda.Stream()
    graphs = []
    norm_backward(other, 70)[1]()
    for n in (70, 500, 3000, 20000, 3000):
        inputs, call = norm_backward(h, n)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = call()
        graphs.append((n, graph, got, inputs, call))  # (the inputs live as long as the graph)
    for n, graph, got, _, _ in graphs + graphs[::-1]:
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, norm_backward(other, n)[1]()):
            assert torch.equal(p, q)
    assert h.status() == 0
    del graphs, graph
    h.close()
    other.close()
