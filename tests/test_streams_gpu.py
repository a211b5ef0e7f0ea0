"""Calls on a stream that is not the current one (``stream=``): their outputs may not lie in memory
on which the current stream's work is not done, and the memory of tensors dropped after a call may
not be handed out before that call has run."""
import pytest
import torch

from ff_util import matrix

pytestmark = pytest.mark.gpu

M, N, K = 512, 1024, 256
T = torch.bfloat16
SLEEP = 40_000_000  # clock cycles: about 20 ms


def setup(h):
    x, w, wu = matrix(M, K, T, 1), matrix(K, N, T, 2, "col"), matrix(K, N, T, 3, "col")
    dy, z, u = (matrix(M, N, T, s) for s in (4, 5, 6))
    rows = matrix(M, N, T, 7)
    _, mean, rstd = h.layer_norm(rows, save=True)
    return {
        "matmul": ((x, w), lambda x, w, **k: [h.matmul(x, w, **k)]),
        "softmax_rows": ((rows,), lambda r, **k: [h.softmax_rows(r, **k)]),
        "matmul_epilogue": ((x, w, dy), lambda x, w, r, **k: h.matmul_epilogue(
            x, w, activation="silu", residual=r, save=True, **k)),
        "matmul_epilogue_backward": ((dy, x, w, z), lambda dy, x, w, z, **k: (
            h.matmul_epilogue_backward(dy, x, w, pre=z, activation="silu", **k))),
        "gated": ((x, w, wu), lambda x, w, wu, **k: h.gated(x, w, wu, save=True, **k)),
        "gated_backward": ((dy, x, w, wu, z, u), lambda *a, **k: h.gated_backward(*a, **k)),
        "layer_norm": ((rows,), lambda r, **k: h.layer_norm(r, save=True, **k)),
        "layer_norm_backward": ((dy, rows, mean, rstd), lambda dy, r, m, s, **k: (
            h.layer_norm_backward(dy, r, None, m, s, **k))),
    }


NAMES = ["matmul", "softmax_rows", "matmul_epilogue", "matmul_epilogue_backward", "gated",
         "gated_backward", "layer_norm", "layer_norm_backward"]


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    hh = g.Gemm(0)
    yield hh
    assert hh.status() == 0
    hh.close()


@pytest.mark.parametrize("name", NAMES)
def test_outputs_off_the_current_streams_pending_work(h, name):
    inputs, call = setup(h)[name]
    want = [t.clone() for t in call(*inputs)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        # memory of the outputs' sizes, still to be written by the current stream when it is dropped
        dropped = [torch.empty_like(t) for t in want for _ in range(4)]
        torch.cuda._sleep(SLEEP)
        for t in dropped:
            t.fill_(7.0)
        del dropped, t
        got = call(*inputs, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_tensors_dropped_before_the_call_has_run(h, name):
    inputs, call = setup(h)[name]
    want = [t.clone() for t in call(*inputs)]
    s = torch.cuda.Stream()
    for _ in range(3):
        copies = [t.clone(memory_format=torch.preserve_format) for t in inputs]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(SLEEP)
        got = call(*copies, stream=s)
        del copies
        new = [torch.full_like(t, 7.0) for t in inputs for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        del new


@pytest.mark.parametrize("name", NAMES)
def test_external_and_current_streams(h, name):
    inputs, call = setup(h)[name]
    want = [t.clone() for t in call(*inputs)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (torch.cuda.ExternalStream(s.cuda_stream), torch.cuda.current_stream(),
                   torch.cuda.default_stream()):
        got = call(*inputs, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    with torch.cuda.stream(s):
        got = call(*inputs, stream=torch.cuda.default_stream())
        assert torch.cuda.current_stream() == s
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
