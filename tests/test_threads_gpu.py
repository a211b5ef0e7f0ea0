"""One handle, one stream and one host thread each, at the same time: the C entries called without
the interpreter's lock (ctypes releases it), from a cold start of what the library keeps for the
whole process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import ctypes, threading
import torch
import dense_tiled_gemm_05_gb300 as g

L = g.lib()
gen = torch.Generator("cuda").manual_seed(1)
rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
SIZES = [(1, 512, 1024), (17, 264, 1024), (64, 1024, 2048), (300, 520, 264), (40, 200, 4096)]
data = [(rnd(M, K), rnd(N, K), rnd(M, N)) for M, N, K in SIZES]
torch.cuda.synchronize()
THREADS = 4
start = threading.Barrier(THREADS)
results, errors = [None] * THREADS, []

def work(t):
    h, s = g.Gemm(0), torch.cuda.Stream()
    outs = [torch.empty_like(r) for _, _, r in data]
    start.wait()
    for _ in range(20):
        for (M, N, K), (x, w, r), y in zip(SIZES, data, outs):
            ep = g.Epilogue()
            ep.residual, ep.ld_residual, ep.activation = r.data_ptr(), N, 4
            code = L.gemm_run_epilogue(h.handle, M, N, K, x.data_ptr(), K, w.data_ptr(), K,
                                       y.data_ptr(), N, 2, 2, 0, 0, 1, ctypes.byref(ep),
                                       ctypes.c_void_p(s.cuda_stream))
            if code:
                errors.append(code)
    s.synchronize()
    if h.status(s):
        errors.append("status")
    results[t] = outs
    h.close()

threads = [threading.Thread(target=work, args=(t,)) for t in range(THREADS)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
h = g.Gemm(0)
for i, (x, w, r) in enumerate(data):
    want = h.matmul_epilogue(x, w.t(), residual=r, activation="silu")
    for t in range(THREADS):
        assert torch.equal(results[t][i], want), (t, i)
print("same")
"""


def test_four_threads_from_a_cold_start():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.strip().endswith("same")
