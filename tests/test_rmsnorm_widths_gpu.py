"""Norms of rows of different widths that share a kernel: called from two host threads at
once, and captured in one graph.  A launch's size must not depend on what another call
has asked of the same function."""
import os
import shutil
import subprocess
import threading

import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from vocabulary_lm_cross_gb300 import build

pytestmark = pytest.mark.gpu

# (T, H) pairs on the kernels that keep rows in flight (their shared memory grows with H)
PAIRS = [((2000, 8192), (2000, 4096)), ((2500, 8189), (2500, 4101)), ((6000, 512), (6000, 1024))]


def setup(T, H, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    x, r, w, dy = randn(T, H), randn(T, H), randn(H), randn(T, H)

    def call():
        a = v.rmsnorm_fwd(x, w, r)
        q = v.rmsnorm_fwd(x, w, r, fp8=True)
        b = v.rmsnorm_bwd(dy, a.residual, w, a.rstd)
        return a.y, a.residual, a.rstd, q.y.view(torch.uint8), q.scale, b.dx, b.dweight

    return call


def equal(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_threads_of_a_c_program_are_never_refused(tmp_path):
    lib = build.build()
    libdir, here = os.path.dirname(lib), os.path.dirname(os.path.abspath(__file__))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    exe = str(tmp_path / "c_norm_threads")
    subprocess.run([shutil.which("gcc") or shutil.which("cc"), "-O2", "-std=gnu11",
                    os.path.join(here, "c_norm_threads.c"), "-o", exe,
                    "-I", os.path.join(os.path.dirname(here), "include"),
                    "-I", os.path.join(cuda, "include"),
                    "-L", libdir, f"-Wl,-rpath,{libdir}", "-lvlmce",
                    "-L", os.path.join(cuda, "lib64"), f"-Wl,-rpath,{os.path.join(cuda, 'lib64')}",
                    "-lcudart", "-lpthread"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("pair", PAIRS)
def test_two_threads_norm_rows_of_different_widths(pair):
    calls = [setup(T, H, i) for i, (T, H) in enumerate(pair)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    start, problems = threading.Barrier(2), []

    def run(i):
        try:
            s = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(s):
                for n in range(100):
                    got = calls[i]()
                    if n % 50 == 49:
                        s.synchronize()
                        if not equal(got, want[i]):
                            problems.append((i, n, "differs"))
        except Exception as e:  # noqa: BLE001
            problems.append((i, repr(e)))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not problems, problems


@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
@pytest.mark.parametrize("pair", PAIRS)
def test_one_graph_norms_rows_of_different_widths(pair, order):
    calls = [setup(*pair[i], i) for i in order]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [c() for c in calls]
    calls[1]()  # eager calls between capture and replay
    graph.replay()
    calls[0]()
    graph.replay()
    torch.cuda.synchronize()
    assert all(equal(a, b) for a, b in zip(got, want))
