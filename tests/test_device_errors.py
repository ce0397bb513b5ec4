"""Errors found on the device after a call has returned reach a caller that gave no error
word: the entry point's refusals (CPU), a wait that runs out and the check that raises
(GPU)."""
import os
import subprocess

import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from vocabulary_lm_cross_gb300 import build, capi

HERE = os.path.dirname(os.path.abspath(__file__))


def test_refusals():
    build.build()
    lib = capi.lib()
    assert lib.vlmce_take_device_errors(None, None) == capi.ERR_INVALID_ARG
    assert lib.vlmce_take_device_errors((1 << 20) + 2, None) == capi.ERR_MISALIGNED


@pytest.mark.gpu
def test_a_wait_that_gives_up_is_reported_without_a_word_of_the_callers(tmp_path):
    lib = build.build()
    libdir, exe = os.path.dirname(lib), str(tmp_path / "wait_gives_up")
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-O2", "-I", build.CSRC,
                    "-I", build.INCLUDE, os.path.join(HERE, "wait_gives_up.cu"), "-o", exe,
                    "-L", libdir, "-Xlinker", f"-rpath={libdir}", "-lvlmce"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "wait ok" in r.stdout, r.stdout + r.stderr


@pytest.mark.gpu
def test_check_after_layers(monkeypatch):
    x = torch.ones((16, 64), device="cuda").bfloat16()
    z = v.glu_fwd(x, x, preact=True).preact
    v.glu_bwd(x[:, :8].contiguous(), x, x, z)
    v.linear_fwd(x, x)
    v.check_device_errors()
    assert v.take_device_errors("cuda:0") == 0

    # what a wait that gave up leaves
    monkeypatch.setattr("vocabulary_lm_cross_gb300.errors.take_device_errors",
                        lambda device=None: capi.DEVERR_TIMEOUT)
    with pytest.raises(RuntimeError, match="gave up"):
        v.check_device_errors()
