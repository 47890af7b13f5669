"""Products of 8-bit tensors whose wait for their sums runs out: the device
error word says so. The library's products are compiled once more with that
wait's limit at nothing; all other waits keep theirs, and so every kernel ends
by itself with its copies and products done."""

import ctypes
import os
import subprocess

import pytest
import torch

import hashed_gram_embedding_gb300 as ple
from hashed_gram_embedding_gb300 import _lib, build
from oracle import eight_bit as oracle

from _helpers import dev_err_word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("mx8") / "impatient.so")
    sources = [os.path.join(build.CSRC, f) for f in ("proj_mx8.cu", "common.cu")]
    run = subprocess.run([build._nvcc(), *build.ARCH, *build.CFLAGS, "-DPLE_SUMS_WAIT_NS=0", "-shared", *sources, "-o", so],
                         capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]
    lib = ctypes.CDLL(so)
    for name in ("ple_gated_mx8", "ple_proj_mx8"):
        getattr(lib, name).argtypes = _lib.SIGNATURES[name]
    return lib


def zeros(rows, columns):
    return (torch.zeros((rows, columns), dtype=torch.uint8, device="cuda"),
            torch.zeros((oracle.scale_bytes(rows, columns),), dtype=torch.uint8, device="cuda"))


# milliseconds of products, of few tokens and of many
@pytest.mark.parametrize("gated,t,columns", [(False, 1, 1 << 26), (False, 100, 1 << 24), (True, 1, 1 << 25), (True, 129, 1 << 23)])
def test_sums_that_do_not_come(impatient, gated, t, columns, monkeypatch):
    rows = 128
    x8, w8 = zeros(t, columns), zeros(rows * 2 if gated else rows, columns)

    def call():
        err = dev_err_word()
        if gated:
            codes, scales = zeros(t, rows)
            ple.ple_gated_mx8(*x8, *w8, codes, scales, dev_err=err)
            return int(err.item()), codes
        out = torch.ones((t, rows), dtype=torch.bfloat16, device="cuda")
        ple.ple_proj_mx8(*x8, *w8, out, dev_err=err)
        return int(err.item()), out

    err, out = call()
    assert err == 0 and (out == 0).all()
    with monkeypatch.context() as m:
        m.setattr(_lib, "_lib", impatient)
        assert call()[0] == ple.PLE_DEVERR_TIMEOUT
    err, out = call()  # as if nothing had been
    assert err == 0 and (out == 0).all()
