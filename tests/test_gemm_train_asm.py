"""The static checks of test_gemm_asm.py on the kernels of gemm_train.hip: no
hazard around the MFMAs issued as asm, no spilled register."""
import os
import subprocess

import pytest

import test_gemm_asm as T

SRC = os.path.join(T.ROOT, "gemm_epilogue_bf16_amd", "csrc", "gemm_train.hip")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    from gemm_epilogue_bf16_amd import build as B

    try:
        cc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("asm") / "gemm_train.s")
    r = subprocess.run([cc, *B.common_flags(), *B.EXTRA_FLAGS["gemm_train.hip"], "-x", "hip", "--cuda-device-only", "-S", SRC,
                        "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return T._kernels(open(out).read())


def test_no_mfma_hazard(kernels):
    assert len(kernels) >= 30
    problems = [f"{k.name[:90]}: {h}" for k in kernels for h in T._hazards(k)]
    assert not problems, "\n".join(problems[:20])


def test_nothing_spilled(kernels):
    for k in kernels:
        assert not any(kind == "I" and "scratch_" in t for kind, t in k.ins), k.name
