"""C ABI checks of the MXFP4 entry points that need no GPU: every one the header declares is
exported, and invalid arguments get their status before anything is launched."""
import os
import re
import subprocess

import pytest

import int4_weight_only_gptq_amd as qg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qgemm_mxfp4.h")
OK, NULL, SHAPE, ALIGN, DTYPE = 0, 1, 2, 3, 4
A16 = 0x10000          # 16-byte aligned fake address: validation rejects the call before any use


@pytest.fixture(scope="module")
def lib():
    return qg.load()


def test_header_functions_are_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^(?:int32_t|int64_t)\s+(\w+)\s*\(", text, flags=re.M)
    out = subprocess.run(["nm", "-D", "--defined-only", qg.lib_path()], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\s[TW]\s(\w+)$", out, flags=re.M))
    assert names and set(names) <= exported
    for n in names:
        assert getattr(lib, n).argtypes is not None


CONVERT = [
    (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE), (dict(rows=-1), SHAPE), (dict(k=-32), SHAPE), (dict(k=48), SHAPE),
    (dict(x=0), NULL), (dict(codes=0), NULL), (dict(scales=0), NULL),
    (dict(ldx=63), SHAPE), (dict(ldc=16), SHAPE), (dict(lds=1), SHAPE),
    (dict(x=A16 + 1), ALIGN), (dict(dtype=2, x=A16 + 2), ALIGN), (dict(codes=A16 + 8), ALIGN), (dict(ldc=40), ALIGN),
    (dict(rows=1 << 31, k=32, ldx=32, ldc=16), SHAPE),
    (dict(ldc=(1 << 22) + 16), SHAPE), (dict(lds=(1 << 22) + 1), SHAPE),
    (dict(rows=0, x=0, codes=0, scales=0), OK), (dict(k=0, x=0, codes=0, scales=0), OK),
]


@pytest.mark.parametrize("kw,code", CONVERT)
def test_quantize_and_dequantize_reject_invalid_arguments(lib, kw, code):
    a = dict(dtype=0, rows=4, k=64, x=A16, ldx=64, codes=A16, ldc=32, scales=A16, lds=2)
    a.update(kw)
    assert lib.mxfp4_quantize(a["dtype"], a["rows"], a["k"], a["x"], a["ldx"], a["codes"], a["ldc"], a["scales"],
                              a["lds"], None) == code
    assert lib.mxfp4_dequantize(a["dtype"], a["rows"], a["k"], a["codes"], a["ldc"], a["scales"], a["lds"], a["x"],
                                a["ldx"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), DTYPE), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-32), SHAPE), (dict(K=80), SHAPE),
    (dict(M=1 << 31), SHAPE), (dict(a=0), NULL), (dict(sa=0), NULL), (dict(b=0), NULL), (dict(sb=0), NULL),
    (dict(c=0), NULL), (dict(lda=16), SHAPE), (dict(lsa=1), SHAPE), (dict(ldb=16), SHAPE), (dict(lsb=1), SHAPE),
    (dict(ldc=7), SHAPE), (dict(a=A16 + 8), ALIGN), (dict(ldb=40), ALIGN), (dict(c=A16 + 1), ALIGN),
    (dict(dtype=2, c=A16 + 2), ALIGN), (dict(M=1 << 30, N=1 << 30, ldc=1 << 30), SHAPE),
    (dict(lda=(1 << 22) + 16), SHAPE), (dict(ldb=(1 << 22) + 16), SHAPE),
    (dict(lsa=(1 << 22) + 1), SHAPE), (dict(lsb=(1 << 22) + 1), SHAPE),
    (dict(M=0, a=0, sa=0, b=0, sb=0, c=0), OK), (dict(N=0, a=0, sa=0, b=0, sb=0, c=0), OK),
])
def test_gemm_mxfp4_rejects_invalid_arguments(lib, kw, code):
    a = dict(dtype=0, M=4, N=8, K=64, a=A16, lda=32, sa=A16, lsa=2, b=A16, ldb=32, sb=A16, lsb=2, c=A16, ldc=8)
    a.update(kw)
    assert lib.gemm_mxfp4(a["dtype"], a["M"], a["N"], a["K"], a["a"], a["lda"], a["sa"], a["lsa"], a["b"], a["ldb"],
                          a["sb"], a["lsb"], a["c"], a["ldc"], None) == code
