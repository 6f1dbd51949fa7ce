"""C ABI checks of the grouped products that need no GPU: every entry point the header
declares is exported, and invalid arguments get their status before anything is launched."""
import os
import re
import subprocess

import pytest

import int4_weight_only_gptq_amd as qg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qgemm_grouped.h")
OK, NULL, SHAPE, ALIGN, DTYPE, LAYOUT, UNSUP = 0, 1, 2, 3, 4, 5, 6
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


def grouped(lib, layout=0, dtype=0, groups=4, off=A16, M=32, N=16, K=64, A=A16, lda=64, B=A16, ldb=64, sb=1024,
            C=A16, ldc=16, sc=0):
    return lib.gemm_grouped(layout, dtype, groups, off, M, N, K, A, lda, B, ldb, sb, C, ldc, sc, None)


@pytest.mark.parametrize("kw,code", [
    (dict(layout=3), LAYOUT), (dict(layout=-1), LAYOUT), (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE),
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-1), SHAPE), (dict(groups=-1), SHAPE),
    (dict(groups=4097), SHAPE), (dict(M=1 << 31), SHAPE), (dict(N=1 << 31, ldc=1 << 31), SHAPE),
    (dict(sb=-1), SHAPE), (dict(sc=-1), SHAPE),
    (dict(off=0), NULL), (dict(A=0), NULL), (dict(B=0), NULL), (dict(C=0), NULL),
    (dict(lda=63), SHAPE), (dict(ldb=63), SHAPE), (dict(ldc=15), SHAPE),
    (dict(layout=1, ldb=15), SHAPE), (dict(layout=2, lda=31), SHAPE), (dict(layout=2, lda=32, ldb=15), SHAPE),
    (dict(layout=2, lda=32, ldb=16, sc=511), SHAPE),         # the groups' outputs overlap
    (dict(A=A16 + 1), ALIGN), (dict(B=A16 + 1), ALIGN), (dict(C=A16 + 1), ALIGN), (dict(off=A16 + 2), ALIGN),
    (dict(dtype=2, A=A16 + 2), ALIGN), (dict(dtype=2, C=A16 + 2), ALIGN),
    (dict(M=1 << 30, N=1 << 30, ldc=1 << 30), SHAPE),        # more tiles than a grid holds
    # nothing to do
    (dict(M=0, off=0, A=0, B=0, C=0), OK), (dict(N=0, off=0, A=0, B=0, C=0), OK),
    (dict(groups=0, off=0, A=0, B=0, C=0), OK),
])
def test_grouped_rejects_invalid_arguments(lib, kw, code):
    assert grouped(lib, **kw) == code


def int4(lib, x=A16, ldx=256, qw=A16, sc=A16, qz=A16, experts=4, off=A16, y=A16, ldy=64, m=8, n=64, k=256, gs=128,
         ws=None, wsb=0):
    return lib.qgemm_int4_grouped(x, ldx, qw, sc, qz, experts, off, y, ldy, m, n, k, gs, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), SHAPE), (dict(n=-8), SHAPE), (dict(k=-128), SHAPE), (dict(experts=-1), SHAPE),
    (dict(experts=4097), SHAPE), (dict(k=200), SHAPE), (dict(n=60), SHAPE), (dict(gs=64), UNSUP),
    (dict(x=0), NULL), (dict(qw=0), NULL), (dict(sc=0), NULL), (dict(y=0), NULL), (dict(off=0), NULL),
    (dict(ldx=128), SHAPE), (dict(ldy=32), SHAPE), (dict(x=A16 + 2), ALIGN), (dict(qw=A16 + 4), ALIGN),
    (dict(sc=A16 + 2), ALIGN), (dict(qz=A16 + 2), ALIGN), (dict(y=A16 + 2), ALIGN), (dict(off=A16 + 2), ALIGN),
    (dict(ws=A16 + 8, wsb=64), ALIGN), (dict(wsb=-1), SHAPE),
    (dict(m=1 << 30, n=1 << 26, ldy=1 << 26, k=1 << 20, ldx=1 << 20), SHAPE),      # more than a grid holds
    (dict(m=0, x=0, qw=0, sc=0, qz=0, y=0, off=0), OK), (dict(experts=0), OK), (dict(n=0, ldy=0), OK),
])
def test_int4_grouped_rejects_invalid_arguments(lib, kw, code):
    assert int4(lib, **kw) == code


def test_int4_grouped_workspace_size(lib):
    f = lib.qgemm_int4_grouped_workspace_size
    assert f(64, 64, 1024, 2048) == 0                                         # strips use none
    assert f(8, 4096, 14336, 4096) == 4096 * 4096 * 2 + 32 * 4096 * 4         # activations and their sums
    assert f(0, 8, 64, 256) == 0 and f(4, 0, 64, 256) == 0
    assert f(4, 8, 60, 256) == -SHAPE and f(4, 8, 64, 100) == -SHAPE and f(-1, 8, 64, 256) == -SHAPE
