"""GPU parity of the products grouped by expert against plain products in fp64.

Tolerances.  bf16 / fp16: the fp32 sum of K products of 16-bit operands is off by at
most gamma_K * sum |a||b| with gamma_K = K u / (1 - K u), u = 2^-24 (any order of
summation; the products are exact in fp32), and the result rounds once, half a step:
eps / 2 relative to the value, plus half the smallest subnormal.  fp32 products round
too: gamma_{K + 1}.
"""
import numpy as np
import pytest

from gpu_helpers import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def tdtype(name):
    import torch

    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def offsets_of(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


def make(layout, dtype, counts, N, K, seed, first=0, behind=0, scale=0.125):
    """CPU operands: (a, b, offsets).  For TN, N and K are the two widths."""
    import torch

    g = torch.Generator().manual_seed(seed)
    rows, groups = first + int(sum(counts)) + behind, len(counts)

    def rnd(*shape):
        return (torch.randn(shape, generator=g) * scale).to(tdtype(dtype))

    off = torch.from_numpy(offsets_of(counts, first))
    if layout == "NT":
        return rnd(rows, K), rnd(groups, N, K), off
    if layout == "NN":
        return rnd(rows, K), rnd(groups, K, N), off
    return rnd(rows, N), rnd(rows, K), off


def reference(layout, a, b, off, absolute=False):
    """fp64 result, NaN in the rows of no group (TN: none)."""
    import torch

    a, b, off = a.double(), b.double(), off.tolist()
    if absolute:
        a, b = a.abs(), b.abs()
    if layout == "TN":
        return torch.stack([a[lo:max(lo, hi)].t() @ b[lo:max(lo, hi)] for lo, hi in zip(off, off[1:])])
    out = torch.full((a.shape[0], b.shape[1 if layout == "NT" else 2]), float("nan"), dtype=torch.float64)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            out[lo:hi] = a[lo:hi] @ (b[e].t() if layout == "NT" else b[e])
    return out


def longest(layout, a, off):
    """Length of the longest sum."""
    o = off.tolist()
    return max([hi - lo for lo, hi in zip(o, o[1:])] + [1]) if layout == "TN" else a.shape[1]


def assert_close(got, layout, dtype, a, b, off, what):
    import torch

    ref, mag = reference(layout, a, b, off), reference(layout, a, b, off, absolute=True)
    K = longest(layout, a, off) + (dtype == "fp32")
    gamma = K * U / (1 - K * U)
    fi = torch.finfo(tdtype(dtype))
    tol = gamma * mag
    if dtype != "fp32":
        tol = tol + (ref.abs() + tol) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2
    got = got.cpu().double()
    held = ~torch.isnan(ref)
    bad = held & ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4])


def run(qg, layout, a, b, off, **kw):
    import torch

    out = qg.gemm_grouped(layout, a.cuda(), b.cuda(), off.cuda(), **kw)
    torch.cuda.synchronize()
    return out


# rows a group: empty groups first, last and in between, one row, tiles that end inside,
# one group with everything
COUNTS = [[3], [0, 1, 0], [1, 0, 2, 0, 0, 5], [17, 0, 33, 1], [130, 64, 0, 7, 70], [0, 300, 0, 20], [0, 0]]
# (N, K): one element; unaligned; aligned to 8 with tails of every tile; whole tiles
SIZES = [(1, 1), (37, 45), (24, 8), (136, 200), (128, 64), (264, 328)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_small_shapes(gpu_lib, layout, dtype):
    for i, counts in enumerate(COUNTS):
        for j, (N, K) in enumerate(SIZES):
            say("grouped", layout, dtype, counts, N, K)
            a, b, off = make(layout, dtype, counts, N, K, seed=100 * i + j)
            assert_close(run(gpu_lib, layout, a, b, off), layout, dtype, a, b, off, (counts, N, K))


# averages that reach every kernel: strips of 16 rows, pipelined tiles of 64, 128 and 256
# rows; k with a tail and a k longer than the strips' waves
AVERAGES = [([1, 3, 0, 12], 5), ([20, 0, 47, 9], 1), ([64, 40, 0, 90], 1), ([100, 200, 1, 99], 1), ([500, 0, 129], 1),
            ([300, 700, 0, 1400], 1)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_every_kernel(gpu_lib, layout, dtype):
    for i, (counts, rep) in enumerate(AVERAGES):
        for N, K in ((512, 2312), (392, 1024)):
            say("grouped kernels", layout, dtype, counts, N, K)
            a, b, off = make(layout, dtype, counts * rep, N, K, seed=1000 + i)
            assert_close(run(gpu_lib, layout, a, b, off), layout, dtype, a, b, off, (counts, N, K))


@pytest.mark.parametrize("groups", [65, 200, 1000])
def test_many_groups(gpu_lib, groups):
    rng = np.random.default_rng(groups)
    counts = (rng.integers(0, 4, groups) * (rng.random(groups) < 0.7)).tolist()
    for layout, N, K in (("NT", 40, 64), ("NN", 40, 64), ("TN", 24, 16), ("NT", 33, 35)):
        say("groups", groups, layout, sum(counts))
        a, b, off = make(layout, "bf16", counts, N, K, seed=groups)
        assert_close(run(gpu_lib, layout, a, b, off), layout, "bf16", a, b, off, (groups, layout))


# more groups than a wave has lanes, in strips, in tiles of 64 and 256 rows and (TN) in tiles
# of 256 x 256 and 128 x 256; a workgroup takes several tiles
@pytest.mark.parametrize("layout,groups,most,N,K", [("NT", 70, 3, 384, 264), ("NN", 70, 3, 384, 264),
                                                    ("NT", 130, 200, 264, 72), ("NN", 130, 200, 264, 72),
                                                    ("NT", 67, 700, 512, 40), ("NN", 67, 700, 512, 40),
                                                    ("TN", 150, 90, 264, 136), ("TN", 70, 60, 512, 512),
                                                    ("TN", 100, 40, 128, 256)])
def test_many_groups_of_many_rows(gpu_lib, layout, groups, most, N, K):
    rng = np.random.default_rng(groups + most)
    counts = (rng.integers(0, most, groups) * (rng.random(groups) < 0.8)).tolist()
    for dtype in ("bf16", "fp16"):
        say("many", layout, groups, sum(counts), N, K, dtype)
        a, b, off = make(layout, dtype, counts, N, K, seed=groups)
        assert_close(run(gpu_lib, layout, a, b, off), layout, dtype, a, b, off, (layout, groups))


@pytest.mark.parametrize("layout", ["NT", "TN"])
@pytest.mark.parametrize("ld", [2 ** 21, 2 ** 21 + 8])
def test_rows_past_32_bits(gpu_lib, layout, ld):
    """Rows whose byte offsets pass 32 bits, at the widest leading dimension of the pipelined
    kernel and past it."""
    import torch

    counts, N, K = [700, 0, 340, 60], 72, 64
    a, b, off = make(layout, "bf16", counts, N, K, seed=21)
    wide = torch.empty((a.shape[0], ld), dtype=torch.bfloat16, device="cuda")
    wide[:, :a.shape[1]] = a.cuda()
    out = None
    if layout == "NT":
        out = torch.empty((a.shape[0], ld), dtype=torch.bfloat16, device="cuda")[:, 8:8 + N]
    got = gpu_lib.gemm_grouped(layout, wide[:, :a.shape[1]], b.cuda(), off.cuda(), out=out)
    torch.cuda.synchronize()
    assert_close(got, layout, "bf16", a, b, off, (layout, ld))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_overlapping_groups_end(gpu_lib, layout, dtype):
    """Offsets that go back and forth (groups that overlap) are not a product's, but the call
    ends and writes nothing outside the output; the next call is right."""
    import torch

    a, b, off = make(layout, dtype, [4] * 200, 72, 64, seed=25)
    shape = (200, 72, 64) if layout == "TN" else (800, 72)
    hold = torch.full((shape[0] + 64,) + shape[1:], 7.0, dtype=tdtype(dtype), device="cuda")
    wild = torch.tensor([0, 800] * 100 + [0], dtype=torch.int32)
    gpu_lib.gemm_grouped(layout, a.cuda(), b.cuda(), wild.cuda(), out=hold[32:-32])
    torch.cuda.synchronize()
    assert torch.all(hold[:32] == 7.0) and torch.all(hold[-32:] == 7.0)
    assert_close(run(gpu_lib, layout, a, b, off), layout, dtype, a, b, off, (layout, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["NT", "NN"])
@pytest.mark.parametrize("counts", [[2, 0, 3], [90, 0, 40]])
def test_rows_of_no_group_stay(gpu_lib, layout, dtype, counts):
    import torch

    N, K, first, behind = 72, 64, 5, 9
    a, b, off = make(layout, dtype, counts, N, K, seed=7, first=first, behind=behind)
    a[:first], a[first + sum(counts):] = float("nan"), float("inf")     # never read
    out = torch.full((a.shape[0], N), 3.0, dtype=tdtype(dtype), device="cuda")
    got = run(gpu_lib, layout, a, b, off, out=out)
    assert got.data_ptr() == out.data_ptr()
    assert torch.all(out[:first] == 3.0) and torch.all(out[first + sum(counts):] == 3.0)
    assert_close(out, layout, dtype, a, b, off, (layout, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_other_groups_do_not_leak(gpu_lib, layout, dtype):
    """A group's result is its own rows' and matrix's: infinities and NaN elsewhere do not reach it."""
    import torch

    for counts in ([5, 3, 8], [100, 61, 150]):
        a, b, off = make(layout, dtype, counts, 64, 72, seed=11)
        lo, hi = int(off[1]), int(off[2])
        clean = run(gpu_lib, layout, a, b, off)
        a2, b2 = a.clone(), b.clone()
        a2[:lo], a2[hi:] = float("nan"), float("inf")
        if layout == "TN":
            b2[:lo], b2[hi:] = float("inf"), float("nan")
        else:
            b2[0], b2[2] = float("nan"), float("inf")
        dirty = run(gpu_lib, layout, a2, b2, off)
        mine = slice(1, 2) if layout == "TN" else slice(lo, hi)
        assert torch.equal(clean[mine], dirty[mine]), (layout, dtype, counts)


@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_strided_operands(gpu_lib, layout):
    """Views with padded rows, a stride between the matrices, unaligned starts, and an
    output view: nothing outside the view is written."""
    import torch

    for dtype, pad, start in (("bf16", 8, 0), ("bf16", 3, 1), ("fp32", 4, 0), ("fp32", 1, 3)):
        counts = [4, 0, 70, 33]
        a, b, off = make(layout, dtype, counts, 48, 56, seed=13)
        wide_a = torch.full((a.shape[0], a.shape[1] + pad + start), float("nan"), dtype=a.dtype)
        wide_a[:, start:start + a.shape[1]] = a
        wide_b = torch.full(tuple(b.shape[:-2]) + (b.shape[-2] + 2, b.shape[-1] + pad + start), float("nan"),
                            dtype=b.dtype)
        wide_b[..., :b.shape[-2], start:start + b.shape[-1]] = b
        va = wide_a.cuda()[:, start:start + a.shape[1]]
        vb = wide_b.cuda()[..., :b.shape[-2], start:start + b.shape[-1]]
        shape = (len(counts), 48, 56) if layout == "TN" else (a.shape[0], 48)
        hold = torch.full(shape[:-2] + (shape[-2] + 1, shape[-1] + pad + start), 7.0, dtype=a.dtype, device="cuda")
        out = hold[..., :shape[-2], start:start + shape[-1]]
        gpu_lib.gemm_grouped(layout, va, vb, off.cuda(), out=out)
        torch.cuda.synchronize()
        assert_close(out, layout, dtype, a, b, off, (layout, dtype, pad, start))
        hold[..., :shape[-2], start:start + shape[-1]] = 7.0
        assert torch.all(hold == 7.0), (layout, dtype, pad, start)


def test_one_matrix_for_every_group(gpu_lib):
    import torch

    a, b, off = make("NT", "bf16", [3, 9, 0, 4], 64, 64, seed=17)
    b = b[:1].cuda().expand(4, -1, -1)                                   # stride 0 between the groups
    got = gpu_lib.gemm_grouped("NT", a.cuda(), b, off.cuda())
    torch.cuda.synchronize()
    assert_close(got, "NT", "bf16", a, b.cpu(), off, "shared")


@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_empty_calls(gpu_lib, layout):
    """No rows, a width of zero, k of zero (zeros in the groups' rows, the others untouched)."""
    import torch

    for counts in ([0, 0, 0], [0]):
        a, b, off = make(layout, "bf16", counts, 24, 32, seed=19)
        got = run(gpu_lib, layout, a, b, off)
        assert torch.all(got == 0) and got.numel() == (len(counts) * 24 * 32 if layout == "TN" else 0)
    a, b, off = make(layout, "bf16", [2, 3], 0, 32, seed=19)
    assert run(gpu_lib, layout, a, b, off).numel() == 0
    if layout != "TN":
        a, b, off = make(layout, "fp16", [2, 3], 24, 0, seed=19, behind=2)
        out = torch.full((7, 24), 5.0, dtype=torch.float16, device="cuda")
        run(gpu_lib, layout, a, b, off, out=out)
        assert torch.all(out[:5] == 0) and torch.all(out[5:] == 5.0)


def test_offsets_are_held_to_the_rows(gpu_lib):
    """Offsets outside 0 .. rows and decreasing ones write nothing outside the output; groups
    whose offsets are in order hold their results."""
    import torch

    a, b, off = make("NT", "bf16", [4, 4, 4, 4], 64, 64, seed=23)
    for bad in ([-5, 4, 8, 12, 99], [0, 4, 2, 12, 16], [-2 ** 31, 4, 8, 12, 2 ** 31 - 1], [16, 0, 0, 0, 0]):
        say("offsets", bad)
        hold = torch.full((16 + 64, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        gpu_lib.gemm_grouped("NT", a.cuda(), b.cuda(), torch.tensor(bad, dtype=torch.int32).cuda(), out=hold[32:48])
        torch.cuda.synchronize()
        assert torch.all(hold[:32] == 7.0) and torch.all(hold[48:] == 7.0)
        o = [min(max(v, 0), 16) for v in bad]
        if o == sorted(o):
            assert_close(hold[32:48], "NT", "bf16", a, b, torch.tensor(o, dtype=torch.int32), bad)


@pytest.mark.parametrize("layout,counts", [("NT", [3, 1]), ("NT", [200, 70]), ("NN", [3, 1]), ("NN", [200, 70]),
                                           ("TN", [200, 70])])
def test_repeatable_and_captured(gpu_lib, layout, counts):
    """The same bits from call to call, on another stream, and from a captured graph whose
    offsets and operands change between its replays, with eager work between them."""
    import torch

    a, b, off = make(layout, "bf16", counts, 136, 192, seed=29)
    da, db, doff = a.cuda(), b.cuda(), off.cuda()
    first = run(gpu_lib, layout, a, b, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = gpu_lib.gemm_grouped(layout, da, db, doff, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.gemm_grouped(layout, da, db, doff, out=out)
    rng = np.random.default_rng(31)
    for i in range(4):
        rows = int(sum(counts))
        cut = int(rng.integers(0, rows + 1))
        o2 = torch.tensor([0, cut, rows], dtype=torch.int32)
        a2 = (a.float() * (i + 1)).to(a.dtype)
        da.copy_(a2)
        doff.copy_(o2)
        graph.replay()
        torch.cuda.synchronize()
        eager = gpu_lib.gemm_grouped(layout, da, db, doff)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), (layout, i, cut)
        assert_close(out, layout, "bf16", a2, b, o2, (layout, i, cut))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_gradients_against_differences(gpu_lib, dtype):
    """NN and TN are the gradients of NT: for L = sum(Y * G), the change of L along a direction
    D of the inputs equals <gradient, D>.  L is linear in X and in W apart, so a difference of
    any step is exact but for rounding: each Y is off by the product's tolerance, each gradient
    likewise, and L adds those over its terms."""
    import torch

    counts, N, K = [5, 0, 40, 12], 56, 64
    x, w, off = make("NT", dtype, counts, N, K, seed=37)
    g = make("TN", dtype, counts, N, K, seed=38)[0]
    y0 = run(gpu_lib, "NT", x, w, off).cpu().double()
    dx = run(gpu_lib, "NN", g, w, off).cpu().double()
    dw = run(gpu_lib, "TN", g, x, off).cpu().double()
    fi = torch.finfo(tdtype(dtype))

    def err(layout, a, b):                          # bound of one product's error, elementwise
        L = longest(layout, a, off) + 1
        sums = L * U / (1 - L * U) * reference(layout, a, b, off, absolute=True)
        return sums + (reference(layout, a, b, off).abs() + sums) * (fi.eps / 2) + fi.smallest_normal

    d = make("NT", dtype, counts, N, K, seed=39)
    for which in ("x", "w"):
        # operands x + d and x (w + d and w), exactly representable: the step is what they differ by
        x1, w1 = (x + d[0], w) if which == "x" else (x, w + d[1])
        step = (x1.double() - x.double()) if which == "x" else (w1.double() - w.double())
        y1 = run(gpu_lib, "NT", x1, w1, off).cpu().double()
        change = ((y1 - y0) * g.double()).sum()
        slope = (dx * step).sum() if which == "x" else (dw * step).sum()
        tol = ((err("NT", x1, w1) + err("NT", x, w)) * g.double().abs()).sum()
        tol = tol + ((err("NN", g, w) if which == "x" else err("TN", g, x)) * step.abs()).sum()
        say("gradient", dtype, which, float(change), float(slope), float(tol))
        assert abs(change - slope) <= tol
        assert tol < 0.05 * ((y1 - y0).abs() * g.double().abs()).sum()      # the bound says something


def test_refusals(gpu_lib):
    import torch

    a, b, off = make("NT", "bf16", [2, 3], 24, 32, seed=41)
    a, b, off = a.cuda(), b.cuda(), off.cuda()
    for bad in (off.long(), off[None], off[:2], off.cpu(), torch.zeros(10, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError):
            gpu_lib.gemm_grouped("NT", a, b, bad)
    with pytest.raises(TypeError):
        gpu_lib.gemm_grouped("NT", a, b.float(), off)
    with pytest.raises(ValueError):
        gpu_lib.gemm_grouped("NT", a[:, :16], b, off)
    with pytest.raises(ValueError):
        gpu_lib.gemm_grouped("NT", a.t().contiguous().t(), b, off)
    with pytest.raises(ValueError):
        gpu_lib.gemm_grouped("XX", a, b, off)
    with pytest.raises(ValueError):
        gpu_lib.gemm_grouped("NT", a, b, off, out=torch.empty((5, 23), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.gemm_grouped("NT", a.cpu(), b.cpu(), off.cpu())
    with pytest.raises(ValueError):
        gpu_lib.gemm_grouped("TN", a, a[:3], off)
