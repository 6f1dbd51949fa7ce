"""GPU parity of the int4 products grouped by expert against plain products in fp64.

Tolerance.  Within a 128-row group of k the kernels sum x (128 + q) and x in fp32 and
take s (sum x (128 + q) - (128 + z) sum x); the groups' values are then added in fp32.
With u = 2^-24 and gamma_j = j u / (1 - j u), every term passes at most 128 additions in
its group, 3 roundings of the correction and the scale, and at most k / 128 + 8 additions
over groups and waves, so the sum is off by at most gamma_{k / 128 + 139} times
sum |x| s (256 + q + z); the result rounds once (half a step: eps / 2 relative to the value,
and half the smallest subnormal).
"""
import numpy as np
import pytest

from gpu_helpers import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def make(counts, n, k, seed, zeros=True, first=0, behind=0):
    import torch

    rng = np.random.default_rng(seed)
    e, rows = len(counts), first + int(sum(counts)) + behind
    words = lambda *shape: torch.from_numpy(rng.integers(0, 1 << 32, shape, dtype=np.uint32).view(np.int32))
    return {"x": torch.from_numpy(rng.standard_normal((rows, k)).astype(np.float32)).to(torch.bfloat16),
            "qweight": words(e, k // 8, n),
            "scales": torch.from_numpy(rng.uniform(0.002, 0.01, (e, k // 128, n)).astype(np.float16)),
            "qzeros": words(e, k // 128, n // 8) if zeros else None,
            "offsets": torch.from_numpy(np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32))}


def nibbles(words, axis):
    w = words.numpy().view(np.uint32)
    parts = np.stack([(w >> np.uint32(4 * t)) & np.uint32(15) for t in range(8)], axis=axis + 1)
    shape = list(w.shape)
    shape[axis] *= 8
    return parts.reshape(shape).astype(np.float64)


def reference(d):
    """(values, magnitudes) in fp64, NaN in the rows of no expert."""
    x = d["x"].double().numpy()
    n, k = d["qweight"].shape[2], x.shape[1]
    ref, mag = np.full((x.shape[0], n), np.nan), np.full((x.shape[0], n), np.nan)
    off = d["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi <= lo:
            continue
        q = nibbles(d["qweight"][e], 0)
        s = np.repeat(d["scales"][e].double().numpy(), 128, axis=0)
        z = np.zeros_like(q) if d["qzeros"] is None else np.repeat(nibbles(d["qzeros"][e], 1), 128, axis=0)
        ref[lo:hi] = x[lo:hi] @ ((q - z) * s)
        mag[lo:hi] = np.abs(x[lo:hi]) @ ((256 + q + z) * s)
    return ref, mag


def assert_close(got, d, what):
    ref, mag = reference(d)
    j = d["x"].shape[1] // 128 + 139
    tol = j * U / (1 - j * U) * mag
    tol = tol + (np.abs(ref) + tol) * 2.0 ** -8 + 2.0 ** -134
    got = got.cpu().double().numpy()
    held = ~np.isnan(ref)
    bad = held & ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4])


def run(qg, d, **kw):
    import torch

    c = lambda t: None if t is None else t.cuda()
    out = qg.qgemm_int4_grouped(c(d["x"]), c(d["qweight"]), c(d["scales"]), c(d["qzeros"]), c(d["offsets"]), **kw)
    torch.cuda.synchronize()
    return out


# strips of 16 and 32 rows, tiles of 64, 128 and 256 rows; empty experts, one row, tiles that
# end inside; one expert with everything
COUNTS = [[1], [0, 1, 0], [3, 0, 1, 17, 0], [20, 0, 47, 9], [64, 40, 0, 90], [100, 200, 1, 99], [500, 0, 129], [0, 300],
          [0, 0]]


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("n,k", [(8, 128), (200, 384), (1032, 2176)])
def test_matches_plain(gpu_lib, n, k, zeros):
    for i, counts in enumerate(COUNTS):
        for workspace in (None, False):
            say("int4 grouped", counts, n, k, zeros, workspace)
            d = make(counts, n, k, seed=10 * i + n, zeros=zeros)
            assert_close(run(gpu_lib, d, workspace=workspace), d, (counts, n, k, zeros, workspace))


def test_wide_strips(gpu_lib):
    # enough strips for 64 columns each, and for 32
    for experts, n in ((64, 1024), (20, 1024), (5, 1024)):
        rng = np.random.default_rng(experts)
        for most in (3, 24):
            counts = rng.integers(0, most, experts).tolist()
            say("int4 strips", counts, n)
            d = make(counts, n, 1280, seed=experts + most)
            assert_close(run(gpu_lib, d), d, (experts, n, most))


@pytest.mark.parametrize("experts,most", [(70, 3), (130, 30), (100, 90), (66, 300), (65, 700)])
def test_more_experts_than_lanes(gpu_lib, experts, most):
    rng = np.random.default_rng(experts)
    counts = (rng.integers(0, most, experts) * (rng.random(experts) < 0.8)).tolist()
    say("int4 experts", experts, sum(counts))
    d = make(counts, 136, 256, seed=experts)
    for workspace in (None, False):
        assert_close(run(gpu_lib, d, workspace=workspace), d, (experts, most, workspace))


@pytest.mark.parametrize("most", [2, 20, 100])
def test_overlapping_experts_end(gpu_lib, most):
    """Offsets that go back and forth end, and write nothing outside the output."""
    import torch

    d = make([most] * 80, 72, 256, seed=13)
    rows = 80 * most
    hold = torch.full((rows + 64, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    wild = {**d, "offsets": torch.tensor([0, rows] * 40 + [0], dtype=torch.int32)}
    run(gpu_lib, wild, out=hold[32:-32])
    assert torch.all(hold[:32] == 7.0) and torch.all(hold[-32:] == 7.0)
    assert_close(run(gpu_lib, d), d, most)


@pytest.mark.parametrize("counts", [[2, 0, 3], [50, 0, 40], [180, 0, 90]])
def test_rows_of_no_expert_stay(gpu_lib, counts):
    import torch

    first, behind = 5, 9
    d = make(counts, 136, 256, seed=3, first=first, behind=behind)
    d["x"][:first], d["x"][first + sum(counts):] = float("nan"), float("inf")      # never read
    hold = torch.full((first + sum(counts) + behind, 144), 3.0, dtype=torch.bfloat16, device="cuda")
    run(gpu_lib, d, out=hold[:, :136])
    assert torch.all(hold[:first] == 3.0) and torch.all(hold[first + sum(counts):] == 3.0)
    assert torch.all(hold[:, 136:] == 3.0)
    assert_close(hold[:, :136], d, counts)


def test_strided_activations(gpu_lib):
    import torch

    for counts in ([2, 5, 0], [60, 70, 1]):
        d = make(counts, 72, 256, seed=5)
        wide = torch.full((sum(counts), 264), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :256] = d["x"].cuda()
        got = gpu_lib.qgemm_int4_grouped(wide[:, :256], d["qweight"].cuda(), d["scales"].cuda(), d["qzeros"].cuda(),
                                         d["offsets"].cuda())
        torch.cuda.synchronize()
        assert_close(got, d, counts)


def test_k_zero_writes_zeros(gpu_lib):
    import torch

    d = make([2, 3], 16, 128, seed=7, behind=2)
    out = torch.full((7, 16), 5.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.qgemm_int4_grouped(d["x"].cuda()[:, :0], d["qweight"].cuda()[:, :0], d["scales"].cuda()[:, :0],
                               d["qzeros"].cuda()[:, :0], d["offsets"].cuda(), out=out)
    torch.cuda.synchronize()
    assert torch.all(out[:5] == 0) and torch.all(out[5:] == 5.0)


@pytest.mark.parametrize("counts", [[3, 1], [40, 20], [300, 100]])
def test_equals_one_expert_at_a_time_and_replays(gpu_lib, counts):
    """Each expert's rows are what qgemm_int4 accepts for them; the same bits from a captured
    graph whose offsets change between replays, with eager calls between."""
    import torch

    d = make(counts, 264, 512, seed=9)
    got = run(gpu_lib, d)
    off = d["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        one = gpu_lib.qgemm_int4(d["x"][lo:hi].cuda(), d["qweight"][e].cuda(), d["scales"][e].cuda(),
                                 d["qzeros"][e].cuda())
        torch.cuda.synchronize()
        part = {**d, "offsets": torch.tensor([0] * (e + 1) + [hi - lo] * (len(counts) - e), dtype=torch.int32),
                "x": d["x"][lo:hi]}
        assert_close(one, part, e)
        assert_close(got[lo:hi], part, e)
    x, off_d, out = d["x"].cuda(), d["offsets"].cuda(), torch.zeros_like(got)
    qw, sc, qz = d["qweight"].cuda(), d["scales"].cuda(), d["qzeros"].cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.qgemm_int4_grouped(x, qw, sc, qz, off_d, out=out)
    for cut in (0, 1, sum(counts) // 2, sum(counts)):
        off_d.copy_(torch.tensor([0, cut, sum(counts)], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eager = gpu_lib.qgemm_int4_grouped(x, qw, sc, qz, off_d)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), cut
        assert_close(out, {**d, "offsets": off_d.cpu()}, cut)


def test_refusals(gpu_lib):
    import torch

    d = make([2, 3], 16, 128, seed=11)
    x, qw, sc, qz, off = (d[k].cuda() for k in ("x", "qweight", "scales", "qzeros", "offsets"))
    f = gpu_lib.qgemm_int4_grouped
    with pytest.raises(TypeError):
        f(x.float(), qw, sc, qz, off)
    with pytest.raises(TypeError):
        f(x, qw, sc.float(), qz, off)
    for bad in ((x, qw[:1], sc, qz, off), (x, qw, sc[:, :, :8], qz, off), (x, qw, sc, qz[:, :, :1], off),
                (x, qw, sc, qz, off[:2]), (x, qw, sc, qz, off.long()), (x, qw.cpu(), sc, qz, off),
                (x, qw.transpose(1, 2).contiguous().transpose(1, 2), sc, qz, off)):
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(gpu_lib.QGemmError):
        f(x, qw, sc, qz, off, group_size=64)
    with pytest.raises(ValueError):
        f(x, qw, sc, qz, off, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(gpu_lib.QGemmError):
        f(x, qw, sc, qz, off, workspace=torch.empty(33, dtype=torch.uint8, device="cuda")[1:])
