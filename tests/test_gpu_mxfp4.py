"""GPU parity of MXFP4 quantisation, reading back and products against plain fp64 forms.

Quantisation and reading back are exact definitions: codes, scales and values are compared
bit for bit (the value in fp16, which the largest scales leave, after one rounding).
Products: every product of two codes and scales is exact in fp32, so the sum of K of them
is off by at most gamma_K sum |a||b|, gamma_K = K u / (1 - K u), u = 2^-24, in any order, and
rounds once to the output's type (half a step: eps / 2 relative, and half the smallest
subnormal)."""
import numpy as np
import pytest

from gpu_helpers import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def tdtype(name):
    import torch

    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def plain_quantize(x):
    """(codes [rows][k/2], scale bytes [rows][k/32]) of an fp64 numpy matrix."""
    rows, k = x.shape
    v = x.reshape(rows, k // 32, 32)
    top = np.abs(v).max(axis=2)
    finite = np.isfinite(v).all(axis=2)
    ex = np.full(top.shape, -127, dtype=np.int64)
    pos = finite & (top > 0)
    ex[pos] = np.clip(np.frexp(top[pos])[1] - 3, -127, 127)
    u = np.abs(np.where(finite[:, :, None], v, 0.0)) / np.exp2(ex.astype(np.float64))[:, :, None]
    d = np.abs(u[..., None] - GRID[:8])
    near = d.min(axis=-1, keepdims=True)
    tie_even = np.where(d == near, np.arange(8) % 2, 2)          # the even code wins a tie
    code = np.argmin(tie_even, axis=-1)
    code = code + 8 * (np.signbit(v) & finite[:, :, None])
    code = code.reshape(rows, k // 2, 2)
    return (code[..., 0] + 16 * code[..., 1]).astype(np.uint8), np.where(finite, ex + 127, 255).astype(np.uint8)


def plain_values(codes, scales):
    nib = np.stack([codes & 15, codes >> 4], axis=2).reshape(codes.shape[0], -1, 32)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (GRID[nib] * s[:, :, None]).reshape(codes.shape[0], -1)


def activations(rows, k, dtype, seed):
    """Rows and blocks of very different size, zero blocks, zeros, ties and the largest codes' edges."""
    import torch

    g = torch.Generator().manual_seed(seed)
    v = torch.randn((rows, k // 32, 32), generator=g, dtype=torch.float64)
    span = 12.0 if dtype == "fp16" else 60.0
    v = v * torch.exp2((torch.rand((rows, k // 32, 1), generator=g, dtype=torch.float64) - 0.5) * 2 * span / 3)
    v[torch.rand((rows, k // 32), generator=g) < 0.1] = 0.0
    v[torch.rand((rows, k // 32, 32), generator=g) < 0.05] = 0.0
    # blocks whose elements are multiples of 1/8: every midpoint between two codes
    ties = torch.rand((rows, k // 32), generator=g) < 0.3
    eighths = torch.randint(-63, 64, (rows, k // 32, 32), generator=g).double() / 8
    v[ties] = eighths[ties]
    return v.reshape(rows, k).to(tdtype(dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 96), (17, 512), (5, 4096), (130, 1056)])
def test_quantize_bit_exact(gpu_lib, dtype, rows, k):
    import torch

    say("quantize", dtype, rows, k)
    x = activations(rows, k, dtype, seed=rows + k)
    codes, scales = gpu_lib.mxfp4_quantize(x.cuda())
    torch.cuda.synchronize()
    want_c, want_s = plain_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    for name in ("bf16", "fp16", "fp32"):
        y = gpu_lib.mxfp4_dequantize(codes, scales, dtype=tdtype(name))
        torch.cuda.synchronize()
        want = torch.from_numpy(plain_values(want_c, want_s)).to(tdtype(name))
        assert y.dtype == tdtype(name) and torch.equal(y.cpu(), want), name


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantize_special_values(gpu_lib, dtype):
    """Infinities, NaN, signed zeros, subnormals, the type's largest and smallest values."""
    import torch

    fi = torch.finfo(tdtype(dtype))
    x = torch.zeros((12, 64), dtype=tdtype(dtype))
    x[0, 3], x[0, 40] = float("inf"), 1.0
    x[1, 5], x[1, 6] = float("-inf"), 2.0
    x[2, 9] = float("nan")
    x[3] = fi.max
    x[4, ::2], x[4, 1::2] = fi.max, -fi.max
    x[5] = fi.tiny
    x[6] = fi.smallest_normal * fi.eps                      # the smallest subnormal
    x[7, 0], x[7, 1] = fi.tiny, fi.smallest_normal * fi.eps
    x[8] = -0.0
    x[9] = torch.linspace(-8, 8, 64).to(tdtype(dtype))
    x[10, 0], x[10, 1:32] = fi.max, fi.tiny
    x[11] = fi.min
    codes, scales = gpu_lib.mxfp4_quantize(x.cuda())
    y = gpu_lib.mxfp4_dequantize(codes, scales, dtype=torch.float32)
    torch.cuda.synchronize()
    want_c, want_s = plain_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert scales[0, 0] == 255 and scales[0, 1] != 255 and scales[1, 0] == 255 and scales[2, 0] == 255
    want = torch.from_numpy(plain_values(want_c, want_s)).float()
    got = y.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(got[0, :32]).all()
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    assert torch.equal(torch.signbit(got[8]), torch.ones(64, dtype=torch.bool))       # -0 stays -0


def test_every_code_and_scale_reads_back(gpu_lib):
    """All 16 codes under all 256 scales, in every type (fp16 overflows to infinity and rounds
    its subnormals; bf16 and fp32 only overflow)."""
    import torch

    codes = np.tile(np.arange(16, dtype=np.uint8) * 16 + np.arange(15, -1, -1, dtype=np.uint8), (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    for name in ("bf16", "fp16", "fp32"):
        y = gpu_lib.mxfp4_dequantize(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), dtype=tdtype(name))
        torch.cuda.synchronize()
        want = torch.from_numpy(plain_values(codes, scales)).to(tdtype(name))
        got = y.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        held = ~torch.isnan(want)
        assert torch.equal(got[held], want[held]), name


def test_quantize_strided(gpu_lib):
    """Padded and unaligned rows in, padded rows out; nothing outside the views is written."""
    import torch

    for dtype, start, pad in (("bf16", 0, 8), ("bf16", 1, 3), ("fp32", 1, 1), ("fp16", 8, 0)):
        x = activations(7, 160, dtype, seed=3)
        wide = torch.full((7, start + 160 + pad), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, start:start + 160] = x.cuda()
        codes = torch.full((8, 96), 0xAB, dtype=torch.uint8, device="cuda")
        scales = torch.full((8, 7), 0xCD, dtype=torch.uint8, device="cuda")
        gpu_lib.mxfp4_quantize(wide[:, start:start + 160], codes[:7, :80], scales[:7, 1:6])
        torch.cuda.synchronize()
        want_c, want_s = plain_quantize(x.double().numpy())
        assert np.array_equal(codes[:7, :80].cpu().numpy(), want_c)
        assert np.array_equal(scales[:7, 1:6].cpu().numpy(), want_s)
        assert torch.all(codes[7] == 0xAB) and torch.all(codes[:, 80:] == 0xAB)
        assert torch.all(scales[7] == 0xCD) and torch.all(scales[:, 0] == 0xCD) and torch.all(scales[:, 6] == 0xCD)
        hold = torch.full((8, start + 160 + pad), 7.0, dtype=x.dtype, device="cuda")
        gpu_lib.mxfp4_dequantize(codes[:7, :80], scales[:7, 1:6], out=hold[:7, start:start + 160])
        torch.cuda.synchronize()
        want = torch.from_numpy(plain_values(want_c, want_s)).to(x.dtype)
        assert torch.equal(hold[:7, start:start + 160].cpu(), want)
        hold[:7, start:start + 160] = 7.0
        assert torch.all(hold == 7.0)


def mx_matrix(rows, k, seed, spread=8):
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 256, (rows, k // 2), dtype=np.uint8),
            rng.integers(127 - spread, 128 + spread, (rows, k // 32)).astype(np.uint8))


def up(m):
    import torch

    return tuple(torch.from_numpy(t).cuda() for t in m)


def assert_product(got, a, b, dtype, what):
    import torch

    va, vb = plain_values(*a), plain_values(*b)
    K = va.shape[1]
    ref, mag = va @ vb.T, np.abs(va) @ np.abs(vb).T
    tol = K * U / (1 - K * U) * mag
    fi = torch.finfo(tdtype(dtype))
    if dtype != "fp32":
        tol = tol + (np.abs(ref) + tol) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2
    g = got.cpu().double().numpy()
    assert g.shape == ref.shape
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), g[bad][:4], ref[bad][:4], np.argwhere(bad)[:4])


# M: one row, strips of 16 and 32 rows, tiles of 64, 128 and 256 rows that end inside; N
# and k that end inside a tile, a chunk and a wave's share
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("K", [32, 160, 512, 1056, 4640])
def test_products(gpu_lib, dtype, K):
    import torch

    spread = 2 if dtype == "fp16" else 8                     # (the values stay inside fp16)
    for M, N in ((1, 1), (1, 257), (15, 33), (17, 40), (32, 16), (33, 130), (64, 65), (100, 257), (257, 300)):
        say("mxfp4", dtype, M, N, K)
        a, b = mx_matrix(M, K, M + K, spread), mx_matrix(N, K, N + K + 1, spread)
        if dtype == "fp16":
            a[1][:] -= 6
        c = gpu_lib.gemm_mxfp4(*up(a), *up(b), dtype=tdtype(dtype))
        torch.cuda.synchronize()
        assert_product(c, a, b, dtype, (M, N, K))


@pytest.mark.parametrize("K", [256, 1312])
def test_large_tiles(gpu_lib, K):
    """Enough 256 x 256 tiles to be chosen, ragged on both sides, against sampled rows and columns."""
    import torch

    M, N = 2500, 5200
    a, b = mx_matrix(M, K, 1), mx_matrix(N, K, 2)
    for dtype in ("bf16", "fp32"):
        say("mxfp4 large", dtype, M, N, K)
        c = gpu_lib.gemm_mxfp4(*up(a), *up(b), dtype=tdtype(dtype))
        torch.cuda.synchronize()
        rows = np.unique(np.concatenate([np.arange(0, M, 37), [255, 256, 2303, 2304, 2499]]))
        cols = np.unique(np.concatenate([np.arange(0, N, 41), [255, 256, 5119, 5120, 5199]]))
        part = c[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()]
        assert_product(part, (a[0][rows], a[1][rows]), (b[0][cols], b[1][cols]), dtype, (dtype, K))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N", [(1500, 12000), (2000, 9300)])
def test_columns_past_whole_rounds(gpu_lib, dtype, M, N):
    """More 256 x 256 tiles than CUs and few in the last round: a second launch takes the columns
    that are left (from 10752 and 8192 on).  The scales' rows start on any byte; the output is a
    view that starts on any element."""
    import torch

    say("mxfp4 columns", dtype, M, N)
    K = 288
    spread = 2 if dtype == "fp16" else 8
    a, b = mx_matrix(M, K, 3, spread), mx_matrix(N, K, 4, spread)
    hold = torch.full((M + 1, N + 5), 7.0, dtype=tdtype(dtype), device="cuda")
    out = gpu_lib.gemm_mxfp4(*up(a), *up(b), out=hold[:M, 3:3 + N])
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([np.arange(0, M, 61), [255, 256, M - 1]]))
    cols = np.unique(np.concatenate([np.arange(0, N, 53), [8191, 8192, min(10751, N - 2), min(10752, N - 2), N - 1]]))
    part = out[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()]
    assert_product(part, (a[0][rows], a[1][rows]), (b[0][cols], b[1][cols]), dtype, (dtype, M, N))
    hold[:M, 3:3 + N] = 7.0
    assert torch.all(hold == 7.0)


@pytest.mark.parametrize("M", [8, 24, 700])
def test_rows_past_32_bits(gpu_lib, M):
    """The widest leading dimensions: offsets of codes, scales and results past 32 bits."""
    import torch

    K, N, ld = 544, 600, 2 ** 22
    a, b = mx_matrix(M, K, 1), mx_matrix(N, K, 2)

    def wide(m):
        hold = torch.empty((m.shape[0], ld), dtype=torch.uint8, device="cuda")
        hold[:, :m.shape[1]] = torch.from_numpy(m).cuda()
        return hold[:, :m.shape[1]]

    out = torch.empty((M, 2 ** 22), dtype=torch.bfloat16, device="cuda")[:, :N]
    gpu_lib.gemm_mxfp4(wide(a[0]), wide(a[1]), wide(b[0]), wide(b[1]), out=out)
    torch.cuda.synchronize()
    assert_product(out, a, b, "bf16", M)


def test_scales_of_every_alignment_and_padding(gpu_lib):
    """Scale rows on 16, 4 and 1 bytes give the same bits; padding behind rows (NaN scales, any
    codes) is never used."""
    import torch

    for M in (3, 24, 50, 200):
        for K in (512, 544, 2080):
            a, b = mx_matrix(M, K, M), mx_matrix(136, K, K)
            first = gpu_lib.gemm_mxfp4(*up(a), *up(b), dtype=torch.float32)
            for pad, start in ((16, 0), (4, 4), (3, 1)):
                ld = (K // 32 + 15) // 16 * 16 + pad
                sa = torch.full((M, start + ld), 255, dtype=torch.uint8, device="cuda")
                sb = torch.full((136, start + ld), 255, dtype=torch.uint8, device="cuda")
                sa[:, start:start + K // 32], sb[:, start:start + K // 32] = up(a)[1], up(b)[1]
                ca = torch.full((M, K // 2 + 32), 0x77, dtype=torch.uint8, device="cuda")
                ca[:, :K // 2] = up(a)[0]
                got = gpu_lib.gemm_mxfp4(ca[:, :K // 2], sa[:, start:start + K // 32], up(b)[0],
                                         sb[:, start:start + K // 32], dtype=torch.float32)
                torch.cuda.synchronize()
                assert torch.equal(first, got), (M, K, pad, start)
            assert_product(first, a, b, "fp32", (M, K))


def test_nan_scale_reaches_its_row_and_column_only(gpu_lib):
    import torch

    for M in (5, 30, 60, 300):
        a, b = mx_matrix(M, 768, 5), mx_matrix(200, 768, 6)
        a[1][2, 7], b[1][150, 20] = 255, 255
        a[0][2], b[0][150] = 0, 0                            # codes of zero: zero times NaN
        c = gpu_lib.gemm_mxfp4(*up(a), *up(b), dtype=torch.float32).cpu()
        want = np.zeros((M, 200), dtype=bool)
        want[2], want[:, 150] = True, True
        assert np.array_equal(torch.isnan(c).numpy(), want), M


def test_output_view_and_zero_sizes(gpu_lib):
    import torch

    for M in (4, 70, 300):
        a, b = mx_matrix(M, 320, 7), mx_matrix(90, 320, 8)
        for dtype in ("bf16", "fp32"):
            hold = torch.full((M + 1, 97), 7.0, dtype=tdtype(dtype), device="cuda")
            gpu_lib.gemm_mxfp4(*up(a), *up(b), out=hold[:M, 3:93])
            torch.cuda.synchronize()
            assert_product(hold[:M, 3:93], a, b, dtype, (M, dtype))
            hold[:M, 3:93] = 7.0
            assert torch.all(hold == 7.0)
    a, b = mx_matrix(5, 0, 9), mx_matrix(6, 0, 9)
    assert torch.all(gpu_lib.gemm_mxfp4(*up(a), *up(b)) == 0)
    a, b = mx_matrix(0, 64, 9), mx_matrix(6, 64, 9)
    assert gpu_lib.gemm_mxfp4(*up(a), *up(b)).shape == (0, 6)
    c, s = gpu_lib.mxfp4_quantize(torch.empty((0, 64), device="cuda"))
    assert gpu_lib.mxfp4_dequantize(c, s).shape == (0, 64)


@pytest.mark.parametrize("M", [1, 20, 60, 150])
def test_layer_captured_with_other_streams(gpu_lib, M):
    """A linear layer as it is used (quantise, multiply) eagerly, on another stream and from a
    graph whose input changes between replays, with eager work between: the same bits."""
    import torch

    wc, ws = gpu_lib.mxfp4_quantize(activations(264, 544, "bf16", seed=M).cuda())
    x = activations(M, 544, "bf16", seed=M + 1).cuda()

    def layer(stream=None):
        c, s = gpu_lib.mxfp4_quantize(x, stream=stream)
        return gpu_lib.gemm_mxfp4(c, s, wc, ws, stream=stream)

    first = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = layer(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    for i in range(4):
        x.copy_(activations(M, 544, "bf16", seed=100 + i).cuda())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer())
        c, s = plain_quantize(x.double().cpu().numpy())
        assert_product(y, (c, s), (wc.cpu().numpy(), ws.cpu().numpy()), "bf16", (M, i))


def test_refusals(gpu_lib):
    import torch

    a, b = up(mx_matrix(4, 64, 1)), up(mx_matrix(8, 64, 2))
    x = torch.zeros((4, 64), device="cuda")
    for bad in (x[:, :40], x[0], x.cpu(), x.t().contiguous().t()):
        with pytest.raises(ValueError):
            gpu_lib.mxfp4_quantize(bad)
    with pytest.raises(TypeError):
        gpu_lib.mxfp4_quantize(x.double())
    with pytest.raises(ValueError):
        gpu_lib.mxfp4_quantize(x, codes=a[0][:3])
    with pytest.raises(gpu_lib.QGemmError):
        gpu_lib.mxfp4_quantize(x, codes=torch.empty((4, 33), dtype=torch.uint8, device="cuda")[:, 1:])
    with pytest.raises(TypeError):
        gpu_lib.mxfp4_dequantize(a[0], a[1], dtype=torch.float64)
    with pytest.raises(TypeError):
        gpu_lib.gemm_mxfp4(a[0].to(torch.int8), a[1], *b)
    for bad in ((a[0], a[1][:, :1], *b), (a[0][:, :16], a[1][:, :1], *b), (a[0], a[1], b[0].cpu(), b[1].cpu()),
                (a[0][0], a[1][0], *b)):
        with pytest.raises(ValueError):
            gpu_lib.gemm_mxfp4(*bad)
    with pytest.raises(ValueError):
        gpu_lib.gemm_mxfp4(*a, *b, out=torch.empty((4, 7), dtype=torch.bfloat16, device="cuda"))
