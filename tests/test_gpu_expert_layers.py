"""The grouped and MXFP4 operators one after the other, as a model's expert layers use them.

Training: tokens sorted by expert, y = relu(x W1_e^T) W2_e^T with its gradients, all in
gemm_grouped.  Every value carries a bound of its error in fp64: a product of a (off by ea)
and b (off by eb) is off by ea |b| + |a| eb + ea eb, by gamma_K (|a| + ea)(|b| + eb) for its fp32
sums, gamma_K = K u / (1 - K u), u = 2^-24, and by one rounding (eps / 2 of the value, half the
smallest subnormal).  relu passes an error on at most as it is; its derivative is taken from the
computed hidden values, as a program does.

Serving: int4 experts, then relu, then a linear layer in MXFP4, eagerly and from a graph."""
import numpy as np
import pytest

from gpu_helpers import say
from test_gpu_grouped import reference
from test_gpu_grouped_int4 import assert_close as assert_int4, make as make_int4
from test_gpu_mxfp4 import activations, assert_product, plain_quantize

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def routed(tokens, experts, top, seed):
    """(token of each row, offsets): every token's `top` experts, rows sorted by expert."""
    import torch

    rng = np.random.default_rng(seed)
    scores = rng.standard_normal((tokens, experts)) + 1.5 * rng.standard_normal(experts)
    chosen = np.argsort(-scores, axis=1)[:, :top]
    order = np.argsort(chosen.reshape(-1), kind="stable")
    counts = np.bincount(chosen.reshape(-1), minlength=experts)
    return (torch.from_numpy(order // top), torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,experts,top,d,f", [(1, 8, 2, 64, 136), (37, 8, 2, 72, 200), (600, 6, 2, 264, 520),
                                                    (50, 3, 1, 35, 51)])
def test_training_layer(gpu_lib, dtype, tokens, experts, top, d, f):
    import torch

    say("expert layer", dtype, tokens, experts, top, d, f)
    t = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dtype]
    fi = torch.finfo(t)
    g = torch.Generator().manual_seed(tokens)
    rnd = lambda *shape: (torch.randn(shape, generator=g) / 8).to(t)
    token, off = routed(tokens, experts, top, tokens)
    x, w1, w2, dy = rnd(tokens, d)[token], rnd(experts, f, d), rnd(experts, d, f), rnd(token.numel(), d)
    run = lambda layout, a, b: gpu_lib.gemm_grouped(layout, a, b, doff)
    doff = off.cuda()
    dx_, w1_, w2_, dy_ = (v.cuda() for v in (x, w1, w2, dy))
    h = run("NT", dx_, w1_)
    a = torch.relu(h)
    y = run("NT", a, w2_)
    da = run("NN", dy_, w2_)
    dh = torch.where(h > 0, da, torch.zeros_like(da))
    gx = run("NN", dh, w1_)
    gw1 = run("TN", dh, dx_)
    gw2 = run("TN", dy_, a)
    torch.cuda.synchronize()

    def product(layout, p, q):          # p, q: (value, error bound), fp64
        (pv, pe), (qv, qe) = p, q
        value = reference(layout, pv, qv, off)
        top_ = reference(layout, pv.abs() + pe, qv.abs() + qe, off)
        carried = top_ - reference(layout, pv, qv, off, absolute=True)
        K = (pv.shape[0] if layout == "TN" else pv.shape[1]) + (dtype == "fp32")
        err = carried.clamp(min=0) + K * U / (1 - K * U) * top_
        if dtype != "fp32":
            err = err + (value.abs() + err) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2
        return value, err * (1 + 1e-9)

    exact = lambda v: (v.double(), torch.zeros_like(v, dtype=torch.float64))
    rh = product("NT", exact(x), exact(w1))
    ra = (rh[0].clamp(min=0), rh[1])
    ry = product("NT", ra, exact(w2))
    rda = product("NN", exact(dy), exact(w2))
    on = (h > 0).cpu().double()
    rdh = (rda[0] * on, rda[1] * on)
    for name, got, (ref, err) in (("h", h, rh), ("y", y, ry), ("da", da, rda), ("gx", gx, product("NN", rdh, exact(w1))),
                                  ("gw1", gw1, product("TN", rdh, exact(x))), ("gw2", gw2, product("TN", exact(dy), ra))):
        diff = (got.cpu().double() - ref).abs()
        assert bool((diff <= err).all()), (name, float((diff - err).max()))


@pytest.mark.parametrize("tokens", [1, 9, 150])
def test_serving_layer(gpu_lib, tokens):
    import torch

    experts, top, k, n, out = 6, 2, 256, 288, 200
    say("serving", tokens)
    token, off = routed(tokens, experts, top, tokens)
    d = make_int4([tokens * top] + [0] * (experts - 1), n, k, seed=tokens)
    d["offsets"] = off
    x, qw, sc, qz, doff = (d[key].cuda() for key in ("x", "qweight", "scales", "qzeros", "offsets"))
    wc, ws = gpu_lib.mxfp4_quantize(activations(out, n, "bf16", seed=5).cuda())

    def layer():
        h = gpu_lib.qgemm_int4_grouped(x, qw, sc, qz, doff)
        a = torch.relu(h)
        codes, scales = gpu_lib.mxfp4_quantize(a)
        return h, a, gpu_lib.gemm_mxfp4(codes, scales, wc, ws)

    def check(h, a, y, what):
        assert_int4(h, {**d, "x": x.cpu(), "offsets": doff.cpu()}, what)
        assert_product(y, plain_quantize(a.double().cpu().numpy()), (wc.cpu().numpy(), ws.cpu().numpy()), "bf16", what)

    check(*layer(), "eager")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, a, y = layer()
    for i in range(3):                   # other tokens, another routing
        x.copy_(make_int4([tokens * top], n, k, seed=50 + i)["x"].cuda())
        doff.copy_(routed(tokens, experts, top, 70 + i)[1].cuda())
        graph.replay()
        torch.cuda.synchronize()
        eager = layer()
        torch.cuda.synchronize()
        for got, want in zip((h, a, y), eager):
            assert torch.equal(got, want), i
        check(h, a, y, i)
