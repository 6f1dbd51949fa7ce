"""What is measured of the experts' products and of the microscaled 4-bit format.

Four operators, each in its plain form (elementary torch operations in 32 bits
or more) and as the framework's own call:

  grouped   matrix products grouped by expert, ragged: rows sorted by expert,
            rows offsets[e] .. offsets[e + 1] belong to expert e (NT forward, NN
            input gradient, TN weight gradient; bf16, fp16, fp32)
  int4      the same forward product with GPTQ int4 expert weights
  mx_quant  rows quantised to MXFP4 (blocks of 32 along the row: 4-bit e2m1
            codes and one power-of-two scale) and read back
  mx_gemm   the product of two MXFP4 matrices, Y = A . B^T
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GROUP = 128      # k rows per int4 scale and zero
BLOCK = 32       # elements per MXFP4 scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # eight sequences decoding one token each, eight experts a token: one or two
        # rows an expert, most of the time goes into reading the chosen experts' weights
        {"name": "grouped_nt_decode", "op": "grouped", "layout": "NT", "dtype": "bf16",
         "tokens": 8, "topk": 8, "experts": 64, "k": 2048, "n": 1024},
        # a prompt (or a training batch) of 2048 tokens through the experts' up projection
        {"name": "grouped_nt_prompt", "op": "grouped", "layout": "NT", "dtype": "bf16",
         "tokens": 2048, "topk": 4, "experts": 32, "k": 2048, "n": 5632},
        # its input gradient at 1024 tokens, in fp16
        {"name": "grouped_nn_dgrad", "op": "grouped", "layout": "NN", "dtype": "fp16",
         "tokens": 1024, "topk": 4, "experts": 16, "k": 5632, "n": 2048},
        # its weight gradient: one matrix for every expert, contracted over that expert's rows
        {"name": "grouped_tn_wgrad", "op": "grouped", "layout": "TN", "dtype": "bf16",
         "tokens": 2048, "topk": 4, "experts": 32, "k": 2048, "n": 5632},
        # fp32 training with sizes that fill no tile
        {"name": "grouped_nt_fp32_ragged", "op": "grouped", "layout": "NT", "dtype": "fp32",
         "tokens": 701, "topk": 2, "experts": 8, "k": 1000, "n": 1416},
        # one sequence decoding one token: eight experts with one row each, the smallest call
        {"name": "int4_grouped_token", "op": "int4", "tokens": 1, "topk": 8, "experts": 64,
         "k": 2048, "n": 1024, "zeros": True},
        # 32 sequences decoding over large experts: a few rows each
        {"name": "int4_grouped_decode", "op": "int4", "tokens": 32, "topk": 2, "experts": 16,
         "k": 4096, "n": 14336, "zeros": True},
        # a prompt of 2048 tokens through the same kind of experts
        {"name": "int4_grouped_prompt", "op": "int4", "tokens": 2048, "topk": 2, "experts": 8,
         "k": 4096, "n": 14336, "zeros": True},
        # one token's activations quantised before a product, and read back
        {"name": "mx_quant_token", "op": "mx_quant", "dtype": "bf16", "m": 1, "k": 4096},
        # a prompt's activations (or a weight matrix when a model is converted)
        {"name": "mx_quant_prompt", "op": "mx_quant", "dtype": "bf16", "m": 4096, "k": 14336},
        # one token through a large MXFP4 layer
        {"name": "mx_gemm_token", "op": "mx_gemm", "dtype": "bf16", "m": 1, "n": 14336, "k": 4096},
        # a prompt of 2000 tokens through a large MXFP4 layer
        {"name": "mx_gemm_prompt", "op": "mx_gemm", "dtype": "bf16", "m": 2000, "n": 25600, "k": 5120},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step between lo and hi, uniform in its logarithm."""
    v = int(round(lo * (hi / lo) ** rng.random() / step)) * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped", "int4", "int4", "mx_quant", "mx_gemm", "mx_gemm"])
    if op == "grouped":
        experts = _log(rng, 2, 64)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        layout = rng.choice(["NT", "NN", "TN"])
        step = rng.choice([64, 8, 8, 1])       # widths that fill tiles, that only align, that do neither
        topk = min(experts, rng.choice([1, 2, 4, 8]))
        case = {"op": op, "layout": layout, "dtype": dtype, "topk": topk, "experts": experts,
                "k": _log(rng, 256, 5632, step), "n": _log(rng, 256, 5632, step)}
        cap = {"bf16": 1.5e11, "fp16": 1.5e11, "fp32": 2.0e10}[dtype] * (0.2 if step == 1 else 1.0)
        if experts * case["k"] * case["n"] > 3.0e8:
            case["n"] = max(step, int(3.0e8 / (experts * case["k"])) // step * step)
        most = max(1, min(4096, int(cap / (2.0 * topk * case["k"] * case["n"]))))
        case["tokens"] = _log(rng, 1, most)
        return case
    if op == "int4":
        experts = _log(rng, 2, 64)
        topk = min(experts, rng.choice([1, 2, 4, 8]))
        case = {"op": op, "topk": topk, "experts": experts, "k": _log(rng, 256, 5120, 128),
                "n": _log(rng, 256, 14336, 8), "zeros": rng.random() < 0.75}
        if experts * case["k"] * case["n"] > 9.0e8:
            case["n"] = max(8, int(9.0e8 / (experts * case["k"])) // 8 * 8)
        most = max(1, min(4096, int(3.0e11 / (2.0 * topk * case["k"] * case["n"]))))
        case["tokens"] = _log(rng, 1, most)
        return case
    if op == "mx_quant":
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "m": _log(rng, 1, 4000),
                "k": _log(rng, 32, 12000, 32)}
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
            "n": _log(rng, 256, 25600, rng.choice([128, 8, 1])), "k": _log(rng, 256, 8192, rng.choice([256, 128, 32]))}
    case["m"] = _log(rng, 1, max(1, min(2048, int(4.0e11 / (2.0 * case["n"] * case["k"])))))
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _route(case, rng):
    """offsets [experts + 1] of rows sorted by expert: every token takes topk different
    experts, some experts being far more popular than others."""
    e, t, k = case["experts"], case["tokens"], case["topk"]
    liking = rng.standard_normal(e) * 0.7
    score = liking[None, :] + rng.gumbel(size=(t, e))
    chosen = np.argpartition(-score, k - 1, axis=1)[:, :k]
    counts = np.bincount(chosen.ravel(), minlength=e)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _uneven(gen, rows, cols, dtype):
    """Activations as a layer meets them: rows of different size, a few channels that stick
    out, and some blocks that are all zero."""
    v = torch.randn((rows, cols), generator=gen, device="cuda", dtype=torch.float32)
    v *= torch.exp(torch.randn((rows, 1), generator=gen, device="cuda"))
    v *= torch.exp(1.5 * torch.randn((1, cols), generator=gen, device="cuda"))
    blank = torch.rand((rows, cols // BLOCK, 1), generator=gen, device="cuda") < 0.02
    v = v.view(rows, cols // BLOCK, BLOCK).masked_fill(blank, 0.0).view(rows, cols)
    return v.clamp(-6e4, 6e4).to(dtype)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op in ("grouped", "int4"):
        off = _route(case, rng)
        st["host_offsets"] = off.tolist()
        st["offsets"] = torch.from_numpy(off).cuda()
        m, k, n, e = int(off[-1]), case["k"], case["n"], case["experts"]
    if op == "grouped":
        dt = DTYPES[case["dtype"]]
        if case["layout"] == "NT":        # x [m][k], w [e][n][k]
            st["a"] = _normal(gen, (m, k), 1.0, dt)
            st["b"] = _normal(gen, (e, n, k), 0.02, dt)
        elif case["layout"] == "NN":      # dy [m][k], w [e][k][n]
            st["a"] = _normal(gen, (m, k), 0.05, dt)
            st["b"] = _normal(gen, (e, k, n), 0.02, dt)
        else:                             # dy [m][n], x [m][k]: gradients [e][n][k]
            st["a"] = _normal(gen, (m, n), 0.05, dt)
            st["b"] = _normal(gen, (m, k), 1.0, dt)
    elif op == "int4":
        st["x"] = _normal(gen, (m, k), 1.0, torch.bfloat16)
        st["qweight"] = torch.randint(-2 ** 31, 2 ** 31, (e, k // 8, n), generator=gen, device="cuda",
                                      dtype=torch.int32)
        st["scales"] = (torch.rand((e, k // GROUP, n), generator=gen, device="cuda") * 0.008
                        + 0.002).to(torch.float16)
        st["qzeros"] = (torch.randint(-2 ** 31, 2 ** 31, (e, k // GROUP, n // 8), generator=gen, device="cuda",
                                      dtype=torch.int32) if case["zeros"] else None)
    elif op == "mx_quant":
        st["x"] = _uneven(gen, case["m"], case["k"], DTYPES[case["dtype"]])
    else:
        st["a"] = _mx_encode(_uneven(gen, case["m"], case["k"], torch.bfloat16))
        parts = [_mx_encode(_normal(gen, (min(4096, case["n"] - r), case["k"]), 0.02, torch.bfloat16))
                 for r in range(0, case["n"], 4096)]
        st["b"] = (torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts]))
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _grouped_plain(st):
    case, a, b, off = st["case"], st["a"], st["b"], st["host_offsets"]
    if case["layout"] == "TN":
        out = torch.zeros((case["experts"], a.shape[1], b.shape[1]), dtype=a.dtype, device=a.device)
        for e in range(case["experts"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                out[e] = (a[lo:hi].float().t() @ b[lo:hi].float()).to(a.dtype)
        return out
    n = case["n"]
    out = torch.empty((a.shape[0], n), dtype=a.dtype, device=a.device)
    for e in range(case["experts"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            w = b[e].float()
            out[lo:hi] = (a[lo:hi].float() @ (w.t() if case["layout"] == "NT" else w)).to(a.dtype)
    return out


def _int4_weights(qweight, scales, qzeros):
    """fp32 [k][n] weights (q - z) * s of one expert."""
    shifts = torch.arange(0, 32, 4, device=qweight.device, dtype=torch.int32)
    q = ((qweight[:, None, :] >> shifts[None, :, None]) & 15).reshape(-1, qweight.shape[1]).float()
    if qzeros is not None:
        z = ((qzeros[:, :, None] >> shifts[None, None, :]) & 15).reshape(qzeros.shape[0], -1).float()
        q = q - z.repeat_interleave(GROUP, dim=0)
    return q * scales.float().repeat_interleave(GROUP, dim=0)


def _int4_plain(st):
    off, x = st["host_offsets"], st["x"]
    out = torch.empty((x.shape[0], st["case"]["n"]), dtype=torch.bfloat16, device=x.device)
    for e in range(st["case"]["experts"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            z = None if st["qzeros"] is None else st["qzeros"][e]
            w = _int4_weights(st["qweight"][e], st["scales"][e], z)
            out[lo:hi] = (x[lo:hi].float() @ w).to(torch.bfloat16)
    return out


def _mx_split(x):
    """e2m1 code values and block exponents of rows in MXFP4: the block's exponent is
    floor(log2(largest magnitude)) - 2, held to -127 .. 127; elements divided by 2^exponent
    round to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), at most 6."""
    v = x.double().view(x.shape[0], -1, BLOCK)
    top = v.abs().amax(dim=2, keepdim=True)
    ex = torch.where(top > 0, torch.frexp(top)[1].double() - 3.0, torch.full_like(top, -127.0)).clamp(-127, 127)
    u = v * torch.exp2(-ex)
    m = u.abs()
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int()
            + (m >= 3.5).int() + (m > 5.0).int())
    return code + 8 * torch.signbit(u).int(), ex


def _mx_encode(x):
    """(codes uint8 [m][k / 2], even elements in the low nibble; scales uint8 [m][k / 32])."""
    code, ex = _mx_split(x)
    code = code.view(x.shape[0], -1, 2)
    return (code[:, :, 0] + 16 * code[:, :, 1]).to(torch.uint8), (ex[:, :, 0] + 127).to(torch.uint8)


def _mx_grid(device, dtype):
    half = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(half + [-h for h in half], device=device, dtype=dtype)


def _mx_quant_plain(st):
    x = st["x"]
    code, ex = _mx_split(x)
    return (_mx_grid(x.device, torch.float64)[code] * torch.exp2(ex)).view(x.shape).to(x.dtype)


def _mx_values(codes, scales):
    """fp32 values of an MXFP4 matrix."""
    nib = torch.stack([codes & 15, codes >> 4], dim=2).view(codes.shape[0], -1, BLOCK)
    s = torch.exp2(scales.float() - 127.0)
    return (_mx_grid(codes.device, torch.float32)[nib.int()] * s[:, :, None]).view(codes.shape[0], -1)


def _mx_gemm_plain(st):
    return (_mx_values(*st["a"]) @ _mx_values(*st["b"]).t()).to(DTYPES[st["case"]["dtype"]])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"grouped": _grouped_plain, "int4": _int4_plain, "mx_quant": _mx_quant_plain,
                "mx_gemm": _mx_gemm_plain}[op](st)
    import int4_weight_only_gptq_amd as qg

    if op == "grouped":
        return qg.gemm_grouped(case["layout"], st["a"], st["b"], st["offsets"])
    if op == "int4":
        return qg.qgemm_int4_grouped(st["x"], st["qweight"], st["scales"], st["qzeros"], st["offsets"])
    if op == "mx_quant":
        codes, scales = qg.mxfp4_quantize(st["x"])
        return qg.mxfp4_dequantize(codes, scales, dtype=st["x"].dtype)
    return qg.gemm_mxfp4(*st["a"], *st["b"], dtype=DTYPES[case["dtype"]])


def _reached(case):
    """Experts that a routing of these sizes gives at least one row, on average over equally
    liked ones."""
    e, t, k = case["experts"], case["tokens"], case["topk"]
    return e * (1.0 - (1.0 - k / e) ** t)


def work(case):
    op = case["op"]
    if op in ("grouped", "int4"):
        rows, k, n = case["tokens"] * case["topk"], case["k"], case["n"]
        flops = 2.0 * rows * k * n
        if op == "int4":
            weights = _reached(case) * (k * n / 2 + (k / GROUP) * n * (2.5 if case["zeros"] else 2.0))
            return {"bytes": 2.0 * rows * (k + n) + weights, "flops": flops}
        size = 4 if case["dtype"] == "fp32" else 2
        matrices = case["experts"] if case["layout"] == "TN" else _reached(case)
        return {"bytes": size * (rows * (k + n) + matrices * k * n), "flops": flops}
    if op == "mx_quant":
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": case["m"] * case["k"] * (2.0 * size), "flops": 4.0 * case["m"] * case["k"]}
    m, n, k = case["m"], case["n"], case["k"]
    size = 4 if case["dtype"] == "fp32" else 2
    return {"bytes": (m + n) * k * (0.5 + 1.0 / BLOCK) + size * m * n, "flops": 2.0 * m * n * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, apart from the plain forms
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "grouped":
        a, b = st["a"].double(), st["b"]
        owner = torch.bucketize(torch.arange(a.shape[0], device="cuda"), st["offsets"].long()[1:], right=True)
        if case["layout"] == "TN":
            out = torch.zeros((case["experts"], a.shape[1], b.shape[1]), dtype=torch.float64, device="cuda")
            for e in range(case["experts"]):
                rows = (owner == e).nonzero()[:, 0]
                out[e] = torch.mm(a[rows].t().contiguous(), b[rows].double())
            return out
        out = torch.zeros((a.shape[0], case["n"]), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            rows = (owner == e).nonzero()[:, 0]
            w = b[e].double()
            out[rows] = torch.mm(a[rows], w if case["layout"] == "NN" else w.t().contiguous())
        return out
    if op == "int4":
        x, n, k = st["x"].double(), case["n"], case["k"]
        owner = torch.bucketize(torch.arange(x.shape[0], device="cuda"), st["offsets"].long()[1:], right=True)
        out = torch.zeros((x.shape[0], n), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            rows = (owner == e).nonzero()[:, 0]
            if rows.numel() == 0:
                continue
            words = st["qweight"][e].long() & 0xFFFFFFFF
            s = st["scales"][e].double()
            z = torch.zeros((k // GROUP, n), dtype=torch.float64, device="cuda")
            if st["qzeros"] is not None:
                zw = st["qzeros"][e].long() & 0xFFFFFFFF
                for t in range(8):
                    z[:, t::8] = ((zw >> (4 * t)) % 16).double()
            w = torch.empty((k, n), dtype=torch.float64, device="cuda")
            for t in range(8):
                w[t::8] = ((words >> (4 * t)) % 16).double()
            w = ((w.view(k // GROUP, GROUP, n) - z[:, None, :]) * s[:, None, :]).view(k, n)
            out[rows] = torch.mm(x[rows], w)
        return out
    if op == "mx_quant":
        # nearest point of the block's own grid, by distance (ties to the even code)
        x = st["x"].double().cpu().numpy().reshape(-1, BLOCK)
        top = np.abs(x).max(axis=1)
        ex = np.full(top.shape, -127.0)
        ex[top > 0] = np.clip(np.floor(np.log2(top[top > 0])) - 2, -127, 127)
        grid = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
        out = np.empty_like(x)
        for lo in range(0, x.shape[0], 1 << 16):
            u = np.abs(x[lo:lo + (1 << 16)]) / np.exp2(ex[lo:lo + (1 << 16), None])
            best, dist = np.zeros(u.shape, dtype=np.int8), np.abs(u)
            for c in range(1, 8):
                d = np.abs(u - grid[c])
                take = (d < dist) | ((d == dist) & (c % 2 == 0))
                best[take], dist[take] = c, d[take]
            out[lo:lo + (1 << 16)] = np.copysign(grid[best], x[lo:lo + (1 << 16)]) * np.exp2(ex[lo:lo + (1 << 16), None])
        return torch.from_numpy(out.reshape(case["m"], case["k"])).cuda()
    vals = []
    for codes, scales in (st["a"], st["b"]):
        full = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device="cuda")
        for half in range(2):
            nib = (codes.long() >> (4 * half)) % 16
            e, man = (nib >> 1) % 4, (nib % 2).double()
            mag = torch.where(e == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2(e.double() - 1.0))
            full[:, half::2] = torch.where(nib >= 8, -mag, mag)
        full.view(codes.shape[0], -1, BLOCK).mul_(torch.exp2(scales.double() - 127.0)[:, :, None])
        vals.append(full)
    return torch.mm(vals[0], vals[1].t().contiguous())
