"""The microscaled (MX) operators, as cases for timing and comparison.

Four operators: quantisation to MX blocks and back, the RMS norm with a
residual whose output is MX, the product of MX activations with an MXFP4 weight,
and that product grouped by expert. With ``own`` false ``run`` computes them in
elementary torch operations; with ``own`` true it makes the library's calls.

An MX block is 32 consecutive elements of a row that share the scale 2^e, stored
as the byte e + 127. Elements are e2m1 (4 bits, two per byte, the lower index in
the low nibble) or e4m3 (one byte). Rows are padded to a multiple of 128
elements (zero codes), and the scale bytes of four consecutive blocks of a row
stand together: scales[k / 128][row][(k / 32) % 4].
"""
import math
import random

import torch

own = False

EMAX = {"e2m1": 2, "e4m3": 8}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LARGEST = 2 * 4096 * 11008 * 4096  # operations of the largest listed product


def listed():
    return [
        # a merged 11008x4096 weight (the 7B up projection) on its way to serving
        {"name": "quantize-w-11008x4096", "op": "quantize", "format": "e2m1", "rows": 11008, "cols": 4096},
        # the input of a down projection for 333 prompt tokens; 11008 + 32 columns: the last 128 are not full
        {"name": "quantize-x-333x11040", "op": "quantize", "format": "e4m3", "rows": 333, "cols": 11040},
        # one token's norm before a projection: latency
        {"name": "norm-1x4096", "op": "norm", "format": "e4m3", "rows": 1, "cols": 4096, "residual": True},
        # a prefill of 4 x 1024 tokens
        {"name": "norm-4096x4096", "op": "norm", "format": "e4m3", "rows": 4096, "cols": 4096, "residual": True},
        # the first norm of a model (nothing to add), odd sizes, 4-bit output
        {"name": "norm-517x5152", "op": "norm", "format": "e2m1", "rows": 517, "cols": 5152, "residual": False},
        # decode: one token through the up projection, bound by the weight's bytes
        {"name": "linear-1x11008x4096", "op": "linear", "format": "e4m3", "rows": 1, "n": 11008, "k": 4096},
        # decode of 16 sequences through the down projection
        {"name": "linear-16x4096x11008", "op": "linear", "format": "e4m3", "rows": 16, "n": 4096, "k": 11008},
        # a short ragged prefill with 4-bit activations, odd sizes
        {"name": "linear-333x4100x4128", "op": "linear", "format": "e2m1", "rows": 333, "n": 4100, "k": 4128},
        # a prefill of 4 x 1024 tokens, bound by the tensor cores
        {"name": "linear-4096x11008x4096", "op": "linear", "format": "e4m3", "rows": 4096, "n": 11008, "k": 4096},
        # one token sent to 8 of 64 experts: 8 rows, most experts empty
        {"name": "grouped-8-of-64", "op": "grouped", "format": "e4m3", "rows": 8, "n": 2048, "k": 2048, "experts": 64,
         "routing": 1},
        # a batch of short prompts over 8 experts, uneven, odd sizes
        {"name": "grouped-1000-of-8", "op": "grouped", "format": "e4m3", "rows": 1000, "n": 4100, "k": 4128,
         "experts": 8, "routing": 2},
        # a prefill of 4096 tokens, two experts each of 16
        {"name": "grouped-8192-of-16", "op": "grouped", "format": "e4m3", "rows": 8192, "n": 4096, "k": 4096,
         "experts": 16, "routing": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "norm", "linear", "grouped"))
    fmt = rng.choice(("e2m1", "e4m3"))
    if op == "quantize":
        cols = 32 * _log(rng, 4, 512)
        return {"op": op, "format": fmt, "rows": _log(rng, 1, max(1, min(20000, 11008 * 4096 // cols))), "cols": cols}
    if op == "norm":
        cols = 32 * _log(rng, 8, 512)
        return {"op": op, "format": fmt, "rows": _log(rng, 1, max(1, min(8192, 4096 * 4096 // cols))), "cols": cols,
                "residual": rng.random() < 0.7}
    if op == "linear":
        n, k = _log(rng, 100, 11008), 32 * _log(rng, 8, 344)
        return {"op": op, "format": fmt, "rows": _log(rng, 1, min(4096, LARGEST // (2 * n * k))), "n": n, "k": k}
    experts = rng.choice((1, 3, 8, 16, 40, 64))
    n, k = _log(rng, 100, 4096), 32 * _log(rng, 8, 128)
    return {"op": op, "format": fmt, "rows": _log(rng, 1, 8192), "n": n, "k": k, "experts": experts,
            "routing": rng.randrange(1, 1 << 20)}


def _sizes(case):
    """Rows of each expert: a softmax of random preferences, as routers give them; some experts get none."""
    rng = random.Random(case["routing"])
    liking = [math.exp(rng.gauss(0.0, 1.0)) for _ in range(case["experts"])]
    if case["rows"] <= case["experts"]:  # one token sent to distinct experts
        sizes = [0] * case["experts"]
        for e in rng.sample(range(case["experts"]), case["rows"]):
            sizes[e] = 1
        return sizes
    cuts, total, run_ = [], sum(liking), 0.0
    for v in liking:
        run_ += v
        cuts.append(int(round(case["rows"] * run_ / total)))
    return [b - a for a, b in zip([0] + cuts[:-1], cuts)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, rows, cols):
    """Normal values with a few channels that are larger, as activations of language models have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = 1.0 + 20.0 * (torch.rand(cols, generator=g, device="cuda") < 0.01).float()
    return (x * loud).to(torch.bfloat16)


def _round_e2m1(v):
    a = v.abs()
    step = 0.5 + 0.5 * (a >= 2).float() + 1.0 * (a >= 4).float()
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)


def _blocks(v, fmt):
    """fp32 [rows, cols] -> (elements, exponents) with v ~ elements * 2^exponents, [rows, cols / 32, 32] and [rows, cols / 32]."""
    b = v.view(v.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - EMAX[fmt], -127).clamp(-127, 127)
    u = torch.ldexp(b, -e.unsqueeze(-1))
    if fmt == "e2m1":
        return _round_e2m1(u), e
    return u.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float(), e


def _values(v, fmt):
    q, e = _blocks(v, fmt)
    return torch.ldexp(q, e.unsqueeze(-1)).view(v.shape)


def _store_weight(w):
    """fp32 [rows, cols] -> the storage of an MXFP4 weight (codes, scales)."""
    rows, cols = w.shape
    padded = -(-cols // 128) * 128
    q, e = _blocks(w, "e2m1")
    table = torch.tensor(E2M1, device=w.device)
    code = torch.searchsorted(table, q.abs().contiguous()) + 8 * torch.signbit(q)
    code = torch.nn.functional.pad(code.view(rows, cols).to(torch.uint8), (0, padded - cols))
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    scales = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, (padded - cols) // 32), value=127)
    return codes.contiguous(), scales.view(rows, padded // 128, 4).permute(1, 0, 2).contiguous()


def _load_weight(codes, scales, rows, cols, first=0, dtype=torch.float32):
    """Rows [first, first + rows) of a stored MXFP4 weight, decoded."""
    c = codes[first:first + rows]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=c.device, dtype=dtype)
    q = table[torch.stack((c & 15, c >> 4), -1).view(rows, -1).int()]
    e = scales[:, first:first + rows].permute(1, 0, 2).reshape(rows, -1, 1).int() - 127
    return torch.ldexp(q.view(rows, -1, 32), e).view(rows, -1)[:, :cols]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "quantize":
        s["x"] = _activations(g, case["rows"], case["cols"]) if case["format"] == "e4m3" else \
            (0.02 * torch.randn(case["rows"], case["cols"], generator=g, device="cuda")).to(torch.bfloat16)
    elif case["op"] == "norm":
        s["x"] = _activations(g, case["rows"], case["cols"])
        s["res"] = _activations(g, case["rows"], case["cols"]) if case["residual"] else None
        s["gamma"] = (1.0 + 0.1 * torch.randn(case["cols"], generator=g, device="cuda")).to(torch.bfloat16)
        s["eps"] = 1e-5
    else:
        experts = case.get("experts", 1)
        s["x"] = _activations(g, case["rows"], case["k"])
        parts = [_store_weight((0.02 * torch.randn(case["n"], case["k"], generator=g, device="cuda"))
                               .to(torch.bfloat16).float()) for _ in range(experts)]
        s["codes"] = torch.cat([p[0] for p in parts])
        s["scales"] = torch.cat([p[1] for p in parts], 1)
        if case["op"] == "grouped":
            s["sizes"] = _sizes(case)
            s["offsets"] = torch.tensor([sum(s["sizes"][:e]) for e in range(experts + 1)], dtype=torch.int32,
                                        device="cuda")
    return s


def _run_own(s):
    import bit_nf4_quantized_absmax_b200 as q
    fmt = q.MX_E2M1 if s["format"] == "e2m1" else q.MX_E4M3
    if s["op"] == "quantize":
        return q.qlora_dequantize_mx(q.qlora_quantize_mx(s["x"], fmt))
    if s["op"] == "norm":
        y, h = q.qlora_rmsnorm_mx(s["x"], s["gamma"], s["eps"], fmt, residual=s["res"])
        return q.qlora_dequantize_mx(y), h
    w = q.MXTensor(s["codes"], s["scales"], s["codes"].shape[0], s["k"], q.MX_E2M1)
    if s["op"] == "linear":
        return q.qlora_mx_linear_fwd(s["x"], w, x_format=fmt)
    return q.qlora_mx_grouped_fwd(s["x"], w, s["offsets"], x_format=fmt)


def run(s):
    if own:
        return _run_own(s)
    fmt = s["format"]
    if s["op"] == "quantize":
        return _values(s["x"].float(), fmt).to(torch.bfloat16)
    if s["op"] == "norm":
        h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(torch.bfloat16)
        f = h.float()
        y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"]) * s["gamma"].float()
        return _values(y, fmt).to(torch.bfloat16), None if s["res"] is None else h
    x = _values(s["x"].float(), fmt)
    if s["op"] == "linear":
        return (x @ _load_weight(s["codes"], s["scales"], s["n"], s["k"]).T).to(torch.bfloat16)
    y = torch.empty(s["rows"], s["n"], dtype=torch.bfloat16, device=x.device)
    at = 0
    for e, m in enumerate(s["sizes"]):
        if m:
            w = _load_weight(s["codes"], s["scales"], s["n"], s["k"], e * s["n"])
            y[at:at + m] = x[at:at + m] @ w.T
            at += m
    return y


def work(case):
    bits = 0.5 + 1 / 32 if case["format"] == "e2m1" else 1 + 1 / 32
    if case["op"] == "quantize":  # bf16 in; the codes and their values out
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 + bits + 2), "flops": 0}
    if case["op"] == "norm":  # x (and the residual) in; the sum, the codes and their values out
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 + (4 if case["residual"] else 0) + bits + 2) + 2 * case["cols"], "flops": 0}
    used = sum(1 for m in _sizes(case) if m) if case["op"] == "grouped" else 1
    m, n, k = case["rows"], case["n"], case["k"]
    return {"bytes": used * n * k * (0.5 + 1 / 32) + 2 * m * k + 2 * m * n, "flops": 2 * m * n * k}


def _exact_values(v, fmt):
    """The MX values of fp64 [rows, cols], from the format's definition: the spacing of the element type's values at
    each magnitude, nearest with ties to even."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    bits, low, top = (1, 0, 6.0) if fmt == "e2m1" else (3, -6, 448.0)
    floor_log2 = lambda a: torch.frexp(a).exponent.double() - 1  # noqa: E731
    e = torch.where(amax > 0, floor_log2(amax) - EMAX[fmt], -127.0).clamp(-127, 127)
    u = b * torch.exp2(-e)
    spacing = torch.exp2(floor_log2(u.abs()).clamp(min=low) - bits)
    spacing = torch.where(u == 0, torch.ones_like(u), spacing)
    return ((torch.round(u / spacing) * spacing).clamp(-top, top) * torch.exp2(e)).view(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    fmt = case["format"]
    if case["op"] == "quantize":
        return _exact_values(s["x"].double(), fmt)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["res"] is not None:
            h = (h + s["res"].double()).to(torch.bfloat16).double()  # the stored sum is the norm's input
        y = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / case["cols"] + s["eps"]) * s["gamma"].double()
        return _exact_values(y, fmt), None if s["res"] is None else s["x"].double() + s["res"].double()
    x = _exact_values(s["x"].double(), fmt)
    sizes = s["sizes"] if case["op"] == "grouped" else [case["rows"]]
    out, at = [], 0
    for e, m in enumerate(sizes):
        if m:
            w = _load_weight(s["codes"], s["scales"], case["n"], case["k"], e * case["n"], torch.float64)
            out.append(x[at:at + m] @ w.transpose(0, 1))
            at += m
    return torch.cat(out)
