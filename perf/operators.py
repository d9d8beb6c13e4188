"""The microscaled operators, measured: block-scaled quantisation and its read-back, the root-mean-square norm with the
residual's addition whose output is quantised in 8 bits, and the product of microscaled activations with 4-bit
microscaled weights.

Format (blocks of 32 along a row): an element is e2m1 (4 bits, +-{0, .5, 1, 1.5, 2, 3, 4, 6}) or e4m3 (8 bits, up to
448), a scale is a power of two, E = floor(log2(max |x|)) - (2 or 8), held as E + 127.  Codes are [rows, row bytes],
rows padded with zeros to 128 elements, two 4-bit codes a byte (even element in the low half).  Scales come in tiles of
128 rows x 4 blocks: byte [row / 128][block / 4][row % 32][row / 32 % 4][block % 4].
"""

import math

import torch

own = False

BLOCK = 32
EPS = 1e-6
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the smallest layer's batch (64 tokens of 256 channels, fp32): latency of quantising and reading back
        {"name": "quantize 64x256 a4 fp32", "op": "quantize", "rows": 64, "d": 256, "bits": 4, "dtype": "fp32"},
        # a ragged batch of a width that is no multiple of 128, in 8 bits
        {"name": "quantize 1001x2016 a8", "op": "quantize", "rows": 1001, "d": 2016, "bits": 8, "dtype": "bf16"},
        # the video batch (21 x 39 x 40 latent patches) before a 4-bit projection
        {"name": "quantize 32760x5120 a4", "op": "quantize", "rows": 32760, "d": 5120, "bits": 4, "dtype": "bf16"},
        # one token (a step of a stream): the norm's latency
        {"name": "norm 1x5120", "op": "norm", "rows": 1, "d": 5120, "bits": 8, "dtype": "bf16", "residual": True},
        # an fp32 residual stream, ragged rows and width, no addition (the first block)
        {"name": "norm 777x2080 fp32", "op": "norm", "rows": 777, "d": 2080, "bits": 8, "dtype": "fp32", "residual": False},
        # the MLP-down input's width at the image batch
        {"name": "norm 4608x12288", "op": "norm", "rows": 4608, "d": 12288, "bits": 8, "dtype": "bf16", "residual": True},
        # a single token through the widest layer: the weights' stream
        {"name": "linear 1 13824-5120 a4", "op": "linear", "rows": 1, "d": 13824, "d_out": 5120, "bits": 4, "y": "fp32"},
        # the stress layer's smallest batch, 8-bit activations
        {"name": "linear 256 13824-5120 a8", "op": "linear", "rows": 256, "d": 13824, "d_out": 5120, "bits": 8, "y": "bf16"},
        # the stress layer at an ordinary batch, 8-bit activations
        {"name": "linear 4096 13824-5120 a8", "op": "linear", "rows": 4096, "d": 13824, "d_out": 5120, "bits": 8, "y": "bf16"},
        # the video projection, 4-bit activations: the largest product
        {"name": "linear 32760 5120-5120 a4", "op": "linear", "rows": 32760, "d": 5120, "d_out": 5120, "bits": 4, "y": "bf16"},
        # the chain of a block's input: residual, norm, 8-bit codes, projection; ragged in all three sizes
        {"name": "block 333 2016-1040", "op": "block", "rows": 333, "d": 2016, "d_out": 1040, "bits": 8, "dtype": "bf16"},
        # the same at the image batch with the MLP-up ratio
        {"name": "block 4608 2560-10240", "op": "block", "rows": 4608, "d": 2560, "d_out": 10240, "bits": 8, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "linear", "linear", "block"])
    while True:
        rows, d, d_out = _log(rng, 1, 32760), 32 * _log(rng, 1, 432), 16 * _log(rng, 1, 768)
        if op in ("quantize", "norm"):
            if rows * d > 32760 * 5120:
                continue
            case = {"op": op, "rows": rows, "d": d, "bits": rng.choice([4, 8]) if op == "quantize" else 8,
                    "dtype": rng.choice(["bf16", "bf16", "fp32"])}
            if op == "norm":
                case["residual"] = rng.random() < 0.75
            return case
        if rows * d * d_out > 32760 * 5120 * 5120 or rows * max(d, d_out) > 32760 * 5120:
            continue
        case = {"op": op, "rows": rows, "d": d, "d_out": d_out}
        if op == "linear":
            return {**case, "bits": rng.choice([4, 8]), "y": rng.choice(["bf16", "bf16", "fp32"])}
        return {**case, "bits": 8, "dtype": rng.choice(["bf16", "bf16", "fp32"])}


# ------------------------------------------------------------------ the plain forms
def _grid(bits):
    """(mantissa bits, least exponent, largest exponent, largest value) of an element type."""
    return (1, 0, 2, 6.0) if bits == 4 else (3, -6, 8, 448.0)


def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127], from its bits (torch.pow and torch.ldexp may be an ulp off on the GPU)."""
    e = e.int()
    return torch.where(e < -126, 1 << 22, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(v, bits):
    """fp32 [rows, d] -> (element values [rows, d / 32, 32], scale exponents [rows, d / 32, 1])."""
    m, emin, emax, top = _grid(bits)
    b = v.reshape(v.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - emax, -127).clamp(min=-127)
    w = b * _pow2(-e)
    step = (torch.frexp(w).exponent - 1).clamp(min=emin) - m
    return (torch.round(w * _pow2(-step)) * _pow2(step)).clamp(-top, top), e


def _values(v, bits):
    """fp32 [rows, d] -> the fp32 values that its codes stand for."""
    q, e = _blocks(v, bits)
    return (q * _pow2(e)).reshape(v.shape)


def _norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["gain"].float()
    return h, n


def _read(codes, scales, rows, d, bits):
    """The fp32 values [rows, d] of codes and scales."""
    if bits == 4:
        c = torch.stack((codes & 15, codes >> 4), -1).reshape(rows, -1).int()
        mag, sign = c & 7, 1 - 2 * (c >> 3)
        v = torch.where(mag < 2, 0.5 * mag, (1.0 + 0.5 * (mag & 1)) * _pow2((mag >> 1) - 1)) * sign
    else:
        v = codes.view(torch.float8_e4m3fn).float()
    e = scales.permute(0, 3, 2, 1, 4).reshape(scales.shape[0] * 128, -1)[:rows].int() - 127
    v = v.reshape(rows, -1, BLOCK)
    return (v * _pow2(e.unsqueeze(-1))).reshape(rows, -1)[:, :d]


# ------------------------------------------------------------------ inputs
def _codes(v, bits):
    """Codes and scales of fp32 [rows, d], laid out as the module's docstring says."""
    rows, d = v.shape
    q, e = _blocks(v, bits)
    kq, rb = -(-d // 128), -(-rows // 128)
    if bits == 4:
        a = q.abs()
        c = (torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)) + 8 * torch.signbit(q)).to(torch.uint8)
    else:
        c = q.to(torch.float8_e4m3fn).view(torch.uint8)
    c = torch.nn.functional.pad(c.reshape(rows, d), (0, kq * 128 - d))
    codes = (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous() if bits == 4 else c.contiguous()
    t = torch.nn.functional.pad((e.squeeze(-1) + 127).to(torch.uint8), (0, kq * 4 - d // BLOCK, 0, rb * 128 - rows))
    return codes, t.reshape(rb, 4, 32, kq, 4).permute(0, 3, 2, 1, 4).contiguous()


def _activations(g, rows, d):
    """Gaussian rows with a log-normal scale each and 1 % of channels twenty times as large, as a transformer's are."""
    x = torch.randn(rows, d, generator=g, device="cuda")
    ch = torch.randperm(d, generator=g, device="cuda")[: max(1, d // 100)]
    x[:, ch] *= 20.0
    return x.mul_(torch.exp(torch.randn(rows, 1, generator=g, device="cuda")))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows, d, bits = case["rows"], case["d"], case["bits"]
    s = {"case": case, "rows": rows, "d": d, "bits": bits}
    if case["op"] == "linear":
        s["codes"], s["scales"] = _codes(_activations(g, rows, d).bfloat16().float(), bits)
    else:
        s["x"] = _activations(g, rows, d).to(DT[case["dtype"]])
    if case["op"] in ("norm", "block"):
        has = case.get("residual", True)
        s["residual"] = _activations(g, rows, d).mul_(2).to(DT[case["dtype"]]) if has else None
        s["gain"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    if case["op"] in ("linear", "block"):
        s["y"] = DT[case.get("y", "bf16")]
        w = 0.02 * torch.randn(case["d_out"], d, generator=g, device="cuda")
        s["wcodes"], s["wscales"] = _codes(w, 4)
        if own:  # the handle that a program keeps for a layer
            from quantized_linear_token_b200 import binding as B
            s["layer"] = B.oq_layer_create(d, case["d_out"], 0, bits, 4, B.OQ_FLAG_MICROSCALED)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op, rows, d, bits = s["case"]["op"], s["rows"], s["d"], s["bits"]
    if op == "quantize":
        return {"values": _values(s["x"].float(), bits).bfloat16()}
    if op == "norm":
        h, n = _norm(s)
        out = {"values": _values(n, bits).bfloat16()}
        return out if s["residual"] is None else {**out, "residual": h.to(s["x"].dtype)}
    w = _read(s["wcodes"], s["wscales"], s["case"]["d_out"], d, 4)
    if op == "linear":
        return {"y": (_read(s["codes"], s["scales"], rows, d, bits) @ w.T).to(s["y"])}
    h, n = _norm(s)
    return {"y": (_values(n, bits) @ w.T).to(s["y"]), "residual": h.to(s["x"].dtype)}


def _run_own(s):
    from quantized_linear_token_b200 import binding as B
    op, d, bits = s["case"]["op"], s["d"], s["bits"]
    if op == "quantize":
        codes, scales = B.oq_mx_quantize(s["x"], bits)
        return {"values": B.oq_mx_dequantize(codes, scales, d, bits, torch.bfloat16)}
    if op == "linear":
        return {"y": B.oq_linear_mx(s["layer"], s["codes"], s["scales"], s["wcodes"], s["wscales"], y_dtype=s["y"])}
    codes, scales, residual = B.oq_rms_norm_mx(s["x"], s["gain"], s["residual"], eps=EPS, bits=bits)
    if op == "norm":
        out = {"values": B.oq_mx_dequantize(codes, scales, d, bits, torch.bfloat16)}
        return out if residual is None else {**out, "residual": residual}
    return {"y": B.oq_linear_mx(s["layer"], codes, scales, s["wcodes"], s["wscales"], y_dtype=s["y"]), "residual": residual}


def work(case):
    rows, d, n = case["rows"], case["d"], case.get("d_out", 0)
    x = rows * d * (4 if case.get("dtype") == "fp32" else 2)
    codes = rows * d * (case["bits"] / 8 + 1 / BLOCK)
    weights = n * d * (0.5 + 1 / BLOCK)
    y = rows * n * (4 if case.get("y") == "fp32" else 2)
    if case["op"] == "quantize":
        return {"bytes": x + 2 * rows * d, "flops": 4 * rows * d}
    if case["op"] == "norm":
        return {"bytes": x * (3 if case["residual"] else 1) + 4 * d + 2 * rows * d, "flops": 10 * rows * d}
    if case["op"] == "linear":
        return {"bytes": codes + weights + y, "flops": 2 * rows * d * n}
    return {"bytes": 3 * x + 4 * d + weights + y, "flops": 2 * rows * d * n + 10 * rows * d}


# ------------------------------------------------------------------ the definitions in 64 bits, written apart
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [(m / 8.0 if e == 0 else 1 + m / 8.0) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127]


def _two(e):
    """2^e in fp64 for whole e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(v, table):
    """|v| -> the nearest entry of an ascending table, halfway to the even index, past its end the last."""
    t = torch.tensor(table, dtype=torch.float64, device=v.device)
    mid = (t[1:] + t[:-1]) / 2
    up, down = torch.searchsorted(mid, v, right=True), torch.searchsorted(mid, v)
    return t[torch.where(up % 2 == 0, up, down)]


def _values64(v, bits):
    rows = []
    for part in v.split(max(1, (1 << 27) // v.shape[1])):
        b = part.reshape(-1, BLOCK)
        amax = b.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200)))
        # log2 may be an ulp off next to a whole number
        e = torch.where(_two(e) > amax, e - 1, torch.where(_two(e + 1) <= amax, e + 1, e))
        scale = _two((e - (2 if bits == 4 else 8)).clamp(min=-127))
        w = b / scale
        rows.append((torch.sign(w) * _nearest(w.abs(), E2M1 if bits == 4 else E4M3) * scale).reshape(part.shape))
    return torch.cat(rows)


def _read64(codes, scales, rows, d, bits):
    if bits == 4:
        t = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device=codes.device)
        v = torch.empty(rows, codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
        v[:, 0::2], v[:, 1::2] = t[(codes % 16).long()], t[(codes // 16).long()]
    else:
        nan = [math.nan]
        t = torch.tensor(E4M3 + nan + [-x for x in E4M3] + nan, dtype=torch.float64, device=codes.device)
        v = t[codes.long()]
    i = torch.arange(rows, device=codes.device)[:, None]
    k = torch.arange(d // BLOCK, device=codes.device)[None, :]
    scale = _two(scales[i // 128, k // 4, i % 32, i // 32 % 4, k % 4].long() - 127)
    return v[:, :d] * scale.repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, rows, d, bits = case["op"], s["rows"], s["d"], s["bits"]
    if op == "quantize":
        return {"values": _values64(s["x"].double(), bits)}
    if op != "linear":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        n = h / torch.sqrt(h.square().sum(-1, keepdim=True) / d + EPS) * s["gain"].double()
        a = _values64(n, bits)
    else:
        a = _read64(s["codes"], s["scales"], rows, d, bits)
    if op == "norm":
        return {"values": a} if s["residual"] is None else {"values": a, "residual": h}
    y = a @ _read64(s["wcodes"], s["wscales"], case["d_out"], d, 4).T
    return {"y": y} if op == "linear" else {"y": y, "residual": h}
