"""Attention with a 4-bit cache and the operators beside it, measured: norms of queries and keys for each head with the
position rotation, the append to a paged cache in microscaled e2m1, attention that reads the cache, and the product
with 4-bit weights that have group scales; and a run of them as one step of a stream makes.

Cache: pages of 128 tokens; heads of 64 channels lie two to a group of 128 channels.  [pages, groups, 272, 64] bytes:
  rows 0-127    K codes, a token's 128 channels a row (e2m1, even channel in the low half)
  rows 128-255  V codes transposed, a channel's 128 tokens a row (even token in the low half)
  rows 256-263  K scales (E8M0, one for 32 channels): byte [token % 32][token / 32][block]
  rows 264-271  V scales: byte [token][block]
Sequence b has lens[b] tokens in the cache, token j in page pages[b, j / 128]; the last cu[b + 1] - cu[b] of them are
this call's.

Weights: code c of 4 bits stands for (c - zero) * scale, one bf16 scale and zero (8 where there are none) for `group`
neighbours of a row.  Rows are padded to 128 codes; in a run of 128 (64 bytes) the 32-bit word 4 q + s holds elements
32 s + 8 q to + 7, and its nibble p the element 2 (p % 4) + p / 4 of those.
"""

import math

import torch

own = False

PAGE = 128
BLOCK = 32
EPS = 1e-6
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of a stream, 40 heads: the latency of norm and rotation
        {"name": "rope 1 40+40x128", "op": "rope", "T": 1, "H": 40, "KH": 40, "D": 128, "rot": 128, "inter": True, "dtype": "bf16"},
        # a ragged fp32 batch, narrow heads, part of the channels rotated in halves
        {"name": "rope 1001 24+8x96 fp32", "op": "rope", "T": 1001, "H": 24, "KH": 8, "D": 96, "rot": 64, "inter": False, "dtype": "fp32"},
        # the video batch (21 x 39 x 40 latent patches) of the 5120-channel layer
        {"name": "rope 32760 40+40x128", "op": "rope", "T": 32760, "H": 40, "KH": 40, "D": 128, "rot": 128, "inter": True, "dtype": "bf16"},
        # a new token for each of 16 streams, grouped heads
        {"name": "append 16x1 32+8x128", "op": "append", "B": 16, "n": 1, "len": 4096, "H": 32, "KH": 8, "D": 128, "inter": False, "ragged": True, "dtype": "bf16"},
        # a latent frame (39 x 40 patches) of the video batch joins the cache
        {"name": "append 1x1560 40+40x128", "op": "append", "B": 1, "n": 1560, "len": 7800, "H": 40, "KH": 40, "D": 128, "inter": True, "ragged": False, "dtype": "bf16"},
        # one token over a short cache, narrow heads: latency
        {"name": "attend 1x1 of 300 16/4x64", "op": "attend", "B": 1, "n": 1, "len": 300, "H": 16, "KH": 4, "D": 64, "causal": True, "window": 0, "ragged": False},
        # one token over the whole video's cache, a key head for each query head
        {"name": "attend 1x1 of 32760 40/40x128", "op": "attend", "B": 1, "n": 1, "len": 32760, "H": 40, "KH": 40, "D": 128, "causal": True, "window": 0, "ragged": False},
        # a served batch of streams of different lengths, grouped heads
        {"name": "attend 64x1 of 8192 32/8x128", "op": "attend", "B": 64, "n": 1, "len": 8192, "H": 32, "KH": 8, "D": 128, "causal": True, "window": 0, "ragged": True},
        # a latent frame over the cache of five, its own among them: every patch sees every other
        {"name": "attend 1x1560 of 7800 40/40x128", "op": "attend", "B": 1, "n": 1560, "len": 7800, "H": 40, "KH": 40, "D": 128, "causal": False, "window": 0, "ragged": False},
        # one conditioning vector through the widest layer: the weights' stream
        {"name": "w4g 1 13824-5120", "op": "w4g", "T": 1, "d": 13824, "d_out": 5120, "group": 128, "zeros": False, "dtype": "bf16", "y": "fp32"},
        # a few ragged tokens, the finest groups with zeros
        {"name": "w4g 13 5120-13824 zeros", "op": "w4g", "T": 13, "d": 5120, "d_out": 13824, "group": 32, "zeros": True, "dtype": "bf16", "y": "bf16"},
        # a step of eight streams: QKV projection, norm, rotation and append, attention, output projection
        {"name": "step 8 of 4096 32/8x128", "op": "step", "B": 8, "n": 1, "len": 4096, "H": 32, "KH": 8, "D": 128, "inter": False, "ragged": True, "group": 128, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "w4g", "w4g", "step"])
    while True:
        if op == "rope":
            D = rng.choice([64, 96, 128, 256])
            c = {"op": op, "T": _log(rng, 1, 32760), "H": rng.randint(1, 48), "KH": rng.randint(1, 48), "D": D,
                 "rot": rng.choice([D, D, D // 2]), "inter": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
            if c["T"] * (c["H"] + c["KH"]) * D * (2 if c["dtype"] == "fp32" else 1) <= 32760 * 80 * 128:
                return c
            continue
        if op == "w4g":
            c = {"op": op, "T": _log(rng, 1, 32), "d": 128 * _log(rng, 1, 108), "d_out": 16 * _log(rng, 4, 1920),
                 "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5,
                 "dtype": rng.choice(["bf16", "bf16", "fp32"]), "y": rng.choice(["bf16", "fp32"])}
            if c["d"] * c["d_out"] <= 13824 * 5120:
                return c
            continue
        KH, D = rng.choice([1, 2, 3, 4, 8, 24, 40]), rng.choice([64, 128])
        H = KH * rng.choice([1, 2, 4, 5, 8])
        if op == "step":
            c = {"op": op, "B": _log(rng, 1, 16), "n": 1, "len": _log(rng, 512, 16384), "H": H, "KH": KH, "D": D,
                 "inter": rng.random() < 0.5, "ragged": rng.random() < 0.7, "group": rng.choice([64, 128]), "dtype": "bf16"}
            if H * D % 128 == 0 and H * D <= 8192 and c["B"] * c["len"] * KH * D <= 16 * 16384 * 8 * 128:
                return c
            continue
        n, B = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 2048)]), _log(rng, 1, 64)
        c = {"op": op, "B": B, "n": n, "len": max(n, _log(rng, 1, 32760)), "H": H, "KH": KH, "D": D,
             "ragged": rng.random() < 0.7}
        if op == "append":
            if B * n * H * D <= 1560 * 40 * 128 and B * c["len"] * KH * D <= 64 * 8192 * 8 * 128:
                return {**c, "inter": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
        elif B * n * H * c["len"] * D <= 1560 * 40 * 7800 * 128 and B * c["len"] * KH * D <= 64 * 8192 * 8 * 128:
            return {**c, "causal": n == 1 or rng.random() < 0.5, "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)])}


def _lengths(case):
    """(tokens of this call, tokens in the cache with them) of each sequence."""
    n, ln = [], []
    for b in range(case["B"]):
        n.append(1 + (case["n"] - 1 + 5 * b) % case["n"] if case["ragged"] else case["n"])
        ln.append(max(n[-1], case["len"] - (7919 * b) % (case["len"] // 2 + 1)) if case["ragged"] else case["len"])
    return n, ln


# ------------------------------------------------------------------ formats
def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127], from its bits."""
    e = e.int()
    return torch.where(e < -126, 1 << 22, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(v):
    """fp32 or fp64 [..., d] -> (e2m1 values [..., d / 32, 32] in fp32, scale exponents [..., d / 32, 1])."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(min=-127)
    w = b * _pow2(-e).to(b.dtype)
    step = (torch.frexp(w).exponent - 1).clamp(min=0) - 1
    return (torch.round(w * _pow2(-step).to(b.dtype)) * _pow2(step).to(b.dtype)).clamp(-6, 6).float(), e


def _nibbles(q):
    """e2m1 values -> codes."""
    a = q.abs()
    return (torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)) + 8 * torch.signbit(q)).to(torch.uint8)


def _e2m1(c):
    c = c.int()
    mag, sign = c & 7, 1 - 2 * (c >> 3)
    return torch.where(mag < 2, 0.5 * mag, (1.0 + 0.5 * (mag & 1)) * _pow2((mag >> 1) - 1)) * sign


def _unpack(b):
    return torch.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1)


def _pack(c):
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()


def _fill(case, g, lens):
    """A cache of random tokens: (cache, pages).  The pages lie in random order and a few belong to no sequence."""
    need = [-(-n // PAGE) for n in lens]
    total, groups = sum(need) + 3, -(-case["KH"] * case["D"] // 128)
    cache = torch.empty(total, groups, 272, 64, dtype=torch.uint8, device="cuda")
    for p0 in range(0, total, 512):
        part = cache[p0:p0 + 512]
        P = part.shape[0]
        # keys with a few strong channels, values even
        k = torch.randn(P, groups, PAGE, 128, generator=g, device="cuda")
        k *= torch.where(torch.rand(groups, 1, 128, generator=g, device="cuda") < 0.03, 6.0, 1.0)
        q, e = _blocks(k)
        part[:, :, :128] = _pack(_nibbles(q).reshape(P, groups, PAGE, 128))
        part[:, :, 256:264] = (e.squeeze(-1) + 127).to(torch.uint8).reshape(P, groups, 4, 32, 4).transpose(2, 3).reshape(P, groups, 8, 64)
        q, e = _blocks(torch.randn(P, groups, PAGE, 128, generator=g, device="cuda"))
        part[:, :, 128:256] = _pack(_nibbles(q).reshape(P, groups, PAGE, 128).transpose(2, 3))
        part[:, :, 264:] = (e.squeeze(-1) + 127).to(torch.uint8).reshape(P, groups, 8, 64)
    order = torch.randperm(total, generator=g, device="cuda").int()
    pages = torch.zeros(case["B"], max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        pages[b, :m] = order[at:at + m]
        at += m
    return cache, pages


def _values(cache, pages, n, KH, D):
    """The first n tokens of a sequence's pages -> K, V [n, KH, D] in fp32."""
    c = cache[pages[:-(-n // PAGE)].long()]
    P, G = c.shape[:2]
    k, v = _e2m1(_unpack(c[:, :, :128])), _e2m1(_unpack(c[:, :, 128:256])).transpose(2, 3)
    ks = c[:, :, 256:264].reshape(P, G, 32, 4, 4).transpose(2, 3).reshape(P, G, PAGE, 4)
    out = []
    for x, s in ((k, ks), (v, c[:, :, 264:].reshape(P, G, PAGE, 4))):
        x = x.reshape(P, G, PAGE, 4, BLOCK) * _pow2(s.int() - 127).unsqueeze(-1)
        x = x.reshape(P, G, PAGE, 128).permute(0, 2, 1, 3).reshape(P * PAGE, -1)
        out.append(x[:n, :KH * D].reshape(n, KH, D))
    return out


def _group_weights(w, group, zeros):
    """fp32 rows [d_out, d] (d a multiple of 128) -> (codes [d_out, d / 2] bytes, scales bf16, zeros or None)."""
    n, d = w.shape
    b = w.reshape(n, -1, group)
    if zeros:
        lo, hi = b.amin(-1, keepdim=True).clamp(max=0), b.amax(-1, keepdim=True).clamp(min=0)
        s = ((hi - lo) / 15).bfloat16()
        z = torch.round(-lo / s.float()).clamp(0, 15)
    else:
        s, z = (b.abs().amax(-1, keepdim=True) / 7).bfloat16(), torch.full_like(b[..., :1], 8)
    c = (torch.round(b / s.float()) + z).clamp(0, 15).to(torch.uint8).reshape(n, d // 128, 4, 4, 4, 2)
    # [run][s][q][element / 2][element % 2] -> [run][q][s][nibble]
    c = c.permute(0, 1, 3, 2, 5, 4).reshape(n, d)
    return _pack(c), s.squeeze(-1).contiguous(), z.squeeze(-1).to(torch.uint8).contiguous() if zeros else None


# ------------------------------------------------------------------ inputs
def _rope_table(positions, rot):
    """(cos, sin) of position / 10000^(2 i / rot) [positions, rot / 2, 2]."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * torch.exp(i * (-2 * math.log(1e4) / rot))
    return torch.stack((a.cos(), a.sin()), -1).float()


def _linear_weights(g, d, d_out, group, zeros):
    return _group_weights(0.02 * torch.randn(d_out, d, generator=g, device="cuda"), group, zeros)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "w4g":
        s["x"] = torch.randn(case["T"], case["d"], generator=g, device="cuda").to(DT[case["dtype"]])
        s["w"] = _linear_weights(g, case["d"], case["d_out"], case["group"], case["zeros"])
        return s
    H, KH, D = case["H"], case["KH"], case["D"]
    if op == "rope":
        T, rot = case["T"], case["rot"]
        s["positions"] = torch.arange(T, dtype=torch.int32, device="cuda")
        s["table"] = _rope_table(T, rot)
    else:
        s["n"], s["lens"] = _lengths(case)
        T, rot = sum(s["n"]), D
        s["cu"] = torch.tensor([sum(s["n"][:b]) for b in range(case["B"] + 1)], dtype=torch.int32, device="cuda")
        s["len"] = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
        s["cache"], s["pages"] = _fill(case, g, s["lens"])
        if op != "attend":
            s["positions"] = torch.cat([torch.arange(m - k, m, dtype=torch.int32, device="cuda")
                                        for k, m in zip(s["n"], s["lens"])])
            s["table"] = _rope_table(max(s["lens"]), rot)
        if own:  # the handle that a program keeps for its heads
            from quantized_linear_token_b200 import binding as B
            s["kv"] = B.oq_kv4_create(H, KH, D)
    if op != "attend":
        s["gq"], s["gk"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in "qk")
    if op == "attend":
        s["q"] = torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
    elif op == "step":
        s["x"] = torch.randn(T, H * D, generator=g, device="cuda").bfloat16()
        s["wqkv"] = _linear_weights(g, H * D, (H + 2 * KH) * D, case["group"], False)
        s["wo"] = _linear_weights(g, H * D, H * D, case["group"], False)
    else:
        # the projection's output: queries, keys (and values) of a token lie in one row
        heads = H + (KH if op == "rope" else 2 * KH)
        x = torch.randn(T, heads, D, generator=g, device="cuda")
        x = x.mul_(torch.exp(0.5 * torch.randn(T, heads, 1, generator=g, device="cuda"))).to(DT[case["dtype"]])
        s["q"], s["k"], s["v"] = x[:, :H], x[:, H:H + KH], x[:, H + KH:]
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _norm_rope(x, gain, table, inter):
    """[T, H, D] of any type, the rows (cos, sin) of its tokens [T, rot / 2, 2]."""
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.to(x.dtype)
    c, t = (table[:, None, :, i].to(x.dtype) for i in (0, 1))
    rot = 2 * c.shape[-1]
    a, b = (n[..., 0:rot:2], n[..., 1:rot:2]) if inter else (n[..., :rot // 2], n[..., rot // 2:rot])
    a, b = a * c - b * t, b * c + a * t
    r = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((r, n[..., rot:]), -1)


def _quantized(x):
    q, e = _blocks(x.reshape(x.shape[0], -1))
    return (q * _pow2(e)).reshape(x.shape)


def _append_plain(s, q, k, v):
    """(q in bf16, the values that k and v have in the cache, in fp32); k in 64 bits: its values lie next to borders
    between codes."""
    case, t = s["case"], s["table"][s["positions"].long()]
    q = _norm_rope(q.float(), s["gq"], t, case["inter"]).bfloat16()
    return q, _quantized(_norm_rope(k.double(), s["gk"], t, case["inter"])), _quantized(v.float())


def _attend_plain(s, q, k_new=None, v_new=None):
    case = s["case"]
    KH, D, G = case["KH"], case["D"], case["H"] // case["KH"]
    y, at = torch.empty_like(q), 0
    for b, (n, ln) in enumerate(zip(s["n"], s["lens"])):
        k, v = _values(s["cache"], s["pages"][b], ln, KH, D)
        if k_new is not None:
            k[ln - n:], v[ln - n:] = k_new[at:at + n], v_new[at:at + n]
        i = torch.arange(ln - n, ln, device="cuda")[:, None]
        j = torch.arange(ln, device="cuda")[None]
        hidden = torch.zeros(n, ln, dtype=torch.bool, device="cuda")
        if case.get("causal", True):
            hidden |= j > i
        if case.get("window", 0):
            hidden |= j <= i - case["window"]
        for h in range(0, KH, step := max(1, (1 << 28) // (G * n * ln))):
            qh = q[at:at + n, h * G:(h + step) * G].float().reshape(n, -1, G, D).permute(1, 2, 0, 3)
            p = qh @ k[:, h:h + step].permute(1, 2, 0)[:, None] * D ** -0.5
            p.masked_fill_(hidden, -math.inf)
            p = torch.exp(p - p.amax(-1, keepdim=True).clamp(min=-1e30))
            o = p @ v[:, h:h + step].transpose(0, 1)[:, None] / p.sum(-1, keepdim=True).clamp(min=1e-30)
            y[at:at + n, h * G:(h + step) * G] = o.permute(2, 0, 1, 3).reshape(n, -1, D).to(y.dtype)
        at += n
    return y


def _linear_plain(x, w, d_out, group, dtype):
    codes, scales, zeros = w
    c = _unpack(codes).reshape(d_out, -1, 4, 4, 2, 4).permute(0, 1, 3, 2, 5, 4).reshape(d_out, -1, group).float()
    c = (c - (8 if zeros is None else zeros.float().unsqueeze(-1))) * scales.float().unsqueeze(-1)
    return (x.float() @ c.reshape(d_out, -1).T).to(dtype)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "w4g":
        return {"y": _linear_plain(s["x"], s["w"], case["d_out"], case["group"], DT[case["y"]])}
    if op == "rope":
        t = s["table"][s["positions"].long()]
        return {x: _norm_rope(s[x].float(), s["g" + x], t, case["inter"]).to(s[x].dtype) for x in "qk"}
    if op == "attend":
        return {"y": _attend_plain(s, s["q"])}
    if op == "append":
        q, k, v = _append_plain(s, s["q"], s["k"], s["v"])
        return {"q": q, "k": k.bfloat16(), "v": v.bfloat16()}
    H, KH, D = case["H"], case["KH"], case["D"]
    x = _linear_plain(s["x"], s["wqkv"], (H + 2 * KH) * D, case["group"], torch.bfloat16).reshape(-1, H + 2 * KH, D)
    o = _attend_plain(s, *_append_plain(s, x[:, :H], x[:, H:H + KH], x[:, H + KH:]))
    return {"y": _linear_plain(o.reshape(-1, H * D), s["wo"], H * D, case["group"], torch.bfloat16)}


def _run_own(s):
    from quantized_linear_token_b200 import binding as B
    case = s["case"]
    op = case["op"]
    if op == "w4g":
        return {"y": B.oq_linear_w4g(s["x"], *s["w"], group=case["group"], y_dtype=DT[case["y"]])}
    if op == "rope":
        q, k = B.oq_qk_norm_rope(s["q"], s["k"], s["gq"], s["gk"], eps=EPS, table=s["table"], positions=s["positions"],
                                 interleaved=case["inter"])
        return {"q": q, "k": k}
    if op == "attend":
        return {"y": B.oq_kv4_attention(s["kv"], s["q"], s["cache"], s["pages"], s["cu"], s["len"], max(s["n"]),
                                        max_len=max(s["lens"]), causal=case["causal"], window=case["window"])}

    def append(q, k, v):
        return B.oq_kv4_append(s["kv"], q, k, v, s["cache"], s["pages"], s["cu"], s["len"], s["gq"], s["gk"], eps=EPS,
                               table=s["table"], positions=s["positions"], interleaved=case["inter"])
    if op == "append":
        q = append(s["q"], s["k"], s["v"])
        k, v = B.oq_kv4_read(s["kv"], s["cache"], s["pages"], s["cu"], s["len"], q.shape[0], dtype=torch.bfloat16)
        return {"q": q, "k": k, "v": v}
    H, KH, D = case["H"], case["KH"], case["D"]
    x = B.oq_linear_w4g(s["x"], *s["wqkv"], group=case["group"], y_dtype=torch.bfloat16).view(-1, H + 2 * KH, D)
    q = append(x[:, :H], x[:, H:H + KH], x[:, H + KH:])
    o = B.oq_kv4_attention(s["kv"], q, s["cache"], s["pages"], s["cu"], s["len"], max(s["n"]), max_len=max(s["lens"]))
    return {"y": B.oq_linear_w4g(o.view(-1, H * D), *s["wo"], group=case["group"], y_dtype=torch.bfloat16)}


def _seen(case):
    """Pairs of a token of this call and a token of the cache that it sees, and cached tokens that any sees."""
    pairs = rows = 0
    for n, ln in zip(*_lengths(case)):
        first = ln
        for i in range(ln - n, ln):
            hi = i + 1 if case.get("causal", True) else ln
            lo = max(0, i - case["window"] + 1) if case.get("window", 0) else 0
            pairs += max(0, hi - lo)
            first = min(first, lo)
        rows += ln - first
    return pairs, rows


def work(case):
    op, size = case["op"], 4 if case.get("dtype") == "fp32" else 2

    def linear(T, d, d_out, group, zeros=False):
        return d * d_out * (0.5 + (3 if zeros else 2) / group), 2 * T * d * d_out
    if op == "w4g":
        b, f = linear(case["T"], case["d"], case["d_out"], case["group"], case["zeros"])
        return {"bytes": b + case["T"] * (case["d"] * size + case["d_out"] * (4 if case["y"] == "fp32" else 2)), "flops": f}
    H, KH, D = case["H"], case["KH"], case["D"]
    if op == "rope":
        x = case["T"] * (H + KH) * D
        return {"bytes": 2 * x * size + 4 * case["T"] * case["rot"], "flops": 8 * x}
    T = sum(_lengths(case)[0])
    if op == "append":
        return {"bytes": T * D * (H * (size + 2) + 2 * KH * (size + 2) + 4), "flops": 10 * T * (H + 2 * KH) * D}
    pairs, rows = _seen(case)
    cache, flops = 2 * rows * KH * D * (0.5 + 1 / BLOCK), 4 * pairs * H * D
    if op == "attend":
        return {"bytes": cache + 4 * T * H * D, "flops": flops}
    b1, f1 = linear(T, H * D, (H + 2 * KH) * D, case["group"])
    b2, f2 = linear(T, H * D, H * D, case["group"])
    return {"bytes": cache + b1 + b2 + 4 * T * H * D, "flops": flops + f1 + f2}


# ------------------------------------------------------------------ the definitions in 64 bits, written apart
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _two(e):
    """2^e in fp64 for whole e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _grid64(x):
    """fp64 [..., d] -> the values of its codes."""
    b = x.reshape(-1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200)))
    e = torch.where(_two(e) > amax, e - 1, torch.where(_two(e + 1) <= amax, e + 1, e))  # log2 may be an ulp off
    scale = _two((e - 2).clamp(min=-127))
    t = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    mid, w = (t[1:] + t[:-1]) / 2, b / scale
    up, down = torch.searchsorted(mid, w.abs(), right=True), torch.searchsorted(mid, w.abs())
    return (torch.sign(w) * t[torch.where(up % 2 == 0, up, down)] * scale).reshape(x.shape)


def _rows64(s, b, n):
    """K, V [n, KH, D] in fp64 of the first n tokens of sequence b, looked up token by token."""
    case, cache = s["case"], s["cache"]
    KH, D = case["KH"], case["D"]
    j, ch = torch.arange(n, device="cuda")[:, None], torch.arange(KH * D, device="cuda")[None]
    p, r, grp, c = s["pages"][b].long()[j // PAGE], j % PAGE, ch // 128, ch % 128
    t = torch.tensor(GRID + [-x for x in GRID], dtype=torch.float64, device="cuda")
    kb, vb = cache[p, grp, r, c // 2], cache[p, grp, 128 + c, r // 2]
    k = t[torch.where(c % 2 == 0, kb % 16, kb // 16).long()]
    v = t[torch.where(r % 2 == 0, vb % 16, vb // 16).long()]
    ka, va = r % 32 * 16 + r // 32 * 4 + c // 32, 512 + r * 4 + c // 32
    k = k * _two(cache[p, grp, 256 + ka // 64, ka % 64].int() - 127)
    v = v * _two(cache[p, grp, 256 + va // 64, va % 64].int() - 127)
    return k.reshape(n, KH, D), v.reshape(n, KH, D)


def _turn64(x, gain, table, inter):
    x = x.double()
    n = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * gain.double()
    half = table.shape[1]
    at = torch.arange(half, device=x.device)
    i, j = (2 * at, 2 * at + 1) if inter else (at, at + half)
    out = n.clone()
    c, t = table[:, None, :, 0].double(), table[:, None, :, 1].double()
    out[..., i] = n[..., i] * c - n[..., j] * t
    out[..., j] = n[..., i] * t + n[..., j] * c
    return out


def _attend64(s, q, k_new=None, v_new=None):
    case = s["case"]
    H, KH, D = case["H"], case["KH"], case["D"]
    out, at = [], 0
    for b, (n, ln) in enumerate(zip(s["n"], s["lens"])):
        k, v = _rows64(s, b, ln)
        if k_new is not None:
            k[ln - n:], v[ln - n:] = k_new[at:at + n], v_new[at:at + n]
        y = torch.zeros(n, H, D, dtype=torch.float64, device="cuda")
        i, j = torch.arange(n, device="cuda")[:, None] + (ln - n), torch.arange(ln, device="cuda")
        see = torch.ones(n, ln, dtype=torch.bool, device="cuda")
        if case.get("causal", True):
            see &= j <= i
        if case.get("window", 0):
            see &= j > i - case["window"]
        for h in range(H):
            z = q[at:at + n, h].double() @ k[:, h * KH // H].T / math.sqrt(D)
            y[:, h] = torch.softmax(z.masked_fill(~see, -math.inf), -1).nan_to_num(0.0) @ v[:, h * KH // H]
        out.append(y)
        at += n
    return torch.cat(out)


def _linear64(x, w, d_out, group):
    codes, scales, zeros = w
    e = torch.arange(codes.shape[1] * 2, device="cuda")
    r = e % 128
    word, nib = e // 128 * 16 + r // 8 % 4 * 4 + r // 32, r % 2 * 4 + r % 8 // 2
    byte = codes[:, word * 4 + nib // 2]
    c = torch.where(nib % 2 == 0, byte % 16, byte // 16).double()
    z = 8.0 if zeros is None else zeros.double()[:, e // group]
    return x.double() @ ((c - z) * scales.double()[:, e // group]).T


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "w4g":
        return {"y": _linear64(s["x"], s["w"], case["d_out"], case["group"])}
    if op == "attend":
        return {"y": _attend64(s, s["q"])}
    H, KH, D = case["H"], case["KH"], case["D"]
    t = s["table"][s["positions"].long()]
    if op == "rope":
        return {x: _turn64(s[x], s["g" + x], t, case["inter"]) for x in "qk"}
    if op == "step":
        x = _linear64(s["x"], s["wqkv"], (H + 2 * KH) * D, case["group"]).reshape(-1, H + 2 * KH, D)
        q, k, v = x[:, :H], x[:, H:H + KH], x[:, H + KH:]
    else:
        q, k, v = s["q"], s["k"], s["v"].double()
    q, k, v = _turn64(q, s["gq"], t, case["inter"]), _grid64(_turn64(k, s["gk"], t, case["inter"])), _grid64(v)
    if op == "append":
        return {"q": q, "k": k, "v": v}
    return {"y": _linear64(_attend64(s, q, k, v).reshape(-1, H * D), s["wo"], H * D, case["group"])}
