"""Cases that measure the microscaled 4-bit (MX4) operators: quantisation and its inverse, the matrix
product grouped by expert, and the mixture-of-experts layer on 4-bit experts.

MX4 is the Open Compute Project's MXFP4: 32 consecutive elements of a row share one scale 2^(s - 127),
s a byte, and each element is one of the E2M1 numbers +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, two to a byte
(the even element in the low half).  For a block with largest magnitude m > 0 the scale is
2^(floor(log2 m) - 2), and an element the E2M1 number nearest to v / scale, ties to the even code,
saturating at +-6; a block of zeros has the scale 1.

  quantize  W^ = the values that the codes and scales of W stand for (bf16 holds each of them exactly)
  grouped   y_n = W^_e x^_n for the rows offsets[e] <= n < offsets[e + 1] of expert e
  layer     p = softmax(x Wr^T), the two largest of 16;  h = bf16(SiLU(W1^_e x^) (W3^_e x^));
            y = bf16(sum over the two experts of p_e (W2^_e h^))
"""
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 32
EXPERTS, TOP_K = 16, 2
# the most that a drawn case may cost: the largest listed one's weights, rows and products
MOST_ELEMENTS = 16 * 4096 * 14336
MOST_LAYER_WEIGHTS = 3 * MOST_ELEMENTS
MOST_ROWS = 16384
MOST_FLOPS = 2 * MOST_ROWS * 4096 * 14336


def listed():
    return [
        # a decode step's activations (64 tokens of hidden size 4096): latency
        {"name": "quantize_activations", "kind": "quantize", "mats": 1, "rows": 64, "cols": 4096},
        # odd rows, five blocks a row
        {"name": "quantize_odd", "kind": "quantize", "mats": 3, "rows": 1237, "cols": 160},
        # the down projections of 16 experts at load time: bandwidth
        {"name": "quantize_experts", "kind": "quantize", "mats": 16, "rows": 4096, "cols": 14336},
        # one token's two experts, down projection: the least work of a serving step
        {"name": "grouped_one_token", "kind": "grouped", "experts": 16, "n": 2, "rows": 4096, "cols": 14336,
         "spread": "even", "out": "bf16"},
        # 64 tokens' assignments, one projection up: every expert's weights are streamed once
        {"name": "grouped_decode", "kind": "grouped", "experts": 16, "n": 128, "rows": 14336, "cols": 4096,
         "spread": "random", "out": "bf16"},
        # many small experts, some without a row, sizes off every tile's edge, fp32 results
        {"name": "grouped_ragged", "kind": "grouped", "experts": 61, "n": 1933, "rows": 1411, "cols": 2176,
         "spread": "skewed", "out": "fp32"},
        # one dense projection: a single group
        {"name": "grouped_dense", "kind": "grouped", "experts": 1, "n": 4096, "rows": 8192, "cols": 8192,
         "spread": "even", "out": "bf16"},
        # 8192 tokens' assignments, one projection up: arithmetic
        {"name": "grouped_prefill", "kind": "grouped", "experts": 16, "n": 16384, "rows": 14336, "cols": 4096,
         "spread": "random", "out": "bf16"},
        # a small layer: launch latency
        {"name": "layer_small", "kind": "layer", "tokens": 37, "d": 256, "ffn": 512},
        # one token through the layer
        {"name": "layer_one_token", "kind": "layer", "tokens": 1, "d": 4096, "ffn": 14336},
        # a decode step of 64 sequences
        {"name": "layer_decode", "kind": "layer", "tokens": 64, "d": 4096, "ffn": 14336},
        # a prompt chunk of 8192 tokens
        {"name": "layer_prefill", "kind": "layer", "tokens": 8192, "d": 4096, "ffn": 14336},
    ]


def _log_int(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, round(low * (high / low) ** rng.random())))


def draw(rng):
    kind = rng.choice(("quantize", "grouped", "grouped", "layer"))
    if kind == "quantize":
        cols = BLOCK * _log_int(rng, 1, 1024)
        mats = _log_int(rng, 1, 16)
        return {"kind": kind, "mats": mats, "rows": _log_int(rng, 1, min(32768, MOST_ELEMENTS // (cols * mats))),
                "cols": cols}
    if kind == "grouped":
        cols = 128 * _log_int(rng, 1, 112)
        experts = _log_int(rng, 1, 256)
        rows = _log_int(rng, 1, min(16384, MOST_ELEMENTS // (cols * experts)))
        n = _log_int(rng, 1, min(MOST_ROWS, MOST_FLOPS // (2 * rows * cols)))
        return {"kind": kind, "experts": experts, "n": n, "rows": rows, "cols": cols,
                "spread": rng.choice(("even", "random", "skewed")), "out": rng.choice(("bf16", "fp32"))}
    d = 128 * _log_int(rng, 1, 64)
    ffn = 128 * _log_int(rng, 1, min(192, MOST_LAYER_WEIGHTS // (3 * EXPERTS * 128 * d)))
    tokens = _log_int(rng, 1, 8192)
    return {"kind": kind, "tokens": tokens, "d": d, "ffn": ffn}


# ------------------------------------------------------------------ the plain form
def _pow2(e):
    """2^e in fp32, e whole numbers of [-126, 127]: the exponent's bits."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _mx4_parts(w):
    """Magnitude codes, signs and scale bytes of rows in blocks of 32, from bf16 values."""
    v = w.float().reshape(*w.shape[:-1], -1, BLOCK)
    m = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(m)[1] - 3).clamp(min=-126)  # frexp: m = f 2^k, 1/2 <= f < 1
    e = torch.where(m == 0, torch.zeros_like(e), e)
    a = v.abs() * _pow2(-e)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code, torch.signbit(v).to(torch.uint8), (e + 127).squeeze(-1).to(torch.uint8)


def _mx4(w):
    """bf16 [..., cols] -> codes uint8 [..., cols / 2] and scales uint8 [..., cols / 32]."""
    code, sign, s = _mx4_parts(w)
    code = (code | (sign << 3)).reshape(w.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def _mx4_values(q, s):
    """The values that codes and scales stand for, in fp32."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    code = torch.stack((q & 15, q >> 4), -1).reshape(*s.shape, BLOCK)
    v = lut.index_select(0, code.reshape(-1).int()).reshape(code.shape)
    return (v * _pow2(s.int() - 127).unsqueeze(-1)).reshape(*q.shape[:-1], -1)


def _grouped(x, expert, slot, cap, w):
    """y_n = w[expert_n] x_n in fp32: the rows of each expert side by side, padded to `cap` rows."""
    side = torch.zeros(w.shape[0], cap, x.shape[-1], device=x.device)
    side[expert, slot] = x
    return torch.bmm(side, w.transpose(1, 2))[expert, slot]


def _layer(s):
    x = s["x"]
    logits = x.float() @ s["router"].T
    top = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids = top.indices[:, :TOP_K]
    p = torch.softmax(logits, -1).gather(1, ids)
    expert = ids.reshape(-1)
    mine = expert.unsqueeze(1) == torch.arange(EXPERTS, device=x.device)
    slot = (mine.int().cumsum(0).gather(1, expert.unsqueeze(1)) - 1).squeeze(1)
    xv = _mx4_values(*_mx4(x)).repeat_interleave(TOP_K, 0)
    gate = _grouped(xv, expert, slot, s["cap"], _mx4_values(s["q1"], s["s1"]))
    up = _grouped(xv, expert, slot, s["cap"], _mx4_values(s["q3"], s["s3"]))
    h = (gate / (1 + torch.exp(-gate)) * up).bfloat16()
    o = _grouped(_mx4_values(*_mx4(h)), expert, slot, s["cap"], _mx4_values(s["q2"], s["s2"]))
    y = (o.reshape(-1, TOP_K, o.shape[-1]) * p.unsqueeze(-1)).sum(1)
    return {"y": y.bfloat16(), "ids": ids.int(), "p": p}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _weights(g, mats, rows, cols):
    """Codes and scales of normally distributed weights, a matrix at a time."""
    q = torch.empty(mats, rows, cols // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(mats, rows, cols // BLOCK, dtype=torch.uint8, device="cuda")
    for i in range(mats):
        q[i], s[i] = _mx4((torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).bfloat16())
    return q, s


def _activations(g, n, cols):
    """Rows of normal values, of levels a few times apart, with some channels far above the others."""
    x = torch.randn(n, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(n, 1, generator=g, device="cuda"))
    x *= 1 + 9 * (torch.rand(1, cols, generator=g, device="cuda") < 0.01)
    return x.bfloat16()


def _counts(case, seed):
    """How many rows each expert has: as even as can be, by chance, or a few experts with the most."""
    e, n = case["experts"], case["n"]
    if case["spread"] == "even":
        return [n // e + (i < n % e) for i in range(e)]
    g = torch.Generator()
    g.manual_seed(seed)
    p = torch.ones(e) if case["spread"] == "random" else torch.exp(1.5 * torch.randn(e, generator=g))
    got = torch.multinomial(p, n, replacement=True, generator=g)
    return torch.bincount(got, minlength=e).tolist()


def prepare(case, seed):
    g = _generator(seed)
    if case["kind"] == "quantize":
        w = torch.randn(case["mats"], case["rows"], case["cols"], generator=g, device="cuda", dtype=torch.bfloat16)
        return {"kind": "quantize", "w": w}
    if case["kind"] == "grouped":
        counts = torch.tensor(_counts(case, seed))
        offsets = torch.cat((torch.zeros(1, dtype=torch.int64), counts.cumsum(0))).int().cuda()
        q, s = _weights(g, case["experts"], case["rows"], case["cols"])
        xq, xs = _mx4(_activations(g, case["n"], case["cols"]))
        return {"kind": "grouped", "q": q, "s": s, "xq": xq.contiguous(), "xs": xs, "offsets": offsets,
                "cap": int(counts.max()), "dtype": torch.bfloat16 if case["out"] == "bf16" else torch.float32}
    t, d, ffn = case["tokens"], case["d"], case["ffn"]
    # tokens whose third expert comes within 1e-3 of the second would be routed by rounding alone: others are taken
    router = torch.randn(EXPERTS, d, generator=g, device="cuda") * d ** -0.5
    x = _activations(g, t + t // 4 + 32, d)
    logits = torch.sort(x.double() @ router.double().T, dim=-1, descending=True).values
    clear = ((logits[:, 0] - logits[:, 1] > 1e-3) & (logits[:, 1] - logits[:, 2] > 1e-3)).nonzero().squeeze(1)[:t]
    state = {"kind": "layer", "router": router, "x": x[clear].contiguous()}
    ids = torch.sort(state["x"].double() @ router.double().T, dim=-1, descending=True).indices[:, :TOP_K]
    state["cap"] = int(torch.bincount(ids.reshape(-1)).max())
    for k, rows, cols in (("1", ffn, d), ("3", ffn, d), ("2", d, ffn)):
        state["q" + k], state["s" + k] = _weights(g, EXPERTS, rows, cols)
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        import int8_expert_weight_b200 as jm

        if state["kind"] == "quantize":
            return jm.jamba_moe_dequantize_mx4(*jm.jamba_moe_quantize_mx4(state["w"]))
        if state["kind"] == "grouped":
            return jm.jamba_moe_grouped_mx4(state["xq"], state["xs"], state["offsets"], state["q"], state["s"],
                                            out_dtype=state["dtype"])
        y, ids, p = jm.jamba_moe_forward_mx4(state["x"], state["router"], None, state["q1"], state["s1"], state["q3"],
                                             state["s3"], state["q2"], state["s2"])
        return {"y": y, "ids": ids, "p": p}
    if state["kind"] == "quantize":
        return _mx4_values(*_mx4(state["w"])).bfloat16()
    if state["kind"] == "grouped":
        n = torch.arange(state["xq"].shape[0], device="cuda", dtype=torch.int32)
        expert = torch.searchsorted(state["offsets"][1:].contiguous(), n, right=True)
        slot = n - state["offsets"][expert]
        x = _mx4_values(state["xq"], state["xs"])
        return _grouped(x, expert, slot, state["cap"], _mx4_values(state["q"], state["s"])).to(state["dtype"])
    return _layer(state)


def _mx4_bytes(elements):
    return elements / 2 + elements / BLOCK


def work(case):
    """Bytes that have to be read and written once, and the products' operations.  Of the experts' weights those
    of experts with a row are counted: at most as many as there are rows."""
    if case["kind"] == "quantize":  # W in, its values out; the codes and scales between the two written and read
        n = case["mats"] * case["rows"] * case["cols"]
        return {"bytes": 4 * n + 2 * _mx4_bytes(n), "flops": 0}
    if case["kind"] == "grouped":
        n, r, k = case["n"], case["rows"], case["cols"]
        live = min(case["experts"], n)
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": _mx4_bytes(live * r * k + n * k) + size * n * r + 4 * (case["experts"] + 1), "flops": 2 * n * r * k}
    t, d, f = case["tokens"], case["d"], case["ffn"]
    live = min(EXPERTS, TOP_K * t)
    return {"bytes": _mx4_bytes(3 * live * d * f) + 2 * (2 * t * d) + 4 * EXPERTS * d + 16 * t,
            "flops": 2 * TOP_K * t * 3 * d * f + 2 * t * d * EXPERTS}


# ------------------------------------------------------------------ the definition in 64 bits
def _scales(device):
    """2^(s - 127) for s = 0 .. 254: a table, as a power function need not be exact."""
    return torch.tensor([2.0 ** (s - 127) for s in range(255)], dtype=torch.float64, device=device)


def _exact_mx4(w):
    """The values that the format's rule gives for rows w, in fp64."""
    v = w.double().reshape(-1, BLOCK)
    m = v.abs().max(1, keepdim=True).values
    powers = _scales(w.device)
    at = torch.searchsorted(powers, torch.where(m > 0, m, 4.0), right=True) - 1  # the last 2^k <= m
    scale = powers[(at - 2).clamp(min=0)]
    a = v.abs() / scale
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.sign(v) * torch.clamp(torch.round(a / step) * step, max=6.0) * scale).reshape(w.shape)


def _exact_values(q, s):
    """fp64 values of one matrix's codes and scales."""
    both = torch.empty(q.shape[0], q.shape[1] * 2, dtype=torch.float64, device=q.device)
    for half, code in ((0, q % 16), (1, q // 16)):
        mag = (code % 8).double()
        whole = torch.where(mag < 4, 1.0, torch.where(mag < 6, 2.0, 4.0)) * (1 + 0.5 * (mag % 2))
        both[:, half::2] = torch.where(mag < 2, 0.5 * mag, whole) * torch.where(code >= 8, -1.0, 1.0)
    return both * _scales(q.device)[s.long()].repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "quantize":
        return torch.stack([_exact_mx4(w) for w in s["w"]])
    if s["kind"] == "grouped":
        at = s["offsets"].tolist()
        y = torch.empty(case["n"], case["rows"], dtype=torch.float64, device="cuda")
        x = _exact_values(s["xq"], s["xs"])
        for e in range(case["experts"]):
            if at[e] < at[e + 1]:
                y[at[e]:at[e + 1]] = x[at[e]:at[e + 1]] @ _exact_values(s["q"][e], s["s"][e]).T
        return y
    x = s["x"]
    logits = x.double() @ s["router"].double().T
    p, ids = torch.topk(torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True)), TOP_K, dim=1)
    xv = _exact_mx4(x)
    y = torch.zeros(x.shape[0], x.shape[1], dtype=torch.float64, device="cuda")
    for e in range(EXPERTS):
        token, k = (ids == e).nonzero(as_tuple=True)
        if token.numel():
            gate, up = (xv[token] @ _exact_values(s["q" + m][e], s["s" + m][e]).T for m in "13")
            h = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16)
            y[token] += p[token, k].unsqueeze(1) * (_exact_mx4(h) @ _exact_values(s["q2"][e], s["s2"][e]).T)
    return {"y": y, "ids": None, "p": p}
