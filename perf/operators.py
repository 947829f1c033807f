"""The cases that the block-scaled FP8 projection and the per-head norm with
rotation are measured on: inputs, plain forms, minimum work and 64-bit values.

    theta_fp8_quantize        W0 -> E4M3 codes, one E8M0 scale per 128 x 128 block
    theta_fp8_quantize_rows   X  -> E4M3 codes, one E8M0 scale per token and 128 columns
    theta_linear_forward_fp8  Y = s * (Xq . W0q^T) + (X . V) . U^T
    theta_qk_norm_rope        RMS norm of each query and key head, then the position rotation
"""
import math

import torch

own = False

BLOCK = 128
LARGEST_BLOCK = 21504 * 5376  # the gate projection of Gemma 4 31B
LARGEST_FORWARD = 2048 * LARGEST_BLOCK
LARGEST_ROWS = 2048 * 21504
LARGEST_HEADS = 8192 * 40 * 256
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # laying out the largest shared block of Gemma 4 31B once, before serving
        {"name": "quantize_31b_gate", "op": "quantize", "O": 21504, "I": 5376, "dt": "bf16"},
        # an fp32 checkpoint, neither size a multiple of the block
        {"name": "quantize_ragged_f32", "op": "quantize", "O": 2000, "I": 1296, "dt": "f32"},
        # the activations of one decode step
        {"name": "rows_decode", "op": "rows", "M": 1, "I": 5376, "dt": "bf16"},
        # the inputs of the 31B down projection for a prefill of 2048 tokens
        {"name": "rows_prefill_down", "op": "rows", "M": 2048, "I": 21504, "dt": "bf16"},
        # decode, Gemma 3 1B gate: a few megabytes, latency counts
        {"name": "forward_1b_gate_m1", "op": "forward", "M": 1, "O": 6912, "I": 1152, "rank": 32},
        # decode, Gemma 4 31B gate: W0 from HBM sets the time
        {"name": "forward_31b_gate_m1", "op": "forward", "M": 1, "O": 21504, "I": 5376, "rank": 64},
        # a batch of decoding sequences, Gemma 4 31B q
        {"name": "forward_31b_q_m16", "op": "forward", "M": 16, "O": 8192, "I": 5376, "rank": 64},
        # a short prompt, sizes that end inside tiles and blocks
        {"name": "forward_ragged_m333", "op": "forward", "M": 333, "O": 2056, "I": 1168, "rank": 24},
        # prefill, Gemma 4 31B gate: the tensor cores set the time
        {"name": "forward_31b_gate_m2048", "op": "forward", "M": 2048, "O": 21504, "I": 5376, "rank": 64},
        # decode, Gemma 3 1B: four query heads and one key head of 256
        {"name": "heads_decode", "op": "heads", "M": 1, "hq": 4, "hk": 1, "D": 256, "rotary": 256, "start": 31000,
         "interleaved": False, "fused": False, "dt": "bf16"},
        # odd sizes: partial rotation of neighbouring pairs, slices of one buffer
        {"name": "heads_ragged_f32", "op": "heads", "M": 333, "hq": 6, "hk": 3, "D": 80, "rotary": 36, "start": 1000000,
         "interleaved": True, "fused": True, "dt": "f32"},
        # prefill, the q and k rows of Gemma 4 31B
        {"name": "heads_prefill", "op": "heads", "M": 8192, "hq": 32, "hk": 8, "D": 256, "rotary": 256, "start": 0,
         "interleaved": False, "fused": False, "dt": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(["quantize", "rows", "forward", "forward", "heads"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    while True:
        if op == "quantize":
            c = {"op": op, "O": _log(rng, 8, 21504), "I": _log(rng, 16, 21504, 16), "dt": dt}
            if c["O"] * c["I"] <= LARGEST_BLOCK // (2 if dt == "f32" else 1):
                return c
        elif op == "rows":
            c = {"op": op, "M": _log(rng, 1, 2048), "I": _log(rng, 16, 21504, 16), "dt": dt}
            if c["M"] * c["I"] <= LARGEST_ROWS // (2 if dt == "f32" else 1):
                return c
        elif op == "forward":
            c = {"op": op, "M": _log(rng, 1, 2048), "O": _log(rng, 64, 21504, 8), "I": _log(rng, 64, 21504, 16),
                 "rank": rng.choice([0, 8, 16, 24, 32, 64, 64, 128])}
            if c["O"] * c["I"] <= LARGEST_BLOCK and c["M"] * c["O"] * c["I"] <= LARGEST_FORWARD:
                return c
        else:
            D = rng.choice([64, 80, 96, 128, 192, 256, 512])
            hk = _log(rng, 1, 16)
            c = {"op": op, "M": _log(rng, 1, 8192), "hq": hk * rng.choice([1, 2, 3, 4, 8]), "hk": hk, "D": D,
                 "rotary": rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)]), "start": _log(rng, 1, 1000000),
                 "interleaved": rng.random() < 0.4, "fused": rng.random() < 0.5, "dt": dt}
            if c["M"] * (c["hq"] + c["hk"]) * D <= LARGEST_HEADS // (2 if dt == "f32" else 1):
                return c


# ------------------------------------------------------------------ plain forms
def _scale_bytes(amax):
    """The byte of the least power of two 2^e with amax <= 448 * 2^e (e + 127); 127 for a block of zeros."""
    m, k = torch.frexp(amax)
    e = torch.where(m <= 0.875, k - 9, k - 8)
    return torch.where(amax > 0, (e + 127).clamp(0, 254), torch.full_like(k, 127)).to(torch.uint8)


def _power(scale_bytes):
    """2^(byte - 127), from its bits: the byte is the fp32 exponent field."""
    b = scale_bytes.to(torch.int32)
    return torch.where(b > 0, b << 23, torch.full_like(b, 1 << 22)).view(torch.float32)


def _encode(x, scale_bytes):
    """E4M3 of x / 2^(byte - 127), scale_bytes broadcast to x's shape."""
    return (x * _power(254 - scale_bytes)).to(torch.float8_e4m3fn)


def _quantize_rows(X):
    M, I = X.shape
    nb = -(-I // BLOCK)
    x = torch.nn.functional.pad(X.float(), (0, nb * BLOCK - I)).view(M, nb, BLOCK)
    b = _scale_bytes(x.abs().amax(dim=2))
    q = _encode(x, b[:, :, None]).view(M, nb * BLOCK)[:, :I].contiguous()
    return q, b.t().contiguous()


def _quantize_blocks(W):
    O, I = W.shape
    no, nb = -(-O // BLOCK), -(-I // BLOCK)
    w = torch.nn.functional.pad(W.float(), (0, nb * BLOCK - I, 0, no * BLOCK - O)).view(no, BLOCK, nb, BLOCK)
    b = _scale_bytes(w.abs().amax(dim=(1, 3)))
    q = _encode(w, b[:, None, :, None]).view(no * BLOCK, nb * BLOCK)[:O, :I].contiguous()
    return q, b


def _forward(st):
    M, I = st["X"].shape
    O = st["s"].shape[0]
    x = st["xq"].float() * _power(st["xs"]).t().repeat_interleave(BLOCK, dim=1)[:, :I]
    w = st["wq"].float() * _power(st["ws"]).repeat_interleave(BLOCK, 0)[:O].repeat_interleave(BLOCK, 1)[:, :I]
    y = (x @ w.t()) * st["s"]
    if st["rank"]:
        y = y + (st["X"].float() @ st["V"].float()) @ st["U"].float().t()
    return y.to(torch.bfloat16)


def _heads(x, w, st):
    M = x.shape[0]
    D, rotary = st["D"], st["rotary"]
    h = x.float().reshape(M, -1, D)
    h = h * torch.rsqrt((h * h).mean(dim=2, keepdim=True) + st["eps"]) * (w.float() + st["offset"])
    angle = st["pos"].double()[:, None] * st["freq"].double()[None, :]
    c, s = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    r, rest = h[:, :, :rotary], h[:, :, rotary:]
    if st["interleaved"]:
        a, b = r[:, :, 0::2], r[:, :, 1::2]
        r = torch.stack((a * c - b * s, b * c + a * s), dim=3).reshape(M, -1, rotary)
    else:
        a, b = r[:, :, :rotary // 2], r[:, :, rotary // 2:]
        r = torch.cat((a * c - b * s, b * c + a * s), dim=2)
    return torch.cat((r, rest), dim=2).reshape(M, -1).to(x.dtype)


# ------------------------------------------------------------------ inputs
def _activations(g, M, I, dt):
    """Activations as a norm leaves them: near unit size, tokens of different size, a few channels far larger."""
    x = torch.randn(M, I, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(M, 1, device="cuda", generator=g))
    big = torch.rand(I, device="cuda", generator=g) < 0.004
    return (x * torch.where(big, 20.0, 1.0)).to(DTYPES[dt])


def _weights(g, O, I, dt):
    w = 0.02 * torch.randn(O, I, device="cuda", generator=g)
    return (w * torch.exp(0.3 * torch.randn(O, 1, device="cuda", generator=g))).to(DTYPES[dt])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    op = case["op"]
    if op == "quantize":
        O, I = case["O"], case["I"]
        W = _weights(g, O, I, case["dt"])
        return {"op": op, "W": W, "codes": torch.empty(O, I, dtype=torch.uint8, device="cuda"),
                "scales": torch.empty(-(-O // BLOCK), -(-I // BLOCK), dtype=torch.uint8, device="cuda")}
    if op == "rows":
        M, I = case["M"], case["I"]
        return {"op": op, "X": _activations(g, M, I, case["dt"]),
                "codes": torch.empty(M, I, dtype=torch.uint8, device="cuda"),
                "scales": torch.empty(-(-I // BLOCK), M, dtype=torch.uint8, device="cuda")}
    if op == "forward":
        M, O, I, r = case["M"], case["O"], case["I"], case["rank"]
        X = _activations(g, M, I, "bf16")
        xq, xs = _quantize_rows(X)
        wq, ws = _quantize_blocks(_weights(g, O, I, "bf16"))
        st = {"op": op, "rank": r, "X": X, "xq": xq, "xs": xs, "wq": wq, "ws": ws,
              "s": 1.0 + 0.05 * torch.randn(O, device="cuda", generator=g),
              "U": (0.05 * torch.randn(O, r, device="cuda", generator=g)).bfloat16() if r else None,
              "V": (0.05 * torch.randn(I, r, device="cuda", generator=g)).bfloat16() if r else None,
              "Y": torch.empty(M, O, dtype=torch.bfloat16, device="cuda"), "work": None,
              "xcodes": xq.view(torch.uint8), "wcodes": wq.view(torch.uint8)}
        return st
    M, D, dt = case["M"], case["D"], DTYPES[case["dt"]]
    nq, nk = case["hq"] * D, case["hk"] * D
    both = (torch.randn(M, nq + nk, device="cuda", generator=g)
            * torch.exp(torch.randn(M, 1, device="cuda", generator=g))).to(dt)
    out = torch.empty_like(both)
    cut = (lambda t: (t[:, :nq], t[:, nq:])) if case["fused"] else \
          (lambda t: (t[:, :nq].contiguous(), t[:, nq:].contiguous()))
    (Q, K), (Qo, Ko) = cut(both), cut(out)
    half = case["rotary"] // 2
    return {"op": op, "D": D, "rotary": case["rotary"], "interleaved": case["interleaved"], "eps": 1e-6, "offset": 1.0,
            "Q": Q, "K": K, "Qo": Qo, "Ko": Ko,
            "wq": (0.1 * torch.randn(D, device="cuda", generator=g)).to(dt),
            "wk": (0.1 * torch.randn(D, device="cuda", generator=g)).to(dt),
            "pos": case["start"] + torch.arange(M, device="cuda"),
            "freq": 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float32) / max(1, half))}


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["op"]
    if own:
        import linear_theta_forward_b200 as theta
        if op == "quantize":
            theta.theta_fp8_quantize(st["W"], st["codes"], st["scales"])
            return st["codes"].view(torch.float8_e4m3fn), st["scales"]
        if op == "rows":
            theta.theta_fp8_quantize_rows(st["X"], st["codes"], st["scales"])
            return st["codes"].view(torch.float8_e4m3fn), st["scales"]
        if op == "forward":
            if st["work"] is None:  # kept by the program that makes the calls
                (M, I), O = st["X"].shape, st["s"].shape[0]
                nbytes = theta.theta_workspace_size(theta.THETA_OP_LINEAR_FORWARD_FP8, M, O, I, st["rank"],
                                                    theta.THETA_BF16)
                st["work"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
            theta.theta_linear_forward_fp8(st["X"], st["xcodes"], st["xs"], st["wcodes"], st["ws"], st["s"], st["U"],
                                           st["V"], st["Y"], st["work"])
            return st["Y"]
        theta.theta_qk_norm_rope(st["Q"], st["K"], st["wq"], st["wk"], st["pos"], st["freq"], st["Qo"], st["Ko"],
                                 st["D"], eps=st["eps"], weight_offset=st["offset"], interleaved=st["interleaved"])
        return st["Qo"], st["Ko"]
    if op == "quantize":
        return _quantize_blocks(st["W"])
    if op == "rows":
        return _quantize_rows(st["X"])
    if op == "forward":
        return _forward(st)
    return _heads(st["Q"], st["wq"], st), _heads(st["K"], st["wk"], st)


def work(case):
    op = case["op"]
    if op in ("quantize", "rows"):
        b = DTYPES[case["dt"]].itemsize
        rows = case["O"] if op == "quantize" else case["M"]
        nb = -(-case["I"] // BLOCK)
        return {"bytes": rows * case["I"] * (b + 1) + (-(-rows // BLOCK) if op == "quantize" else rows) * nb,
                "flops": 2 * rows * case["I"]}
    if op == "forward":
        M, O, I, r = case["M"], case["O"], case["I"], case["rank"]
        nb = -(-I // BLOCK)
        moved = O * I + -(-O // BLOCK) * nb + 4 * O + M * I + M * nb + 2 * M * O
        if r:
            moved += 2 * r * (O + I) + 2 * M * I
        return {"bytes": moved, "flops": 2 * M * (O * I + r * (O + I))}
    b, n = DTYPES[case["dt"]].itemsize, case["M"] * (case["hq"] + case["hk"]) * case["D"]
    return {"bytes": 2 * b * n + 8 * case["M"] + 2 * case["rotary"] + 2 * b * case["D"], "flops": 8 * n}


# ------------------------------------------------------------------ 64-bit values
def _pow2(e):
    """2^e in fp64 for whole numbers e, from the bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3_nearest(v):
    """The E4M3 value nearest to v (|v| <= 448), ties to the even one: multiples of 2^(floor(log2|v|) - 3), of 2^-9 at least."""
    unit = _pow2((torch.frexp(v)[1] - 4).clamp(min=-9))
    return torch.round(v / unit) * unit


def _least_exponent(a):
    """The least e >= -127 with a <= 448 * 2^e; 0 where a is 0."""
    e = torch.ceil(torch.log2(a.clamp(min=2.0 ** -160) / 448.0))
    e = torch.where(a > 448.0 * _pow2(e), e + 1, e)
    e = torch.where(a <= 448.0 * _pow2(e - 1), e - 1, e)
    return torch.where(a > 0, e.clamp(min=-127.0), torch.zeros_like(e))


def _e4m3_table():
    c = torch.arange(256, device="cuda")
    f, m = ((c >> 3) & 15).double(), (c & 7).double()
    v = torch.where(f > 0, (1 + m / 8) * _pow2(f - 7), m / 8 * 2.0 ** -6)
    return torch.where(c >= 128, -v, v)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("quantize", "rows"):
        x = (st["W"] if op == "quantize" else st["X"]).double()
        rows, I = x.shape
        height = BLOCK if op == "quantize" else 1
        values = torch.empty_like(x)
        scales = torch.empty(-(-rows // height), -(-I // BLOCK), dtype=torch.uint8, device="cuda")
        for b in range(scales.shape[1]):
            part = x[:, b * BLOCK:(b + 1) * BLOCK]
            a = part.abs().amax(dim=1)
            if height > 1:
                a = torch.stack([p.amax() for p in a.split(height)])
            e = _least_exponent(a)
            scales[:, b] = (e + 127).to(torch.uint8)
            values[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3_nearest(
                part * _pow2(-e).repeat_interleave(height)[:rows, None])
        return values, scales if op == "quantize" else scales.t().contiguous()
    if op == "forward":
        table = _e4m3_table()
        M, I = st["X"].shape
        O = st["s"].shape[0]
        y = torch.zeros(M, O, dtype=torch.float64, device="cuda")
        row_block = torch.arange(O, device="cuda") // BLOCK
        for b in range(-(-I // BLOCK)):
            cols = slice(b * BLOCK, min(I, (b + 1) * BLOCK))
            x, w = table[st["xcodes"][:, cols].long()], table[st["wcodes"][:, cols].long()]
            ex, ew = st["xs"][b].long() - 127, st["ws"][:, b].long()[row_block] - 127
            y += (x * _pow2(ex)[:, None]) @ (w * _pow2(ew)[:, None]).t()
        y *= st["s"].double()
        if st["rank"]:
            y += st["X"].double() @ (st["V"].double() @ st["U"].double().t())
        return y
    D, rotary = case["D"], case["rotary"]
    i = torch.arange(rotary // 2, device="cuda")
    first = 2 * i if case["interleaved"] else i
    second = 2 * i + 1 if case["interleaved"] else i + rotary // 2
    turn = st["pos"].double()[:, None] * st["freq"].double()
    out = []
    for x, w in ((st["Q"], st["wq"]), (st["K"], st["wk"])):
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for h in range(x.shape[1] // D):
            v = x[:, h * D:(h + 1) * D].double()
            v = v / torch.sqrt(v.square().sum(dim=1, keepdim=True) / D + st["eps"]) * (w.double() + st["offset"])
            z = v.clone()
            z[:, first] = v[:, first] * torch.cos(turn) - v[:, second] * torch.sin(turn)
            z[:, second] = v[:, second] * torch.cos(turn) + v[:, first] * torch.sin(turn)
            y[:, h * D:(h + 1) * D] = z
        out.append(y)
    return tuple(out)
