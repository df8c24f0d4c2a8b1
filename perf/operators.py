"""Cases for the operators around the sharded optimizer step: what they compute in plain torch, and how a user calls them.

  adamw   AdamW over the many tensors of a shard, its two moments in fp32 or in blockwise E4M3, with an optional
          16-bit copy of the weights (the model's own).
  trip    an MXFP4 payload and back: quantise a matrix along its rows, or along its columns (the payload of its
          transpose), and dequantise it as the receiver does.
  matmul  the product of two MXFP4 payloads, C = A B^T.
  linear  forward and backward of a linear layer whose three products run on MXFP4 payloads.

MXFP4: 32 values along a row share a scale 2^(e - 127), e = max(exponent field of the fp32 absmax - 2, 0); a value is
the nearest of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} times it, ties to the even code, 6 beyond.  Rows are padded with zeros
to whole 128 values: 64 code bytes (even value in the low four bits) and 4 scale bytes.

E4M3 moments: m and r = sqrt(v), each with a power-of-two scale per block of G values, the smallest at which the
block's absmax is at most 448.  They are rounded up or down at random: value i gets 32 hash bits of (i, seed, step),
the low half for m and the high half for r, and goes up where its fraction of the spacing plus (half / 65536) reaches 1.
A positive r never becomes zero.
"""
import math
import random

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LR, BETA1, BETA2, EPS, DECAY, CLIP = 3e-4, 0.9, 0.999, 1e-8, 0.1, 0.37
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# One decoder layer of the 8B-parameter model and of the 70B-parameter model this repository's workloads are shaped by.
LAYER_8B = [4096 * 4096, 4096 * 4096, 4096 * 1024, 4096 * 1024] + 3 * [4096 * 14336]
LAYER_70B = [8192 * 28672, 8192 * 8192, 8192 * 8192]
MOST_ADAMW, MOST_TRIP, MOST_MATMUL, MOST_LINEAR = sum(LAYER_70B), 8192 * 28672, 8192 * 8192 * 28672, 2048 * 4096 * 14336


def sizes_text(sizes):
    return ",".join(str(int(n)) for n in sizes)


def ragged(rng, count, total):
    """`count` sizes of very different orders that add up to about `total`."""
    w = [math.exp(rng.uniform(0, 7)) for _ in range(count)]
    return [max(1, int(total * x / sum(w))) for x in w]


def listed():
    r = random.Random(20)
    return [
        # the update of one norm's weights: nothing but latency
        {"name": "adamw one vector", "op": "adamw", "state": "f32", "sizes": "4096", "grad": "f32", "copy": "none", "G": 128, "step": 1},
        # one rank's eighth of an 8B decoder layer, on the fp32 sums that the gradient reduce leaves
        {"name": "adamw shard", "op": "adamw", "state": "f32", "sizes": sizes_text(n // 8 for n in LAYER_8B), "grad": "f32", "copy": "bf16", "G": 128, "step": 1000},
        # the norms, biases and small matrices of a model: many tensors, few values, odd sizes
        {"name": "adamw ragged e4m3", "op": "adamw", "state": "e4m3", "sizes": sizes_text(ragged(r, 96, 700_001)), "grad": "bf16", "copy": "none", "G": 128, "step": 10},
        # a whole 70B decoder layer with its moments in 8 bits
        {"name": "adamw layer e4m3", "op": "adamw", "state": "e4m3", "sizes": sizes_text(LAYER_70B), "grad": "bf16", "copy": "bf16", "G": 128, "step": 1000},
        # a small odd matrix, its last block short
        {"name": "trip small odd", "op": "trip", "rows": 37, "cols": 1003, "dtype": "f32", "transpose": False},
        # the forward gather of one 8B projection
        {"name": "trip projection", "op": "trip", "rows": 14336, "cols": 4096, "dtype": "bf16", "transpose": False},
        # the backward gather of a 70B projection: blocks along the other axis
        {"name": "trip transposed", "op": "trip", "rows": 28672, "cols": 8192, "dtype": "f16", "transpose": True},
        # one token through a gathered 8B projection
        {"name": "matmul token", "op": "matmul", "M": 1, "N": 14336, "K": 4096, "out": "bf16"},
        # sizes that are no multiples of anything
        {"name": "matmul ragged", "op": "matmul", "M": 77, "N": 1001, "K": 1111, "out": "f32"},
        # a training batch through a 70B projection
        {"name": "matmul batch", "op": "matmul", "M": 8192, "N": 8192, "K": 28672, "out": "bf16"},
        # the last, short batch of a small head
        {"name": "linear ragged", "op": "linear", "tokens": 77, "in": 520, "out": 1032},
        # 2048 tokens through an 8B projection and back
        {"name": "linear layer", "op": "linear", "tokens": 2048, "in": 4096, "out": 14336},
    ]


def logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("adamw", "adamw", "trip", "matmul", "linear"))
    if op == "adamw":
        state = rng.choice(("f32", "e4m3"))
        total = logint(rng, 100, MOST_ADAMW // 2 if state == "f32" else MOST_ADAMW)
        return {"op": op, "state": state, "sizes": sizes_text(ragged(rng, logint(rng, 1, 96), total * 0.95)), "grad": rng.choice(("f32", "bf16", "f16")),
                "copy": rng.choice(("none", "bf16", "f16")), "G": rng.choice((32, 64, 128, 256, 512, 1024)), "step": logint(rng, 1, 100_000)}
    if op == "trip":
        rows = logint(rng, 1, 28672)
        return {"op": op, "rows": rows, "cols": logint(rng, 1, min(28672, MOST_TRIP // rows)), "dtype": rng.choice(("f32", "bf16", "f16")), "transpose": rng.random() < 0.5}
    if op == "matmul":
        M, N = logint(rng, 1, 8192), logint(rng, 16, 28672)
        return {"op": op, "M": M, "N": N, "K": logint(rng, 32, min(28672, max(32, MOST_MATMUL // (M * N)))), "out": rng.choice(("f32", "bf16", "f16"))}
    T, I = logint(rng, 1, 4096), logint(rng, 32, 14336)
    return {"op": op, "tokens": T, "in": I, "out": logint(rng, 32, min(14336, max(32, MOST_LINEAR // (T * I))))}


def up(n, m):
    return (n + m - 1) // m * m


def work(case):
    op = case["op"]
    if op == "adamw":
        sizes, width = [int(n) for n in case["sizes"].split(",")], {"none": 0, "f32": 4, "bf16": 2, "f16": 2}
        n, blocks = sum(sizes), sum(up(k, case["G"]) // case["G"] for k in sizes)
        each = 8 + width[case["grad"]] + width[case["copy"]] + (16 if case["state"] == "f32" else 4)
        return {"bytes": n * each + (0 if case["state"] == "f32" else 16 * blocks), "flops": 20 * n}
    if op == "trip":
        R, C = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        return {"bytes": 2 * R * C * (4 if case["dtype"] == "f32" else 2) + 2 * R * up(C, 32) * 17 // 32, "flops": 4 * R * C}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * up(K, 32) * 17 // 32 + M * N * (4 if case["out"] == "f32" else 2), "flops": 2 * M * N * K}
    T, I, O = case["tokens"], case["in"], case["out"]
    return {"bytes": 4 * (T * I + O * I + T * O), "flops": 6 * T * I * O}


# ---------------------------------------------------------------------------- inputs


def offsets(case):
    """[(first value, size)] of each tensor in the flat buffers: every tensor starts a new block."""
    got, at = [], 0
    for n in (int(k) for k in case["sizes"].split(",")):
        got.append((at, n))
        at += up(n, case["G"])
    return got, at


def plain_encode(x):
    """[rows, cols] fp32 -> the payload of its MXFP4 form (codes, scales), rows padded to whole 128 values."""
    value, scale = plain_blocks(x)
    v = value.abs()
    code = torch.where(v < 2, 2 * v, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.uint8) | (torch.signbit(value).to(torch.uint8) << 3)
    code = code.view(x.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), scale


def prepare(case, seed):
    dev, gen = "cuda", torch.Generator(device="cuda")
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731

    def weight(rows, cols):  # N(0, 0.02) and now and then an outlier of 20 sigma
        w = normal(rows, cols).mul_(0.02)
        return torch.where(torch.rand(rows, cols, generator=gen, device=dev) < 0.001, torch.sign(w) * 0.4, w)

    def activation(rows, cols):  # channels of different sizes
        return normal(rows, cols) * torch.exp(0.7 * normal(1, cols))

    s = {"case": case, "seed": int(seed)}
    if case["op"] == "adamw":
        at, total = offsets(case)
        inside = torch.zeros(total + 1, dtype=torch.int32, device=dev)
        starts = torch.tensor([a for a, _ in at], device=dev)
        ends = torch.tensor([a + n for a, n in at], device=dev)
        inside = inside.index_add_(0, starts, torch.ones_like(starts, dtype=torch.int32)).index_add_(0, ends, -torch.ones_like(ends, dtype=torch.int32))
        inside = inside.cumsum(0, dtype=torch.int32)[:total].to(torch.float32)  # 1 within a tensor, 0 in what pads its last block
        s["p"] = normal(total).mul_(0.02).mul_(inside)
        spread = torch.exp(normal(total // case["G"], 1)).expand(-1, case["G"]).reshape(-1)
        s["g"] = (normal(total) * spread * inside).mul_(1e-3).to(DTYPE[case["grad"]])
        s["copy"] = None if case["copy"] == "none" else s["p"].to(DTYPE[case["copy"]])
        s["clip"] = torch.tensor([CLIP], device=dev)
        if case["step"] == 1:
            m, r = torch.zeros(total, device=dev), torch.zeros(total, device=dev)
        else:
            m, r = (normal(total) * spread * inside).mul_(1e-4), (normal(total).abs_().add_(0.1) * spread * inside).mul_(4e-4)
        if case["state"] == "f32":
            s["m"], s["v"] = m, r * r
        else:
            for name, x in (("m", m), ("v", r)):
                scale, over = pow2_scale(x.view(-1, case["G"]).abs().amax(1, keepdim=True))
                s[name] = (x.view(-1, case["G"]) * over).reshape(-1).to(torch.float8_e4m3fn).view(torch.uint8)
                s[name + "_scales"] = scale.reshape(-1)
        s["params"] = [s["p"][a:a + n] for a, n in at]
        s["grads"] = [s["g"][a:a + n] for a, n in at]
        s["copies"] = None if s["copy"] is None else [s["copy"][a:a + n] for a, n in at]
    elif case["op"] == "trip":
        s["x"] = weight(case["rows"], case["cols"]).to(DTYPE[case["dtype"]])
    elif case["op"] == "matmul":
        s["a"] = plain_encode(activation(case["M"], case["K"]))
        s["b"] = plain_encode(weight(case["N"], case["K"]))
    else:
        s["x"] = activation(case["tokens"], case["in"]).to(torch.bfloat16).requires_grad_()
        s["w"] = weight(case["out"], case["in"]).to(torch.bfloat16).requires_grad_()
        s["dy"] = (normal(case["tokens"], case["out"]) * 1e-3).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------- the plain forms


def pow2_scale(absmax):
    """(scale, 1 / scale): 2^k with the smallest k >= -126 at which absmax / 2^k <= 448; a block of zeros has scale 0."""
    e = (((absmax.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp_(min=1)
    return torch.where(absmax == 0, 0.0, (e << 23).view(torch.float32)), ((254 - e) << 23).view(torch.float32)


def mix(x):
    """Scrambles 32 bits held in int64."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def key_of(seed, step):
    k = 0
    for word in (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF, step & 0xFFFFFFFF, step >> 32):
        k = mix((k + word + 0x9E3779B9) & 0xFFFFFFFF)
    return k


def to_e4m3(x, half, G):
    """fp32 values -> (codes, scales), rounded by the 16 random bits `half` of each."""
    scale, over = pow2_scale(x.view(-1, G).abs().amax(1, keepdim=True))
    q = (x.view(-1, G) * over).view(-1)
    small = torch.where(q.abs() < 2.0 ** -6, 2.0 ** -6, 0.0)  # below it the spacing stays 2^-9
    t = (((q.abs() + small).view(torch.int32) + (half << 4).to(torch.int32)) & ~0xFFFFF).view(torch.float32) - small
    return torch.copysign(t, q), scale.view(-1)


def plain_adamw(s):
    c, G = s["case"], s["case"]["G"]
    eight = c["state"] == "e4m3"
    value = lambda name: (s[name].view(torch.float8_e4m3fn).to(torch.float32).view(-1, G) * s[name + "_scales"].view(-1, 1)).view(-1)  # noqa: E731
    g = s["g"].to(torch.float32) * s["clip"]
    m = (value("m") if eight else s["m"]) * BETA1 + g * (1 - BETA1)
    v = (value("v").square() if eight else s["v"]) * BETA2 + (g * g) * (1 - BETA2)
    r = torch.sqrt(v)
    s["p"].mul_(1 - LR * DECAY).sub_(m * (LR / (1 - BETA1 ** c["step"])) / (r * (1 / math.sqrt(1 - BETA2 ** c["step"])) + EPS))
    if s["copy"] is not None:
        s["copy"].copy_(s["p"])
    if not eight:
        s["m"].copy_(m), s["v"].copy_(v)
        return {"p": s["p"], "copy": s["copy"], "m": s["m"], "v": s["v"]}
    h = mix(torch.arange(m.numel(), device=m.device) ^ key_of(s["seed"], c["step"]))
    t, scale = to_e4m3(m, h & 0xFFFF, G)
    s["m"].copy_(t.to(torch.float8_e4m3fn).view(torch.uint8)), s["m_scales"].copy_(scale)
    t, scale = to_e4m3(r, h >> 16, G)
    s["v"].copy_(torch.where(r > 0, t.clamp(min=2.0 ** -9), 0.0).to(torch.float8_e4m3fn).view(torch.uint8)), s["v_scales"].copy_(scale)
    return adamw_outputs(s)


def adamw_outputs(s):
    f8 = torch.float8_e4m3fn
    return {"p": s["p"], "copy": s["copy"], "m": s["m"].view(f8), "m_scales": s["m_scales"], "v": s["v"].view(f8), "v_scales": s["v_scales"]}


def plain_blocks(x):
    """[rows, cols] fp32 -> (E2M1 values of the padded rows before their scale, scale bytes)."""
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % 128)).view(x.shape[0], -1, 32)
    e = ((x.abs().amax(2).view(torch.int32) >> 23) - 2).clamp_(min=0)
    q = x * ((254 - e) << 23).view(torch.float32).unsqueeze(2)
    a = q.abs()
    spacing = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    value = torch.copysign((torch.round(a / spacing) * spacing).clamp_(max=6), q)
    return value.view(x.shape[0], -1), e.to(torch.uint8)


def scale_value(e):
    e = e.to(torch.int32)
    return torch.where(e == 0, 2.0 ** -127, (e << 23).view(torch.float32))


def plain_round(x):
    """fp32 -> fp32: through MXFP4 along the rows and back."""
    value, e = plain_blocks(x)
    return (value.view(x.shape[0], -1, 32) * scale_value(e).unsqueeze(2)).view(x.shape[0], -1)[:, :x.shape[1]]


def plain_decode(payload):
    codes, scales = payload
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    value = grid[torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1).to(torch.int32)]
    return (value.view(codes.shape[0], -1, 32) * scale_value(scales).unsqueeze(2)).view(codes.shape[0], -1)


def plain(s):
    c = s["case"]
    if c["op"] == "adamw":
        return plain_adamw(s)
    if c["op"] == "trip":
        x = s["x"].to(torch.float32)
        return plain_round(x.t().contiguous() if c["transpose"] else x).to(s["x"].dtype)
    if c["op"] == "matmul":
        return torch.matmul(plain_decode(s["a"]), plain_decode(s["b"]).t()).to(DTYPE[c["out"]])
    x, w, dy = (s[k].detach().to(torch.float32) for k in ("x", "w", "dy"))
    along = lambda t: plain_round(t.t().contiguous())  # blocks along the columns: the transpose's rows  # noqa: E731
    y = torch.matmul(plain_round(x), plain_round(w).t())
    dx = torch.matmul(plain_round(dy), along(w).t())
    dw = torch.matmul(along(dy), along(x).t())
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


# ---------------------------------------------------------------------------- the framework's calls


def run(s):
    if not own:
        return plain(s)
    import quantized_collective_payloads_amd as qcp
    c = s["case"]
    if c["op"] == "adamw":
        if "optimizer" not in s:  # the handle that a program keeps beside its tensors
            s["optimizer"] = qcp.AdamW(s["params"], copies=s["copies"], state=c["state"], G=c["G"], m=s["m"], v=s["v"], m_scales=s.get("m_scales"), v_scales=s.get("v_scales"))
        qcp.adamw_step(s["optimizer"], s["grads"], c["step"], LR, BETA1, BETA2, EPS, DECAY, grad_scale=s["clip"], seed=s["seed"])
        return {"p": s["p"], "copy": s["copy"], "m": s["m"], "v": s["v"]} if c["state"] == "f32" else adamw_outputs(s)
    if c["op"] == "trip":
        codes, scales = qcp.mxfp4_quantize(s["x"], transpose=c["transpose"])
        return qcp.mxfp4_dequantize(codes, scales, c["rows"] if c["transpose"] else c["cols"], s["x"].dtype)
    if c["op"] == "matmul":
        return qcp.mxfp4_matmul(*s["a"], *s["b"], dtype=DTYPE[c["out"]])
    y = qcp.mxfp4_linear(s["x"], s["w"])
    dx, dw = torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
    return {"y": y.detach(), "dx": dx, "dw": dw}


# ---------------------------------------------------------------------------- the definitions in 64 bits


def power_of_two(k):
    """2^k in float64, from its bits: torch's own powers may be an ulp off, which moves ties."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def exact_payload(x):
    """float64 [rows, cols] -> what its MXFP4 payload stands for, float64 [rows, cols]."""
    rows, cols = x.shape
    t = torch.zeros(rows, up(cols, 32), dtype=torch.float64, device=x.device)
    t[:, :cols] = x
    t = t.view(rows, -1, 32)
    big = t.abs().amax(2, keepdim=True)
    power = torch.where(big > 0, torch.frexp(big)[1] - 1 - 2, -127).clamp(min=-127)
    unit = power_of_two(power)
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    a = (t / unit).abs()
    at = torch.bucketize(a, middle)
    tie = (a == middle[at.clamp(max=6)]) & (at < 7) & (at % 2 == 1)
    return (torch.sign(t) * grid[at + tie] * unit).view(rows, -1)[:, :cols]


def exact_decode(payload):
    codes, scales = payload
    c = torch.stack((codes % 16, codes // 16), 2).view(codes.shape[0], -1).to(torch.float64)
    sign, c = torch.where(c >= 8, -1.0, 1.0).to(torch.float64), torch.remainder(c, 8)
    e, half = torch.div(c, 2, rounding_mode="floor"), torch.remainder(c, 2)
    value = torch.where(e == 0, half / 2, power_of_two(e - 1) * (1 + half / 2)) * sign
    return (value.view(codes.shape[0], -1, 32) * power_of_two(scales.to(torch.int64) - 127).unsqueeze(2)).view(codes.shape[0], -1)


def exact_hash(count, key, device):
    x = torch.arange(count, device=device, dtype=torch.int64).to(torch.int32) ^ torch.tensor(key, device=device).to(torch.int32)
    logical = lambda v, k: (v >> k) & ((1 << (32 - k)) - 1)  # noqa: E731
    x = (x ^ logical(x, 16)) * 0x6A09E667
    x = (x ^ logical(x, 15)) * (0xBB67AE85 - (1 << 32))
    x = x ^ logical(x, 16)
    return x & 0xFFFF, logical(x, 16)


def exact_e4m3(x, half, G, least):
    x = x.view(-1, G)
    mantissa, power = torch.frexp(x.abs().amax(1, keepdim=True) / 448)
    power = torch.where(mantissa == 0.5, power - 1, power).clamp(min=-126)
    scale = power_of_two(power)
    q = (x / scale).abs()
    unit = power_of_two((torch.frexp(q)[1] - 1).clamp(min=-6) - 3)
    q = torch.floor(q / unit + half.view(-1, G).to(torch.float64) / 65536) * unit
    q = torch.where(x != 0, q.clamp(min=2.0 ** -9 if least else 0.0), 0.0)
    return (torch.sign(x) * q).view(-1), torch.where(mantissa == 0, 0.0, scale).view(-1)


def exact(case, seed):
    s = prepare(case, seed)
    wide = lambda t: t.detach().to(torch.float64)  # noqa: E731
    if case["op"] == "adamw":
        G, eight = case["G"], case["state"] == "e4m3"
        held = lambda name: (wide(s[name].view(torch.float8_e4m3fn)).view(-1, G) * wide(s[name + "_scales"]).view(-1, 1)).view(-1)  # noqa: E731
        g = wide(s["g"]) * CLIP
        m = BETA1 * (held("m") if eight else wide(s["m"])) + (1 - BETA1) * g
        v = BETA2 * (held("v") ** 2 if eight else wide(s["v"])) + (1 - BETA2) * g ** 2
        p = wide(s["p"])
        p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** case["step"])) / (torch.sqrt(v / (1 - BETA2 ** case["step"])) + EPS)
        out = {"p": p, "copy": None if s["copy"] is None else p, "m": m, "v": v}
        if eight:
            low, high = exact_hash(m.numel(), key_of(s["seed"], case["step"]), m.device)
            out["m"], out["m_scales"] = exact_e4m3(m, low, G, False)
            out["v"], out["v_scales"] = exact_e4m3(torch.sqrt(v), high, G, True)
        return out
    if case["op"] == "trip":
        return exact_payload(wide(s["x"]).t().contiguous() if case["transpose"] else wide(s["x"]))
    if case["op"] == "matmul":
        return torch.matmul(exact_decode(s["a"]), exact_decode(s["b"]).t())
    x, w, dy = wide(s["x"]), wide(s["w"]), wide(s["dy"])
    columns = lambda t: exact_payload(t.t().contiguous())  # noqa: E731
    return {"y": torch.matmul(exact_payload(x), exact_payload(w).t()), "dx": torch.matmul(exact_payload(dy), columns(w).t()), "dw": torch.matmul(columns(dy), columns(x).t())}
