"""The operators around the NVFP4 block that finish a training step, and answer with single tokens: the 8-bit
floating-point linear layer with one scale per block of 128 (language-model head, sensitive projections), the
log probabilities of tokens with entropy, top alternatives and gradient, and the AdamW step over many tensors
with states in 8 or 32 bits.

``listed()`` and ``draw()`` say at which sizes they are measured, ``prepare()`` makes what a program has in hand
before the call, ``run()`` makes one call (the plain form, or with ``own`` the framework's kernels), ``exact()``
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.95, 1e-8, 3e-4, 0.1


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # One token of a sequence being generated, through the 1B model's MLP up-projection: all weights are read
        # for one row, latency counts.
        {"name": "fp8_fwd_one_token", "op": "fp8_fwd", "tokens": 1, "n": 5632, "k": 2048, "save": False},
        # A batch of sequences being generated, one token each, through the down-projection.
        {"name": "fp8_fwd_token_batch", "op": "fp8_fwd", "tokens": 96, "n": 2048, "k": 5632, "save": False},
        # Scoring one text of odd length with a vocabulary of odd size.
        {"name": "fp8_fwd_odd_vocabulary", "op": "fp8_fwd", "tokens": 1021, "n": 32003, "k": 2048, "save": False},
        # The language-model head in training: 8192 tokens of width 2048 to 32000 logits, the input's column form
        # kept for the weight gradient.
        {"name": "fp8_fwd_head", "op": "fp8_fwd", "tokens": 8192, "n": 32000, "k": 2048, "save": True},
        # A short ragged micro-batch's backward pass: both gradients of a projection.
        {"name": "fp8_bwd_ragged", "op": "fp8_bwd", "tokens": 777, "n": 5003, "k": 2048},
        # The head's backward pass: gradient of the hidden states and of the weights.
        {"name": "fp8_bwd_head", "op": "fp8_bwd", "tokens": 8192, "n": 32000, "k": 2048},
        # Serving: four sequences, one new token each, with the twenty likeliest alternatives.
        {"name": "logprobs_one_token", "op": "lp_fwd", "tokens": 4, "vocab": 131072, "dtype": "bf16", "top": 20,
         "masked": False, "temperature": 0.7},
        # Evaluation with constrained vocabularies: FP32 logits, banned entries at -inf (one row bans all), prompt
        # tokens that do not count, five alternatives.
        {"name": "logprobs_masked_f32", "op": "lp_fwd", "tokens": 515, "vocab": 50021, "dtype": "f32", "top": 5,
         "masked": True, "temperature": 1.0},
        # The training loss of the head above.
        {"name": "logprobs_train", "op": "lp_fwd", "tokens": 8192, "vocab": 32000, "dtype": "bf16", "top": 0,
         "masked": False, "temperature": 1.0},
        # Its gradient, with an entropy term.
        {"name": "logprobs_bwd_train", "op": "lp_bwd", "tokens": 8192, "vocab": 32000, "dtype": "bf16", "top": 0,
         "masked": False, "temperature": 1.0},
        # Norm weights and biases of a few layers, kept in 32 bits: many small tensors, latency counts.
        {"name": "adamw_small_f32", "op": "adamw", "tensors": 40, "largest": 5632, "smallest": 64, "bits": 32,
         "grad": "f32", "sr": False, "copy": False},
        # The matrices and norms of several layers with 8-bit states, BF16 gradients and a BF16 copy for the model.
        {"name": "adamw_layers_8bit", "op": "adamw", "tensors": 32, "largest": 2048 * 5632, "smallest": 2048,
         "bits": 8, "grad": "bf16", "sr": True, "copy": True},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fp8_fwd", "fp8_fwd", "fp8_bwd", "lp_fwd", "lp_bwd", "adamw"])
    if op in ("fp8_fwd", "fp8_bwd"):
        while True:
            t, n, k = _log_uniform(rng, 1, 8192), _log_uniform(rng, 256, 32003), _log_uniform(rng, 256, 8192)
            if rng.random() < 0.5:  # the sizes of most models
                n, k = n + 15 & ~15, k + 127 & ~127
            if 4.0 * t * n * k <= 4.0 * 8192 * 32000 * 2048 and (t * n + t * k + n * k) <= 600_000_000:
                break
        c = {"op": op, "tokens": t, "n": n, "k": k}
        if op == "fp8_fwd":
            c["save"] = rng.random() < 0.4
        return c
    if op in ("lp_fwd", "lp_bwd"):
        while True:
            t, v = _log_uniform(rng, 1, 8192), _log_uniform(rng, 1000, 131072)
            f32 = rng.random() < 0.4
            if t * v * (2 if f32 else 1) <= 8192 * 32000:
                break
        return {"op": op, "tokens": t, "vocab": v, "dtype": "f32" if f32 else "bf16",
                "top": rng.choice([0, 1, 5, 20, 32]), "masked": rng.random() < 0.4,
                "temperature": rng.choice([1.0, 1.0, 0.7, 1.3])}
    while True:
        count, largest = _log_uniform(rng, 1, 200), _log_uniform(rng, 1000, 2048 * 5632)
        if count * largest <= 32 * 2048 * 5632:
            break
    bits = rng.choice([8, 8, 32])
    return {"op": "adamw", "tensors": count, "largest": largest, "smallest": max(1, largest // 200), "bits": bits,
            "grad": rng.choice(["bf16", "f32"]), "sr": bits == 8 and rng.random() < 0.7, "copy": rng.random() < 0.5}


def _adamw_sizes(case):
    """Half of the tensors at the largest size, the rest spread down to the smallest, with odd ones among them."""
    n, hi, lo = case["tensors"], case["largest"], case["smallest"]
    sizes = []
    for i in range(n):
        if i % 2 == 0:
            sizes.append(hi)
        else:
            f = (i // 2 + 1) / max(1, n // 2)
            s = int(hi * (lo / hi) ** f)
            sizes.append(max(lo, s | 1 if i % 4 == 1 else s))
    return sizes


def work(case):
    op = case["op"]
    if op == "fp8_fwd":
        t, n, k = case["tokens"], case["n"], case["k"]
        saved = t * k * (1 + 1 / BLOCK) if case["save"] else 0
        return {"bytes": 2 * t * k + n * k + (n * k) / (BLOCK * BLOCK) + 2 * t * n + saved, "flops": 2.0 * t * n * k}
    if op == "fp8_bwd":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": 2 * t * n + n * k + t * k * (1 + 1 / BLOCK) + 2 * t * k + 2 * n * k, "flops": 4.0 * t * n * k}
    if op in ("lp_fwd", "lp_bwd"):
        t, v, size = case["tokens"], case["vocab"], 4 if case["dtype"] == "f32" else 2
        small = t * (8 + 4 + 4 + 8) + t * case["top"] * 12
        return {"bytes": t * v * size * (2 if op == "lp_bwd" else 1) + small, "flops": (5.0 if op == "lp_fwd" else 6.0) * t * v}
    n = sum(_adamw_sizes(case))
    per = 8 + (2 if case["grad"] == "bf16" else 4) + (16 if case["bits"] == 32 else 4 + 4 / BLOCK)
    return {"bytes": n * (per + (2 if case["copy"] else 0)), "flops": 15.0 * n}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _fp8_inputs(case, seed):
    g = _generator(seed)
    t, n, k = case["tokens"], case["n"], case["k"]
    x = torch.randn((t, k), device=DEV, generator=g)
    # a few channels of the hidden states are much larger than the rest
    x *= torch.where(torch.rand(k, device=DEV, generator=g) < 0.004, 20.0, 1.0)
    w = torch.randn((n, k), device=DEV, generator=g) * 0.02
    got = {"x": x.bfloat16(), "w": w.bfloat16()}
    if case["op"] == "fp8_bwd":
        # gradients differ by orders of magnitude from token to token
        size = torch.exp(torch.randn((t, 1), device=DEV, generator=g)) * 1e-4
        got["dy"] = (torch.randn((t, n), device=DEV, generator=g) * size).bfloat16()
    return got


def _logprob_inputs(case, seed):
    g = _generator(seed)
    t, v = case["tokens"], case["vocab"]
    z = torch.randn((t, v), device=DEV, generator=g) * 2.0
    targets = torch.randint(0, v, (t,), device=DEV, generator=g)
    # a model that has learnt something: the right token stands out in most rows
    z.scatter_add_(1, targets[:, None], torch.randn((t, 1), device=DEV, generator=g) * 3.0 + 6.0)
    if case["masked"]:
        banned = torch.rand(v, device=DEV, generator=g) < 0.3
        z.masked_fill_(banned[None, :] & (torch.rand((t, 1), device=DEV, generator=g) < 0.5), -math.inf)
        targets.masked_fill_(torch.rand(t, device=DEV, generator=g) < 0.2, -100)
        if t > 2:
            z[t // 2].fill_(-math.inf)
    z = z if case["dtype"] == "f32" else z.bfloat16()
    got = {"logits": z, "targets": targets}
    if case["op"] == "lp_bwd":
        got["g_logprob"] = -torch.rand(t, device=DEV, generator=g) / t
        got["g_entropy"] = -0.01 * torch.rand(t, device=DEV, generator=g) / t
        got["g_top"] = torch.randn((t, case["top"]), device=DEV, generator=g) * 0.1 / t if case["top"] else None
    return got


def _scale_bytes(amax, top):
    """The power-of-two scale of a block as its biased exponent: the least 2^e with amax <= 1.75 * 2^(top + e)."""
    bits = amax.contiguous().view(torch.int32)
    return ((bits >> 23) - top + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(0, 254)


def _power(byte):
    """2^(byte - 127) in FP32 (byte 0 is a subnormal number)."""
    return torch.where(byte == 0, 0x400000, byte.int() << 23).view(torch.float32)


def _adamw_inputs(case, seed):
    g = _generator(seed)
    sizes = _adamw_sizes(case)
    blocks = [(s + BLOCK - 1) // BLOCK for s in sizes]
    total = sum(blocks) * BLOCK
    valid = torch.zeros(total, dtype=torch.bool, device=DEV)
    at = 0
    places = []
    for s, b in zip(sizes, blocks):
        valid[at:at + s] = True
        places.append((at, s))
        at += b * BLOCK
    level = torch.exp(torch.randn((total // BLOCK, 1), device=DEV, generator=g))
    noise = lambda: (torch.randn((total // BLOCK, BLOCK), device=DEV, generator=g) * level).view(-1)  # noqa: E731
    keep = lambda a: torch.where(valid, a, torch.zeros((), device=DEV))  # noqa: E731
    got = {"places": places, "blocks": blocks, "step": 100}
    got["param"] = keep(torch.randn(total, device=DEV, generator=g) * 0.02)
    grad = keep(noise() * 1e-3)
    got["grad"] = grad.bfloat16() if case["grad"] == "bf16" else grad
    m = keep(noise() * 3e-4)
    v = keep(torch.square(noise() * 1e-3) + torch.square(noise() * 1e-4))
    got["copy"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV) if case["copy"] else None
    if case["bits"] == 32:
        got["m"], got["v"], got["m_scale"], got["v_scale"] = m, v, None, None
    else:
        for name, a, top, kind in (("m", m, 8, torch.float8_e4m3fn), ("v", v, 15, torch.float8_e5m2)):
            a = a.view(-1, BLOCK)
            byte = _scale_bytes(a.abs().amax(1), top)
            got[name] = (a / _power(byte)[:, None]).to(kind).view(-1)
            got[name + "_scale"] = byte.to(torch.uint8)
    decay = [0.0 if s <= 2048 else DECAY for s in sizes]
    got["decay"] = decay
    return got


def prepare(case, seed):
    if case["op"] == "adamw":
        s = _adamw_inputs(case, seed)
        s["case"] = case
        if own:
            import nvfp4_quantized_pretraining_gb300 as F
            cut = lambda a: None if a is None else [a[o:o + n] for o, n in s["places"]]  # noqa: E731
            ends = [0]
            for b in s["blocks"]:
                ends.append(ends[-1] + b)
            scales = lambda a: None if a is None else [a[i:j] for i, j in zip(ends, ends[1:])]  # noqa: E731
            s["plan"] = F.AdamWTensors(cut(s["param"]), cut(s["grad"]), cut(s["m"]), cut(s["v"]),
                                       scales(s["m_scale"]), scales(s["v_scale"]), model=cut(s["copy"]),
                                       weight_decay=s["decay"])
        else:
            count = torch.tensor(s["blocks"], device=DEV)
            nb = int(sum(s["blocks"]))
            tensor = torch.repeat_interleave(torch.arange(len(s["blocks"]), device=DEV), count, output_size=nb)
            first = torch.cumsum(count, 0) - count
            s["tensor"], s["block"] = tensor, torch.arange(nb, device=DEV) - first[tensor]
            s["factor"] = torch.tensor([1.0 - LR * d for d in s["decay"]], device=DEV, dtype=torch.float32)[tensor]
        return s
    if case["op"] in ("lp_fwd", "lp_bwd"):
        s = _logprob_inputs(case, seed)
        s["case"] = case
        if case["op"] == "lp_bwd":  # what the forward pass left
            if own:
                import nvfp4_quantized_pretraining_gb300 as F
                s["saved"] = F.fp4_token_logprobs(s["logits"], s["targets"], top_k=case["top"],
                                                  temperature=case["temperature"])
            else:
                s["saved"] = _logprobs_plain(s["logits"], s["targets"], case["top"], case["temperature"])
        return s
    s = _fp8_inputs(case, seed)
    s["case"] = case
    w = s.pop("w")
    if own:
        import nvfp4_quantized_pretraining_gb300 as F
        if case["op"] == "fp8_fwd":
            s["wq"] = F.fp4_fp8_quantize(w, block_rows=BLOCK)
        else:
            s["wqT"] = F.fp4_fp8_quantize_transposed(w, block_rows=BLOCK)
            s["xqT"] = F.fp4_fp8_quantize_transposed(s.pop("x"))
    else:
        s["wq"] = _quantize_plain(w, BLOCK)
        if case["op"] == "fp8_bwd":
            s["xqT"] = _quantize_plain(s.pop("x").t(), 1)
    return s


# ---------------------------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------------------------
def _quantize_plain(x, block_rows):
    """E4M3 values of x (rows x cols) with a power-of-two scale for each block of block_rows x 128; and the scales
    as biased exponents."""
    rows, cols = x.shape
    r, c = -(-rows // block_rows), -(-cols // BLOCK)
    p = torch.zeros((r * block_rows, c * BLOCK), device=x.device)
    p[:rows, :cols] = x.float()
    p = p.view(r, block_rows, c, BLOCK)
    byte = _scale_bytes(p.abs().amax((1, 3)), 8)
    codes = (p / _power(byte)[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(r * block_rows, c * BLOCK)[:rows, :cols], byte


def _dequantize_plain(q, block_rows):
    codes, byte = q
    scale = _power(byte).repeat_interleave(block_rows, 0).repeat_interleave(BLOCK, 1)
    return codes.float() * scale[:codes.shape[0], :codes.shape[1]]


def _fp8_fwd_plain(s):
    x = s["x"]
    y = torch.matmul(_dequantize_plain(_quantize_plain(x, 1), 1), _dequantize_plain(s["wq"], BLOCK).t()).bfloat16()
    return {"y": y, "saved": _quantize_plain(x.t(), 1)[0]} if s["case"]["save"] else {"y": y}


def _fp8_bwd_plain(s):
    dy = s["dy"]
    dx = torch.matmul(_dequantize_plain(_quantize_plain(dy, 1), 1), _dequantize_plain(s["wq"], BLOCK))
    dw = torch.matmul(_dequantize_plain(_quantize_plain(dy.t(), 1), 1), _dequantize_plain(s["xqT"], 1).t())
    return {"dx": dx.bfloat16(), "dw": dw.bfloat16()}


def _logprobs_plain(logits, targets, top, temperature):
    inv = 1.0 / temperature
    z = logits.float()
    most = z.amax(1, keepdim=True)
    empty = most == -math.inf
    x = torch.where(z == -math.inf, z, (z - most) * inv)  # (an empty row has -inf throughout)
    e = torch.exp(x)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    # entropy = log sum e^x - sum e^x x / sum e^x; a banned entry adds nothing
    mean = torch.where(z == -math.inf, 0.0, e * x).sum(1, keepdim=True) / total
    entropy = torch.where(empty, 0.0, log_total - mean)[:, 0]
    at = targets.clamp(min=0)[:, None]
    logprob = torch.where(empty, -math.inf, x.gather(1, at) - log_total)[:, 0]
    logprob = torch.where(targets < 0, 0.0, logprob)
    got = {"logprob": logprob, "entropy": entropy, "most": most[:, 0], "total": total[:, 0]}
    if top:
        index = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :top]
        got["top_index"] = index
        got["top_logprob"] = torch.where(empty, -math.inf, x.gather(1, index) - log_total)
    return got


def _logprobs_bwd_plain(s):
    c, z, f = s["case"], s["logits"].float(), s["saved"]
    inv = 1.0 / c["temperature"]
    counts = s["targets"] >= 0
    g = torch.where(counts, s["g_logprob"], 0.0)
    all_g = g + s["g_top"].sum(1) if c["top"] else g
    masked = z == -math.inf
    x = (z - f["most"][:, None]) * inv
    p = torch.where(masked, 0.0, torch.exp(x) / f["total"][:, None])
    logp = torch.where(masked, 0.0, x - torch.log(f["total"])[:, None])
    d = p * (-all_g[:, None] - s["g_entropy"][:, None] * (logp + f["entropy"][:, None]))
    d.scatter_add_(1, s["targets"].clamp(min=0)[:, None], g[:, None])
    if c["top"]:
        d.scatter_add_(1, f["top_index"], s["g_top"])
    return {"dlogits": torch.where(masked, 0.0, d * inv).to(s["logits"].dtype)}


def _philox_plain(low, stream, step, seed):
    """The four 32-bit words of Philox4x32-10 of the counters (low, 0, stream, step), as int64."""
    mask = 0xFFFFFFFF
    c0, c1, c2, c3 = low, torch.zeros_like(low), stream, torch.full_like(low, step)
    k0, k1 = seed & mask, seed >> 32
    for _ in range(10):  # the generator's rounds
        h0 = (c0 >> 16) * 0xD2511F53 + ((c0 & 0xFFFF) * 0xD2511F53 >> 16) >> 16
        h1 = (c2 >> 16) * 0xCD9E8D57 + ((c2 & 0xFFFF) * 0xCD9E8D57 >> 16) >> 16
        l0, l1 = c0 * 0xD2511F53 & mask, c2 * 0xCD9E8D57 & mask
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = k0 + 0x9E3779B9 & mask, k1 + 0xBB67AE85 & mask
    return c0, c1, c2, c3


def _random16_plain(s, which, step, seed):
    """16 random bits for each element, [blocks, 128]: group j of eight elements of tensor t takes the halves of the
    words of counter (j, 0, 2 t + which, step), low half first."""
    j = s["block"][:, None] * 16 + torch.arange(16, device=DEV)
    words = torch.stack(_philox_plain(j, (2 * s["tensor"] + which)[:, None].expand_as(j).contiguous(), step, seed), 2)
    return torch.stack((words & 0xFFFF, words >> 16), 3).view(-1, BLOCK).int()


def _store8_plain(a, top, shift, kind, random):
    """a [blocks, 128] FP32 in 8 bits: one power-of-two scale per block, stochastic rounding by 16 random bits, or to
    nearest even; a positive number of the unsigned kind stays above zero."""
    byte = _scale_bytes(a.abs().amax(1), top)
    # a * 2^-e * 2^-(126 - least normal exponent): the code is then the top bits of the FP32 pattern
    y = a / _power(byte)[:, None] * (2.0 ** -120 if shift == 20 else 2.0 ** -112)
    bits = y.view(torch.int32)
    size = bits & 0x7FFFFFFF
    if random is not None:
        code = size + (random << (shift - 16)) >> shift
    else:
        code = size + ((1 << (shift - 1)) - 1) + (size >> shift & 1) >> shift
    if shift == 21:
        code = torch.where((code == 0) & (a > 0), 1, code)
    code = code | (bits >> 24 & 0x80)
    return code.to(torch.uint8).view(kind).view(-1), byte.to(torch.uint8)


def _adamw_plain(s):
    c, step = s["case"], s["step"]
    s["step"] += 1
    blocks = lambda a: a.view(-1, BLOCK)  # noqa: E731
    g = blocks(s["grad"]).float()
    if c["bits"] == 8:
        m = blocks(s["m"]).float() * _power(s["m_scale"].int())[:, None]
        v = blocks(s["v"]).float() * _power(s["v_scale"].int())[:, None]
    else:
        m, v = blocks(s["m"]), blocks(s["v"])
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * (g * g)
    size, root = LR / (1.0 - BETA1 ** step), 1.0 / math.sqrt(1.0 - BETA2 ** step)
    p = blocks(s["param"]) * s["factor"][:, None] - size * (m / (torch.sqrt(v) * root + EPS))
    s["param"] = p.view(-1)
    if c["bits"] == 8:
        r = [_random16_plain(s, w, step, 1234) if c["sr"] else None for w in (0, 1)]
        s["m"], s["m_scale"] = _store8_plain(m, 8, 20, torch.float8_e4m3fn, r[0])
        s["v"], s["v_scale"] = _store8_plain(v, 15, 21, torch.float8_e5m2, r[1])
    else:
        s["m"], s["v"] = m.view(-1), v.view(-1)
    if c["copy"]:
        s["copy"] = s["param"].bfloat16()
    return _adamw_outputs(s)


def _adamw_outputs(s):
    names = ("param", "m", "v", "m_scale", "v_scale", "copy")
    return {n: s[n] for n in names if s[n] is not None}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "fp8_fwd":
            return _fp8_fwd_plain(s)
        if op == "fp8_bwd":
            return _fp8_bwd_plain(s)
        if op == "lp_fwd":
            return _logprobs_plain(s["logits"], s["targets"], c["top"], c["temperature"])
        return _logprobs_bwd_plain(s) if op == "lp_bwd" else _adamw_plain(s)
    import nvfp4_quantized_pretraining_gb300 as F
    if op == "fp8_fwd":
        y, saved = F.fp4_fp8_linear_fwd(s["x"], s["wq"], save=c["save"])
        return {"y": y, "saved": saved.values()} if c["save"] else {"y": y}
    if op == "fp8_bwd":
        dx, dw = F.fp4_fp8_linear_bwd(s["dy"], s["wqT"], s["xqT"])
        return {"dx": dx, "dw": dw}
    if op == "lp_fwd":
        r = F.fp4_token_logprobs(s["logits"], s["targets"], top_k=c["top"], temperature=c["temperature"])
        got = {"logprob": r.logprob, "entropy": r.entropy, "most": r.stats[:, 0], "total": r.stats[:, 1]}
        if c["top"]:
            got["top_index"], got["top_logprob"] = r.top_index, r.top_logprob
        return got
    if op == "lp_bwd":
        return {"dlogits": F.fp4_token_logprobs_bwd(s["logits"], s["saved"], s["targets"], g_logprob=s["g_logprob"],
                                                    g_entropy=s["g_entropy"], g_top=s["g_top"])}
    F.fp4_adamw_step(s["plan"], s["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS,
                     round_mode=F.SR if c["sr"] else F.RTN, seed=1234)
    s["step"] += 1
    return _adamw_outputs(s)


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_power(e):
    return (e.long() + 1023 << 52).view(torch.float64)


def _exact_exponent(amax, largest):
    """The least e, not below -127, with amax <= largest * 2^e."""
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, 2.0 ** -140)) / largest))
    e = torch.where(largest * _exact_power(e - 1) >= amax, e - 1, e)
    return torch.where(largest * _exact_power(e) < amax, e + 1, e).clamp(min=-127)


def _exact_e4m3(x, block_rows):
    """Values (FP64) of x rounded to E4M3 under the block's scale, the codes' values, by counting in steps."""
    rows, cols = x.shape
    x = x.double()
    r, c = -(-rows // block_rows), -(-cols // BLOCK)
    x = torch.nn.functional.pad(x, (0, c * BLOCK - cols, 0, r * block_rows - rows))
    x = x.reshape(r, block_rows, c, BLOCK).transpose(1, 2)
    e = _exact_exponent(x.abs().amax((2, 3), keepdim=True), 448.0)
    y = x * _exact_power(-e)
    least = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))  # the binade; below 2^-6 the steps stay 2^-9
    step = _exact_power(least - 3)
    y = torch.round(y / step) * step
    back = lambda a: a.transpose(1, 2).reshape(r * block_rows, c * BLOCK)[:rows, :cols]  # noqa: E731
    return back(y * _exact_power(e)), back(y)


def _exact_fp8(case, seed):
    i = _fp8_inputs(case, seed)
    w = _exact_e4m3(i["w"], BLOCK)[0]
    if case["op"] == "fp8_fwd":
        y = torch.matmul(_exact_e4m3(i["x"], 1)[0], w.t())
        return {"y": y, "saved": _exact_e4m3(i["x"].t(), 1)[1]} if case["save"] else {"y": y}
    dx = torch.matmul(_exact_e4m3(i["dy"], 1)[0], w)
    dw = torch.matmul(_exact_e4m3(i["dy"].t(), 1)[0], _exact_e4m3(i["x"].t(), 1)[0].t())
    return {"dx": dx, "dw": dw}


def _exact_logprobs(case, seed):
    i = _logprob_inputs(case, seed)
    z = i["logits"].double()
    t, top = case["tokens"], case["top"]
    a = z / case["temperature"]
    most = z.amax(1)
    empty = torch.isinf(most)
    lse = torch.logsumexp(a, 1)
    lp = torch.where(empty[:, None], -math.inf, a - torch.where(empty, 0.0, lse)[:, None])
    p = torch.exp(lp)
    entropy = -torch.xlogy(p, p).sum(1)
    valid = i["targets"] >= 0
    rows = torch.arange(t, device=DEV)
    to = torch.where(valid, i["targets"], 0)
    order = torch.argsort(z, dim=1, descending=True, stable=True)[:, :top] if top else None
    if case["op"] == "lp_fwd":
        got = {"logprob": torch.where(valid, lp[rows, to], 0.0), "entropy": entropy, "most": most,
               "total": torch.where(empty, 0.0, torch.exp(lse - most / case["temperature"]))}
        if top:
            got["top_index"], got["top_logprob"] = None, lp.gather(1, order)
        return got
    # the gradient of sum(g_logprob logprob + g_entropy entropy + g_top top_logprob)
    gl, gh = torch.where(valid, i["g_logprob"].double(), 0.0), i["g_entropy"].double()
    onto = torch.zeros_like(z)
    onto[rows, to] += gl
    if top:
        onto.scatter_add_(1, order, i["g_top"].double())
    d = onto - onto.sum(1, keepdim=True) * p - gh[:, None] * (torch.xlogy(p, p) + p * entropy[:, None])
    return {"dlogits": torch.where(torch.isinf(z), 0.0, d / case["temperature"])}


def _exact_adamw(case, seed):
    i = _adamw_inputs(case, seed)
    step = i["step"]
    spread = lambda b: _exact_power(b.long() - 127).repeat_interleave(BLOCK)  # noqa: E731
    m, v, g = i["m"].double(), i["v"].double(), i["grad"].double()
    if case["bits"] == 8:
        m, v = m * spread(i["m_scale"]), v * spread(i["v_scale"])
    decay = torch.cat([torch.full((b * BLOCK,), d, device=DEV, dtype=torch.float64)
                       for b, d in zip(i["blocks"], i["decay"])])
    m += (g - m) * (1.0 - BETA1)
    v += (g * g - v) * (1.0 - BETA2)
    p = i["param"].double()
    p = p - LR * decay * p - LR * (m / (1.0 - BETA1 ** step)) / (torch.sqrt(v / (1.0 - BETA2 ** step)) + EPS)
    got = {"param": p, "m": m, "v": v}
    if case["bits"] == 8:  # the moments in units of their block's scale, before they are rounded to 8 bits
        for name, largest in (("m", 448.0), ("v", 57344.0)):
            a = got[name].view(-1, BLOCK)
            got[name] = (a * _exact_power(-_exact_exponent(a.abs().amax(1, keepdim=True), largest))).view(-1)
            got[name + "_scale"] = None
    if case["copy"]:
        got["copy"] = p
    return got


def exact(case, seed):
    if case["op"] == "adamw":
        return _exact_adamw(case, seed)
    return _exact_logprobs(case, seed) if case["op"] in ("lp_fwd", "lp_bwd") else _exact_fp8(case, seed)
