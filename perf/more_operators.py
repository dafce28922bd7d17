"""Measured cases of the optimiser step, the 8-bit head and the beam search operators.

A case is one call (or the two that belong together) of a user's program: an
AdamW step over a list of tensors, bringing a matrix to 8 bits with a scale for
each block, the logits of an 8-bit head, the choice of the next beams over the
vocabulary, or the reordering of the beams' states.  ``own`` selects the
framework's kernels; otherwise the same results come from elementary torch
operations.
"""
import math

import torch

own = False

V_WIDE = 151936  # the framework's vocabulary (inputs.V_QWEN3)
D_HEAD = 4096    # the width of its lm_head
BLOCK = 128      # elements that share a scale


def listed():
    return [
        # The biases and norms of a model, fp32 throughout: launch latency.
        {"name": "adamw_small", "op": "adamw", "n": 16, "lo": 1, "hi": 5000, "p": "f32", "g": "f32",
         "bits": 32, "max": 0.0, "random": False},
        # A bf16 model's tensors with states of 8 bits, gradients clipped on the way, roundings drawn.
        {"name": "adamw_model_8bit", "op": "adamw", "n": 20, "lo": 1000, "hi": 20000000, "p": "bf16", "g": "bf16",
         "bits": 8, "max": 1.0, "random": True},
        # The activations of a small odd layer, a scale for each run of 128 in a row.
        {"name": "quantize_rows", "op": "quantize", "T": 333, "K": 1000, "dtype": "f32", "rows": 1, "pad": 8},
        # The head's weight after an optimiser step, a scale for each block of 128 x 128.
        {"name": "quantize_head", "op": "quantize", "T": V_WIDE, "K": D_HEAD, "dtype": "bf16", "rows": 128, "pad": 0},
        # The logits of one sequence's next token: the weight is read once.
        {"name": "head_one", "op": "head", "T": 1, "N": V_WIDE, "K": D_HEAD, "dtype": "bf16", "out": "bf16"},
        # A rollout batch of odd size, fp32 logits for the sampler.
        {"name": "head_batch_f32", "op": "head", "T": 201, "N": V_WIDE, "K": D_HEAD, "dtype": "bf16", "out": "f32"},
        # Scoring prompts: every position's logits.
        {"name": "head_prompts", "op": "head", "T": 4096, "N": V_WIDE, "K": D_HEAD, "dtype": "bf16", "out": "bf16"},
        # One request with four beams, eight candidates of which some may end: latency.
        {"name": "beams_one", "op": "beams", "B": 1, "beams": 4, "n": 8, "V": V_WIDE, "dtype": "bf16", "pad": 0,
         "flat": 0.0, "mask": 0.0, "dead": 0.0},
        # A small vocabulary of odd size in padded fp32 rows, half of it masked (a grammar), some beams dead.
        {"name": "beams_grammar", "op": "beams", "B": 33, "beams": 3, "n": 6, "V": 10007, "dtype": "f32", "pad": 9,
         "flat": 0.0, "mask": 0.5, "dead": 0.2},
        # A served batch of wide searches.
        {"name": "beams_batch", "op": "beams", "B": 64, "beams": 16, "n": 32, "V": V_WIDE, "dtype": "bf16", "pad": 0,
         "flat": 0.02, "mask": 0.0, "dead": 0.0},
        # Recurrent states of a small search, into a second set of buffers.
        {"name": "reorder_small", "op": "reorder", "B": 4, "beams": 5, "tensors": 12, "heads": 1, "length": 1, "room": 1,
         "width": 1000, "dtype": "f32", "place": False},
        # The filled part of a key and value cache, in place.
        {"name": "reorder_cache", "op": "reorder", "B": 16, "beams": 8, "tensors": 8, "heads": 8, "length": 1501, "room": 2048,
         "width": 128, "dtype": "bf16", "place": True},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["adamw", "adamw", "quantize", "head", "head", "beams", "beams", "reorder"])
    if op == "adamw":
        lo = spread(1, 10000)
        bits = rng.choice([8, 32])
        return {"op": op, "n": spread(1, 20), "lo": lo, "hi": lo + spread(1, 12000000),
                "p": rng.choice(["bf16", "f32"]), "g": rng.choice(["bf16", "f32"]), "bits": bits,
                "max": rng.choice([0.0, 1.0, 1e6]), "random": rng.random() < 0.6}
    if op == "quantize":
        rows = rng.choice([1, 128])
        return {"op": op, "T": spread(1, 60000), "K": 8 * spread(1, 1024), "dtype": rng.choice(["bf16", "f32"]),
                "rows": rows, "pad": rng.choice([0, 0, 8, rng.randint(1, 64)])}
    if op == "head":
        N = rng.choice([V_WIDE, spread(1000, V_WIDE), spread(1000, V_WIDE) | 1])
        return {"op": op, "T": spread(1, 3000), "N": N, "K": 16 * spread(8, D_HEAD // 16),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "out": rng.choice(["bf16", "f32"])}
    if op == "beams":
        beams = spread(1, 24)
        V = rng.choice([V_WIDE, spread(2000, V_WIDE), spread(2000, V_WIDE) | 1])
        return {"op": op, "B": max(1, spread(1, 700) // beams), "beams": beams,
                "n": max(1, min(48, rng.choice([beams, 2 * beams, 2 * beams + 1]))), "V": V,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "pad": rng.choice([0, 0, 8, rng.randint(1, 64)]),
                "flat": rng.choice([0.0, 0.0, 0.1]), "mask": rng.choice([0.0, 0.0, 0.3]),
                "dead": rng.choice([0.0, 0.0, 0.3])}
    beams = spread(1, 16)
    length = spread(1, 1500)
    return {"op": op, "B": max(1, spread(1, 100) // beams), "beams": beams, "tensors": spread(1, 12),
            "heads": rng.choice([1, 2, 8]), "length": length, "room": length + rng.choice([0, 1, spread(1, 600)]),
            "width": rng.choice([1, 64, 128, rng.randint(1, 300)]), "dtype": rng.choice(["bf16", "f32"]),
            "place": rng.random() < 0.5}


# ---- inputs -----------------------------------------------------------------

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


LR, BETA1, BETA2, EPS, DECAY = 1e-4, 0.9, 0.999, 1e-8, 0.01
STEP = 250


def _adamw_sizes(case):
    rng = torch.Generator().manual_seed(7)  # the shapes are the model's, not the seed's
    u = torch.rand(case["n"], generator=rng, dtype=torch.float64)
    lo, hi = math.log(case["lo"]), math.log(case["hi"])
    return [int(round(math.exp(lo + float(x) * (hi - lo)))) for x in u]


def _slices(flat, sizes):
    """Tensors one behind another in a flat buffer, each from a multiple of 128 elements."""
    out, at = [], 0
    for n in sizes:
        out.append(flat[at:at + n])
        at += -(-n // BLOCK) * BLOCK
    return out


def _prepare_adamw(case, seed, g):
    sizes = _adamw_sizes(case)
    total = sum(-(-n // BLOCK) * BLOCK for n in sizes)

    def flat(dtype):
        return torch.zeros(total, dtype=dtype, device="cuda")

    s = {"seed": seed * 7919 + 13 if case["random"] else None, "max": case["max"],
         "p_flat": flat(_type(case["p"])), "g_flat": flat(_type(case["g"]))}
    s["p"], s["g"] = _slices(s["p_flat"], sizes), _slices(s["g_flat"], sizes)
    if case["bits"] == 32:
        s["m_flat"], s["v_flat"] = flat(torch.float32), flat(torch.float32)
        s["m"], s["v"] = _slices(s["m_flat"], sizes), _slices(s["v_flat"], sizes)
    else:  # codes, and behind them one scale for each block
        s["m"] = [torch.zeros(n + -(-n // BLOCK), dtype=torch.uint8, device="cuda") for n in sizes]
        s["v"] = [torch.zeros_like(x) for x in s["m"]]
        s["m_out"], s["v_out"] = flat(torch.float32), flat(torch.float32)
        s["out"] = (_slices(s["m_out"], sizes), _slices(s["v_out"], sizes))
    for i, n in enumerate(sizes):
        # gradients of a layer's own size, wide within it; moments of a run in progress
        size = 10.0 ** (-2 - i % 4) * torch.exp(torch.randn(n, generator=g, device="cuda"))
        s["p"][i].copy_(0.05 * torch.randn(n, generator=g, device="cuda"))
        s["g"][i].copy_(size * torch.randn(n, generator=g, device="cuda"))
        m = 0.3 * size * torch.randn(n, generator=g, device="cuda")
        v = (size * (0.5 + torch.rand(n, generator=g, device="cuda"))).square()
        v[::101] = 0.0
        if case["bits"] == 32:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
        else:
            draws = torch.full((n,), 1 << 19, dtype=torch.int64, device="cuda")
            s["m"][i].copy_(_encode(m, draws, 14, True)[0])
            s["v"][i].copy_(_encode(v, draws, 30, False)[0])
    total_sq = s["g_flat"].double().square().sum()
    s["norm"] = torch.sqrt(total_sq).float()
    return s


def _logits(case, T, g):
    """Language-model-like rows: a bulk N(0, 2^2) and, but for the share `flat`
    of rows, 48 columns raised by up to 14 to 24; `mask` of the columns at -inf."""
    V, dt = case["V"], _type(case["dtype"])
    store = torch.zeros(T, V + case["pad"], dtype=dt, device="cuda")
    out = store[:, :V]
    n_flat = int(round(case["flat"] * T))
    for r0 in range(0, T, 256):
        n = min(256, T - r0)
        z = torch.randn(n, V, generator=g, device="cuda").mul_(2.0)
        height = 14.0 + 10.0 * torch.rand(n, 1, generator=g, device="cuda")
        cols = torch.randint(0, V, (n, 48), generator=g, device="cuda")
        rise = height * torch.rand(n, 48, generator=g, device="cuda")
        rise[:max(0, min(n, n_flat - r0))] = 0.0
        z.scatter_add_(1, cols, rise)
        if case["mask"] > 0:
            off = torch.rand(n, V, generator=g, device="cuda") < case["mask"]
            off[:, :2] = False
            z[off] = -math.inf
        out[r0:r0 + n] = z.to(dt)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "adamw":
        s.update(_prepare_adamw(case, seed, g))
    elif case["op"] == "quantize":
        T, K = case["T"], case["K"]
        store = torch.empty(T, K + case["pad"], dtype=_type(case["dtype"]), device="cuda")
        wide = 0.02 if case["rows"] == 128 else 1.0
        store.copy_(wide * torch.randn(T, K + case["pad"], generator=g, device="cuda"))
        s["x"] = store[:, :K]
        s["x"][:, ::97] *= 30  # a few loud channels
        s["x"][:, :min(K, BLOCK)][T // 2:T // 2 + 1] = 0  # a block of zeros
    elif case["op"] == "head":
        T, N, K = case["T"], case["N"], case["K"]
        x = torch.randn(T, K, generator=g, device="cuda")
        x[:, ::97] *= 10
        s["x"] = x.to(_type(case["dtype"]))
        # a head of 8 bits as a checkpoint holds it, with scales of its own
        s["W"] = torch.empty(N, K, dtype=torch.float8_e4m3fn, device="cuda")
        for r in range(0, N, 16384):
            w = 60.0 * torch.randn(min(16384, N - r), K, generator=g, device="cuda")
            s["W"][r:r + 16384] = w.clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["Ws"] = 0.0003 * (0.5 + torch.rand(-(-N // BLOCK), -(-K // BLOCK), generator=g, device="cuda"))
    elif case["op"] == "beams":
        B, beams = case["B"], case["beams"]
        s["z"] = _logits(case, B * beams, g)
        s["scores"] = -20.0 * torch.rand(B, beams, generator=g, device="cuda")
        s["scores"][torch.rand(B, beams, generator=g, device="cuda") < case["dead"]] = -math.inf
    else:
        B, beams = case["B"], case["beams"]
        s["parents"] = torch.randint(0, beams, (B, beams), generator=g, device="cuda")
        s["states"], s["out"] = [], []
        for _ in range(case["tensors"]):
            shape = (B * beams, case["heads"], case["room"], case["width"])
            x = torch.empty(shape, dtype=_type(case["dtype"]), device="cuda").normal_(generator=g)
            s["states"].append(x[:, :, :case["length"]])
            s["out"].append(torch.empty_like(x)[:, :, :case["length"]])
    return s


# ---- the plain form -----------------------------------------------------------

def _mix(x, key):
    """32 bits that are as good as random, for the counters x of one key."""
    low = 0xFFFFFFFF
    x = (x ^ key) & low
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & low
    x = x ^ (x >> 15)
    x = (x + key) & low
    x = (x * 0xBB67AE85) & low
    return x ^ (x >> 16)


def _key(seed, tensor):
    key = _mix(seed & 0xFFFFFFFF, 0x9E3779B9)
    key = _mix(key ^ (seed >> 32 & 0xFFFFFFFF), 0x3C6EF372)
    return _mix(key ^ tensor, 0xDAA66D2B)


def _draws(seed, tensor, n):
    """(20 bits for the first moment, for the second, 16 for the parameter) of every element."""
    if seed is None:
        half = torch.full((n,), 1 << 19, dtype=torch.int64, device="cuda")
        return half, half, None
    key = _key(seed, tensor)
    r = _mix(torch.arange(n, dtype=torch.int64, device="cuda"), key)
    return (r >> 16) << 4 | 8, (r & 0xFFFF) << 4 | 8, _mix(r, key ^ 0xA54FF53A) >> 16


def _encode(x, draws, depth, signed):
    """8-bit codes with one exponent for each block of 128, and the values they
    stand for: three bits of mantissa and an exponent that reaches `depth`
    binary orders below the block's largest, rounded where the draw says."""
    n = x.numel()
    bits = x.view(torch.int32).to(torch.int64) & 0x7FFFFFFF
    lost = bits >= 0x7F800000
    rest = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.int64, device="cuda")
    rest[:n] = torch.where(lost, torch.zeros_like(bits), bits)
    top = rest.view(-1, BLOCK).amax(dim=1) >> 23
    base = torch.clamp((top - depth) * 8, min=0).repeat_interleave(BLOCK)[:n]
    code = ((bits + draws) >> 20) - base
    below = (bits >> 20) - base < 1
    least = ((base + 1) << 20).to(torch.int32).view(torch.float32)
    if signed:  # below the least value: that or zero
        up = x.abs() > least * (draws.float() * 2.0**-20)
        code = torch.where(below, up.to(torch.int64), code)
    else:  # never from above zero to zero: an update is divided by the root
        code = torch.where(bits > 0, torch.where(below, torch.ones_like(code), code), torch.zeros_like(code))
    value = torch.where(code > 0, (code + base) << 20, torch.zeros_like(code)).to(torch.int32).view(torch.float32)
    value = torch.where(lost, torch.full_like(value, math.nan), value)
    code = torch.where(lost, torch.full_like(code, 127 if signed else 255), code)
    if signed:
        negative = torch.signbit(x)
        value = torch.where(negative, -value, value)
        code = code + negative.to(torch.int64) * 128
    return torch.cat([code, top]).to(torch.uint8), value


def _decode(state, n, depth, signed):
    code, top = state[:n].to(torch.int64), state[n:].to(torch.int64)
    base = torch.clamp((top - depth) * 8, min=0).repeat_interleave(BLOCK)[:n]
    c = code & 127 if signed else code
    value = torch.where(c > 0, (c + base) << 20, torch.zeros_like(c)).to(torch.int32).view(torch.float32)
    value = torch.where(c == (127 if signed else 255), torch.full_like(value, math.nan), value)
    return torch.where(code >= 128, -value, value) if signed else value


def _adamw_plain(s):
    factor = torch.ones((), device="cuda")
    if s["max"] > 0:
        factor = torch.clamp(torch.full_like(s["norm"], s["max"]) / s["norm"], max=1.0)
    small = s["bits"] == 8
    step_size = LR / (1 - BETA1**STEP)
    root = 1 / math.sqrt(1 - BETA2**STEP)
    for i, (p, g) in enumerate(zip(s["p"], s["g"])):
        n = p.numel()
        to_m, to_v, to_p = _draws(s["seed"], i, n)
        m = _decode(s["m"][i], n, 14, True) if small else s["m"][i]
        v = _decode(s["v"][i], n, 30, False) if small else s["v"][i]
        g = g.float() * factor
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + g * g * (1 - BETA2)
        new = p.float() * (1 - LR * DECAY) - step_size * (m / (torch.sqrt(v) * root + EPS))
        if p.dtype == torch.bfloat16 and to_p is not None:
            b = new.view(torch.int32).to(torch.int64) & 0xFFFFFFFF
            b = (b + to_p) & 0xFFFF0000
            new = torch.where(b >= 1 << 31, b - (1 << 32), b).to(torch.int32).view(torch.float32)
        p.copy_(new)
        if small:
            code, value = _encode(m, to_m, 14, True)
            s["m"][i].copy_(code)
            s["out"][0][i].copy_(value)
            code, value = _encode(v, to_v, 30, False)
            s["v"][i].copy_(code)
            s["out"][1][i].copy_(value)
        else:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
    return (s["p_flat"], s["m_out"], s["v_out"]) if small else (s["p_flat"], s["m_flat"], s["v_flat"])


def _blocks(x, rows):
    """x in blocks of rows x 128, padded with zeros: [row blocks, rows, column blocks, 128]."""
    T, K = x.shape
    Tb, Kb = -(-T // rows), -(-K // BLOCK)
    out = torch.zeros(Tb * rows, Kb * BLOCK, dtype=torch.float32, device="cuda")
    out[:T, :K] = x
    return out.view(Tb, rows, Kb, BLOCK)


def _quantize_plain(x, rows):
    """The values that the codes stand for, over the scale, and the scales: the
    least power of two that brings a block's largest to 448 or less."""
    T, K = x.shape
    b = _blocks(x, rows)
    top = b.abs().amax(dim=(1, 3))
    exponent = ((top.view(torch.int32) + 0x1FFFFF) >> 23) - 127 - 8
    exponent = torch.where(top == 0, torch.zeros_like(exponent), torch.clamp(exponent, min=-126))
    scale = ((exponent + 127) << 23).view(torch.float32)
    q = (b / scale[:, None, :, None]).reshape(b.shape[0] * rows, -1)[:T, :K].to(torch.float8_e4m3fn)
    return q, scale


def _spread_scale(scale, rows, T, K):
    return scale.repeat_interleave(rows, 0)[:T].repeat_interleave(BLOCK, 1)[:, :K]


def _head_plain(s):
    q, scale = _quantize_plain(s["x"], 1)
    x = q.float() * _spread_scale(scale, 1, *q.shape)
    W = s["W"].float() * _spread_scale(s["Ws"], BLOCK, *s["W"].shape)
    return (x @ W.T).to(_type(s["out"]))


def _beams_plain(s):
    B, beams, n, V = s["B"], s["beams"], s["n"], s["V"]
    z = s["z"].double()
    top = z.amax(dim=1, keepdim=True)
    log_total = torch.log(torch.exp(z - top).sum(dim=1, keepdim=True))
    total = s["scores"].double().view(-1, 1) - top - log_total + z
    total, order = torch.sort(total.view(B, beams * V), dim=1, descending=True, stable=True)
    total, order = total[:, :n], order[:, :n]
    none = total == -math.inf
    parent, token = order // V, order % V
    return (total.float(), torch.where(none, torch.full_like(parent, -1), parent),
            torch.where(none, torch.full_like(token, -1), token))


def _reorder_plain(s):
    rows = s["parents"] + torch.arange(s["B"], device="cuda")[:, None] * s["beams"]
    outs = s["states"] if s["place"] else s["out"]
    for x, o in zip(s["states"], outs):
        o.copy_(x.index_select(0, rows.view(-1)))
    return outs


def run(s):
    if own:
        from vocab_wide_token_gb300 import pstat

        if s["op"] == "adamw":
            limit = {"norm": s["norm"], "max_norm": s["max"]} if s["max"] > 0 else {}
            pstat.adamw_step(s["p"], s["g"], s["m"], s["v"], STEP, LR, (BETA1, BETA2), EPS, DECAY, seed=s["seed"], **limit)
            if s["bits"] == 32:
                return s["p_flat"], s["m_flat"], s["v_flat"]
            pstat.adamw_moments(s["m"], s["v"], s["p"], out=s["out"])
            return s["p_flat"], s["m_out"], s["v_out"]
        if s["op"] == "quantize":
            return pstat.fp8_quantize(s["x"], s["rows"])
        if s["op"] == "head":
            q, scale = pstat.fp8_quantize(s["x"], 1)
            return pstat.fp8_logits(q, scale, s["W"], s["Ws"], _type(s["out"]))
        if s["op"] == "beams":
            return pstat.beam_select(s["z"], s["scores"], s["n"])
        return pstat.beam_reorder(s["states"], s["parents"], out=s["states"] if s["place"] else s["out"])
    if s["op"] == "adamw":
        return _adamw_plain(s)
    if s["op"] == "quantize":
        return _quantize_plain(s["x"], s["rows"])
    if s["op"] == "head":
        return _head_plain(s)
    return _beams_plain(s) if s["op"] == "beams" else _reorder_plain(s)


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    def size(name):
        return 2 if name == "bf16" else 4

    if case["op"] == "adamw":
        n = sum(_adamw_sizes(case))
        # parameter in and out, gradient, moments in and out; 8-bit moments also as values
        each = 2 * size(case["p"]) + size(case["g"]) + (16 if case["bits"] == 32 else 4 + 8 + 4 / BLOCK)
        return {"bytes": n * each, "flops": 15 * n}
    if case["op"] == "quantize":
        n = case["T"] * case["K"]
        return {"bytes": n * (size(case["dtype"]) + 1) + 4 * n / (BLOCK * case["rows"]), "flops": 3 * n}
    if case["op"] == "head":
        T, N, K = case["T"], case["N"], case["K"]
        nbytes = T * K * size(case["dtype"]) + N * K + 4 * N * K / BLOCK**2 + T * N * size(case["out"])
        return {"bytes": nbytes, "flops": 2 * T * N * K}
    if case["op"] == "beams":
        T = case["B"] * case["beams"]
        return {"bytes": T * case["V"] * size(case["dtype"]) + 4 * T + 20 * case["B"] * case["n"],
                "flops": 4 * T * case["V"]}
    # Of `beams` rows, drawn as parents at random, this share is some beam's parent; in place
    # a beam that is its own parent is written to nobody.
    k = case["beams"]
    share = 1 - (1 - 1 / k)**k
    cells = case["B"] * k * case["heads"] * case["length"] * case["width"] * case["tensors"]
    if case["place"]:
        moved = 1 - (1 - 1 / k)**(k - 1) + 1 - 1 / k  # read by another beam, written
        return {"bytes": cells * size(case["dtype"]) * moved + 8 * case["B"] * k, "flops": 0}
    return {"bytes": cells * size(case["dtype"]) * (share + 1) + 8 * case["B"] * k, "flops": 0}


# ---- the definition in 64 bits -----------------------------------------------------

def _round(x, t):
    return x.to(t).double()


def _exact_codes(x, draws, depth, signed):
    """The value each element is rounded to, from its neighbours on the grid:
    the upper one where the draw's share of the step is passed."""
    n = x.numel()
    pad = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.float64, device="cuda")
    pad[:n] = x.abs()
    top = torch.frexp(pad.view(-1, BLOCK).amax(dim=1))[1].double() - 1  # 2^top <= largest < 2^(top + 1)
    least = (1.125 * torch.exp2(torch.clamp(top - depth, min=-127.0))).repeat_interleave(BLOCK)[:n]
    a = x.abs()
    step = torch.exp2(torch.frexp(torch.maximum(a, least))[1].double() - 1 - 3)
    low = torch.floor(a / step) * step
    share = draws.double() / 2.0**20
    value = low + torch.where((a - low) / step + share >= 1.0, step, torch.zeros_like(step))
    below = a < least
    if signed:
        value = torch.where(below, torch.where(a > least * share, least, torch.zeros_like(a)), value)
    else:
        value = torch.where(below & (a > 0), least, value)
    return torch.copysign(value, x)


def _exact_adamw(case, seed):
    s = prepare(case, seed)
    f32 = torch.float32
    factor = 1.0
    if s["max"] > 0:
        factor = min(1.0, float(_round(torch.tensor(s["max"] / float(s["norm"]), dtype=torch.float64), f32)))
    p_all = s["p_flat"].double()
    m_all, v_all = torch.zeros_like(p_all), torch.zeros_like(p_all)
    b1, c1, b2, c2 = BETA1, 1 - BETA1, BETA2, 1 - BETA2
    at = 0
    for i, g in enumerate(s["g"]):
        n = g.numel()
        g, p = g.double() * factor, p_all[at:at + n]
        if case["bits"] == 32:
            m, v = s["m"][i].double() * b1 + g * c1, s["v"][i].double() * b2 + g * g * c2
            m_all[at:at + n], v_all[at:at + n] = m, v
        else:
            # Which of two codes a value gets is decided on its 32-bit form, by definition:
            # every product and sum rounded once (64 bits hold them before that).
            to_m, to_v, _ = _draws(s["seed"], i, n)
            one = [float(_round(torch.tensor(x, dtype=torch.float64), f32)) for x in (b1, c1, b2, c2)]
            g = _round(g, f32)
            m = _round(_round(_decode(s["m"][i], n, 14, True).double() * one[0], f32) + _round(g * one[1], f32), f32)
            v = _round(_round(_decode(s["v"][i], n, 30, False).double() * one[2], f32)
                       + _round(_round(g * g, f32) * one[3], f32), f32)
            m_all[at:at + n], v_all[at:at + n] = _exact_codes(m, to_m, 14, True), _exact_codes(v, to_v, 30, False)
        update = (m / (1 - b1**STEP)) / (torch.sqrt(v / (1 - b2**STEP)) + EPS)
        p_all[at:at + n] = p - LR * DECAY * p - LR * update
        at += -(-n // BLOCK) * BLOCK
    return p_all, m_all, v_all


def _exact_quantize(x, rows):
    """Scales from the binary exponents, codes to the nearest of the 8-bit numbers, ties to even."""
    T, K = x.shape
    b = _blocks(x, rows).double()
    top = b.abs().amax(dim=(1, 3))
    exponent = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448.0))
    exponent = torch.where(448.0 * torch.exp2(exponent - 1) >= top, exponent - 1, exponent)
    exponent = torch.where(448.0 * torch.exp2(exponent) < top, exponent + 1, exponent)
    exponent = torch.where(top == 0, torch.zeros_like(exponent), torch.clamp(exponent, min=-126))
    scale = torch.exp2(exponent)
    y = (b / scale[:, None, :, None]).reshape(b.shape[0] * rows, -1)[:T, :K]
    step = torch.exp2(torch.clamp(torch.frexp(y)[1].double() - 1, min=-6) - 3)
    return torch.round(y / step) * step, scale


def exact(case, seed):
    if case["op"] == "adamw":
        return _exact_adamw(case, seed)
    s = prepare(case, seed)
    if case["op"] == "quantize":
        if case["T"] * case["K"] > 700_000_000:
            return None
        return _exact_quantize(s["x"], case["rows"])
    if case["op"] == "head":
        T, N, K = case["T"], case["N"], case["K"]
        if T * N * K > 3e12:
            return None
        q, scale = _exact_quantize(s["x"], 1)
        x = q * _spread_scale(scale, 1, T, K)
        out = torch.empty(T, N, dtype=torch.float64, device="cuda")
        for r in range(0, N, 16384):
            w = s["W"][r:r + 16384].double()
            w *= _spread_scale(s["Ws"][r // BLOCK:(r + 16384) // BLOCK].double(), BLOCK, *w.shape)
            out[:, r:r + 16384] = x @ w.T
        return out
    if case["op"] == "beams":
        B, beams, n, V = case["B"], case["beams"], case["n"], case["V"]
        k = min(n, V)
        rows = []
        for t in range(B * beams):
            z = s["z"][t].double()
            base = float(s["scores"].view(-1)[t]) - float(torch.logsumexp(z, 0))
            cut = torch.topk(z, k).values[-1]
            cols = (z >= cut).nonzero()[:, 0]
            rows.append([(-(base + x), t % beams, c) for x, c in zip(z[cols].tolist(), cols.tolist())
                         if base + x > -math.inf])
        found = []
        for b in range(B):
            best = sorted(x for row in rows[b * beams:(b + 1) * beams] for x in row)[:n]
            found.append(best + [(math.inf, -1, -1)] * (n - len(best)))
        return (torch.tensor([[-x[0] for x in f] for f in found], dtype=torch.float64),
                torch.tensor([[x[1] for x in f] for f in found]), torch.tensor([[x[2] for x in f] for f in found]))
    rows = [b * case["beams"] + p for b, r in enumerate(s["parents"].tolist()) for p in r]
    return [torch.stack([x[r] for r in rows]).double() for x in s["states"]]
