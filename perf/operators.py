"""Measured cases of the sampling, truncated-policy and gradient-clipping operators.

A case is one call that a user's program makes of them: drawing the next token
of every sequence of a decode batch, scoring and differentiating the drawn
tokens under the distribution they were drawn from, or taking the global norm
of a list of gradients and clipping by it.  ``own`` selects the framework's
kernels; otherwise the same results come from elementary torch operations.
"""
import math

import torch

own = False

V_WIDE = 151936  # the framework's vocabulary (inputs.V_QWEN3)
IGNORE = -100


def listed():
    return [
        # One chat stream: the latency of a single token's draw.
        {"name": "sample_one", "op": "sample", "T": 1, "V": V_WIDE, "dtype": "bf16", "pad": 0,
         "t": 0.8, "k": 50, "p": 0.95, "m": 0.0, "per_row": False, "flat": 0.0, "mask": 0.0},
        # A served batch in which every request has its own settings (some greedy, some unfiltered).
        {"name": "sample_requests", "op": "sample", "T": 64, "V": V_WIDE, "dtype": "bf16", "pad": 0,
         "t": 1.0, "k": 0, "p": 1.0, "m": 0.0, "per_row": True, "flat": 0.0, "mask": 0.0},
        # fp32 logits with nucleus sampling; every 32nd row is one the model is unsure of.
        {"name": "sample_nucleus_f32", "op": "sample", "T": 256, "V": V_WIDE, "dtype": "f32", "pad": 0,
         "t": 0.7, "k": 0, "p": 0.9, "m": 0.0, "per_row": False, "flat": 0.03, "mask": 0.0},
        # A small vocabulary of odd size in padded rows, part of it masked (a grammar), min-p.
        {"name": "sample_grammar", "op": "sample", "T": 333, "V": 10007, "dtype": "bf16", "pad": 9,
         "t": 1.2, "k": 0, "p": 1.0, "m": 0.05, "per_row": False, "flat": 0.0, "mask": 0.5},
        # An RL rollout step over many sequences: the policy itself, no truncation.
        {"name": "sample_rollout", "op": "sample", "T": 2048, "V": V_WIDE, "dtype": "bf16", "pad": 0,
         "t": 1.0, "k": 0, "p": 1.0, "m": 0.0, "per_row": False, "flat": 0.0, "mask": 0.0},
        # The framework's smallest training workload (64 rows of 1000 fp32 logits), top-k.
        {"name": "train_tiny", "op": "train", "T": 64, "V": 1000, "dtype": "f32", "pad": 0,
         "t": 0.9, "k": 40, "p": 1.0, "m": 0.0, "per_row": False, "flat": 1.0, "mask": 0.0},
        # Scoring and gradient of rollouts that were drawn with temperature and top-p.
        {"name": "train_nucleus", "op": "train", "T": 2048, "V": V_WIDE, "dtype": "bf16", "pad": 0,
         "t": 0.8, "k": 0, "p": 0.95, "m": 0.0, "per_row": False, "flat": 0.0, "mask": 0.0},
        # fp32 logits, temperature alone.
        {"name": "train_tempered_f32", "op": "train", "T": 512, "V": V_WIDE, "dtype": "f32", "pad": 0,
         "t": 1.3, "k": 0, "p": 1.0, "m": 0.0, "per_row": False, "flat": 0.5, "mask": 0.0},
        # The norm of many small tensors (biases, norms): launch latency.
        {"name": "norm_small", "op": "norm", "n": 16, "lo": 1, "hi": 5000, "dtype": "mixed", "max": 0.0},
        # The norm of a model's gradients, 300 ragged tensors of both types.
        {"name": "norm_model", "op": "norm", "n": 300, "lo": 100, "hi": 4000000, "dtype": "mixed", "max": 0.0},
        # Clipping ragged bf16 gradients into the optimiser's buffers.
        {"name": "clip_model", "op": "clip", "n": 48, "lo": 1000, "hi": 8000000, "dtype": "bf16", "max": 1.0},
        # The lm_head's own gradients: dW [151936, 4096] and dhidden [16384, 4096], fp32.
        {"name": "clip_lmhead", "op": "clip", "n": 0, "lo": 0, "hi": 0, "dtype": "f32", "max": 1.0},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["sample", "sample", "sample", "train", "train", "norm", "clip"])
    if kind in ("norm", "clip"):
        lo = spread(1, 10000)
        return {"op": kind, "n": spread(1, 300) if kind == "norm" else spread(1, 48), "lo": lo,
                "hi": lo + spread(1, 6000000), "dtype": rng.choice(["bf16", "f32", "mixed"]),
                "max": 0.0 if kind == "norm" else rng.choice([0.5, 1.0, 1e6])}
    dtype = rng.choice(["bf16", "f32"])
    V = rng.choice([V_WIDE, spread(2000, V_WIDE), spread(2000, V_WIDE) | 1])
    T = spread(1, 2048 if dtype == "bf16" else 512)
    return {"op": kind, "T": T, "V": V, "dtype": dtype, "pad": rng.choice([0, 0, 8, rng.randint(1, 64)]),
            "t": rng.choice([1.0, round(rng.uniform(0.3, 1.5), 3)]),
            "k": rng.choice([0, 0, spread(1, 200), spread(1, 5000)]),
            "p": rng.choice([1.0, 1.0, 0.9, round(rng.uniform(0.2, 0.99), 3)]),
            "m": rng.choice([0.0, 0.0, round(rng.uniform(0.01, 0.3), 3)]),
            "per_row": rng.random() < 0.25, "flat": rng.choice([0.0, 0.0, 0.1]),
            "mask": rng.choice([0.0, 0.0, 0.3])}


# ---- inputs -----------------------------------------------------------------

def _logits(case, g):
    """Language-model-like rows: a bulk N(0, 2^2) over the vocabulary and, but
    for the share `flat` of rows, 48 columns raised by up to 14 to 24 (entropies
    from about 0 to 3 nats, a tail of 0.01 to 10 per cent); `mask` of the
    columns at -inf."""
    T, V = case["T"], case["V"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    store = torch.zeros(T, V + case["pad"], dtype=dt, device="cuda")
    out = store[:, :V]
    n_flat = int(round(case["flat"] * T))
    n_up = min(48, V)
    for r0 in range(0, T, 256):
        n = min(256, T - r0)
        z = torch.randn(n, V, generator=g, device="cuda").mul_(2.0)
        height = 14.0 + 10.0 * torch.rand(n, 1, generator=g, device="cuda")
        cols = torch.randint(0, V, (n, n_up), generator=g, device="cuda")
        rise = height * torch.rand(n, n_up, generator=g, device="cuda")
        rise[:max(0, min(n, n_flat - r0))] = 0.0
        z.scatter_add_(1, cols, rise)
        if case["mask"] > 0:
            off = torch.rand(n, V, generator=g, device="cuda") < case["mask"]
            off[:, :2] = False
            z[off] = -math.inf
        out[r0:r0 + n] = z.to(dt)
    return out


def _settings(case, g):
    """The four filters: plain numbers, or one value for each row."""
    T = case["T"]
    if not case["per_row"]:
        return case["t"], case["k"], case["p"], case["m"]

    def pick(values, dt):
        i = torch.randint(0, len(values), (T,), generator=g, device="cuda")
        return torch.tensor(values, device="cuda", dtype=dt)[i]

    cold = 0.0 if case["op"] == "sample" else 0.25
    return (pick([cold, 0.5, 0.7, 0.9, 1.0, 1.0, 1.2], torch.float32),
            pick([0, 0, 0, 1, 20, 50, 200], torch.int32),
            pick([1.0, 1.0, 0.8, 0.9, 0.95], torch.float32),
            pick([0.0, 0.0, 0.0, 0.05, 0.1], torch.float32))


def _grad_sizes(case, seed):
    if case["n"] == 0:
        return [(V_WIDE, 4096), (16384, 4096)]
    rng = torch.Generator().manual_seed(7)  # the shapes are the model's, not the seed's
    u = torch.rand(case["n"], generator=rng, dtype=torch.float64)
    lo, hi = math.log(case["lo"]), math.log(case["hi"])
    return [(int(round(math.exp(lo + float(x) * (hi - lo)))),) for x in u]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("norm", "clip"):
        grads = []
        for i, shape in enumerate(_grad_sizes(case, seed)):
            x = torch.randn(*shape, generator=g, device="cuda").mul_(10.0 ** (-(i % 4)))
            bf16 = case["dtype"] == "bf16" or (case["dtype"] == "mixed" and i % 2 == 0)
            grads.append(x.to(torch.bfloat16) if bf16 else x)
        state = {"op": case["op"], "grads": grads, "max": case["max"]}
        if case["op"] == "clip":
            state["out"] = [torch.empty_like(x) for x in grads]
        return state
    T, V = case["T"], case["V"]
    z = _logits(case, g)
    t, k, p, m = _settings(case, g)
    state = {"op": case["op"], "z": z, "t": t, "k": k, "p": p, "m": m}
    if case["op"] == "sample":
        state["u"] = torch.rand(T, generator=g, device="cuda")
        return state
    # Labels as a rollout draws them (from the tempered rows, so that a few lie
    # outside the truncation), some ignored; advantages with a loss mask.
    y = torch.empty(T, dtype=torch.int64, device="cuda")
    tt = t[:, None] if isinstance(t, torch.Tensor) else t
    for r0 in range(0, T, 256):
        zz = z[r0:r0 + 256].float() / (tt[r0:r0 + 256] if isinstance(tt, torch.Tensor) else tt)
        noise = torch.rand(zz.shape, generator=g, device="cuda").clamp_(1e-30)
        y[r0:r0 + 256] = torch.argmax(zz - torch.log(-torch.log(noise)), dim=1)
    y[torch.rand(T, generator=g, device="cuda") < 0.05] = IGNORE
    w = torch.randn(T, generator=g, device="cuda")
    state["y"] = y
    state["w"] = w * (torch.rand(T, generator=g, device="cuda") >= 0.2).float()
    return state


# ---- the plain form -----------------------------------------------------------

def _column(x, T, dtype):
    if isinstance(x, torch.Tensor):
        return x.to(dtype)[:, None]
    # a number means what its 32-bit value means, as a tensor of such numbers would
    return torch.full((T, 1), x, device="cuda").to(torch.float32 if dtype.is_floating_point else dtype).to(dtype)


def _truncate(z, t, k, p, m):
    """x = (z - M)/t in 64 bits, the kept columns, the cut and the greedy rows."""
    T, V = z.shape
    t, p, m = (_column(a, T, torch.float64) for a in (t, p, m))
    k = _column(k, T, torch.int64)
    greedy = t == 0
    t = torch.where(greedy, torch.ones_like(t), t)
    k = torch.where(greedy, torch.ones_like(k), torch.where(k <= 0, torch.full_like(k, V), k))
    z = z + 0.0  # -0 and +0 are one value
    values, order = torch.sort(z, dim=1, descending=True, stable=True)
    top = values[:, :1].double()
    xs = (values.double() - top) / t
    rank = torch.arange(V, device=z.device)[None, :]
    keep = (rank < k) & (values > -math.inf)
    mass = torch.cumsum(torch.where(keep, torch.exp(xs), torch.zeros_like(xs)), dim=1)
    before = torch.cat([torch.zeros_like(mass[:, :1]), mass[:, :-1]], dim=1)
    keep = keep & ((before < p * mass[:, -1:]) | (p >= 1))
    keep = keep & ((xs >= torch.log(m)) | (m <= 0))
    last = keep.sum(dim=1, keepdim=True) - 1
    tau = values.gather(1, last)[:, 0].float()
    index = order.gather(1, last)[:, 0]
    free = ((k >= V) & (p >= 1) & (m <= 0))[:, 0]
    tau = torch.where(free, torch.full_like(tau, -math.inf), tau)
    index = torch.where(free, torch.full_like(index, V - 1), index)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    return (z.double() - top) / t, kept, top[:, 0], tau, index, t


def _sample_plain(s):
    x, kept, _, _, _, _ = _truncate(s["z"], s["t"], s["k"], s["p"], s["m"])
    total = torch.cumsum(torch.where(kept, torch.exp(x), torch.zeros_like(x)), dim=1)
    token = (total <= s["u"].double()[:, None] * total[:, -1:]).sum(dim=1)
    logprob = x.gather(1, token[:, None])[:, 0] - torch.log(total[:, -1])
    return token, logprob.float()


def _train_plain(s):
    x, kept, top, tau, index, t = _truncate(s["z"], s["t"], s["k"], s["p"], s["m"])
    y, w = s["y"], s["w"]
    e = torch.where(kept, torch.exp(x), torch.zeros_like(x))
    total = e.sum(dim=1)
    log_total = torch.log(total)
    entropy = log_total - torch.where(kept, e * x, torch.zeros_like(x)).sum(dim=1) / total
    ignored = y == IGNORE
    col = torch.where(ignored, torch.zeros_like(y), y)[:, None]
    hit = kept.gather(1, col)[:, 0]
    logprob = torch.where(hit, x.gather(1, col)[:, 0] - log_total, torch.full_like(log_total, -math.inf))
    logprob = torch.where(ignored, torch.zeros_like(logprob), logprob)
    scale = torch.where(ignored | ~hit, torch.zeros_like(w), w).double()[:, None] / t
    grad = -(e / total[:, None])
    grad.scatter_add_(1, col, torch.ones_like(grad[:, :1]))
    grad = torch.where(scale == 0, torch.zeros_like(grad), grad * scale).to(s["z"].dtype)
    rowstats = torch.stack([top, log_total], dim=1).float()
    return logprob.float(), entropy.float(), rowstats, tau, index, grad


def _norm_plain(grads):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for x in grads:
        total = total + (x.double() * x.double()).sum()
    return torch.sqrt(total)


def _clip_plain(s):
    norm = _norm_plain(s["grads"])
    factor = torch.clamp(s["max"] / norm, max=1.0).float()
    for x, o in zip(s["grads"], s["out"]):
        o.copy_(x.float() * factor)
    return [norm.float()] + s["out"]


def run(state):
    if own:
        from vocab_wide_token_gb300 import pstat

        if state["op"] == "sample":
            return pstat.sample(state["z"], state["u"], state["t"], state["k"], state["p"], state["m"])
        if state["op"] == "train":
            lp, ent, rs, tau, index = pstat.filtered_forward(
                state["z"], state["y"], state["t"], state["k"], state["p"], state["m"], IGNORE)
            grad = pstat.filtered_backward(
                state["z"], state["y"], state["w"], rs, tau, index, state["t"], IGNORE)
            return lp, ent, rs, tau, index, grad
        if state["op"] == "norm":
            return pstat.grad_norm(state["grads"])
        norm, out = pstat.clip_grad_norm(state["grads"], state["max"], out=state["out"])
        return [norm] + out
    if state["op"] == "sample":
        return _sample_plain(state)
    if state["op"] == "train":
        return _train_plain(state)
    if state["op"] == "norm":
        return _norm_plain(state["grads"]).float()
    return _clip_plain(state)


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    if case["op"] in ("norm", "clip"):
        nbytes = n = 0
        for i, shape in enumerate(_grad_sizes(case, 0)):
            size = math.prod(shape)
            bf16 = case["dtype"] == "bf16" or (case["dtype"] == "mixed" and i % 2 == 0)
            nbytes += size * (2 if bf16 else 4)
            n += size
        clip = case["op"] == "clip"
        return {"bytes": nbytes * (2 if clip else 1) + 4, "flops": n * (3 if clip else 2)}
    T, V, es = case["T"], case["V"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        return {"bytes": T * V * es + T * 16, "flops": 4 * T * V}
    return {"bytes": 2 * T * V * es + T * 48, "flops": 9 * T * V}


# ---- the definition in 64 bits, by groups of equal logits -----------------------------

def _one_row(z, t, k, p, m):
    """(x, kept, cut value, cut index) of one row: equal logits form a group,
    groups are taken from the top, and the last group is split by index."""
    V = z.numel()
    z = z.double()
    finite = z > -math.inf
    top = z.max()
    if t == 0:
        index = int((z == top).nonzero()[0])
        kept = torch.zeros(V, dtype=torch.bool, device=z.device)
        kept[index] = True
        return z - top, kept, float(top), index
    x = (z - top) / t
    values, counts = torch.unique(z[finite], return_counts=True)
    values, counts = values.flip(0), counts.flip(0)
    weight = torch.exp((values - top) / t)
    want = int(finite.sum())
    if k > 0:
        want = min(want, k)
    cum = torch.cumsum(counts, 0)
    if p < 1:
        in_top = torch.clamp(want - (cum - counts), min=0).minimum(counts).double()
        mass = torch.cumsum(in_top * weight, 0)
        target = p * mass[-1]
        gi = int((mass < target).sum())
        prior = float(mass[gi - 1]) if gi else 0.0
        need = max(1, math.ceil((float(target) - prior) / float(weight[gi])))
        want = min(want, int(cum[gi] - counts[gi]) + need)
    if m > 0:
        want = min(want, int((x >= math.log(m)).sum()))
    gi = int((cum < want).sum())
    value = values[gi]
    ties = (z == value).nonzero()[:, 0]
    index = int(ties[want - int(cum[gi] - counts[gi]) - 1])
    kept = (z > value) | ((z == value) & (torch.arange(V, device=z.device) <= index))
    if not (0 < k < V) and p >= 1 and m <= 0:
        return x, finite, -math.inf, V - 1
    return x, kept, float(value), index


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        squares = [float(torch.linalg.vector_norm(x.reshape(-1), dtype=torch.float64)) for x in s["grads"]]
        norm = math.sqrt(math.fsum(v * v for v in squares))
        if case["op"] == "norm":
            return torch.tensor(norm, dtype=torch.float64)
        factor = min(1.0, s["max"] / norm)
        if sum(x.numel() for x in s["grads"]) > 200_000_000:
            return [torch.tensor(norm, dtype=torch.float64)] + [None] * len(s["grads"])
        return [torch.tensor(norm, dtype=torch.float64)] + [x.double() * factor for x in s["grads"]]
    T, V = case["T"], case["V"]
    if T * V > 80_000_000:
        return None

    def at(x, i):
        return float(x[i]) if isinstance(x, torch.Tensor) else float(torch.tensor(x, dtype=torch.float32))

    rows = []
    for i in range(T):
        t = at(s["t"], i)
        k = int(s["k"][i]) if isinstance(s["k"], torch.Tensor) else s["k"]
        x, kept, tau, index = _one_row(s["z"][i], t, k, at(s["p"], i), at(s["m"], i))
        cols = kept.nonzero()[:, 0]
        e = torch.exp(x[cols])
        run_sum = torch.cumsum(e, 0)
        total = run_sum[-1]
        if case["op"] == "sample":
            j = int(torch.searchsorted(run_sum, s["u"][i].double() * total, right=True))
            rows.append((int(cols[j]), float(x[cols[j]] - torch.log(total))))
            continue
        y, w = int(s["y"][i]), float(s["w"][i])
        log_total = float(torch.log(total))
        entropy = log_total - float((e * x[cols]).sum() / total)
        grad = torch.zeros(V, dtype=torch.float64, device="cuda")
        if y == IGNORE:
            logprob = 0.0
        elif not bool(kept[y]):
            logprob = -math.inf
        else:
            logprob = float(x[y]) - log_total
            if w != 0:
                grad[cols] = -(w / t) * e / total
                grad[y] += w / t
        rows.append((logprob, entropy, float(s["z"][i].max()), log_total, tau, index, grad))
    if case["op"] == "sample":
        return (torch.tensor([r[0] for r in rows]), torch.tensor([r[1] for r in rows], dtype=torch.float64))
    f = [torch.tensor([r[j] for r in rows], dtype=torch.float64) for j in range(5)]
    return (f[0], f[1], torch.stack([f[2], f[3]], dim=1), f[4], torch.tensor([r[5] for r in rows]),
            torch.stack([r[6] for r in rows]))
