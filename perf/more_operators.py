"""The matrix products next to the gated activations: what is measured, and their plain forms.

Two kinds of case, told apart by ``case["op"]``:

``gated``    a gated MLP's up half in one operator: both projections of the rows, the
             activation of the gate and the product, ``act(x Wg') * (x Wu')``; of one block or
             of a batch of experts with their own row counts; forward, or forward and backward.
``entropy``  the cross entropy of ``x W'`` against a target in a large vocabulary, the logits
             never kept; forward, or forward and backward.

``own`` selects the library's kernels; otherwise ``run`` computes the same in elementary
torch operations in 32 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
K, C = math.sqrt(2.0 / math.pi), 0.044715
DEAD = -100                   # the target of a token that takes no part


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # serving: one token through an expert-sized block; launch latency
        {"name": "gated decode 1 token", "op": "gated", "pass": "forward", "act": "silu",
         "experts": 1, "rows": 1, "k": 2048, "d": 768, "live": 1.0, "dtype": "bf16"},
        # serving: a batch of 16 sequences, one token each, through a wide dense block
        {"name": "gated decode 16 tokens wide", "op": "gated", "pass": "forward", "act": "gelu",
         "experts": 1, "rows": 16, "k": 4096, "d": 16384, "live": 1.0, "dtype": "bf16"},
        # serving: 256 choices of a decode batch spread over 128 experts, most with a row or two
        {"name": "gated decode experts", "op": "gated", "pass": "forward", "act": "silu",
         "experts": 128, "rows": 32, "k": 2048, "d": 768, "live": 0.0625, "dtype": "bf16"},
        # serving: a prompt
        {"name": "gated prefill", "op": "gated", "pass": "forward", "act": "gelu",
         "experts": 1, "rows": 2048, "k": 4096, "d": 16384, "live": 1.0, "dtype": "bf16"},
        # odd sizes throughout: no row but the first starts on a 16-byte boundary
        {"name": "gated step odd", "op": "gated", "pass": "step", "act": "silu",
         "experts": 1, "rows": 1001, "k": 1101, "d": 2731, "live": 1.0, "dtype": "fp16"},
        # training a dense block
        {"name": "gated step dense", "op": "gated", "pass": "step", "act": "silu",
         "experts": 1, "rows": 4096, "k": 4096, "d": 8192, "live": 1.0, "dtype": "bf16"},
        # training a mixture of experts: buffers of fixed capacity, 70% filled
        {"name": "gated step experts", "op": "gated", "pass": "step", "act": "silu",
         "experts": 32, "rows": 1024, "k": 2048, "d": 768, "live": 0.7, "dtype": "bf16"},
        # scoring a short answer
        {"name": "entropy forward 64 tokens", "op": "entropy", "pass": "forward", "tokens": 64,
         "k": 1024, "vocab": 32000, "live": 1.0, "dtype": "bf16"},
        # scoring long texts
        {"name": "entropy forward batch", "op": "entropy", "pass": "forward", "tokens": 8192,
         "k": 2048, "vocab": 65536, "live": 1.0, "dtype": "bf16"},
        # training on answers alone: the prompts' tokens, 60% of the batch, take no part
        {"name": "entropy step answers", "op": "entropy", "pass": "step", "tokens": 4096,
         "k": 1024, "vocab": 65536, "live": 0.4, "dtype": "bf16"},
        # odd sizes throughout
        {"name": "entropy step odd", "op": "entropy", "pass": "step", "tokens": 777,
         "k": 1001, "vocab": 50001, "live": 0.9, "dtype": "fp16"},
        # training with a large vocabulary
        {"name": "entropy step batch", "op": "entropy", "pass": "step", "tokens": 4096,
         "k": 2048, "vocab": 131072, "live": 1.0, "dtype": "bf16"},
    ]


MOST = 6 * 4096 * 2048 * 131072       # operations of the largest listed case


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width of a model: odd or even as it comes, or a multiple of 64."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.4 else max(lo, n // 64 * 64)


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    step = rng.choice(["forward", "step"])
    if rng.random() < 0.5:
        k, vocab = _width(rng, 64, 4096), _width(rng, 1000, 131072)
        most = min(8192, MOST // (6 * k * vocab), (1 << 30) // vocab)
        return {"op": "entropy", "pass": step, "tokens": _log(rng, 1, most), "k": k,
                "vocab": vocab, "live": rng.choice([1.0, 1.0, 0.9, 0.4]), "dtype": dtype}
    experts = rng.choice([1, 1, 1, 4, 16, 64])
    k = _width(rng, 64, 8192 if experts == 1 else 2048)
    d = _width(rng, 64, 16384 if experts == 1 else 2048)
    most = min(8192, MOST // (12 * experts * k * d), (1 << 27) // (experts * max(k, d)))
    return {"op": "gated", "pass": step, "act": rng.choice(["silu", "gelu"]), "experts": experts,
            "rows": _log(rng, 1, max(1, most)), "k": k, "d": d,
            "live": 1.0 if experts == 1 else rng.choice([1.0, 0.7, 0.3]), "dtype": dtype}


# --------------------------------------------------------------------- inputs

def _counts(case, seed):
    """Live rows of each expert: about ``live`` of the capacity, unevenly."""
    if case["live"] >= 1:
        return [case["rows"]] * case["experts"]
    rng = random.Random(seed)
    mean = case["rows"] * case["live"]
    return [min(case["rows"], int(mean * 2 * rng.random() + 0.5)) for _ in range(case["experts"])]


def _dead(case):
    """How many tokens take no part."""
    return case["tokens"] - max(1, int(case["tokens"] * case["live"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    dtype, k = DTYPES[case["dtype"]], case["k"]
    s = {"case": case}
    if case["op"] == "entropy":
        t, v = case["tokens"], case["vocab"]
        weight = (2 * k ** -0.5 * normal(v, k)).to(dtype)
        targets = torch.randint(v, (t,), generator=gen, device="cuda")
        # a hidden state leans towards its target's row, some strongly and some not at all
        x = normal(t, k)
        for a in range(0, t, 1024):
            x[a:a + 1024] += 3 * uniform(min(1024, t - a), 1) * weight[targets[a:a + 1024]].float()
        s["x"], s["weight"] = x.to(dtype), weight
        n = _dead(case)
        if n:
            targets[torch.randperm(t, generator=gen, device="cuda")[:n]] = DEAD
        s["targets"] = targets
        # the mean over the live tokens, each with a weight; fp16 under a loss scale
        s["grad_loss"] = (0.5 + uniform(t)) * ((4096 if case["dtype"] == "fp16" else 1) / (t - n))
        return s

    e, m, d = case["experts"], case["rows"], case["d"]
    # normed rows with a few strong channels; projections of about unit size
    x = normal(e, m, k) * (1 + 3 * (uniform(1, 1, k) < 0.01))
    s["x"] = x.to(dtype)
    s["weight"] = torch.empty(e, 2 * d, k, dtype=dtype, device="cuda")
    for i in range(e):
        s["weight"][i] = (1.2 * k ** -0.5 * normal(2 * d, k)).to(dtype)
    s["grad"] = normal(e, m, d).to(dtype) if case["pass"] == "step" else None
    s["n_rows"] = None
    if case["live"] < 1:
        s["n_rows"] = torch.tensor(_counts(case, seed), dtype=torch.int32, device="cuda")
        # the buffers of fixed capacity that a block keeps: rows past the live ones stay 0
        s["out"] = torch.zeros(e, m, d, dtype=dtype, device="cuda")
        if case["pass"] == "step":
            s["grad_x"] = torch.zeros(e, m, k, dtype=dtype, device="cuda")
    elif e == 1:
        for name in ("x", "weight", "grad"):
            s[name] = s[name][0] if s[name] is not None else None
    return s


# ---------------------------------------------------------------- plain forms

def _silu(g):
    sig = 1 / (1 + torch.exp(-g))
    return g * sig, sig * (1 + g * (1 - sig))


def _gelu(g):
    t = torch.tanh(K * (g + C * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * (K + 3 * K * C * g * g)


def _plain_gated(s, case):
    act = _silu if case["act"] == "silu" else _gelu
    dtype, d = s["x"].dtype, case["d"]
    x, w = s["x"].float(), s["weight"].float()
    if s["n_rows"] is not None:
        live = torch.arange(case["rows"], device=x.device)[None, :, None] < s["n_rows"][:, None, None]
        x = torch.where(live, x, torch.zeros_like(x))
    h = x @ w.mT
    g, u = h[..., :d], h[..., d:]
    a, slope = act(g)
    got = {"out": (a * u).to(dtype)}
    if case["pass"] == "step":
        grad = s["grad"].float()
        if s["n_rows"] is not None:
            grad = torch.where(live, grad, torch.zeros_like(grad))
        grad_h = torch.cat([grad * u * slope, grad * a], -1)
        got["grad_x"] = (grad_h @ w).to(dtype)
        got["grad_weight"] = (grad_h.mT @ x).to(dtype)
    return got


def _plain_entropy(s, case):
    dtype, targets = s["x"].dtype, s["targets"]
    live = targets >= 0
    at = targets.clamp(min=0)[:, None]
    x, w = s["x"].float(), s["weight"].float()
    logits = x @ w.T
    top = logits.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))
    nothing = torch.zeros_like(lse[:, 0])
    got = {"loss": torch.where(live, (lse - logits.gather(1, at))[:, 0], nothing),
           "lse": torch.where(live, lse[:, 0], nothing)}
    if case["pass"] == "step":
        p = torch.exp(logits - lse)
        p.scatter_add_(1, at, -torch.ones_like(lse))
        p *= torch.where(live, s["grad_loss"], nothing)[:, None]
        got["grad_x"] = (p @ w).to(dtype)
        got["grad_weight"] = (p.T @ x).to(dtype)
    return got


# ------------------------------------------------------------------------ run

def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return (_plain_gated if case["op"] == "gated" else _plain_entropy)(state, case)


def _run_own(s, case):
    import gated_activation_gb300 as ga
    step = case["pass"] == "step"
    if case["op"] == "entropy":
        kept = ga.linear_cross_entropy(s["x"], s["weight"], s["targets"])
        got = {"loss": kept.loss, "lse": kept.lse}
        if step:
            got["grad_x"], got["grad_weight"] = ga.linear_cross_entropy_backward(
                s["grad_loss"], s["x"], s["weight"], s["targets"], kept)
        return got
    forward, backward = ((ga.linear_silu_and_mul, ga.linear_silu_and_mul_backward)
                         if case["act"] == "silu" else
                         (ga.linear_gelu_and_mul, ga.linear_gelu_and_mul_backward))
    if not step:
        return {"out": forward(s["x"], s["weight"], n_rows=s["n_rows"], out=s.get("out"))}
    out, kept = forward(s["x"], s["weight"], n_rows=s["n_rows"], keep=True, out=s.get("out"))
    grad_x, grad_weight = backward(s["grad"], s["x"], s["weight"], kept, n_rows=s["n_rows"],
                                   grad_in=s.get("grad_x"))
    return {"out": out, "grad_x": grad_x, "grad_weight": grad_weight}


# ----------------------------------------------------------------------- work

def work(case):
    """Bytes of inputs and outputs, each once, and two operations for each product; a step
    has three products of the forward pass's size.  Elementwise operations are left out."""
    k = case["k"]
    if case["op"] == "entropy":
        t, v = case["tokens"] - _dead(case), case["vocab"]
        once = 2 * (t * k + v * k) + 8 * case["tokens"] + 8 * case["tokens"]
        if case["pass"] == "forward":
            return {"bytes": once, "flops": 2 * t * v * k}
        return {"bytes": once + 2 * (t * k + v * k) + 4 * case["tokens"], "flops": 6 * t * v * k}
    counts, d = _counts(case, 0), case["d"]
    rows, used = sum(counts), sum(n > 0 for n in counts)
    once = 2 * (rows * (k + d) + used * 2 * d * k)
    if case["pass"] == "forward":
        return {"bytes": once, "flops": 4 * rows * k * d}
    # an expert without rows has a weight gradient of zeros to write
    return {"bytes": once + 2 * (rows * (k + d) + case["experts"] * 2 * d * k),
            "flops": 12 * rows * k * d}


# ---------------------------------------------------------------------- exact

def _exact_gated(s, case, seed):
    d, k, m = case["d"], case["k"], case["rows"]
    step = case["pass"] == "step"
    x, w = s["x"].view(-1, m, k), s["weight"].view(-1, 2 * d, k)
    grad = s["grad"].view(-1, m, d) if step else None
    new = dict(dtype=torch.float64, device=x.device)
    out, gx = torch.zeros(len(x), m, d, **new), torch.zeros(len(x), m, k, **new)
    gw = torch.zeros(len(x), 2 * d, k, **new)
    for e, n in enumerate(_counts(case, seed)):
        xe, wg, wu = x[e, :n].double(), w[e, :d].double(), w[e, d:].double()
        g, u = xe @ wg.T, xe @ wu.T
        # both activations are g sigmoid(y)
        if case["act"] == "silu":
            y, dy = g, torch.ones_like(g)
        else:
            y, dy = 2 * K * (g + C * g ** 3), 2 * K * (1 + 3 * C * g ** 2)
        sig = torch.sigmoid(y)
        out[e, :n] = g * sig * u
        if step:
            up = grad[e, :n].double()
            dg, du = up * u * (sig + g * sig * (1 - sig) * dy), up * g * sig
            gx[e, :n] = dg @ wg + du @ wu
            gw[e, :d], gw[e, d:] = dg.T @ xe, du.T @ xe
    got = {"out": out, "grad_x": gx, "grad_weight": gw} if step else {"out": out}
    return got if s["x"].dim() == 3 else {name: v[0] for name, v in got.items()}


def _exact_entropy(s, case):
    t, targets = case["tokens"], s["targets"]
    rows = (targets >= 0).nonzero()[:, 0]
    new = dict(dtype=torch.float64, device=targets.device)
    w = s["weight"].double()
    got = {"loss": torch.zeros(t, **new), "lse": torch.zeros(t, **new)}
    step = case["pass"] == "step"
    if step:
        got["grad_x"], got["grad_weight"] = torch.zeros(t, case["k"], **new), torch.zeros_like(w)
    for part in rows.split(1024):
        x, goal = s["x"][part].double(), targets[part]
        logits = x @ w.T
        lse = torch.logsumexp(logits, 1)
        got["lse"][part] = lse
        got["loss"][part] = lse - logits[torch.arange(len(part), device=goal.device), goal]
        if step:
            p = torch.softmax(logits, 1)
            p[torch.arange(len(part), device=goal.device), goal] -= 1
            p *= s["grad_loss"][part].double()[:, None]
            got["grad_x"][part] = p @ w
            got["grad_weight"] += p.T @ x
    return got


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return _exact_gated(s, case, seed) if case["op"] == "gated" else _exact_entropy(s, case)
