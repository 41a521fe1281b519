"""The operators that train a gated MLP block: what is measured, and their plain forms.

Four kinds of case, told apart by ``case["op"]``:

``step``     the 8-bit checkpoint of silu_and_mul or gelu_and_mul: one forward pass that
             keeps the input in 8 bits, and the backward pass that reads it back.
``sparse``   the same of gelu_and_mul_sparse, the forward pass (with the values that its
             checkpoint stands for) or the backward pass alone.
``norm``     layer norm: the forward pass alone, or forward and backward.
``balance``  the balance loss of a router, its per-expert counts and its gradient.

``own`` selects the library's kernels; otherwise ``run`` computes the same in elementary
torch operations in 32 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
Z95 = 1.6448536269514722      # inverse normal CDF of a target sparsity of 0.95
BLOCK = 32                    # elements that share one scale of a checkpoint
K, C = math.sqrt(2.0 / math.pi), 0.044715
COEF, EPS = 1e-2, 1e-5


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # an expert's few rows at the end of a micro-batch: launch latency
        {"name": "silu step 64 rows", "op": "step", "act": "silu", "rows": 64, "d": 768,
         "dtype": "bf16", "live": 1.0},
        # a full MoE layer's rows (expert width 768) in a buffer that is 80% filled
        {"name": "silu step moe rows", "op": "step", "act": "silu", "rows": 16384, "d": 768,
         "dtype": "bf16", "live": 0.8},
        # a dense GeGLU block with an odd width: no row but the first starts aligned
        {"name": "gelu step odd width", "op": "step", "act": "gelu", "rows": 1000, "d": 4099,
         "dtype": "fp16", "live": 1.0},
        # the sparse-GELU block at its prefill shape, forward
        {"name": "sparse forward prefill", "op": "sparse", "pass": "forward", "rows": 2048,
         "d": 16384, "dtype": "bf16", "z": Z95},
        # and its backward pass
        {"name": "sparse backward prefill", "op": "sparse", "pass": "backward", "rows": 2048,
         "d": 16384, "dtype": "bf16", "z": Z95},
        # a short sequence's backward pass in full precision
        {"name": "sparse backward 8 rows", "op": "sparse", "pass": "backward", "rows": 8,
         "d": 8192, "dtype": "fp32", "z": Z95},
        # the norm in front of the block for a few tokens: launch latency
        {"name": "norm forward 16 rows", "op": "norm", "pass": "forward", "rows": 16, "d": 2048,
         "dtype": "bf16", "params": "bf16", "bias": True},
        # a training batch at a model width of 2048, parameters kept in 32 bits
        {"name": "norm step batch", "op": "norm", "pass": "step", "rows": 16384, "d": 2048,
         "dtype": "bf16", "params": "fp32", "bias": True},
        # wide rows
        {"name": "norm step wide", "op": "norm", "pass": "step", "rows": 2048, "d": 16384,
         "dtype": "bf16", "params": "bf16", "bias": True},
        # full precision, an odd width, no bias
        {"name": "norm step odd width", "op": "norm", "pass": "step", "rows": 1001, "d": 4097,
         "dtype": "fp32", "params": "fp32", "bias": False},
        # a router with few tokens
        {"name": "balance 64 tokens", "op": "balance", "tokens": 64, "experts": 128, "k": 8,
         "dtype": "fp32", "live": 1.0},
        # a router over a long packed batch, a tenth of it padding
        {"name": "balance batch", "op": "balance", "tokens": 65536, "experts": 128, "k": 8,
         "dtype": "bf16", "live": 0.9},
    ]


def _log(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n == 3 * 1024 else n


def draw(rng):
    op = rng.choice(["step", "sparse", "norm", "balance"])
    if op == "balance":
        experts = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
        return {"op": op, "tokens": _log(rng, 1, (1 << 23) // experts), "experts": experts,
                "k": rng.choice([1, 2, 4, 6, 8]), "dtype": rng.choice(list(DTYPES)),
                "live": rng.choice([1.0, 0.95, 0.5])}
    dtype = rng.choice(list(DTYPES))
    most = (1 << 25) * 2 // BYTES[dtype]            # elements of one half, or of one tensor
    d = _log(rng, 48, 32768)
    if rng.random() < 0.5:
        d = max(64, d // 96 * 96 if d % 2 else d // 128 * 128)
        d -= 32 * (d == 3 * 1024)
    rows = _log(rng, 1, min(16384, most // d))
    if op == "step":
        return {"op": op, "act": rng.choice(["silu", "gelu"]), "rows": rows, "d": d,
                "dtype": dtype, "live": rng.choice([1.0, 0.75])}
    if op == "sparse":
        return {"op": op, "pass": rng.choice(["forward", "backward"]), "rows": rows, "d": d,
                "dtype": dtype, "z": rng.choice([0.0, Z95])}
    return {"op": op, "pass": rng.choice(["forward", "step"]), "rows": rows, "d": d,
            "dtype": dtype, "params": rng.choice([dtype, "fp32"]), "bias": rng.random() < 0.7}


# --------------------------------------------------------------------- inputs

def _live_rows(case):
    return max(1, int(case["rows"] * case["live"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"] == "balance":
        t, e = case["tokens"], case["experts"]
        logits = 1.5 * normal(t, e) + 0.5 * normal(1, e)
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["ids"] = torch.topk(s["logits"], case["k"], dim=1).indices
        s["live"] = uniform(t) < case["live"] if case["live"] < 1 else None
        s["grad_loss"] = 0.5 + uniform(1)
        return s

    m, d, dtype = case["rows"], case["d"], DTYPES[case["dtype"]]
    if case["op"] == "norm":
        # a residual stream: a mean and a scale of each row's own, a few strong channels
        x = normal(m, d) * (0.5 + 1.5 * uniform(m, 1)) + normal(m, 1)
        s["x"] = (x * (1 + 4 * (uniform(1, d) < 0.01))).to(dtype)
        s["weight"] = (1 + 0.1 * normal(d)).to(DTYPES[case["params"]])
        s["bias"] = (0.1 * normal(d)).to(DTYPES[case["params"]]) if case["bias"] else None
        s["grad"] = normal(m, d).to(dtype)
        return s

    # gate rows with a mean and a scale of their own and 1% outliers, up rows N(0, 1)
    gate = normal(m, d) * (0.5 + 1.5 * uniform(m, 1)) + (2 * uniform(m, 1) - 1)
    gate = torch.where(uniform(m, d) < 0.01, 4 * gate, gate)
    s["grad"] = normal(m, d).to(dtype)
    if case["op"] == "sparse" and case["pass"] == "backward":
        # what the forward pass left: the checkpoint of (gate - cutoff, up), and the deviations
        std, delta = _deviation(gate, case["z"])
        up = normal(m, d).to(dtype).float()
        halves = [_encode(delta, keep_sign=True), _encode(up)]
        s["codes"] = torch.cat([h[0] for h in halves], 1)
        s["scales"] = torch.cat([h[1] for h in halves], 1)
        s["std"] = std.squeeze(1)
        return s
    s["x"] = torch.cat([gate, normal(m, d)], 1).to(dtype)
    if case["op"] == "step":
        s["n_rows"] = torch.tensor([_live_rows(case)], dtype=torch.int32, device="cuda") \
            if case["live"] < 1 else None
    return s


# ---------------------------------------------------------------- plain forms

def _encode(v, keep_sign=False):
    """Codes [M, d] and scales [M, ceil(d/32)] of the 32-bit values ``v``: in each block the
    smallest power of two that brings its largest magnitude within 127, and the multiples of
    it nearest to the values; ``keep_sign`` gives every positive value a positive code."""
    m, d = v.shape
    blocks = -(-d // BLOCK)
    padded = torch.nn.functional.pad(v, (0, blocks * BLOCK - d)).view(m, blocks, BLOCK)
    top = padded.abs().amax(2, keepdim=True)
    scale = (((top.view(torch.int32) + 0x10000) >> 23) - 6).clamp(0, 248)
    bad = ~torch.isfinite(top)
    q = torch.round(padded * ((254 - scale) << 23).view(torch.float32)).clamp(-127, 127)
    if keep_sign:
        q = torch.where(padded > 0, q.clamp(min=1), q)
    q = torch.where(bad, torch.zeros_like(q), q)
    scale = torch.where(bad, torch.full_like(scale, 255), scale)
    codes = q.to(torch.int8).view(m, blocks * BLOCK)[:, :d].contiguous()
    return codes, scale.to(torch.uint8).squeeze(2)


def _decode(codes, scales):
    """The 32-bit values of one half's codes and scales."""
    bits = scales.to(torch.int32) << 23            # 2^(scale - 127), by its bits
    bits = torch.where(scales == 0, torch.full_like(bits, 0x00400000), bits)
    power = torch.where(scales == 255, torch.full_like(bits, 0x7FC00000), bits)
    power = power.view(torch.float32)
    return codes.float() * power.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _deviation(gate, z):
    """Each row's standard deviation, and gate - cutoff."""
    mean = gate.mean(1, keepdim=True)
    std = (gate - mean).square().mean(1, keepdim=True).sqrt()
    return std, gate - (mean + std * z)


def _silu(g):
    sig = 1 / (1 + torch.exp(-g))
    return g * sig, sig * (1 + g * (1 - sig))


def _gelu(g):
    t = torch.tanh(K * (g + C * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * (K + 3 * K * C * g * g)


ACTIVATIONS = {"silu": _silu, "gelu": _gelu}


def _plain_step(s, act, live):
    x, grad = s["x"][:live].float(), s["grad"][:live].float()
    dtype, d = s["x"].dtype, s["grad"].shape[1]
    a, _ = act(x[:, :d])
    out = (a * x[:, d:]).to(dtype)
    gate, up = _decode(*_encode(x[:, :d])), _decode(*_encode(x[:, d:]))
    a, slope = act(gate)
    grad_x = torch.cat([grad * up * slope, grad * a], 1).to(dtype)
    return {"out": out, "grad_x": grad_x, "again": (a * up).to(dtype)}


def _plain_sparse_forward(s, z):
    d = s["grad"].shape[1]
    x = s["x"].float()
    std, delta = _deviation(x[:, :d], z)
    a, _ = _gelu(delta.clamp(min=0))
    values = [_decode(*_encode(delta, keep_sign=True)), _decode(*_encode(x[:, d:]))]
    return {"out": (a * x[:, d:]).to(s["x"].dtype), "std": std.squeeze(1),
            "values": torch.cat(values, 1).to(torch.bfloat16)}


def _plain_sparse_backward(s, z):
    d = s["grad"].shape[1]
    n = s["scales"].shape[1] // 2
    grad, std = s["grad"].float(), s["std"][:, None]
    delta = _decode(s["codes"][:, :d], s["scales"][:, :n])
    up = _decode(s["codes"][:, d:], s["scales"][:, n:])
    a, slope = _gelu(delta.clamp(min=0))
    h = torch.where(delta <= 0, torch.zeros_like(grad), grad * up * slope)
    share = torch.where(std == 0, torch.zeros_like(delta), (delta + z * std) / std)
    gate = h - h.sum(1, keepdim=True) / d * (1 + z * share)
    dtype = s["grad"].dtype
    return {"grad_x": torch.cat([gate, grad * a], 1).to(dtype), "again": (a * up).to(dtype)}


def _plain_norm(s, step):
    x, w = s["x"].float(), s["weight"].float()
    dtype, d = s["x"].dtype, s["x"].shape[1]
    mean = x.sum(1, keepdim=True) / d
    rstd = 1 / torch.sqrt((x - mean).square().sum(1, keepdim=True) / d + EPS)
    hat = (x - mean) * rstd
    out = hat * w
    if s["bias"] is not None:
        out = out + s["bias"].float()
    got = {"out": out.to(dtype), "mean": mean.squeeze(1), "rstd": rstd.squeeze(1)}
    if step:
        grad = s["grad"].float()
        gw = grad * w
        inner = gw - gw.sum(1, keepdim=True) / d - hat * ((gw * hat).sum(1, keepdim=True) / d)
        got["grad_x"] = (rstd * inner).to(dtype)
        got["grad_weight"] = (grad * hat).sum(0)
        if s["bias"] is not None:
            got["grad_bias"] = grad.sum(0)
    return got


def _plain_balance(s):
    logits, ids, live = s["logits"].float(), s["ids"], s["live"]
    t, e = logits.shape
    k = ids.shape[1]
    if live is None:
        live = torch.ones(t, dtype=torch.bool, device=logits.device)
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = torch.where(live[:, None], p / p.sum(1, keepdim=True), torch.zeros_like(p))
    chosen = torch.where(live[:, None], ids, torch.full_like(ids, e)).view(-1)
    counts = torch.zeros(e + 1, dtype=torch.int32, device=ids.device)
    counts = counts.index_add_(0, chosen, torch.ones_like(chosen, dtype=torch.int32))[:e]
    tokens = live.sum(dtype=torch.int32).view(1)
    n = tokens.float().clamp(min=1)
    mean_p = p.sum(0) / n
    loss = COEF * e * (counts.float() / (n * k) * mean_p).sum().view(1)
    mixed = (p * counts.float()).sum(1, keepdim=True)
    grad = s["grad_loss"] * (COEF * e / (n * n * k)) * p * (counts.float() - mixed)
    return {"loss": loss, "counts": counts, "tokens": tokens, "mean_p": mean_p,
            "grad_logits": grad.to(s["logits"].dtype)}


# ------------------------------------------------------------------------ run

def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "step":
        return _plain_step(state, ACTIVATIONS[case["act"]], _live_rows(case))
    if case["op"] == "sparse":
        plain = _plain_sparse_forward if case["pass"] == "forward" else _plain_sparse_backward
        return plain(state, case["z"])
    if case["op"] == "norm":
        return _plain_norm(state, case["pass"] == "step")
    return _plain_balance(state)


def _run_own(s, case):
    import gated_activation_gb300 as ga
    if case["op"] == "step":
        forward, backward = ((ga.silu_and_mul_checkpoint, ga.silu_and_mul_backward)
                             if case["act"] == "silu" else
                             (ga.gelu_and_mul_checkpoint, ga.gelu_and_mul_backward))
        out, kept = forward(s["x"], n_rows=s["n_rows"])
        grad_x, again = backward(s["grad"], kept, n_rows=s["n_rows"], recompute=True)
        live = _live_rows(case)                # rows past the live ones are not written
        return {"out": out[:live], "grad_x": grad_x[:live], "again": again[:live]}
    if case["op"] == "sparse":
        if case["pass"] == "forward":
            out, kept = ga.gelu_and_mul_sparse_checkpoint(s["x"], case["z"])
            return {"out": out, "std": kept.std, "values": ga.checkpoint_values(kept)}
        kept = ga.Checkpoint(s["codes"], s["scales"], s["std"])
        grad_x, again = ga.gelu_and_mul_sparse_backward(s["grad"], kept, case["z"], recompute=True)
        return {"grad_x": grad_x, "again": again}
    if case["op"] == "norm":
        out, mean, rstd = ga.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
        got = {"out": out, "mean": mean, "rstd": rstd}
        if case["pass"] == "step":
            grad_x, grad_weight, grad_bias = ga.layer_norm_backward(
                s["grad"], s["x"], s["weight"], mean, rstd, bias=s["bias"] is not None)
            got["grad_x"], got["grad_weight"] = grad_x, grad_weight
            if grad_bias is not None:
                got["grad_bias"] = grad_bias
        return got
    kept = ga.moe_balance_loss(s["logits"], s["ids"], COEF, live=s["live"])
    grad = ga.moe_balance_loss_backward(s["grad_loss"], s["logits"], kept, live=s["live"])
    return {"loss": kept.loss, "counts": kept.counts, "tokens": kept.tokens,
            "mean_p": kept.mean_p, "grad_logits": grad}


# ----------------------------------------------------------------------- work

def work(case):
    """Bytes that each pass cannot do without; operations counted per element, a special
    function as one."""
    if case["op"] == "balance":
        t, e, size = case["tokens"], case["experts"], BYTES[case["dtype"]]
        read = 2 * e * size + 8 * case["k"]        # of a live token, in the two passes
        always = e * size + (2 if case["live"] < 1 else 0)
        n = t * case["live"]
        return {"bytes": n * read + t * always + 12 * e, "flops": 14 * n * e}
    m, d, size = case["rows"], case["d"], BYTES[case["dtype"]]
    held = 2 * d + 2 * -(-d // BLOCK)              # one row's codes and scales
    if case["op"] == "step":
        m = _live_rows(case)
        forward = 2 * d * size + d * size + held
        backward = d * size + held + 2 * d * size + d * size
        return {"bytes": m * (forward + backward), "flops": 50 * m * d}
    if case["op"] == "sparse":
        if case["pass"] == "forward":              # then the values: codes read, bf16 written
            return {"bytes": m * (3 * d * size + held + 4 + held + 4 * d), "flops": 35 * m * d}
        return {"bytes": m * (4 * d * size + held + 4), "flops": 40 * m * d}
    params = d * BYTES[case["params"]] * (2 if case["bias"] else 1)
    work_ = {"bytes": m * (2 * d * size + 8) + params, "flops": 8 * m * d}
    if case["pass"] == "step":
        work_["bytes"] += m * (3 * d * size + 8) + d * BYTES[case["params"]] \
            + 4 * d * (2 if case["bias"] else 1)
        work_["flops"] += 16 * m * d
    return work_


# ---------------------------------------------------------------------- exact

def _power(k):
    """2^k in 64 bits, exactly."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_to_block(v, keep_sign=False):
    """The values that the checkpoint of ``v`` (64 bits) stands for, from its definition."""
    m, d = v.shape
    blocks = -(-d // BLOCK)
    b = torch.zeros(m, blocks * BLOCK, dtype=torch.float64, device=v.device)
    b[:, :d] = v
    b = b.view(m, blocks, BLOCK)
    top = b.abs().max(2, keepdim=True).values
    # top = f 2^e with f in [1/2, 1): f 2^7 < 128 is the first candidate's largest code
    f, e = torch.frexp(top)
    k = torch.where(f * 128 >= 127.5, e - 6, e - 7).clamp(-127, 121)
    step = _power(k)
    q = (b / step).round().clamp(-127, 127)
    if keep_sign:
        q = torch.where((b > 0) & (q < 1), torch.ones_like(q), q)
    return (q * step).view(m, blocks * BLOCK)[:, :d]


def _from_codes(codes, scales):
    step = _power(scales.to(torch.int64) - 127)
    wide = step[:, :, None].expand(-1, -1, BLOCK).reshape(codes.shape[0], -1)
    return codes.to(torch.float64) * wide[:, :codes.shape[1]]


def _exact_act(name, g):
    if name == "silu":
        sig = torch.sigmoid(g)
        return g * sig, sig + g * sig * (1 - sig)
    # gelu_tanh(g) = g sigmoid(2y)
    sig = torch.sigmoid(2 * K * (g + C * g ** 3))
    return g * sig, sig + g * sig * (1 - sig) * 2 * K * (1 + 3 * C * g ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "step":
            live, d = _live_rows(case), case["d"]
            x, grad = s["x"][:live].double(), s["grad"][:live].double()
            out = _exact_act(case["act"], x[:, :d])[0] * x[:, d:]
            gate, up = _round_to_block(x[:, :d]), _round_to_block(x[:, d:])
            a, slope = _exact_act(case["act"], gate)
            return {"out": out, "grad_x": torch.cat([grad * up * slope, grad * a], 1),
                    "again": a * up}
        if case["op"] == "sparse":
            z, d = case["z"], case["d"]
            if case["pass"] == "forward":
                x = s["x"].double()
                gate, up = x[:, :d], x[:, d:]
                std = torch.std(gate, 1, correction=0, keepdim=True)
                delta = gate - gate.mean(1, keepdim=True) - z * std
                out = torch.where(delta > 0, _exact_act("gelu", delta)[0], delta * 0) * up
                values = torch.cat([_round_to_block(delta, True), _round_to_block(up)], 1)
                return {"out": out, "std": std[:, 0], "values": values}
            n = s["scales"].shape[1] // 2
            delta = _from_codes(s["codes"][:, :d], s["scales"][:, :n])
            up = _from_codes(s["codes"][:, d:], s["scales"][:, n:])
            grad, std = s["grad"].double(), s["std"].double()[:, None]
            a, slope = _exact_act("gelu", delta)
            a, slope = a * (delta > 0), slope * (delta > 0)
            h = grad * up * slope
            cutoff = torch.where(std > 0, 1 + z * (delta / std + z), torch.ones_like(delta))
            gate = h - h.mean(1, keepdim=True) * cutoff
            return {"grad_x": torch.cat([gate, grad * a], 1), "again": a * up}
        if case["op"] == "norm":
            x, w = s["x"].double(), s["weight"].double()
            var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
            rstd = (var + EPS) ** -0.5
            hat = (x - mean) * rstd
            out = hat * w + (s["bias"].double() if s["bias"] is not None else 0)
            got = {"out": out, "mean": mean[:, 0], "rstd": rstd[:, 0]}
            if case["pass"] == "step":
                grad = s["grad"].double()
                g = grad * w
                g = g - g.mean(1, keepdim=True)
                got["grad_x"] = rstd * (g - hat * (g * hat).mean(1, keepdim=True))
                got["grad_weight"] = (grad * hat).sum(0)
                if s["bias"] is not None:
                    got["grad_bias"] = grad.sum(0)
            return got
        live = s["live"]
        keep = torch.arange(case["tokens"], device="cuda") if live is None else live.nonzero()[:, 0]
        e, k, n = case["experts"], case["k"], max(1, len(keep))
        p = torch.softmax(s["logits"].double()[keep], 1)
        counts = torch.bincount(s["ids"][keep].reshape(-1), minlength=e).double()
        share = counts / (n * k)
        grad = torch.zeros(case["tokens"], e, dtype=torch.float64, device="cuda")
        g = p * (share - (p @ share)[:, None]) * (COEF * e / n)
        grad[keep] = s["grad_loss"].double() * g
        return {"loss": COEF * e * (share * p.sum(0) / n).sum().view(1), "counts": None,
                "tokens": None, "mean_p": p.sum(0) / n, "grad_logits": grad}
