"""Plain 64-bit forms of the training operators, written from their definitions, and the
bounds that the kernels' outputs are held to.

The kernels compute in fp32 and round each output once, to nearest even.  An output of value
``ref`` whose terms have the absolute sum ``mag`` is computed to within ARITH * mag before it is
rounded: 2^-18 is 64 fp32 roundings, more than any element passes through (the longest sums here
are trees over threads after at most a few dozen terms each, and the special functions are within
a few units).  Rounding is monotonic, so the output lies between the roundings of ref - ARITH mag
and ref + ARITH mag: no allowance for the rounding itself is needed.  Two terms go with that:
a product that falls below fp32's normal range is rounded to a multiple of 2^-149, so UNDER, four
such roundings, is added; and where a result is an exponential e^a, the up to four roundings of its
argument count as 4 |a| 2^-24 of it, so ``mag`` grows by 1 + |a| / 16.
"""
import torch

ARITH = 2.0 ** -18
UNDER = 4 * 2.0 ** -150
K2 = 2.0 * (2.0 / torch.pi) ** 0.5
CUBIC = 0.044715


def check(got, ref, mag, dtype, what):
    got, ref = got.double().cpu(), ref.cpu()
    assert got.shape == ref.shape, what
    off = ARITH * mag.cpu() + UNDER
    low, high = ((ref + s * off).to(dtype).double() for s in (-1, 1))
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    bad = ((got < low) | (got > high)) & ~nan
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside their bounds, "
                             f"first at {list(i)}: {got[i]} for {ref[i]} "
                             f"({low[i]} to {high[i]})")


def power(k):
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def blocks(v):
    """[M, d] as blocks of 32, the last one filled with zeros: [M, B, 32]."""
    m, d = v.shape
    b = -(-d // 32)
    out = torch.zeros(m, b * 32, dtype=v.dtype)
    out[:, :d] = v
    return out.view(m, b, 32)


def encode(v):
    """(codes int8 [M, d], scales uint8 [M, B]) of 64-bit values by the definition: the
    smallest k in [-127, 121] with rint(max |v| 2^-k) <= 127, found by trying; past that the
    codes stop at 127."""
    m, d = v.shape
    b = blocks(v)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    k = torch.full(top.shape, -127, dtype=torch.int64)
    clean = torch.where(bad, torch.zeros_like(top), top)
    for e in range(-127, 121):
        k = torch.where((clean * 2.0 ** -e).round() > 127, torch.full_like(k, e + 1), k)
    q = (b / power(k)[..., None]).round().clamp(-127, 127)
    q = torch.where(bad[..., None], torch.zeros_like(q), q)
    scales = torch.where(bad, torch.full_like(k, 255), k + 127)
    return q.reshape(m, -1)[:, :d].to(torch.int8), scales.to(torch.uint8)


def steps(scales, d):
    """The step of every element, [M, d]: NaN in bad blocks."""
    s = power(scales.to(torch.int64) - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return s.repeat_interleave(32, 1)[:, :d]


def values(codes, scales):
    """[M, 2d] values of a checkpoint."""
    d, b = codes.shape[1] // 2, scales.shape[1] // 2
    codes, scales = codes.cpu(), scales.cpu()
    return torch.cat([codes[:, :d].double() * steps(scales[:, :b], d),
                      codes[:, d:].double() * steps(scales[:, b:], d)], 1)


def act(name, g):
    """(act(g), act'(g), sum of the magnitudes of the slope's terms, growth of the bound)."""
    if name == "silu":
        a, da = g, torch.ones_like(g)
    else:
        a, da = K2 * (g + CUBIC * g ** 3), K2 * (1 + 3 * CUBIC * g ** 2)
    s, c = torch.sigmoid(a), torch.sigmoid(-a)
    second = torch.nan_to_num(g * s * c * da, nan=0.0) + 0 * torch.isnan(g) * g
    return g * s, s + second, s + second.abs(), 1 + a.abs() / 16


def act_backward(name, v, dy):
    """({"grad", "out"}: (ref, mag)) of the elementwise backward pass at values v = (g, u)."""
    d = dy.shape[1]
    g, u = v[:, :d], v[:, d:]
    a, slope, mag, grow = act(name, g)
    return {"grad": (torch.cat([dy * u * slope, dy * a], 1),
                     torch.cat([(dy * u).abs() * mag * grow, (dy * a).abs() * grow], 1)),
            "out": (a * u, (a * u).abs() * grow)}


def sparse_stats(x, d, z):
    g = x[:, :d]
    mean = g.mean(1, keepdim=True)
    std = ((g - mean) ** 2).mean(1, keepdim=True).sqrt()
    return mean, std, g - (mean + std * z)


def sparse_backward(v, dy, std, z):
    d = dy.shape[1]
    delta, u = v[:, :d], v[:, d:]
    s = torch.where(delta > 0, delta, delta * 0)
    a, slope, mag, grow = act("gelu", s)
    on = ~(delta <= 0)
    h = torch.where(on, dy * u * slope, torch.zeros_like(dy))
    hm = torch.where(on, (dy * u).abs() * mag * grow, torch.zeros_like(dy))
    std = std[:, None]
    term = torch.where(std == 0, torch.zeros_like(delta), z * (delta + z * std) / std)
    tmag = torch.where(std == 0, torch.zeros_like(delta), abs(z) * (delta.abs() + abs(z) * std) / std)
    grad = h - h.sum(1, keepdim=True) / d * (1 + term)
    gmag = hm + hm.sum(1, keepdim=True) / d * (1 + tmag)
    return {"grad": (torch.cat([grad, dy * a], 1), torch.cat([gmag, (dy * a).abs() * grow], 1)),
            "out": (a * u, (a * u).abs() * grow)}


def layer_norm(x, w, b, eps):
    """{"out", "mean", "rstd"}: (ref, mag); the magnitudes carry what the mean's rounding
    (relative to the row's mean magnitude) does to x - mean."""
    d = x.shape[1]
    mean = x.mean(1, keepdim=True)
    rstd = 1 / (((x - mean) ** 2).mean(1, keepdim=True) + eps).sqrt()
    hat = (x - mean) * rstd
    big = x.abs().mean(1, keepdim=True)
    hat_mag = hat.abs() * (1 + big * rstd) + big * rstd + rstd * x.abs() * 2.0 ** -5
    out = hat * w + (b if b is not None else 0)
    return {"out": (out, hat_mag * w.abs() + (b.abs() if b is not None else 0)),
            "mean": (mean[:, 0], big[:, 0]),
            "rstd": (rstd[:, 0], (rstd * (1 + big * rstd))[:, 0]),
            "hat": (hat, hat_mag)}


def layer_norm_backward(x, dy, w, eps):
    f = layer_norm(x, w, None, eps)
    hat, hat_mag = f["hat"]
    rstd = f["rstd"][0][:, None]
    g = dy * w
    a, b = g.mean(1, keepdim=True), (g * hat).mean(1, keepdim=True)
    grad = rstd * (g - a - hat * b)
    bm = (g.abs() * hat_mag).mean(1, keepdim=True)
    mag = rstd * (g.abs() + g.abs().mean(1, keepdim=True) + hat_mag * b.abs() + hat.abs() * bm)
    grow = 1 + f["rstd"][1][:, None] / rstd            # rstd's own relative error
    return {"grad": (grad, mag * grow),
            "weight": ((dy * hat).sum(0), (dy.abs() * hat_mag).sum(0)),
            "bias": (dy.sum(0), dy.abs().sum(0))}


def balance(logits, ids, live, coef):
    """{"loss", "mean_p", "grad"}: (ref, mag), with "counts" and "tokens"."""
    t, e = logits.shape
    k = ids.shape[1]
    on = torch.ones(t, dtype=torch.bool) if live is None else live.bool()
    x = logits[on]
    top = x.amax(1, keepdim=True) if len(x) else x[:, :1]
    top = torch.where(top == -float("inf"), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(1, keepdim=True)
    p = torch.where(total == 0, p, p / total)
    span = (x - top).abs().nan_to_num(posinf=0.0).amax(1, keepdim=True) if len(x) else total
    kept = ids[on].reshape(-1)
    kept = kept[(kept >= 0) & (kept < e)]
    counts = torch.bincount(kept, minlength=e)
    n = max(1, int(on.sum()))
    c = counts.double()
    mean_p = p.sum(0) / n
    share = c / (n * k)
    scale = coef * e / (n * n * k)
    mid = c - c.mean()
    grad = torch.zeros(t, e, dtype=torch.float64)
    mag = torch.zeros(t, e, dtype=torch.float64)
    grad[on] = scale * p * (c - (p * c).sum(1, keepdim=True))
    mag[on] = (1 + span / 16) * scale * p * (mid.abs() + 1 + (p * (mid.abs() + 1)).sum(1, keepdim=True))
    pm = ((1 + span / 16) * p).sum(0) / n
    return {"counts": counts.to(torch.int32), "tokens": int(on.sum()),
            "mean_p": (mean_p, pm), "loss": (coef * e * (share * mean_p).sum().view(1),
                                            coef * e * (share * pm).sum().view(1)),
            "grad": (grad, mag)}
