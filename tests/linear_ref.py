"""Plain 64-bit forms of the gated projections and the cross entropy of a linear layer, written
from their definitions, and the bounds that the kernels' outputs are held to.

Where the bounds come from.  A product of k terms is summed in fp32 from exact products, 16 terms
to an instruction, each sum possibly cut off instead of rounded: at most k / 16 + 16 steps of
2^-23 of the terms' absolute sum, so ``acc(k) = (k / 16 + 16) 2^-23`` of it.  Elementwise fp32
arithmetic is within ARITH = 2^-18 of its terms (64 roundings, more than any element passes
through).  Rounding to an element type adds half a step, ``eps / 2`` of the value, or half the
smallest subnormal number.  What a sum is made of carries its own errors into it: those are
propagated to first order with the absolute values of the factors (times 1.01 for the rest).
Where the two passes meet, the projections that the forward pass keeps are off by half of a code's
step, 2^-15 of their block's largest magnitude.
"""
import torch

ARITH = 2.0 ** -18
MORE = 1.01
K2 = 2.0 * (2.0 / torch.pi) ** 0.5
CUBIC = 0.044715


def acc(k):
    return (k / 16 + 16) * 2.0 ** -23


def half_step(x, dtype):
    f = torch.finfo(dtype)
    return x.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def act(name, g):
    """act, its slope, and a bound on its second derivative (0.5 for silu, at 0; for gelu_tanh
    2 k2 / 2 + ... < 1.6 = K2 at 0, where it is largest)."""
    if name == "silu":
        y, dy, second = g, torch.ones_like(g), 0.5
    else:
        y, dy, second = K2 * (g + CUBIC * g ** 3), K2 * (1 + 3 * CUBIC * g ** 2), K2
    s = torch.sigmoid(y)
    far = torch.sigmoid(-y)
    return g * s, s + g * s * far * dy, second


def check(got, ref, bound, what):
    """got within bound of ref.  A value past the type's largest number rounds to infinity: that
    is right where ref may lie there (fp16: 65504)."""
    most = torch.finfo(got.dtype).max
    got, ref = got.double(), ref.to(got.device)
    assert got.shape == ref.shape, f"{what}: shape"
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    bad = ~nan & ~((got - ref).abs() <= bound)
    bad &= ~((got == ref) | (torch.isinf(got) & (got.sign() * ref + bound >= most)))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside their bounds, first "
                             f"at {list(i)}: {got[i]} for {ref[i]} (bound {bound[i]})")


def forward(name, x, w, dtype):
    """(out, its bound, g, u, their bounds) of rows x [n, k] and weight w [2d, k], in 64 bits."""
    d, k = w.shape[0] // 2, w.shape[1]
    h, off = x @ w.T, acc(k) * (x.abs() @ w.abs().T)
    g, u, og, ou = h[:, :d], h[:, d:], off[:, :d], off[:, d:]
    a, slope, _ = act(name, g)
    out = a * u
    # |slope| <= 1.13; the exponent's own roundings grow with |g|
    bound = MORE * (u.abs() * 1.13 * og + a.abs() * ou) + ARITH * (1 + g.abs()) * out.abs() \
        + half_step(out, dtype) + 1e-30
    return out, bound, g, u, og, ou


def block_top(v):
    """The largest magnitude of each element's block of 32 in its row."""
    n, d = v.shape
    b = -(-d // 32)
    p = torch.zeros(n, b * 32, dtype=v.dtype, device=v.device)
    p[:, :d] = v.abs()
    return p.view(n, b, 32).amax(2).repeat_interleave(32, 1)[:, :d]


def backward(name, dy, x, w, dtype):
    """((grad_in, bound), (grad_weight, bound)) from the definition, in 64 bits."""
    n, d, k = len(x), w.shape[0] // 2, w.shape[1]
    _, _, g, u, og, ou = forward(name, x, w, dtype)
    a, slope, second = act(name, g)
    step = 2.0 ** -15 * MORE
    og, ou = og + step * block_top(g), ou + step * block_top(u)
    dg, du = dy * u * slope, dy * a
    rows = torch.cat([dg, du], 1)
    off = torch.cat([dy.abs() * (1.13 * ou + u.abs() * second * og), dy.abs() * 1.13 * og], 1)
    off = MORE * off + ARITH * (1 + torch.cat([g, g], 1).abs()) * torch.cat(
        [(dy * u).abs() * 1.13, du.abs()], 1) + half_step(rows, dtype)
    gi, gw = rows @ w, rows.T @ x
    bi = MORE * (off @ w.abs()) + acc(2 * d) * (rows.abs() @ w.abs()) + half_step(gi, dtype)
    bw = MORE * (off.T @ x.abs()) + acc(n) * (rows.abs().T @ x.abs()) + half_step(gw, dtype)
    return (gi, bi + 1e-30), (gw, bw + 1e-30)


def entropy(x, w, goal):
    """(loss, bound, lse, bound, logits, their bound) of live rows."""
    k = w.shape[1]
    logits, off = x @ w.T, acc(k) * (x.abs() @ w.abs().T)
    lse = torch.logsumexp(logits, 1)
    at = logits.gather(1, goal[:, None])[:, 0]
    # lse is an average of the logits' errors; sums of positive terms in fp32
    worst = off.amax(1) + ARITH * (1 + logits.abs().amax(1))
    bound = worst + 2.0 ** -22 * lse.abs()
    return lse - at, bound + off.gather(1, goal[:, None])[:, 0] + 2.0 ** -22 * at.abs(), lse, bound, logits, off


def entropy_backward(gl, x, w, goal, dtype):
    """((grad_in, bound), (grad_weight, bound)) of live rows."""
    n, v = len(x), len(w)
    _, _, lse, olse, logits, off = entropy(x, w, goal)
    p = torch.exp(logits - lse[:, None])
    y = p.clone()
    y[torch.arange(n, device=y.device), goal] -= 1
    # y / c, c = 1 - p_target, is an operand (the target's -1 exact), f = gl c stands outside, and f x is the other
    # operand.  y's own error, in units of y: the logits' and the loss's; then the roundings, half a step each:
    # y's of all but the target's column, and f x's.  c is within the loss's error of its own value.
    oy = MORE * p * (off + 2 * olse[:, None] + ARITH * (1 + logits.abs())) + 2.0 ** -21 * (p + y.abs())
    oy = oy + y.abs() * (2 * olse[:, None] + ARITH)
    weight, half = gl[:, None].abs(), torch.finfo(dtype).eps / 2 * MORE
    c = 1 - torch.exp(logits.gather(1, goal[:, None]) - lse[:, None])
    f = gl.abs()[:, None] * c
    power = 2.0 ** (torch.floor(torch.log2(f.max())) + 1) if n and f.max() > 0 else 1.0
    # fp16: half a subnormal step, of y under its 2^14 and of f x under the power of two above every f
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    off_in = weight * (oy + half * p) + f * tiny * 2.0 ** -14
    off_w = weight * (oy + half * (p + y.abs())) + f * tiny * 2.0 ** -14
    rows = gl[:, None] * y
    gi, gw = rows @ w, rows.T @ x
    # sums over pieces of the vocabulary add fp32 roundings
    bi = MORE * (off_in @ w.abs()) + (acc(v) + 2.0 ** -18) * (rows.abs() @ w.abs()) + half_step(gi, dtype)
    bw = MORE * (off_w.T @ x.abs()) + acc(n) * (rows.abs().T @ x.abs()) + half_step(gw, dtype) \
        + (tiny * power * (y.abs() / c.clamp(min=1e-30)).sum(0)[:, None] if n else 0.0)
    return (gi, bi + 1e-30), (gw, bw + 1e-30)
