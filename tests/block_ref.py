"""Plain 64-bit forms of the 8-bit layer, the norm between blocks and the scoring
of logits, with the error that the kernels' 32-bit arithmetic may add.

A rounding to nearest is off by at most half a step: 2^-24 of the value in fp32,
2^-8 in bf16, 2^-11 in fp16 (and half of the smallest subnormal, 2^-25), 2^-4 in
e4m3 (and 2^-10). The bounds below count those, and are derived beside each form;
they were written down before the kernels' results were compared with them.
"""
import math

import torch

U = 2.0 ** -24
E4M3 = torch.float8_e4m3fn
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, E4M3: 2.0 ** -4}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, E4M3: 2.0 ** -10}
C448 = torch.tensor(1.0 / 448.0, dtype=torch.float32)


def blocks(x, rows):
    R, K = x.shape
    rb, kb = -(-R // rows), -(-K // 128)
    p = x.new_zeros(rb * rows, kb * 128)
    p[:R, :K] = x
    return p.view(rb, rows, kb, 128)


def quant(x, rows):
    """The quantiser as it is defined, in fp32 on the CPU: the kernel has to give the same bits."""
    R, K = x.shape
    b = blocks(x.float().cpu(), rows)
    a = b.abs().amax(dim=(1, 3))  # carries a NaN on
    s = a * C448
    s = torch.where(s < 2.0 ** -126, torch.full_like(s, 2.0 ** -126), s)
    v = (b * (1.0 / s)[:, None, :, None]).clamp(-448.0, 448.0)
    q = v.to(E4M3).view(b.shape[0] * rows, -1)[:R, :K]
    return q, s.t().contiguous()


def widen(q, s, rows):
    """The values that codes and scales stand for, in 64 bits."""
    R, K = q.shape
    i = torch.arange(R, device=q.device) // rows
    j = torch.arange(K, device=q.device) // 128
    return q.double() * s.double()[j[None, :], i[:, None]]


def operand(R, K, rows, gen, std=1.0, device="cuda"):
    """Random codes (every finite e4m3 value may appear) and scales of an operand."""
    x = torch.randn(R, K, generator=gen) * std
    q, s = quant(x, rows)
    s = s * (0.5 + torch.rand(s.shape, generator=gen))
    return q.to(device), s.to(device)


def product(x, xs, w, ws):
    """y = x w^T and the bound on the fp32 kernels' error.

    Products of e4m3 values are exact. A block's 128 products are summed by the
    tensor core, whose fp32 additions need not round to nearest: a whole step
    (2 U) of the running magnitude each. The scale is rounded once, and every
    block's promotion and every partial sum of a cluster (at most 8) adds a rounding.
    """
    X, W = widen(x, xs, 1), widen(w, ws, 128)
    mag = X.abs() @ W.abs().t()
    nkb = -(-X.shape[1] // 128)
    return X @ W.t(), 2 * U * (128 + nkb + 12) * mag


def rounded(y, err, dtype):
    """The bound once y is rounded to dtype."""
    return err + HALF[dtype] * (y.abs() + err) + TINY[dtype] if dtype != torch.float32 else err + U * y.abs()


ACT = {
    "silu": lambda g: g * torch.sigmoid(g),
    "gelu": lambda g: 0.5 * g * torch.erfc(-g / math.sqrt(2.0)),
    "gelu_tanh": lambda g: g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)),
    "relu": torch.relu,
}


def gated(x, xs, wg, gs, wu, us, act):
    """h = act(g) u and its bound: the slope of every activation is below 1.2. silu's exponential is off by
    2 + 1.2 |g| steps (its documented bound), its division by 2 more; the forms of gelu as 1 plus a function within
    [-1, 1] that is good to a few steps of 1 (8 with its argument's) leave |g| / 2 times that; relu is exact."""
    g, eg = product(x, xs, wg, gs)
    u, eu = product(x, xs, wu, us)
    a = ACT[act](g)
    if act == "silu":
        ea = a.abs() * 2 * U * (6 + 1.2 * g.abs())
    elif act == "relu":
        ea = torch.zeros_like(a)
    else:
        ea = g.abs() * 8 * U
    ea = ea + 1.2 * eg
    return a * u, ea * (u.abs() + eu) + a.abs() * eu + 2 * U * (a * u).abs()


def check_close(got, want, bound, what=""):
    got = got.double()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst ratio "
                           f"{float(((got - want).abs() / bound.clamp_min(1e-300))[bad].max())}")


def check_quantised(q, s, h, err, what=""):
    """Codes and scales of h in blocks of 128 columns: the scale to its roundings and h's error, the codes to half
    a step of theirs (a value on a border may fall to either side by its error)."""
    b = blocks(h, 1)
    a, ea = b.abs().amax(3)[:, 0].t(), blocks(err, 1).amax(3)[:, 0].t()
    S = (a / 448.0).clamp_min(2.0 ** -126)
    check_close(s, S, 4 * U * S + ea / 448.0 * (1 + 1e-6) + 1e-45, what + " scales")
    v = widen(q, s, 1)
    step = widen(torch.ones_like(h), s, 1)
    check_close(v, h, (2.0 ** -4 * (h.abs() + err) + step * 2.0 ** -10) * (1 + 1e-5) + err, what + " codes")


def _unit(v, ev, kind, eps, w, b, add):
    """kind(v) * w + b and its bound, v itself being off by ev. Sums of a row: at most 32 values in a thread, 5 + 4
    levels of a tree and a few more: 48 roundings, each U of the sum of magnitudes; the root, its Newton step and
    the products add 8."""
    if kind == "none":
        y, ey = v, ev
    else:
        n = v.shape[1]
        mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
        em = 48 * U * v.abs().mean(1, keepdim=True) + ev.mean(1, keepdim=True) if kind == "layer" else mean
        c = v - mean
        ec = ev + em + U * c.abs()
        ms = (c * c).sum(1, keepdim=True) / n + eps
        ems = 48 * U * ms + (2 * c.abs() * ec + ec * ec).sum(1, keepdim=True) / n
        r = ms.rsqrt()
        # r as a function of ms, to second order: its relative change is ems / ms at most while that is below 1/2
        rel = (ems / ms).clamp(max=0.5) + 8 * U
        y = c * r
        ey = (ec * r + y.abs() * rel) * (1 + rel)
    if w is not None:
        w = w.double() + add
        y, ey = y * w, ey * w.abs() + 3 * U * (y * w).abs()
    if b is not None:
        y, ey = y + b.double(), ey + 2 * U * (y + b.double()).abs() + 2 * U * y.abs()
    return y, ey + 2 * U * y.abs()


def norm(x, weight, bias, eps, kind, block=None, post="none", post_weight=None, post_bias=None, post_eps=None,
         gate=None, scale=1.0, unit_offset=False):
    """(n, its bound, r, its bound)."""
    add = 1.0 if unit_offset else 0.0
    r, er = x.double(), torch.zeros_like(x, dtype=torch.float64)
    if block is not None:
        v = block.double()
        z, ez = _unit(v, torch.zeros_like(v), post, eps if post_eps is None else post_eps, post_weight, post_bias, add)
        if gate is not None:
            g = gate.double().expand_as(z)
            z, ez = z * g, ez * g.abs() + 2 * U * (z * g).abs()
        z, ez = scale * z, abs(scale) * ez + 2 * U * (scale * z).abs()
        r, er = r + z, ez + 2 * U * (r + z).abs()
    n, en = _unit(r, er, kind, eps, weight, bias, add)
    return n, en, r, er


def logprobs(x, targets, temp, k):
    """(logprob, entropy, top_logprob, top_index, bound [T, 1] of the normaliser, bound of the entropy)."""
    raw = x.double()
    T, V = x.shape
    m = raw.amax(1, keepdim=True)
    empty = torch.isneginf(m)
    d = (raw - torch.where(empty, torch.zeros_like(m), m)) / temp
    d = torch.where(torch.isneginf(raw), torch.full_like(d, -math.inf), d)
    e = torch.exp(d)
    S = e.sum(1, keepdim=True)
    lp = d - torch.log(S)
    p = torch.where(empty, torch.zeros_like(e), e / S)
    away = torch.where(p > 0, p * d.abs(), torch.zeros_like(p)).sum(1, keepdim=True)
    H = torch.where(empty, torch.zeros_like(S), torch.log(S) + away)[:, 0]
    lp = torch.where(empty | torch.isneginf(raw), torch.full_like(lp, -math.inf), lp)
    order = torch.argsort(-raw, dim=1, stable=True)[:, :k]
    if order.shape[1] < k:
        order = torch.cat([order, order.new_zeros(T, k - order.shape[1])], 1)
        gone = torch.arange(k, device=x.device)[None, :] >= V
    else:
        gone = torch.zeros(1, k, dtype=torch.bool, device=x.device)
    top = lp.gather(1, order)
    gone = gone | torch.isneginf(raw.gather(1, order))
    idx = torch.where(gone, torch.full_like(order, -1), order)
    top = torch.where(gone, torch.full_like(top, -math.inf), top)
    at = None
    if targets is not None:
        at = lp.gather(1, targets.clamp_min(0)[:, None])[:, 0]
        at = torch.where(targets < 0, torch.zeros_like(at), at)
    # The sum: V / 256 values in a thread (in two lanes, then joined) and 20 more joins, U of the sum each; an
    # exponential is off by 4 U and by its argument's roundings, 4 U of the argument. Then the logarithm: 2 steps.
    n = V / 256 + 24
    es = (n + 8) * U + 4 * U * away
    elog = es + 4 * U * torch.log(S).abs() + 2 * U
    eh = elog + (n + 12) * U * away + 8 * U * (away + away ** 2) + 4 * U * H[:, None].abs()
    return at, H, top, idx, torch.where(empty, torch.zeros_like(elog), elog), torch.where(empty, torch.zeros_like(eh), eh)[:, 0]
