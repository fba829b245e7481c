"""The 8-bit layer, the norm between blocks and the scoring of logits: what is measured of them.

Five operators, each as a user's program calls it:
  quant     blocks of 128 (rows) or 128 x 128 (weights) to e4m3 with an fp32 scale each
  gemm      y = x W^T on such operands
  gated     h = act(x Wg^T) * (x Wu^T) on such operands, also requantised for the next product
  norm      norm after a block, gate, residual scale and the next block's norm in one pass
  logprobs  log probabilities of given tokens, entropy and the top alternatives of a row of logits
Where `own` is false `run` computes them in elementary torch operations in 32 bits.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": E4M3}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
DEV = "cuda"


def listed():
    return [
        # One token's activations before an 8-bit layer (decode; latency).
        {"name": "quant_row_T1", "op": "quant", "T": 1, "K": 4096, "rows": 1, "dtype": "bf16"},
        # A gate projection's weights when a model is loaded.
        {"name": "quant_weight", "op": "quant", "T": 11008, "K": 4096, "rows": 128, "dtype": "f16"},
        # Attention output projection, one token.
        {"name": "gemm_T1", "op": "gemm", "T": 1, "N": 4096, "K": 4096, "out": "bf16"},
        # Down projection of a small batch of decoding sequences.
        {"name": "gemm_T16_down", "op": "gemm", "T": 16, "N": 4096, "K": 11008, "out": "f32"},
        # A ragged prompt: odd token count, odd output width.
        {"name": "gemm_T333_odd", "op": "gemm", "T": 333, "N": 4099, "K": 4096, "out": "bf16"},
        # The large skewed prefill layer in 8 bits.
        {"name": "gemm_T4096_large", "op": "gemm", "T": 4096, "N": 28672, "K": 8192, "out": "bf16"},
        # Gate and up projections, eight decoding sequences, ready for the down projection.
        {"name": "gated_T8", "op": "gated", "T": 8, "N": 11008, "K": 4096, "out": "e4m3", "act": "silu"},
        # Gate and up projections of a prompt.
        {"name": "gated_T2048", "op": "gated", "T": 2048, "N": 11008, "K": 4096, "out": "e4m3", "act": "silu"},
        # Between two blocks of one decoding sequence: fp32 block output, bf16 residual stream.
        {"name": "norm_T1", "op": "norm", "T": 1, "D": 4096, "block": "f32", "x": "bf16", "out": "bf16",
         "post": "none", "kind": "rms", "gate": "none"},
        # Between two blocks of a long prompt, norms on both sides, a gate per channel, e4m3 out.
        {"name": "norm_T8192", "op": "norm", "T": 8192, "D": 4096, "block": "bf16", "x": "bf16", "out": "e4m3",
         "post": "rms", "kind": "rms", "gate": "channel"},
        # Sampling step of a few sequences: fp32 logits as the GEMMs give them.
        {"name": "logprobs_T4", "op": "logprobs", "T": 4, "V": 32000, "dtype": "f32", "top": 20, "masked": False},
        # Scoring a prompt (perplexity) over a large odd vocabulary, some entries masked.
        {"name": "logprobs_T2048", "op": "logprobs", "T": 2048, "V": 128001, "dtype": "bf16", "top": 5, "masked": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "gated", "norm", "logprobs"])
    if op == "quant":
        return {"op": op, "T": _log(rng, 1, 8192), "K": _log(rng, 1, 11008), "rows": rng.choice([1, 128]),
                "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op in ("gemm", "gated"):
        c = {"op": op, "T": _log(rng, 1, 4096), "N": _log(rng, 1, 11008), "K": 16 * _log(rng, 1, 688)}
        if op == "gemm":
            return {**c, "out": rng.choice(["f32", "bf16", "f16"])}
        c["out"] = rng.choice(["e4m3", "e4m3", "bf16", "f32"])
        return {**c, "N": -(-c["N"] // 16) * 16 if c["out"] == "e4m3" else c["N"],
                "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"])}
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 8192), "D": _log(rng, 8, 8192), "block": rng.choice(["f32", "bf16", "f16"]),
                "x": rng.choice(["f32", "bf16"]), "out": rng.choice(["e4m3", "bf16", "f16", "f32"]),
                "post": rng.choice(["none", "rms", "layer"]), "kind": rng.choice(["rms", "layer"]),
                "gate": rng.choice(["none", "channel", "token", "full"])}
    return {"op": op, "T": _log(rng, 1, 2048), "V": _log(rng, 100, 131072), "dtype": rng.choice(["f32", "bf16", "f16"]),
            "top": rng.choice([0, 1, 5, 20, 32]), "masked": rng.choice([True, False])}


# ---- inputs ------------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFF)


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * std


def _activations(g, T, K):
    """Unit activations with a few outlier channels, as between two layers of a language model."""
    loud = 1.0 + 9.0 * (torch.rand(K, generator=g, device=DEV) < 0.005).float()
    return _normal(g, T, K) * loud


def _operand(g, R, K, rows, weight):
    """An e4m3 operand [R, K] and its scales [ceil(K/128), ceil(R/rows)], as a program has them in hand."""
    x = _normal(g, R, K, std=0.02) if weight else _activations(g, R, K)
    kb, rb = -(-K // 128), -(-R // rows)
    s = torch.rand(kb, rb, generator=g, device=DEV) * 0.5 + 0.75
    s = s * ((4.5 * 0.02 if weight else 4.0) / 448.0)
    full = s.repeat_interleave(rows, 1)[:, :R].repeat_interleave(128, 0)[:K].t()
    q = (x / full).clamp_(-448.0, 448.0).to(E4M3)
    return q, s


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"case": case}
    if op == "quant":
        x = _normal(g, case["T"], case["K"], std=0.02) if case["rows"] == 128 else _activations(g, case["T"], case["K"])
        s["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "gemm":
        s["x"], s["xs"] = _operand(g, case["T"], case["K"], 1, False)
        s["w"], s["ws"] = _operand(g, case["N"], case["K"], 128, True)
    elif op == "gated":
        s["x"], s["xs"] = _operand(g, case["T"], case["K"], 1, False)
        s["wg"], s["gs"] = _operand(g, case["N"], case["K"], 128, True)
        s["wu"], s["us"] = _operand(g, case["N"], case["K"], 128, True)
    elif op == "norm":
        T, D = case["T"], case["D"]
        s["x"] = _activations(g, T, D).to(DTYPES[case["x"]])
        s["block"] = _normal(g, T, D, std=0.7).to(DTYPES[case["block"]])
        s["weight"] = (1.0 + _normal(g, D, std=0.1)).bfloat16()
        s["bias"] = _normal(g, D, std=0.1).bfloat16() if case["kind"] == "layer" else None
        s["post_weight"] = (1.0 + _normal(g, D, std=0.1)).bfloat16() if case["post"] != "none" else None
        s["post_bias"] = _normal(g, D, std=0.1).bfloat16() if case["post"] == "layer" else None
        shape = {"none": None, "channel": (D,), "token": (T, 1), "full": (T, D)}[case["gate"]]
        s["gate"] = _normal(g, *shape, std=0.5).bfloat16() if shape else None
    else:
        T, V = case["T"], case["V"]
        x = _normal(g, T, V, std=2.5)
        s["targets"] = torch.randint(0, V, (T,), generator=g, device=DEV)
        if case["masked"]:  # vocabulary entries that a grammar or padding shuts out
            x = x.masked_fill(torch.rand(T, V, generator=g, device=DEV) < 0.3, float("-inf"))
        s["x"] = x.to(DTYPES[case["dtype"]])
    return s


# ---- the plain forms ---------------------------------------------------------------------


def _blocks(x, rows):
    """x [R, K] in blocks: [ceil(R/rows), rows, ceil(K/128), 128], zeros in the padding."""
    R, K = x.shape
    kb, rb = -(-K // 128), -(-R // rows)
    p = x.new_zeros(rb * rows, kb * 128)
    p[:R, :K] = x
    return p.view(rb, rows, kb, 128)


def _quant(x, rows):
    R, K = x.shape
    b = _blocks(x.float(), rows)
    s = torch.clamp_min(b.abs().amax(dim=(1, 3)) / 448.0, 2.0 ** -126)
    r = 1.0 / s
    q = (b * r[:, None, :, None]).clamp_(-448.0, 448.0).to(E4M3)
    return q.view(q.shape[0] * rows, -1)[:R, :K].contiguous(), s.t().contiguous()


def _widen(q, s, rows):
    """The values an e4m3 operand stands for, in fp32."""
    b = _blocks(q.float(), rows)
    return (b * s.t()[:, None, :, None]).view(b.shape[0] * rows, -1)[:q.shape[0], :q.shape[1]]


def _act(g, name):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))
    return torch.clamp_min(g, 0.0)


def _norm(v, kind, weight, bias, eps=1e-6):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + eps) * weight.to(v.dtype)
    return v if bias is None else v + bias.to(v.dtype)


def _run_plain(s, case):
    op = case["op"]
    if op == "quant":
        return _quant(s["x"], case["rows"])
    if op == "gemm":
        return (_widen(s["x"], s["xs"], 1) @ _widen(s["w"], s["ws"], 128).t()).to(DTYPES[case["out"]])
    if op == "gated":
        x = _widen(s["x"], s["xs"], 1)
        h = _act(x @ _widen(s["wg"], s["gs"], 128).t(), case["act"]) * (x @ _widen(s["wu"], s["us"], 128).t())
        return _quant(h, 1) if case["out"] == "e4m3" else h.to(DTYPES[case["out"]])
    if op == "norm":
        z = _norm(s["block"].float(), case["post"], s["post_weight"], s["post_bias"])
        if s["gate"] is not None:
            z = z * s["gate"].float()
        r = s["x"].float() + 0.5 * z
        n = _norm(r, case["kind"], s["weight"], s["bias"])
        n = _quant(n, 1) if case["out"] == "e4m3" else n.to(DTYPES[case["out"]])
        return n, r.to(DTYPES[case["x"]])
    x = s["x"].float()
    m = x.amax(1, keepdim=True)
    d = (x - m) / 0.8
    e = torch.exp(d)
    S = e.sum(1, keepdim=True)
    log_s = torch.log(S)
    entropy = (log_s - (e * torch.clamp_min(d, -1e30)).sum(1, keepdim=True) / S)[:, 0]
    lp = d - log_s
    top = torch.sort(s["x"], dim=1, descending=True, stable=True)[1][:, :case["top"]]
    return lp.gather(1, s["targets"][:, None])[:, 0], entropy, lp.gather(1, top), top.to(torch.int32)


def _run_own(s, case):
    import token_adaptive_mixed_b200 as mobi
    op = case["op"]
    if op == "quant":
        return mobi.mobi_fp8_quant(s["x"], block_rows=case["rows"])
    if op == "gemm":
        return mobi.mobi_fp8_gemm(s["x"], s["xs"], s["w"], s["ws"], out_dtype=DTYPES[case["out"]])
    if op == "gated":
        return mobi.mobi_fp8_gated(s["x"], s["xs"], s["wg"], s["gs"], s["wu"], s["us"], act=case["act"],
                                   out_dtype=DTYPES[case["out"]])
    if op == "norm":
        return mobi.mobi_norm(s["x"], s["weight"], s["bias"], eps=1e-6, kind=case["kind"], block=s["block"],
                              post=case["post"], post_weight=s["post_weight"], post_bias=s["post_bias"],
                              gate=s["gate"], scale=0.5, out_dtype=DTYPES[case["out"]])
    return mobi.mobi_logprobs(s["x"], s["targets"], temperature=0.8, top_k=case["top"])


def run(state):
    return _run_own(state, state["case"]) if own else _run_plain(state, state["case"])


# ---- what a pass cannot do without ---------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "quant":
        n, kb, rb = case["T"] * case["K"], -(-case["K"] // 128), -(-case["T"] // case["rows"])
        return {"bytes": n * (SIZE[case["dtype"]] + 1) + 4 * kb * rb, "flops": 3 * n}
    if op in ("gemm", "gated"):
        T, N, K = case["T"], case["N"], case["K"]
        kb, nb, w = -(-K // 128), -(-N // 128), 2 if op == "gated" else 1
        out = T * N * SIZE[case["out"]] + (4 * T * nb if case["out"] == "e4m3" else 0)
        return {"bytes": T * K + w * N * K + 4 * kb * (T + w * nb) + out, "flops": 2 * w * T * N * K}
    if op == "norm":
        T, D = case["T"], case["D"]
        per = SIZE[case["block"]] + 2 * SIZE[case["x"]] + SIZE[case["out"]] + (2 if case["gate"] == "full" else 0)
        return {"bytes": T * D * per + (4 * T * -(-D // 128) if case["out"] == "e4m3" else 0), "flops": 12 * T * D}
    return {"bytes": case["T"] * case["V"] * SIZE[case["dtype"]] + case["T"] * (16 + 8 * case["top"]),
            "flops": 6 * case["T"] * case["V"]}


# ---- from the definitions, in 64 bits -------------------------------------------------------


def _grid(v):
    """v (float64) rounded to the nearest e4m3 value, ties to even, saturating at 448."""
    a = v.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 1).clamp(min=-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def _spread(s, R, K, rows):
    """Block scales [kb, rb] for each element of an [R, K] operand, in 64 bits."""
    i = torch.arange(R, device=s.device) // rows
    j = torch.arange(K, device=s.device) // 128
    return s.double()[j[None, :], i[:, None]]


def _quant64(x, rows):
    R, K = x.shape
    kb, rb = -(-K // 128), -(-R // rows)
    i = torch.arange(R, device=x.device) // rows
    j = torch.arange(K, device=x.device) // 128
    at = (j[None, :] * rb + i[:, None]).reshape(-1)
    a = torch.zeros(kb * rb, dtype=torch.float64, device=x.device).scatter_reduce(
        0, at, x.abs().reshape(-1), "amax", include_self=True)
    s = (a / 448.0).clamp(min=2.0 ** -126).view(kb, rb)
    return _grid(x / s.view(-1)[at].view(R, K)), s


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quant":
        return _quant64(s["x"].double(), case["rows"])
    if op in ("gemm", "gated"):
        T, N, K = case["T"], case["N"], case["K"]
        x = s["x"].double() * _spread(s["xs"], T, K, 1)
        if op == "gemm":
            return torch.matmul(x, (s["w"].double() * _spread(s["ws"], N, K, 128)).T)
        g = torch.matmul(x, (s["wg"].double() * _spread(s["gs"], N, K, 128)).T)
        u = torch.matmul(x, (s["wu"].double() * _spread(s["us"], N, K, 128)).T)
        a = {"silu": lambda v: v * torch.sigmoid(v), "relu": torch.relu,
             "gelu": lambda v: v * 0.5 * torch.erfc(-v / math.sqrt(2.0)),
             "gelu_tanh": lambda v: v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))}
        h = a[case["act"]](g) * u
        return _quant64(h, 1) if case["out"] == "e4m3" else h
    if op == "norm":
        def unit(v, kind, w, b):
            if kind == "none":
                return v
            mean = v.sum(1, keepdim=True) / v.shape[1] if kind == "layer" else torch.zeros_like(v[:, :1])
            var = ((v - mean) ** 2).sum(1, keepdim=True) / v.shape[1]
            out = (v - mean) / torch.sqrt(var + 1e-6) * w.double()
            return out + b.double() if b is not None else out
        z = unit(s["block"].double(), case["post"], s["post_weight"], s["post_bias"])
        r = s["x"].double() + 0.5 * (z if s["gate"] is None else s["gate"].double() * z)
        n = unit(r, case["kind"], s["weight"], s["bias"])
        return _quant64(n, 1) if case["out"] == "e4m3" else n, r
    x = s["x"].double() / 0.8
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    entropy = -torch.xlogy(p, p).sum(1)
    raw = s["x"].double()
    # Distinct sort keys: larger values first, the lower index first among equal ones.
    order = torch.argsort(-raw, dim=1, stable=True)[:, :case["top"]]
    at = torch.gather(x, 1, order) - lse[:, None]
    target = torch.gather(x, 1, s["targets"][:, None])[:, 0] - lse
    return target, entropy, at, order.to(torch.int32)
