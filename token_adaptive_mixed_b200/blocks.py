"""What a model runs around the mixed-bit layer: the 8-bit layer with a scale per
block of 128, the step between two blocks (norms, gate, residual) and the
scoring of logits. Bindings of the calls of the same names in include/mobi.h.

Unlike the mixed-bit calls these take row pitches, so a tensor may be a slice of
a larger one as long as its last dimension is contiguous, and they run on the
tensors' device, on that device's current stream. Tensors of one call live on
one device. Outputs are allocated unless given. With `stream` (a stream of that
device, or its handle) the whole call runs as under torch.cuda.stream(stream):
new outputs belong to that stream too, since memory that the current stream has
freed may still be in use by work queued there. The inputs are kept alive, and
ready, by the caller, as for any work queued on another stream.

They serve and have no backward pass: where gradients are recorded, a tensor that
requires one is refused, since its part of the gradient would be lost in silence.
Under torch.no_grad() or torch.inference_mode() it is taken as any other.
"""
from __future__ import annotations

import ctypes
import struct

import torch

E4M3 = torch.float8_e4m3fn
_F32 = torch.float32
_DT = {_F32: 0, torch.bfloat16: 1, torch.float16: 2, E4M3: 3}
_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
_NORM = {"none": 0, None: 0, "rms": 1, "layer": 2}

_raw_stream = torch._C._cuda_getCurrentRawStream
_get_device = torch._C._cuda_getDevice


class NormArgs(ctypes.Structure):
    """mobi_norm_args (include/mobi.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "block", "gate", "weight", "bias", "post_weight", "post_bias",
                                                "r_out", "n_out", "n_scale")]
                + [(n, ctypes.c_int64) for n in ("T", "D", "ldx", "ldb", "ldr", "ldn", "gate_st", "gate_sd")]
                + [(n, ctypes.c_int) for n in ("x_dtype", "block_dtype", "gate_dtype", "weight_dtype", "out_dtype",
                                               "post", "kind")]
                + [(n, ctypes.c_float) for n in ("eps", "post_eps", "scale")]
                + [("unit_offset", ctypes.c_int)])


# The same record packed in one step. struct pads between fields as C does, but not at the end of a record: "0P" does.
_NORM_ARGS = struct.Struct("".join({ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int: "i",
                                   ctypes.c_float: "f"}[t] for _, t in NormArgs._fields_) + "0P").pack

# The other calls' arguments as words of mobi_call_words: one foreign argument
# instead of 10 to 18, which ctypes converts at 0.1 us each.
_QUANT, _GEMM, _GATED, _LOGPROBS = range(4)
_WORDS = {_QUANT: struct.Struct("10q").pack, _GEMM: struct.Struct("13q").pack, _GATED: struct.Struct("18q").pack,
          _LOGPROBS: struct.Struct("6qf4x6q").pack}
_NAMES = ("mobi_fp8_quant", "mobi_fp8_gemm", "mobi_fp8_gated", "mobi_logprobs", "mobi_norm")

SYMBOLS = _NAMES + ("mobi_call_words", "mobi_debug_fp8_plan")


def bind(L: ctypes.CDLL) -> None:
    """Argument types of the calls of this module."""
    p, i64, ci, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.mobi_fp8_quant.argtypes = [p, ci, i64, i64, i64, ci, p, i64, p, p]
    L.mobi_fp8_gemm.argtypes = [p, i64, p, i64, i64, p, i64, p, i64, ci, p, i64, p]
    L.mobi_fp8_gated.argtypes = [p, i64, p, i64, i64, p, i64, p, p, i64, p, i64, ci, ci, p, i64, p, p]
    L.mobi_norm.argtypes = [p, p]
    L.mobi_logprobs.argtypes = [p, ci, i64, i64, i64, p, f32, ci, p, p, p, p, p]
    L.mobi_call_words.argtypes = [ci, p, ci]
    L.mobi_debug_fp8_plan.argtypes = [i64, i64, i64, ci, ci, p]
    for n in SYMBOLS:
        getattr(L, n).restype = ci


_lib: list = []


def _library() -> ctypes.CDLL:
    from . import lib
    _lib.append(lib())
    return _lib[0]


def _under(stream, t: torch.Tensor):
    """What makes `stream` the current one for a call on t's device."""
    _on(t, "the input")
    if not hasattr(stream, "cuda_stream"):
        h = int(stream)
        stream = torch.cuda.ExternalStream(h, device=t.device) if h else torch.cuda.default_stream(t.device)
    elif stream.device != t.device:
        raise ValueError("the stream is of another device")
    return torch.cuda.stream(stream)


def _call(call: int, device: int, *words) -> None:
    """Run a call of mobi_call_words on `device`, on its current stream."""
    w = _WORDS[call](*words, _raw_stream(device))
    L = _lib[0] if _lib else _library()
    if _get_device() == device:
        status = L.mobi_call_words(call, w, len(w) >> 3)
    else:
        with torch.cuda.device(device):
            status = L.mobi_call_words(call, w, len(w) >> 3)
    if status:
        from . import _check
        _check(_NAMES[call], status)


def _refuse_gradient(what: str) -> None:
    """For a tensor that requires a gradient."""
    if torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient and this call has no backward pass: call it under "
                         "torch.no_grad(), or detach the tensor")


def _matrix(t: torch.Tensor, what: str, device: int):
    """(rows, columns, row pitch) of a matrix on CUDA device `device` whose rows are contiguous."""
    if t.requires_grad:
        _refuse_gradient(what)
    if t.get_device() != device or device < 0:
        _on(t, what, device)
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D")
    (R, C), (ld, sd) = t.shape, t.stride()
    if sd != 1 and C > 1:
        raise ValueError(f"the rows of {what} must be contiguous")
    if ld < C:
        if R > 1:
            raise ValueError(f"the rows of {what} overlap")
        ld = C
    return R, C, ld or 1


def _on(t: torch.Tensor, what: str, device: int | None = None) -> None:
    if not t.is_cuda:
        raise ValueError("libmobi takes CUDA tensors only (no CPU path)")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{what} is on another device")


def _vector(t, n: int, what: str, device, dtype=None) -> int:
    """The address of a contiguous vector of n elements (None: 0)."""
    if t is None:
        return 0
    if t.requires_grad:
        _refuse_gradient(what)
    _on(t, what, device)
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous vector of {n} elements")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype}")
    return t.data_ptr()


def _scales(s: torch.Tensor, kb: int, rb: int, what: str, device: int) -> int:
    if s.requires_grad:
        _refuse_gradient(f"the scale tensor {what}")
    if s.get_device() != device:
        _on(s, f"the scale tensor {what}", device)
    if s.dtype is not _F32 or s.shape != (kb, rb) or not s.is_contiguous():
        raise ValueError(f"the scale tensor {what} must be contiguous fp32 of shape ({kb}, {rb})")
    return s.data_ptr()


def _out(t, T: int, N: int, dtype, what, device, dev):
    """(output, its row pitch): a given one checked, or a new one. Rows of a new e4m3 output start at multiples of
    16 bytes, as the products take them. (Sizes are passed to torch.empty one by one: a tuple costs another 0.7 us.)"""
    if t is None:
        if dtype is E4M3 and N & 15:
            ld = (N + 15) & ~15
            return torch.empty(T, ld, dtype=E4M3, device=dev)[:, :N], ld
        return torch.empty(T, N, dtype=dtype, device=dev), N
    if t.dtype is not dtype or t.dim() != 2 or t.shape[0] != T or t.shape[1] != N:
        raise ValueError(f"{what} must be {dtype} of shape ({T}, {N})")
    return t, _matrix(t, what, device)[2]


def _new_scales(t, kb: int, rb: int, what, device, dev):
    """(scales, their address): given ones checked, or new ones."""
    if t is None:
        t = torch.empty(kb, rb, dtype=_F32, device=dev)
        return t, t.data_ptr()
    return t, _scales(t, kb, rb, what, device)


def mobi_fp8_quant(X: torch.Tensor, block_rows: int = 1, Q: torch.Tensor | None = None,
                   scale: torch.Tensor | None = None, stream=None):
    """X [T, K] (fp32, bf16 or fp16) in blocks of 1 x 128 (activations) or 128 x 128 (block_rows=128, weights)
    -> (Q e4m3 [T, K], scale fp32 [ceil(K/128), ceil(T/block_rows)]); Q * scale stands for X."""
    if stream is not None:
        with _under(stream, X):
            return mobi_fp8_quant(X, block_rows, Q, scale)
    d = X.get_device()
    T, K, ldx = _matrix(X, "X", d)
    dt = _DT.get(X.dtype, 3)
    if dt == 3:
        raise ValueError("X must be fp32, bf16 or fp16")
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    dev = X.device
    kb, rb = (K + 127) >> 7, T if block_rows == 1 else (T + 127) >> 7
    Q, ldq = _out(Q, T, K, E4M3, "Q", d, dev)
    scale, sp = _new_scales(scale, kb, rb, "scale", d, dev)
    _call(_QUANT, d, X.data_ptr(), dt, T, K, ldx, block_rows, Q.data_ptr(), ldq, sp)
    return Q, scale


def _operand(Q, scale, what, scale_name, rows, K, device):
    """(rows, columns, pitch, codes address, scales address) of an e4m3 operand; rows per scale `rows`."""
    if Q.dtype is not E4M3:
        raise ValueError(f"{what} must be e4m3")
    R, k, ld = _matrix(Q, what, device)
    if K is not None and k != K:
        raise ValueError(f"{what} has {k} columns, X has {K}")
    if R <= 1:
        ld = (ld + 15) & ~15  # one row: the pitch is never used
    return R, k, ld, Q.data_ptr(), _scales(scale, (k + 127) >> 7, (R + rows - 1) // rows, scale_name, device)


def mobi_fp8_gemm(X: torch.Tensor, xs: torch.Tensor, W: torch.Tensor, ws: torch.Tensor, out_dtype=torch.float32,
                  Y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The 8-bit layer Y = X W^T: X e4m3 [T, K] with xs (block_rows=1), W e4m3 [N, K] with ws (block_rows=128)
    -> Y [T, N] in out_dtype (fp32, bf16 or fp16)."""
    if stream is not None:
        with _under(stream, X):
            return mobi_fp8_gemm(X, xs, W, ws, out_dtype, Y)
    d = X.get_device()
    T, K, ldx, xp, xsp = _operand(X, xs, "X", "xs", 1, None, d)
    N, _, ldw, wp, wsp = _operand(W, ws, "W", "ws", 128, K, d)
    dt = _DT.get(out_dtype, 3)
    if dt == 3:
        raise ValueError("out_dtype must be fp32, bf16 or fp16")
    Y, ldy = _out(Y, T, N, out_dtype, "Y", d, X.device)
    _call(_GEMM, d, xp, ldx, xsp, T, K, wp, ldw, wsp, N, dt, Y.data_ptr(), ldy)
    return Y


def mobi_fp8_gated(X: torch.Tensor, xs: torch.Tensor, Wg: torch.Tensor, gs: torch.Tensor, Wu: torch.Tensor,
                   us: torch.Tensor, act: str = "silu", out_dtype=torch.bfloat16, H: torch.Tensor | None = None,
                   hs: torch.Tensor | None = None, stream=None):
    """act(X Wg^T) * (X Wu^T) in one kernel, operands as mobi_fp8_gemm; act "silu", "gelu", "gelu_tanh" or "relu".
    -> H [T, N] in out_dtype, or (H e4m3, hs fp32 [ceil(N/128), T]) for out_dtype torch.float8_e4m3fn."""
    if stream is not None:
        with _under(stream, X):
            return mobi_fp8_gated(X, xs, Wg, gs, Wu, us, act, out_dtype, H, hs)
    d, dev = X.get_device(), X.device
    T, K, ldx, xp, xsp = _operand(X, xs, "X", "xs", 1, None, d)
    N, _, ldg, gp, gsp = _operand(Wg, gs, "Wg", "gs", 128, K, d)
    Nu, _, ldu, up, usp = _operand(Wu, us, "Wu", "us", 128, K, d)
    if Nu != N:
        raise ValueError("Wg and Wu must have as many rows")
    if act not in _ACT:
        raise ValueError(f"act must be one of {sorted(_ACT)}")
    dt = _DT.get(out_dtype)
    if dt is None:
        raise ValueError("out_dtype must be fp32, bf16, fp16 or e4m3")
    H, ldh = _out(H, T, N, out_dtype, "H", d, dev)
    hsp = 0
    if dt == 3:
        hs, hsp = _new_scales(hs, (N + 127) >> 7, T, "hs", d, dev)
    _call(_GATED, d, xp, ldx, xsp, T, K, gp, ldg, gsp, up, ldu, usp, N, _ACT[act], dt, H.data_ptr(), ldh, hsp)
    return (H, hs) if dt == 3 else H


def mobi_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
              eps: float = 1e-6, kind: str = "rms", block: torch.Tensor | None = None, post: str = "none",
              post_weight: torch.Tensor | None = None, post_bias: torch.Tensor | None = None,
              post_eps: float | None = None, gate: torch.Tensor | None = None, scale: float = 1.0,
              unit_offset: bool = False, out_dtype=torch.bfloat16, N: torch.Tensor | None = None,
              n_scale: torch.Tensor | None = None, R: torch.Tensor | None = None, stream=None):
    """The step between two blocks in one pass: r = x + scale * gate * post(block), n = kind(r) * weight + bias.

    x [T, D] is the residual stream, block [T, D] the block's output (None: a plain norm of x), gate anything that
    broadcasts to [T, D]; kind and post are "rms", "layer" or "none". -> (n, r), or n alone without a block; n is
    a pair (codes, scales) for out_dtype torch.float8_e4m3fn. R=x updates the residual stream in place."""
    if stream is not None:
        with _under(stream, x):
            return mobi_norm(x, weight, bias, eps, kind, block, post, post_weight, post_bias, post_eps, gate, scale,
                             unit_offset, out_dtype, N, n_scale, R)
    d, dev = x.get_device(), x.device
    T, D, ldx = _matrix(x, "x", d)
    xdt, odt = _DT.get(x.dtype, 3), _DT.get(out_dtype)
    if xdt == 3 or odt is None:
        raise ValueError("x must be fp32, bf16 or fp16, out_dtype one of these or e4m3")
    if kind not in _NORM or post not in _NORM:
        raise ValueError('kind and post must be "rms", "layer" or "none"')
    wdt = None
    for w in (weight, bias, post_weight, post_bias):
        if w is not None:
            if wdt is not None and w.dtype is not wdt:
                raise ValueError("the weights and biases must have one type")
            wdt = w.dtype
    wdt = 0 if wdt is None else _DT.get(wdt, 3)
    if wdt == 3:
        raise ValueError("the weights and biases must be fp32, bf16 or fp16")
    wp, bp = _vector(weight, D, "weight", d), _vector(bias, D, "bias", d)
    block_p = gate_p = pwp = pbp = rp = nsp = 0
    ldb = ldr = gate_st = gate_sd = bdt = gdt = 0
    if block is not None:
        if block.shape != x.shape:
            raise ValueError("block must have the shape of x")
        ldb = _matrix(block, "block", d)[2]
        block_p, bdt = block.data_ptr(), _DT.get(block.dtype, 3)
        if bdt == 3:
            raise ValueError("block must be fp32, bf16 or fp16")
        pwp, pbp = _vector(post_weight, D, "post_weight", d), _vector(post_bias, D, "post_bias", d)
        if gate is not None:
            if gate.requires_grad:
                _refuse_gradient("gate")
            _on(gate, "gate", d)
            gdt = _DT.get(gate.dtype, 3)
            if gdt == 3:
                raise ValueError("gate must be fp32, bf16 or fp16")
            gate_st, gate_sd = gate.expand(T, D).stride()
            gate_p = gate.data_ptr()
        R, ldr = _out(R, T, D, x.dtype, "R", d, dev)
        rp = R.data_ptr()
    elif R is not None or gate is not None or post_weight is not None or post_bias is not None:
        raise ValueError("R, gate and the post norm's weights need a block")
    N, ldn = _out(N, T, D, out_dtype, "N", d, dev)
    if odt == 3:
        n_scale, nsp = _new_scales(n_scale, (D + 127) >> 7, T, "n_scale", d, dev)
    a = _NORM_ARGS(x.data_ptr(), block_p, gate_p, wp, bp, pwp, pbp, rp, N.data_ptr(), nsp, T, D, ldx, ldb, ldr, ldn,
                   gate_st, gate_sd, xdt, bdt, gdt, wdt, odt, _NORM[post], _NORM[kind], eps,
                   eps if post_eps is None else post_eps, scale, unit_offset)
    L = _lib[0] if _lib else _library()
    if _get_device() == d:
        status = L.mobi_norm(a, _raw_stream(d))
    else:
        with torch.cuda.device(d):
            status = L.mobi_norm(a, _raw_stream(d))
    if status:
        from . import _check
        _check("mobi_norm", status)
    n = (N, n_scale) if odt == 3 else N
    return n if block is None else (n, R)


def mobi_logprobs(logits: torch.Tensor, targets: torch.Tensor | None = None, temperature: float = 1.0,
                  top_k: int = 0, entropy: bool = True, stream=None):
    """Scoring of logits [T, V] (fp32, bf16 or fp16) -> (logprob [T] of the int64 targets, entropy [T],
    top_logprob [T, top_k], top_index int32 [T, top_k]); logprob is None without targets, entropy without
    entropy=True. A negative target is ignored (log probability 0); one >= V is reported by mobi_sync_check."""
    if stream is not None:
        with _under(stream, logits):
            return mobi_logprobs(logits, targets, temperature, top_k, entropy)
    d, dev = logits.get_device(), logits.device
    T, V, ld = _matrix(logits, "logits", d)
    dt = _DT.get(logits.dtype, 3)
    if dt == 3:
        raise ValueError("logits must be fp32, bf16 or fp16")
    tp = _vector(targets, T, "targets", d, torch.int64)
    k = int(top_k)
    lp = None if targets is None else torch.empty(T, dtype=_F32, device=dev)
    en = torch.empty(T, dtype=_F32, device=dev) if entropy else None
    top = torch.empty(T, max(k, 0), dtype=_F32, device=dev)
    idx = torch.empty(T, max(k, 0), dtype=torch.int32, device=dev)
    _call(_LOGPROBS, d, logits.data_ptr(), dt, T, V, ld, tp, temperature, k, 0 if lp is None else lp.data_ptr(),
          0 if en is None else en.data_ptr(), top.data_ptr(), idx.data_ptr())
    return lp, en, top, idx
