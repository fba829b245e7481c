"""CPU checks of the 8-bit layer, the norm between blocks and the scoring of
logits: every refusal happens on the host, before a launch."""
import ctypes

import pytest
import torch

import token_adaptive_mixed_b200 as mobi
from token_adaptive_mixed_b200 import blocks
from token_adaptive_mixed_b200 import build as mobi_build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    mobi_build.build()
    return mobi.lib()


def test_quant_refusals(L):
    def call(X=FAKE, dt=1, T=8, K=256, ldx=256, rows=1, Q=FAKE, ldq=256, s=FAKE):
        return L.mobi_fp8_quant(X, dt, T, K, ldx, rows, Q, ldq, s, None)
    assert call(T=0) == 0 and call(K=0) == 0
    assert call(T=-1) == 1 and call(K=-1) == 1
    assert call(dt=3) == 1 and call(dt=-1) == 1
    assert call(rows=64) == 1
    assert call(X=None) == 1 and call(Q=None) == 1 and call(s=None) == 1
    assert call(ldx=255) == 1 and call(ldq=255) == 1
    assert call(X=FAKE + 1) == 3 and call(dt=0, X=FAKE + 2) == 3 and call(s=FAKE + 2) == 3
    assert call(T=1 << 29) == 2 and call(K=1 << 24, ldx=1 << 24, ldq=1 << 24) == 2
    assert call(T=1 << 28, K=1 << 28, ldx=1 << 28, ldq=1 << 28, rows=128) == 2


def test_gemm_refusals(L):
    def call(X=FAKE, ldx=256, xs=FAKE, T=8, K=256, W=FAKE, ldw=256, ws=FAKE, N=64, dt=0, Y=FAKE, ldy=64):
        return L.mobi_fp8_gemm(X, ldx, xs, T, K, W, ldw, ws, N, dt, Y, ldy, None)
    assert call(T=0) == 0 and call(N=0) == 0
    assert call(T=-1) == 1 and call(N=-1) == 1 and call(K=-1) == 1
    assert call(K=0) == 2 and call(T=1 << 29) == 2
    assert call(dt=3) == 1 and call(dt=4) == 1
    for k in ("X", "xs", "W", "ws", "Y"):
        assert call(**{k: None}) == 1, k
    assert call(ldx=240) == 1 and call(ldw=240) == 1 and call(ldy=63) == 1
    assert call(X=FAKE + 8) == 3 and call(W=FAKE + 8) == 3 and call(ldx=264) == 3 and call(ldw=264) == 3
    assert call(xs=FAKE + 2) == 3 and call(Y=FAKE + 2) == 3 and call(dt=1, Y=FAKE + 1) == 3


def test_gated_refusals(L):
    def call(X=FAKE, xs=FAKE, T=8, K=256, Wg=FAKE, gs=FAKE, Wu=FAKE, us=FAKE, N=64, act=0, dt=1, H=FAKE, ldh=64,
             hs=FAKE, ldu=256):
        return L.mobi_fp8_gated(X, 256, xs, T, K, Wg, 256, gs, Wu, ldu, us, N, act, dt, H, ldh, hs, None)
    assert call(T=0) == 0 and call(N=0) == 0
    assert call(act=4) == 1 and call(act=-1) == 1 and call(dt=4) == 1 and call(dt=-1) == 1
    for k in ("X", "xs", "Wg", "gs", "Wu", "us", "H"):
        assert call(**{k: None}) == 1, k
    assert call(dt=3, hs=None) == 1 and call(dt=3, hs=FAKE + 2) == 3
    assert call(ldu=250) == 1 and call(Wu=FAKE + 4) == 3 and call(ldh=63) == 1


def test_norm_refusals(L):
    def call(**kw):
        a = blocks.NormArgs()
        d = dict(x=FAKE, n_out=FAKE, T=4, D=64, ldx=64, ldn=64, kind=1, eps=1e-6, x_dtype=1, out_dtype=1)
        for k, v in {**d, **kw}.items():
            setattr(a, k, v)
        return L.mobi_norm(ctypes.addressof(a), None)
    blk = dict(block=FAKE, ldb=64, block_dtype=0, scale=1.0, post_eps=1e-6)
    assert L.mobi_norm(None, None) == 1
    assert call(T=0) == 0 and call(T=0, **blk) == 0
    assert call(T=-1) == 1 and call(D=0) == 1 and call(D=16385, ldx=16385, ldn=16385) == 2 and call(T=1 << 29) == 2
    assert call(x=None) == 1 and call(n_out=None) == 1 and call(out_dtype=3) == 1  # no scales
    assert call(x_dtype=3) == 1 and call(out_dtype=4) == 1 and call(kind=3) == 1 and call(kind=-1) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(ldx=63) == 1 and call(ldn=63) == 1
    assert call(weight=FAKE, weight_dtype=3) == 1
    assert call(**{**blk, "ldb": 63}) == 1 and call(**{**blk, "block_dtype": 3}) == 1
    assert call(**{**blk, "scale": float("nan")}) == 1 and call(**{**blk, "post_eps": -1.0}) == 1
    assert call(gate=FAKE, gate_dtype=3, **blk) == 1 and call(post=3, **blk) == 1
    assert call(r_out=FAKE, ldr=63, **blk) == 1
    assert call(r_out=FAKE, ldr=72, ldx=64, **blk) == 1  # in place with another pitch
    assert call(x=FAKE + 1) == 3 and call(weight=FAKE + 1, weight_dtype=1) == 3 and call(n_out=FAKE + 1) == 3
    assert call(gate=FAKE + 2, gate_dtype=0, **blk) == 3 and call(r_out=FAKE + 1, ldr=64, **blk) == 3


def test_logprobs_refusals(L):
    def call(x=FAKE, dt=0, T=4, V=100, ld=100, tg=FAKE, temp=1.0, k=5, lp=FAKE, en=FAKE, tl=FAKE, ti=FAKE):
        return L.mobi_logprobs(x, dt, T, V, ld, tg, temp, k, lp, en, tl, ti, None)
    assert call(T=0) == 0
    assert call(T=-1) == 1 and call(V=0) == 1 and call(dt=3) == 1 and call(k=-1) == 1 and call(k=33) == 1
    assert call(V=1 << 29, ld=1 << 29) == 2
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e-31):
        assert call(temp=t) == 1, t
    assert call(x=None) == 1 and call(ld=99) == 1 and call(lp=None) == 1
    assert call(tl=None) == 1 and call(ti=None) == 1
    assert call(x=FAKE + 2) == 3 and call(dt=1, x=FAKE + 1) == 3 and call(tg=FAKE + 4) == 3 and call(ti=FAKE + 2) == 3


def test_binding_takes_cuda_tensors_only():
    x = torch.zeros(4, 128)
    q, s = x.to(torch.float8_e4m3fn), torch.ones(1, 4)
    for f in (lambda: mobi.mobi_fp8_quant(x), lambda: mobi.mobi_fp8_gemm(q, s, q, s),
              lambda: mobi.mobi_fp8_gated(q, s, q, s, q, s), lambda: mobi.mobi_norm(x),
              lambda: mobi.mobi_logprobs(x), lambda: mobi.mobi_fp8_quant(x, stream=0),
              lambda: mobi.mobi_norm(x, stream=0)):
        with pytest.raises(ValueError):
            f()


def test_reference_quantiser():
    """The tests' own quantiser against hand-made values: the scale, ties to even, the floor of the scale, a NaN."""
    import block_ref as ref
    x = torch.zeros(2, 128)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 448.0, 17.0, 19.0, -0.0009765625  # 17: between 16 and 18; 2^-10: half of 2^-9
    x[1, 5] = float("nan")
    q, s = ref.quant(x, 1)
    assert s[0, 0] == 1.0 and torch.isnan(s[0, 1])
    assert q[0, :4].float().tolist() == [448.0, 16.0, 20.0, 0.0]
    assert torch.isnan(q[1].float()).all()
    q, s = ref.quant(torch.zeros(1, 5), 1)
    assert s[0, 0] == 2.0 ** -126 and (q.float() == 0).all()


def test_reference_logprobs():
    """The tests' own scoring against torch's."""
    import block_ref as ref
    g = torch.Generator().manual_seed(0)
    x = torch.randn(3, 50, generator=g) * 3
    x[1, 7] = float("-inf")
    t = torch.tensor([4, 7, -1])
    lp, H, top, idx, _, _ = ref.logprobs(x, t, 0.7, 4)
    want = torch.log_softmax(x.double() / 0.7, 1)
    assert torch.allclose(lp[:1], want[:1, 4]) and lp[1] == float("-inf") and lp[2] == 0
    p = want.exp()
    assert torch.allclose(H, -torch.xlogy(p, p).sum(1))
    assert torch.equal(idx, x.topk(4, 1)[1])
    assert torch.allclose(top, want.gather(1, idx))


def test_words_refusals(L):
    """mobi_call_words: the number of words, the call, ints that do not fit; the rest is refused by the call itself."""
    import struct
    q = [0x1000, 1, 4, 128, 128, 1, 0x2000, 128, 0x3000, 0]
    call = lambda c, w, n=None: L.mobi_call_words(c, struct.pack(f"{len(w)}q", *w), len(w) if n is None else n)  # noqa: E731
    assert L.mobi_call_words(0, None, 10) == 1
    assert call(-1, q) == 1 and call(4, q) == 1 and call(0, q, 9) == 1 and call(1, q) == 1 and call(3, q) == 1
    for i in (1, 5):
        assert call(0, q[:i] + [q[i] + (1 << 32)] + q[i + 1:]) == 1
    assert call(0, q[:5] + [64] + q[6:]) == 1 and call(0, q[:8] + [0x3001, 0]) == L.mobi_fp8_quant(
        0x1000, 1, 4, 128, 128, 1, 0x2000, 128, 0x3001, None)
    assert call(0, [0, 0, 0, 128, 128, 1, 0, 128, 0, 0]) == 0 and call(1, [0] * 13) == 0 and call(2, [0] * 18) == 0
    temp = struct.unpack("q", struct.pack("f4x", 1.0))[0]
    assert call(3, [0, 0, 0, 5, 5, 0, temp, 0, 0, 0, 0, 0, 0]) == 0 and call(3, [0, 0, 0, 5, 5] + [0] * 8) == 1


def test_packed_records_have_their_size():
    """What the binding hands over in place of arguments is as long as what the C side reads, and says the same."""
    names = [n for n, _ in blocks.NormArgs._fields_]
    values = [i + 1 for i in range(len(names))]
    record = blocks._NORM_ARGS(*values)
    assert len(record) == ctypes.sizeof(blocks.NormArgs)
    a = blocks.NormArgs.from_buffer_copy(record)
    assert [getattr(a, n) for n in names] == values
    for call, n in ((blocks._QUANT, 10), (blocks._GEMM, 13), (blocks._GATED, 18), (blocks._LOGPROBS, 13)):
        assert len(blocks._WORDS[call](*range(n))) == 8 * n


def _plan(L, T, N, K, gated, sms=148):
    p = (ctypes.c_int64 * 5)()
    assert L.mobi_debug_fp8_plan(T, N, K, gated, sms, p) == 0
    return tuple(p)


def test_plan_refusals(L):
    p = (ctypes.c_int64 * 5)()
    call = lambda T=4, N=4, K=4, g=0, sms=148, q=p: L.mobi_debug_fp8_plan(T, N, K, g, sms, q)  # noqa: E731
    assert call() == 0
    assert call(T=0) == 1 and call(N=0) == 1 and call(K=0) == 1 and call(g=2) == 1 and call(sms=1) == 1
    assert call(q=None) == 1 and call(T=1 << 29) == 2


@pytest.mark.parametrize("gated", [0, 1])
def test_every_plan_has_a_gpu_test(L, gated):
    """Whatever kernel, tile and cluster a size can be given, a size of the GPU tests is given it too, and the wide
    kernel's tests have pairs that take three tiles in a row or more."""
    import test_gpu_blocks as gpu
    tested = {_plan(L, *s, gated)[:3] for s in (gpu.PLANS_GATED if gated else gpu.PLANS)}
    steps = lambda top: sorted({round(2 ** (i / 4)) for i in range(4 * top)})  # noqa: E731
    reached = {_plan(L, T, N, K, gated)[:3] for T in steps(13) for N in steps(15) for K in steps(14)}
    assert reached <= tested, reached - tested
    most = {}
    for s in gpu.PLANS_GATED if gated else gpu.PLANS:
        p = _plan(L, *s, gated)
        most[p[:2]] = max(most.get(p[:2], 0), p[4])
    assert all(most[w] >= 3 for w in ([(1, 256)] if gated else [(1, 128), (1, 256)])), most


def test_plan_covers_the_output(L):
    """Tiles times their size reach every output, and the cluster divides no K below one block for each CTA."""
    for gated in (0, 1):
        for T in (1, 17, 64, 129, 333, 5000):
            for N in (1, 128, 4099, 28672):
                for K in (1, 300, 4096):
                    wide, cols, share, tiles, row = _plan(L, T, N, K, gated)
                    tt, tn = (256, 128 if gated else cols) if wide else (cols, 128)
                    assert tiles == -(-T // tt) * -(-N // tn)
                    assert row == (-(-tiles // 74) if wide else 1)
                    assert share == 2 if wide else 1 <= share <= max(1, -(-K // 128) // 2)


def test_gradients_are_refused():
    """No call has a backward pass: a tensor that requires a gradient is refused where gradients are recorded (before
    anything else is looked at, so also here), and taken under no_grad (here: refused as a CPU tensor)."""
    x = torch.zeros(4, 128, requires_grad=True)
    q, s = torch.zeros(4, 128).to(torch.float8_e4m3fn), torch.ones(1, 4, requires_grad=True)
    for f in (lambda: mobi.mobi_fp8_quant(x), lambda: mobi.mobi_norm(x), lambda: mobi.mobi_logprobs(x),
              lambda: blocks._vector(x[0], 128, "weight", 0), lambda: blocks._scales(s, 1, 4, "xs", 0),
              lambda: blocks._out(x, 4, 128, torch.float32, "Y", 0, x.device)):
        with pytest.raises(ValueError, match="requires a gradient"):
            f()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensors only"):
            f()
