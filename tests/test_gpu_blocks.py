"""The 8-bit layer, the norm between blocks and the scoring of logits against
their plain 64-bit forms (block_ref.py has the forms and the bounds)."""
import math

import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def mobi():
    import token_adaptive_mixed_b200 as m
    from token_adaptive_mixed_b200 import build
    build.build()
    m.lib()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def same_codes(q, want):
    return torch.equal(q.contiguous().view(torch.uint8).cpu(), want.contiguous().view(torch.uint8))


# ---- quantiser: bit-exact ---------------------------------------------------------------


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("T,K", [(1, 128), (1, 1), (3, 100), (17, 512), (130, 300), (257, 1037), (128, 4096)])
def test_quant(mobi, T, K, rows, dtype):
    g = gen(T * 10007 + K)
    x = (torch.randn(T, K, generator=g) * torch.exp(torch.randn(T, 1, generator=g) * 3)).clamp(-6e4, 6e4).to(dtype)
    q, s = mobi.mobi_fp8_quant(x.to(DEV), block_rows=rows)
    wq, ws = ref.quant(x, rows)
    assert torch.equal(s.cpu(), ws) and same_codes(q, wq)


@pytest.mark.parametrize("rows", [1, 128])
def test_quant_edges(mobi, rows):
    """Zero blocks, the scale's floor, the largest values, infinities and NaN; rows that are a slice of others."""
    x = torch.randn(256, 640, generator=gen(1))
    x[:, :128] = 0
    x[:128, 128:256] *= 1e-42
    x[3, 256] = float("nan")
    x[200, 300] = float("inf")
    x[:, 400] = 3.4e38
    x[5, 639] = -0.0
    q, s = mobi.mobi_fp8_quant(x.to(DEV), block_rows=rows)
    wq, ws = ref.quant(x, rows)
    assert torch.equal(s.cpu().view(torch.int32)[~torch.isnan(ws)], ws.view(torch.int32)[~torch.isnan(ws)])
    assert torch.equal(torch.isnan(s.cpu()), torch.isnan(ws))
    a, b = q.float().cpu(), wq.float()
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a[~torch.isnan(b)], b[~torch.isnan(b)])
    big = x.to(DEV)
    for part in (big[:, 3:500], big[1:, 8:], big[::3, 16:400]):
        q, s = mobi.mobi_fp8_quant(part, block_rows=rows)
        wq, ws = ref.quant(part.cpu(), rows)
        assert torch.equal(torch.nan_to_num(s.cpu()), torch.nan_to_num(ws))
        assert torch.equal(torch.nan_to_num(q.float().cpu()), torch.nan_to_num(wq.float()))


# ---- products -------------------------------------------------------------------------------

# Both kernels, one block of K to eight CTAs, ragged K, odd N and T (every kernel, tile and cluster: PLANS below).
GEMM = [(1, 128, 128), (1, 1, 16), (1, 4096, 4096), (2, 300, 1000), (16, 129, 2048), (17, 640, 272), (32, 77, 1536),
        (33, 500, 640), (64, 1024, 512), (65, 200, 128), (128, 257, 1040), (129, 384, 3200), (200, 4096, 1024),
        (256, 256, 128), (333, 4099, 512), (1000, 1500, 384), (2049, 513, 272), (37, 9000, 144), (100, 16, 8192)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,N,K", GEMM)
def test_gemm(mobi, T, N, K, dtype):
    g = gen(T + 1009 * N + K)
    x, xs = ref.operand(T, K, 1, g, device=DEV)
    w, ws = ref.operand(N, K, 128, g, 0.02, device=DEV)
    x, w = _pitched(x), _pitched(w)
    buf = torch.full((T + 2, N + 8), 7.0, dtype=dtype, device=DEV)
    y = mobi.mobi_fp8_gemm(x, xs, w, ws, out_dtype=dtype, Y=buf[1:T + 1, 3:N + 3])
    mobi.mobi_sync_check()
    want, err = ref.product(x, xs, w, ws)
    ref.check_close(y, want, ref.rounded(want, err, dtype), f"{T}x{N}x{K}")
    buf[1:T + 1, 3:N + 3] = 7.0
    assert (buf == 7.0).all(), "written outside Y"


def _pitched(q):
    """The same codes with rows 16 bytes apart or more (K need not be a multiple of 16)."""
    R, K = q.shape
    p = torch.empty((R, (K + 15) // 16 * 16 + 16), dtype=E4M3, device=q.device)
    p.view(torch.uint8).fill_(0x7f)  # NaN codes beside the rows: they must not be read as values
    p[:, :K] = q
    return p[:, :K]


@pytest.mark.parametrize("K", [1, 15, 129, 250])
def test_gemm_any_k(mobi, K):
    for T, N in ((5, 40), (300, 300)):
        g = gen(K)
        x, xs = ref.operand(T, K, 1, g, device=DEV)
        w, ws = ref.operand(N, K, 128, g, device=DEV)
        x, w = _pitched(x), _pitched(w)
        want, err = ref.product(x, xs, w, ws)
        ref.check_close(mobi.mobi_fp8_gemm(x, xs, w, ws), want, ref.rounded(want, err, F32))


@pytest.mark.parametrize("T", [3, 700])
def test_gemm_single_blocks(mobi, T):
    """One block at a time has to count, with its own scales: the others' codes are zero."""
    N, K = 384, 640
    g = gen(T)
    x, xs = ref.operand(T, K, 1, g, device=DEV)
    w, ws = ref.operand(N, K, 128, g, device=DEV)
    for b in range(5):
        xb = torch.zeros_like(x)
        xb[:, 128 * b:128 * b + 128] = x[:, 128 * b:128 * b + 128]
        want, err = ref.product(xb, xs, w, ws)
        assert want.abs().max() > 0
        ref.check_close(mobi.mobi_fp8_gemm(xb, xs, w, ws), want, ref.rounded(want, err, F32))


@pytest.mark.parametrize("T", [9, 400])
def test_gemm_nan_stays_in_its_row(mobi, T):
    N, K = 300, 512
    g = gen(5)
    x = torch.randn(T, K, generator=g)
    x[2, 200] = float("nan")
    x[4, 10] = float("inf")
    q, s = mobi.mobi_fp8_quant(x.to(DEV))
    w, ws = ref.operand(N, K, 128, g, device=DEV)
    y = mobi.mobi_fp8_gemm(q, s, w, ws)
    bad = torch.zeros(T, dtype=torch.bool)
    bad[2] = bad[4] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()
    h, hs = mobi.mobi_fp8_gated(q, s, w, ws, w, ws, out_dtype=E4M3)
    assert torch.isnan(h.float()[bad]).all() and torch.isfinite(h.float()[~bad]).all()
    assert torch.isnan(hs[:, bad]).all() and torch.isfinite(hs[:, ~bad]).all()


GATED = [(1, 128, 128), (1, 16, 48), (7, 144, 272), (8, 2048, 1024), (16, 100, 2048), (20, 640, 512), (32, 1000, 272),
         (33, 300, 640), (64, 200, 1024), (130, 129, 256), (200, 4096, 512), (300, 1000, 400), (1030, 700, 256)]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("T,N,K", GATED)
def test_gated(mobi, T, N, K, act):
    g = gen(T + 7 * N + K)
    x, xs = ref.operand(T, K, 1, g, device=DEV)
    wg, gs = ref.operand(N, K, 128, g, 0.05, device=DEV)
    wu, us = ref.operand(N, K, 128, g, 0.05, device=DEV)
    h, err = ref.gated(x, xs, wg, gs, wu, us, act)
    for dtype in (F32, BF16, F16):
        y = mobi.mobi_fp8_gated(x, xs, wg, gs, wu, us, act=act, out_dtype=dtype)
        ref.check_close(y, h, ref.rounded(h, err, dtype), f"{dtype}")
    buf = torch.full((T + 2, (N + 15) // 16 * 16 + 16), 3.0, device=DEV).to(E4M3)
    q, s = mobi.mobi_fp8_gated(x, xs, wg, gs, wu, us, act=act, out_dtype=E4M3, H=buf[1:T + 1, :N])
    mobi.mobi_sync_check()
    ref.check_quantised(q, s, h, err)
    buf.view(torch.uint8)[1:T + 1, :N] = torch.full((1,), 3.0).to(E4M3).view(torch.uint8).to(DEV)
    assert (buf.float() == 3.0).all(), "written outside H"


def test_products_do_not_depend_on_timing(mobi):
    """The same call gives the same bits, alone and beside another on a second stream."""
    g = gen(3)
    x, xs = ref.operand(48, 4096, 1, g, device=DEV)
    w, ws = ref.operand(2000, 4096, 128, g, device=DEV)
    u, us = ref.operand(2000, 4096, 128, g, device=DEV)
    first = mobi.mobi_fp8_gemm(x, xs, w, ws)
    gat = mobi.mobi_fp8_gated(x, xs, w, ws, u, us)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(10):
        with torch.cuda.stream(a):
            y = mobi.mobi_fp8_gemm(x, xs, w, ws)
        h = mobi.mobi_fp8_gated(x, xs, w, ws, u, us, stream=b)
        outs.append((y, h))
    torch.cuda.synchronize()
    mobi.mobi_sync_check()
    assert all(torch.equal(y, first) and torch.equal(h, gat) for y, h in outs)


@pytest.mark.parametrize("T", [8, 64, 600])
def test_product_timeout_is_reported(mobi, T):
    """A wait that runs out ends the kernel with an error status; the next call is right again."""
    N, K = 1024, 4096
    g = gen(T)
    x, xs = ref.operand(T, K, 1, g, device=DEV)
    w, ws = ref.operand(N, K, 128, g, device=DEV)
    u, us = ref.operand(N, K, 128, g, device=DEV)
    for call in (lambda: mobi.mobi_fp8_gemm(x, xs, w, ws),
                 lambda: mobi.mobi_fp8_gated(x, xs, w, ws, u, us, out_dtype=E4M3)[0]):
        good = call()
        mobi.mobi_sync_check()
        mobi.mobi_debug_set_wait_limit(1)
        try:
            call()
            with pytest.raises(mobi.MobiError) as e:
                mobi.mobi_sync_check()
            assert e.value.status == 6  # MOBI_ERR_TIMEOUT
        finally:
            mobi.mobi_debug_set_wait_limit(0)
        again = call()
        mobi.mobi_sync_check()
        assert torch.equal(again.view(torch.uint8), good.view(torch.uint8))


# ---- norm -----------------------------------------------------------------------------------


def norm_case(T, D, xd, bd, wd, gate, post, kind, g, out):
    x = torch.randn(T, D, generator=g) * 3 + 0.5
    b = torch.randn(T, D, generator=g) * 0.7 - 0.2
    vec = lambda s: (1.0 + torch.randn(D, generator=g) * s).to(wd).to(DEV)  # noqa: E731
    shape = {"none": None, "channel": (D,), "token": (T, 1), "full": (T, D), "one": (1,)}[gate]
    return dict(x=x.to(xd).to(DEV), weight=vec(0.1), bias=vec(0.2) if kind == "layer" else None, eps=1e-5, kind=kind,
                block=b.to(bd).to(DEV) if bd is not None else None,
                **(dict(post=post, post_weight=vec(0.1) if post != "none" else None,
                        post_bias=vec(0.3) if post == "layer" else None, post_eps=1e-4,
                        gate=(torch.randn(*shape, generator=g)).to(F16 if gate == "token" else BF16).to(DEV)
                        if shape else None, scale=0.7) if bd is not None else {}))


def check_norm(mobi, case, out, **more):
    got = mobi.mobi_norm(out_dtype=out, **case, **more)
    mobi.mobi_sync_check()
    n, en, r, er = ref.norm(**case)
    if case["block"] is not None:
        got, rr = got
        ref.check_close(rr, r, ref.rounded(r, er, rr.dtype), "r")
    if out is E4M3:
        ref.check_quantised(got[0], got[1], n, en, "n")
    else:
        ref.check_close(got, n, ref.rounded(n, en, out), "n")


@pytest.mark.parametrize("D", [1, 7, 8, 100, 128, 250, 512, 1000, 4096, 4097, 5000, 8192, 11008, 16384])
@pytest.mark.parametrize("T,kind,post,gate,out", [
    (1, "rms", "none", "none", BF16), (5, "layer", "rms", "channel", F32), (3, "rms", "layer", "token", E4M3),
    (9, "layer", "none", "full", F16), (2, "none", "rms", "one", F32)])
def test_norm(mobi, T, D, kind, post, gate, out):
    g = gen(T * 31 + D)
    for xd, bd, wd in ((BF16, F32, BF16), (F32, BF16, F32), (F16, F16, F16)):
        check_norm(mobi, norm_case(T, D, xd, bd, wd, gate, post, kind, g, out), out)


@pytest.mark.parametrize("T,D", [(1, 4096), (700, 512), (2000, 4096), (1200, 96), (800, 6000), (650, 77), (600, 16384)])
def test_norm_many_rows(mobi, T, D):
    g = gen(D)
    check_norm(mobi, norm_case(T, D, BF16, BF16, BF16, "channel", "rms", "rms", g, E4M3), E4M3)
    check_norm(mobi, norm_case(T, D, F32, F32, F32, "full", "layer", "layer", g, F32), F32)
    check_norm(mobi, norm_case(T, D, BF16, None, BF16, "none", "none", "rms", g, BF16), BF16)


@pytest.mark.parametrize("D", [264, 265])
def test_norm_slices_in_place_and_offset(mobi, D):
    """Rows of larger tensors, the residual stream updated in place, weights counted as 1 + w, no weights at all."""
    g = gen(D)
    T = 40
    big = torch.randn(T, D + 32, generator=g).to(BF16).to(DEV)
    for off in (0, 8, 3):
        x = big.clone()[:, off:off + D]
        keep = x.clone()
        blk = torch.randn(T, D + 16, generator=g).to(DEV)[:, 8:8 + D]
        w = (torch.randn(D, generator=g) * 0.1).to(DEV)
        n, en, r, er = ref.norm(keep, w, None, 1e-6, "rms", block=blk, scale=1.0, unit_offset=True)
        y, rr = mobi.mobi_norm(x, w, block=blk, unit_offset=True, R=x)
        assert rr.data_ptr() == x.data_ptr()
        ref.check_close(x, r, ref.rounded(r, er, BF16), "r")
        ref.check_close(y, n, ref.rounded(n, en, BF16), "n")
        n, en, _, _ = ref.norm(keep, None, None, 1e-6, "layer")
        out = torch.full((T, D + 9), 5.0, device=DEV)
        mobi.mobi_norm(keep, kind="layer", out_dtype=F32, N=out[:, 4:4 + D])
        ref.check_close(out[:, 4:4 + D], n, ref.rounded(n, en, F32), "plain")
        assert (out[:, :4] == 5.0).all() and (out[:, 4 + D:] == 5.0).all()


def test_norm_special_rows(mobi):
    """A zero row, rows with an infinity or a NaN, constant rows: the others are untouched by them."""
    T, D = 6, 520
    x = torch.randn(T, D, generator=gen(9))
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3] = 2.5
    for kind in ("rms", "layer"):
        for out in (F32, E4M3):
            y = mobi.mobi_norm(x.to(DEV), kind=kind, out_dtype=out, eps=1e-6)
            v = (y[0] if out is E4M3 else y).float()
            n, en, _, _ = ref.norm(x.to(DEV), None, None, 1e-6, kind)
            assert (v[0] == 0).all() and torch.isnan(v[2]).any()
            if out is F32:
                ref.check_close(v[4:], n[4:], ref.rounded(n, en, F32)[4:])
                ref.check_close(v[3], n[3], ref.rounded(n, en, F32)[3])


# ---- scoring --------------------------------------------------------------------------------


def check_scores(mobi, x, targets, temp, k):
    lp, H, top, idx = mobi.mobi_logprobs(x, targets, temperature=temp, top_k=k)
    wl, wH, wt, wi, elog, eH = ref.logprobs(x, targets, temp, k)
    assert torch.equal(idx, wi.to(torch.int32)), "alternatives"

    def close(got, want, bound, what):
        inf = torch.isneginf(want)
        assert torch.equal(torch.isneginf(got), inf), what
        z = torch.zeros_like(want)
        ref.check_close(torch.where(inf, z.float(), got), torch.where(inf, z, want),
                        torch.where(inf, z, bound) + 1e-300, what)
    # (x - m) / t: a rounding each, and the difference from ln S.
    if targets is not None:
        ignored = targets < 0
        assert (lp[ignored] == 0).all()
        close(lp, wl, elog[:, 0] + 6 * ref.U * wl.abs() + 3 * ref.U * elog[:, 0], "log probability")
    else:
        assert lp is None
    close(H, wH, eH, "entropy")
    close(top, wt, elog + 6 * ref.U * wt.abs(), "top")


SHAPES = [(1, 1), (2, 7), (3, 33), (5, 1000), (4, 4099), (2, 32000), (1, 131073), (150, 5000), (300, 700)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,V", SHAPES)
def test_logprobs(mobi, T, V, dtype):
    g = gen(T * 7 + V)
    x = (torch.randn(T, V, generator=g) * 3).to(dtype).to(DEV)
    t = torch.randint(-1, V, (T,), generator=g).to(DEV)
    for temp, k in ((1.0, 5), (0.6, 0), (3.0, 20), (1.0, 32)):
        check_scores(mobi, x, t, temp, k)
    check_scores(mobi, x, None, 1.0, 1)
    mobi.mobi_sync_check()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,V", [(2, 7), (3, 1000), (4, 32000), (2, 131073), (200, 3000)])
@pytest.mark.parametrize("mask", ["some", "few", "empty", "ties", "constant", "rounded"])
def test_logprobs_masks_and_ties(mobi, T, V, dtype, mask):
    """Masked entries, rows with fewer left than asked for, rows with nothing left, equal entries (the lowest index)."""
    g = gen(V)
    x = torch.randn(T, V, generator=g) * 2
    drop = torch.rand(T, V, generator=g)
    if mask == "some":
        x[drop < 0.5] = float("-inf")
    elif mask == "few":
        x[drop > 4.0 / V] = float("-inf")
    elif mask == "empty":
        x[T // 2] = float("-inf")
    elif mask == "ties":
        x = torch.where(drop < 0.01, 5.0, torch.where(drop < 0.5, 4.0, -1.0))
    elif mask == "constant":
        x[:] = -2.5
    else:
        x = x.round()
    t = torch.randint(0, V, (T,), generator=g).to(DEV)
    for k in (1, 20, 32):
        check_scores(mobi, x.to(dtype).to(DEV), t, 0.9, k)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,V", [(3, 1000), (2, 40000), (160, 2000)])
def test_logprobs_lowest_value_masks(mobi, T, V, dtype):
    """A mask of the type's lowest value: those entries are finite, so they stand behind the rest by index, with a
    probability of 0 beside any other and of 1/n among themselves."""
    g = gen(V + 1)
    low = torch.finfo(dtype).min
    x = torch.randn(T, V, generator=g) * 2
    x[torch.rand(T, V, generator=g) > 8.0 / V] = low
    x[0] = low
    x[1, ::2] = float("-inf")
    x[1, 1::2] = low
    x = x.clamp_min(low).to(dtype) if dtype != F16 else x.to(dtype)
    x[1, ::2] = float("-inf")
    d = x.to(DEV)
    for k in (0, 5, 32):
        lp, H, top, idx = mobi.mobi_logprobs(d, torch.full((T,), 1, device=DEV), temperature=1.3, top_k=k)
        order = torch.argsort(-d.double(), dim=1, stable=True)[:, :k]
        assert torch.equal(idx, order.to(torch.int32))
        n = [V, V // 2]
        for row in (0, 1):
            tol = (V / 256 + 40) * ref.U * 16 + 8 * ref.U * math.log(V)
            assert abs(lp[row].item() + math.log(n[row])) <= tol and abs(H[row].item() - math.log(n[row])) <= 2 * tol
            if k:
                assert (top[row].double() + math.log(n[row])).abs().max().item() <= tol


def test_logprobs_extremes(mobi):
    """Large logits and temperatures, an infinity, a NaN, a target outside the vocabulary, rows of a larger tensor."""
    g = gen(4)
    x = torch.randn(6, 500, generator=g)
    x[1] *= 1e30
    x[2] *= 1e-30
    for temp in (1e-3, 1.0, 1e6):
        check_scores(mobi, x[[0, 2, 3]].to(DEV), torch.tensor([3, 4, 5], device=DEV), temp, 8)
    lp, H, top, idx = mobi.mobi_logprobs(x[1:2].to(DEV), torch.tensor([7], device=DEV), top_k=1)
    best = int(x[1].argmax())
    assert idx[0, 0] == best and top[0, 0] == 0 and H[0] == 0
    y = x.clone()
    y[0, 3] = float("nan")
    y[4, 9] = float("inf")
    lp, H, top, idx = mobi.mobi_logprobs(y.to(DEV), torch.zeros(6, dtype=torch.int64, device=DEV), top_k=3)
    assert torch.isnan(lp[[0, 4]]).all() and torch.isnan(H[[0, 4]]).all() and torch.isfinite(lp[[2, 3, 5]]).all()
    mobi.mobi_sync_check()
    lp, _, _, _ = mobi.mobi_logprobs(x.to(DEV), torch.tensor([0, 0, 0, 500, 0, 0], device=DEV))
    assert torch.isnan(lp[3]) and torch.isfinite(lp[[0, 2, 4, 5]]).all()
    with pytest.raises(mobi.MobiError) as e:
        mobi.mobi_sync_check()
    assert e.value.status == 1
    mobi.mobi_sync_check()
    big = torch.randn(9, 1100, generator=g).to(BF16).to(DEV)
    for part in (big[:, 1:1000], big[::2, 8:900], big[:, 3:4]):
        check_scores(mobi, part, torch.zeros(part.shape[0], dtype=torch.int64, device=DEV), 1.0, 4)


# ---- together -------------------------------------------------------------------------------


def test_empty_calls(mobi):
    z = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    q, s = mobi.mobi_fp8_quant(z(0, 256))
    assert q.shape == (0, 256) and s.shape == (2, 0)
    w, ws = mobi.mobi_fp8_quant(torch.ones(64, 256, device=DEV), block_rows=128)
    assert mobi.mobi_fp8_gemm(q, s, w, ws).shape == (0, 64)
    h, hs = mobi.mobi_fp8_gated(q, s, w, ws, w, ws, out_dtype=E4M3)
    assert h.shape == (0, 64) and hs.shape == (1, 0)
    assert mobi.mobi_norm(z(0, 256)).shape == (0, 256)
    lp, H, top, idx = mobi.mobi_logprobs(z(0, 100), z(0, dtype=torch.int64), top_k=3)
    assert lp.shape == (0,) and top.shape == (0, 3)
    mobi.mobi_sync_check()


def test_refusals_of_the_binding(mobi):
    x = torch.randn(4, 256, device=DEV)
    q, s = mobi.mobi_fp8_quant(x)
    w, ws = mobi.mobi_fp8_quant(x, block_rows=128)
    bad = [lambda: mobi.mobi_fp8_quant(x, block_rows=64), lambda: mobi.mobi_fp8_quant(x.t()),
           lambda: mobi.mobi_fp8_quant(x.double()), lambda: mobi.mobi_fp8_quant(x[0]),
           lambda: mobi.mobi_fp8_gemm(q, s, w, s), lambda: mobi.mobi_fp8_gemm(q, s, w[:, :128], ws),
           lambda: mobi.mobi_fp8_gemm(q.float(), s, w, ws), lambda: mobi.mobi_fp8_gemm(q, s, w, ws, out_dtype=E4M3),
           lambda: mobi.mobi_fp8_gemm(q, s, w, ws, Y=torch.empty(4, 5, device=DEV)),
           lambda: mobi.mobi_fp8_gated(q, s, w, ws, w[:2], ws), lambda: mobi.mobi_fp8_gated(q, s, w, ws, w, ws, act="x"),
           lambda: mobi.mobi_norm(x, torch.ones(255, device=DEV)), lambda: mobi.mobi_norm(x, kind="group"),
           lambda: mobi.mobi_norm(x, block=x[:2]), lambda: mobi.mobi_norm(x, gate=x),
           lambda: mobi.mobi_norm(x, torch.ones(256, device=DEV), torch.ones(256, device=DEV).half()),
           lambda: mobi.mobi_norm(x, block=x, gate=torch.ones(3, 1, device=DEV)),
           lambda: mobi.mobi_logprobs(x, torch.zeros(4, dtype=torch.int32, device=DEV)),
           lambda: mobi.mobi_logprobs(x, top_k=33), lambda: mobi.mobi_logprobs(x, temperature=0.0)]
    for f in bad:
        with pytest.raises((ValueError, RuntimeError)):
            f()
    mobi.mobi_sync_check()


def _layer(mobi, T, seed):
    """A block's feed-forward half and the head, as a user would chain them; returns a function of (x, y) and its parts."""
    D, F, V = 256, 640, 1000
    g = gen(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DEV)  # noqa: E731
    ws = {k: mobi.mobi_fp8_quant(rnd(n, m, std=0.06), block_rows=128) for k, n, m in
          (("g", F, D), ("u", F, D), ("d", D, F))}
    head, sz = mobi.mobi_pack(rnd(((V + 15) // 16) * 16, D, std=0.1).half())
    wr = rnd(D, 3, std=0.05)
    w1, w2 = (1 + rnd(D, std=0.1)).bfloat16(), (1 + rnd(D, std=0.1)).bfloat16()
    gate = rnd(D, std=0.5).bfloat16()

    def run(x, y, targets):
        (n, ns), r = mobi.mobi_norm(x, w1, block=y, post="rms", post_weight=w2, gate=gate, scale=0.5, out_dtype=E4M3)
        h, hs = mobi.mobi_fp8_gated(n, ns, *ws["g"], *ws["u"], out_dtype=E4M3)
        d = mobi.mobi_fp8_gemm(h, hs, *ws["d"])
        f, r2 = mobi.mobi_norm(r, w2, block=d)
        logits, k_t, _, _ = mobi.mobi_linear(f, wr, None, head, sz, ((V + 15) // 16) * 16)
        return (n, ns, r, h, hs, d, f, r2, logits, k_t) + mobi.mobi_logprobs(logits[:, :V], targets, top_k=5)
    return run, ws, (w1, w2, gate), rnd, V


@pytest.mark.parametrize("T", [1, 12, 100, 500])
def test_run_together(mobi, T):
    """Norm -> gated product -> down projection -> norm -> mixed-bit head -> scoring, each step against its plain form
    on the inputs that it got."""
    run, ws, (w1, w2, gate), rnd, V = _layer(mobi, T, 11)
    x, y = rnd(T, 256).bfloat16(), rnd(T, 256)
    t = torch.randint(0, V, (T,), generator=gen(T)).to(DEV)
    n, ns, r, h, hs, d, f, r2, logits, k_t, lp, H, top, idx = run(x, y, t)
    mobi.mobi_sync_check()
    wn, en, wr_, er = ref.norm(x, w1, None, 1e-6, "rms", block=y, post="rms", post_weight=w2, gate=gate, scale=0.5)
    ref.check_close(r, wr_, ref.rounded(wr_, er, BF16), "r")
    ref.check_quantised(n, ns, wn, en, "n")
    wh, eh = ref.gated(n, ns, *ws["g"], *ws["u"], "silu")
    ref.check_quantised(h, hs, wh, eh, "h")
    wd, ed = ref.product(h, hs, *ws["d"])
    ref.check_close(d, wd, ref.rounded(wd, ed, F32), "d")
    wf, ef, w2r, e2r = ref.norm(r, w2, None, 1e-6, "rms", block=d)
    ref.check_close(f, wf, ref.rounded(wf, ef, BF16), "f")
    ref.check_close(r2, w2r, ref.rounded(w2r, e2r, BF16), "r2")
    wl, wH, wt, wi, elog, eH = ref.logprobs(logits[:, :V], t, 1.0, 5)
    assert torch.equal(idx, wi.to(torch.int32))
    ref.check_close(lp, wl, elog[:, 0] + 6 * ref.U * wl.abs(), "lp")


@pytest.mark.parametrize("T", [4, 300])
def test_captured_and_replayed(mobi, T):
    """The chain captured into two graphs that are replayed in turn with new inputs gives what eager calls give."""
    run, _, _, rnd, V = _layer(mobi, T, 12)
    bufs = [(rnd(T, 256).bfloat16(), rnd(T, 256), torch.randint(0, V, (T,), generator=gen(i)).to(DEV)) for i in range(2)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for b in bufs:
            run(*b)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b in bufs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(run(*b))
        graphs.append(gr)
    for rep in range(3):
        for b in bufs:
            b[0].copy_(rnd(T, 256))
            b[1].copy_(rnd(T, 256))
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        mobi.mobi_sync_check()
        got = [[o.clone() for o in out] for out in outs]
        for b, out in zip(bufs, got):
            for a, e in zip(out, run(*b)):
                assert torch.equal(a.contiguous().view(torch.uint8), e.contiguous().view(torch.uint8))


@pytest.mark.parametrize("handle", [False, True])
def test_given_stream(mobi, handle):
    """Calls on a given stream, or on its handle, give what they give on the current one, and their new outputs stay out
    of memory that the current stream has freed (work queued there may still use it)."""
    g = gen(21)
    x, xs = ref.operand(70, 512, 1, g, device=DEV)
    w, ws = ref.operand(384, 512, 128, g, device=DEV)
    v = torch.randn(70, 512, generator=g).to(DEV)
    y = torch.randint(0, 512, (70,), generator=g).to(DEV)
    calls = [lambda **k: mobi.mobi_fp8_quant(v, **k), lambda **k: (mobi.mobi_fp8_gemm(x, xs, w, ws, **k),),
             lambda **k: (mobi.mobi_fp8_gated(x, xs, w, ws, w, ws, **k),), lambda **k: mobi.mobi_norm(v, block=v, **k),
             lambda **k: mobi.mobi_logprobs(v, y, top_k=4, **k)]
    side = torch.cuda.Stream()
    for call in calls:
        want = call()
        freed = [torch.empty_like(o) for o in want]
        at = {o.data_ptr() for o in freed}
        torch.cuda.synchronize()
        del freed
        got = call(stream=side.cuda_stream if handle else side)
        torch.cuda.synchronize()
        assert not at & {o.data_ptr() for o in got}
        for a, b in zip(got, want):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    out = torch.empty(70, 384, device=DEV)
    torch.cuda.synchronize()
    assert mobi.mobi_fp8_gemm(x, xs, w, ws, Y=out, stream=0) is out
    torch.cuda.synchronize()
    assert torch.equal(out, mobi.mobi_fp8_gemm(x, xs, w, ws))
    mobi.mobi_sync_check()


def test_graphs_replayed_at_once(mobi):
    """Two captured chains replayed on two streams at the same time: nothing is shared between them."""
    run, _, _, rnd, V = _layer(mobi, 40, 13)
    args = [(rnd(40, 256).bfloat16(), rnd(40, 256), torch.randint(0, V, (40,), generator=gen(i)).to(DEV))
            for i in range(2)]
    want = [run(*a) for a in args]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in args:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(run(*a))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    mobi.mobi_sync_check()
    for out, w in zip(outs, want):
        for a, b in zip(out, w):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_rows_far_apart(mobi):
    """Rows more than 4 GiB apart, read and written: the same as close ones."""
    g = gen(31)
    pitch = (1 << 32) + 256  # bytes
    store = [torch.empty(pitch + 4096, dtype=torch.uint8, device=DEV) for _ in range(2)]

    def far(t, i=0):
        v = store[i].view(t.dtype).as_strided(t.shape, (pitch // t.element_size(), 1))
        v.copy_(t)
        return v

    x = torch.randn(2, 512, generator=g).to(BF16).to(DEV)
    w = (1 + 0.1 * torch.randn(512, generator=g)).to(BF16).to(DEV)
    q, s = mobi.mobi_fp8_quant(x)
    got = mobi.mobi_fp8_quant(far(x), Q=far(torch.zeros_like(q), 1))
    assert torch.equal(got[0].contiguous().view(torch.uint8), q.view(torch.uint8)) and torch.equal(got[1], s)
    m, ms = ref.operand(300, 512, 128, g, device=DEV)
    y = mobi.mobi_fp8_gemm(q, s, m, ms)
    assert torch.equal(mobi.mobi_fp8_gemm(far(q), s, m, ms, Y=far(torch.zeros_like(y), 1)), y)
    h = mobi.mobi_fp8_gated(q, s, m, ms, m, ms)
    assert torch.equal(mobi.mobi_fp8_gated(far(q), s, m, ms, m, ms, H=far(torch.zeros_like(h), 1)), h)
    n, r = mobi.mobi_norm(far(x), w, block=x, post="rms", scale=0.5, R=far(torch.zeros_like(x), 1))
    wn, en, wr, er = ref.norm(x, w, None, 1e-6, "rms", block=x, post="rms", scale=0.5)
    ref.check_close(r, wr, ref.rounded(wr, er, BF16), "r")
    ref.check_close(n, wn, ref.rounded(wn, en, BF16), "n")
    t = torch.tensor([3, 500], device=DEV)
    for a, b in zip(mobi.mobi_logprobs(far(x), t, top_k=5), mobi.mobi_logprobs(x, t, top_k=5)):
        assert torch.equal(a, b)
    mobi.mobi_sync_check()


@pytest.mark.parametrize("D", [4096, 4095, 16384, 16383])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_range_of_the_squares(mobi, D, kind):
    """Rows on both sides of the stated limit of the sum of squares, 1.8e19 / sqrt(D), before and after the residual
    sum; rows just above the smallest root mean square where eps is 0."""
    sign = (torch.arange(D) % 2 * -2 + 1).float()
    limit = math.sqrt(torch.finfo(torch.float32).max) / math.sqrt(D)
    x = torch.stack([0.97 * limit * sign, 1.03 * limit * sign, 3.0 * sign]).to(DEV)
    y = mobi.mobi_norm(x, kind=kind, out_dtype=F32)
    n, en, _, _ = ref.norm(x, None, None, 1e-6, kind)
    ref.check_close(y[[0, 2]], n[[0, 2]], ref.rounded(n, en, F32)[[0, 2]])
    assert (y[1] == 0).all()
    q, s = mobi.mobi_norm(x, kind=kind, out_dtype=E4M3)
    ref.check_quantised(q[[0, 2]], s[:, [0, 2]], n[[0, 2]], en[[0, 2]])
    assert (q[1].float() == 0).all() and (s[:, 1] == 2.0 ** -126).all()
    base = torch.randn(3, D, generator=gen(D)).to(DEV)
    case = dict(x=base, weight=None, bias=None, eps=1e-6, kind="rms", block=x, post=kind, post_eps=1e-6)
    y, r = mobi.mobi_norm(out_dtype=F32, **case)
    n, en, wr, er = ref.norm(**case)
    for got, want, err in ((y, n, en), (r, wr, er)):
        ref.check_close(got[[0, 2]], want[[0, 2]], ref.rounded(want, err, F32)[[0, 2]])
    assert torch.equal(r[1], base[1])
    small = 1e-18 * sign[None].to(DEV)
    n, en, _, _ = ref.norm(small, None, None, 0.0, kind)
    ref.check_close(mobi.mobi_norm(small, kind=kind, eps=0.0, out_dtype=F32), n, ref.rounded(n, en, F32))
    assert torch.isnan(mobi.mobi_norm(torch.zeros(1, D, device=DEV), kind=kind, eps=0.0, out_dtype=F32)).all()


# ---- every division of a product -------------------------------------------------------------

# One call or more for each kernel, tile and cluster that a call of any size can be given (test_blocks.py holds the
# lists against the library's own choice), with odd sizes and ragged blocks of K; the last ones of each list are the
# wide kernel's: one tile, then two to five tiles that a pair takes in a row, ragged at both ends.
PLANS = [(1, 1, 1), (3, 200, 386), (5, 77, 642), (9, 333, 901), (2, 1000, 1154), (13, 141, 1409), (16, 300, 1665),
         (1, 500, 1923), (17, 45, 100), (21, 99, 385), (25, 207, 647), (31, 130, 899), (32, 300, 1179),
         (19, 400, 1413), (27, 151, 1665), (30, 260, 1969), (34, 9551, 1126), (40, 8822, 2966), (35, 6482, 2195),
         (37, 5518, 2148), (57, 300, 1665), (64, 190, 1925), (38, 13777, 2435), (38, 19484, 2041), (73, 3660, 2948),
         (258, 1084, 2959), (92, 1956, 2422), (131, 907, 2400), (99, 230, 2064), (140, 130, 2088), (69, 300, 1683),
         (130, 150, 1667), (80, 140, 1926), (133, 270, 1988), (333, 700, 270), (600, 4099, 1024), (1000, 8200, 2050),
         (2049, 4099, 640), (2100, 2993, 1040), (4096, 4099, 1040), (4097, 8192, 144)]
PLANS_GATED = [(1, 1, 1), (3, 200, 386), (5, 77, 642), (9, 333, 901), (2, 1000, 1154), (13, 141, 1409), (16, 300, 1665),
               (1, 500, 1923), (17, 45, 100), (21, 99, 385), (25, 207, 647), (31, 130, 899), (32, 300, 1179),
               (19, 400, 1413), (27, 151, 1665), (30, 260, 1969), (38, 11822, 1136), (35, 7007, 2458), (281, 1359, 2758),
               (48, 150, 1034), (66, 140, 1034), (37, 300, 903), (100, 200, 901), (33, 140, 1163), (65, 260, 1163),
               (50, 300, 1419), (127, 200, 1438), (38, 131, 1665), (70, 300, 1689), (64, 260, 1940), (70, 140, 1921),
               (77, 500, 300), (2100, 1300, 400), (1000, 5000, 1040), (2100, 2993, 1040), (2049, 4099, 272)]


def guarded(T, N, dtype, off):
    """A matrix [T, N] whose rows start `off` elements into rows of a larger tensor full of 7, and a check of the rest."""
    buf = torch.full((T + 2, (N + 15) // 16 * 16 + 32), 7.0, device=DEV).to(dtype)
    kept = buf.clone()

    def check():
        raw, want = buf.view(torch.uint8), kept.view(torch.uint8)
        at = slice(off * buf.element_size(), (off + N) * buf.element_size())
        raw[1:T + 1, at] = want[1:T + 1, at]
        assert torch.equal(raw, want), "written outside the output"
    return buf[1:T + 1, off:off + N], check


@pytest.mark.parametrize("T,N,K", PLANS)
def test_gemm_every_plan(mobi, T, N, K):
    g = gen(T + 31 * N + K)
    x, xs = ref.operand(T, K, 1, g, device=DEV)
    w, ws = ref.operand(N, K, 128, g, 0.02, device=DEV)
    x, w = _pitched(x), _pitched(w)
    want, err = ref.product(x, xs, w, ws)
    for dtype, off in ((F32, 16), (BF16, 16), (F16, 3), (F32, 1)):  # rows at multiples of 16 bytes, and others
        y, check = guarded(T, N, dtype, off)
        mobi.mobi_fp8_gemm(x, xs, w, ws, out_dtype=dtype, Y=y)
        mobi.mobi_sync_check()
        ref.check_close(y, want, ref.rounded(want, err, dtype), f"{dtype}")
        check()
    again = mobi.mobi_fp8_gemm(x, xs, w, ws)
    assert all(torch.equal(mobi.mobi_fp8_gemm(x, xs, w, ws), again) for _ in range(3))


@pytest.mark.parametrize("T,N,K", PLANS_GATED)
def test_gated_every_plan(mobi, T, N, K):
    g = gen(T + 37 * N + K)
    x, xs = ref.operand(T, K, 1, g, device=DEV)
    wg, gs = ref.operand(N, K, 128, g, 0.05, device=DEV)
    wu, us = ref.operand(N, K, 128, g, 0.05, device=DEV)
    x, wg, wu = _pitched(x), _pitched(wg), _pitched(wu)
    for act in (("silu", "gelu"), ("relu", "gelu_tanh"))[(T + N) % 2]:
        h, err = ref.gated(x, xs, wg, gs, wu, us, act)
        for dtype, off in ((F32, 16), (BF16, 16), (F16, 3)):
            y, check = guarded(T, N, dtype, off)
            mobi.mobi_fp8_gated(x, xs, wg, gs, wu, us, act=act, out_dtype=dtype, H=y)
            mobi.mobi_sync_check()
            ref.check_close(y, h, ref.rounded(h, err, dtype), f"{dtype}")
            check()
        for off in (16, 5):
            q, check = guarded(T, N, E4M3, off)
            scales = torch.full(((N + 127) // 128, T), 7.0, device=DEV)
            mobi.mobi_fp8_gated(x, xs, wg, gs, wu, us, act=act, out_dtype=E4M3, H=q, hs=scales)
            mobi.mobi_sync_check()
            ref.check_quantised(q, scales, h, err)
            check()
    first = mobi.mobi_fp8_gated(x, xs, wg, gs, wu, us, out_dtype=E4M3)
    for _ in range(3):
        q, s = mobi.mobi_fp8_gated(x, xs, wg, gs, wu, us, out_dtype=E4M3)
        assert torch.equal(q.view(torch.uint8), first[0].view(torch.uint8)) and torch.equal(s, first[1])


@pytest.mark.parametrize("T,N,K", [(2049, 4099, 640), (4096, 4099, 1040)])
def test_tiles_in_a_row_single_blocks(mobi, T, N, K):
    """Every tile that a pair takes after its first uses its own rows' scales and each block of K counts: all blocks but
    one are zero, and the scales differ by powers of two from tile to tile."""
    g = gen(T)
    x, xs = ref.operand(T, K, 1, g, device=DEV)
    w, ws = ref.operand(N, K, 128, g, device=DEV)
    xs *= torch.exp2((torch.arange(T, device=DEV) // 128 % 7 - 3).float())[None]
    ws *= torch.exp2((torch.arange(ws.shape[1], device=DEV) % 5 - 2).float())[None]
    last = (K - 1) // 128
    for b in (0, 2, last):
        xb = torch.zeros_like(x)
        xb[:, 128 * b:128 * b + 128] = x[:, 128 * b:128 * b + 128]
        want, err = ref.product(xb, xs, w, ws)
        ref.check_close(mobi.mobi_fp8_gemm(xb, xs, w, ws), want, ref.rounded(want, err, F32))
    mobi.mobi_sync_check()


def test_tiles_in_a_row_beside_another_call(mobi):
    """Calls whose pairs take several tiles, on two streams at once and captured into a graph: the bits of a call alone."""
    g = gen(17)
    x, xs = ref.operand(2100, 1040, 1, g, device=DEV)
    w, ws = ref.operand(2993, 1040, 128, g, 0.05, device=DEV)
    u, us = ref.operand(2993, 1040, 128, g, 0.05, device=DEV)
    y, (h, hs) = mobi.mobi_fp8_gemm(x, xs, w, ws), mobi.mobi_fp8_gated(x, xs, w, ws, u, us, out_dtype=E4M3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = (mobi.mobi_fp8_gemm(x, xs, w, ws), *mobi.mobi_fp8_gated(x, xs, w, ws, u, us, out_dtype=E4M3))
    a, b, c = (torch.cuda.Stream() for _ in range(3))
    outs = []
    for _ in range(5):
        with torch.cuda.stream(a):
            p = mobi.mobi_fp8_gemm(x, xs, w, ws)
        with torch.cuda.stream(b):
            q = mobi.mobi_fp8_gated(x, xs, w, ws, u, us, out_dtype=E4M3)
        with torch.cuda.stream(c):
            graph.replay()
        outs.append((p, *q))
    torch.cuda.synchronize()
    mobi.mobi_sync_check()
    for out in outs + [held]:
        for got, want in zip(out, (y, h, hs)):
            assert torch.equal(got.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


@pytest.mark.parametrize("T,N,K", [(2100, 2993, 1040), (4096, 4099, 1040)])
def test_timeout_with_tiles_in_a_row(mobi, T, N, K):
    """A wait that runs out before the first of several tiles ends the kernel with an error status."""
    g = gen(T)
    x, xs = ref.operand(T, K, 1, g, device=DEV)
    w, ws = ref.operand(N, K, 128, g, 0.05, device=DEV)
    u, us = ref.operand(N, K, 128, g, 0.05, device=DEV)
    want, err = ref.product(x, xs, w, ws)
    h, eh = ref.gated(x, xs, w, ws, u, us, "silu")
    mobi.mobi_sync_check()
    for call in (lambda: mobi.mobi_fp8_gemm(x, xs, w, ws), lambda: mobi.mobi_fp8_gated(x, xs, w, ws, u, us),
                 lambda: mobi.mobi_fp8_gated(x, xs, w, ws, u, us, out_dtype=E4M3)):
        mobi.mobi_debug_set_wait_limit(1)
        try:
            call()
            with pytest.raises(mobi.MobiError) as e:
                mobi.mobi_sync_check()
            assert e.value.status == 6  # MOBI_ERR_TIMEOUT
        finally:
            mobi.mobi_debug_set_wait_limit(0)
        mobi.mobi_sync_check()
    ref.check_close(mobi.mobi_fp8_gemm(x, xs, w, ws), want, ref.rounded(want, err, F32))
    q, s = mobi.mobi_fp8_gated(x, xs, w, ws, u, us, out_dtype=E4M3)
    ref.check_quantised(q, s, h, eh)
    mobi.mobi_sync_check()


@pytest.mark.parametrize("D,off", [(520, 0), (521, 0), (520, 3), (4096, 0), (4097, 0), (97, 0), (9000, 0), (9001, 0)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("where", ["x", "block", "gate", "post"])
def test_norm_rows_that_are_not_finite(mobi, D, off, kind, where):
    """Infinities and NaN in some rows, from every input: those rows follow the definition (NaN where it gives NaN, 0
    where an infinite sum of squares leaves 0, and the scales and codes of their blocks), all others keep their bounds.
    With more rows than CTAs, so that a row follows a bad one in the same threads; both kernels (odd D, odd starts)."""
    T, inf, nan = 1500, float("inf"), float("nan")
    g = gen(D + off)
    bad = {1: inf, 2: nan, 4: -inf, 700: nan, 701: inf, 1498: inf}
    wide = lambda t: torch.cat([t.new_zeros(T, off), t], 1).to(DEV)[:, off:]  # noqa: E731
    base = torch.randn(T, D, generator=g) * 2
    base[0], base[3] = 0.0, 2.5
    block, gate = torch.randn(T, D, generator=g), torch.randn(T, D, generator=g) * 0.5 + 1.5
    block[0] = block[3] = 0.0
    at = {"x": base, "block": block, "gate": gate, "post": block}[where]
    for t, v in bad.items():
        at[t, (t * 7) % D] = v
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(DEV)
    case = dict(x=wide(base), weight=w, bias=None, eps=1e-6, kind=kind)
    if where != "x":
        case.update(block=wide(block), gate=wide(gate), post="rms" if where == "post" else "none", post_eps=1e-5, scale=0.5)
    n, en, r, er = ref.norm(**case)
    good = torch.ones(T, dtype=torch.bool, device=DEV)
    good[list(bad)] = False
    assert torch.isfinite(n[good]).all() and torch.isnan(n[~good]).any(1).all()
    assert ((n == 0) | torch.isnan(n))[~good].all()

    def same(got, want, bound, dtype, what):
        got = got.double()
        ref.check_close(got[good], want[good], ref.rounded(want, bound, dtype)[good], what)
        assert torch.equal(torch.isnan(got[~good]), torch.isnan(want[~good])), what
        return got[~good], want[~good]

    for dtype in (F32, BF16):
        y = mobi.mobi_norm(out_dtype=dtype, **case)
        if where != "x":
            y, rr = y
            a, b = same(rr, r, er, F32, "r")
            assert torch.equal(torch.isinf(a), torch.isinf(b)) and torch.equal(a[torch.isinf(b)], b[torch.isinf(b)])
        a, b = same(y, n, en, dtype, "n")
        assert torch.equal(a.nan_to_num(1.0), b.nan_to_num(1.0))
    y = mobi.mobi_norm(out_dtype=E4M3, **case)
    q, s = y if where == "x" else y[0]
    ref.check_quantised(q[good], s[:, good], n[good], en[good], "codes")
    broken = torch.isnan(ref.blocks(n[~good], 1)).any(3)[:, 0]  # [rows, blocks]
    assert torch.equal(torch.isnan(s[:, ~good].t()), broken) and (s[:, ~good].t()[~broken] == 2.0 ** -126).all()
    v = ref.blocks(q[~good].float(), 1)[:, 0]
    inside = (torch.arange(v[0].numel(), device=DEV) < D).view(v[0].shape)
    for i in range(len(bad)):
        assert torch.isnan(v[i][broken[i]][inside[broken[i]]]).all() and (v[i][~broken[i]] == 0).all()
    mobi.mobi_sync_check()


@pytest.mark.parametrize("T,D", [(5, 264), (600, 2048), (600, 264), (5, 4104), (5, 8200), (5, 1001), (600, 4097), (5, 8201)])
@pytest.mark.parametrize("xd", [F32, BF16, F16])
@pytest.mark.parametrize("bd", [None, F32, BF16, F16])
def test_norm_types(mobi, T, D, xd, bd):
    """Each type of x with each of the block, the weights and the gate, and each shape of the gate, in every form of both
    kernels (one, two and four octets of a thread, few rows and many)."""
    g = gen(T + D)
    outs = [BF16, E4M3, F32, F16]
    for i, wd in enumerate((F32, BF16, F16)):
        for j, gate in enumerate(("channel", "token", "full") if bd is not None else ("none",)):
            case = norm_case(T, D, xd, bd, wd, "none", ("rms", "layer", "none")[(i + j) % 3], ("layer", "rms")[j % 2], g, F32)
            if bd is not None:
                shape = {"channel": (D,), "token": (T, 1), "full": (T, D)}[gate]
                case["gate"] = torch.randn(*shape, generator=g).to((F32, F16, BF16)[(i + 2 * j) % 3]).to(DEV)
            check_norm(mobi, case, outs[(i + j + (bd is None)) % 4])


def test_gradients_are_refused(mobi):
    """Each input in turn requires a gradient: refused where gradients are recorded, the same bits under no_grad."""
    x, b, g = torch.randn(4, 256, device=DEV), torch.randn(4, 256, device=DEV), torch.randn(4, 1, device=DEV)
    v = [torch.randn(256, device=DEV) for _ in range(4)]
    q, s = mobi.mobi_fp8_quant(x)
    w, ws = mobi.mobi_fp8_quant(x, block_rows=128)
    norm = lambda x, b, g, w, c, p, d: mobi.mobi_norm(x, w, c, block=b, gate=g, post="rms", post_weight=p,  # noqa: E731
                                                      post_bias=d)
    calls = [(lambda x: mobi.mobi_fp8_quant(x), [x]), (lambda x: mobi.mobi_logprobs(x, top_k=2), [x]),
             (lambda s, ws: mobi.mobi_fp8_gemm(q, s, w, ws), [s, ws]),
             (lambda s, gs, us: mobi.mobi_fp8_gated(q, s, w, gs, w, us), [s, ws, ws.clone()]), (norm, [x, b, g, *v])]
    flat = lambda o: [t for t in (o if isinstance(o, tuple) else (o,)) if t is not None]  # noqa: E731
    for call, args in calls:
        want = flat(call(*args))
        for i in range(len(args)):
            some = [a.clone().requires_grad_(i == j) for j, a in enumerate(args)]
            with pytest.raises(ValueError, match="requires a gradient"):
                call(*some)
            with torch.no_grad():
                got = flat(call(*some))
            for a, e in zip(got, want):
                assert torch.equal(a.view(torch.uint8), e.view(torch.uint8)) and not a.requires_grad
    mobi.mobi_sync_check()


@pytest.mark.parametrize("first", ["quant", "gemm", "gated", "norm", "logprobs"])
def test_first_call_of_a_process_is_captured(first):
    """Each call as the first of its process, inside a capture: what it sets up once per device may happen there."""
    import os
    import subprocess
    import sys
    code = """
import sys, torch
import block_ref as ref
import token_adaptive_mixed_b200 as mobi
first = sys.argv[1]
g = torch.Generator().manual_seed(2)
v = torch.randn(40, 256, generator=g).cuda()
x, xs = ref.operand(40, 256, 1, g)
w, ws = ref.operand(300, 256, 128, g)
t = torch.arange(40).cuda()
call = {"quant": lambda: mobi.mobi_fp8_quant(v), "gemm": lambda: (mobi.mobi_fp8_gemm(x, xs, w, ws),),
        "gated": lambda: (mobi.mobi_fp8_gated(x, xs, w, ws, w, ws),), "norm": lambda: mobi.mobi_norm(v, block=v),
        "logprobs": lambda: mobi.mobi_logprobs(v, t, top_k=3)}[first]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = call()
graph.replay()
torch.cuda.synchronize()
mobi.mobi_sync_check()
for a, b in zip(held, call()):
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
print("same")
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "PYTHONPATH": os.pathsep.join([os.path.dirname(here), here])}
    out = subprocess.run([sys.executable, "-c", code, first], env=env, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]


def test_outputs_past_32_bits(mobi):
    """More than 2^31 elements in and out: the last rows are what a call on them alone gives."""
    g = gen(41)
    last = torch.tensor([0, 1, 255, 256, -300, -2, -1])

    def pick(t, dim=0):
        return t.index_select(dim, (last % t.shape[dim]).to(DEV)).contiguous().view(torch.uint8)

    x = torch.randn(1024, 8192, generator=g).to(BF16).to(DEV).repeat(270, 1)[:275001]
    x[-300:] *= 3
    part = x[(last % x.shape[0]).to(DEV)]
    w = (1 + 0.1 * torch.randn(8192, generator=g)).to(BF16).to(DEV)
    for rows in (1, 128):
        q, s = mobi.mobi_fp8_quant(x, block_rows=rows)
        assert q.numel() > 1 << 31
        if rows == 1:
            a, b = mobi.mobi_fp8_quant(part)
            assert torch.equal(pick(q), a.view(torch.uint8)) and torch.equal(pick(s, 1), b.view(torch.uint8))
        else:
            at = 128 * (x.shape[0] // 128)
            a, b = mobi.mobi_fp8_quant(x[at:], block_rows=128)
            assert torch.equal(q[at:].view(torch.uint8), a.view(torch.uint8)) and torch.equal(s[:, -1:], b)
        del q, s
    y = mobi.mobi_norm(x, w)
    n, en, _, _ = ref.norm(part, w, None, 1e-6, "rms")
    ref.check_close(y[(last % x.shape[0]).to(DEV)], n, ref.rounded(n, en, BF16))
    del y, x
    x = torch.randn(64, 128001, generator=g).to(BF16).to(DEV).repeat(270, 1)
    t = torch.randint(0, 128001, (x.shape[0],), generator=g).to(DEV)
    at = (last % x.shape[0]).to(DEV)
    assert x.numel() > 1 << 31
    lp, H, top, idx = (o[at] for o in mobi.mobi_logprobs(x, t, top_k=4))
    wl, wH, wt, wi, elog, eH = ref.logprobs(x[at], t[at], 1.0, 4)
    assert torch.equal(idx, wi.to(torch.int32))
    ref.check_close(lp, wl, elog[:, 0] + 6 * ref.U * wl.abs() + 3 * ref.U * elog[:, 0], "log probability")
    ref.check_close(H, wH, eH, "entropy")
    ref.check_close(top, wt, elog + 6 * ref.U * wt.abs(), "top")
    del x
    T, N, K = 60001, 40003, 144
    q, s = ref.operand(T, K, 1, g, device=DEV)
    w, ws = ref.operand(N, K, 128, g, device=DEV)
    y = mobi.mobi_fp8_gemm(q, s, w, ws, out_dtype=BF16)
    h, hs = mobi.mobi_fp8_gated(q, s, w, ws, w, ws, out_dtype=E4M3)
    assert y.numel() > 1 << 31
    mobi.mobi_sync_check()
    at = (last % T).to(DEV)
    qs, ss = q.view(torch.uint8)[at].view(E4M3), s[:, at].contiguous()
    want, err = ref.product(qs, ss, w, ws)
    ref.check_close(y[at], want, ref.rounded(want, err, BF16))
    want, err = ref.gated(qs, ss, w, ws, w, ws, "silu")
    ref.check_quantised(h.view(torch.uint8)[at].view(E4M3), hs[:, at].contiguous(), want, err)


@pytest.mark.parametrize("T", [11, 300])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_activations_keep_their_relative_accuracy(mobi, act, T):
    """g is every finite e4m3 value times a power of two, exactly, and u is 1: h is the activation alone, also far to the
    left, where it nears 0. Bounds relative to the value (U = 2^-24): the fast exponential of w is off by 2 + 1.2 |w|
    steps (2 U each), w itself by 6 U |w|, the division by 2 steps, the sum by half of one. gelu with z = |g| / sqrt 2:
    2 U (7 + z (2 z + 1.5)), from an erfc good to 4 steps whose argument's two roundings, 2 U z, meet a slope of its
    logarithm of at most 2 z + 1.5, and two products; a polynomial's 14 U and three roundings of z^2 fit into it.
    Where e^-w passes 2^126 the fast division gives 0, and values below 2^-119 are not held to a relative bound."""
    codes = torch.arange(256, dtype=torch.uint8).view(E4M3)
    codes = codes[torch.isfinite(codes.float())]
    N = codes.numel()
    x = torch.zeros(T, 128)
    x[:, 0] = 1.0
    wg, wu = torch.zeros(N, 128), torch.zeros(N, 128)
    wg[:, 0], wu[:, 0] = codes.float(), 1.0
    xs = torch.exp2(-(torch.arange(T) % 11).float())[None].to(DEV)
    gs, us = torch.ones(1, 2, device=DEV), torch.ones(1, 2, device=DEV)
    x, wg, wu = (t.to(E4M3).to(DEV) for t in (x, wg, wu))
    g = codes.double().to(DEV)[None] * xs.double().t()
    assert torch.equal(mobi.mobi_fp8_gemm(x, xs, wg, gs).double(), g)
    want = ref.ACT[act](g)
    if act == "silu":
        rel = 2 * ref.U * (6 + 1.2 * g.abs())
    elif act == "gelu_tanh":
        rel = 2 * ref.U * (6 + 4.2 * (2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)).abs())
    elif act == "gelu":
        z = g.abs() / math.sqrt(2.0)
        rel = 2 * ref.U * (7 + z * (2 * z + 1.5))
    else:
        rel = torch.zeros_like(g)
    # u = 1 for the same xs: the product's other side takes 1 / xs through us, one call for each power of two.
    for j in range(11):
        rows = slice(j, T, 11)
        h = mobi.mobi_fp8_gated(x, xs, wg, gs, wu, us * 2.0 ** j, act=act, out_dtype=F32)
        ref.check_close(h[rows], want[rows], want[rows].abs() * rel[rows] + 2.0 ** -119, f"{act} 2^-{j}")
    mobi.mobi_sync_check()


@pytest.mark.parametrize("T,D", [(1, 256), (7, 256), (700, 512), (7, 257), (1, 1), (5, 8)])
@pytest.mark.parametrize("xd", [F32, BF16])
def test_norm_gates_of_any_layout(mobi, T, D, xd):
    """Whatever broadcasts to the rows: a scalar, one value, a row, a column, transposed, every other column, columns of
    a larger tensor at odd starts, rows that overlap."""
    g = gen(T * 3 + D)
    rnd = lambda *s, dtype=F32: torch.randn(*s, generator=g).to(dtype).to(DEV)  # noqa: E731
    x, b, w = (rnd(*s, dtype=xd) for s in ((T, D), (T, D), (D,)))
    for gd in (F32, BF16):
        r = lambda *s: rnd(*s, dtype=gd)  # noqa: E731
        gates = [r(1)[0], r(1), r(1, D), r(T, 1), r(1, 1), r(D, T).t(), r(T, 2 * D)[:, ::2], r(T, D + 9)[:, 5:5 + D],
                 r(T, D + 16)[:, 8:8 + D], r(2 * T, D)[::2], r(T + D).as_strided((T, D), (1, 1)), r(T, 3)[:, 1:2],
                 r(D, 1).t().expand(T, D), r(D, 3)[:, 1]]
        for i, gate in enumerate(gates):
            check_norm(mobi, dict(x=x, weight=w, bias=None, eps=1e-6, kind="rms", block=b, gate=gate, scale=-1.5),
                       (F32, E4M3)[i % 2])


@pytest.mark.parametrize("T,K", [(1, 128), (7, 300), (130, 513), (260, 1024)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quant_and_norm_into_given_outputs(mobi, T, K, dtype):
    """Codes and scales written where the caller says, at rows on multiples of 16 bytes and off them, and nowhere else."""
    g = gen(T + K)
    x = torch.randn(T, K, generator=g).to(dtype)
    d = x.to(DEV)
    kb = (K + 127) // 128
    n, en, _, _ = ref.norm(d, None, None, 1e-6, "rms")
    for off in (0, 16, 3):
        for rows in (1, 128):
            q, check = guarded(T, K, E4M3, off)
            room = torch.full((kb * (T if rows == 1 else (T + 127) // 128) + 2,), 7.0, device=DEV)
            s = room[1:-1].view(kb, -1)
            a, b = mobi.mobi_fp8_quant(d, block_rows=rows, Q=q, scale=s)
            assert a is q and b is s
            wq, ws = ref.quant(x, rows)
            assert same_codes(q, wq) and torch.equal(s.cpu(), ws) and (room[[0, -1]] == 7.0).all()
            check()
        q, check = guarded(T, K, E4M3, off)
        room = torch.full((kb * T + 2,), 7.0, device=DEV)
        s = room[1:-1].view(kb, T)
        a, b = mobi.mobi_norm(d, out_dtype=E4M3, N=q, n_scale=s)
        assert a is q and b is s
        ref.check_quantised(q, s, n, en)
        assert (room[[0, -1]] == 7.0).all()
        check()
        y, check = guarded(T, K, dtype, off)
        r, checked = guarded(T, K, dtype, 16 - off)
        o, rr = mobi.mobi_norm(d, block=d, scale=0.0, out_dtype=dtype, N=y, R=r)
        assert o is y and rr is r and torch.equal(r, d)
        ref.check_close(y, n, ref.rounded(n, en, dtype))
        check()
        checked()
    mobi.mobi_sync_check()


@pytest.mark.parametrize("T", [11, 300])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_activations_of_infinities_and_nan(mobi, act, T):
    """g beyond fp32's range (the scales' product overflows) and NaN, u = 1: what the formula gives in 64 bits, in those
    rows alone."""
    N = 260
    g = gen(T)
    x = torch.zeros(T, 128)
    x[:, 0] = 1.0
    wg, wu = torch.zeros(N, 128), torch.zeros(N, 128)
    wg[:, 0], wu[:, 0] = torch.randn(N, generator=g), 1.0
    wg[7, 0] = 0.0
    xs = torch.ones(1, T)
    xs[0, 3], xs[0, 5] = 2.0 ** 127, float("nan")
    gs, us = torch.full((1, 3), 4.0, device=DEV), torch.full((1, 3), 2.0 ** -127, device=DEV)
    x, wg, wu = (t.to(E4M3).to(DEV) for t in (x, wg, wu))
    xs = xs.to(DEV)
    v = wg.double()[:, 0]
    big = torch.where(v == 0, math.nan, v.sign() * math.inf)  # 0 times an infinite scale
    h = mobi.mobi_fp8_gated(x, xs, wg, gs, wu, us, act=act, out_dtype=F32)
    for row, want in ((3, ref.ACT[act](big)), (5, torch.full_like(v, math.nan))):
        assert torch.equal(torch.isnan(h[row]), torch.isnan(want))
        assert torch.equal(h[row][~torch.isnan(want)].double(), want[~torch.isnan(want)])
    rest = [t for t in range(T) if t not in (3, 5)]
    assert torch.isfinite(h[rest]).all()
    mobi.mobi_sync_check()
