"""The norm's and the orthogonalised update's entry points reject bad arguments on the host, before anything reaches
the GPU (CPU only: no compute call is made here)."""
import ctypes

import pytest
import torch

import grouped_expert_ffn_router_amd as m

L = m.lib
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x10002)
BIG = ctypes.c_void_p(0x100000)
F32, BF16, FP8 = m.MOE_DTYPE_F32, m.MOE_DTYPE_BF16, m.MOE_DTYPE_FP8_E4M3


def norm(**k):
    return L.moe_norm(k.get("x", FAKE), k.get("ldx", 256), k.get("res"), k.get("ldr", 256), k.get("dt", BF16),
                      k.get("T", 10), k.get("H", 256), k.get("kind", 0), k.get("w", FAKE), k.get("b"),
                      k.get("wdt", BF16), k.get("eps", 1e-5), k.get("sum"), k.get("y", FAKE), k.get("ys"),
                      k.get("ydt", BF16), k.get("mean", FAKE), k.get("rstd", FAKE), None)


def back(**k):
    return L.moe_norm_backward(k.get("dy", FAKE), k.get("ld_dy", 256), k.get("s", FAKE), k.get("ld_s", 256),
                               k.get("dsum"), k.get("ld_ds", 256), k.get("dt", BF16), k.get("T", 10), k.get("H", 256),
                               k.get("kind", 0), k.get("w", FAKE), k.get("wdt", BF16), k.get("mean", FAKE),
                               k.get("rstd", FAKE), k.get("dx", FAKE), k.get("dw", FAKE), k.get("db"),
                               k.get("ws", BIG), k.get("wsb", 1 << 30), None)


def orth(**k):
    return L.moe_orthogonalize(k.get("g", FAKE), k.get("dt", F32), k.get("B", 2), k.get("m", 64), k.get("n", 96),
                               k.get("steps", 5), *k.get("coeffs", m.ORTHOGONALIZE_COEFFS), k.get("eps", 1e-7),
                               k.get("scale", 1.0), k.get("out", FAKE), k.get("odt", BF16), k.get("ws", BIG),
                               k.get("wsb", 1 << 30), None)


@pytest.mark.parametrize("bad,says", [
    (dict(dt=7), "dtype"), (dict(wdt=7), "dtype"), (dict(ydt=9), "dtype"), (dict(kind=2), "kind"), (dict(T=-1), "T ="),
    (dict(T=1 << 31), "T ="), (dict(H=0), "H ="), (dict(H=65537, ldx=65537), "H ="), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(ldx=255), "stride"),
    (dict(ldx=1 << 31), "stride"), (dict(res=FAKE, ldr=255, sum=FAKE), "stride"), (dict(x=None), "x is NULL"),
    (dict(w=None), "weight"), (dict(y=None), "y is NULL"), (dict(res=FAKE), "sum is NULL"),
    (dict(dt=F32, ydt=F32, x=ODD), "aligned"), (dict(mean=ODD), "mean"), (dict(rstd=ODD), "rstd"),
    (dict(ydt=FP8), "y_scales"), (dict(ydt=FP8, H=250, ldx=256, ys=FAKE), "multiple of 128"),
    (dict(ydt=FP8, ys=FAKE, y=ODD), "16-byte"), (dict(ydt=FP8, ys=ODD), "y_scales"),
])
def test_norm_refuses(bad, says):
    assert norm(**bad) == m.MOE_ERR_INVALID_ARG
    assert says in L.moe_last_error().decode()


def test_norm_unsupported_and_empty():
    assert norm(dt=FP8) == m.MOE_ERR_UNSUPPORTED
    assert norm(wdt=FP8) == m.MOE_ERR_UNSUPPORTED
    assert norm(dt=F32) == m.MOE_ERR_UNSUPPORTED  # fp32 rows, bf16 result
    assert norm(T=0, x=None, w=None, y=None) == m.MOE_OK


@pytest.mark.parametrize("bad,says", [
    (dict(dt=7), "dtype"), (dict(kind=5), "kind"), (dict(T=-1), "T ="), (dict(H=0), "H ="), (dict(ld_dy=255), "stride"),
    (dict(ld_s=255), "stride"), (dict(dsum=FAKE, ld_ds=255), "stride"), (dict(dw=None), "dweight"),
    (dict(db=ODD), "dbias"), (dict(dy=None), "dy"), (dict(s=None), "s is NULL"), (dict(mean=None), "mean"),
    (dict(rstd=None), "rstd"), (dict(dx=None), "dx"), (dict(w=None), "weight"),
])
def test_norm_backward_refuses(bad, says):
    assert back(**bad) == m.MOE_ERR_INVALID_ARG
    assert says in L.moe_last_error().decode()


def test_norm_backward_workspace():
    need = m.moe_norm_backward_workspace_bytes(10, 256)
    assert need >= 2 * 256 * 4  # at least one partial row of each
    assert back(wsb=need - 1) == m.MOE_ERR_WORKSPACE
    assert back(ws=None) == m.MOE_ERR_WORKSPACE
    assert back(ws=ODD) == m.MOE_ERR_WORKSPACE
    assert back(dt=FP8) == m.MOE_ERR_UNSUPPORTED
    for T, H in ((-1, 256), (10, 0), (10, 1 << 17), (1 << 31, 256)):
        assert m.moe_norm_backward_workspace_bytes(T, H) == 0


@pytest.mark.parametrize("bad,says", [
    (dict(dt=7), "dtype"), (dict(odt=7), "dtype"), (dict(B=-1), "batch"), (dict(B=1 << 24), "batch"), (dict(m=0), "m ="),
    (dict(n=65537), "n ="), (dict(steps=0), "steps"), (dict(steps=33), "steps"), (dict(eps=0.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(scale=float("inf")), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(B=(1 << 24) - 1, m=65536, n=65536), "too large"),
    (dict(B=(1 << 22) + 1, m=100, n=65), "too large"),
    (dict(coeffs=(4.0, 0.0, 0.0)), "bounded"), (dict(coeffs=(2.0, 0.0, 0.0)), "bounded"),
    (dict(coeffs=(1.0, float("nan"), 0.0)), "bounded"), (dict(coeffs=(1.0, -20.0, 20.0)), "bounded"),
    (dict(g=None), "g is NULL"), (dict(out=None), "out"), (dict(g=ODD), "aligned"),
])
def test_orthogonalize_refuses(bad, says):
    assert orth(**bad) == m.MOE_ERR_INVALID_ARG
    assert says in L.moe_last_error().decode()


def test_orthogonalize_workspace_and_types():
    need = m.moe_orthogonalize_workspace_bytes(2, 64, 96)
    assert need > 0
    assert (m.moe_orthogonalize_workspace_bytes(4, 2048, 4096, torch.float32)
            > m.moe_orthogonalize_workspace_bytes(4, 2048, 4096))
    assert m.moe_orthogonalize_workspace_bytes(2, 96, 64) == need
    assert orth(wsb=need - 1) == m.MOE_ERR_WORKSPACE
    assert orth(ws=None) == m.MOE_ERR_WORKSPACE
    assert orth(ws=ODD) == m.MOE_ERR_WORKSPACE
    assert orth(dt=FP8) == m.MOE_ERR_UNSUPPORTED
    assert orth(odt=FP8) == m.MOE_ERR_UNSUPPORTED
    assert orth(B=0, g=None, out=None, ws=None) == m.MOE_OK
    for B, mm, n in ((-1, 4, 4), (1, 0, 4), (1, 4, 1 << 17)):
        assert m.moe_orthogonalize_workspace_bytes(B, mm, n) == 0
    # the coefficient sets in use: the usual one for any number of steps, and the convergent ones
    for steps in (1, 5, 10, 32):
        assert orth(steps=steps, g=None) == m.MOE_ERR_INVALID_ARG and "g is NULL" in L.moe_last_error().decode()
    for c in ((1.5, -0.5, 0.0), (1.875, -1.25, 0.375)):
        assert orth(coeffs=c, steps=32, g=None) == m.MOE_ERR_INVALID_ARG
        assert "g is NULL" in L.moe_last_error().decode()


def test_wrappers_refuse():
    x = torch.zeros(4, 256)
    w = torch.ones(256)
    cases = [
        (lambda: m.moe_norm(x, w), "on the GPU"),
        (lambda: m.moe_norm(x, w, kind="batch"), "kind"),
        (lambda: m.moe_norm(x[0], w), r"\[T, H\]"),
        (lambda: m.moe_norm(x.double(), w), "float32 or bfloat16"),
        (lambda: m.moe_norm(x, w[:255]), "weight has shape"),
        (lambda: m.moe_norm(x, torch.ones(512)[::2]), "contiguous"),
        (lambda: m.moe_norm(x, w, bias=w.bfloat16()), "bias has dtype"),
        (lambda: m.moe_norm(x.T, torch.ones(4)), "rows must be contiguous"),
        (lambda: m.moe_norm(torch.zeros(256).expand(4, 256), w), "overlap"),
        (lambda: m.moe_norm(x, w, residual=x.bfloat16()), "residual has dtype"),
        (lambda: m.moe_norm(x, w, residual=x[:3]), "residual has shape"),
        (lambda: m.moe_norm(x[:, :100], w[:100], out_dtype=torch.uint8), "multiple of 128"),
        (lambda: m.moe_norm(x, w, y=torch.zeros(4, 256), out_dtype=torch.uint8), "y has dtype"),
        (lambda: m.moe_norm_backward(x, x, w, None, torch.ones(4)), "means"),
        (lambda: m.moe_norm_backward(x, x, w, torch.ones(4), torch.ones(3)), "rstd has shape"),
        (lambda: m.moe_norm_backward(x[:, :8], x, w, torch.ones(4), torch.ones(4)), "dy has shape"),
        (lambda: m.moe_norm_backward(x, x, w, torch.ones(4), torch.ones(4)), "on the GPU"),
        (lambda: m.moe_orthogonalize(x), "on the GPU"),
        (lambda: m.moe_orthogonalize(x[0]), r"\[B, m, n\]"),
        (lambda: m.moe_orthogonalize(x.T), "contiguous"),
        (lambda: m.moe_orthogonalize(x.half()), "dtype"),
        (lambda: m.moe_orthogonalize(x, coeffs=(1.0, 2.0)), "three"),
        (lambda: m.moe_orthogonalize(x, out_dtype=torch.float16), "float32 or bfloat16"),
        (lambda: m.moe_orthogonalize(x, out=x, out_dtype=torch.bfloat16), "out has dtype"),
    ]
    for call, says in cases:
        with pytest.raises(ValueError, match=says):
            call()
    with pytest.raises(NotImplementedError):
        m.moe_norm(x, w, out_dtype=torch.bfloat16)


def test_layer_refuses():
    for kw, says in ((dict(norm="batch"), "norm"), (dict(norm="rms"), "norm_weight"),
                     (dict(norm_weight=torch.ones(256)), "need norm")):
        with pytest.raises(ValueError, match=says):
            m.MoELayer(4, 256, 2, 1, 256, torch.bfloat16, torch.zeros(2, 256, 256), None, None, **kw)
