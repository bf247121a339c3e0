"""The norm and its backward against the definition in 64 bits.

Bounds, from the kernels' arithmetic (u32 = 2^-24, half a step of fp32; u half a step of the stored type).  A sum of n
terms added in any order is off by at most n u32 sum|terms|; a row's sums have at most 64 terms per thread, then at most
6 + 16 exchanges, so n <= N = 96 covers them with the division and the products.
  mean:   N u32 mean|s|
  rstd:   the sum of squares has relative error N u32, an error d of the mean adds d^2 to it (the differences from the
          exact mean sum to zero), and sqrt and division round once each: r (N u32 + (r d)^2)
  y:      |w| r d + |z w| (rel(rstd) + 4 u32) + 2 u32 |y - b| + 2 u32 |b| + u |y|
  dx:     r N u32 (|t| + mean|t| + |z| mean|t z|) + u32 |dsum| + u |dx|, t = dy w
  dw, db: sums over rows: a workgroup adds at most T / 256 + 1 rows (256 workgroups or more, or one pass), 16 groups, and
          the partials in 32 + 32: (T / 256 + 112) u32 sum|dy z|.  Wide rows have 64 workgroups or more a column and no
          groups, T / 64 + 1 + 64 terms: less than that up to T = 4000
"""
import math

import pytest
import torch

import grouped_expert_ffn_router_amd as m

pytestmark = pytest.mark.gpu
U32 = 2.0**-24
N = 96
HALF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8}


def normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def forward64(x, w, b, residual, kind, eps):
    """y, the stored rows, mean, rstd and the bounds of the kernel's errors in them (before the rounding of y)."""
    s = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    v = s.double()
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros(len(v), 1, dtype=torch.float64, device=v.device)
    d = N * U32 * v.abs().mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(mean)
    r = 1 / torch.sqrt(((v - mean) ** 2).mean(1, keepdim=True) + eps)
    rel = N * U32 + (r * d) ** 2
    z = (v - mean) * r
    yw = z * w.double()
    y = yw + (0 if b is None else b.double())
    ey = w.double().abs() * r * d + yw.abs() * (rel + 6 * U32) + (0 if b is None else 2 * U32 * b.double().abs())
    return y, s, mean, r, ey, d, r * rel


def check_forward(r, x, w, b, residual, kind, eps):
    y, s, mean, rstd, ey, d, er = forward64(x, w, b, residual, kind, eps)
    if residual is not None:
        assert torch.equal(r.sum, s)
    if kind == "layer":
        assert ((r.mean.double() - mean[:, 0]).abs() <= d[:, 0] + U32 * mean[:, 0].abs()).all()
    assert ((r.rstd.double() - rstd[:, 0]).abs() <= er[:, 0] + U32 * rstd[:, 0]).all()
    if r.y_scales is None:
        bound = ey + HALF[r.y.dtype] * (y.abs() + ey) + 2.0**-149
        assert ((r.y.double() - y).abs() <= bound).all(), float(((r.y.double() - y).abs() / bound).max())
        return
    # codes: half a step (2^-4 of the value, 2^-10 below the normal range), after a division that rounds once
    codes = r.y.view(torch.float8_e4m3fn).double()
    T, H = y.shape
    amax = y.view(T, -1, 128).abs().amax(2)
    eb = ey.view(T, -1, 128).amax(2)
    sc = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    assert ((r.y_scales.double() - sc).abs() <= eb / 448 + 2 * U32 * sc).all()
    scale = r.y_scales.double().repeat_interleave(128, 1)
    bound = (2.0**-4 + 4 * U32) * y.abs() + 2.0**-10 * scale + 1.1 * ey + 448 * (scale - sc.repeat_interleave(128, 1)).abs()
    assert ((codes * scale - y).abs() <= bound).all()


CASES = [  # T, H, rows, weights, kind, bias, residual
    (1, 1, torch.float32, torch.float32, "layer", True, False),
    (1, 7168, torch.bfloat16, torch.bfloat16, "rms", False, True),
    (5, 8, torch.bfloat16, torch.float32, "layer", True, True),
    (17, 13, torch.float32, torch.bfloat16, "rms", True, False),
    (33, 128, torch.float32, torch.float32, "layer", True, True),
    (300, 256, torch.bfloat16, torch.bfloat16, "layer", True, False),
    (129, 264, torch.bfloat16, torch.float32, "rms", False, True),
    (70, 1000, torch.bfloat16, torch.bfloat16, "layer", False, True),
    (1001, 1537, torch.float32, torch.float32, "layer", True, True),
    (65, 2047, torch.bfloat16, torch.bfloat16, "layer", True, True),
    (40, 2048, torch.float32, torch.bfloat16, "rms", False, False),
    (2049, 4096, torch.bfloat16, torch.bfloat16, "layer", True, True),
    (66, 5120, torch.bfloat16, torch.float32, "layer", True, False),
    (20, 8192, torch.float32, torch.float32, "rms", False, True),
    (7, 12289, torch.bfloat16, torch.bfloat16, "layer", True, False),
    (600, 9000, torch.float32, torch.bfloat16, "layer", True, True),
    (9, 16381, torch.bfloat16, torch.float32, "rms", False, True),
    (21, 1111, torch.bfloat16, torch.bfloat16, "layer", True, True),
    (30, 3000, torch.bfloat16, torch.float32, "layer", True, False),
    (11, 6144, torch.bfloat16, torch.bfloat16, "rms", False, True),
    (5, 9216, torch.bfloat16, torch.bfloat16, "layer", True, True),
    (3, 10240, torch.float32, torch.float32, "rms", False, True),
    (500, 17000, torch.bfloat16, torch.float32, "layer", True, True),
    (9, 16384, torch.bfloat16, torch.bfloat16, "rms", False, True),
    (3, 16392, torch.bfloat16, torch.bfloat16, "layer", True, True),
    (2, 65536, torch.float32, torch.float32, "layer", True, False),
    (2, 65535, torch.bfloat16, torch.bfloat16, "layer", True, False),
]


def inputs(T, H, dt, wdt, bias, residual, seed=3):
    x = (normal(seed, T, H) * torch.exp(normal(seed + 1, T, 1)) + 2 * normal(seed + 2, H)).to(dt)
    w = (1 + 0.3 * normal(seed + 3, H)).to(wdt)
    b = normal(seed + 4, H).to(wdt) if bias else None
    res = normal(seed + 5, T, H).to(dt) if residual else None
    return x, w, b, res


@pytest.mark.parametrize("T,H,dt,wdt,kind,bias,residual", CASES)
def test_forward(T, H, dt, wdt, kind, bias, residual):
    x, w, b, res = inputs(T, H, dt, wdt, bias, residual)
    check_forward(m.moe_norm(x, w, b, res, kind, 1e-5), x, w, b, res, kind, 1e-5)


@pytest.mark.parametrize("T,H,dt,kind,bias,residual", [
    (1, 128, torch.bfloat16, "rms", False, False), (37, 128, torch.float32, "layer", True, True),
    (130, 384, torch.bfloat16, "layer", True, True), (64, 7168, torch.bfloat16, "rms", False, True),
    (19, 2176, torch.float32, "rms", False, False), (12, 5120, torch.bfloat16, "layer", True, True),
    (3, 16512, torch.bfloat16, "layer", True, False),
    (2, 32896, torch.float32, "rms", False, True)])
@pytest.mark.parametrize("code", [torch.uint8, torch.float8_e4m3fn])
def test_forward_to_e4m3(T, H, dt, kind, bias, residual, code):
    x, w, b, res = inputs(T, H, dt, dt, bias, residual)
    w[:128] = 0  # a block of zeros has scale 1 (the bias alone, where there is one)
    r = m.moe_norm(x, w, b, res, kind, 1e-5, out_dtype=code)
    assert r.y.dtype == code
    check_forward(r, x, w, b, res, kind, 1e-5)
    if not bias:
        assert (r.y_scales[:, 0] == 1).all() and (r.y.view(torch.uint8)[:, :128] & 0x7F == 0).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_strides_offsets_and_canaries(dt):
    """Rows of a wider buffer, at every alignment, give the bits of their contiguous copies; nothing around the outputs
    is written."""
    T, H = 37, 520
    wide = normal(5, T, 2 * H + 40).to(dt)
    w, b = normal(6, H).to(dt), normal(7, H).to(dt)
    ref = {}
    for off in (0, 8, 1, 3):
        x, res = wide[:, off:off + H], wide[:, H + 20 + off:2 * H + 20 + off]
        buf = torch.full((T * H + 64,), -7.0, device="cuda", dtype=dt)
        y = buf[32:32 + T * H].view(T, H)
        r = m.moe_norm(x, w, b, res, "layer", 1e-5, y=y)
        check_forward(r, x, w, b, res, "layer", 1e-5)
        assert (buf[:32] == -7).all() and (buf[32 + T * H:] == -7).all()
        c = m.moe_norm(x.contiguous(), w, b, res.contiguous(), "layer", 1e-5)
        assert torch.equal(c.y, r.y) and torch.equal(c.rstd, r.rstd)
        ref[off] = r
        dbuf = torch.full((T * H + 64,), -7.0, device="cuda", dtype=dt)
        out = dict(dx=dbuf[32:32 + T * H].view(T, H), dweight=torch.empty(H, device="cuda"),
                   dbias=torch.empty(H, device="cuda"))
        m.moe_norm_backward(res, r.sum, w, r.mean, r.rstd, dsum=x, out=out)
        assert (dbuf[:32] == -7).all() and (dbuf[32 + T * H:] == -7).all()
        check_backward(out, res, r.sum, w, r.mean, r.rstd, "layer", x)


def test_unaligned_rows_to_e4m3():
    T, H = 21, 384
    wide = normal(4, T, 2 * H + 30).bfloat16()
    w = normal(6, H + 1).bfloat16()[1:]
    x, res = wide[:, 1:1 + H], wide[:, H + 7:2 * H + 7]
    r = m.moe_norm(x, w, residual=res, kind="rms", out_dtype=torch.uint8)
    check_forward(r, x, w, None, res, "rms", 1e-5)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_aligned_strides_keep_the_bits(dt):
    T, H = 37, 520
    wide = normal(8, T, 2 * H + 48).to(dt)
    w, b = normal(6, H).to(dt), normal(7, H).to(dt)
    x, res = wide[:, 8:8 + H], wide[:, H + 24:2 * H + 24]
    r, c = m.moe_norm(x, w, b, res), m.moe_norm(x.contiguous(), w, b, res.contiguous())
    assert torch.equal(r.y, c.y) and torch.equal(r.sum, c.sum) and torch.equal(r.rstd, c.rstd)
    a = m.moe_norm_backward(res, r.sum, w, r.mean, r.rstd, dsum=x)
    d = m.moe_norm_backward(res.contiguous(), r.sum, w, r.mean, r.rstd, dsum=x.contiguous())
    assert all(torch.equal(a[k], d[k]) for k in a)


def test_in_place_sum_and_gradient():
    T, H = 50, 1024
    x, w, b, res = inputs(T, H, torch.bfloat16, torch.bfloat16, True, True)
    want = m.moe_norm(x, w, b, res)
    for alias in ("x", "residual"):
        x2, r2 = x.clone(), res.clone()
        got = m.moe_norm(x2, w, b, r2, sum=x2 if alias == "x" else r2)
        assert torch.equal(got.y, want.y) and torch.equal(got.sum, want.sum) and torch.equal(got.rstd, want.rstd)
    dy, ds = normal(1, T, H).bfloat16(), normal(2, T, H).bfloat16()
    ref = m.moe_norm_backward(dy, want.sum, w, want.mean, want.rstd, dsum=ds)
    for alias in ("dy", "dsum"):
        dy2, ds2 = dy.clone(), ds.clone()
        out = dict(dx=dy2 if alias == "dy" else ds2, dweight=torch.empty(H, device="cuda"),
                   dbias=torch.empty(H, device="cuda"))
        m.moe_norm_backward(dy2, want.sum, w, want.mean, want.rstd, dsum=ds2, out=out)
        assert all(torch.equal(out[k], ref[k]) for k in ref)


def test_rows_of_extremes():
    """Constant rows, rows far from zero, tiny and huge rows, and rows with infinities or NaN, which stay in their own
    row."""
    H = 640
    x = normal(9, 10, H)
    x[1] = 0
    x[2] = 3.0
    x[3] = x[3] * 1e-3 + 1e4
    x[4] *= 1e-30
    x[5] *= 1e15
    x[6, 5] = float("inf")
    x[7, 600] = float("nan")
    x[8, 0] = float("-inf")
    w, b = 1 + 0.1 * normal(10, H), normal(11, H)
    fine = [0, 1, 2, 3, 4, 5, 9]
    for kind in ("layer", "rms"):
        r = m.moe_norm(x, w, b, kind=kind)
        f = m.moe_norm(x[fine], w, b, kind=kind)
        assert torch.equal(r.y[fine], f.y) and torch.isfinite(f.y).all()
        check_forward(f, x[fine], w, b, None, kind, 1e-5)
        if kind == "layer":
            assert torch.equal(f.y[1], b) and torch.isnan(r.y[6:9]).all()
        else:  # an infinity makes rstd 0: NaN at its own place, the bias elsewhere
            assert torch.isnan(r.y[7]).all() and torch.isnan(r.y[6, 5]) and torch.equal(r.y[6, 6:], b[6:])
        q = m.moe_norm(x, w, b, kind=kind, out_dtype=torch.float8_e4m3fn)
        assert torch.equal(torch.isnan(q.y.float()), torch.isnan(r.y)) and torch.isfinite(q.y_scales).all()
        out = m.moe_norm_backward(torch.ones_like(x), x, w, r.mean, r.rstd, kind)
        assert torch.isfinite(out["dx"][fine]).all()


def test_eps_zero_and_large():
    x, w = normal(1, 6, 256), torch.ones(256, device="cuda")
    for eps in (0.0, 1e-12, 10.0):
        check_forward(m.moe_norm(x, w, eps=eps), x, w, None, None, "layer", eps)


def backward64(dy, s, w, mean, rstd, kind, dsum):
    v, g, r = s.double(), dy.double(), rstd.double()[:, None]
    z = (v - (mean.double()[:, None] if kind == "layer" else 0)) * r
    t = g * w.double()
    c1 = t.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(r)
    c2 = (t * z).mean(1, keepdim=True)
    dx = r * (t - c1 - z * c2) + (0 if dsum is None else dsum.double())
    edx = r * N * U32 * (t.abs() + t.abs().mean(1, keepdim=True) + z.abs() * (t * z).abs().mean(1, keepdim=True))
    if dsum is not None:
        edx = edx + 2 * U32 * dsum.double().abs()
    n = (len(v) / 256 + 112) * U32
    return dx, (g * z).sum(0), g.sum(0), edx, n * (g * z).abs().sum(0), n * g.abs().sum(0)


def check_backward(out, dy, s, w, mean, rstd, kind, dsum):
    dx, dw, db, edx, ew, eb = backward64(dy, s, w, mean, rstd, kind, dsum)
    bound = edx + HALF[s.dtype] * (dx.abs() + edx) + 2.0**-149
    assert ((out["dx"].double() - dx).abs() <= bound).all(), float(((out["dx"].double() - dx).abs() / bound).max())
    assert ((out["dweight"].double() - dw).abs() <= ew + 2.0**-149).all()
    if out["dbias"] is not None:
        assert ((out["dbias"].double() - db).abs() <= eb + 2.0**-149).all()


@pytest.mark.parametrize("T,H,dt,wdt,kind,bias,residual", CASES)
def test_backward(T, H, dt, wdt, kind, bias, residual):
    x, w, b, res = inputs(T, H, dt, wdt, bias, residual)
    f = m.moe_norm(x, w, b, res, kind, 1e-5)
    dy = normal(20, T, H).to(dt)
    ds = normal(21, T, H).to(dt) if residual else None
    out = m.moe_norm_backward(dy, f.sum, w, f.mean, f.rstd, kind, ds, want_bias=bias)
    assert (out["dbias"] is not None) == bias
    check_backward(out, dy, f.sum, w, f.mean, f.rstd, kind, ds)
    again = m.moe_norm_backward(dy, f.sum, w, f.mean, f.rstd, kind, ds, want_bias=bias)
    assert all(out[k] is None or torch.equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward_against_differences(kind):
    """<dx, v> and <dw, u> against the change of L = <dy, y> along v and u, by differences of the 64-bit forward with two
    step lengths (h and h / 2; their disagreement bounds what is left of the h^2 term)."""
    T, H, eps = 6, 96, 1e-5
    x, w, b, _ = inputs(T, H, torch.float32, torch.float32, True, False)
    f = m.moe_norm(x, w, b, kind=kind, eps=eps)
    dy = normal(30, T, H)
    out = m.moe_norm_backward(dy, x, w, f.mean, f.rstd, kind, want_bias=True)

    def L(x64, w64, b64):
        c = x64 - x64.mean(1, keepdim=True) if kind == "layer" else x64
        y = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * w64 + b64
        return float((dy.double() * y).sum())

    _, _, _, edx, ew, eb = backward64(dy, x, w, f.mean, f.rstd, kind, None)
    x64, w64, b64 = x.double(), w.double(), b.double()
    # mean and rstd reach the kernel in fp32: relative changes of u32 in each move dx by a few u32 of its terms
    edx = 2 * edx + 8 * U32 * out["dx"].double().abs()
    for name, got, err, arg in (("x", out["dx"], edx, 0), ("w", out["dweight"], 2 * ew, 1), ("b", out["dbias"], 2 * eb, 2)):
        v = normal(40 + arg, *got.shape).double()
        def at(h):
            a = [x64, w64, b64]
            a[arg] = a[arg] + h * v
            return L(*a)
        d = [(at(h) - at(-h)) / (2 * h) for h in (1e-4, 5e-5)]
        want = d[1] + (d[1] - d[0]) / 3
        tol = float((err * v.abs()).sum()) + abs(d[1] - d[0]) + 1e-9 * float((dy.double().abs()).sum())
        assert abs(float((got.double() * v).sum()) - want) <= tol, name


def test_no_rows():
    w = torch.ones(256, device="cuda")
    x = torch.empty(0, 256, device="cuda")
    r = m.moe_norm(x, w)
    assert r.y.shape == (0, 256)
    out = dict(dx=torch.empty_like(x), dweight=torch.full((256,), 5.0, device="cuda"),
               dbias=torch.full((256,), 5.0, device="cuda"))
    m.moe_norm_backward(x, x, w, r.mean, r.rstd, out=out)
    assert (out["dweight"] == 0).all() and (out["dbias"] == 0).all()


@pytest.mark.parametrize("T,H", [(1, 64), (64, 128), (65, 128), (300, 1000), (9, 5000), (700, 2048), (33, 20000), (40, 12000)])
def test_workspace_is_enough(T, H):
    x, w, b, _ = inputs(T, H, torch.bfloat16, torch.bfloat16, True, False)
    f = m.moe_norm(x, w, b)
    dy = normal(60, T, H).bfloat16()
    need = m.moe_norm_backward_workspace_bytes(T, H)
    outs = []
    for fill in (0, 255):
        buf = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        outs.append(m.moe_norm_backward(dy, x, w, f.mean, f.rstd, workspace=buf[:need]))
        assert (buf[need:] == fill).all()
    assert all(torch.equal(outs[0][k], outs[1][k]) for k in outs[0])
    check_backward(outs[0], dy, x, w, f.mean, f.rstd, "layer", None)


def test_other_stream_and_two_calls():
    """Calls on two streams at once, each with its own workspace, give the results of one after the other."""
    T, H = 700, 2048
    x, w, b, _ = inputs(T, H, torch.bfloat16, torch.bfloat16, True, False)
    f = m.moe_norm(x, w, b)
    dys = [normal(50 + i, T, H).bfloat16() for i in range(2)]
    want = [m.moe_norm_backward(d, x, w, f.mean, f.rstd) for d in dys]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dys]
    got = [m.moe_norm_backward(d, x, w, f.mean, f.rstd, stream=s) for d, s in zip(dys, streams)]
    torch.cuda.synchronize()
    for a, c in zip(want, got):
        assert all(torch.equal(a[k], c[k]) for k in a)
    with pytest.raises(ValueError):
        m.moe_norm(x, w, stream=streams[0].cuda_stream)  # a raw handle: the caller passes every buffer


def test_e4m3_of_values_that_have_no_scale():
    """A block whose largest value / 448 is 0 in fp32 (below 448 * 2^-150) has scale 1, and codes of 0."""
    x = normal(31, 3, 256).bfloat16()
    w = torch.zeros(256, device="cuda")
    w[5], w[200] = 1e-43, 1.0
    r = m.moe_norm(x, w, kind="rms", out_dtype=torch.float8_e4m3fn)
    assert torch.equal(r.y_scales[:, 0], torch.ones(3, device="cuda"))
    assert (r.y.view(torch.uint8)[:, :128] & 0x7F == 0).all()
    assert (r.y.float()[:, 200].abs() == 448).all()


@pytest.mark.parametrize("H,residual", [(1, False), (3, True)])
def test_more_rows_than_one_grid_holds(H, residual):
    """16 threads a row, 2^28 rows and more: 2^32 threads.  Rows around the places where a grid may end, and the last ones."""
    T = (1 << 28) + 37
    x = torch.arange(T * H, device="cuda", dtype=torch.int32).remainder_(251).to(torch.bfloat16).view(T, H)
    w = torch.tensor([1.0, -2.0, 0.5], device="cuda")[:H].contiguous()
    b = None if residual else w + 1
    r = m.moe_norm(x, w, b, residual=x if residual else None, kind="rms", eps=1.0)
    for lo in (0, (1 << 27) - 20, (1 << 28) - 20, T - 40):
        rows = x[lo:lo + 40]
        want = m.moe_norm(rows, w, b, residual=rows if residual else None, kind="rms", eps=1.0)
        assert torch.equal(r.y[lo:lo + 40], want.y) and torch.equal(r.rstd[lo:lo + 40], want.rstd)
        if residual:
            assert torch.equal(r.sum[lo:lo + 40], want.sum)


def test_e4m3_scales_of_every_size():
    """Blocks from 1e-43 to 1e37: the codes are those of the same rows at 1, where the scale is the same power of two larger;
    NaN and infinities keep to their own codes and blocks."""
    x = normal(32, 40, 128)
    w = torch.ones(128, device="cuda")
    base = m.moe_norm(x, w, kind="rms", out_dtype=torch.uint8)
    for p in (-100, -90, -81, -79, -60, 60, 99, 101, 117):  # scales of about 2^-7: normal ones throughout
        r = m.moe_norm(x, w * 2.0**p, kind="rms", out_dtype=torch.uint8)
        assert torch.equal(r.y, base.y) and torch.equal(r.y_scales, base.y_scales * 2.0**p), p
    for f in (1e-43, 1e-40):  # y itself and the scale are a few of fp32's smallest steps
        r = m.moe_norm(x, w * f, kind="rms", out_dtype=torch.float8_e4m3fn)
        assert torch.isfinite(r.y.float()).all() and (r.y_scales > 0).all()
    w[7] = float("inf")
    r = m.moe_norm(x, w, kind="rms", out_dtype=torch.float8_e4m3fn)
    assert torch.isinf(r.y_scales).all() and torch.isnan(r.y[:, 7].float()).all()
    assert (r.y.float()[:, 8:] == 0).all()
    w[7] = float("nan")
    r = m.moe_norm(x, w, kind="rms", out_dtype=torch.uint8)
    assert (r.y[:, 7] & 0x7F == 0x7F).all() and (r.y[:, 8:] & 0x7F < 0x7F).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("base", [0, 16, 640, 2048])
def test_every_rest_of_a_row(base, dt):
    """Widths of each remainder by 8, rows that end where NaN begins: none of it is read into a row, and none is overwritten."""
    for H in range(base + 1, base + 10):
        T = 9
        wide = [torch.full((T, H + 3), float("nan"), device="cuda", dtype=dt) for _ in range(4)]
        x, res, dy, ds = (t[:, 1:H + 1] for t in wide)
        for k, t in enumerate((x, res, dy, ds)):
            t.copy_(normal(50 + k, T, H))
        w, b = normal(54, H).to(dt), normal(55, H).to(dt)
        f = m.moe_norm(x, w, b, res, "layer", 1e-5)
        check_forward(f, x, w, b, res, "layer", 1e-5)
        for kind, g in (("layer", f), ("rms", m.moe_norm(x, w, None, res, "rms", 1e-5))):
            out = m.moe_norm_backward(dy, g.sum, w, g.mean, g.rstd, kind, ds, want_bias=True)
            check_backward(out, dy, g.sum, w, g.mean, g.rstd, kind, ds)
        assert all(torch.isnan(t[:, 0]).all() and torch.isnan(t[:, H + 1:]).all() for t in wide)
