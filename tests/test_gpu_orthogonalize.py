"""Orthogonalised updates against the definition in 64 bits.

Tolerances.  Operands of the products are rounded by at most h = 2^-11 of their value (fp16), or 2^-22 as hi + lo.  Rounding
errors are even over the interval and independent, so a rounded matrix is off by about 0.4 h of its norm.  A step's result
takes |B| <= 2.81 of X's rounding (b s^2 + c s^4 is at most b^2 / (4 c) in size), as much of B's, and through B = b A + c A A
those of A: |b| 1.46 sqrt(3) 0.4 h (A = X X^T with |X|^2 <= 1.46, two operands and its own rounding).  Together
sqrt(2 (2.81 * 0.4)^2 + (4.775 * 1.46 * 0.69)^2) h = 5.1 h a step; the derivative of the step's map is below 1.2 in size over
most of [0.68, 1.21], where the values are from the second or third step on, so two to three steps' errors add: 12 h, and
the tests allow 16 h of the result's norm, plus the result's own rounding (2^-8 bf16, 2^-24 fp32 at most).  fp32 accumulation
over K terms adds about sqrt(K) 2^-24 of the same kind: (16 + sqrt(K)) 2^-22 for fp32 results.
A single value is held to 10 times that on the root mean square: the largest of 10^6 normal values is 4.9 deviations.
Low ranks: X itself keeps 22 bits; what rounding leaves outside the rank grows by a = 3.4445 a step, 485 in five, to at most
485 * 2^-23 = 6e-5 of the norm.
Values near zero: X is held in units of 2^-24 (fp16's smallest step) / 2^12, so each value of X_0 is off by at most 2^-37
whatever its size, and the result by at most 485 * 2^-37 sqrt(m n) in norm.  That shows where |g| is far below eps (a
gradient of 1e-36 gives 1e-26 by the definition and 0 here).
"""
import pytest
import torch

import grouped_expert_ffn_router_amd as m

pytestmark = pytest.mark.gpu
COEFFS = m.ORTHOGONALIZE_COEFFS


def normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def definition(g, steps=5, coeffs=COEFFS, eps=1e-7):
    a, b, c = coeffs
    out = []
    for x in g.double():
        x = x / (x.norm() + eps)
        flip = x.shape[0] > x.shape[1]
        x = x.T.contiguous() if flip else x
        for _ in range(steps):
            A = x @ x.T.contiguous()
            x = a * x + (b * A + c * A @ A) @ x
        out.append(x.T.contiguous() if flip else x)
    return torch.stack(out)


def tolerance(out_dtype, q, low_rank=False):
    if out_dtype == torch.bfloat16:
        return 16 * 2.0**-11 + 2.0**-8
    return (16 + q**0.5) * 2.0**-22 + (485 * 2.0**-22 if low_rank else 0)


def check(got, want, low_rank=False):
    tol = tolerance(got.dtype, max(got.shape[1:]), low_rank)
    err = got.double() - want
    for e, w in zip(err, want):
        floor = 485 * 2.0**-37
        assert float(e.norm()) <= tol * float(w.norm()) + floor * w.numel() ** 0.5
        rms = float(w.norm()) / w.numel() ** 0.5
        assert float((e.abs() - 10 * tol * torch.clamp(w.abs(), min=rms)).max()) <= 10 * floor


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("g_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,mm,n", [(1, 1, 1), (2, 1, 9), (2, 7, 1), (1, 64, 64), (8, 128, 256), (3, 129, 257),
                                    (2, 333, 100), (2, 100, 333), (1, 640, 512), (5, 130, 96)])
def test_sizes(B, mm, n, g_dtype, out_dtype):
    g = (normal(B + mm + n, B, mm, n) * 0.01).to(g_dtype)
    check(m.moe_orthogonalize(g, out_dtype=out_dtype), definition(g))


@pytest.mark.parametrize("B,mm,n,out_dtype", [(4, 2048, 2048, torch.bfloat16), (70, 512, 520, torch.bfloat16),
                                              (40, 384, 1000, torch.float32), (26, 1300, 520, torch.bfloat16),
                                              (70, 128, 1000, torch.bfloat16), (70, 1000, 100, torch.float32),
                                              (90, 60, 2000, torch.float32), (33, 192, 1100, torch.bfloat16),
                                              (1, 1700, 5000, torch.bfloat16), (1, 5000, 1100, torch.float32)])
def test_large_tiles(B, mm, n, out_dtype):
    """Every tile size, whole and shared tiles, the one-launch form of narrow matrices and the sizes past it."""
    g = normal(1, B, mm, n) * 1e-3
    out = m.moe_orthogonalize(g, out_dtype=out_dtype)
    check(out, definition(g))


# sides and batches for which tiles of 256 x 192 leave the least of a last round empty
@pytest.mark.parametrize("B,mm,n", [(4, 768, 4090), (4, 4090, 768), (1, 2301, 4000), (2, 1500, 4096)])
def test_rectangular_tiles(B, mm, n):
    g = normal(2, B, mm, n) * 0.02
    check(m.moe_orthogonalize(g, out_dtype=torch.bfloat16), definition(g))


# One step with b = c = 0 gives a X_0.  a = 1 + 2^-11 is halfway between two fp16 values: with B rounded to fp16 alone every
# value comes out 2^-11 too small.  The errors' mean along the result shows it, for what single roundings add to it is small:
# 0.41 * 2^-8 of a value each over N normal values is sqrt(3 / N) 0.41 2^-8, 1.2e-5 at N = 60 000; five of these are 2^-14.
# The last product's X is the fp16 hi part, though, and 11 bits rounded to bf16's 8 are not even: a value m 2^e (1 <= m < 2)
# lies at k / 8 of a bf16 step (2^-7 2^e), k = 0 .. 7 equally likely, and a moves it on by f / 8, f = m / 2.  Those with
# k >= 4 round up, the others down: (4 - 8 f) / 64 of a step on average, (1 - m) / 16, which is (m - 1) / m 2^-11 of the value
# and at most 2^-12.  So 2^-12 + 2^-14 (3.1e-4) is allowed, and a rounded a is 4.9e-4 off.
@pytest.mark.parametrize("B,mm,n", [(16, 60, 1000), (64, 1000, 60), (64, 128, 500), (40, 1000, 100), (33, 192, 1100),
                                    (20, 1100, 192), (6, 512, 2048), (6, 2000, 512), (4, 768, 4090), (4, 4090, 768),
                                    (4, 2048, 2048), (1, 363, 3263)])
def test_a_is_not_rounded_with_the_diagonal(B, mm, n):
    a = 1 + 2.0**-11
    g = normal(8, B, mm, n)
    got = m.moe_orthogonalize(g, steps=1, coeffs=(a, 0.0, 0.0), out_dtype=torch.bfloat16).double()
    for e, x in zip(got, g.double()):
        w = a * x / (x.norm() + 1e-7)
        assert abs(float(((e - w) * w).sum() / (w * w).sum())) <= 2.0**-12 + 2.0**-14


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rank", [1, 3, 40])
def test_low_rank(rank, out_dtype):
    g = torch.matmul(normal(rank, 3, 200, rank), normal(rank + 1, 3, rank, 520))
    check(m.moe_orthogonalize(g, out_dtype=out_dtype), definition(g), low_rank=True)


def test_spectrum_and_zeros():
    """Singular values over four decades, matrices of zeros, with one value, and with rows of zeros (which stay)."""
    g = torch.zeros(5, 160, 224, device="cuda")
    g[0] = normal(1, 160, 160) @ torch.diag(torch.logspace(0, -4, 160, device="cuda")) @ normal(2, 160, 224)
    g[2, 3, 5] = -2.5
    g[3] = normal(3, 160, 224)
    g[3, 10:50] = 0
    g[4] = normal(4, 160, 224) * 1e-38
    for dt in (torch.bfloat16, torch.float32):
        out = m.moe_orthogonalize(g, out_dtype=dt)
        check(out, definition(g), low_rank=True)
        assert (out[1] == 0).all() and (out[3, 10:50] == 0).all()
        assert (out[2] != 0).sum() == 1


def test_large_and_small_gradients():
    """|g| past the range where fp32 squares hold."""
    g = normal(1, 3, 96, 160)
    want = definition(g, eps=1e-40)
    for f in (1e30, 1e-30):
        check(m.moe_orthogonalize(g * f, eps=1e-40), want)
    check(m.moe_orthogonalize(g * 1e-9), definition(g * 1e-9))  # |g| near eps


def test_infinities_stay_in_their_matrix():
    g = normal(1, 4, 130, 200)
    clean = m.moe_orthogonalize(g)
    g2 = g.clone()
    g2[1, 5, 6] = float("inf")
    g2[3, 100, 0] = float("nan")
    out = m.moe_orthogonalize(g2)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    assert torch.isnan(out[1]).all() and torch.isnan(out[3]).all()


@pytest.mark.parametrize("steps,coeffs", [(1, COEFFS), (2, (1.5, -0.5, 0.0)), (10, (1.875, -1.25, 0.375)),
                                          (7, (1.5, -0.5, 0.0))])
def test_steps_and_coefficients(steps, coeffs):
    g = normal(2, 2, 120, 180)
    check(m.moe_orthogonalize(g, steps=steps, coeffs=coeffs), definition(g, steps, coeffs))


def test_orthogonal_in_the_limit():
    """With the convergent coefficients the result's rows are orthonormal: |O O^T - 1| within the operands' rounding."""
    g = normal(3, 2, 96, 400)
    o = m.moe_orthogonalize(g, steps=14, coeffs=(1.5, -0.5, 0.0), out_dtype=torch.float32).double()
    gram = torch.matmul(o, o.transpose(1, 2).contiguous())
    # O's relative error (16 + 20) 2^-22, twice, in units of |1|_F = sqrt(96)
    assert float((gram - torch.eye(96, device="cuda", dtype=torch.float64)).norm(dim=(1, 2)).max()) <= 2 * 36 * 2.0**-22 * 96**0.5


def test_scale_and_one_matrix():
    g = normal(4, 90, 140)
    one = m.moe_orthogonalize(g, out_dtype=torch.float32)
    assert one.shape == g.shape
    check(one[None], definition(g[None]))
    check(m.moe_orthogonalize(g, scale=-0.02, out_dtype=torch.float32)[None], -0.02 * definition(g[None]))
    assert (m.moe_orthogonalize(g, scale=0.0) == 0).all()


def test_canaries_repeats_and_unaligned():
    """Nothing around out is written, results repeat bit for bit, unaligned inputs and outputs give the same bits, and
    what the workspace held does not matter."""
    B, mm, n = 3, 70, 136
    g = normal(5, B, mm, n)
    want = m.moe_orthogonalize(g)
    ws = torch.full((m.moe_orthogonalize_workspace_bytes(B, mm, n),), 255, dtype=torch.uint8, device="cuda")
    for off in (0, 1, 8):
        buf = torch.full((B * mm * n + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
        src = torch.empty(B * mm * n + 8, device="cuda")
        gi = src[off % 8:off % 8 + B * mm * n].view(B, mm, n).copy_(g)
        out = buf[16 + off:16 + off + B * mm * n].view(B, mm, n)
        m.moe_orthogonalize(gi, out=out, workspace=ws)
        assert torch.equal(out, want)
        assert (buf[:16 + off] == 9).all() and (buf[16 + off + B * mm * n:] == 9).all()
    flip = g.transpose(1, 2).contiguous()
    o = m.moe_orthogonalize(flip)
    check(o, definition(flip))


@pytest.mark.parametrize("B,mm,n,dt", [(2, 60, 300, torch.float32), (8, 128, 256, torch.bfloat16),
                                       (20, 128, 2000, torch.float32), (3, 1001, 333, torch.float32),
                                       (4, 512, 512, torch.bfloat16), (1, 1536, 2100, torch.bfloat16),
                                       (9, 1300, 1000, torch.bfloat16), (5, 1100, 1030, torch.float32)])
def test_workspace_is_enough(B, mm, n, dt):
    """The bytes behind the workspace stay, and the result does not depend on what the workspace held."""
    g = normal(8, B, mm, n)
    need = m.moe_orthogonalize_workspace_bytes(B, mm, n, dt)
    assert need % 256 == 0
    outs = []
    for fill in (0, 255):
        buf = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        outs.append(m.moe_orthogonalize(g, out_dtype=dt, workspace=buf[:need]))
        assert (buf[need:] == fill).all()
    assert torch.equal(*outs)
    check(outs[0], definition(g))


def test_batches_are_independent():
    g = normal(6, 6, 150, 140)
    a = m.moe_orthogonalize(g)
    p = torch.tensor([3, 0, 5, 1, 4, 2], device="cuda")
    assert torch.equal(m.moe_orthogonalize(g[p].contiguous()), a[p])
    assert m.moe_orthogonalize(g[:0]).shape == (0, 150, 140)


def test_refusals_on_the_gpu():
    g = normal(7, 2, 64, 64)
    with pytest.raises(ValueError, match="overlap"):
        m.moe_orthogonalize(g, out=g)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        m.moe_orthogonalize(g, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        m.moe_orthogonalize(g, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="bounded"):
        m.moe_orthogonalize(g, coeffs=(3.0, 0.0, 0.0))
