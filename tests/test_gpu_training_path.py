"""The norm, the layer, its backward, the norm's backward and the update of the expert weights, run together as a training
step runs them."""
import numpy as np
import pytest
import torch

import grouped_expert_ffn_router_amd as m
import moe_inputs
from test_gpu_graph import _capture_and_check, _dev
from test_gpu_orthogonalize import check as check_orthogonal, definition

pytestmark = pytest.mark.gpu
U32 = 2.0**-24


def build(dtype, norm, train, T=200, H=256, E=6, k=2, F=384, seed=11, form=None, bias=None):
    wl = moe_inputs.Workload("step", T=T, H=H, E=E, k=k, F=F, dtype=dtype, logits="gauss", seed=seed)
    inp = moe_inputs.make_inputs(wl)
    tdt = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}[dtype]
    sc = [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
          for a in (inp.s_gate, inp.s_up, inp.s_down)]
    w = [_dev(a, dtype) for a in (inp.w_gate, inp.w_up, inp.w_down)]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rdt = torch.bfloat16 if dtype == "fp8" else tdt
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    nw = (1 + 0.2 * rnd(H)).to(rdt)
    nb = (0.1 * rnd(H)).to(rdt) if (norm == "layer" if bias is None else bias) else None
    layer = m.MoELayer(T, H, E, k, F, tdt, *w, *sc, train=train, form=form, norm=norm, norm_weight=nw, norm_bias=nb)
    plain = m.MoELayer(T, H, E, k, F, tdt, *w, *sc, form=form)
    x, res = (1 + rnd(T, H)).to(rdt), rnd(T, H).to(rdt)
    return layer, plain, x, res, rnd(H, E) / H**0.5, rnd


@pytest.mark.parametrize("dtype,norm,form", [("bf16", "rms", "permuted"), ("fp8", "rms", "gather"), ("fp8", "layer", "fused"),
                                             ("f32", "layer", "permuted")])
def test_forward_x_is_the_calls_in_a_row(dtype, norm, form):
    layer, plain, x, res, wr, _ = build(dtype, norm, False, form=form)
    out = layer.forward_x(x, wr, residual=res).clone()
    n = m.moe_norm(x, layer.norm_weight, layer.norm_bias, res, norm,
                   out_dtype=torch.uint8 if dtype == "fp8" else None)
    assert torch.equal(layer.norm_rows, n.sum) and torch.equal(layer.xn, n.y)
    want = plain.forward_x(n.y, wr, x_scales=n.y_scales)
    assert torch.equal(out, want) and torch.equal(layer.topk_idx, plain.topk_idx)
    with pytest.raises(ValueError, match="norm"):
        plain.forward_x(n.y, wr, x_scales=n.y_scales, residual=res)


def test_gradients_of_a_step():
    """Loss <out, dout> + <rows, dsum> of an fp32 layer: the gradients against autograd in 64 bits on the CPU with the same
    picks.  Each of the five products between the rows and their gradient adds at most K <= 2 F terms in fp32, off by at
    most K 2^-24 of the sum of their magnitudes, which for values of random sign is about sqrt(K) times the result:
    5 K^1.5 2^-24 bounds the relative error in norm."""
    layer, _, x, res, wr, rnd = build("f32", "layer", True)
    T, H, E, k, F = layer.T, layer.H, layer.E, layer.k, layer.F
    xn, _ = layer.normalize(x, res)
    layer.route_x(xn, wr)
    layer.dispatch(xn)
    layer.forward_train()
    layer.combine()
    dout, dsum = rnd(T, H), rnd(T, H)
    g = layer.backward(dout)
    ng = layer.normalize_backward(g["dx"] + g["d_logits"] @ wr.T, dsum)
    up = layer.orthogonalize(out_dtype=torch.float32)
    torch.cuda.synchronize()

    c = lambda t: t.detach().double().cpu()  # noqa: E731
    X = (c(x + res)).requires_grad_()
    nw, nb = c(layer.norm_weight).requires_grad_(), c(layer.norm_bias).requires_grad_()
    W = [c(t).requires_grad_() for t in layer.w_nat]
    z = X - X.mean(1, keepdim=True)
    n = z / torch.sqrt((z * z).mean(1, keepdim=True) + 1e-5) * nw + nb
    logits = n @ c(wr)
    idx = layer.topk_idx.cpu().long()
    w = torch.softmax(logits.gather(1, idx), 1)
    out = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        h = torch.nn.functional.silu(n[t] @ W[0][e]) * (n[t] @ W[1][e])
        out = out.index_add(0, t, w[t, j, None] * (h @ W[2][e]))
    ((out * c(dout)).sum() + (X * c(dsum)).sum()).backward()
    tol = 5 * (2 * F) ** 1.5 * U32
    for name, got, want in (("out", layer.out, out.detach()), ("dx", ng["dx"], X.grad), ("dweight", ng["dweight"], nw.grad),
                            ("dbias", ng["dbias"], nb.grad), ("dw_gate", g["dw_gate"], W[0].grad),
                            ("dw_up", g["dw_up"], W[1].grad), ("dw_down", g["dw_down"], W[2].grad)):
        assert float((c(got) - want).norm() / want.norm()) <= tol, name
    for name in ("w_gate", "w_up", "w_down"):
        # an expert's gradient has at most its rows' rank: about 400 / 6 of 256, so the bound of low ranks is the one that holds
        check_orthogonal(up[name], definition(g["d" + name]), low_rank=True)


def test_updates_of_another_type_leave_a_captured_call_alone():
    layer, _, x, res, wr, rnd = build("f32", "layer", True)
    for g in layer.grads.values():
        g.copy_(torch.randn_like(g))
    first = layer.orthogonalize(out_dtype=torch.bfloat16)
    pointers = {k: u.data_ptr() for k, u in first.items()}
    other = layer.orthogonalize(out_dtype=torch.float32)
    again = layer.orthogonalize(out_dtype=torch.bfloat16)
    assert {k: u.data_ptr() for k, u in again.items()} == pointers
    assert not set(pointers.values()) & {u.data_ptr() for u in other.values()}
    assert other["w_gate"].dtype == torch.float32 and layer.updates is again


def test_step_in_one_graph():
    layer, _, x, res, wr, rnd = build("bf16", "rms", True, T=512, H=512, E=4, F=512)
    dout = rnd(512, 512).bfloat16()

    def step():
        xn, _ = layer.normalize(x, res)
        layer.route_x(xn, wr)
        layer.dispatch(xn)
        layer.forward_train()
        layer.combine()
        g = layer.backward(dout)
        layer.normalize_backward(g["dx"], dout)
        layer.orthogonalize()

    step()
    _capture_and_check(step, lambda: [layer.out, layer.norm_grads["dx"], layer.norm_grads["dweight"],
                                      layer.updates["w_gate"], layer.updates["w_up"], layer.updates["w_down"]])


def test_small_batches_in_one_graph():
    """The one-launch form of narrow matrices and the shared tiles, captured."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    gs = [torch.randn(s, generator=g, device="cuda") for s in ((8, 128, 256), (2, 333, 1001), (4, 1536, 1024))]
    outs = [torch.empty(t.shape, device="cuda", dtype=dt) for t, dt in zip(gs, (torch.float32, torch.float32, torch.bfloat16))]
    ws = [torch.empty(m.moe_orthogonalize_workspace_bytes(*t.shape, o.dtype), dtype=torch.uint8, device="cuda")
          for t, o in zip(gs, outs)]

    def step():
        for t, o, w in zip(gs, outs, ws):
            m.moe_orthogonalize(t, out=o, workspace=w)

    _capture_and_check(step, lambda: outs)


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, give the bits of one after the other."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    a = torch.randn((3, 300, 700), generator=g, device="cuda")
    b = torch.randn((3, 700, 300), generator=g, device="cuda")
    want = [m.moe_orthogonalize(t) for t in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [m.moe_orthogonalize(t, stream=s) for t, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_a_norm_without_training_and_back():
    layer, plain, x, res, _, _ = build("bf16", "rms", False)
    layer.normalize(x)
    assert layer.norm_rows is x
    for call in (lambda: layer.normalize_backward(x), layer.orthogonalize, lambda: plain.normalize(x)):
        with pytest.raises(ValueError):
            call()
    trained = build("bf16", "rms", True)[0]
    with pytest.raises(ValueError, match="follows"):
        trained.normalize_backward(x)
