"""A router's training step as a user runs it: logits, general gates, grouping, experts, combine, and
back through the combine and the gates, against 64-bit automatic differentiation of the whole and
against differences of the loss."""
import numpy as np
import pytest
import torch

from mixture_experts_zero_b200 import binding as B
from mixture_experts_zero_b200 import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_router_gradient_of_the_layer(cuda_device, score, renorm):
    w = inputs.scaled(inputs.WORKLOADS["tiny"], T=50)
    t = inputs.make(w, device="cuda", grid=True)
    opts = dict(score=score, groups=4, top_groups=3, group_rank=2, renorm=renorm, scale=1.5)
    z = B.lc_moe_router_logits(t["x"], t["wr"])
    idx, gate = B.lc_moe_gate(z, t["bias"], w.K, w.N, **opts)
    off, _, pair, xp = B.lc_moe_permute(idx, w.N, w.E, x=t["x"])
    _, y = B.lc_moe_expert_ffn(xp, off, t["w13"], t["w2"], w.T, w.K)
    out = B.lc_moe_combine(t["x"], y, gate, pair)
    dout = torch.randn(w.T, w.d, device="cuda").bfloat16()
    dy, dgate, dx = B.lc_moe_combine_backward(dout, t["x"], y, gate, pair)
    dz = B.lc_moe_gate_backward(z, idx, dgate, score=score, renorm=renorm, scale=1.5)
    torch.cuda.synchronize()

    # the same loss in 64 bits, with the experts' rows as the layer computed them
    z64 = z.double().cpu().requires_grad_()
    x64 = t["x"].double().cpu().requires_grad_()
    M = int(off[-1])
    y64 = y[:M].double().cpu().requires_grad_()
    i, p = idx.long().cpu(), pair.long().cpu()
    s = torch.softmax(z64, 1) if score == "softmax" else torch.sigmoid(z64)
    c = torch.gather(s, 1, i)
    g = 1.5 * (c / c.sum(1, keepdim=True) if renorm else c)
    v = torch.where((p >= 0)[:, :, None], y64[p.clamp_min(0)], x64[:, None, :])
    o = (g[:, :, None] * v).sum(1)
    loss = (o * dout.double().cpu()).sum()
    loss.backward()
    assert np.allclose(gate.double().cpu(), g.detach(), rtol=1e-5, atol=0)
    # out: K terms in fp32 and one rounding to bf16
    size = (g[:, :, None] * v).abs().sum(1).detach()
    assert ((out.double().cpu() - o.detach()).abs() <= 2.0 ** -8 * o.detach().abs() + 2.0 ** -20 * size).all()
    # dz: fp32 sums of d products in dgate (d / 8 + 16 half steps of the sizes), then K of them
    bound = (v.abs() * dout.double().cpu().abs()[:, None, :]).sum(2).max().item() * 1.5
    assert ((dz.double().cpu() - z64.grad).abs() <= (w.d / 8 + 100) * 2.0 ** -24 * 4 * bound).all()
    assert ((dy[:M].double().cpu() - y64.grad).abs() <= (2.0 ** -8 + 2.0 ** -20) * y64.grad.abs()).all()
    assert ((dx.double().cpu() - x64.grad).abs() <= (2.0 ** -8 + 2.0 ** -20) * x64.grad.abs()).all()

    # differences of the loss along one direction of the logits: error h^2 / 6 times a third derivative
    direction = torch.randn(z64.shape, dtype=torch.float64)

    def at(h):
        zz = z64.detach() + h * direction
        s = torch.softmax(zz, 1) if score == "softmax" else torch.sigmoid(zz)
        c = torch.gather(s, 1, i)
        gg = 1.5 * (c / c.sum(1, keepdim=True) if renorm else c)
        return ((gg[:, :, None] * v.detach()).sum(1) * dout.double().cpu()).sum().item()
    diff = (at(1e-3) - at(-1e-3)) / 2e-3
    got = (dz.double().cpu() * direction).sum().item()
    assert abs(diff - got) <= 1e-4 * (z64.grad * direction).abs().sum().item() + 1e-4 * bound
