"""Gradient of the combine on the device against its formula in 64 bits.

dgate: products of two bf16 values are exact in fp32, and a sum of n terms in at least 8 chains is
within (n / 8 + 16) half steps of fp32 times the sum of the sizes. dY and dx: one fp32 rounding of
the product (and of the sum of K gates), then the rounding to bf16."""
import numpy as np
import pytest
import torch

from mixture_experts_zero_b200 import binding as B
from tests.operator_ref import U16, U32

pytestmark = pytest.mark.gpu

SENTINEL = 0x7BCD  # a bf16 pattern no result takes


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, d, K, N, Z, seed, spare=3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    key = torch.rand(T, N + Z, generator=g, device="cuda")
    idx = key.argsort(1)[:, :K].to(torch.int32).contiguous()
    _, _, pair_row, _ = B.lc_moe_permute(idx, N, N + Z)
    rows = int((pair_row >= 0).sum())
    def n(*s):
        return torch.randn(*s, generator=g, device="cuda")
    return dict(dout=n(T, d).bfloat16(), x=n(T, d).bfloat16(), y=n(rows + spare, d).bfloat16(),
                gate=torch.rand(T, K, generator=g, device="cuda"), pair_row=pair_row)


def reference(c):
    dout, x, y, gate, pr = f64(c["dout"]), f64(c["x"]), f64(c["y"]), f64(c["gate"]), c["pair_row"].cpu().numpy()
    T, K = pr.shape
    dgate, size = np.zeros((T, K)), np.zeros((T, K))
    dy = np.full(y.shape, np.nan)
    dx = np.where(pr < 0, gate, 0.0).sum(1)[:, None] * dout
    for r in range(K):
        v = np.where((pr[:, r] >= 0)[:, None], y[np.maximum(pr[:, r], 0)], x) if len(y) else x
        dgate[:, r] = (v * dout).sum(1)
        size[:, r] = np.abs(v * dout).sum(1)
        f = pr[:, r] >= 0
        dy[pr[f, r]] = gate[f, r][:, None] * dout[f]
    return dy, dgate, size, dx


def check(c, dy, dgate, dx):
    rdy, rdg, size, rdx = reference(c)
    d = rdx.shape[1]
    K = rdg.shape[1]
    assert np.all(np.abs(f64(dgate) - rdg) <= (d / 8 + 16) * U32 * size + 1e-30)
    assert np.all(np.abs(f64(dx) - rdx) <= (U16 + (K + 2) * U32) * np.abs(rdx))
    used = ~np.isnan(rdy[:, 0]) if len(rdy) else np.zeros(0, bool)
    assert np.all(np.abs(f64(dy)[used] - rdy[used]) <= (U16 + 2 * U32) * np.abs(rdy[used]))
    rest = dy.view(torch.int16).cpu().numpy()[~used]
    assert np.all(rest == SENTINEL)


def fresh(y):
    return torch.full(y.shape, SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16)


@pytest.mark.parametrize("T,d,K,N,Z", [
    (1, 64, 1, 1, 0), (1, 64, 3, 1, 4), (5, 128, 12, 8, 8), (33, 1024, 6, 64, 32), (100, 192, 32, 40, 24),
    (1, 6144, 12, 512, 256), (7, 6144, 12, 512, 256), (700, 320, 4, 16, 0), (1200, 2048, 12, 512, 256),
    (3, 8256, 5, 8, 4),
])
def test_combine_gradient(cuda_device, T, d, K, N, Z):
    c = make(T, d, K, N, Z, T + d)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dy = fresh(c["y"])
    out = B.lc_moe_combine_backward(**c, dy=dy, ws=ws)
    assert out[0] is dy and B.lc_moe_read_status(ws) == 0
    check(c, *out)


def test_no_ffn_picks_and_no_rows(cuda_device):
    c = make(9, 128, 4, 1, 8, 0, spare=0)
    c["pair_row"] = torch.full((9, 4), -1, dtype=torch.int32, device="cuda")
    c["y"] = c["y"][:0]
    dy, dgate, dx = B.lc_moe_combine_backward(**c)
    _, rdg, size, rdx = reference(c)
    assert dy.shape == (0, 128)
    assert np.all(np.abs(f64(dgate) - rdg) <= 32 * U32 * size)
    assert np.all(np.abs(f64(dx) - rdx) <= (U16 + 8 * U32) * np.abs(rdx))


def test_rows_out_of_range_are_reported_and_skipped(cuda_device):
    c = make(6, 128, 3, 8, 4, 1)
    rows = c["y"].shape[0]
    pr = c["pair_row"].clone()
    t, r = (pr >= 0).nonzero()[0].tolist()
    c["pair_row"] = pr
    pr[t, r] = rows
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dy, dgate, dx = B.lc_moe_combine_backward(**c, dy=fresh(c["y"]), ws=ws)
    assert B.lc_moe_read_status(ws, raise_on_error=False) == B.DEV_IDX_RANGE
    assert float(dgate[t, r]) == 0.0
    c["pair_row"] = pr.clone()
    good = dict(c)
    good["pair_row"] = torch.where(pr == rows, torch.full_like(pr, -1), pr)
    want = B.lc_moe_combine_backward(**good, dy=fresh(c["y"]))
    dgate[t, r] = want[1][t, r] = 0
    assert torch.equal(dgate, want[1]) and torch.equal(dy.view(torch.int16), want[0].view(torch.int16))
    w = torch.where(pr < 0, c["gate"], torch.zeros_like(c["gate"])).double().sum(1, keepdim=True)
    assert np.all(np.abs(f64(dx) - f64(w) * f64(c["dout"])) <= (U16 + 8 * U32) * np.abs(f64(w) * f64(c["dout"])))


def test_combine_gradient_against_differences(cuda_device):
    """The combine is linear in each of its inputs: a difference of the 64-bit forward is the
    gradient up to rounding."""
    c = make(3, 64, 4, 6, 3, 4, spare=0)
    dy, dgate, dx = B.lc_moe_combine_backward(**c)
    dout, x, y, gate, pr = f64(c["dout"]), f64(c["x"]), f64(c["y"]), f64(c["gate"]), c["pair_row"].cpu().numpy()

    def loss(x, y, gate):
        v = np.where((pr >= 0)[:, :, None], y[np.maximum(pr, 0)], x[:, None, :])
        return ((gate[:, :, None] * v).sum(1) * dout).sum()
    base = loss(x, y, gate)
    rng = np.random.default_rng(0)
    for a, got in ((x, f64(dx)), (y, f64(dy)), (gate, f64(dgate))):
        step = rng.standard_normal(a.shape)
        args = [b + step if b is a else b for b in (x, y, gate)]
        # each gradient element is within a bf16 half step (dgate: far less)
        lim = 2 * U16 * np.abs(got * step).sum() + 1e-9
        assert abs((loss(*args) - base) - (got * step).sum()) <= lim


def test_repeats_other_streams_and_graphs_give_the_same_bits(cuda_device):
    c = make(150, 1024, 6, 64, 32, 8)
    want = B.lc_moe_combine_backward(**c)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = B.lc_moe_combine_backward(**c, stream=st)
    st.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    outs = [torch.zeros_like(a) for a in want]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.lc_moe_combine_backward(**c, dy=outs[0], dgate=outs[1], dx=outs[2], ws=ws)
    for _ in range(2):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
