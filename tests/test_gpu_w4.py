"""4-bit experts on the device: the quantiser's codes and scales (whole numbers: equal), and the
grouped products against float64 products of the same codes, scales and bf16 rows.

Products: a code times a bf16 value is exact in fp32; the sums of one output run through at most 28
dependent steps of the tensor cores and of fp32 additions, each within 2 steps of fp32 of the sizes
added so far: 2^-17 of the sum of the sizes |w x|. The SwiGLU then moves an error of g by at most
1.1 |u| and one of u by |silu(g)|, and evaluates silu within 2^-19 (1 + |g|) of itself (the argument
of the exponential is rounded to fp32, the fast exponential and quotient are within a few steps).
H and Y add their rounding to bf16."""
import numpy as np
import pytest
import torch

import oracle
from mixture_experts_zero_b200 import binding as B
from mixture_experts_zero_b200 import inputs
from tests import operator_ref as R
from tests.gpu_util import assert_out_close, np_bits

pytestmark = pytest.mark.gpu

ACC = 2.0 ** -17
SENTINEL = 0x7BCD


def f64(t):
    return t.detach().double().cpu().numpy()


def weights(N, d, I, group, seed, std=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w13 = (torch.randn(N, 2 * I, d, generator=g, device="cuda") * (std or d ** -0.5)).bfloat16()
    w2 = (torch.randn(N, d, I, generator=g, device="cuda") * (std or I ** -0.5)).bfloat16()
    q13, q2 = B.lc_moe_quantize_w4(w13, group), B.lc_moe_quantize_w4(w2, group)
    return w13, w2, q13 + q2


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,cols", [(16, 128), (48, 256), (160, 640), (4096, 128), (16, 6144)])
def test_quantiser(cuda_device, rows, cols, group):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + cols)
    w = (torch.randn(rows, cols, generator=g, device="cuda") * 0.02).bfloat16()
    w[3] = 0                      # groups whose scale would be 0
    w[5] *= 1e-38                 # far below the smallest normal value
    w[7, :32] = 1.0
    w[8] = (w[8].float() * 1e37).bfloat16()
    codes, scale = B.lc_moe_quantize_w4(w, group)
    q, s = R.w4_quantize(f64(w), group)
    sc = f64(scale)
    flat = sc.reshape(rows // 16, cols // group, 8, 2).transpose(0, 3, 2, 1).reshape(rows, cols // group)
    np.testing.assert_array_equal(flat, s)
    got = R.w4_unpack(codes.cpu().numpy(), np.ones_like(sc), rows, cols, group)
    np.testing.assert_array_equal(got, q)
    # a code is within half a step of its weight (the scale's own rounding moves amax by 2^-8 of it)
    full = R.w4_unpack(codes.cpu().numpy(), sc, rows, cols, group)
    step = np.repeat(s, group, 1)
    live = np.repeat(np.abs(f64(w)).reshape(rows, -1, group).max(2) > 1e-36, group, 1)
    assert np.all((np.abs(full - f64(w)) <= 0.5 * step * (1 + 1e-6))[live])


def test_quantiser_of_stacked_matrices_and_64_columns(cuda_device):
    w = torch.randn(3, 32, 64, device="cuda").bfloat16()
    codes, scale = B.lc_moe_quantize_w4(w, 64)
    assert codes.shape == (3, 32, 32) and scale.shape == (3, 2, 1, 16)
    for e in range(3):
        c, s = B.lc_moe_quantize_w4(w[e].contiguous(), 64)
        assert torch.equal(c, codes[e]) and torch.equal(s, scale[e])


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def check_ffn(x, counts, q, group, d, I, h, y, first=0):
    """H against the products of x, Y against the products of the H that was stored."""
    at = first
    hb, yb = f64(h), f64(y)
    for e, n in enumerate(counts):
        if not n:
            continue
        w13 = R.w4_unpack(q[0][e].cpu().numpy(), f64(q[1][e]), 2 * I, d, group)
        w2 = R.w4_unpack(q[2][e].cpu().numpy(), f64(q[3][e]), d, I, group)
        xs = f64(x[at:at + n])
        gu, size = xs @ w13.T, np.abs(xs) @ np.abs(w13).T
        g, u = gu[:, :I], gu[:, I:]
        want = silu(g) * u
        tol = R.U16 * np.abs(want) + 1.1 * np.abs(u) * ACC * size[:, :I] + (np.abs(silu(g)) + ACC * size[:, :I]) * ACC * size[:, I:] \
            + 2.0 ** -19 * (1 + np.abs(g)) * np.abs(want) + 1e-37
        err = np.abs(hb[at:at + n] - want)
        assert np.all(err <= tol), ("h", e, float((err / tol).max()))
        hs = hb[at:at + n]
        want, size = hs @ w2.T, np.abs(hs) @ np.abs(w2).T
        tol = R.U16 * np.abs(want) + ACC * size + 1e-37
        err = np.abs(yb[at:at + n] - want)
        assert np.all(err <= tol), ("y", e, float((err / tol).max()))
        at += n
    return at


def run_ffn(counts, d, I, group, seed=0, tail=5, K=1, std=None, **kw):
    N, rows = len(counts), sum(counts) + tail
    rows = -(-rows // K) * K
    w13, w2, q = weights(N, d, I, group, seed, std)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    x = torch.randn(rows, d, generator=g, device="cuda").bfloat16()
    x[sum(counts):] = float("nan")  # rows behind the last expert's are not read
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    h = torch.full((rows, I), SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    y = torch.full((rows, d), SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.lc_moe_expert_ffn_w4(x, off, *q, rows // K, K, h=h, y=y, ws=ws, **kw)
    assert B.lc_moe_read_status(ws) == 0
    end = check_ffn(x, counts, q, group, d, I, h, y)
    assert (h[end:].view(torch.int16) == SENTINEL).all() and (y[end:].view(torch.int16) == SENTINEL).all()


@pytest.mark.parametrize("d,I,group", [(64, 64, 32), (64, 64, 64), (128, 192, 64), (192, 320, 32), (256, 128, 128),
                                       (1024, 256, 32), (128, 1024, 128), (640, 64, 64), (6144, 128, 128)])
def test_ffn_at_every_row_count(cuda_device, d, I, group):
    run_ffn([1, 0, 7, 8, 9, 16, 17, 33], d, I, group, seed=d + I)


@pytest.mark.parametrize("counts", [[1], [0, 0, 1], [0], [0, 0, 0], [2, 0, 0, 3], [100, 1, 0, 65], [31, 32, 63, 64, 128]])
def test_ffn_row_counts(cuda_device, counts):
    run_ffn(counts, 128, 128, 32, seed=len(counts))


def test_ffn_many_experts(cuda_device):
    rng = np.random.default_rng(0)
    run_ffn([int(v) for v in rng.integers(0, 4, 2048)], 64, 64, 32, seed=3)


def test_ffn_full_width(cuda_device):
    run_ffn([1, 3, 0, 12], 6144, 2048, 64, seed=9, K=3)
    run_ffn([40, 1], 6144, 2048, 128, seed=10)


def test_ffn_large_activations(cuda_device):
    """Rows of very different sizes, and values near the ends of the bf16 range in one row."""
    N, d, I, group = 2, 256, 128, 64
    _, _, q = weights(N, d, I, group, 4)
    x = torch.randn(6, d, device="cuda")
    x[0] *= 1e-30
    x[1] *= 1e12
    x[2, ::2] *= 1e4
    x = x.bfloat16()
    off = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
    h, y = B.lc_moe_expert_ffn_w4(x, off, *q, 6, 1)
    check_ffn(x, [4, 2], q, group, d, I, h, y)


def test_a_row_of_nan_or_infinity_stays_by_itself(cuda_device):
    N, d, I, group, counts = 3, 192, 128, 64, [5, 11, 20]
    _, _, q = weights(N, d, I, group, 14)
    rows = sum(counts)
    x = torch.randn(rows, d, device="cuda").bfloat16()
    off = torch.tensor([0, 5, 16, 36], dtype=torch.int32, device="cuda")
    h, y = B.lc_moe_expert_ffn_w4(x, off, *q, rows, 1)
    bad = x.clone()
    for r, v in ((4, float("nan")), (7, float("inf")), (15, float("nan")), (30, float("-inf"))):
        bad[r, 3] = v
    h2, y2 = B.lc_moe_expert_ffn_w4(bad, off, *q, rows, 1)
    keep = [r for r in range(rows) if r not in (4, 7, 15, 30)]
    assert torch.equal(h[keep], h2[keep]) and torch.equal(y[keep], y2[keep])
    for r in (4, 7, 15, 30):
        assert not torch.isfinite(y2[r].float()).any()


def test_rows_before_the_first_expert_stay(cuda_device):
    N, d, I, group = 2, 64, 64, 32
    _, _, q = weights(N, d, I, group, 15)
    x = torch.randn(12, d, device="cuda").bfloat16()
    off = torch.tensor([3, 3, 10], dtype=torch.int32, device="cuda")
    h = torch.full((12, I), SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    y = torch.full((12, d), SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    B.lc_moe_expert_ffn_w4(x, off, *q, 12, 1, h=h, y=y)
    for v in (h, y):
        assert (v[:3].view(torch.int16) == SENTINEL).all() and (v[10:].view(torch.int16) == SENTINEL).all()
    check_ffn(x, [0, 7], q, group, d, I, h, y, first=3)


def test_ffn_on_two_streams_at_once(cuda_device):
    N, d, I, group, counts = 4, 512, 256, 64, [2, 30, 0, 9]
    _, _, q = weights(N, d, I, group, 16)
    rows = sum(counts)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    xs = [torch.randn(rows, d, device="cuda").bfloat16() for _ in range(2)]
    want = [B.lc_moe_expert_ffn_w4(x, off, *q, rows, 1) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[B.lc_moe_expert_ffn_w4(x, off, *q, rows, 1, stream=s) for x, s in zip(xs, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_offsets_are_reported_and_skipped(cuda_device):
    N, d, I, group = 3, 64, 64, 32
    _, _, q = weights(N, d, I, group, 6)
    x = torch.randn(8, d, device="cuda").bfloat16()
    for bad in ([0, 3, 2, 8], [0, 3, 6, 9], [-1, 3, 6, 8], [0, 100, 6, 8]):
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        h, y = torch.zeros(8, I, device="cuda").bfloat16(), torch.zeros(8, d, device="cuda").bfloat16()
        B.lc_moe_expert_ffn_w4(x, off, *q, 8, 1, h=h, y=y, ws=ws)
        assert B.lc_moe_read_status(ws, raise_on_error=False) == B.DEV_IDX_RANGE


def test_y_over_its_rows(cuda_device):
    """H is complete before Y begins, so Y may take the place of x_perm; rows of no expert stay."""
    N, d, I, group, counts = 4, 512, 1024, 64, [3, 40, 0, 17]
    _, _, q = weights(N, d, I, group, 18)
    x = torch.randn(sum(counts) + 4, d, device="cuda").bfloat16()
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    h, y = B.lc_moe_expert_ffn_w4(x, off, *q, 64, 1)
    for _ in range(5):
        over = x.clone()
        h2, y2 = B.lc_moe_expert_ffn_w4(over, off, *q, 64, 1, y=over)
        assert y2 is over and torch.equal(h[:60], h2[:60]) and torch.equal(y[:60], over[:60])
        assert torch.equal(over[60:], x[60:])


@pytest.mark.parametrize("rows,offsets,taken", [
    (8, [0, 3, 2, 8], [0]),            # expert 2 begins inside expert 0
    (8, [0, 3, 6, 9], [0, 1]),
    (8, [-1, 3, 6, 8], [1, 2]),
    (8, [0, 100, 6, 8], [2]),
    (40, [0, 9, 4, 12, 12, 40], [0, 4]),
    (40, [20, 10, 15, 15, 41, 30, 40], [1, 5]),
    (8, [8, 0, 0, -5, -9, 2 ** 31 - 1, 7], []),
    (8, [0, -1, 0, 9, 8], []),
])
def test_experts_beside_bad_offsets(cuda_device, rows, offsets, taken):
    """Only the rows of experts that are not skipped are written, with what good offsets give."""
    N, d, I, group = len(offsets) - 1, 64, 64, 32
    _, _, q = weights(N, d, I, group, 7)
    x = torch.randn(rows, d, device="cuda").bfloat16()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    h = torch.full((rows, I), SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    y = torch.full((rows, d), SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    B.lc_moe_expert_ffn_w4(x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), *q, rows, 1, h=h, y=y, ws=ws)
    assert B.lc_moe_read_status(ws, raise_on_error=False) == B.DEV_IDX_RANGE
    rest = np.ones(rows, bool)
    for e in taken:
        a, b = offsets[e], offsets[e + 1]
        check_ffn(x, [0] * e + [b - a], q, group, d, I, h, y, first=a)
        rest[a:b] = False
    for v in (h, y):
        assert np.all(v.view(torch.int16).cpu().numpy()[rest] == SENTINEL)


def test_offsets_that_give_many_experts_the_same_rows(cuda_device):
    """1024 experts that all claim rows 0..64: the first has them, and no sum runs over."""
    rows, N, d, I, group = 64, 2048, 64, 64, 32
    _, _, q = weights(N, d, I, group, 8)
    x = torch.randn(rows, d, device="cuda").bfloat16()
    off = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    off[1::2] = rows
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    h, y = B.lc_moe_expert_ffn_w4(x, off, *q, rows, 1, ws=ws)
    assert B.lc_moe_read_status(ws, raise_on_error=False) == B.DEV_IDX_RANGE
    check_ffn(x, [rows], q, group, d, I, h, y)


def test_ffn_on_another_stream_in_a_graph_and_repeated(cuda_device):
    N, d, I, group, counts = 6, 256, 192, 64, [3, 0, 9, 20, 1, 2]
    _, _, q = weights(N, d, I, group, 12)
    rows = sum(counts)
    x = torch.randn(rows, d, device="cuda").bfloat16()
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    want = B.lc_moe_expert_ffn_w4(x, off, *q, rows, 1)
    check_ffn(x, counts, q, group, d, I, *want)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = B.lc_moe_expert_ffn_w4(x, off, *q, rows, 1, stream=st)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    h, y = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.lc_moe_expert_ffn_w4(x, off, *q, rows, 1, h=h, y=y, ws=ws)
    for _ in range(2):
        h.zero_(), y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want[0]) and torch.equal(y, want[1])


# ------------------------------------------------------------------------------ the layer --

GATE = dict(score="sigmoid", groups=4, top_groups=2, group_rank=2, scale=2.5)


def layer(T=64, seed=0, group=32):
    w = inputs.scaled(inputs.WORKLOADS["tiny"], T=T, I=128, seed=seed)
    t = inputs.make(w, device="cuda", grid=True)
    q = B.lc_moe_quantize_w4(t["w13"], group) + B.lc_moe_quantize_w4(t["w2"], group)
    return w, t, q


@pytest.mark.parametrize("T", [1, 7, 64, 300])
@pytest.mark.parametrize("opts", [None, GATE, dict(renorm=False)])
def test_layer_is_the_run_of_its_stages(cuda_device, T, opts):
    w, t, q = layer(T)
    idx = torch.empty(T, w.K, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, w.K, dtype=torch.float32, device="cuda")
    counts = torch.zeros(w.E, dtype=torch.int32, device="cuda")
    ws = B.new_workspace(B.Shape(T, w.d, w.N, w.Z, w.K, w.I), B.OP_FORWARD_W4)
    out = B.lc_moe_forward_w4(t["x"], t["wr"], t["bias"], *q, w.K, opts=opts, idx=idx, gate=gate, counts=counts, ws=ws)
    assert B.lc_moe_read_status(ws) == 0
    if opts is None:
        i2, g2 = B.lc_moe_route(t["x"], t["wr"], t["bias"], w.K, w.N)
    else:
        i2, g2 = B.lc_moe_gate(B.lc_moe_router_logits(t["x"], t["wr"]), t["bias"], w.K, w.N, **opts)
    assert torch.equal(idx, i2) and torch.equal(gate, g2)
    assert torch.equal(counts, torch.bincount(idx.flatten().long(), minlength=w.E).int())
    off, _, pair, xp = B.lc_moe_permute(i2, w.N, w.E, x=t["x"])
    _, y = B.lc_moe_expert_ffn_w4(xp, off, *q, T, w.K)
    assert torch.equal(out, B.lc_moe_combine(t["x"], y, g2, pair))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("opts", [None, GATE])
def test_layer_against_64_bits(cuda_device, opts, group):
    """The whole layer on grid inputs (exact logits): picks equal, output against the formula with
    bf16 at H and Y, at the tolerance of the other forwards."""
    w, t, q = layer(80, 3, group)
    idx = torch.empty(w.T, w.K, dtype=torch.int32, device="cuda")
    out = B.lc_moe_forward_w4(t["x"], t["wr"], t["bias"], *q, w.K, opts=opts, idx=idx)
    z = f64(t["x"]) @ f64(t["wr"]).T
    o = {**dict(score="softmax", groups=1, top_groups=1, group_rank=1, renorm=True, scale=1.0), **(opts or {})}
    s = R.scores(z, o["score"])
    if opts is None:
        want_idx = oracle.route(z.astype(np.float32), t["bias"].cpu().numpy(), w.K)[0]
    else:
        want_idx = R.picks(s, f64(t["bias"]), w.K, o["groups"], o["top_groups"], o["group_rank"])
    np.testing.assert_array_equal(idx.cpu().numpy(), want_idx)
    g = R.gates(z, s, want_idx, o["score"], o["renorm"], o["scale"])
    x, exact = f64(t["x"]), np.zeros((w.T, w.d))
    w13 = [R.w4_unpack(q[0][e].cpu().numpy(), f64(q[1][e]), 2 * w.I, w.d, group) for e in range(w.N)]
    w2 = [R.w4_unpack(q[2][e].cpu().numpy(), f64(q[3][e]), w.d, w.I, group) for e in range(w.N)]
    for tok in range(w.T):
        for r in range(w.K):
            e = want_idx[tok, r]
            v = x[tok]
            if e < w.N:
                gu = w13[e] @ x[tok]
                v = w2[e] @ (silu(gu[:w.I]) * gu[w.I:])
            exact[tok] += g[tok, r] * v
    assert_out_close(np_bits(out), exact, what="4-bit layer")


def test_layer_in_a_graph_and_decode_of_one_token(cuda_device):
    w, t, q = layer(1, 5)
    want = B.lc_moe_forward_w4(t["x"], t["wr"], t["bias"], *q, w.K, opts=GATE)
    ws = B.new_workspace(B.Shape(1, w.d, w.N, w.Z, w.K, w.I), B.OP_FORWARD_W4)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.lc_moe_forward_w4(t["x"], t["wr"], t["bias"], *q, w.K, opts=GATE, out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert B.lc_moe_read_status(ws) == 0


def test_empty_calls(cuda_device):
    w, t, q = layer(4, 6)
    x = t["x"][:0]
    idx, gate = B.lc_moe_gate(torch.empty(0, w.E, device="cuda"), t["bias"], w.K, w.N)
    assert idx.shape == gate.shape == (0, w.K)
    assert B.lc_moe_gate_backward(torch.empty(0, w.E, device="cuda"), idx, gate).shape == (0, w.E)
    dy, dgate, dx = B.lc_moe_combine_backward(x, x, t["x"], gate, idx)
    assert dy.eq(0).all() and dgate.shape == (0, w.K) and dx.shape == (0, w.d)
    off = torch.zeros(w.N + 1, dtype=torch.int32, device="cuda")
    h, y = B.lc_moe_expert_ffn_w4(x, off, *q, 0, w.K)
    assert h.shape == (0, w.I) and y.shape == (0, w.d)
    torch.cuda.synchronize()


def test_layer_without_tokens_and_without_a_bias(cuda_device):
    w, t, q = layer(4, 6)
    assert B.lc_moe_forward_w4(t["x"][:0], t["wr"], t["bias"], *q, w.K).shape == (0, w.d)
    a = B.lc_moe_forward_w4(t["x"], t["wr"], None, *q, w.K, opts={})
    b = B.lc_moe_forward_w4(t["x"], t["wr"], torch.zeros_like(t["bias"]), *q, w.K, opts={})
    assert torch.equal(a, b)
    with pytest.raises(ValueError, match="bias"):
        B.lc_moe_forward_w4(t["x"], t["wr"], None, *q, w.K)
