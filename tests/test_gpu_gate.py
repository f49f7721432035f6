"""General gates and their gradient on the device, against plain 64-bit forms (tests/operator_ref.py).

Picks have to be equal. Gates: expf is within 2 steps, its argument z - m is rounded once (|z - m|
half steps relative to the result), the sum and the quotient add a few more, in numerator and
denominator: (2 R + 64) half steps of fp32 with R the range of a row's logits. Gradients: the same
factor times the sizes of the terms added (the reference's bound), plus the rounding of a bf16
result."""
import math

import numpy as np
import pytest
import torch

from mixture_experts_zero_b200 import binding as B
from tests import operator_ref as R

pytestmark = pytest.mark.gpu

CASES = [
    # T, E, K, groups, top, rank
    (1, 1, 1, 1, 1, 1), (1, 768, 12, 1, 1, 1), (37, 12, 3, 4, 2, 2), (64, 33, 7, 1, 1, 1), (5, 2048, 32, 1, 1, 1),
    (9, 2048, 32, 32, 7, 2), (130, 768, 12, 8, 4, 2), (33, 96, 6, 3, 1, 1), (20, 333, 7, 9, 5, 2), (17, 64, 32, 32, 16, 2),
    (11, 31, 31, 31, 31, 2), (21, 1025, 9, 1, 1, 1), (13, 40, 8, 8, 8, 1), (700, 130, 5, 2, 1, 2), (15, 32, 16, 32, 16, 2), (9, 30, 10, 3, 1, 2),
    (8, 62, 2, 31, 1, 1),
]


def logits_of(T, E, seed, bf16, std=2.0):
    z = torch.from_numpy(np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32) * std)
    return (z.to(torch.bfloat16) if bf16 else z).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def span(z):
    """The range of a row's logits; a logit more than 110 below the largest adds nothing in fp32."""
    z = np.where(np.isinf(z), 0.0, z)
    return min(110.0, float((z.max(1) - z.min(1)).max()))


def check_gate(z, b, K, N, score, groups=1, top=1, rank=1, renorm=True, scale=1.0, **kw):
    E = z.shape[1]
    counts = torch.full((E,), 3, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    idx, gate = B.lc_moe_gate(z, b, K, N, score=score, groups=groups, top_groups=top, group_rank=rank, renorm=renorm,
                              scale=scale, counts=counts, ws=ws, **kw)
    assert B.lc_moe_read_status(ws) == 0
    s = R.scores(f64(z), score)
    want = R.picks(s, None if b is None else f64(b), K, groups, top, rank)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    ref = R.gates(f64(z), s, want, score, renorm, scale)
    tol = (2 * span(f64(z)) + 64) * R.U32 * np.abs(ref) + 1e-37
    err = np.abs(f64(gate) - ref)
    assert np.all(err <= tol), float((err / tol).max())
    np.testing.assert_array_equal(counts.cpu().numpy() - 3, np.bincount(want.ravel(), minlength=E))
    return idx, gate


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", CASES)
def test_gate_against_64_bits(cuda_device, case, score):
    T, E, K, groups, top, rank = case
    rng = np.random.default_rng(hash(case) % 1000)
    for bf16 in (False, True):
        z = logits_of(T, E, E + T, bf16)
        for renorm, scale, bias in ((True, 1.0, True), (False, 2.5, True), (True, 2.5, False)):
            b = torch.from_numpy((rng.random(E) * 0.2 - 0.1).astype(np.float32)).cuda() if bias else None
            check_gate(z, b, K, max(1, E // 2), score, groups, top, rank, renorm, scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens(cuda_device, score):
    """Enough tokens that some have keys closer to each other than fp32 resolves."""
    z = logits_of(6000, 96, 5, False, std=4.0)
    b = torch.from_numpy((np.random.default_rng(0).random(96) * 1e-3).astype(np.float32)).cuda()
    check_gate(z, b, 8, 64, score)
    check_gate(z, b, 8, 64, score, groups=8, top=3, rank=2, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_experts_with_crowded_keys(cuda_device, score):
    """2048 experts whose scores the biases level out, so that neighbours in the order are close."""
    z = logits_of(400, 2048, 6, False, std=0.5)
    b = -torch.from_numpy(R.scores(f64(z[:1]), score)[0].astype(np.float32)).cuda()
    check_gate(z, b, 32, 1024, score)
    check_gate(z[:50], b, 32, 1024, score, groups=16, top=5, rank=2)
    check_gate(z[:1], b, 32, 1024, score)      # every key is a rounding error


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_keys_that_fp32_cannot_tell_apart(cuda_device, score):
    """Neighbouring fp32 logits and biases that nearly undo their differences."""
    rng = np.random.default_rng(3)
    E, K = 80, 9
    base = np.float32(1.25) + np.arange(E, dtype=np.float32) * np.float32(2.0 ** -22)
    z = np.stack([rng.permutation(base) for _ in range(40)]).astype(np.float32)
    for b in (None, np.zeros(E, np.float32), (rng.integers(-3, 4, E) * 2.0 ** -26).astype(np.float32)):
        bt = None if b is None else torch.from_numpy(b).cuda()
        check_gate(torch.from_numpy(z).cuda(), bt, K, 40, score)
        check_gate(torch.from_numpy(z).cuda(), bt, K, 40, score, groups=8, top=3, rank=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_index(cuda_device, score):
    rng = np.random.default_rng(1)
    for (T, E, K, groups, top, rank) in [(40, 12, 3, 1, 1, 1), (64, 65, 32, 1, 1, 1), (3, 2048, 32, 1, 1, 1),
                                         (50, 96, 6, 8, 3, 2), (50, 96, 6, 8, 3, 1)]:
        z = torch.from_numpy(rng.integers(-1, 2, (T, E)).astype(np.float32)).cuda()
        z[0] = 0.0  # every key equal
        check_gate(z, None, K, max(1, E // 2), score, groups, top, rank)
        check_gate(z.to(torch.bfloat16), None, K, max(1, E // 2), score, groups, top, rank, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_logits_and_switched_off_experts(cuda_device, score):
    """-inf and lowest logits, rows that leave nothing, -inf biases, fewer live experts than K."""
    E, K = 48, 5
    z = logits_of(9, E, 7, False)
    z[0, 3:] = -math.inf
    z[1, :] = -math.inf
    z[2, 1::2] = torch.finfo(torch.float32).min
    z[3, :] = torch.finfo(torch.float32).min
    z[4, :] = -300.0
    z[4, 7] = -299.0
    b = torch.zeros(E, device="cuda")
    for renorm in (True, False):
        check_gate(z, None, K, 24, score, renorm=renorm)
        check_gate(z, b, K, 24, score, renorm=renorm, scale=2.5)
    b[4:] = -math.inf
    check_gate(z, b, K, 24, score)
    b[:] = -math.inf
    check_gate(z, b, K, 24, score)
    b[:] = 0
    b[::3] = -math.inf
    check_gate(z, b, K, 24, score, groups=8, top=3, rank=1)
    check_gate(z, b, K, 24, score, groups=8, top=3, rank=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_below_fp32_behind_masked_experts(cuda_device, score):
    """Masked experts (score 0) tie in fp32 with scores that only 64 bits can hold: a run of equal keys
    across the K-th place hides an expert behind it that belongs before it."""
    E, K = 22, 5
    low = -300.0 if score == "softmax" else -120.0
    z = torch.full((6, E), -math.inf, device="cuda")
    z[:, 4] = 1.0
    z[0, 15] = low
    z[1, 15], z[1, 20] = low, low + 1
    z[2, 0] = low
    z[3, 5:] = low
    z[4, 21] = low
    z[5, 6], z[5, 21] = low, low
    for b in (None, torch.zeros(E, device="cuda")):
        check_gate(z, b, K, E, score)
        check_gate(z, b, K, E, score, renorm=False)
        check_gate(z, b, K, E, score, groups=2, top=1, rank=2)
        check_gate(z.repeat(1, 3), None if b is None else b.repeat(3), K, E, score, groups=3, top=2, rank=2)


def test_small_shares_of_sigmoid_gates(cuda_device):
    """A chosen score whose e^-z does not fit fp32 still has its share of the gates."""
    z = torch.tensor([[-30.0, -90.0, -95.0, -200.0], [3.0, -70.0, -88.0, -100.0], [-39.0, -89.5, -101.0, -110.0]],
                     device="cuda")
    for scale in (1.0, 2.5):
        check_gate(z, None, 3, 4, "sigmoid", scale=scale)
        check_gate(z, torch.zeros(4, device="cuda"), 3, 4, "sigmoid", scale=scale)


def test_all_masked_row_has_zero_gates(cuda_device):
    z = torch.full((2, 16), -math.inf, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx, gate = B.lc_moe_gate(z, None, 4, 16, score=score, renorm=renorm)
            assert gate.eq(0).all() and idx.cpu().tolist() == [[0, 1, 2, 3]] * 2
            d = B.lc_moe_gate_backward(z, idx, torch.ones(2, 4, device="cuda"), score=score, renorm=renorm)
            assert d.eq(0).all()


def test_extreme_biases(cuda_device):
    """Biases far larger than the scores, and of both signs: the key is the rounded 64-bit sum."""
    z = logits_of(30, 64, 2, False)
    b = torch.from_numpy((np.random.default_rng(5).standard_normal(64) * 1e4).astype(np.float32)).cuda()
    for score in ("softmax", "sigmoid"):
        check_gate(z, b, 8, 64, score)
        check_gate(z, b, 8, 64, score, groups=8, top=2, rank=2)
        check_gate(z, torch.full((64,), 1e3, device="cuda"), 8, 64, score)


def test_nan_keys_are_reported(cuda_device):
    for bad, score in ((math.nan, "softmax"), (math.nan, "sigmoid"), (math.inf, "softmax")):
        z = logits_of(6, 40, 1, False)
        clean = z.clone()
        z[2, 9] = bad
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        idx, gate = B.lc_moe_gate(z, None, 4, 40, score=score, ws=ws)
        assert B.lc_moe_read_status(ws, raise_on_error=False) == B.DEV_NAN_KEY
        assert idx[2].cpu().tolist() == [0, 1, 2, 3] and gate[2].isnan().all()
        ref, rg = B.lc_moe_gate(clean, None, 4, 40, score=score)
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(idx[keep], ref[keep]) and torch.equal(gate[keep], rg[keep])
    z = logits_of(2, 8, 1, False)
    b = torch.zeros(8, device="cuda")
    b[0], b[1] = math.inf, -math.inf
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.lc_moe_gate(z, b, 2, 8, groups=4, top_groups=2, group_rank=2, ws=ws)
    assert B.lc_moe_read_status(ws, raise_on_error=False) == B.DEV_NAN_KEY


def test_infinite_sigmoid_logit_is_a_score_of_one(cuda_device):
    z = logits_of(3, 20, 4, False)
    z[1, 5] = math.inf
    idx, gate = B.lc_moe_gate(z, None, 2, 20, score="sigmoid", renorm=False)
    assert int(idx[1, 0]) == 5 and float(gate[1, 0]) == 1.0


def test_unaligned_rows_and_default_options(cuda_device):
    """Logits that start on an odd element, and the C call with NULL options."""
    import ctypes
    for bf16 in (False, True):
        z = logits_of(21, 77, 8, bf16)
        flat = torch.zeros(21 * 77 + 1, dtype=z.dtype, device="cuda")
        flat[1:] = z.view(-1)
        v = flat[1:].view(21, 77)
        idx, gate = check_gate(v, None, 6, 70, "softmax")
        idx2, gate2 = torch.empty_like(idx), torch.empty_like(gate)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        s = B.Shape(21, 64, 70, 7, 6, 64)
        rc = B.library().lc_moe_gate(ctypes.byref(s), None, B._ptr(v), int(bf16), None, B._ptr(idx2), B._ptr(gate2),
                                     None, B._ptr(ws), 256, B._stream(None))
        torch.cuda.synchronize()
        assert rc == 0 and torch.equal(idx, idx2) and torch.equal(gate, gate2)
        d = B.lc_moe_gate_backward(v, idx, torch.ones_like(gate), renorm=False)
        check_backward(v, idx, torch.ones_like(gate), "softmax", False, 1.0, d)


@pytest.mark.parametrize("low", [torch.finfo(torch.float32).min, -3e38])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_lowest_value_biases_beside_infinite_ones(cuda_device, score, low):
    """Two keys at the end of the fp32 range make a finite group score in 64 bits, above one of -inf; two
    at the other end make one that is below +inf."""
    inf = math.inf
    z = logits_of(5, 8, 21, False)
    for b in ([0, 0, -inf, -inf, low, low, -inf, -inf], [-inf, -inf, -inf, 0, low, low, low, low],
              [low, low, -inf, -inf, 0, 0, low, 0], [-low, -low, 0, 0, -low, 0, -low, -low],
              [low, -inf, low, low, low, 0, -inf, -inf]):
        b = torch.tensor(b, device="cuda", dtype=torch.float32)
        for top, K in ((1, 2), (2, 3), (3, 5)):
            check_gate(z, b, K, 8, score, groups=4, top=top, rank=2)
            check_gate(z, b, K, 8, score, groups=4, top=top, rank=1)
        check_gate(z, b, 6, 8, score)


@pytest.mark.filterwarnings("ignore::RuntimeWarning")  # infinities in the plain form
@pytest.mark.parametrize("K", [1, 2, 3])
def test_sigmoid_logits_whose_scores_are_all_one(cuda_device, K):
    """1 / (1 + e^-z) is 1 in 64 bits from z = 37 on: such logits tie, whatever they are."""
    inf = math.inf
    rng = np.random.default_rng(2)
    z = torch.from_numpy(np.minimum(rng.standard_normal((6, 40)), 5.0).astype(np.float32)).cuda()
    for row, at in enumerate(({3: 37.5, 20: inf}, {0: 37.5, 9: 1e25, 30: inf}, {7: 100.0, 8: 90.0, 9: 3e38, 39: inf},
                              {1: inf, 2: 40.0}, {5: 79.0, 6: 81.0, 38: 2e20}, {i: 50.0 + i for i in range(40)})):
        for i, v in at.items():
            z[row, i] = v
    for bf16 in (False, True):
        v = z.bfloat16() if bf16 else z
        for renorm in (True, False):
            check_gate(v, None, K, 40, "sigmoid", renorm=renorm)
            check_gate(v, torch.zeros(40, device="cuda"), K, 40, "sigmoid", renorm=renorm)
            for groups, top in ((8, 1), (8, 3), (2, 1)):
                check_gate(v, None, K, 40, "sigmoid", groups=groups, top=top, rank=1, renorm=renorm)
                check_gate(v, None, K, 40, "sigmoid", groups=groups, top=top, rank=2, renorm=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_uncertain_key_behind_two_certain_ones(cuda_device, score):
    """The K-th and the key behind it are biases of experts without a score, which fp32 holds exactly and tells
    apart; a third key, a score near e^-60 that fp32 holds within tens of steps, lies above both in 64 bits
    and may lie below both in fp32."""
    rng = np.random.default_rng(17)
    zs = (-60.0 - 10.0 * rng.random(96)).astype(np.float32)
    for z3 in zs:
        # softmax: all of the rest is with expert 0, which is switched off
        row = np.array([0.0 if score == "softmax" else -110.0, -110.0, -110.0, z3, -110.0, -110.0], np.float32)
        s3 = R.scores(row[None], score)[0, 3]
        for above in (6.0, 14.0):
            b1 = np.float32(s3 * (1 - above * 2.0 ** -23))
            b = [-math.inf, b1, b1 * np.float32(1 - 5 * 2.0 ** -23), 0.0, b1 * np.float32(0.5), -math.inf]
            bt, zt = torch.tensor(b, dtype=torch.float32, device="cuda"), torch.from_numpy(row[None]).cuda()
            for K in (1, 2):
                idx, _ = B.lc_moe_gate(zt, bt, K, 6, score=score)
                assert idx[0].cpu().tolist() == [3, 1][:K], (float(z3), above)


# ------------------------------------------------------------------------------- gradient --

def check_backward(z, idx, dg, score, renorm, scale, got):
    dz, bound = R.gate_backward(f64(z), idx.cpu().numpy(), f64(dg), score, renorm, scale)
    tol = (2 * span(f64(z)) + 64) * R.U32 * bound + 1e-37
    if z.dtype == torch.bfloat16:
        tol = tol * (1 + R.U16) + R.U16 * np.abs(dz)
    err = np.abs(f64(got) - dz)
    assert got.dtype == z.dtype
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 2048, 32), (77, 333, 7), (257, 768, 12), (50, 12, 12)])
def test_gate_gradient_against_the_formula(cuda_device, T, E, K, renorm, score):
    for bf16 in (False, True):
        z = logits_of(T, E, T + E, bf16)
        idx, gate = B.lc_moe_gate(z, None, K, E, score=score, renorm=renorm, scale=1.5)
        dg = torch.from_numpy(np.random.default_rng(K).standard_normal((T, K)).astype(np.float32)).cuda()
        out = torch.full_like(z, 7.0)
        got = B.lc_moe_gate_backward(z, idx, dg, score=score, renorm=renorm, scale=1.5, dlogits=out)
        assert got is out
        check_backward(z, idx, dg, score, renorm, 1.5, got)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(cuda_device, renorm, score):
    """Central differences of the 64-bit gates with the picks held fixed: their error is h^2 / 6 times
    a third derivative (below 8 for scores in 0..1 and quotients of them), 2e-6 at h = 1e-3."""
    T, E, K = 4, 24, 5
    z = logits_of(T, E, 11, False, std=1.0)
    idx, _ = B.lc_moe_gate(z, None, K, E, score=score, renorm=renorm)
    dg = torch.from_numpy(np.random.default_rng(2).standard_normal((T, K)).astype(np.float32)).cuda()
    got = f64(B.lc_moe_gate_backward(z, idx, dg, score=score, renorm=renorm))
    z64, i, w = f64(z), idx.cpu().numpy(), f64(dg)
    h = 1e-3

    def total(zz):
        return (R.gates(zz, R.scores(zz, score), i, score, renorm, 1.0) * w).sum(1)
    for e in range(E):
        up, down = z64.copy(), z64.copy()
        up[:, e] += h
        down[:, e] -= h
        diff = (total(up) - total(down)) / (2 * h)
        assert np.abs(got[:, e] - diff).max() <= 2e-6 * np.abs(w).sum(1).max() + 1e-6


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_a_pick_with_nearly_all_of_the_share(cuda_device, score):
    """The largest pick's gradient is a sum over the others, not the difference of two numbers that are
    nearly equal: relative to itself it is within (2 R + 64) half steps, one half step more for each of
    K differences."""
    z = torch.tensor([[9.0, -9.0, -12.0, -30.0], [40.0, 3.0, 2.0, 1.0]], device="cuda")
    idx = torch.tensor([[0, 1, 2], [0, 1, 2]], dtype=torch.int32, device="cuda")
    dg = torch.tensor([[0.7, -1.3, 2.1], [1.0, 0.9, -4.0]], device="cuda")
    got = f64(B.lc_moe_gate_backward(z, idx, dg, score=score))
    s = R.scores(f64(z), score)[:, :3]
    if score == "sigmoid":  # 1 - s without its rounding
        f = 1.0 / (1.0 + np.exp(f64(z)[:, :3]))
    else:
        f = np.ones((2, 3))
    p = s / s.sum(1, keepdims=True)
    d = f64(dg)
    want = p * f * (p[:, None, :] * (d[:, :, None] - d[:, None, :])).sum(2)
    size = p * f * (p[:, None, :] * np.abs(d[:, :, None] - d[:, None, :])).sum(2)
    assert np.all(np.abs(got[:, :3] - want) <= (2 * 39 + 64 + 3) * R.U32 * size)
    assert np.all(got[:, 3] == 0)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E", [12, 77, 96, 1000, 2048])
def test_dense_gradient_of_a_row_that_is_nearly_one_hot(cuda_device, E, bf16):
    """The same for softmax gates that are not renormalised: 1 - s is the sum of the other shares. The
    fast exponential of -x is within 2 + 1.7 x steps, 4 + 3.4 x half steps, in each of the factors."""
    K = 5
    z = logits_of(4, E, E, False)
    z[:, 3] = 30.0
    z = z.bfloat16() if bf16 else z
    idx = torch.tensor([[3, 0, 1, 2, 5]] * 3 + [[4, 0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    dg = torch.from_numpy(np.random.default_rng(E).standard_normal((4, K)).astype(np.float32)).cuda()
    got = f64(B.lc_moe_gate_backward(z, idx, dg, renorm=False))
    z64, i, d = f64(z), idx.cpu().numpy(), f64(dg)
    s = R.scores(z64, "softmax")
    at = np.arange(4)[:, None]
    p = s[at, i]
    others = s.copy()
    others[at, i] = 0.0
    u = others.sum(1)[:, None]
    # s_r (sum_q p_q (d_r - d_q) + d_r u) at the picks, -s D elsewhere
    diff = d[:, :, None] - d[:, None, :]
    want, size = -s * (p * d).sum(1)[:, None], s * (p * np.abs(d)).sum(1)[:, None]
    want[at, i] = p * ((p[:, None, :] * diff).sum(2) + d * u)
    size[at, i] = p * ((p[:, None, :] * np.abs(diff)).sum(2) + np.abs(d) * u)
    tol = 2 * (3.4 * span(z64) + 100) * R.U32 * size + 1e-37
    if bf16:
        tol = tol * (1 + R.U16) + R.U16 * np.abs(want)
    err = np.abs(got - want)
    assert np.all(err <= tol), float((err / tol).max())


def dense_gradient(z64, i, d):
    """(dz, size) of softmax gates that are not renormalised, without a difference of nearly equal numbers:
    s_e (sum over the picked experts u of s_u (ds_e - ds_u) + ds_e (sum of the other shares)) at the picks, where
    ds_e is the sum of dgate over e's picks, and -s_i D elsewhere. size bounds the terms added; a sum over
    several picks of an expert is rounded before it enters a difference, by as many half steps at most."""
    T, E = z64.shape
    s = R.scores(z64, "softmax")
    want, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        picked = sorted(set(i[t].tolist()))
        ds = np.array([d[t][i[t] == e].sum() for e in picked])
        mag = np.array([np.abs(d[t][i[t] == e]).sum() for e in picked])
        many = np.array([(i[t] == e).sum() for e in picked])
        su = s[t, picked]
        rest = np.delete(s[t], picked).sum()
        want[t], size[t] = -s[t] * (su * ds).sum(), s[t] * (su * mag).sum()
        diff = ds[:, None] - ds[None, :]
        lost = R.U32 * ((many - 1) * mag)
        want[t, picked] = su * ((su * diff).sum(1) + ds * rest)
        size[t, picked] = su * ((su * np.abs(diff)).sum(1) + np.abs(ds) * rest) \
            + su * (su * (lost[:, None] + lost[None, :])).sum(1) / R.U32
    return want, size


def check_dense(z, idx, dg, scale=1.0):
    got = f64(B.lc_moe_gate_backward(z, idx, dg, renorm=False, scale=scale))
    z64 = f64(z)
    want, size = dense_gradient(z64, idx.cpu().numpy(), f64(dg))
    want, size = scale * want, scale * size
    tol = 2 * (3.4 * span(z64) + 100) * R.U32 * size + 1e-37
    if z.dtype == torch.bfloat16:
        tol = tol * (1 + R.U16) + R.U16 * np.abs(want)
    err = np.abs(got - want)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E", [12, 77, 768, 2048])
def test_dense_gradient_where_the_picks_hold_the_mass_together(cuda_device, E, bf16):
    """Picks of comparable share with equal or nearly equal dgate: ds - D is what little the others hold."""
    rng = np.random.default_rng(E)
    for K in (2, 3, 5):
        z = logits_of(8, E, E + K, False)
        idx = np.stack([rng.permutation(E)[:K] for _ in range(8)]).astype(np.int32)
        for t in range(8):
            z[t, idx[t].tolist()] = torch.from_numpy((6.0 + 4 * t + rng.random(K)).astype(np.float32)).cuda()
        z = z.bfloat16() if bf16 else z
        it = torch.from_numpy(idx).cuda()
        for dg in (np.ones((8, K)), 1 + 1e-6 * rng.standard_normal((8, K)), -3 + 0.1 * rng.random((8, K)),
                   rng.standard_normal((8, K))):
            dt = torch.from_numpy(dg.astype(np.float32)).cuda()
            check_dense(z, it, dt)
            check_dense(z, it, dt, scale=2.5)
        # the first expert picked twice
        rep = it.clone()
        rep[:, -1] = rep[:, 0]
        for dg in (np.full((8, K), 0.75), rng.standard_normal((8, K))):
            check_dense(z, rep, torch.from_numpy(dg.astype(np.float32)).cuda())


def test_gate_gradient_repeated_and_bad_picks(cuda_device):
    z = logits_of(4, 30, 3, False)
    idx = torch.tensor([[1, 1, 5, 1], [0, 29, 0, 29], [2, -1, 30, 4], [7, 8, 9, 10]], dtype=torch.int32, device="cuda")
    dg = torch.from_numpy(np.random.default_rng(9).standard_normal((4, 4)).astype(np.float32)).cuda()
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
            got = B.lc_moe_gate_backward(z, idx, dg, score=score, renorm=renorm, ws=ws)
            assert B.lc_moe_read_status(ws, raise_on_error=False) == B.DEV_IDX_RANGE
            check_backward(z, idx, dg, score, renorm, 1.0, got)


def test_gate_on_another_stream_and_in_a_graph(cuda_device):
    z = logits_of(300, 96, 1, False)
    b = torch.linspace(-0.1, 0.1, 96, device="cuda")
    kw = dict(score="sigmoid", groups=8, top_groups=4, group_rank=2, scale=2.5)
    want = B.lc_moe_gate(z, b, 6, 64, **kw)
    dg = torch.ones(300, 6, device="cuda")
    want_d = B.lc_moe_gate_backward(z, want[0], dg, score="softmax", renorm=False)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = B.lc_moe_gate(z, b, 6, 64, stream=st, **kw)
    got_d = B.lc_moe_gate_backward(z, got[0], dg, score="softmax", renorm=False, stream=st)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got_d, want_d)
    idx, gate, d = torch.zeros_like(want[0]), torch.zeros_like(want[1]), torch.zeros_like(z)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.lc_moe_gate(z, b, 6, 64, idx=idx, gate=gate, ws=ws, **kw)
        B.lc_moe_gate_backward(z, idx, dg, score="softmax", renorm=False, dlogits=d, ws=ws)
    for _ in range(2):
        idx.zero_(), gate.zero_(), d.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, want[0]) and torch.equal(gate, want[1]) and torch.equal(d, want_d)


def test_binding_refuses_wrong_tensors(cuda_device):
    z = logits_of(6, 16, 0, False)
    b = torch.zeros(16, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        B.lc_moe_gate(z.t().contiguous().t(), b, 2, 16)
    with pytest.raises(TypeError, match="bias"):
        B.lc_moe_gate(z, b.double(), 2, 16)
    with pytest.raises(ValueError, match="bias"):
        B.lc_moe_gate(z, b[:8], 2, 16)
    with pytest.raises(ValueError, match="ws"):
        B.lc_moe_gate(z, b, 2, 16, ws=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(B.LcMoeError, match="unsupported shape"):
        B.lc_moe_gate(z, b, 17, 16)
    with pytest.raises(B.LcMoeError, match="workspace"):
        B.lc_moe_gate(z, b, 2, 16, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    idx, gate = B.lc_moe_gate(z, b, 2, 16)
    with pytest.raises(B.LcMoeError, match="invalid argument"):
        B.lc_moe_gate_backward(z, idx, gate, dlogits=z)
    with pytest.raises(TypeError, match="dlogits"):
        B.lc_moe_gate_backward(z, idx, gate, dlogits=z.bfloat16())
    x = torch.zeros(6, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.LcMoeError, match="invalid argument"):
        B.lc_moe_combine_backward(x, x.clone(), x.clone(), gate, idx, dx=x)
    with pytest.raises(B.LcMoeError):
        B._shape_arg(2 ** 32 + 5, 64, 1, 0, 1, 64)


def test_calls_on_two_streams_at_once(cuda_device):
    """Two streams, one status word: nothing else is shared between calls."""
    z = [logits_of(3000, 96, s, False) for s in (1, 2)]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = [B.lc_moe_gate(v, None, 6, 64, score="sigmoid", groups=8, top_groups=4, group_rank=2) for v in z]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        got.append([B.lc_moe_gate(v, None, 6, 64, score="sigmoid", groups=8, top_groups=4, group_rank=2, ws=ws, stream=s)
                    for v, s in zip(z, streams)])
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
