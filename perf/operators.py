"""Cases of the routing and 4-bit expert operators: their inputs, plain forms and exact values.

Four operators of the MoE layer, each reached through the package's entry points:

  gate          logits [T, E] -> K experts per token and their gates (``lc_moe_gate``): softmax or
                sigmoid scores, a balance bias that steers the choice only, a first choice among
                groups of experts, gates renormalised or not, times a factor
  gate_bwd      the gradient of those gates for the logits (``lc_moe_gate_backward``)
  combine_bwd   the gradient of the layer's weighted sum for the experts' rows, the gates and the
                tokens that zero-computation experts hand through (``lc_moe_combine_backward``)
  ffn_w4        the SwiGLU experts on rows grouped by expert, with 4-bit weights and a bf16 scale
                per group of 32, 64 or 128 input columns (``lc_moe_expert_ffn_w4``)

``run`` computes them from elementary torch operations, or through the package where ``own`` is
set; ``exact`` gives the same outputs in 64 bits, written apart from both.
"""
import math

import numpy as np
import torch

own = False

# --------------------------------------------------------------------------------- the cases --


def _gate(name, T, E, K, **kw):
    case = dict(name=name, op="gate", T=T, E=E, K=K, score="softmax", groups=1, top_groups=1, group_rank=1,
                renorm=True, scale=1.0, bias=True, off=0, bf16=False)
    case.update(kw)
    return case


def listed():
    return [
        # routing of one decoded token at the LongCat-Flash router width (512 FFN + 256 zero
        # experts): latency
        _gate("gate_one", 1, 768, 12),
        # a decode batch of a layer with 96 experts in 8 groups, some experts switched off
        _gate("gate_decode_groups", 128, 96, 6, score="sigmoid", groups=8, top_groups=4, group_rank=2,
              scale=2.5, off=5),
        # a prefill batch at the LongCat-Flash router width
        _gate("gate_prefill", 16384, 768, 12),
        # the same batch with sigmoid scores and a choice of 4 of 8 groups first
        _gate("gate_prefill_groups", 16384, 768, 12, score="sigmoid", groups=8, top_groups=4, group_rank=2,
              scale=2.5),
        # ragged: a token count and an expert count that divide by nothing, bf16 logits (equal
        # logits are common), gates not renormalised, no bias
        _gate("gate_odd", 4099, 333, 7, renorm=False, bias=False, bf16=True),
        # training: the gradient of softmax gates that are not renormalised reaches every logit
        dict(name="gate_bwd_prefill", op="gate_bwd", T=16384, E=768, K=12, score="softmax", renorm=False,
             scale=1.0, bf16=False),
        # training, ragged: renormalised sigmoid gates on bf16 logits
        dict(name="gate_bwd_odd", op="gate_bwd", T=1023, E=333, K=7, score="sigmoid", renorm=True,
             scale=2.5, bf16=True),
        # training: a micro-batch of a small layer
        dict(name="combine_bwd_small", op="combine_bwd", T=100, d=1024, K=6, N=64, Z=32),
        # training: the prefill batch at the LongCat-Flash width, a third of the picks zero experts
        dict(name="combine_bwd_prefill", op="combine_bwd", T=16384, d=6144, K=12, N=512, Z=256),
        # serving: one token through its 8 experts at the LongCat-Flash expert shape
        dict(name="ffn_w4_one", op="ffn_w4", T=1, d=6144, I=2048, K=8, N=32, Z=0, group=128, zipf=0.0),
        # serving: a decode batch of 128 tokens over 512 experts, about 2 rows for each
        dict(name="ffn_w4_decode", op="ffn_w4", T=128, d=6144, I=2048, K=12, N=512, Z=256, group=64, zipf=0.0),
        # serving: a batch of a small layer with uneven experts, from none to hundreds of rows
        dict(name="ffn_w4_uneven", op="ffn_w4", T=700, d=1024, I=256, K=6, N=64, Z=32, group=32, zipf=1.1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_bwd", "combine_bwd", "ffn_w4", "ffn_w4"])
    if op in ("gate", "gate_bwd"):
        groups = rng.choice([1, 1, 2, 3, 4, 8, 16]) if op == "gate" else 1
        E = groups * _log(rng, max(2, 8 // groups), 2048 // groups)
        T = _log(rng, 1, max(1, min(20000, 16384 * 768 // E)))
        top = rng.randint(1, groups)
        K = rng.randint(1, min(32, top * (E // groups), 16))
        case = dict(op=op, T=T, E=E, K=K, score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5, rng.uniform(0.5, 3.0)]), bf16=rng.random() < 0.4)
        if op == "gate":
            case.update(groups=groups, top_groups=top, group_rank=rng.choice([1, 2]), bias=rng.random() < 0.7,
                        off=0)
            if case["bias"] and rng.random() < 0.3:
                case["off"] = rng.randint(1, max(1, E // 8))
        return case
    if op == "combine_bwd":
        d = 64 * _log(rng, 1, 96)
        T = _log(rng, 1, min(16384, 16384 * 6144 // d))
        N = _log(rng, 4, 512)
        Z = rng.choice([0, N // 2, N])
        return dict(op=op, T=T, d=d, K=rng.randint(1, min(12, N + Z)), N=N, Z=Z)
    group = rng.choice([32, 64, 128])
    unit = max(64, group)
    d, I = unit * _log(rng, 1, 6144 // unit), unit * _log(rng, 1, 2048 // unit)
    N = _log(rng, 1, max(1, min(512, 128 * 6144 * 2048 // (d * I))))
    Z = rng.choice([0, N // 2])
    K = rng.randint(1, min(12, N + Z))
    T = _log(rng, 1, 600)
    return dict(op=op, T=T, d=d, I=I, K=K, N=N, Z=Z, group=group, zipf=rng.choice([0.0, 1.1]))


# ------------------------------------------------------------------------------------ inputs --


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _logits(case, g):
    # a router's logits: the dot products of unit-variance activations with its rows
    z = torch.randn(case["T"], case["E"], generator=g, device="cuda") * 2.0
    return z.to(torch.bfloat16) if case["bf16"] else z


def _picks(T, K, N, Z, g, zipf=0.0):
    """K distinct experts of N + Z for each token, as a router's top-K of noisy scores."""
    key = -torch.log(-torch.log(torch.rand(T, N + Z, generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)))
    if zipf:
        rank = torch.randperm(N + Z, generator=g, device="cuda") + 1
        key = key - zipf * torch.log(rank.float())
    return torch.sort(key, dim=1, descending=True).indices[:, :K].contiguous()


def _w4(rows, cols, group, experts, g):
    """4-bit weights of ``experts`` matrices [rows, cols]: normal weights quantised to -7..7 with a
    bf16 scale per group of columns. Codes are stored as the value plus 8 in 512-byte tiles of 16
    rows x 64 columns: byte 16 * (4 * (r % 8) + (c % 32) // 8) + 4 * (2 * (c % 64 // 32) + r % 16 // 8)
    onward holds a 32-bit word of the 8 columns c - c % 8 ..., whose nibble p is column
    2 * (p % 4) + p // 4 of the 8. Scales are stored [rows / 16, cols / group, 8, 2]: row
    16 a + 8 h + b at [a, :, b, h]."""
    codes = torch.empty(experts, rows, cols // 2, dtype=torch.uint8, device="cuda")
    scale = torch.empty(experts, rows // 16, cols // group, 16, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(rows, cols, device="cuda")
    for e in range(experts):
        # the largest of a group of normal values is about 2.5 deviations: a step of 2.5 / 7
        q.normal_(generator=g).mul_(2.8).round_().clamp_(-7, 7).add_(8)
        n = q.to(torch.uint8).view(rows // 16, 2, 8, cols // 64, 2, 4, 4, 2)
        n = n.permute(0, 3, 2, 5, 4, 1, 7, 6).reshape(-1, 2)
        codes[e] = (n[:, 0] | (n[:, 1] << 4)).view(rows, cols // 2)
        s = torch.rand(scale[e].shape, generator=g, device="cuda") * 0.5 + 0.75
        scale[e] = s / (2.8 * math.sqrt(cols))
    return codes, scale


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("gate", "gate_bwd"):
        T, E, K = case["T"], case["E"], case["K"]
        s["logits"] = _logits(case, g)
        s["status"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        if op == "gate":
            s["bias"] = None
            if case["bias"]:
                s["bias"] = torch.rand(E, generator=g, device="cuda") * 0.2 - 0.1
                if case["off"]:
                    # experts that a deployment has switched off
                    s["bias"][torch.randperm(E, generator=g, device="cuda")[:case["off"]]] = -math.inf
        else:
            key = s["logits"].float() + torch.randn(T, E, generator=g, device="cuda") * 0.5
            s["idx"] = torch.sort(key, dim=1, descending=True).indices[:, :K].to(torch.int32).contiguous()
            s["dgate"] = torch.randn(T, K, generator=g, device="cuda")
        return s
    T, K, N, Z, d = case["T"], case["K"], case["N"], case["Z"], case["d"]
    pick = _picks(T, K, N, Z, g, case.get("zipf", 0.0))
    # rows grouped by expert, in token order within one
    flat = pick.reshape(-1)
    order = torch.sort(torch.where(flat < N, flat, N), stable=True).indices
    counts = torch.bincount(flat, minlength=N + Z)[:N]
    rows = int(counts.sum())
    s["status"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    if op == "combine_bwd":
        pair_row = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
        pair_row[order[:rows]] = torch.arange(rows, dtype=torch.int32, device="cuda")
        s["pair_row"] = pair_row.view(T, K)
        s["gate"] = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), dim=1)
        # y holds a row for every pick, the first ``rows`` of them in use
        for name, n in (("dout", T), ("x", T), ("y", T * K)):
            s[name] = torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16)
        s["dy"] = torch.zeros_like(s["y"])
        return s
    I = case["I"]
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["counts"] = counts.tolist()
    s["x"] = torch.randn(T * K, d, generator=g, device="cuda").to(torch.bfloat16)
    s["w13q"], s["w13_scale"] = _w4(2 * I, d, case["group"], N, g)
    s["w2q"], s["w2_scale"] = _w4(d, I, case["group"], N, g)
    # rows behind the last expert's stay as they are
    s["h"] = torch.zeros(T * K, I, dtype=torch.bfloat16, device="cuda")
    s["y"] = torch.zeros(T * K, d, dtype=torch.bfloat16, device="cuda")
    return s


# -------------------------------------------------------------------------------- plain forms --


def _scores(z, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    m = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return e / e.sum(dim=1, keepdim=True).clamp_min(1.0)


def _plain_gate(s, c):
    # 64 bits: two keys that lie next to each other decide which experts are picked
    score = _scores(s["logits"].double(), c["score"])
    key = score if s["bias"] is None else score + s["bias"].double()
    T, E = key.shape
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    if c["groups"] > 1:
        of = key.view(T, c["groups"], E // c["groups"])
        best = torch.sort(of, dim=2, descending=True).values[:, :, :c["group_rank"]].sum(dim=2)
        top = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros(T, c["groups"], device=key.device).scatter_(1, top, 1.0)
        kept = torch.gather(kept, 1, order // (E // c["groups"]))
        order = torch.gather(order, 1, torch.sort(kept, dim=1, descending=True, stable=True).indices)
    idx = order[:, :c["K"]]
    gate = torch.gather(score, 1, idx)
    if c["renorm"]:
        total = gate.sum(dim=1, keepdim=True)
        gate = torch.where(total > 0, gate / total, torch.zeros_like(gate))
    return idx.to(torch.int32), (gate * c["scale"]).float()


def _plain_gate_bwd(s, c):
    score = _scores(s["logits"].float(), c["score"])
    idx = s["idx"].long()
    chosen, dgate = torch.gather(score, 1, idx), s["dgate"] * c["scale"]
    if c["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        dgate = (dgate - (dgate * chosen).sum(dim=1, keepdim=True) / total) / total
    dscore = torch.zeros_like(score).scatter_add_(1, idx, dgate)
    if c["score"] == "sigmoid":
        dz = dscore * score * (1.0 - score)
    else:
        dz = score * (dscore - (dscore * score).sum(dim=1, keepdim=True))
    return dz.to(s["logits"].dtype)


def _plain_combine_bwd(s, c):
    T, K, d = c["T"], c["K"], c["d"]
    zero = s["pair_row"] < 0
    row = s["pair_row"].long().clamp_min(0)
    dout = s["dout"].float()
    v = torch.where(zero[:, :, None], s["x"][:, None, :], s["y"][row.view(-1)].view(T, K, d)).float()
    dgate = (v * dout[:, None, :]).sum(dim=2)
    del v
    token = torch.arange(T, device=dout.device)[:, None].expand(T, K)[~zero]
    dy = s["dy"].clone()
    dy[row[~zero]] = (s["gate"][~zero][:, None] * dout[token]).to(torch.bfloat16)
    dx = torch.where(zero, s["gate"], torch.zeros_like(s["gate"])).sum(dim=1, keepdim=True) * dout
    return dy, dgate, dx.to(torch.bfloat16)


def _plain_w4(codes, scale, rows, cols):
    """One expert's matrix [rows, cols] in fp32 from its codes and scales."""
    b = codes.view(-1)
    n = torch.stack([b & 15, b >> 4], dim=1).float().sub_(8.0)
    w = n.view(rows // 16, cols // 64, 8, 4, 2, 2, 2, 4).permute(0, 5, 2, 1, 4, 3, 7, 6).reshape(rows, cols)
    s = scale.float().view(rows // 16, -1, 8, 2).permute(0, 3, 2, 1).reshape(rows, -1, 1)
    return w.view(rows, s.shape[1], -1).mul(s).view(rows, cols)


def _plain_ffn_w4(s, c):
    d, I = c["d"], c["I"]
    h, y = s["h"], s["y"]
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            x = s["x"][at:at + n].float()
            gu = x @ _plain_w4(s["w13q"][e], s["w13_scale"][e], 2 * I, d).t()
            g, u = gu[:, :I], gu[:, I:]
            # H is an output of the operator: what it holds in bf16 is what the second product reads
            h[at:at + n] = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)
            y[at:at + n] = (h[at:at + n].float() @ _plain_w4(s["w2q"][e], s["w2_scale"][e], d, I).t()).to(torch.bfloat16)
            at += n
    return h, y


# ---------------------------------------------------------------------------------------- run --


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return dict(gate=_plain_gate, gate_bwd=_plain_gate_bwd, combine_bwd=_plain_combine_bwd,
                    ffn_w4=_plain_ffn_w4)[op](s, c)
    import mixture_experts_zero_b200 as moe
    if op == "gate":
        return moe.lc_moe_gate(s["logits"], s["bias"], c["K"], c["E"], score=c["score"], groups=c["groups"],
                               top_groups=c["top_groups"], group_rank=c["group_rank"], renorm=c["renorm"],
                               scale=c["scale"], ws=s["status"])
    if op == "gate_bwd":
        return moe.lc_moe_gate_backward(s["logits"], s["idx"], s["dgate"], score=c["score"], renorm=c["renorm"],
                                        scale=c["scale"], ws=s["status"])
    if op == "combine_bwd":
        return moe.lc_moe_combine_backward(s["dout"], s["x"], s["y"], s["gate"], s["pair_row"], dy=s["dy"],
                                           ws=s["status"])
    return moe.lc_moe_expert_ffn_w4(s["x"], s["offsets"], s["w13q"], s["w13_scale"], s["w2q"], s["w2_scale"],
                                    c["T"], c["K"], h=s["h"], y=s["y"], ws=s["status"])


def work(case):
    c, op = case, case["op"]
    T, K = c["T"], c["K"]
    if op in ("gate", "gate_bwd"):
        wide = 2 if c["bf16"] else 4
        # gate: logits in, picks and gates out; its gradient: picks and dgate in, dlogits out, and the
        # logits in (all of them only where the gates are a softmax over all experts)
        logits = T * c["E"] * wide
        if op == "gate":
            return dict(bytes=logits + T * K * 8 + (c["E"] * 4 if c["bias"] else 0), flops=T * c["E"] * 4)
        dense = c["score"] == "softmax" and not c["renorm"]
        return dict(bytes=logits + T * K * 8 + (logits if dense else T * K * wide), flops=T * c["E"] * 4)
    share = K * c["N"] / (c["N"] + c["Z"])  # FFN experts per token, on average
    if op == "combine_bwd":
        d = c["d"]
        zeros = 1 if c["Z"] else 0
        # dout (and x) in, each FFN row in and its gradient out, dx out, gates and picks in, dgate out
        return dict(bytes=T * d * 2 * (2 + zeros) + T * share * d * 4 + T * K * 12, flops=T * d * (2 * K + share))
    d, I, N = c["d"], c["I"], c["N"]
    rows = T * share
    # experts that at least one of the T * share picks falls on, were they spread evenly
    live = N * (1.0 - (1.0 - min(1.0, K / (N + c["Z"]))) ** T)
    weights = live * 3 * d * I * (0.5 + 2.0 / c["group"])
    return dict(bytes=weights + rows * (2 * d + 2 * I) * 2, flops=rows * 6 * d * I)


# -------------------------------------------------------------------------------------- exact --


def exact(case, seed):
    s = prepare(case, seed)
    return dict(gate=_exact_gate, gate_bwd=_exact_gate_bwd, combine_bwd=_exact_combine_bwd,
                ffn_w4=_exact_ffn_w4)[case["op"]](s, case)


def _exact_scores(s, c):
    z = s["logits"].double().cpu().numpy()
    if c["score"] == "sigmoid":
        return np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))
    e = np.exp(z - z.max(axis=1)[:, None])
    return e / e.sum(axis=1)[:, None]


def _exact_gate(s, c):
    score = _exact_scores(s, c)
    key = score.copy() if s["bias"] is None else score + s["bias"].double().cpu().numpy()
    T, E = key.shape
    allowed = np.ones((T, E), bool)
    if c["groups"] > 1:
        size = E // c["groups"]
        best = -np.sort(-key.reshape(T, c["groups"], size), axis=2)[:, :, :c["group_rank"]].sum(axis=2)
        rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1, kind="stable")
        allowed = np.repeat(rank < c["top_groups"], size, axis=1)
    # experts of the groups left out come after every other, also after those with a key of -inf
    tail = np.where(allowed, np.where(np.isinf(key), 1e30, -key), 2e30)
    idx = np.argsort(tail, axis=1, kind="stable")[:, :c["K"]]
    gate = np.take_along_axis(score, idx, axis=1)
    if c["renorm"]:
        gate = gate / gate.sum(axis=1)[:, None]
    return idx.astype(np.int32), gate * c["scale"]


def _exact_gate_bwd(s, c):
    score = _exact_scores(s, c)
    T, E = score.shape
    at = np.arange(T)[:, None]
    idx = s["idx"].cpu().numpy()
    dg = s["dgate"].double().cpu().numpy() * c["scale"]
    p = score[at, idx]
    # dg/dz through d(score)/dz first: J = dscore_r/dz_i, then the quotient's derivative
    if c["renorm"]:
        q = p.sum(axis=1)[:, None]
        ds = dg / q - (dg * p).sum(axis=1)[:, None] / q ** 2
    else:
        ds = dg
    dz = np.zeros((T, E))
    if c["score"] == "sigmoid":
        np.add.at(dz, (at, idx), ds * p * (1.0 - p))
    else:
        dz -= (ds * p).sum(axis=1)[:, None] * score
        np.add.at(dz, (at, idx), ds * p)
    return dz


def _exact_combine_bwd(s, c):
    T, K, d = c["T"], c["K"], c["d"]
    dout, pair = s["dout"].double(), s["pair_row"].long()
    dy = s["dy"].double()
    dgate = torch.empty(T, K, dtype=torch.float64, device="cuda")
    dx = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for r in range(K):
        own_row = pair[:, r] >= 0
        source = s["x"].double()
        source[own_row] = s["y"][pair[own_row, r]].double()
        dgate[:, r] = torch.einsum("td,td->t", source, dout)
        part = s["gate"][:, r].double()[:, None] * dout
        dy[pair[own_row, r]] = part[own_row]
        dx[~own_row] += part[~own_row]
    return dy, dgate, dx


def _exact_w4(codes, scale, rows, cols, group):
    r = torch.arange(rows, device="cuda")[:, None]
    k = torch.arange(cols, device="cuda")[None, :]
    tile = (r // 16) * (cols // 64) + k // 64
    byte = tile * 512 + 16 * (4 * (r % 8) + (k % 32) // 8) + 4 * (2 * ((k % 64) // 32) + (r % 16) // 8)
    p = (k % 8) // 2 + 4 * (k % 2) + 0 * r
    code = (codes.reshape(-1)[byte + p // 2].long() >> (4 * (p % 2))) & 15
    step = scale.reshape(rows // 16, cols // group, 16)[r // 16, k // group, 2 * (r % 8) + (r % 16) // 8]
    return (code - 8).double() * step.double()


def _exact_ffn_w4(s, c):
    d, I = c["d"], c["I"]
    h, y = s["h"].double(), s["y"].double()
    ends = s["offsets"].tolist()
    for e in range(c["N"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        w = _exact_w4(s["w13q"][e], s["w13_scale"][e], 2 * I, d, c["group"])
        g, u = torch.split(torch.matmul(s["x"][a:b].double(), w.T), I, dim=1)
        h[a:b] = g * torch.sigmoid(g) * u
        w = _exact_w4(s["w2q"][e], s["w2_scale"][e], d, I, c["group"])
        y[a:b] = torch.matmul(h[a:b].to(torch.bfloat16).double(), w.T)
    return h, y
