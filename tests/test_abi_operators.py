"""Host-side checks of the general gates, the gradients and the 4-bit experts: bad arguments are
refused before any CUDA call, in the library and in the binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

from mixture_experts_zero_b200 import binding as B
from mixture_experts_zero_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.library()


P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(257)


def opts(score=0, groups=1, top_groups=1, group_rank=1, renorm=1, scale=1.0):
    return ctypes.byref(B.GateOpts(score, groups, top_groups, group_rank, renorm, scale))


def shape(T=16, d=128, N=8, Z=4, K=3, I=64):
    return ctypes.byref(B.Shape(T, d, N, Z, K, I))


def gate(lib, s=None, o=None, logits=P, kind=0, bias=P, idx=P, gate=P, counts=None, ws=P, n=256):
    return lib.lc_moe_gate(s or shape(), o, logits, kind, bias, idx, gate, counts, ws, n, None)


INV, SHAPE, SMALL, MIS = B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED_SHAPE, B.ERR_WORKSPACE_TOO_SMALL, B.ERR_MISALIGNED


@pytest.mark.parametrize("o,code", [
    (dict(score=2), INV), (dict(score=-1), INV), (dict(groups=0), INV), (dict(top_groups=0), INV),
    (dict(groups=2, top_groups=3), INV), (dict(group_rank=0), INV), (dict(group_rank=3), INV),
    (dict(renorm=2), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(groups=5), SHAPE),                # 12 experts
    (dict(groups=6, top_groups=1), SHAPE),  # 2 experts stay, K = 3
])
def test_gate_options_are_checked(lib, o, code):
    assert gate(lib, o=opts(**o)) == code
    assert lib.lc_moe_gate_backward(shape(), opts(**o), P, 0, P, P, ctypes.c_void_p(512), P, 256, None) == code
    assert lib.lc_moe_forward_w4(shape(), opts(**o), P, P, P, P, P, P, P, 32, P, None, None, None, P, 1 << 40,
                                 None) == code


def test_more_than_32_groups_are_refused(lib):
    s = shape(N=64, Z=2, K=2)
    assert gate(lib, s=s, o=opts(groups=33, top_groups=33)) == SHAPE


def test_gate_arguments(lib):
    for name in ("logits", "idx", "gate", "ws"):
        assert gate(lib, **{name: None}) == INV
    assert gate(lib, kind=2) == INV
    assert gate(lib, n=255) == SMALL
    assert gate(lib, logits=ctypes.c_void_p(258)) == MIS
    assert gate(lib, ws=ODD) == MIS
    assert gate(lib, s=shape(K=13)) == SHAPE
    assert gate(lib, s=shape(T=0)) == B.OK


def test_gate_backward_arguments(lib):
    good = [P, 0, P, P, ctypes.c_void_p(512), P, 256, None]
    def call(s=None, **kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return lib.lc_moe_gate_backward(s or shape(), None, *a)
    for k in ("a0", "a2", "a3", "a4", "a5"):
        assert call(**{k: None}) == INV
    assert call(a4=P) == INV                    # dlogits is the logits' buffer
    assert call(a1=7) == INV
    assert call(a6=10) == SMALL
    assert call(a4=ctypes.c_void_p(514)) == MIS
    assert call(s=shape(T=0)) == B.OK


def test_combine_backward_arguments(lib):
    def call(s=None, dout=P, x=P, y=P, rows=48, g=P, pr=P, dy=P, dg=P, dx=P, ws=P, n=256):
        return lib.lc_moe_combine_backward(s or shape(), dout, x, y, rows, g, pr, dy, dg, dx, ws, n, None)
    for k in ("dout", "x", "y", "g", "pr", "dy", "dg", "dx", "ws"):
        assert call(**{k: None}) == INV
    assert call(rows=-1) == INV
    a, b, c = (ctypes.c_void_p(v) for v in (4096, 8192, 12288))
    assert call(y=a, dy=a, dx=b) == INV         # in place
    assert call(y=a, dy=b, x=c, dx=c) == INV
    assert call(y=a, dy=b, dout=c, dx=c) == INV
    assert call(n=0) == SMALL
    for k in ("dout", "x", "y", "dy", "dx", "ws"):
        assert call(**{k: ctypes.c_void_p(264)}) == MIS
    assert call(s=shape(T=0)) == B.OK


def test_w4_arguments(lib):
    q = lib.lc_moe_quantize_w4
    assert q(P, 16, 64, 48, P, P, None) == INV
    assert q(P, 15, 64, 32, P, P, None) == INV
    assert q(P, 16, 96, 32, P, P, None) == INV
    assert q(P, 16, 64, 128, P, P, None) == INV
    assert q(None, 16, 64, 32, P, P, None) == INV
    assert q(ODD, 16, 64, 32, P, P, None) == MIS
    assert q(None, 0, 64, 32, None, None, None) == B.OK

    def ffn(s=None, group=32, n=256, **kw):
        a = dict(x=P, off=P, w13=P, s13=P, w2=P, s2=P, h=P, y=P, ws=P)
        a.update(kw)
        return lib.lc_moe_expert_ffn_w4(s or shape(), a["x"], a["off"], a["w13"], a["s13"], a["w2"], a["s2"], group,
                                        a["h"], a["y"], a["ws"], n, None)
    for k in ("x", "off", "w13", "s13", "w2", "s2", "h", "y", "ws"):
        assert ffn(**{k: None}) == INV
    for k in ("x", "w13", "s13", "w2", "s2", "h", "y", "ws"):
        assert ffn(**{k: ctypes.c_void_p(264)}) == MIS
    assert ffn(group=16) == INV
    assert ffn(group=128) == SHAPE              # I = 64
    assert ffn(n=255) == SMALL
    assert ffn(s=shape(T=0)) == B.OK

    def fwd(s=None, o=None, group=32, n=1 << 40, **kw):
        a = dict(x=P, wr=P, bias=P, w13=P, s13=P, w2=P, s2=P, out=P, ws=P)
        a.update(kw)
        return lib.lc_moe_forward_w4(s or shape(), o, a["x"], a["wr"], a["bias"], a["w13"], a["s13"], a["w2"], a["s2"],
                                     group, a["out"], None, None, None, a["ws"], n, None)
    for k in ("x", "wr", "bias", "w13", "s13", "w2", "s2", "out", "ws"):
        assert fwd(**{k: None}) == INV          # without options the bias is required
    need = B.lc_moe_workspace_bytes(B.Shape(16, 128, 8, 4, 3, 64), B.OP_FORWARD_W4)
    assert need > 0 and fwd(n=need - 1) == SMALL
    assert fwd(group=8) == INV
    assert fwd(group=128) == SHAPE
    assert fwd(s=shape(T=0)) == B.OK


def test_valid_calls_without_a_device_report_a_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert gate(lib) == B.ERR_CUDA
    assert lib.lc_moe_quantize_w4(P, 16, 64, 32, P, P, None) == B.ERR_CUDA


def test_binding_refuses_host_tensors_types_and_names():
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        B.lc_moe_gate(z, None, 2, 8)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        B.lc_moe_gate(z.double(), None, 2, 8)
    with pytest.raises(ValueError, match="dimensions"):
        B.lc_moe_gate(z[0], None, 2, 8)
    with pytest.raises(ValueError, match="score"):
        B._gate_opts("tanh", 1, 1, 1, True, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        B.lc_moe_quantize_w4(torch.zeros(16, 64, dtype=torch.bfloat16))


class _Elsewhere:
    """A tensor of another device than the current one, for the check alone."""
    is_cuda = True
    device = torch.device("cuda", 7)

    def is_contiguous(self):
        return True


def test_binding_refuses_tensors_of_another_device():
    with pytest.raises(ValueError, match="current device"):
        B._one_device(x=_Elsewhere())


def _options(*a):
    return B._gate_opts(*a)._obj


@pytest.mark.parametrize("make", [torch.tensor, np.array], ids=["tensor", "array"])
def test_options_follow_a_scalar_that_changes(make):
    """A factor held in a 0-d tensor or array is read anew by every call."""
    scale = make(1.5)
    assert _options("softmax", 1, 1, 1, True, scale).scale == 1.5
    scale += 1.5
    assert _options("softmax", 1, 1, 1, True, scale).scale == 3.0
    groups, renorm = make(4), make(True)
    first = _options("softmax", groups, groups, 1, renorm, 1.0)
    assert (first.groups, first.top_groups, first.renorm) == (4, 4, 1)
    groups *= 2
    renorm &= False
    second = _options("softmax", groups, groups, 1, renorm, 1.0)
    assert (second.groups, second.top_groups, second.renorm) == (8, 8, 0)
    assert (first.groups, first.renorm) == (4, 1)


def test_shapes_follow_a_scalar_that_changes():
    k = torch.tensor(3)
    assert B._shape_arg(5, 64, 8, 4, k, 64)._obj.K == 3
    k += 1
    assert B._shape_arg(5, 64, 8, 4, k, 64)._obj.K == 4
    assert B._shape_arg(5, 64, torch.tensor(8), torch.tensor(4), k, 64)._obj.N == 8


def test_options_keep_the_sign_of_zero_and_refuse_what_is_no_number():
    for scale in (0.0, -0.0, 0.0):
        assert math.copysign(1.0, _options("softmax", 1, 1, 1, True, scale).scale) == math.copysign(1.0, scale)
    for bad in ("1.5", None):
        with pytest.raises(TypeError):
            B._gate_opts("softmax", 1, 1, 1, True, bad)
    with pytest.raises(TypeError):
        B._gate_opts("softmax", 1.0, 1, 1, True, 1.0)


@pytest.mark.parametrize("at", [0, 1, 2])
def test_options_beyond_32_bits_are_refused(at):
    """The struct's fields are 32 bits wide: 2^32 + 1 is not 1."""
    for v in (2 ** 32 + 1, 2 ** 31, -2 ** 32 + 1):
        a = [1, 1, 1]
        a[at] = v
        with pytest.raises(B.LcMoeError, match="invalid argument"):
            B._gate_opts("softmax", *a, True, 1.0)


def _at(v):
    return ctypes.c_void_p(v)


# one token row of d = 128 is 256 bytes, T = 16 rows 4096; K = 3
ROOM = dict(dout=1 << 16, x=2 << 16, y=3 << 16, g=4 << 16, pr=5 << 16, dy=6 << 16, dg=7 << 16, dx=8 << 16)


@pytest.mark.parametrize("out,rows", [("dy", 48), ("dx", 16)])
@pytest.mark.parametrize("other", ["dout", "x", "y", "dy", "dx", "g", "pr", "dg"])
def test_combine_backward_refuses_buffers_that_overlap(lib, out, rows, other):
    """Whatever a pick reads, another pick's write must not reach: one buffer for two, or parts of one."""
    if out == other:
        return
    size = dict(dout=4096, x=4096, y=48 * 256, dy=48 * 256, dx=4096, g=192, pr=192, dg=192)
    for delta in (0, size[other] // 16 * 16 - 16, 16 - rows * 256):
        a = {k: _at(v) for k, v in ROOM.items()}
        a[out] = _at(ROOM[other] + delta)
        assert lib.lc_moe_combine_backward(shape(), a["dout"], a["x"], a["y"], 48, a["g"], a["pr"], a["dy"], a["dg"], a["dx"],
                                           P, 256, None) == INV, delta
    # next to it
    for at in (ROOM[other] + size[other], ROOM[other] - rows * 256):
        a = {k: _at(v) for k, v in ROOM.items()}
        a[out] = _at(at)
        if not torch.cuda.is_available():
            assert lib.lc_moe_combine_backward(shape(), a["dout"], a["x"], a["y"], 48, a["g"], a["pr"], a["dy"], a["dg"],
                                               a["dx"], P, 256, None) == B.ERR_CUDA


def test_combine_backward_refuses_dgate_over_the_gates(lib):
    """The gates of a token are read by every block that has some of its picks."""
    a = {k: _at(v) for k, v in ROOM.items()}
    for other in ("g", "pr"):
        for delta in (0, 188, -188):
            assert lib.lc_moe_combine_backward(shape(), a["dout"], a["x"], a["y"], 48, a["g"], a["pr"], a["dy"],
                                               _at(ROOM[other] + delta), a["dx"], P, 256, None) == INV


@pytest.mark.parametrize("kind,width", [(0, 4), (1, 2)])
def test_gate_backward_refuses_buffers_that_overlap(lib, kind, width):
    """dlogits [16, 12] over a part of the logits, of idx or of dgate."""
    n, z, i, g = 16 * 12 * width, 1 << 16, 2 << 16, 3 << 16
    for at in (z, z + n - width, z - n + width, i + 188, i - n + 4, g + 188, g - n + 4):
        assert lib.lc_moe_gate_backward(shape(), None, _at(z), kind, _at(i), _at(g), _at(at), P, 256, None) == INV
    if not torch.cuda.is_available():
        for at in (z + n, z - n, i + 192, g - n):
            assert lib.lc_moe_gate_backward(shape(), None, _at(z), kind, _at(i), _at(g), _at(at), P, 256, None) == B.ERR_CUDA


def test_w4_ffn_refuses_h_over_its_inputs(lib):
    """H [48, 64] is written while rows of x_perm [48, 128] are read, and read while Y [48, 128] is written."""
    x, h, y, off = 1 << 20, 2 << 20, 3 << 20, 4 << 20

    def call(h, y):
        return lib.lc_moe_expert_ffn_w4(shape(), _at(x), _at(off), P, P, P, P, 32, _at(h), _at(y), P, 256, None)
    for at in (x, x + 48 * 256 - 16, x - 48 * 128 + 16, y, y + 48 * 256 - 16, y - 48 * 128 + 16, off, off + 16):
        assert call(at, y) == INV
    assert call(h, off - 48 * 256 + 16) == INV
    if not torch.cuda.is_available():
        for at in (x + 48 * 256, y - 48 * 128):
            assert call(at, y) == B.ERR_CUDA
        assert call(h, x) == B.ERR_CUDA     # Y over x_perm: H is complete before Y begins
