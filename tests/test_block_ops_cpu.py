"""Host-side checks of the operators around the layer: every refusal returns its
code before anything is launched (the pointers are never dereferenced), sizes,
and the binding's argument checks (no GPU needed)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_30_b200 import binding as B
from mixture_experts_layer_30_b200 import build as BUILD

FAKE = ctypes.c_void_p(0x10000)
BIG = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def at(offset):
    return ctypes.c_void_p(0x10000 + offset)


@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.lib()


def norm(lib, **over):
    a = dict(T=4, d=64, dtype=B.MOE_BF16, x=FAKE, residual=FAKE, weight=FAKE, eps=1e-5,
             sum_out=at(4096), y=FAKE, inv=FAKE, q=FAKE, sf=FAKE)
    a.update(over)
    return lib.moe_rmsnorm(a["T"], a["d"], a["dtype"], a["x"], a["residual"], a["weight"],
                           a["eps"], a["sum_out"], a["y"], a["inv"], a["q"], a["sf"], None)


@pytest.mark.parametrize("over,code,word", [
    (dict(dtype=7), INVALID, b"dtype"),
    (dict(T=-1), INVALID, b"bad shape"),
    (dict(d=0), INVALID, b"bad shape"),
    (dict(d=60, q=None, sf=None), UNSUPPORTED, b"multiple of 8"),
    (dict(d=62, dtype=B.MOE_F32, q=None, sf=None), UNSUPPORTED, b"multiple of 4"),
    (dict(eps=-1e-5), INVALID, b"eps"),
    (dict(eps=float("nan")), INVALID, b"eps"),
    (dict(eps=float("inf")), INVALID, b"eps"),
    (dict(sf=None), INVALID, b"together"),
    (dict(q=None), INVALID, b"together"),
    (dict(y=None, q=None, sf=None), INVALID, b"neither"),
    (dict(d=72), UNSUPPORTED, b"MXFP8"),
    (dict(dtype=B.MOE_F32), UNSUPPORTED, b"MXFP8"),
    (dict(x=None), INVALID, b"x is NULL"),
    (dict(x=at(8)), INVALID, b"x must be"),
    (dict(residual=at(4)), INVALID, b"residual"),
    (dict(weight=None), INVALID, b"weight"),
    (dict(sum_out=None), INVALID, b"sum_out"),
    (dict(residual=None), INVALID, b"sum_out"),
    (dict(y=at(4096)), INVALID, b"same buffer"),
    (dict(inv=at(2)), INVALID, b"inv_rms"),
])
def test_rmsnorm_refusals(lib, over, code, word):
    assert norm(lib, **over) == code
    assert word in lib.moe_last_error()


def test_rmsnorm_of_no_rows_launches_nothing(lib):
    before = B.kernel_launches()
    assert norm(lib, T=0) == 0
    assert B.kernel_launches() == before


def test_rmsnorm_backward_refusals(lib):
    need = lib.moe_rmsnorm_workspace_bytes(4, 64)
    assert need >= 256 + 4 * 64 * 4
    assert lib.moe_rmsnorm_workspace_bytes(-1, 64) == 0
    assert lib.moe_rmsnorm_workspace_bytes(4, 0) == 0

    def call(**over):
        a = dict(T=4, d=64, s=FAKE, w=FAKE, inv=FAKE, dy=FAKE, dsum=None, dx=FAKE, dw=FAKE,
                 ws=FAKE, n=need)
        a.update(over)
        return lib.moe_rmsnorm_backward(a["T"], a["d"], B.MOE_BF16, a["s"], a["w"], a["inv"],
                                        a["dy"], a["dsum"], a["dx"], a["dw"], a["ws"], a["n"],
                                        None)
    assert call(n=need - 256) == WORKSPACE
    assert call(ws=None) == INVALID
    assert call(ws=at(8)) == INVALID
    assert call(d=60, n=BIG) == UNSUPPORTED
    for name in ("s", "w", "inv", "dy", "dx", "dw"):
        assert call(**{name: None}) == INVALID, name
    assert call(dsum=at(2)) == INVALID


def test_permute_mxfp8_rows_refusals(lib):
    s = B.make_shape(16, 256, 4, 2, 2, 128, "bf16")
    nb = B.workspace_bytes(s)

    def call(shape=s, q=FAKE, sf=FAKE, off=FAKE, out=FAKE, n=nb):
        return lib.moe_permute_mxfp8_rows(ctypes.byref(shape), q, sf, FAKE, FAKE, off, FAKE, FAKE,
                                          out, FAKE, FAKE, n, None)
    assert call(q=None) == INVALID
    assert b"x_q" in lib.moe_last_error()
    assert call(sf=at(8)) == INVALID
    assert call(off=None) == INVALID
    assert call(out=at(4)) == INVALID
    assert call(n=nb - 256) == WORKSPACE
    assert call(shape=B.make_shape(16, 192, 4, 2, 2, 128, "bf16"), n=BIG) == UNSUPPORTED
    assert call(shape=B.make_shape(16, 256, 4, 2, 2, 128, "f32"), n=BIG) == UNSUPPORTED


def test_w4_sizes(lib):
    # blocks of 16 rows x 128 columns: 1024 bytes of codes, 16 * 128 / group scales
    assert lib.moe_w4_code_bytes(3, 16, 128) == 3 * 1024
    assert lib.moe_w4_code_bytes(3, 17, 129) == 3 * 4 * 1024
    assert lib.moe_w4_scale_bytes(3, 17, 129, 32) == 3 * 4 * 16 * 4 * 2
    assert lib.moe_w4_scale_bytes(1, 16, 128, 128) == 32
    assert lib.moe_w4_scale_bytes(1, 16, 128, 48) == 0
    assert lib.moe_w4_code_bytes(-1, 16, 128) == 0
    # offsets beyond 32 bits
    assert lib.moe_w4_code_bytes(512, 2048, 6144) == 512 * 2048 * 6144 // 2


def test_w4_refusals(lib):
    s = B.make_shape(16, 256, 4, 2, 2, 128, "bf16")
    nb = B.workspace_bytes(s)

    def quantize(n=1, rows=16, cols=128, group=32, dtype=B.MOE_BF16, src=FAKE, q=FAKE, sc=FAKE):
        return lib.moe_quantize_weights_w4(n, rows, cols, group, dtype, src, q, sc, None)
    assert quantize(group=48) == UNSUPPORTED
    assert quantize(dtype=3) == INVALID
    assert quantize(rows=-1) == INVALID
    assert quantize(src=None) == INVALID
    assert quantize(q=at(8)) == INVALID
    assert quantize(sc=None) == INVALID
    assert quantize(rows=0) == 0
    assert quantize(n=1 << 20, rows=1 << 20) == UNSUPPORTED

    def gate_up(shape=s, group=64, x=FAKE, rt=FAKE, q1=FAKE, s1=FAKE, q3=FAKE, s3=FAKE, off=FAKE,
                h=FAKE, n=nb):
        return lib.moe_expert_gate_up_w4(ctypes.byref(shape), group, x, rt, q1, s1, q3, s3, off, h,
                                         FAKE, n, None)
    assert gate_up(group=16) == UNSUPPORTED
    assert gate_up(n=nb - 256) == WORKSPACE
    for name in ("x", "q1", "s1", "q3", "s3", "off", "h"):
        assert gate_up(**{name: None}) == INVALID, name
    assert gate_up(rt=at(2)) == INVALID
    odd = B.make_shape(16, 256, 4, 2, 2, 124, "bf16")
    assert gate_up(shape=odd, n=BIG) == UNSUPPORTED
    assert b"I=124" in lib.moe_last_error()

    def down(shape=s, group=64, h=FAKE, q2=FAKE, s2=FAKE, off=FAKE, y=FAKE, n=nb):
        return lib.moe_expert_down_w4(ctypes.byref(shape), group, h, q2, s2, off, y, FAKE, n, None)
    assert down(group=0) == UNSUPPORTED
    assert down(n=nb - 256) == WORKSPACE
    for name in ("h", "q2", "s2", "off", "y"):
        assert down(**{name: None}) == INVALID, name
    assert down(shape=odd, n=BIG) == UNSUPPORTED
    # an empty batch reads and writes no rows
    empty = B.make_shape(0, 256, 4, 2, 2, 128, "bf16")
    before = B.kernel_launches()
    assert gate_up(shape=empty, x=None, rt=None, h=None) == 0
    assert down(shape=empty, h=None, y=None) == 0
    assert B.kernel_launches() == before


def grads(*entries):
    return (B._Grad * max(1, len(entries)))(*[B._Grad(*e) for e in entries])


def test_gradient_refusals(lib):
    nb = lib.moe_grad_workspace_bytes(2)
    assert lib.moe_grad_workspace_bytes(-1) == 0
    assert lib.moe_grad_workspace_bytes(1000) > lib.moe_grad_workspace_bytes(1) > 256
    ok = grads((0x1000, 0x1000, 8, 0), (0x2002, 0x2002, 3, 1))

    def norm_(n=2, lst=ok, out=FAKE, ws=FAKE, size=nb):
        return lib.moe_grad_norm(n, lst, out, ws, size, None)
    assert norm_(n=-1) == INVALID
    assert norm_(lst=None) == INVALID
    assert norm_(out=None) == INVALID
    assert norm_(ws=None) == INVALID
    assert norm_(ws=at(64)) == INVALID
    assert norm_(size=nb - 256) == WORKSPACE
    assert norm_(n=1, lst=grads((0x1000, 0x1000, 8, 5))) == INVALID
    assert norm_(n=1, lst=grads((0x1000, 0x1000, -8, 0))) == INVALID
    assert norm_(n=1, lst=grads((None, None, 8, 0))) == INVALID
    assert norm_(n=1, lst=grads((0x1002, 0x1002, 8, 0))) == INVALID   # fp32 off its 4 bytes
    assert b"tensor 0" in lib.moe_last_error()

    def clip(n=2, lst=ok, limit=1.0, nrm=FAKE):
        return lib.moe_grad_clip(n, lst, limit, nrm, None)
    assert clip(limit=-1.0) == INVALID
    assert clip(limit=float("nan")) == INVALID
    assert clip(nrm=None) == INVALID
    assert clip(n=1, lst=grads((0x1000, None, 8, 0))) == INVALID
    assert clip(n=1, lst=grads((0x1000, 0x1001, 8, 1))) == INVALID
    before = B.kernel_launches()
    assert clip(n=0, lst=None) == 0
    assert clip(n=1, lst=grads((None, None, 0, 0))) == 0
    assert B.kernel_launches() == before


def _list(tensors, out=None):
    """The list's own checks, without the workspace that needs a device."""
    glist = B.GradientList.__new__(B.GradientList)
    glist.tensors = tensors
    glist.out = tensors if out is None else out
    glist._check_overlap()


def test_overlapping_gradients_are_refused():
    a = torch.zeros(64)
    b = torch.zeros(64)
    _list([a[:32], a[32:], b])
    _list([a], [b])
    _list([a, a[:0], b], None)
    _list([a[:16], a[16:32]], [b[:16], b[16:32]])
    for tensors, out in (([a, a], None),                     # the same tensor twice
                         ([a[:33], a[32:]], None),
                         ([a, b], [b, a]),                   # an output over another gradient
                         ([a[:32], a[32:]], [b[:32], b[16:48]]),
                         ([a[:32]], [a[8:40]]),              # shifted over itself
                         ([a, b[:4]], [b, torch.zeros(4)])):
        with pytest.raises(ValueError, match="overlaps"):
            _list(tensors, out)


def test_binding_checks_sizes_before_the_call():
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError, match="2-d"):
        B._rows(torch.zeros(4))
    with pytest.raises(ValueError, match="2-d"):
        B._rows(torch.zeros((4, 64), dtype=torch.float16))
    with pytest.raises(ValueError, match="dy has shape"):
        B._same(x, (("dy", torch.zeros((3, 64))),))
    with pytest.raises(ValueError, match="weight has 32"):
        B._size(torch.zeros(32), 64, "weight")
    with pytest.raises(ValueError, match="do not hold"):
        B._w4((torch.zeros(1024, dtype=torch.uint8), torch.zeros(16, dtype=torch.bfloat16)), 1, 17,
              128, 128, "w1")


@pytest.mark.parametrize("shape", [(2 ** 31, 8), (2 ** 32 + 5, 8), (1, 2 ** 32 + 8)])
def test_rows_past_32_bits_are_refused(shape):
    """As 32-bit numbers these would be negative or another, small size."""
    with pytest.raises(ValueError, match="more than"):
        B._rows(torch.empty(shape, dtype=torch.bfloat16, device="meta"))


@pytest.mark.parametrize("T,K", [(2 ** 31 - 1, 1), (2 ** 30 - 32, 2)])
def test_w4_rows_next_to_32_bits_are_refused(lib, T, K):
    """The end of the last chunk would not be a 32-bit number."""
    s = B.make_shape(T, 8, 2, 0, K, 8, "bf16")
    for code in (lib.moe_expert_gate_up_w4(ctypes.byref(s), 32, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                           FAKE, FAKE, FAKE, BIG, None),
                 lib.moe_expert_down_w4(ctypes.byref(s), 32, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                        BIG, None)):
        assert code == UNSUPPORTED and b"past int32" in lib.moe_last_error()


@pytest.mark.parametrize("rows,blocks,name", [(15, 16 * 8, "x_q"), (16, 16 * 8 - 1, "x_sf")])
def test_dispatch_of_short_8bit_rows_is_refused(lib, rows, blocks, name):
    """Codes or scales of fewer tokens than the shape has would be read past their end."""
    s = B.make_shape(16, 256, 4, 2, 2, 128, "bf16")
    q, sf = torch.zeros((rows, 256), dtype=torch.uint8), torch.zeros(blocks, dtype=torch.uint8)
    ints, out = torch.zeros(64, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match=f"{name} has"):
        B.permute_mxfp8_rows(s, q, sf, ints, ints, ints, ints, ints, out, out, out)
