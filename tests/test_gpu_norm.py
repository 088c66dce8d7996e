"""Residual RMS norm and its backward pass against their formulas in 64 bits.

Tolerances.  A sum of n fp32 terms is off by at most (additions in a chain) *
2^-24 times the sum of the terms' magnitudes; the longest chain of a row's sum is
at most d/32 additions in a thread and 12 across threads (CHAIN below), and of a
column's sum at most T rows and 20 across CTAs.  A result of type t is rounded
once, by at most eps(t)/2 of its value."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_30_b200 import binding as B
from oracle import moe_oracle as orc
from tests import parity as P

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def half(dt):
    return torch.finfo(dt).eps / 2


def chain(d):
    return d / 32 + 12


def make(T, d, dt, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, d), generator=g) * torch.exp(torch.randn((T, 1), generator=g))).to(dt)
    r = torch.randn((T, d), generator=g).to(dt) if residual else None
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(dt)
    return x.cuda(), None if r is None else r.cuda(), w.cuda()


def run(x, r, w, eps=1e-5, mx=False, want_y=True, in_place=False):
    T, d = x.shape
    y = torch.full_like(x, 7) if want_y else None
    s = None if r is None else (r if in_place else torch.full_like(x, 7))
    inv = torch.full((T,), 7.0, device="cuda")
    q = torch.full((T, d), 7, dtype=torch.uint8, device="cuda") if mx else None
    sf = torch.full((T, d // 32), 7, dtype=torch.uint8, device="cuda") if mx else None
    B.rmsnorm(x, w, eps, y, residual=r, sum_out=s, inv_rms=inv, y_q=q, y_sf=sf)
    torch.cuda.synchronize()
    return y, s, inv, q, sf


def check_forward(x, r, w, y, s, inv, eps=1e-5):
    d = x.shape[1]
    if r is not None:
        want = x.double() + r.double()
        # an fp32 addition and the rounding to the type
        assert ((s.double() - want).abs() <= want.abs() * (half(x.dtype) * (1 + 2.0 ** -12)
                                                           + U32)).all()
        base = s.double()
    else:
        base = x.double()
    inv64 = (base.square().mean(1) + eps).rsqrt()
    assert ((inv.double() - inv64).abs() <= inv64 * (chain(d) / 2 + 4) * U32).all()
    y64 = base * inv64[:, None] * w.double()
    tol = y64.abs() * (half(x.dtype) + (chain(d) / 2 + 8) * U32) * (1 + 2.0 ** -7) + 1e-38
    assert ((y.double() - y64).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 64), (16, 2048), (5, 1000), (129, 256), (7, 6144),
                                 (2, 20480), (3, 70000), (2, 131072), (300, 32)])
def test_forward(T, d, dtype):
    dt = DT[dtype]
    x, r, w = make(T, d, dt, T + d)
    y, s, inv, _, _ = run(x, r, w)
    check_forward(x, r, w, y, s, inv)
    y, _, inv, _, _ = run(x, None, w)
    check_forward(x, None, w, y, None, inv)


@pytest.mark.parametrize("T,d", [(1, 32), (16, 2048), (33, 96), (9, 6144), (2, 20480), (2, 98304)])
@pytest.mark.parametrize("residual", [True, False])
def test_mxfp8_output_is_the_quantised_y(T, d, residual):
    x, r, w = make(T, d, torch.bfloat16, 5 * T + d, residual)
    x[0, :32] = 0
    if residual:
        r[0, :32] = 0  # a block of zeros
    y, s, inv, q, sf = run(x, r, w, mx=True)
    check_forward(x, r, w, y, s, inv)
    codes, scales, _ = orc.mxfp8_quantize(P.to_f64(y))
    np.testing.assert_array_equal(q.cpu().numpy(), codes)
    np.testing.assert_array_equal(sf.cpu().numpy().astype(np.int64), scales + 127)
    # without y in 16 bits the codes are the same
    _, _, _, q2, sf2 = run(x, r, w, mx=True, want_y=False)
    assert torch.equal(q, q2) and torch.equal(sf, sf2)


@pytest.mark.parametrize("d", [256, 20480, 131072])
def test_in_place(d):
    x, r, w = make(4, d, torch.bfloat16, 3)
    y, s, inv, _, _ = run(x, r, w)
    y2, s2, inv2, _, _ = run(x, r.clone(), w, in_place=True)  # the sum over the residual
    assert torch.equal(y, y2) and torch.equal(s, s2) and torch.equal(inv, inv2)
    x2 = x.clone()
    B.rmsnorm(x2, w, 1e-5, y2, residual=r, sum_out=x2)        # the sum over x
    assert torch.equal(y, y2) and torch.equal(s, x2)
    want, _, _, _, _ = run(x, None, w)
    x2 = x.clone()
    B.rmsnorm(x2, w, 1e-5, x2)                                # y over x
    assert torch.equal(want, x2)


def test_special_rows():
    x, _, w = make(6, 64, torch.float32, 1, residual=False)
    x[0] = 0                       # 1 / sqrt(eps)
    x[1, 3] = float("nan")
    x[2, 3] = float("inf")         # inv = 0: finite entries 0, the infinite one NaN
    x[3] = 1e-30
    x[4] *= 1e15
    y, _, inv, _, _ = run(x, None, w)
    assert (y[0] == 0).all() and abs(float(inv[0]) * 1e-5 ** 0.5 - 1) < 1e-6
    assert torch.isnan(y[1]).all()
    assert float(inv[2]) == 0 and torch.isnan(y[2, 3])
    assert (y[2, :3] == 0).all()
    rest = torch.tensor([3, 4, 5], device="cuda")
    check_forward(x[rest], None, w, y[rest], None, inv[rest])
    # without eps a zero row is 0 * inf
    y, _, inv, _, _ = run(x[:1], None, w, eps=0.0)
    assert torch.isinf(inv).all() and torch.isnan(y).all()


def bwd(s, w, inv, dy, dsum, dx=None):
    T, d = s.shape
    dx = torch.full_like(s, 7) if dx is None else dx
    dw = torch.full_like(w, 7)
    ws = B.new_rmsnorm_workspace(T, d)
    ws.fill_(0xff)  # nothing may be expected of the workspace
    B.rmsnorm_backward(s, w, inv, dy, dx, dw, ws, dsum=dsum)
    torch.cuda.synchronize()
    return dx, dw


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_dsum", [True, False])
@pytest.mark.parametrize("T,d", [(1, 8), (2, 64), (16, 2048), (333, 1000), (700, 256), (65, 6144),
                                 (3, 20480), (2, 70000), (1500, 32)])
def test_backward(T, d, with_dsum, dtype):
    dt = DT[dtype]
    s, dsum, w = make(T, d, dt, T + 3 * d, with_dsum)
    g = torch.Generator().manual_seed(T * d)
    dy = torch.randn((T, d), generator=g).to(dt).cuda()
    inv = (s.double().square().mean(1) + 1e-5).rsqrt().float()
    dx, dw = bwd(s, w, inv, dy, dsum)
    i64, s64, dy64, w64 = inv.double()[:, None], s.double(), dy.double(), w.double()
    xhat = s64 * i64
    wdy = w64 * dy64
    c = (wdy * xhat).mean(1, keepdim=True)
    dx64 = i64 * (wdy - xhat * c)
    # fp32 error: the products, and the row mean's chain
    mag = i64 * (6 * wdy.abs() + xhat.abs() * (chain(d) + 8)
                 * (wdy * xhat).abs().mean(1, keepdim=True))
    if dsum is not None:
        dx64 = dx64 + dsum.double()
        mag = mag + 2 * dsum.double().abs()
    tol = (dx64.abs() * half(dt) + mag * U32) * (1 + 2.0 ** -7)
    assert ((dx.double() - dx64).abs() <= tol).all()
    dw64 = (dy64 * xhat).sum(0)
    tol = (dw64.abs() * half(dt) + (dy64 * xhat).abs().sum(0) * (T + 24) * U32) * (1 + 2.0 ** -7)
    assert ((dw.double() - dw64).abs() <= tol).all()
    # bit-reproducible; the gradient may be written over dy or dsum
    dx2, dw2 = bwd(s, w, inv, dy, dsum)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    if dsum is not None:
        over = dsum.clone()
        bwd(s, w, inv, dy, over, dx=over)
        assert torch.equal(dx, over)
    over = dy.clone()
    bwd(s, w, inv, over, dsum, dx=over)
    assert torch.equal(dx, over)


def test_backward_against_differences():
    """The gradient of sum(y * dy) + sum(s * dsum) against central differences of the
    64-bit formula: their error is O(h^2) of third derivatives of order one, below
    1e-5 at h = 1e-3; the fp32 gradients' error (above) is below that too."""
    T, d, eps, h = 3, 16, 1e-5, 1e-3
    s, dsum, w = make(T, d, torch.float32, 11)
    g = torch.Generator().manual_seed(2)
    dy = torch.randn((T, d), generator=g).cuda()
    _, _, inv, _, _ = run(s, None, w, eps)
    dx, dw = bwd(s, w, inv, dy, dsum)

    def loss(a, b):
        y = a * (a.square().mean(1, keepdim=True) + eps).rsqrt() * b
        return float((y * dy.double()).sum() + (a * dsum.double()).sum())
    s64, w64 = s.double(), w.double()
    scale = s64.abs().max().item()
    for t in range(T):
        for j in range(d):
            e = torch.zeros_like(s64)
            e[t, j] = h * max(1.0, scale)
            num = (loss(s64 + e, w64) - loss(s64 - e, w64)) / (2 * float(e[t, j]))
            assert abs(num - float(dx[t, j])) <= 2e-4 * (1 + abs(num)), (t, j)
    for j in range(d):
        e = torch.zeros_like(w64)
        e[j] = h
        num = (loss(s64, w64 + e) - loss(s64, w64 - e)) / (2 * h)
        assert abs(num - float(dw[j])) <= 1e-5 * (1 + abs(num)), j


def test_no_rows():
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    inv = torch.empty(0, device="cuda")
    B.rmsnorm(x, w, 1e-5, torch.empty_like(x), inv_rms=inv)
    _, dw = bwd(x, w, inv, x, None)
    assert (dw == 0).all()


def test_other_stream_and_graph():
    x, r, w = make(64, 512, torch.bfloat16, 9)
    want = run(x, r, w, mx=True)
    st = torch.cuda.Stream()
    y, s, inv = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device="cuda")
    q = torch.empty((64, 512), dtype=torch.uint8, device="cuda")
    sf = torch.empty((64, 16), dtype=torch.uint8, device="cuda")
    dy = torch.randn_like(x)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = B.new_rmsnorm_workspace(64, 512)
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        B.rmsnorm(x, w, 1e-5, y, residual=r, sum_out=s, inv_rms=inv, y_q=q, y_sf=sf, stream=st)
        B.rmsnorm_backward(s, w, inv, dy, dx, dw, ws, stream=st)
    for _ in range(2):
        for t in (y, s, inv, q, sf, dx, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((y, s, inv, q, sf), want):
            assert torch.equal(a, b)
        dx2, dw2 = bwd(s, w, inv, dy, None)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
