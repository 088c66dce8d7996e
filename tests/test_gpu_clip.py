"""Global gradient norm and clipping against 64 bits.

Tolerances.  Squares and the sums of at most 8 of them are fp32 (one rounding
each, so at most 9 * 2^-24 of the sum of squares, halved by the root), the rest
is fp64; the norm is rounded once: 6 * 2^-24 of its value.  The factor adds an
addition, a division and the product (3 * 2^-24), the result one rounding of its
type."""
import math

import pytest
import torch

from mixture_experts_layer_30_b200 import binding as B

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def tensors(spec, seed, std=0.02, offset=0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n + offset, generator=g) * std).to(dt).cuda()[offset:]
            for n, dt in spec]


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def check(ts, max_norm, out=None):
    before = [t.clone() for t in ts]
    glist = B.GradientList(ts, out=out)
    norm = torch.full((1,), 7.0, device="cuda")
    B.clip_gradients(glist, max_norm, norm)
    torch.cuda.synchronize()
    want = norm64(before)
    assert abs(float(norm) - want) <= 6 * U32 * want
    coef = min(1.0, max_norm / (want + 1e-6))
    for b, o in zip(before, ts if out is None else out):
        w = b.double() * coef
        tol = w.abs() * (torch.finfo(b.dtype).eps / 2 + 12 * U32) * (1 + 2.0 ** -7) + 1e-38
        assert ((o.double() - w).abs() <= tol).all()
        if coef == 1.0:
            assert torch.equal(o, b)
    if out is not None:
        assert all(torch.equal(b, t) for b, t in zip(before, ts))
    return float(norm)


SPECS = [
    [(1, F32)], [(1, BF16)], [(7, BF16), (3, F32), (8, BF16)],
    [(4096 * 3 + 5, BF16), (4096, F32), (100_001, F32), (65_537, BF16)],
    [(17 * i + 1, BF16 if i % 2 else F32) for i in range(300)],      # several tables
    [(0, F32), (5, BF16), (0, BF16)],
    [(3_000_001, BF16), (2_000_003, F32)],
]


@pytest.mark.parametrize("spec", SPECS, ids=lambda s: f"{len(s)}x{s[0][0]}")
@pytest.mark.parametrize("max_norm", [0.01, 1e6, 0.0])
def test_clip(spec, max_norm):
    check(tensors(spec, 1), max_norm)
    ts = tensors(spec, 2)
    check(ts, max_norm, out=[torch.full_like(t, 7) for t in ts])


@pytest.mark.parametrize("offset", [1, 2, 3, 5, 8])
def test_tensors_that_start_inside_their_16_bytes(offset):
    spec = [(5, BF16), (4097, F32), (40_000, BF16), (2, F32)]
    ts = tensors(spec, 3, offset=offset)
    check(ts, 0.05)
    ts = tensors(spec, 4, offset=offset)
    out = tensors(spec, 5)  # another place in the 16 bytes than the gradients
    check(ts, 0.05, out=out)
    # neighbours of a slice stay as they were
    base = torch.full((64,), 3.0, device="cuda")
    check([base[offset:offset + 20]], 0.1)
    assert (base[:offset] == 3).all() and (base[offset + 20:] == 3).all()


def test_no_tensors():
    norm = torch.full((1,), 7.0, device="cuda")
    B.clip_gradients(B.GradientList([]), 1.0, norm)
    assert float(norm) == 0
    B.clip_gradients(B.GradientList([torch.empty(0, device="cuda")]), 1.0, norm)
    assert float(norm) == 0


def test_nan_and_infinity():
    a = torch.ones(100, device="cuda")
    a[7] = float("inf")
    norm = torch.zeros(1, device="cuda")
    B.clip_gradients(B.GradientList([a]), 1.0, norm)
    assert math.isinf(float(norm))
    assert torch.isnan(a[7]) and (a[:7] == 0).all() and (a[8:] == 0).all()
    b = torch.ones(100, dtype=BF16, device="cuda")
    b[3] = float("nan")
    B.clip_gradients(B.GradientList([b]), 1.0, norm)
    assert math.isnan(float(norm)) and torch.isnan(b).all()


def test_norm_is_reproducible_and_leaves_the_gradients():
    ts = tensors([(1_000_003, BF16), (70_001, F32)], 6)
    keep = [t.clone() for t in ts]
    glist = B.GradientList(ts)
    seen = set()
    for _ in range(5):
        norm = torch.zeros(1, device="cuda")
        B.gradient_norm(glist, norm)
        seen.add(float(norm))
    assert len(seen) == 1
    assert all(torch.equal(a, b) for a, b in zip(ts, keep))


def test_large_offsets():
    """More than 2^32 bytes and 2^31 elements in one tensor."""
    n = 2 ** 31 + 5
    t = torch.zeros(n, dtype=BF16, device="cuda")
    t[-3:] = 3.0
    t[0] = 4.0
    norm = torch.zeros(1, device="cuda")
    B.clip_gradients(B.GradientList([t]), 1.0, norm)
    want = math.sqrt(43.0)
    assert abs(float(norm) - want) <= 6 * U32 * want
    tol = 3 / want * 2.0 ** -7
    assert abs(float(t[-1]) - 3 / want) <= tol and abs(float(t[0]) - 4 / want) <= 2 * tol
    assert float(t[1:-3].abs().max()) == 0


def test_graph_replay_sees_new_gradients():
    ts = tensors([(5000, BF16), (33, F32)], 8)
    norm = torch.zeros(1, device="cuda")
    st = torch.cuda.Stream()
    out = [torch.empty_like(t) for t in ts]
    with torch.cuda.stream(st):
        glist = B.GradientList(ts, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        B.clip_gradients(glist, 0.5, norm, stream=st)
    for scale in (1.0, 3.0):
        for t in ts:
            t.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        want = norm64(ts)
        assert abs(float(norm) - want) <= 6 * U32 * want
        coef = min(1.0, 0.5 / (want + 1e-6))
        for t, o in zip(ts, out):
            w = t.double() * coef
            assert ((o.double() - w).abs()
                    <= w.abs() * (torch.finfo(t.dtype).eps / 2 + 12 * U32) * 1.01).all()


def test_lists_that_cannot_be_taken_are_refused():
    a = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        B.GradientList([a[::2]])
    with pytest.raises(ValueError, match="dtype"):
        B.GradientList([a.half()])
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.GradientList([torch.zeros(4)])
    with pytest.raises(ValueError, match="overlaps"):
        B.GradientList([a, a])
    with pytest.raises(ValueError, match="elements"):
        B.GradientList([a], out=[a[:3]])
    with pytest.raises(ValueError, match="outputs"):
        B.GradientList([a], out=[])
