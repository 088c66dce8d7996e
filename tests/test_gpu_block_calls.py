"""Calls of the operators around the layer beyond the plain ones: streams, several calls at
once, replayed graphs on changed inputs, the host's two paths to a call, and the sizes at
which a call changes its kernel."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_30_b200 import binding as B
from tests.test_gpu_block import dispatch, routed
from tests.test_gpu_norm import make, run
from tests.test_gpu_w4 import close, decode, offsets_of

pytestmark = pytest.mark.gpu


def few_rows(N, d, I, group, seed):
    """One to three rows of every expert, N experts [d, I]."""
    g = torch.Generator().manual_seed(seed)
    counts = torch.randint(1, 4, (N,), generator=g).tolist()
    R = sum(counts)
    shape = B.make_shape(R, d, N, 0, 1, I, "bf16")
    w = torch.randn((N, d, I), generator=g) * 0.05
    return (shape, counts, offsets_of(counts).cuda(),
            B.quantize_weights_w4(w.to(torch.bfloat16).cuda(), group),
            torch.randn((R, I), generator=g).to(torch.bfloat16).cuda(), B.new_workspace(shape))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("d,I", [(4096, 136), (4104, 72), (4096, 384)])
def test_w4_many_pieces_of_few_rows(d, I, group):
    """Enough row blocks for two slices of the contraction: one, two and three of its
    128-column blocks, so that a slice has none, one or two steps."""
    shape, counts, off, w, h, ws = few_rows(48, d, I, group, d + I)
    y = torch.full((shape.T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    B.expert_down_w4(shape, group, h, w, off, y, ws)
    torch.cuda.synchronize()
    assert B.device_status(ws) == 0
    at = 0
    for e in range(0, 48):
        a, b = at, at + counts[e]
        at = b
        if e % 12:
            continue
        one = decode((w[0][e:e + 1], w[1][e:e + 1]), d, I, group)[0]
        v = h[a:b].double().cpu().numpy()
        close(y[a:b], v @ one.T, np.abs(v) @ np.abs(one).T, I, torch.bfloat16, f"expert {e}")


@pytest.mark.parametrize("T,N,K", [(8192, 16, 3), (8193, 16, 3), (8161, 5, 5), (1000, 512, 12),
                                   (4100, 1024, 2)])
def test_dispatch_layout_sizes(T, N, K):
    """Around the largest batch that one launch lays out, with tables of every size."""
    shape, x, idx, counts = routed(T, 256, N, 3 if N < 1000 else 0, K, T + N)
    ws = B.new_workspace(shape)
    y, q, sf = (torch.empty((T, n), dtype=t, device="cuda")
                for n, t in ((256, torch.bfloat16), (256, torch.uint8), (8, torch.uint8)))
    B.rmsnorm(x, torch.ones(256, dtype=torch.bfloat16, device="cuda"), 1e-5, y, y_q=q, y_sf=sf)
    want = dispatch(shape, lambda *o: B.permute_mxfp8(shape, y, idx, counts, *o, ws))
    got = dispatch(shape, lambda *o: B.permute_mxfp8_rows(shape, q, sf, idx, counts, *o, ws))
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert B.device_status(ws) == 0


def test_calls_on_another_stream():
    """stream= and torch's current stream are the same thing; the default stream is not
    touched."""
    x, r, w = make(64, 1024, torch.bfloat16, 1)
    want = run(x, r, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for explicit in (False, True):
        y, s = torch.empty_like(x), torch.empty_like(x)
        inv = torch.empty(64, device="cuda")
        torch.cuda.synchronize()
        if explicit:
            B.rmsnorm(x, w, 1e-5, y, residual=r, sum_out=s, inv_rms=inv, stream=side)
        else:
            with torch.cuda.stream(side):
                B.rmsnorm(x, w, 1e-5, y, residual=r, sum_out=s, inv_rms=inv)
        side.synchronize()
        outs.append((y, s, inv))
    for y, s, inv in outs:
        assert torch.equal(y, want[0]) and torch.equal(s, want[1]) and torch.equal(inv, want[2])


def test_products_on_two_streams_at_once():
    """Two calls in flight, each with its own workspace, give what they give alone."""
    a, b = few_rows(24, 1024, 512, 64, 1), few_rows(24, 1024, 512, 64, 2)

    def call(s, stream=None):
        y = torch.empty((s[0].T, 1024), dtype=torch.bfloat16, device="cuda")
        B.expert_down_w4(s[0], 64, s[4], s[3], s[2], y, s[5], stream=stream)
        return y
    alone = call(a), call(b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        both = [call(s, st) for s, st in zip((a, b), streams)]
        torch.cuda.synchronize()
        assert torch.equal(both[0], alone[0]) and torch.equal(both[1], alone[1])


def test_replayed_training_calls():
    """Norm, its backward pass and clipping captured once, replayed on other values."""
    T, d = 40, 512
    x, r, w = make(T, d, torch.bfloat16, 3)
    dy = torch.randn((T, d), device="cuda").to(torch.bfloat16)
    ws, norm = B.new_rmsnorm_workspace(T, d), torch.empty(1, device="cuda")
    buf = {k: torch.empty((T, d), dtype=torch.bfloat16, device="cuda") for k in ("y", "s", "dx")}
    inv, dw = torch.empty(T, device="cuda"), torch.empty(d, dtype=torch.bfloat16, device="cuda")
    clipped = torch.empty_like(dw)
    grads = B.GradientList([dw], out=[clipped])

    def step():
        B.rmsnorm(x, w, 1e-5, buf["y"], residual=r, sum_out=buf["s"], inv_rms=inv)
        B.rmsnorm_backward(buf["s"], w, inv, dy, buf["dx"], dw, ws)
        B.clip_gradients(grads, 0.25, norm)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn((T, d), generator=g))
        dy.copy_(torch.randn((T, d), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (buf["y"], buf["s"], buf["dx"], dw, clipped, norm)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (buf["y"], buf["s"], buf["dx"], dw, clipped, norm)):
            assert torch.equal(a, b)


def test_both_paths_of_a_call_agree(monkeypatch):
    """The native path of a call and the checked Python path behind it."""
    class Refuses:
        def __getattr__(self, name):
            return lambda *args: -1

    x, r, w = make(33, 256, torch.bfloat16, 5)
    y, s, inv, q, sf = run(x, r, w, mx=True)
    dy = torch.randn_like(x)
    ws = B.new_rmsnorm_workspace(33, 256)
    p = few_rows(6, 256, 128, 32, 3)
    shape, rx, idx, counts = routed(20, 256, 8, 4, 3, 1)
    dws = B.new_workspace(shape)
    grads = [torch.randn(1000, device="cuda"), torch.randn(77, device="cuda").to(torch.bfloat16)]
    outs = [torch.empty_like(g) for g in grads]
    plan, norm = B.GradientList(grads, out=outs), torch.empty(1, device="cuda")
    x2 = torch.randn((p[0].T, 256), device="cuda").to(torch.bfloat16)
    w1 = B.quantize_weights_w4(torch.randn((6, 128, 256), device="cuda"), 32)

    def everything():
        n = run(x, r, w, mx=True)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        B.rmsnorm_backward(s, w, inv, dy, dx, dw, ws)
        d = dispatch(shape, lambda *o: B.permute_mxfp8_rows(shape, q[:20], sf[:20], idx, counts,
                                                            *o, dws))
        h = torch.empty((p[0].T, 128), dtype=torch.bfloat16, device="cuda")
        yy = torch.empty((p[0].T, 256), dtype=torch.bfloat16, device="cuda")
        B.expert_gate_up_w4(p[0], 32, x2, None, w1, w1, p[2], h, p[5])
        B.expert_down_w4(p[0], 32, p[4], p[3], p[2], yy, p[5])
        B.clip_gradients(plan, 1.0, norm)
        n2 = B.gradient_norm(plan, torch.empty(1, device="cuda"))
        torch.cuda.synchronize()
        return [*n, dx, dw, *d, h, yy, norm.clone(), n2, *(o.clone() for o in outs)]
    want = everything()
    monkeypatch.setattr(B, "_native", lambda: Refuses())
    got = everything()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_refusals_name_the_argument():
    x, r, w = make(4, 64, torch.bfloat16, 1)
    y, s = torch.empty_like(x), torch.empty_like(x)
    with pytest.raises(ValueError, match="y has dtype"):
        B.rmsnorm(x, w, 1e-5, y.float())
    with pytest.raises(ValueError, match="residual has shape"):
        B.rmsnorm(x, w, 1e-5, y, residual=r[:2], sum_out=s)
    with pytest.raises(ValueError, match="weight must be contiguous"):
        B.rmsnorm(x, torch.stack([w, w], 1)[:, 0], 1e-5, y)
    with pytest.raises(ValueError, match="y must be a CUDA tensor"):
        B.rmsnorm(x, w, 1e-5, y.cpu())
    with pytest.raises(B.MoEError, match="sum_out"):
        B.rmsnorm(x, w, 1e-5, y, sum_out=s)
    with pytest.raises(B.MoEError, match="eps"):
        B.rmsnorm(x, w, float("nan"), y)
    ws = B.new_rmsnorm_workspace(4, 64)
    inv, dw = torch.ones(4, device="cuda"), torch.empty_like(w)
    with pytest.raises(B.MoEError, match="workspace"):
        B.rmsnorm_backward(x, w, inv, y, s, dw, ws[:256])
    with pytest.raises(ValueError, match="inv_rms has 3 elements"):
        B.rmsnorm_backward(x, w, inv[:3], y, s, dw, ws)
    plan = B.GradientList([torch.ones(3, device="cuda")])
    with pytest.raises(B.MoEError, match="max_norm"):
        B.clip_gradients(plan, -1.0, torch.empty(1, device="cuda"))
    with pytest.raises(ValueError, match="norm has 2 elements"):
        B.clip_gradients(plan, 1.0, torch.empty(2, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [8, 40, 256, 520, 1032, 2048, 3080, 6152, 12296, 16384, 20480])
def test_norm_backward_widths(d, dtype):
    """One width for each way a row is laid over threads, against 64 bits (tolerances as for the
    norm's other tests: half a step of the type, and the sums' chains)."""
    for T in (1, 3, 11):
        s, dsum, w = make(T, d, dtype, T + d)
        dy = torch.randn((T, d), generator=torch.Generator().manual_seed(d)).to(dtype).cuda()
        inv = (s.double().square().mean(1) + 1e-5).rsqrt().float()
        dx, dw = torch.empty_like(s), torch.empty_like(w)
        B.rmsnorm_backward(s, w, inv, dy, dx, dw, B.new_rmsnorm_workspace(T, d), dsum=dsum)
        torch.cuda.synchronize()
        i64 = inv.double()[:, None]
        xhat, wdy = s.double() * i64, w.double() * dy.double()
        dx64 = i64 * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True)) + dsum.double()
        half, u32 = torch.finfo(dtype).eps / 2, 2.0 ** -24
        mag = i64 * (6 * wdy.abs() + xhat.abs() * (d / 32 + 20)
                     * (wdy * xhat).abs().mean(1, keepdim=True)) + 2 * dsum.double().abs()
        assert ((dx.double() - dx64).abs() <= (dx64.abs() * half + mag * u32) * (1 + 2.0 ** -7)).all()
        each = dy.double() * xhat
        tol = (each.sum(0).abs() * half + each.abs().sum(0) * (T + 24) * u32) * (1 + 2.0 ** -7)
        assert ((dw.double() - each.sum(0)).abs() <= tol).all()


def test_infinite_max_norm_leaves_the_gradients():
    """The factor is 1 then, and inf / inf = NaN for an infinite norm."""
    g = torch.linspace(-3, 3, 1001, device="cuda")
    out, norm = torch.empty_like(g), torch.empty(1, device="cuda")
    B.clip_gradients(B.GradientList([g], out=[out]), float("inf"), norm)
    assert torch.equal(out, g) and torch.isfinite(norm).all()
    g[500] = float("inf")
    B.clip_gradients(B.GradientList([g], out=[out]), float("inf"), norm)
    assert torch.isinf(norm).all() and torch.isnan(out).all()
