"""The operators around the layer together, as a block of a model runs them: norm,
8-bit dispatch and MXFP8 experts; norm and 4-bit experts in a graph; a training
step from the norm to the clipped gradients."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_30_b200 import binding as B
from mixture_experts_layer_30_b200 import configs as C
from mixture_experts_layer_30_b200 import inputs as IN
from tests import parity as P

pytestmark = pytest.mark.gpu


def routed(T, d, N, Z, K, seed, I=128):
    g = torch.Generator().manual_seed(seed)
    shape = B.make_shape(T, d, N, Z, K, I, "bf16")
    x = torch.randn((T, d), generator=g).to(torch.bfloat16).cuda()
    idx = torch.rand((T, N + Z), generator=g).topk(K, 1).indices.to(torch.int32)
    counts = torch.bincount(idx.reshape(-1).long(), minlength=N + Z).to(torch.int32)
    return shape, x, idx.cuda().contiguous(), counts.cuda()


def dispatch(shape, call):
    R = max(1, shape.T * shape.K)
    off = torch.full((shape.N + 1,), -7, dtype=torch.int32, device="cuda")
    rt = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    sp = torch.full((max(1, shape.T), shape.K), -7, dtype=torch.int32, device="cuda")
    q = torch.full((R, shape.d), 7, dtype=torch.uint8, device="cuda")
    sf = torch.full((R, shape.d // 32), 7, dtype=torch.uint8, device="cuda")
    call(off, rt, sp, q, sf)
    torch.cuda.synchronize()
    return off, rt, sp, q, sf


@pytest.mark.parametrize("T,d,N,Z,K", [(1, 256, 4, 0, 1), (5, 512, 8, 4, 3), (256, 2048, 64, 32, 6),
                                       (257, 2048, 64, 32, 6), (300, 6144, 512, 256, 12),
                                       (40, 2304, 16, 100, 40), (2000, 256, 1000, 0, 2),
                                       (64, 8448, 481, 20, 5), (255, 256, 600, 60, 3)])
def test_dispatch_of_8bit_rows_equals_the_quantising_dispatch(T, d, N, Z, K):
    shape, x, idx, counts = routed(T, d, N, Z, K, T + d)
    ws = B.new_workspace(shape)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    q = torch.empty((T, d), dtype=torch.uint8, device="cuda")
    sf = torch.empty((T, d // 32), dtype=torch.uint8, device="cuda")
    B.rmsnorm(x, w, 1e-5, y, y_q=q, y_sf=sf)
    want = dispatch(shape, lambda *o: B.permute_mxfp8(shape, y, idx, counts, *o, ws))
    got = dispatch(shape, lambda *o: B.permute_mxfp8_rows(shape, q, sf, idx, counts, *o, ws))
    for a, b in zip(want, got):
        assert torch.equal(a, b)  # rows behind the last one too: neither call writes them
    assert B.device_status(ws) == 0


def test_dispatch_reports_bad_indices_and_counts():
    shape, x, idx, counts = routed(20, 256, 8, 4, 3, 1)
    ws = B.new_workspace(shape)
    q = torch.zeros((20, 256), dtype=torch.uint8, device="cuda")
    sf = torch.zeros((20, 8), dtype=torch.uint8, device="cuda")
    bad = idx.clone()
    bad[3, 1] = 12
    dispatch(shape, lambda *o: B.permute_mxfp8_rows(shape, q, sf, bad, counts, *o, ws))
    assert B.device_status(ws) & B.DEV_BAD_EXPERT_INDEX
    dispatch(shape, lambda *o: B.permute_mxfp8_rows(shape, q, sf, idx, counts + 1, *o, ws))
    assert B.device_status(ws) == B.DEV_COUNT_MISMATCH


def test_dispatch_of_an_empty_batch():
    shape = B.make_shape(0, 256, 4, 2, 2, 128, "bf16")
    ws = B.new_workspace(shape)
    counts = torch.zeros(6, dtype=torch.int32, device="cuda")
    off, _, _, q, _ = dispatch(shape, lambda *o: B.permute_mxfp8_rows(
        shape, torch.empty((0, 256), dtype=torch.uint8, device="cuda"),
        torch.empty((0, 8), dtype=torch.uint8, device="cuda"),
        torch.empty((0, 2), dtype=torch.int32, device="cuda"), counts, *o, ws))
    assert (off == 0).all() and (q == 7).all()


def block_inputs(cfg, seed=0):
    L = IN.make_layer_inputs(cfg, device="cuda")
    g = torch.Generator().manual_seed(seed)
    L["res"] = torch.randn((cfg.T, cfg.d), generator=g).to(L["x"].dtype).cuda()
    L["norm"] = (1 + 0.2 * torch.randn(cfg.d, generator=g)).to(L["x"].dtype).cuda()
    return L


@pytest.mark.parametrize("cfg", [C.DECODE_T64, C.LONGCAT_SLICE], ids=lambda c: c.name)
def test_mxfp8_block(cfg):
    """Norm with 8-bit output, then the layer on those rows: bit-equal to the layer that
    quantises the normed rows itself."""
    L = block_inputs(cfg)
    shape = B.shape_of(cfg)
    W = [B.quantize_weights_mxfp8(L[k]) for k in ("w1", "w3", "w2")]
    nb = B.PreNormBuffers(shape, mx=True)
    buf, fb = B.LayerBuffers(shape), B.Mxfp8Buffers(shape)
    y = B.prenorm(nb, L["x"], L["res"], L["norm"])
    out = B.forward_mxfp8(buf, fb, y, L["w_router"], *W, L["bias"], x_q=nb.x_q).clone()
    want = B.forward_mxfp8(buf, fb, y, L["w_router"], *W, L["bias"])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and B.device_status(buf.ws) == 0
    s64 = L["x"].double() + L["res"].double()
    assert ((nb.s.double() - s64).abs() <= s64.abs() * 2.0 ** -8 * (1 + 2.0 ** -12)).all()


def test_w4_block_in_a_graph():
    """A decode step with 4-bit experts, captured once and replayed on new tokens, is the
    eager step."""
    cfg = C.DECODE_T16
    L = block_inputs(cfg)
    shape = B.shape_of(cfg)
    W = [B.quantize_weights_w4(L[k], 128) for k in ("w1", "w3", "w2")]
    buf, nb = B.LayerBuffers(shape), B.PreNormBuffers(shape)
    x, res = L["x"].clone(), L["res"].clone()

    def step(b, n):
        y = B.prenorm(n, x, res, L["norm"])
        return B.forward_w4(b, 128, y, L["w_router"], *W, L["bias"])
    step(buf, nb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(buf, nb)
    other, nb2 = B.LayerBuffers(shape), B.PreNormBuffers(shape)
    for seed in (1, 2):
        x.copy_(torch.randn_like(x))
        graph.replay()
        want = step(other, nb2)
        torch.cuda.synchronize()
        assert torch.equal(buf.out, want) and torch.equal(nb.s, nb2.s)
    assert B.device_status(buf.ws) == 0 and B.device_status(other.ws) == 0


def test_training_step():
    """fp32: norm -> layer -> gradients -> norm's gradients -> clipping, against torch's
    gradients of the same formulas in 64 bits with the selection held fixed."""
    cfg = C.TINY_F32.with_T(48, "tiny")
    L = block_inputs(cfg, 3)
    shape = B.shape_of(cfg)
    nb = B.PreNormBuffers(shape, train=True)
    buf, bb = B.LayerBuffers(shape, with_probs=True), B.BackwardBuffers(shape)
    g = torch.Generator().manual_seed(4)
    dout = torch.randn((cfg.T, cfg.d), generator=g).cuda()
    dsum = torch.randn((cfg.T, cfg.d), generator=g).cuda()
    y = B.prenorm(nb, L["x"], L["res"], L["norm"])
    out = B.forward_train(buf, bb, y, L["w_router"], L["w1"], L["w3"], L["w2"], L["bias"])
    B.backward(buf, bb, y, L["w_router"], L["w1"], L["w3"], L["w2"], dout)
    B.prenorm_backward(nb, L["norm"], bb.dx, dsum=dsum)
    grads = [nb.dweight, bb.dw_router, bb.dw1, bb.dw3, bb.dw2]
    before = [t.clone() for t in grads]
    norm = torch.zeros(1, device="cuda")
    B.clip_gradients(B.GradientList(grads), 0.5, norm)
    torch.cuda.synchronize()
    assert B.device_status(buf.ws) == 0 and B.device_status(bb.bws) == 0

    v = {k: L[k].double().cpu().requires_grad_() for k in ("x", "norm", "w_router", "w1", "w3",
                                                           "w2")}
    s = v["x"] + L["res"].double().cpu()
    yy = s * (s.square().mean(1, keepdim=True) + 1e-5).rsqrt() * v["norm"]
    probs = torch.softmax(yy @ v["w_router"].T, 1)
    idx = buf.topk_idx.cpu().long()
    total = torch.zeros_like(yy)
    for t in range(cfg.T):
        row = 0
        for e in idx[t].tolist():
            if e >= cfg.N:
                row = row + probs[t, e] * yy[t]
            else:
                a = v["w1"][e] @ yy[t]
                row = row + probs[t, e] * (v["w2"][e] @ (a * torch.sigmoid(a) * (v["w3"][e] @ yy[t])))
        total[t] = row
    loss = (total * dout.double().cpu()).sum() + (s * dsum.double().cpu()).sum()
    loss.backward()
    P.assert_close(P.to_f64(out), total.detach().numpy(), "f32", "out")
    P.assert_close(P.to_f64(nb.dx), v["x"].grad.numpy(), "f32", "dx")
    want = [v[k].grad for k in ("norm", "w_router", "w1", "w3", "w2")]
    for a, b in zip(before, want):
        P.assert_close(P.to_f64(a), b.numpy(), "f32", "gradient")
    n64 = float(torch.sqrt(sum(w.square().sum() for w in want)))
    assert abs(float(norm) / n64 - 1) <= 1e-4
    coef = min(1.0, 0.5 / (float(norm) + 1e-6))
    assert coef < 1
    for a, b in zip(before, grads):
        np.testing.assert_allclose(b.double().cpu().numpy(), a.double().cpu().numpy() * coef,
                                   rtol=2.0 ** -21, atol=1e-38)


def test_dispatch_of_more_experts_than_the_call_before():
    """Large shared tables: a call with more experts follows one with fewer."""
    for N in (900, 1000, 1024):
        shape, x, idx, counts = routed(600, 256, N, 0, 2, N)
        ws = B.new_workspace(shape)
        want = dispatch(shape, lambda *o: B.permute_mxfp8(shape, x, idx, counts, *o, ws))
        off = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
        off[1:] = counts[:N].cumsum(0)
        assert torch.equal(want[0], off) and B.device_status(ws) == 0
