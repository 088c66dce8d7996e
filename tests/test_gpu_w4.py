"""4-bit expert path: quantiser bit for bit, expert products against 64 bits on the
weights that the codes stand for.

Tolerances.  Codes are small integers and activations have 8 (bf16) or 24 bits, so
a product rounds at most once; a sum of K products in any of the kernels' orders
is off by at most (K / 2 + 32) * 2^-23 of the sum of magnitudes (sequential
rounding is the largest, the tensor core's truncation within 16 products and the
joining of pieces are below it), and the scales add two roundings.  The result is
rounded once, by at most eps/2.  Over a whole output the roundings average, so
its 2-norm error is also held to eps/2 of the 2-norm."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_30_b200 import binding as B
from mixture_experts_layer_30_b200 import configs as C
from mixture_experts_layer_30_b200 import inputs as IN
from oracle import moe_oracle as orc
from tests import parity as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def decode(pair, rows, cols, group):
    """Weights [n, rows, cols] in float64, each value looked up where the format
    keeps it."""
    codes, scales = (t.cpu() for t in pair)
    n, rb, sp, _ = codes.shape
    codes = codes.reshape(n, rb * sp * 1024).numpy()
    scales = scales.double().reshape(n, rb * sp * 16 * (128 // group)).numpy()
    r, c = np.arange(rows)[:, None], np.arange(cols)[None, :]
    block = (r // 16) * sp + c // 128
    cc = c % 128
    nib = (cc % 8) // 2 + 4 * (cc % 2)
    byte = block * 1024 + (r % 16) * 64 + 16 * ((cc % 32) // 8) + 4 * (cc // 32) + nib // 2
    v = (codes[:, byte] >> (4 * (nib % 2))) & 15
    s = scales[:, (block * 16 + r % 16) * (128 // group) + cc // group]
    return (v.astype(np.float64) - 8.0) * s


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,cols", [(2, 48, 256), (1, 1, 1), (3, 17, 131), (1, 100, 1000)])
def test_quantiser_is_bit_exact(n, rows, cols, dtype, group):
    g = torch.Generator().manual_seed(rows + cols)
    w = torch.randn((n, rows, cols), generator=g) * torch.exp(2 * torch.randn((n, rows, 1),
                                                                              generator=g))
    w[0, 0, :32] = 0.0
    w = w.to(DT[dtype])
    q, s = B.quantize_weights_w4(w.cuda(), group)
    torch.cuda.synchronize()
    # the definition in fp32: scale = bf16(amax / 7), code = rint(w / scale)
    pad = -(-cols // 128) * 128
    wf = torch.zeros((n, rows, pad))
    wf[:, :, :cols] = w.float()
    blocks = wf.view(n, rows, pad // group, group)
    scale = (blocks.abs().amax(3) / 7.0).to(torch.bfloat16).float()
    code = torch.round(blocks / scale.unsqueeze(3)).clamp(-8, 7)
    code = torch.where(scale.unsqueeze(3) > 0, code, torch.zeros_like(code))
    want = (code.double() * scale.double().unsqueeze(3)).view(n, rows, pad)[:, :, :cols].numpy()
    np.testing.assert_array_equal(decode((q, s), rows, cols, group), want)
    # half a step of the group's scale (its bf16 rounding moves the largest by 7 * 2^-9 of a step)
    err = np.abs(want - w.double().numpy())
    lim = scale.double().repeat_interleave(group, 2)[:, :, :cols].numpy() * (0.5 + 7 * 2.0 ** -8)
    assert (err <= lim * (1 + 2.0 ** -20)).all()
    # padding holds zeros
    full = decode((q, s), -(-rows // 16) * 16, pad, group)
    assert (full[:, rows:] == 0).all() and (full[:, :, cols:] == 0).all()


def offsets_of(counts):
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.tensor(counts, dtype=torch.int32).cumsum(0)
    return off


def close(got, want, mag, K, dt, what):
    """mag: what a relative error of the sums moves the result by."""
    got, want, mag = got.double().cpu().numpy(), np.asarray(want), np.asarray(mag)
    u = torch.finfo(dt).eps / 2
    tol = (np.abs(want) * u + mag * (K / 2 + 32) * 2.0 ** -23) * (1 + 2.0 ** -6) + 1e-37
    bad = np.abs(got - want) > tol
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4])
    if want.size and dt == torch.bfloat16:
        assert P.rel_l2(got, want) <= u * (1 + 2.0 ** -4), (what, P.rel_l2(got, want))


def sigmoid(a):
    return 1.0 / (1.0 + np.exp(-a))


def products(counts, T, d, I, group, dtype, seed, Z=0, K=1, gather=True, extreme=False):
    """Runs both halves on made-up routed rows; returns what the checks need."""
    dt = DT[dtype]
    N, R = len(counts), sum(counts)
    assert R <= T * K
    g = torch.Generator().manual_seed(seed)
    shape = B.make_shape(T, d, N, Z, K, I, dtype)
    ws = B.new_workspace(shape)
    off = offsets_of(counts).cuda()
    W = {}
    for name, rows, cols in (("w1", I, d), ("w3", I, d), ("w2", d, I)):
        w = torch.randn((N, rows, cols), generator=g) * 0.05
        if extreme:
            w = w * torch.exp(3 * torch.randn((N, rows, 1), generator=g))
        W[name] = B.quantize_weights_w4(w.to(dt).cuda(), group)
    src = torch.randn((T if gather else T * K, d), generator=g).to(dt).cuda()
    rt = torch.randint(0, T, (T * K,), generator=g, dtype=torch.int32).cuda()
    h = torch.full((T * K, I), 7.0, dtype=dt, device="cuda")
    y = torch.full((T * K, d), 7.0, dtype=dt, device="cuda")
    B.expert_gate_up_w4(shape, group, src, rt if gather else None, W["w1"], W["w3"], off, h, ws)
    hin = torch.randn((T * K, I), generator=g).to(dt).cuda()
    B.expert_down_w4(shape, group, hin, W["w2"], off, y, ws)
    torch.cuda.synchronize()
    assert B.device_status(ws) == 0
    # rows behind the last expert's stay as they were
    assert (h[R:] == 7).all() and (y[R:] == 7).all()
    x64 = src.double().cpu().numpy()
    rows = rt[:R].cpu().numpy() if gather else np.arange(R)
    at = 0
    for e, m in enumerate(counts):
        if m == 0:
            continue
        a, b = at, at + m
        at = b
        one = {k: decode((v[0][e:e + 1], v[1][e:e + 1]), I if k != "w2" else d,
                         d if k != "w2" else I, group)[0] for k, v in W.items()}
        x = x64[rows[a:b]]
        p, u = x @ one["w1"].T, x @ one["w3"].T
        mp, mu = np.abs(x) @ np.abs(one["w1"]).T, np.abs(x) @ np.abs(one["w3"]).T
        act = p * sigmoid(p)
        # |SiLU'| <= 1.1; expf and the division stay within 8 units of the result
        mag = 1.1 * np.abs(u) * mp + np.abs(act) * mu + np.abs(act * u)
        close(h[a:b], act * u, mag, d, dt, f"gate/up of expert {e}")
        v = hin[a:b].double().cpu().numpy()
        close(y[a:b], v @ one["w2"].T, np.abs(v) @ np.abs(one["w2"]).T, I, dt,
              f"down of expert {e}")
    return shape, W, src, rt, off, h, y, ws, hin


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts,d,I", [
    ([1], 128, 128),
    ([1, 0, 2, 8, 9], 256, 128),
    ([0, 0, 0], 256, 128),                  # every expert empty
    ([16, 17, 31, 32, 33], 384, 256),
    ([3, 1], 1000, 616),                    # edges inside a block
    ([5, 24, 64, 65], 72, 8),               # smaller than one block
    ([2, 0, 7], 2048, 1024),
    ([150, 1, 40], 264, 136),               # many rows of one expert
])
def test_products(counts, d, I, group, dtype):
    T = max(4, sum(counts))
    products(counts, T, d, I, group, dtype, seed=sum(counts) + d + group)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_in_place_and_wide_scales(dtype):
    products([4, 11, 0, 3], 10, 512, 256, 32, dtype, seed=5, K=2, gather=False, extreme=True)


def test_longcat_geometry():
    products([1, 0, 13, 20], 34, 6144, 2048, 128, "bf16", seed=6)


def test_one_value_per_row():
    """fp32 rows of one 16-byte vector."""
    products([3, 2], 5, 4, 4, 64, "f32", seed=7)
    products([3, 2], 5, 8, 8, 64, "bf16", seed=8)


def test_many_experts_with_few_rows():
    counts = [0] * 700
    for e in (0, 3, 255, 256, 511, 699):
        counts[e] = e % 3 + 1
    products(counts, sum(counts), 128, 128, 64, "bf16", seed=9)


def test_bad_row_token_is_reported_and_reads_row_0():
    counts, d, I, group = [2, 3], 256, 128, 64
    shape, W, src, rt, off, h, _, ws, _ = products(counts, 5, d, I, group, "bf16", seed=10)
    bad, zero = rt.clone(), rt.clone()
    bad[1], bad[4] = 5, -1
    zero[1], zero[4] = 0, 0
    want = torch.empty_like(h)
    B.expert_gate_up_w4(shape, group, src, zero, W["w1"], W["w3"], off, want, ws)
    got = torch.empty_like(h)
    B.expert_gate_up_w4(shape, group, src, bad, W["w1"], W["w3"], off, got, ws)
    torch.cuda.synchronize()
    assert torch.equal(got[:5], want[:5])
    assert B.device_status(ws) == B.DEV_BAD_OFFSETS


def test_bad_offsets_count_as_empty():
    shape, W, src, rt, off, h, _, ws, hin = products([2, 3], 5, 256, 128, 64, "bf16", seed=12)
    bad = torch.tensor([0, 9, 5], dtype=torch.int32).cuda()   # 9 rows of 5; then backwards
    out = torch.full_like(h, 7)
    B.expert_gate_up_w4(shape, 64, src, rt, W["w1"], W["w3"], bad, out, ws)
    y = torch.full((5, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    B.expert_down_w4(shape, 64, hin, W["w2"], bad, y, ws)
    torch.cuda.synchronize()
    assert (out == 7).all() and (y == 7).all()
    assert B.device_status(ws) == B.DEV_BAD_OFFSETS


def test_nan_stays_in_its_row():
    shape, W, src, rt, off, h, y, ws, hin = products([9, 4], 13, 384, 256, 32, "bf16", seed=13)
    hin2 = hin.clone()
    hin2[2, 5] = float("nan")
    y2 = torch.empty_like(y)
    B.expert_down_w4(shape, 32, hin2, W["w2"], off, y2, ws)
    torch.cuda.synchronize()
    assert torch.isnan(y2[2]).all()
    keep = [r for r in range(13) if r != 2]
    assert torch.equal(y2[keep], y[:13][keep])


def test_results_do_not_depend_on_the_call():
    shape, W, src, rt, off, h, y, ws, hin = products([9, 4, 20], 33, 1024, 512, 64, "bf16",
                                                     seed=14)
    for _ in range(3):
        h2, y2 = torch.full_like(h, 7), torch.full_like(y, 7)
        B.expert_gate_up_w4(shape, 64, src, rt, W["w1"], W["w3"], off, h2, ws)
        B.expert_down_w4(shape, 64, hin, W["w2"], off, y2, ws)
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(y, y2)


def test_wrong_weight_sizes_are_refused():
    shape, W, src, rt, off, h, y, ws, hin = products([2, 3], 5, 256, 128, 64, "bf16", seed=15)
    with pytest.raises(ValueError, match="do not hold"):
        B.expert_down_w4(shape, 128, hin, W["w2"], off, y, ws)
    with pytest.raises(ValueError, match="do not hold"):
        B.expert_gate_up_w4(shape, 64, src, rt, (W["w1"][0][:1], W["w1"][1]), W["w3"], off, h, ws)
    with pytest.raises(B.MoEError):
        B.quantize_weights_w4(torch.zeros((16, 128), device="cuda"), group=16)


@pytest.mark.parametrize("cfg", [C.TINY_F32, C.DECODE_T16, C.DECODE_T256, C.LONGCAT_SLICE],
                         ids=lambda c: c.name)
def test_w4_layer(cfg):
    """The whole layer with 4-bit experts: selection and dispatch against the oracle,
    the output against the oracle's FFN on the decoded weights."""
    T = min(cfg.T, 64) if cfg.d == 6144 else cfg.T
    L = IN.make_layer_inputs(cfg.with_T(T, cfg.name), device="cuda")
    shape = B.shape_of(cfg, T=T)
    group = 64
    W = {k: B.quantize_weights_w4(L[k], group) for k in ("w1", "w3", "w2")}
    buf = B.LayerBuffers(shape, with_probs=True)
    B.forward_w4(buf, group, L["x"], L["w_router"], W["w1"], W["w3"], W["w2"], L["bias"])
    torch.cuda.synchronize()
    assert B.device_status(buf.ws) == 0
    x64, wr64 = P.to_f64(L["x"]), P.to_f64(L["w_router"])
    R = int(buf.offsets[-1])
    g = dict(dtype=cfg.dtype, probs=buf.probs.cpu().numpy().astype(np.float64),
             idx=buf.topk_idx.cpu().numpy(),
             gate=buf.topk_gate.cpu().numpy().astype(np.float64), counts=buf.counts.cpu().numpy(),
             n_ffn=buf.n_ffn.cpu().numpy(), offsets=buf.offsets.cpu().numpy(),
             row_token=buf.row_token[:R].cpu().numpy(), slot_pos=buf.slot_pos.cpu().numpy(),
             x_perm=None, R=R)
    idx_ref, probs, _ = P.check_routing_and_dispatch(g, x64, wr64, L["bias"], cfg.N, cfg.K)
    off, rt, sp = orc.canonical_permutation(idx_ref, cfg.N)
    rows = {"w1": (cfg.I, cfg.d), "w3": (cfg.I, cfg.d), "w2": (cfg.d, cfg.I)}
    y = np.zeros((R, cfg.d))
    for e in range(cfg.N):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        w = {k: decode((W[k][0][e:e + 1], W[k][1][e:e + 1]), *rows[k], group)[0] for k in W}
        p = x64[rt[a:b]] @ w["w1"].T
        y[a:b] = (p * sigmoid(p) * (x64[rt[a:b]] @ w["w3"].T)) @ w["w2"].T
    P.assert_close(P.to_f64(buf.y_perm[:R]), y, cfg.dtype, "y_perm")
    gate = orc.gates(probs, idx_ref)
    P.assert_close(P.to_f64(buf.out), orc.combine(x64, y, idx_ref, gate, sp, cfg.N), cfg.dtype,
                   "out")
