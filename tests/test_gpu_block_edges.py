"""Calls of the operators around the layer at the edges of what they take."""
import pytest
import torch

from mixture_experts_layer_30_b200 import binding as B
from tests.test_gpu_w4 import decode, offsets_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_w4_rows_behind_a_short_row_token_are_not_read(dtype, native, monkeypatch):
    """row_token holds the rows of the first two experts only: the third counts as empty."""
    if not native:
        class Refuses:
            def __getattr__(self, name):
                return lambda *args: -1
        monkeypatch.setattr(B, "_native", lambda: Refuses())
    counts, d, I = [3, 0, 9, 5], 128, 64
    R = sum(counts)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(1)
    shape = B.make_shape(R, d, 4, 0, 1, I, dtype)
    ws = B.new_workspace(shape)
    w1, w3 = (B.quantize_weights_w4(torch.randn((4, I, d), generator=g).to(dt).cuda(), 32)
              for _ in range(2))
    x = torch.randn((R, d), generator=g).to(dt).cuda()
    rt = torch.arange(R, dtype=torch.int32).flip(0).cuda()
    off = offsets_of(counts).cuda()
    want = torch.full((R, I), 7.0, dtype=dt, device="cuda")
    B.expert_gate_up_w4(shape, 32, x, rt, w1, w3, off, want, ws)
    torch.cuda.synchronize()
    assert B.device_status(ws) == 0
    for held, rows in ((R, R), (R - 1, 12), (12, 12), (11, 3), (0, 0)):
        h = torch.full_like(want, 7.0)
        B.expert_gate_up_w4(shape, 32, x, rt[:held].clone(), w1, w3, off, h, ws)
        torch.cuda.synchronize()
        assert torch.equal(h[:rows], want[:rows]) and (h[rows:] == 7).all(), held
        assert B.device_status(ws) == (0 if held == R else B.DEV_BAD_OFFSETS), held


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prenorm_of_a_first_block(dtype):
    """Without a residual prenorm is rmsnorm of x, and its backward pass that of x; the next
    block's call with a residual on the same buffers is unchanged by it."""
    shape = B.make_shape(9, 256, 4, 2, 2, 128, dtype)
    dt = B.torch_dtype(shape)
    g = torch.Generator().manual_seed(2)
    x, r, dy = (torch.randn((9, 256), generator=g).to(dt).cuda() for _ in range(3))
    w = (1 + 0.2 * torch.randn(256, generator=g)).to(dt).cuda()
    mx = dtype == "bf16"
    nb = B.PreNormBuffers(shape, mx=mx, train=True)
    ws = B.new_rmsnorm_workspace(9, 256)
    for res in (None, r, None):
        nb.s.fill_(float("nan"))
        y = B.prenorm(nb, x, res, w)
        B.prenorm_backward(nb, w, dy, dsum=r)
        s = x if res is None else torch.empty_like(x)
        y2, inv = torch.empty_like(x), torch.empty(9, device="cuda")
        q, sf = (torch.empty_like(t) for t in nb.x_q) if mx else (None, None)
        B.rmsnorm(x, w, 1e-5, y2, residual=res, sum_out=None if res is None else s, inv_rms=inv,
                  y_q=q, y_sf=sf)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        B.rmsnorm_backward(s, w, inv, dy, dx, dw, ws, dsum=r)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(nb.inv_rms, inv)
        assert torch.equal(nb.dx, dx) and torch.equal(nb.dweight, dw)
        if mx:
            assert torch.equal(nb.x_q[0], q) and torch.equal(nb.x_q[1], sf)
        s64 = s.double()
        want = s64 * (s64.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w.double()
        # fp32 arithmetic (a sum of 256, its root, two products) and one rounding of the type
        tol = want.abs() * (torch.finfo(dt).eps / 2 + 24 * 2.0 ** -24)
        assert ((y.double() - want).abs() <= tol * (1 + 2.0 ** -7)).all()


def test_clip_by_a_joined_norm():
    """Two ranks' lists, each clipped by the norm of both, are one list clipped by its own: the
    factor's rounding (3 * 2^-24), the norm's (6 * 2^-24 on each side) and the result's."""
    g = torch.Generator().manual_seed(3)
    lists = [[(torch.randn(n, generator=g) * 0.1).to(dt).cuda() for n, dt in spec]
             for spec in (((1001, torch.float32), (70_000, torch.bfloat16)),
                          ((5, torch.bfloat16), (33_333, torch.float32)))]
    before = [[t.clone() for t in ts] for ts in lists]
    norms = [torch.empty(1, device="cuda") for _ in lists]
    plans = [B.GradientList(ts) for ts in lists]
    for p, n in zip(plans, norms):
        B.gradient_norm(p, n)
    joined = (norms[0].double().square() + norms[1].double().square()).sqrt().float()
    for p in plans:
        assert B.clip_by_norm(p, 0.5, joined) is joined
    torch.cuda.synchronize()
    n64 = sum(float(t.double().square().sum()) for ts in before for t in ts) ** 0.5
    assert abs(float(joined) - n64) <= 7 * 2.0 ** -24 * n64
    for ts, old in zip(lists, before):
        for a, b in zip(ts, old):
            w = b.double() * (0.5 / (n64 + 1e-6))
            tol = w.abs() * (torch.finfo(a.dtype).eps / 2 + 16 * 2.0 ** -24) * (1 + 2.0 ** -7)
            assert ((a.double() - w).abs() <= tol + 1e-38).all()
    with pytest.raises(B.MoEError, match="max_norm"):
        B.clip_by_norm(plans[0], -1.0, joined)
    with pytest.raises(ValueError, match="norm has 2 elements"):
        B.clip_by_norm(plans[0], 1.0, torch.empty(2, device="cuda"))


def test_a_gradient_list_is_ready_for_any_stream():
    """Made on a stream that is busy, used at once on another: the workspace is clear by then
    (its memory held ones before)."""
    n = B.lib().moe_grad_workspace_bytes(1)
    g = torch.linspace(-1, 1, 4097, device="cuda")
    want = float(g.double().norm())
    busy, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for explicit in (False, True):
        norm = torch.zeros(1, device="cuda")
        with torch.cuda.stream(busy):
            torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")  # freed, taken again below
            torch.cuda._sleep(20_000_000)
            if not explicit:
                plan = B.GradientList([g])
        if explicit:
            plan = B.GradientList([g], stream=busy)
        B.gradient_norm(plan, norm, stream=other)
        torch.cuda.synchronize()
        assert abs(float(norm) - want) <= 6 * 2.0 ** -24 * want


def test_a_gradient_list_made_in_a_capture():
    """Its clearing becomes part of the graph, in front of the calls on it."""
    g = torch.linspace(-1, 1, 4097, device="cuda")
    norm = torch.zeros(1, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        plan = B.GradientList([g])
        B.gradient_norm(plan, norm)
    for scale in (1.0, 2.0):
        g.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        want = float(g.double().norm())
        assert abs(float(norm) - want) <= 6 * 2.0 ** -24 * want
    del plan, graph


def test_a_norm_after_two_at_once_is_right():
    """Two calls of one list in flight at once are not promised a norm, but they leave the
    workspace as they found it."""
    ts = [torch.full((3_000_001,), 0.5, device="cuda"), torch.full((77,), 2.0, device="cuda")]
    plan = B.GradientList(ts)
    want = (3_000_001 * 0.25 + 77 * 4.0) ** 0.5
    streams, norms = [torch.cuda.Stream() for _ in range(2)], torch.zeros(3, 1, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        for st, n in zip(streams, norms):
            B.gradient_norm(plan, n, stream=st)
        torch.cuda.synchronize()
        norms[2].zero_()
        B.gradient_norm(plan, norms[2])
        assert abs(float(norms[2]) - want) <= 6 * 2.0 ** -24 * want
        assert int(plan.ws[4:8].view(torch.int32)) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1e-37, 1e-30, 1e-22, 3e-23, 2e-23, 1e-19, 1e-16, 1e16, 1e19,
                                   1e20, 1e30])
def test_norm_of_gradients_whose_squares_leave_fp32(scale, dtype):
    """Below 1e-19 the squares lose their bits in fp32, above 1.8e19 they are infinite.  In 64 bits
    every square of such a vector is exact; where the sum of 4 or 8 is formed in fp32 it is at
    least 2^-110, so that a square below the normal range adds at most 2^-149: the bound of the
    other sizes holds."""
    g = torch.Generator().manual_seed(4)
    for n in (1, 5, 8, 8191, 100_003):
        base = (torch.randn(n + 3, generator=g) * scale).to(dtype).cuda()
        for start in (0, 3):
            t = base[start:start + n]
            norm = torch.zeros(1, device="cuda")
            B.gradient_norm(B.GradientList([t]), norm)
            want = float(t.double().square().sum().sqrt())
            assert 0 < want < 3.4e38
            assert abs(float(norm) - want) <= 6 * 2.0 ** -24 * want + 2.0 ** -150


def test_one_large_entry_leaves_the_other_gradients():
    """A finite entry above 1.8e19 has a finite norm: the factor is small, not 0."""
    g = torch.full((1000,), 1e15, device="cuda")
    g[17] = 1e20
    keep = g.double()
    norm = torch.zeros(1, device="cuda")
    B.clip_gradients(B.GradientList([g]), 1.0, norm)
    want = float(keep.norm())
    assert abs(float(norm) - want) <= 6 * 2.0 ** -24 * want
    w = keep / want
    assert ((g.double() - w).abs() <= w * (13 * 2.0 ** -24) * (1 + 2.0 ** -7)).all()


def test_norm_of_ordinary_and_extreme_entries_together():
    """Small entries beside an ordinary one in the same vector, zeros, and a norm below fp32's
    smallest normal number."""
    t = torch.zeros(4096, device="cuda")
    t[0], t[1], t[4000] = 3.0, 1e-25, 1e-25
    norm = torch.zeros(1, device="cuda")
    B.gradient_norm(B.GradientList([t]), norm)
    assert float(norm) == 3.0
    t.zero_()
    B.gradient_norm(B.GradientList([t]), norm)
    assert float(norm) == 0.0
    t[7] = 2.0 ** -140
    B.gradient_norm(B.GradientList([t]), norm)
    assert float(norm) == 2.0 ** -140


@pytest.mark.parametrize("T", [592, 1184, 4000])
def test_fp32_weight_gradient_keeps_small_rows(T):
    """s = weight = inv_rms = 1, so a column's terms are dy itself: 1 in the first 32 rows, then
    2^-25, which an fp32 sum of ones drops.  A CTA's own rows are summed in fp32, exactly here:
    a CTA has at most 7 of them, at a stride of the grid, so all but 32 CTAs sum small terms
    alone and those 32 lose at most 6 * 2^-25 each.  The join of the CTAs is fp64 and the result is
    rounded once: 2^-24 of it."""
    d = 2048
    one = torch.ones((T, d), device="cuda")
    dy = torch.full((T, d), 2.0 ** -25, device="cuda")
    dy[:32] = 1.0
    dw, dx = torch.empty(d, device="cuda"), torch.empty_like(one)
    B.rmsnorm_backward(one, one[0].clone(), torch.ones(T, device="cuda"), dy, dx, dw,
                       B.new_rmsnorm_workspace(T, d))
    torch.cuda.synchronize()
    want = 32 + (T - 32) * 2.0 ** -25
    per = -(-T // 592)
    tol = want * 2.0 ** -24 + 32 * (per - 1) * 2.0 ** -25
    assert (T - 32) * 2.0 ** -25 > 2 * tol  # an fp32 join would be seen
    assert float((dw.double() - want).abs().max()) <= tol


def test_w4_work_whose_cost_passes_32_bits():
    """Runs are cut by cost * parts: in 64 bits where the product does not fit 32.  A contraction
    of 8 and 65536 output columns reach that with small weights; every output is checked
    (tolerance as for the other products: (K / 2 + 32) * 2^-23 of the sums' magnitude)."""
    d, I, counts = 8, 65536, [25_003, 0, 15_006]
    R = sum(counts)
    ctas = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    chunks = sum(c // 16 for c in counts)
    assert chunks * 6 * (I // 64) * ctas >= 2 ** 32
    g = torch.Generator().manual_seed(6)
    shape = B.make_shape(R, d, 3, 0, 1, I, "bf16")
    ws = B.new_workspace(shape)
    W = [B.quantize_weights_w4(torch.randn((3, I, d), generator=g).to(torch.bfloat16).cuda(), 64)
         for _ in range(2)]
    x = torch.randn((R, d), generator=g).to(torch.bfloat16).cuda()
    h = torch.full((R, I), float("nan"), dtype=torch.bfloat16, device="cuda")
    off = offsets_of(counts)
    B.expert_gate_up_w4(shape, 64, x, None, *W, off.cuda(), h, ws)
    torch.cuda.synchronize()
    assert B.device_status(ws) == 0
    for e, m in enumerate(counts):
        if m == 0:
            continue
        w1, w3 = (torch.from_numpy(decode((q[e:e + 1], s[e:e + 1]), I, d, 64)[0]).cuda()
                  for q, s in W)
        for a in range(int(off[e]), int(off[e + 1]), 1000):
            b = min(a + 1000, int(off[e + 1]))
            v = x[a:b].double()
            p, u = v @ w1.T, v @ w3.T
            act = p * torch.sigmoid(p)
            want = act * u
            mag = (1.1 * u.abs() * (v.abs() @ w1.abs().T) + act.abs() * (v.abs() @ w3.abs().T)
                   + want.abs())
            tol = (want.abs() * 2.0 ** -8 + mag * (d / 2 + 32) * 2.0 ** -23) * (1 + 2.0 ** -6)
            assert ((h[a:b].double() - want).abs() <= tol + 1e-37).all(), (e, a)


def test_short_tensors_on_the_device_are_refused():
    """The native path of a call checks lengths too (nothing is launched)."""
    T, d, N, Z, K, I = 16, 256, 4, 2, 2, 128
    R = T * K
    shape = B.make_shape(T, d, N, Z, K, I, "bf16")
    ws = B.new_workspace(shape)
    dev = dict(device="cuda")
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    w1, w2 = (B.quantize_weights_w4(torch.zeros(s, dtype=bf, **dev), 64)
              for s in ((N, I, d), (N, d, I)))
    sizes = {"x_q": (T * d, u8), "x_sf": (T * d // 32, u8), "topk_idx": (R, i32),
             "counts": (N + Z, i32), "offsets": (N + 1, i32), "row_token": (R, i32),
             "slot_pos": (R, i32), "x_perm_q": (R * d, u8), "x_perm_sf": (R * d // 32, u8)}
    before = B.kernel_launches()
    for name in sizes:
        a = [torch.zeros(n - (k == name), dtype=t, **dev) for k, (n, t) in sizes.items()]
        with pytest.raises(ValueError, match=f"{name} has"):
            B.permute_mxfp8_rows(shape, *a, ws)

    def up(x=T * d, rows=R, off=N + 1, h=R * I):
        B.expert_gate_up_w4(shape, 64, torch.zeros(x, dtype=bf, **dev),
                            None if rows is None else torch.zeros(rows, dtype=i32, **dev), w1, w1,
                            torch.zeros(off, dtype=i32, **dev), torch.zeros(h, dtype=bf, **dev), ws)

    def down(h=R * I, off=N + 1, y=R * d):
        B.expert_down_w4(shape, 64, torch.zeros(h, dtype=bf, **dev), w2,
                         torch.zeros(off, dtype=i32, **dev), torch.zeros(y, dtype=bf, **dev), ws)
    for call, args, name in ((up, dict(x=T * d - 1), "x"), (up, dict(rows=None), "x"),
                             (up, dict(off=N), "offsets"), (up, dict(h=R * I - 1), "h"),
                             (down, dict(h=R * I - 1), "h"), (down, dict(off=N), "offsets"),
                             (down, dict(y=R * d - 1), "y_perm")):
        with pytest.raises(ValueError, match=f"^{name} has"):
            call(**args)
    assert B.kernel_launches() == before
    up()
    up(x=R * d, rows=None)
    down()
    torch.cuda.synchronize()
    assert B.device_status(ws) == 0
