"""The measured cases of the operators around and inside the MoE layer: the
residual RMS norm and its backward pass, the dispatch of 8-bit rows, the 4-bit
expert products, and the global gradient norm with clipping.

``run`` computes an operator either through the package (``own``) or in plain
torch; ``exact`` is its definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
MAX_NORM = 1.0

# Layer shapes: (d, N, Z, K, I) of this repository's workloads, and two odd ones.
SHAPES = {
    "tiny": (256, 16, 8, 4, 128),
    "mid": (2048, 64, 32, 6, 1024),
    "slice": (6144, 32, 16, 12, 2048),   # the LongCat expert geometry on 32 experts
    "odd": (1000, 7, 3, 3, 616),
    "ragged": (1832, 24, 0, 2, 1176),
}
DISPATCH = {"mid": (2048, 64, 32, 6), "slice": (6144, 32, 16, 12), "longcat": (6144, 512, 256, 12)}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decode batch entering the layer: the smallest call, latency counts
        {"name": "norm decode bf16", "op": "norm", "T": 16, "d": 2048, "dtype": "bf16",
         "residual": True, "mx": False},
        # a prefill batch entering the layer with MXFP8 experts: bandwidth counts
        {"name": "norm prefill bf16 mx", "op": "norm", "T": 8192, "d": 6144, "dtype": "bf16",
         "residual": True, "mx": True},
        # a training step's norm, gradient of the residual stream joined
        {"name": "norm backward bf16", "op": "norm_bwd", "T": 8192, "d": 6144, "dtype": "bf16",
         "dsum": True},
        # a small fp32 model's training step, odd sizes, no residual branch
        {"name": "norm backward f32 odd", "op": "norm_bwd", "T": 333, "d": 1000, "dtype": "f32",
         "dsum": False},
        # a mid-sized batch of 8-bit rows sent to its experts
        {"name": "dispatch 8-bit mid", "op": "dispatch", "shape": "mid", "T": 1024},
        # the full prefill batch, two thirds of its slots on FFN experts
        {"name": "dispatch 8-bit longcat", "op": "dispatch", "shape": "longcat", "T": 8192},
        # one token being generated
        {"name": "gate_up w4 one token", "op": "gate_up", "shape": "mid", "T": 1, "group": 128},
        # the largest decode batch of the mid layer, about 16 rows an expert
        {"name": "gate_up w4 T=256", "op": "gate_up", "shape": "mid", "T": 256, "group": 64},
        # the second half at the same batch
        {"name": "down w4 T=256", "op": "down", "shape": "mid", "T": 256, "group": 128},
        # a few users at the LongCat expert geometry, an odd batch and the finest groups
        {"name": "down w4 slice T=13", "op": "down", "shape": "slice", "T": 13, "group": 32},
        # the gradients of one mid layer after its backward pass
        {"name": "clip mid layer bf16", "op": "clip", "tensors": 4, "total": 402849792,
         "dtype": "bf16"},
        # many small tensors of odd sizes, both types (a whole small model)
        {"name": "clip 53 odd tensors", "op": "clip", "tensors": 53, "total": 1500007,
         "dtype": "mixed"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "dispatch", "gate_up", "down", "clip"])
    if op in ("norm", "norm_bwd"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        mx = op == "norm" and dtype == "bf16" and rng.random() < 0.5
        d = 8 * _log_int(rng, 16, 768)
        if mx:
            d = max(32, d // 32 * 32)
        T = _log_int(rng, 1, 8192 if dtype == "bf16" else 4096)
        if op == "norm":
            return {"op": op, "T": T, "d": d, "dtype": dtype, "residual": rng.random() < 0.7,
                    "mx": mx}
        return {"op": op, "T": T, "d": d, "dtype": dtype, "dsum": rng.random() < 0.7}
    if op == "dispatch":
        shape = rng.choice(sorted(DISPATCH))
        return {"op": op, "shape": shape, "T": _log_int(rng, 1, 8192)}
    if op in ("gate_up", "down"):
        shape = rng.choice(sorted(SHAPES))
        return {"op": op, "shape": shape, "T": _log_int(rng, 1, 64 if shape == "slice" else 256),
                "group": rng.choice([32, 64, 128])}
    return {"op": op, "tensors": _log_int(rng, 1, 60), "total": _log_int(rng, 1000, 200000000),
            "dtype": rng.choice(["bf16", "f32", "mixed"])}


# --- inputs ---------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _tensor_sizes(case):
    """Sizes of the gradient list: one small tensor and even large ones (a layer's
    router and expert weights), or a ragged spread over two decades."""
    n, total = case["tensors"], case["total"]
    if n == 4:
        first = min(96 * 2048, total // 4)
        each = (total - first) // 3
        return [first, each, each, total - first - 2 * each]
    share = [10.0 ** (2.0 * ((7 * i) % n) / n) for i in range(n)]
    s = sum(share)
    return [max(1, int(total * v / s)) for v in share]


def _tensor_dtypes(case):
    if case["dtype"] == "mixed":
        return [DTYPES["f32" if i % 3 == 1 else "bf16"] for i in range(case["tensors"])]
    return [DTYPES[case["dtype"]]] * case["tensors"]


def _routing(T, N, Z, K, g):
    """Distinct experts per token with a mild preference among them, and the dispatch
    layout of the FFN slots: rows of an expert in token order.  The loads are the
    same for every seed (so that outputs have one size), which expert and which
    token has them is not."""
    E = N + Z
    load = _gen(E + 1000 * K)
    score = torch.rand((T, E), generator=load, device="cuda")
    score += 0.3 * torch.rand((1, E), generator=load, device="cuda")
    name = torch.cat([torch.randperm(N, generator=g, device="cuda"),
                      N + torch.randperm(Z, generator=g, device="cuda")])
    idx = name[score.topk(K, dim=1).indices[torch.randperm(T, generator=g, device="cuda")]]
    flat = idx.reshape(-1)
    rows = (flat < N).nonzero().squeeze(1)
    order = torch.argsort(flat[rows], stable=True)
    expert = flat[rows][order]
    count = torch.bincount(expert, minlength=N)
    offsets = torch.zeros(N + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = count.cumsum(0)
    return {"topk_idx": idx.to(torch.int32).contiguous(),
            "counts": torch.bincount(flat, minlength=E).to(torch.int32),
            "offsets": offsets.to(torch.int32),
            "row_token": (rows[order] // K).to(torch.int32).contiguous(),
            "row_expert": expert, "R": int(offsets[-1])}


def _w4(n, rows, cols, group, g):
    """4-bit weights as the package lays them out: codes in blocks of 16 rows by 128
    columns (rows and columns padded with zeros), one bf16 scale a row and group."""
    rb, sp = -(-rows // 16), -(-cols // 128)
    codes = torch.empty((n, rb, sp, 1024), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (rb * sp * 2048))
    for m in range(0, n, step):
        k = min(step, n - m)
        v = torch.randn((k, rb, sp, 1024, 2), generator=g, device="cuda").mul_(2.4).round_()
        v = v.clamp_(-8, 7).add_(8).to(torch.uint8)
        codes[m:m + k] = v[..., 0] | (v[..., 1] << 4)
    scales = torch.rand((n, rb, sp, 16, 128 // group), generator=g, device="cuda")
    scales = (scales * 0.01 + 0.004).to(torch.bfloat16)
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("norm", "norm_bwd"):
        T, d, dt = case["T"], case["d"], DTYPES[case["dtype"]]
        s["w"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        # token rows of different magnitudes, as the residual stream has them
        mag = torch.exp(0.5 * torch.randn((T, 1), generator=g, device="cuda"))
        s["x"] = (torch.randn((T, d), generator=g, device="cuda") * mag).to(dt)
        if op == "norm":
            s["res"] = _randn((T, d), g, dt) if case["residual"] else None
            s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["y"] = torch.empty_like(s["x"])
            s["inv"] = torch.empty(T, device="cuda")
            if case["mx"]:
                s["q"] = torch.empty((T, d), dtype=torch.uint8, device="cuda")
                s["sf"] = torch.empty((T, d // 32), dtype=torch.uint8, device="cuda")
        else:
            s["inv"] = (s["x"].double().square().mean(1) + EPS).rsqrt().float()
            s["dy"] = _randn((T, d), g, dt)
            s["dsum"] = _randn((T, d), g, dt) if case["dsum"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty_like(s["w"])
    elif op == "dispatch":
        d, N, Z, K = DISPATCH[case["shape"]]
        T = case["T"]
        s.update(_routing(T, N, Z, K, g))
        s["dims"] = (T, d, N, Z, K, 128)
        v = torch.randn((T, d), generator=g, device="cuda").mul_(80.0).clamp_(-448.0, 448.0)
        s["q"] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        s["sf"] = torch.randint(112, 124, (T, d // 32), generator=g, device="cuda").to(torch.uint8)
        i32 = dict(dtype=torch.int32, device="cuda")
        s["out_offsets"] = torch.empty(N + 1, **i32)
        s["out_row_token"] = torch.empty(T * K, **i32)
        s["out_slot_pos"] = torch.empty((T, K), **i32)
        s["xq"] = torch.empty((T * K, d), dtype=torch.uint8, device="cuda")
        s["xsf"] = torch.empty((T * K, d // 32), dtype=torch.uint8, device="cuda")
    elif op in ("gate_up", "down"):
        d, N, Z, K, I = SHAPES[case["shape"]]
        T = case["T"]
        s.update(_routing(T, N, Z, K, g))
        s["dims"] = (T, d, N, Z, K, I)
        # the experts that have rows, and each row's place in a batch padded by expert:
        # the plan of the plain form
        s["touched"], s["slot"] = s["row_expert"].unique(return_inverse=True)
        s["row"] = (torch.arange(s["R"], device="cuda") - s["offsets"].long()[s["row_expert"]])
        s["most"] = int(s["row"].max()) + 1 if s["R"] else 0
        if op == "gate_up":
            s["x"] = _randn((T, d), g, torch.bfloat16)
            s["w1"], s["w3"] = (_w4(N, I, d, case["group"], g) for _ in range(2))
            s["out"] = torch.empty((T * K, I), dtype=torch.bfloat16, device="cuda")
        else:
            s["h"] = _randn((T * K, I), g, torch.bfloat16, 0.3)
            s["w2"] = _w4(N, d, I, case["group"], g)
            s["out"] = torch.empty((T * K, d), dtype=torch.bfloat16, device="cuda")
    else:
        s["grads"] = [_randn((n,), g, dt, 0.02)
                      for n, dt in zip(_tensor_sizes(case), _tensor_dtypes(case))]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        s["norm"] = torch.empty(1, device="cuda")
    return s


# --- one pass -------------------------------------------------------------------

def _run_own(s):
    from mixture_experts_layer_30_b200 import binding as B
    op = s["op"]
    if op == "norm":
        mx = s["case"]["mx"]
        B.rmsnorm(s["x"], s["w"], EPS, s["y"], residual=s["res"], sum_out=s["sum"],
                  inv_rms=s["inv"], y_q=s["q"] if mx else None, y_sf=s["sf"] if mx else None)
        out = {"y": s["y"], "inv": s["inv"], "sum": s["sum"]}
        if mx:
            out["q"] = s["q"].view(torch.float8_e4m3fn)
            out["scale"] = s["sf"].view(torch.float8_e8m0fnu)
        return out
    if op == "norm_bwd":
        if "ws" not in s:
            s["ws"] = B.new_rmsnorm_workspace(*s["x"].shape)
        B.rmsnorm_backward(s["x"], s["w"], s["inv"], s["dy"], s["dx"], s["dw"], s["ws"],
                           dsum=s["dsum"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "clip":
        if "plan" not in s:
            s["plan"] = B.GradientList(s["grads"], out=s["out"])
        B.clip_gradients(s["plan"], MAX_NORM, s["norm"])
        return {"norm": s["norm"], "grads": s["out"]}
    if "layer" not in s:
        s["layer"] = B.make_shape(*s["dims"], "bf16")
        s["ws"] = B.new_workspace(s["layer"])
    R = s["R"]
    if op == "dispatch":
        B.permute_mxfp8_rows(s["layer"], s["q"], s["sf"], s["topk_idx"], s["counts"],
                             s["out_offsets"], s["out_row_token"], s["out_slot_pos"], s["xq"],
                             s["xsf"], s["ws"])
        return {"offsets": s["out_offsets"], "row_token": s["out_row_token"][:R],
                "slot_pos": s["out_slot_pos"], "q": s["xq"][:R], "sf": s["xsf"][:R]}
    group = s["case"]["group"]
    if op == "gate_up":
        B.expert_gate_up_w4(s["layer"], group, s["x"], s["row_token"], s["w1"], s["w3"],
                            s["offsets"], s["out"], s["ws"])
    else:
        B.expert_down_w4(s["layer"], group, s["h"], s["w2"], s["offsets"], s["out"], s["ws"])
    return {"out": s["out"][:R]}


def _mx_round(y):
    """MXFP8 of y: E4M3 with the smallest 2^s per 32 values that holds the largest."""
    T, d = y.shape
    blocks = y.float().view(T, d // 32, 32)
    m, e = torch.frexp(blocks.abs().amax(2))
    s = torch.where(m <= 0.875, e - 9, e - 8)
    s = torch.where(m == 0, torch.zeros_like(s), s)
    codes = torch.ldexp(blocks, -s.unsqueeze(2)).to(torch.float8_e4m3fn)
    return codes.view(T, d), (s + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _w4_values(w, experts, rows, cols, dtype):
    """The weights [experts, rows, cols] that codes and scales stand for."""
    codes, scales = (t[experts] for t in w)
    n, rb, sp, _ = codes.shape
    # block bytes: row half, row, lane quad t, 32-column piece j, byte; nibble p of the
    # four bytes holds column 2p (p < 4) or 2(p - 4) + 1 of the lane's eight
    c = codes.view(n, rb, sp, 2, 8, 4, 4, 4, 1)
    c = torch.cat([c & 15, c >> 4], dim=-1).view(n, rb, sp, 2, 8, 4, 4, 2, 4)
    c = c.permute(0, 1, 3, 4, 2, 6, 5, 8, 7).reshape(n, rb * 16, sp * 128)
    gps = scales.shape[-1]
    sc = scales.permute(0, 1, 3, 2, 4).reshape(n, rb * 16, sp * gps, 1).to(dtype)
    v = (c.to(dtype) - 8.0).view(n, rb * 16, sp * gps, 128 // gps) * sc
    return v.view(n, rb * 16, sp * 128)[:, :rows, :cols]


def _by_expert(s, a, dtype):
    """Rows of `a` in a batch [touched experts, most rows, columns] padded with zeros."""
    p = torch.zeros((s["touched"].numel(), s["most"], a.shape[1]), dtype=dtype, device="cuda")
    p[s["slot"], s["row"]] = a.to(dtype)
    return p


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "norm":
        t = s["x"]
        if s["res"] is not None:
            t = (t.float() + s["res"].float()).to(t.dtype)
        f = t.float()
        inv = torch.rsqrt((f * f).mean(1) + EPS)
        y = (f * inv.unsqueeze(1) * s["w"].float()).to(t.dtype)
        out = {"y": y, "inv": inv, "sum": t if s["res"] is not None else None}
        if s["case"]["mx"]:
            out["q"], out["scale"] = _mx_round(y)
        return out
    if op == "norm_bwd":
        xhat = s["x"].float() * s["inv"].unsqueeze(1)
        dy = s["dy"].float()
        g = dy * s["w"].float()
        dx = (g - xhat * (g * xhat).mean(1, keepdim=True)) * s["inv"].unsqueeze(1)
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        dw = (dy * xhat).sum(0, dtype=torch.float64)
        return {"dx": dx.to(s["x"].dtype), "dw": dw.to(s["w"].dtype)}
    if op == "dispatch":
        T, d, N, Z, K, _ = s["dims"]
        flat = s["topk_idx"].reshape(-1).long()
        key = torch.where(flat < N, flat, torch.full_like(flat, N))
        order = torch.argsort(key, stable=True)[:s["R"]]
        slot = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
        slot[order] = torch.arange(s["R"], dtype=torch.int32, device="cuda")
        bounds = torch.arange(N, device="cuda").unsqueeze(1)
        counts = (key.unsqueeze(0) == bounds).sum(1)
        offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)]).to(torch.int32)
        rt = order // K
        return {"offsets": offsets, "row_token": rt.to(torch.int32),
                "slot_pos": slot.view(T, K), "q": s["q"][rt], "sf": s["sf"][rt]}
    if op == "clip":
        sq = [t.float().square().sum(dtype=torch.float64) for t in s["grads"]]
        norm = torch.stack(sq).sum().sqrt().float().view(1)
        coef = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
        return {"norm": norm, "grads": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}
    T, d, N, Z, K, I = s["dims"]
    if op == "gate_up":
        x = _by_expert(s, s["x"][s["row_token"].long()], torch.float32)
        a = torch.bmm(x, _w4_values(s["w1"], s["touched"], I, d, x.dtype).transpose(1, 2))
        u = torch.bmm(x, _w4_values(s["w3"], s["touched"], I, d, x.dtype).transpose(1, 2))
        y = a * torch.sigmoid(a) * u
    else:
        x = _by_expert(s, s["h"][:s["R"]], torch.float32)
        y = torch.bmm(x, _w4_values(s["w2"], s["touched"], d, I, x.dtype).transpose(1, 2))
    return {"out": y[s["slot"], s["row"]].to(torch.bfloat16)}


# --- what a pass cannot do without ----------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        T, d, e = case["T"], case["d"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm":
            b = T * d * e * (4 if case["residual"] else 2) + d * e + 4 * T
            b += T * d * 33 // 32 if case["mx"] else 0
            return {"bytes": b, "flops": T * d * (5 if case["residual"] else 4)}
        return {"bytes": T * d * e * (4 if case["dsum"] else 3) + 2 * d * e + 4 * T,
                "flops": 10 * T * d}
    if op == "dispatch":
        d, N, Z, K = DISPATCH[case["shape"]]
        rows = case["T"] * K * N / (N + Z)
        return {"bytes": (case["T"] + rows) * d * 33 / 32 + 4 * (2 * case["T"] * K + rows + 2 * N),
                "flops": 0}
    if op == "clip":
        e = 2 if case["dtype"] == "bf16" else 4 if case["dtype"] == "f32" else 8 / 3
        return {"bytes": 2 * e * case["total"], "flops": 3 * case["total"]}
    d, N, Z, K, I = SHAPES[case["shape"]]
    rows = case["T"] * K * N / (N + Z)
    touched = N * (1 - (1 - K / (N + Z)) ** case["T"])
    mats = 2 if op == "gate_up" else 1
    b = mats * touched * I * d * (0.5 + 2 / case["group"])
    b += (case["T"] * d + rows * I if op == "gate_up" else rows * (I + d)) * 2
    return {"bytes": b, "flops": 2 * mats * rows * I * d}


# --- the definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        return None  # whole numbers only
    if op == "norm":
        x = s["x"].double()
        total = None
        if s["res"] is not None:
            x = total = (x + s["res"].double()).to(s["x"].dtype).double()
        inv = 1.0 / torch.sqrt(torch.einsum("td,td->t", x, x) / x.shape[1] + EPS)
        y = torch.einsum("td,t,d->td", x, inv, s["w"].double())
        out = {"y": y, "inv": inv, "sum": total}
        if case["mx"]:
            out["q"] = out["scale"] = None  # next to a border of 8 bits either code is right
        return out
    if op == "norm_bwd":
        x, dy, w, inv = (s[k].double() for k in ("x", "dy", "w", "inv"))
        proj = torch.einsum("td,td,d->t", x, dy, w) * inv ** 3 / x.shape[1]
        dx = torch.einsum("td,d,t->td", dy, w, inv) - x * proj[:, None]
        if s["dsum"] is not None:
            dx += s["dsum"].double()
        return {"dx": dx, "dw": torch.einsum("td,td,t->d", dy, x, inv)}
    if op == "clip":
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(t.double())) ** 2
                             for t in s["grads"]))
        coef = min(1.0, MAX_NORM / (norm + 1e-6))
        return {"norm": torch.tensor([norm], dtype=torch.float64),
                "grads": [t.double() * coef for t in s["grads"]]}
    T, d, N, Z, K, I = s["dims"]
    cols = I if op == "gate_up" else d
    y = torch.zeros((s["R"], cols), dtype=torch.float64, device="cuda")
    off = s["offsets"].tolist()
    rt = s["row_token"].long()
    for e in range(N):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        at = torch.tensor([e], device="cuda")
        if op == "gate_up":
            x = s["x"][rt[a:b]].double()
            gate = x @ _w4_table(s["w1"], at, I, d).T
            y[a:b] = gate / (1.0 + torch.exp(-gate)) * (x @ _w4_table(s["w3"], at, I, d).T)
        else:
            y[a:b] = s["h"][a:b].double() @ _w4_table(s["w2"], at, d, I).T
    return {"out": y}


def _w4_table(w, at, rows, cols):
    """One expert's weights by looking each (row, column) up where the format keeps it."""
    codes, scales = w[0][at[0]].reshape(-1), w[1][at[0]]
    sp, gps = w[0].shape[2], w[1].shape[-1]
    r = torch.arange(rows, device="cuda").unsqueeze(1)
    c = torch.arange(cols, device="cuda").unsqueeze(0)
    in_span, in8 = c % 128, c % 8
    block = (r // 16) * sp + c // 128
    nibble = in8 // 2 + 4 * (in8 % 2)
    byte = (r % 16) * 64 + (in_span % 32) // 8 * 16 + in_span // 32 * 4 + nibble // 2
    v = codes[block * 1024 + byte].int()
    v = torch.where(nibble % 2 == 1, v >> 4, v & 15)
    sc = scales[r // 16, c // 128, r % 16, in_span * gps // 128]
    return (v.double() - 8.0) * sc.double()
