"""Calls of the operators around the layer at the edges of what they take."""
import pytest
import torch

from mixture_experts_layer_30_b200 import binding as B
from tests.test_gpu_w4 import offsets_of

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
