"""Host-side checks of the operators around the layer at their edges: every tensor that is
too short for its shape is refused before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_30_b200 import binding as B
from mixture_experts_layer_30_b200 import build as BUILD

FAKE = ctypes.c_void_p(0x10000)
U8, I32, BF16 = torch.uint8, torch.int32, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.lib()


def flat(n, dtype):
    return torch.zeros(n, dtype=dtype)


T, D, N, Z, K, I = 16, 256, 4, 2, 2, 128
R = T * K
DISPATCH = {"x_q": (T * D, U8), "x_sf": (T * D // 32, U8), "topk_idx": (R, I32),
            "counts": (N + Z, I32), "offsets": (N + 1, I32), "row_token": (R, I32),
            "slot_pos": (R, I32), "x_perm_q": (R * D, U8), "x_perm_sf": (R * D // 32, U8)}


@pytest.mark.parametrize("name", sorted(DISPATCH))
def test_short_tensors_of_the_8bit_dispatch_are_refused(lib, name):
    """The kernels' extents come from the shape alone: one element less would be read or
    written past its end."""
    s = B.make_shape(T, D, N, Z, K, I, "bf16")
    a = {k: flat(n - (k == name), dt) for k, (n, dt) in DISPATCH.items()}
    with pytest.raises(ValueError, match=f"{name} has"):
        B.permute_mxfp8_rows(s, *a.values(), flat(1024, U8))


def w4_pair(rows, cols, group):
    blocks = N * -(-rows // 16) * -(-cols // 128)
    return flat(blocks * 1024, U8), flat(blocks * 2048 // group, BF16)


@pytest.mark.parametrize("name,gather", [("x", True), ("x", False), ("offsets", True),
                                         ("h", True), ("h", False)])
def test_short_tensors_of_the_4bit_gate_up_are_refused(lib, name, gather):
    s = B.make_shape(T, D, N, Z, K, I, "bf16")
    n = {"x": (T if gather else R) * D, "offsets": N + 1, "h": R * I}
    n[name] -= 1
    with pytest.raises(ValueError, match=f"{name} has"):
        B.expert_gate_up_w4(s, 64, flat(n["x"], BF16), flat(R, I32) if gather else None,
                            w4_pair(I, D, 64), w4_pair(I, D, 64), flat(n["offsets"], I32),
                            flat(n["h"], BF16), flat(1024, U8))


@pytest.mark.parametrize("name", ["h", "offsets", "y_perm"])
def test_short_tensors_of_the_4bit_down_are_refused(lib, name):
    s = B.make_shape(T, D, N, Z, K, I, "bf16")
    n = {"h": R * I, "offsets": N + 1, "y_perm": R * D}
    n[name] -= 1
    with pytest.raises(ValueError, match=f"{name} has"):
        B.expert_down_w4(s, 64, flat(n["h"], BF16), w4_pair(D, I, 64), flat(n["offsets"], I32),
                         flat(n["y_perm"], BF16), flat(1024, U8))


def test_row_count_of_the_4bit_gate_up_stays_within_the_shape(lib):
    s = B.make_shape(T, D, N, Z, K, I, "bf16")
    for rows in (-1, R + 1):
        code = lib.moe_expert_gate_up_w4_rows(ctypes.byref(s), 64, rows, FAKE, FAKE, FAKE, FAKE,
                                              FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None)
        assert code == 1 and b"n_rows" in lib.moe_last_error()


def test_prenorm_without_a_residual_norms_x_itself(lib, monkeypatch):
    """A model's first block has no residual yet: no sum is asked for, and the backward pass
    reads x, not a buffer that nothing wrote."""
    calls = []
    monkeypatch.setattr(B, "rmsnorm", lambda *a, **k: calls.append((a, k)))
    monkeypatch.setattr(B, "rmsnorm_backward", lambda *a, **k: calls.append((a, k)))
    nb = B.PreNormBuffers(B.make_shape(4, 64, 4, 2, 2, 64, "f32"), device="cpu", train=True)
    x, r, w, dy = (torch.zeros((4, 64)) for _ in range(4))
    B.prenorm(nb, x, None, w)
    assert calls[-1][1]["residual"] is None and calls[-1][1]["sum_out"] is None
    B.prenorm_backward(nb, w, dy)
    assert calls[-1][0][0] is x
    B.prenorm(nb, x, r, w)
    assert calls[-1][1]["residual"] is r and calls[-1][1]["sum_out"] is nb.s
    B.prenorm_backward(nb, w, dy)
    assert calls[-1][0][0] is nb.s


class _Compiled(Exception):
    pass


def test_native_module_of_another_torch_is_built_again(lib, monkeypatch):
    """It uses torch's C++ interface: one compiled against another version is not fresh,
    however new its file is; the CUDA library does not depend on torch and stays."""
    commands = []

    def record(cmd, **kw):
        commands.append(cmd)
        raise _Compiled
    monkeypatch.setattr(BUILD.subprocess, "Popen", record)
    monkeypatch.setattr(BUILD.subprocess, "run", record)
    BUILD.build()
    assert not commands
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(_Compiled):
        BUILD.build()
    assert [c for c in commands if BUILD.CALLS_SRC in c] and not [c for c in commands
                                                                  if BUILD.SOURCES[0] in c]


def test_calls_go_on_without_the_native_module(lib, monkeypatch):
    """It only shortens the host's part: where it cannot be loaded, the binding's checked path
    makes the same calls, with a warning.  The CUDA library itself has no stand-in."""
    import sys

    import mixture_experts_layer_30_b200 as package
    monkeypatch.delattr(package, "_calls", raising=False)
    monkeypatch.setitem(sys.modules, package.__name__ + "._calls", None)
    monkeypatch.setattr(B, "_calls", None)
    s = B.make_shape(T, D, N, Z, K, I, "bf16")
    with pytest.warns(RuntimeWarning, match="_calls"):
        with pytest.raises(ValueError, match="y_perm has"):
            B.expert_down_w4(s, 64, flat(R * I, BF16), w4_pair(D, I, 64), flat(N + 1, I32),
                             flat(R * D - 1, BF16), flat(1024, U8))
    monkeypatch.setattr(B, "_lib", None)
    monkeypatch.setattr(B, "_calls", None)
    monkeypatch.setattr(B, "LIB_PATH", "/nowhere/libmoe_b200.so")
    with pytest.raises(RuntimeError, match="missing"):
        B._native()


def test_w4_sizes_next_to_32_bits(lib):
    assert lib.moe_w4_code_bytes(1, 2 ** 31 - 1, 1) == 2 ** 27 * 1024
    assert lib.moe_w4_code_bytes(1, 1, 2 ** 31 - 1) == 2 ** 24 * 1024
    assert lib.moe_w4_scale_bytes(1, 2 ** 31 - 1, 1, 128) == 2 ** 27 * 32
    # the end of the last block of columns would not be a 32-bit number
    for d, I in ((2 ** 31 - 8, 8), (8, 2 ** 31 - 8)):
        s = B.make_shape(1, d, 1, 0, 1, I, "bf16")
        for code in (lib.moe_expert_gate_up_w4(ctypes.byref(s), 32, FAKE, FAKE, FAKE, FAKE, FAKE,
                                               FAKE, FAKE, FAKE, FAKE, 1 << 60, None),
                     lib.moe_expert_down_w4(ctypes.byref(s), 32, FAKE, FAKE, FAKE, FAKE, FAKE,
                                            FAKE, 1 << 60, None)):
            assert code == 2 and b"past int32" in lib.moe_last_error()


@pytest.mark.parametrize("shape", [(2 ** 31, 1, 1), (1, 2 ** 32 + 16, 1), (1, 1, 2 ** 31)])
def test_4bit_weights_past_32_bits_are_refused(lib, shape):
    """As 32-bit numbers these would be negative or another, small size."""
    with pytest.raises(ValueError, match="more than"):
        B.quantize_weights_w4(torch.empty(shape, dtype=BF16, device="meta"))
