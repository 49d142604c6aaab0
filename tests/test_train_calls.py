"""The training entry points' calls on the CPU: refusals, and what the native binding does
around a call.  Nothing is launched: there is no device, or the call is refused before."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import binding_stub

P = ctypes.c_void_p
OKP = 1 << 20          # an aligned address; nothing is launched without a device


@pytest.fixture(scope="module")
def M():
    import expert_layer_dual_b200.moe as moe
    return moe


@pytest.mark.parametrize("change,code", [
    ({"op": 3}, 1), ({"op": -1}, 1), ({"block": -1}, 1), ({"limit": 0}, 1), ({"limit": 999}, 1), ({"limit": 1000001}, 1), ({"N": 100}, 2),
    ({"a": None}, 1), ({"out": OKP + 4}, 1), ({"ws": None}, 1), ({"ws_bytes": 128}, 4), ({"op": 2, "M": 9000000}, 2)])
def test_selftest_refusals(M, change, code):
    a = {"op": 0, "a": OKP, "a_s": OKP, "b": OKP, "b_s": OKP, "M": 5, "N": 256, "K": 128, "out": OKP, "block": 0,
         "limit": 1000, "ws": OKP, "ws_bytes": 256, **change}
    assert M._lib.moe_selftest_product_timeout(
        a["op"], P(a["a"]), P(a["a_s"]), P(a["b"]), P(a["b_s"]), a["M"], a["N"], a["K"], P(a["out"]), 0, a["block"],
        a["limit"], P(a["ws"]), a["ws_bytes"], None) == code


@pytest.mark.parametrize("op,shapes", [(0, ((9, 384), (9, 3), (256, 384), (2, 3), (9, 256))),
                                       (1, ((9, 256), (9, 2), (256, 384), (2, 3), (9, 384))),
                                       (2, ((256, 128), (1, 256), (384, 128), (1, 384), (256, 384)))])
def test_selftest_checks_its_tensors(M, op, shapes):
    types = (torch.uint8, torch.float32, torch.uint8, torch.float32, torch.float32)
    good = [torch.zeros(s, dtype=t) for s, t in zip(shapes, types)]
    ws = torch.zeros(256, dtype=torch.uint8)
    call = lambda t: M.selftest_product_timeout(op, *t[:4], 9, t[4], False, 0, 1000, ws, stream=0)  # noqa: E731
    with pytest.raises(ValueError, match="current CUDA device"):
        call(good)
    for i, name in enumerate(("a", "a_s", "b", "b_s", "out")):
        for bad in (good[i][:-1], good[i].to(torch.bfloat16)):
            with pytest.raises(ValueError, match="expected"):
                call([*good[:i], bad, *good[i + 1:]])


@pytest.mark.parametrize("change,want", [
    ({"x": torch.zeros((4, 256), dtype=torch.float16)}, "1024 elements or more of bfloat16"),
    ({"x": torch.zeros((4, 256))}, "of bfloat16"),
    ({"q": torch.zeros((4, 255), dtype=torch.uint8)}, "1024 elements or more of uint8"),
    ({"q": torch.zeros((4, 256), dtype=torch.bfloat16)}, "of uint8"),
    ({"q": torch.zeros((0, 256), dtype=torch.uint8)}, "of uint8"),
    ({"s": torch.zeros((4, 1))}, "8 elements or more of float32"),
    ({"s": torch.zeros((4, 2), dtype=torch.float64)}, "of float32"),
    ({"s": torch.zeros((8,), dtype=torch.bfloat16)}, "of float32")])
def test_row_quantiser_checks_types_and_room(M, change, want):
    """A buffer that is too small would be written past its end on the device, values of
    another type read as bf16 bits."""
    a = {"x": torch.zeros((4, 256), dtype=torch.bfloat16), "q": torch.zeros((4, 256), dtype=torch.uint8),
         "s": torch.zeros((4, 2)), **change}
    with pytest.raises(ValueError, match=want):
        M._native.quantize_act_fp8(0, 0, a["x"], a["q"], a["s"])


def test_row_quantiser_takes_empty_tensors_of_any_device(M):
    """No rows: nothing is read or written, so nothing is asked of the buffers."""
    q, s = torch.zeros((0, 256), dtype=torch.uint8), torch.zeros((0, 2))
    for x in (torch.zeros((0, 256), dtype=torch.bfloat16), torch.zeros((0, 256), dtype=torch.int16)):
        assert M._native.quantize_act_fp8(0, 0, x, q, s) == M.OK
        assert M._native.quantize_act_fp8(-1, 0, x, None, None) == M.OK
        assert M._native.quantize_act_fp8(-1, 0, x, torch.zeros(9, dtype=torch.uint8), torch.zeros(9)) == M.OK
        M.quantize_act_fp8(x, q, s, stream=0)


def test_row_quantiser_refuses_memory_that_the_device_does_not_reach(M):
    x, q, s = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2))
    assert M._lib.moe_device_address(x.data_ptr()) is None
    with pytest.raises(ValueError, match="reaches"):
        M.quantize_act_fp8(x, q, s, stream=0)


def test_a_call_lets_other_threads_run(tmp_path):
    got = binding_stub.run(str(tmp_path), """
call("quantize_act_fp8", 0, 0, torch.zeros((0, 128), dtype=torch.bfloat16), None, None)
""")
    assert got == {"quantize_act_fp8": 0}


@pytest.mark.parametrize("make", [lambda *s: torch._neg_view(torch.ones(s)),
                                  lambda *s: torch._efficientzerotensor(s)], ids=["negated", "zero"])
def test_tensors_whose_memory_does_not_hold_their_values_are_refused(M, make):
    """The imaginary part of a conjugate is such a negated view; a mask of such zeros would
    come without an address, as if there were no mask."""
    n, z = M._native, torch.zeros
    ids, i = z((4, 2), dtype=torch.int32), z(8, dtype=torch.int32)
    assert torch.ones((1, 1), dtype=torch.complex64).conj().imag.is_neg()
    with pytest.raises(ValueError, match="logits: a negated view or a zero"):
        n.balance_loss(0, 0, make(4, 8), ids, None, 0.1, z(1), i, z(8), z(1), z(256))
    with pytest.raises(ValueError, match="logits: a negated view or a zero"):
        n.route_backward(0, 0, make(4, 8), ids, None, None, None, True, z(1), 0.1, i, i, z(4, 8))
    with pytest.raises(ValueError, match="x: a negated view or a zero"):
        n.quantize_act_fp8(0, 0, make(4, 128), z(4, 128, dtype=torch.uint8), z(4, 1))
    with pytest.raises(ValueError, match="x: a negated view or a zero"):
        n.quantize_fp8_tokens(0, 0, make(4, 128), None, z(128, 128), z(1, 128))
    with pytest.raises(ValueError, match="dw: a negated view or a zero"):
        n.gemm_fp8_wgrad(0, 0, i, i, i, i, None, 4, make(128, 128), False, z(256))


def test_another_torch_does_not_load_the_binding():
    """The binding is compiled against one torch; under another the training calls raise, and
    what does not need it works, the row quantiser with the same checks."""
    code = """
import torch
torch.__version__ = "0.0.1"
import expert_layer_dual_b200.moe as M
z = torch.zeros
bf, u8 = torch.bfloat16, torch.uint8
assert M.workspace_bytes(M.moe_shape(4, 256, 8, 2, 128, 0, 0, 1)) > 0 and M.fp8_token_rows(5) == 128
assert not hasattr(M._native, "__wrapped__")  # as inspect and doctest ask
try:
    M._native.gemm_fp8(0, 0, *[z(1)] * 7)
except ImportError as e:
    assert "torch-0.0.1" in str(e) and "expert_layer_dual_b200.build" in str(e), e
else:
    raise AssertionError("loaded")
M.quantize_act_fp8(z((0, 256), dtype=bf), z((0, 256), dtype=u8), z((0, 2)), stream=0)
M.quantize_act_fp8(z((0, 256), dtype=bf), None, None, stream=0)
x, q, s = z((4, 256), dtype=bf), z((4, 256), dtype=u8), z((4, 2))
for bad, name in (((x.half(), q, s), "x"), ((x, q[:3], s), "codes"), ((x, q, s.double()), "scales"), ((x, q, s), "x")):
    try:
        M.quantize_act_fp8(*bad, stream=0)
    except ValueError as e:
        assert str(e).startswith(name), e
    else:
        raise AssertionError(name)
print("fine")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
