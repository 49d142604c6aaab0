"""The training entry points' calls on the GPU: memory of several kinds, and what the native
binding does around a call."""
import pytest
import torch

import binding_stub
import train_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expert_layer_dual_b200.moe as M

DEV = "cuda"


@pytest.mark.parametrize("pinned", ["x", "q", "s", "xqs"])
def test_row_quantiser_on_pinned_host_memory(pinned):
    x = torch.randn((37, 384), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    q, s = ref.quantise_rows(x)
    buf = {"x": x, "q": torch.zeros((37, 384), dtype=torch.uint8), "s": torch.zeros((37, 3))}
    buf = {n: t.pin_memory() if n in pinned else t.to(DEV) for n, t in buf.items()}
    M.quantize_act_fp8(buf["x"], buf["q"], buf["s"])
    torch.cuda.synchronize()
    assert torch.equal(buf["q"].cpu(), q) and torch.equal(buf["s"].cpu(), s)


def test_row_quantiser_refuses_pageable_memory():
    x, q, s = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2))
    for cpu in range(3):
        with pytest.raises(ValueError, match="reaches"):
            M.quantize_act_fp8(*[t if i == cpu else t.to(DEV) for i, t in enumerate((x, q, s))])


def test_row_quantiser_on_larger_buffers_of_another_shape():
    x = torch.randn((5, 256), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    q, s = ref.quantise_rows(x)
    gq, gs = torch.full((2000,), 9, dtype=torch.int8, device=DEV), torch.full((4, 5), 9.0, device=DEV)
    M.quantize_act_fp8(x.to(DEV).view(torch.int16), gq, gs)
    assert torch.equal(gq[:1280].view(torch.uint8).view(5, 256).cpu(), q) and bool((gq[1280:] == 9).all())
    assert torch.equal(gs.view(-1)[:10].view(5, 2).cpu(), s) and bool((gs.view(-1)[10:] == 9.0).all())


def test_every_call_lets_other_threads_run(tmp_path):
    """A launch waits while the stream's queue is full; the interpreter lock held meanwhile
    would stop the Python callback that could empty it."""
    got = binding_stub.run(str(tmp_path), """
z = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t, device="cuda")
f, i, b = torch.float32, torch.int32, torch.bfloat16
logits, ids, w, ws = z(8, 16, t=f), z(8, 2, t=i), z(8, 2, t=f), z(256)
one, n, counts = z(1, t=f), z(1, t=i), z(16, t=i)
call("balance_loss", 0, 0, logits, ids, None, 0.1, one, counts, z(16, t=f), n, ws)
call("route_backward", 0, 0, logits, ids, w, w, None, True, one, 0.1, counts, n, z(8, 16, t=f))
a, s, m, ms = z(8, 128), z(8, 1, t=f), z(128, 128), z(1, 1, t=f)
call("gemm_fp8", 0, 0, a, s, m, ms, None, z(8, 128, t=b), ws)
call("gemm_fp8_dgrad", 0, 0, a, s, m, ms, None, z(8, 128, t=b), ws)
call("quantize_act_fp8", 0, 0, z(8, 128, t=b), a, s)
call("quantize_fp8_tokens", 0, 0, z(8, 128, t=b), None, m, z(1, 128, t=f))
call("gemm_fp8_wgrad", 0, 0, m, z(1, 128, t=f), m, z(1, 128, t=f), None, 8, z(128, 128, t=f), False, ws)
""")
    assert got == {e.removeprefix("moe_"): 0 for e in binding_stub.ENTRIES}


def _calls():
    """{entry: (function, its outputs by name)}: each with small inputs."""
    f, i, b = torch.float32, torch.int32, torch.bfloat16
    z = lambda *s, t=torch.uint8: torch.full(s, 1, dtype=t, device=DEV)  # noqa: E731
    ws = z(256)
    logits, ids, w, one, n, counts = z(8, 16, t=f), z(8, 2, t=i), z(8, 2, t=f), z(1, t=f), z(1, t=i), z(16, t=i)
    a, s, m, ms, x, t = z(8, 128), z(8, 1, t=f), z(128, 128), z(1, 1, t=f), z(8, 128, t=b), z(1, 128, t=f)
    return {
        "balance_loss": (lambda loss, counts, mean, tokens, ws: M.balance_loss(
            logits, ids, None, 0.1, loss, counts, mean, tokens, ws),
            {"loss": (1, f), "counts": (16, i), "mean": (16, f), "tokens": (1, i), "ws": (256, torch.uint8)}),
        "route_backward": (lambda dlogits: M.route_backward(
            logits, ids, w, w, None, True, one, 0.1, counts, n, dlogits), {"dlogits": ((8, 16), f)}),
        "gemm_fp8": (lambda y, ws: M.gemm_fp8(a, s, m, ms, None, y, ws),
                     {"y": ((8, 128), b), "ws": (256, torch.uint8)}),
        "gemm_fp8_dgrad": (lambda y: M.gemm_fp8_dgrad(a, s, m, ms, None, y, ws), {"y": ((8, 128), f)}),
        "quantize_act_fp8": (lambda q, s: M.quantize_act_fp8(x, q, s), {"q": ((8, 128), torch.uint8), "s": ((8, 1), f)}),
        "quantize_fp8_tokens": (lambda q, s: M.quantize_fp8_tokens(x, None, q, s),
                                {"q": ((128, 128), torch.uint8), "s": ((1, 128), f)}),
        "gemm_fp8_wgrad": (lambda dw: M.gemm_fp8_wgrad(m, t, m, t, None, 8, dw, True, ws), {"dw": ((128, 128), f)}),
    }


@pytest.mark.parametrize("entry", ["balance_loss", "route_backward", "gemm_fp8", "gemm_fp8_dgrad", "quantize_act_fp8",
                                   "quantize_fp8_tokens", "gemm_fp8_wgrad"])
def test_outputs_that_are_lazily_cloned_get_storage_of_their_own(entry):
    """What a lazy clone shares with its source until it is written stays as it was."""
    call, outputs = _calls()[entry]
    plain = {n: torch.full(s if isinstance(s, tuple) else (s,), 5, dtype=t, device=DEV) for n, (s, t) in outputs.items()}
    source = {n: t.clone() for n, t in plain.items()}
    cloned = {n: torch._lazy_clone(t) for n, t in source.items()}
    call(**plain)
    call(**cloned)
    for n, t in cloned.items():
        assert bool((source[n] == 5).all()), f"{n}: the source was written"
        assert torch.equal(t, plain[n]), n


def test_row_quantiser_without_the_binding(monkeypatch):
    """The same call, the same kernel, through ctypes."""
    x = torch.randn((37, 384), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    want = ref.quantise_rows(x)
    monkeypatch.setattr(M, "_native", M._NoBinding("none"))
    for place in (lambda t: t.to(DEV), lambda t: t.pin_memory()):
        q, s = place(torch.zeros((37, 384), dtype=torch.uint8)), place(torch.zeros((37, 3)))
        M.quantize_act_fp8(place(x), q, s)
        torch.cuda.synchronize()
        assert torch.equal(q.cpu(), want[0]) and torch.equal(s.cpu(), want[1])
    with pytest.raises(ImportError):
        M.gemm_fp8(q.to(DEV), s.to(DEV), q.to(DEV), s.to(DEV), None, q.to(DEV), q.to(DEV))


@pytest.mark.parametrize("shape", [(1, 128), (3, 128), (4097, 128), (60001, 128), (30001, 384), (12001, 640), (7001, 1152)],
                         ids=lambda s: "x".join(map(str, s)))
def test_row_quantiser_on_short_rows(shape):
    """Groups of neighbouring rows share a warp; their number need not be even."""
    x = (torch.randn(shape, generator=torch.Generator().manual_seed(shape[0])) * 3).to(torch.bfloat16)
    want = ref.quantise_rows(x)
    q, s = torch.full(shape, 9, dtype=torch.uint8, device=DEV), torch.full((shape[0], shape[1] // 128), 9.0, device=DEV)
    M.quantize_act_fp8(x.to(DEV), q, s)
    assert torch.equal(q.cpu(), want[0]) and torch.equal(s.cpu(), want[1])
