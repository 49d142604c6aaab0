"""The training entry points' calls on the GPU: memory of several kinds, and what the native
binding does around a call."""
import pytest
import torch

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
