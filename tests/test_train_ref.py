"""The 64-bit formulas of the training operators against differences, and the
host-side refusals of their entry points (no GPU)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import train_ref as ref


def forward64(l, ids, w_of, dw, dloss, coef, counts, n):
    """dloss * balance loss + <dw, w> as a function of the logits, counts fixed."""
    P = ref.softmax64(l)
    f = counts.double() * l.shape[1] / (ids.shape[1] * n)
    return float(dloss * coef * (f * P.mean(0)).sum() + (dw * w_of(l, P)).sum())


@pytest.mark.parametrize("renorm", [True, False])
def test_logit_gradient_against_differences(renorm):
    T, E, k = 6, 9, 3
    g = torch.Generator().manual_seed(3)
    l = torch.randn((T, E), generator=g, dtype=torch.float64)
    ids = torch.topk(l, k, dim=1).indices.int()
    dw = torch.randn((T, k), generator=g, dtype=torch.float64)
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E)

    def w_of(l, P):
        top = P.gather(1, ids.long())
        return top / top.sum(1, keepdim=True) if renorm else top

    w = w_of(l, ref.softmax64(l))
    d, size = ref.route_backward(l, ids, w, dw, None, renorm, 1.3, 0.4, counts, T)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            ends = []
            for s in (h, -h):
                m = l.clone()
                m[t, e] += s
                ends.append(forward64(m, ids, w_of, dw, 1.3, 0.4, counts, T))
            # truncation h^2, rounding 2^-52 * |value| / h
            assert abs((ends[0] - ends[1]) / (2 * h) - float(d[t, e])) < 1e-8
    assert bool((size >= d.abs() - 1e-15).all())


def test_block_quantisation_round_trip():
    g = torch.Generator().manual_seed(4)
    x = torch.randn((5, 256), generator=g).to(torch.bfloat16)
    x[2, :128] = 0
    q, s = ref.quantise_rows(x)
    assert float(s[2, 0]) == 1.0 and bool((q[2, :128] == 0).all())
    err = (ref.rows64(q, s) - x.double()).abs().reshape(5, 2, 128)
    # half an e4m3 step (2^-4 relative) plus the subnormal step 2^-10 of the scale
    assert bool((err <= 2.0 ** -4 * x.double().abs().reshape(5, 2, 128) + 2.0 ** -10 * s.double()[:, :, None]
                 + 1e-12).all())
    w = torch.randn((2, 256, 128), generator=g).to(torch.bfloat16)
    q, s = ref.quantise_weights(w)
    assert q.shape == w.shape and s.shape == (2, 2, 1)
    assert float((ref.weights64(q, s) - w.double()).abs().max()) <= 2.0 ** -4 * float(w.abs().max())


def test_token_layout_and_adjoints():
    """Padding and order of the token-block layout, and <dy, x W^T> = <dy W, x> =
    <dy^T x, W> on the values that the codes stand for."""
    g = torch.Generator().manual_seed(5)
    M, N, K = 200, 128, 256
    off = torch.tensor([0, 130, 130, 200], dtype=torch.int32)
    x = torch.randn((M, K), generator=g).to(torch.bfloat16)
    q, s, blocks = ref.quantise_tokens(x, off, 512)
    assert blocks == 3
    assert bool((q[:, 130:256] == 0).all()) and bool((q[:, 256 + 70: 384] == 0).all())
    dy64 = torch.randn((M, N), generator=g, dtype=torch.float64)
    x64 = torch.randn((M, K), generator=g, dtype=torch.float64)
    w64 = torch.randn((3, N, K), generator=g, dtype=torch.float64)
    y, _, cov = ref.grouped(x64, w64, off, M, True)
    dx, _, _ = ref.grouped(dy64, w64, off, M, False)
    assert bool(cov.all())
    dw = torch.stack([dy64[a:b].T @ x64[a:b] for a, b in ((0, 130), (130, 130), (130, 200))])
    a, b, c = (dy64 * y).sum(), (dx * x64).sum(), (dw * w64).sum()
    assert abs(a - b) < 1e-9 * abs(a) + 1e-8 and abs(a - c) < 1e-9 * abs(a) + 1e-8


def _rn(x):
    """A positive fraction rounded to FP32 (nearest, ties to even; normal range)."""
    f = np.float32(float(x))
    near = [np.nextafter(f, np.float32(0)), f, np.nextafter(f, np.float32(np.inf))]
    return min(near, key=lambda c: (abs(Fraction(float(c)) - x), int(c.view(np.uint32)) & 1))


def test_corrected_quotient_is_the_rounded_one():
    """The quantisers' quotient: the product with the reciprocal, corrected by one
    FMA residual, equals fp32(v / s) for every bf16 significand v and the scale s =
    fp32(b / 448) of every bf16 significand b, with the reciprocal one ulp off
    either way too; and s itself comes out of the same correction."""
    def corrected(v, r, s):
        q = _rn(Fraction(v) * Fraction(float(r)))
        e = Fraction(v) - Fraction(float(q)) * s
        e32 = Fraction(float(_rn(abs(e)))) * (1 if e > 0 else -1) if e else e
        return _rn(e32 * Fraction(float(r)) + Fraction(float(q)))

    for b in range(128, 256):
        s = _rn(Fraction(b, 448))
        assert corrected(b, _rn(Fraction(1, 448)), Fraction(448)) == s
        r0 = _rn(1 / Fraction(float(s)))
        for r in (np.nextafter(r0, np.float32(0)), r0, np.nextafter(r0, np.float32(np.inf))):
            for v in range(128, 256):
                assert corrected(v, r, Fraction(float(s))) == _rn(Fraction(v) / Fraction(float(s)))


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def M():
    from expert_layer_dual_b200 import build
    build.build()
    from expert_layer_dual_b200 import moe
    return moe


P = ctypes.c_void_p
OKP = 1 << 20          # an aligned address; nothing is launched without a device


def test_sizes(M):
    assert M.balance_workspace_bytes(64, 256) == 256
    assert M.balance_workspace_bytes(1 << 20, 256) >= 256 + 296 * 256 * 8
    assert M.balance_workspace_bytes(-1, 256) == 0 and M.balance_workspace_bytes(4, 257) == 0
    assert M.balance_workspace_bytes(4, 0) == 0
    assert [M.fp8_token_rows(*a) for a in ((0, 1), (1, 1), (128, 1), (129, 1), (300, 4), (3, 256))] == \
        [0, 128, 128, 256, 768, 384]
    assert M.fp8_token_rows(-1, 1) == 0 and M.fp8_token_rows(5, 0) == 0


@pytest.mark.parametrize("change,code", [
    ({"T": -1}, 1), ({"E": 0}, 1), ({"k": 0}, 1), ({"E": 257}, 2), ({"k": 9}, 2), ({"E": 4, "k": 5}, 2),
    ({"T": 1 << 30}, 2), ({"logits": None}, 1), ({"ids": None}, 1), ({"loss": None}, 1),
    ({"counts": None}, 1), ({"prob_mean": None}, 1), ({"tokens": None}, 1), ({"logits": OKP + 4}, 1),
    ({"ws": None}, 1), ({"ws": OKP + 16}, 1), ({"ws_bytes": 255}, 4)])
def test_balance_refusals(M, change, code):
    a = {"logits": OKP, "ids": OKP, "mask": None, "T": 64, "E": 8, "k": 2, "coef": 0.1, "loss": OKP,
         "counts": OKP, "prob_mean": OKP, "tokens": OKP, "ws": OKP, "ws_bytes": 256, **change}
    assert M._lib.moe_balance_loss(
        P(a["logits"]), P(a["ids"]), P(a["mask"]), a["T"], a["E"], a["k"], a["coef"], P(a["loss"]),
        P(a["counts"]), P(a["prob_mean"]), P(a["tokens"]), P(a["ws"]), a["ws_bytes"], None) == code


@pytest.mark.parametrize("change,code", [
    ({"T": -1}, 1), ({"T": 0}, 0), ({"E": 300}, 2), ({"k": 9}, 2), ({"dw": None, "dloss": None}, 1),
    ({"ids": None}, 1), ({"w": None}, 1), ({"counts": None}, 1), ({"tokens": None}, 1),
    ({"logits": None}, 1), ({"dlogits": None}, 1), ({"logits": OKP + 8}, 1), ({"dlogits": OKP + 8}, 1)])
def test_route_backward_refusals(M, change, code):
    a = {"logits": OKP, "ids": OKP, "w": OKP, "dw": OKP, "T": 4, "E": 8, "k": 2, "dloss": OKP,
         "counts": OKP, "tokens": OKP, "dlogits": OKP, **change}
    assert M._lib.moe_route_backward(
        P(a["logits"]), P(a["ids"]), P(a["w"]), P(a["dw"]), None, a["T"], a["E"], a["k"], 1,
        P(a["dloss"]), 0.1, P(a["counts"]), P(a["tokens"]), P(a["dlogits"]), None) == code


@pytest.mark.parametrize("entry", ["moe_gemm_fp8", "moe_gemm_fp8_dgrad"])
@pytest.mark.parametrize("change,code", [
    ({"M": -1}, 1), ({"M": 0, "a": None}, 0), ({"G": 0}, 1), ({"G": 2}, 1), ({"G": 257, "off": OKP}, 2),
    ({"N": 0}, 1), ({"N": 200}, 2), ({"K": 64}, 2), ({"G": 256, "off": OKP, "N": 1 << 23}, 2),
    ({"a": None}, 1), ({"a_s": None}, 1), ({"w": None}, 1), ({"w_s": None}, 1), ({"out": None}, 1),
    ({"a": OKP + 8}, 1), ({"w": OKP + 8}, 1), ({"out": OKP + 8}, 1), ({"type": 3}, 2), ({"type": -1}, 2),
    ({"ws": None}, 1), ({"ws": OKP + 32}, 1), ({"ws_bytes": 8}, 4)])
def test_product_refusals(M, entry, change, code):
    a = {"a": OKP, "a_s": OKP, "w": OKP, "w_s": OKP, "off": None, "G": 1, "M": 5, "N": 256, "K": 128,
         "out": OKP, "type": 0, "ws": OKP, "ws_bytes": 256, **change}
    assert getattr(M._lib, entry)(
        P(a["a"]), P(a["a_s"]), P(a["w"]), P(a["w_s"]), P(a["off"]), a["G"], a["M"], a["N"], a["K"],
        P(a["out"]), a["type"], P(a["ws"]), a["ws_bytes"], None) == code


@pytest.mark.parametrize("change,code", [
    ({"M": -1}, 1), ({"G": 3}, 1), ({"N": 130}, 2), ({"K": 130}, 2), ({"dw": None}, 1), ({"dw": OKP + 4}, 1),
    ({"a": None}, 1), ({"a_s": None}, 1), ({"b": None}, 1), ({"b_s": None}, 1), ({"a": OKP + 1}, 1),
    ({"b": OKP + 2}, 1), ({"ws": None}, 1), ({"ws_bytes": 0}, 4), ({"M": 9000000}, 2)])
def test_weight_gradient_refusals(M, change, code):
    a = {"a": OKP, "a_s": OKP, "b": OKP, "b_s": OKP, "off": None, "G": 1, "M": 5, "N": 256, "K": 128,
         "dw": OKP, "ws": OKP, "ws_bytes": 256, **change}
    assert M._lib.moe_gemm_fp8_wgrad(
        P(a["a"]), P(a["a_s"]), P(a["b"]), P(a["b_s"]), P(a["off"]), a["G"], a["M"], a["N"], a["K"],
        P(a["dw"]), 0, P(a["ws"]), a["ws_bytes"], None) == code


@pytest.mark.parametrize("change,code", [
    ({"M": -1}, 1), ({"M": 0, "x": None}, 0), ({"G": 2}, 1), ({"cols": 100}, 2), ({"x": None}, 1),
    ({"q": None}, 1), ({"s": None}, 1), ({"x": OKP + 2}, 1), ({"q": OKP + 4}, 1), ({"M": 9000000}, 2)])
def test_token_quantiser_refusals(M, change, code):
    a = {"x": OKP, "off": None, "G": 1, "M": 5, "cols": 128, "q": OKP, "s": OKP, **change}
    assert M._lib.moe_quantize_fp8_tokens(P(a["x"]), P(a["off"]), a["G"], a["M"], a["cols"], P(a["q"]),
                                          P(a["s"]), None) == code


def test_binding_refuses_tensors_off_the_current_device(M):
    t = torch.zeros((4, 128), dtype=torch.uint8)
    s = torch.zeros((4, 1))
    with pytest.raises(ValueError, match="current CUDA device"):
        M.gemm_fp8(t, s, torch.zeros((128, 128), dtype=torch.uint8), torch.zeros((1, 1)), None,
                   torch.zeros((4, 128)), torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="current CUDA device"):
        M.balance_loss(s, t, None, 0.1, s, t, s, t, t)


def test_native_binding_checks_before_it_calls(M):
    """The native layer itself (device 0, stream 0): nothing is launched for
    tensors elsewhere, of another rank, or that are no tensors."""
    n = M._native
    t, s = torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((4, 1))
    w, ws = torch.zeros((128, 128), dtype=torch.uint8), torch.zeros((1, 1))
    for f in (n.gemm_fp8, n.gemm_fp8_dgrad):
        with pytest.raises(ValueError, match="current CUDA device"):
            f(0, 0, t, s, w, ws, None, s, t)
        with pytest.raises(ValueError, match="a matrix"):
            f(0, 0, t[0], s, w, ws, None, s, t)
        with pytest.raises(ValueError, match="not a tensor"):
            f(0, 0, t, s, None, ws, None, s, t)
        with pytest.raises(ValueError, match="offsets"):
            f(0, 0, t, s, torch.zeros((2, 128, 128), dtype=torch.uint8), ws, None, s, t)
        with pytest.raises(TypeError):
            f(0, 0, t)
    with pytest.raises(ValueError):
        n.quantize_act_fp8(0, 0, torch.zeros((4, 128)).to_sparse(), t, s)
    with pytest.raises(ValueError):
        n.quantize_fp8_tokens(0, 0, torch.zeros((4, 128), device="meta"), None, t, s)
    with pytest.raises(ValueError):
        n.route_backward(0, 0, s, t, None, None, None, True, s, 0.1, t, t, s)
    with pytest.raises(ValueError):
        n.gemm_fp8_wgrad(0, 0, t, s, t, s, None, 4, w, False, t)
    with pytest.raises(TypeError):
        n.gemm_fp8_wgrad(0, 0, t, s, t, s, None, "4", w, False, t)
