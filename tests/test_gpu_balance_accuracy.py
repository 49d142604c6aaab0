"""How far the balance loss and the gradient of the router logits may be off: many rows, and
logits of a wide spread.

Bounds, from the arithmetic, in steps of u = 2^-24, S the largest max - l of a row:
  - the exponential is the hardware's exp2 (4 u) of (l - m) log2(e), whose difference,
    product and constant round by u, u and u / 4: relative ln 2 * 2.25 S log2(e) u = 2.25 S u;
  - the row's sum has terms as far off, and 15 + 4 additions; its reciprocal and the
    product with it round by u each: a probability is within (4.5 S + 29) u;
  - at most 64 rows of a lane, two lanes and a block's 16 warps are added in FP32 (64 + 1 +
    16 u; or 2 + 1 + 32 u in one block); what a lane's further rows round away is kept; the
    mean (u), the loss (u) and its coefficient (u) are rounded once, all other sums are in
    FP64: the means and the loss are within (4.5 S + 113) u, for any number of rows;
  - a term of the gradient is a product of a probability with f - 1 (3 u), dloss coef / n (3 u)
    and, in the second term, the row's sum of (f - 1) P (as far off as a probability, f - 1,
    and 16 + 4 additions), in at most 6 more roundings: (9 S + 93) u of the terms' magnitudes.
What lies below 2^-126 is flushed to zero."""
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expert_layer_dual_b200.moe as M

DEV = "cuda"
U = 2.0 ** -24
TINY = 2.0 ** -125


def balance(logits, ids, mask, coef):
    T, E = logits.shape
    o = {"loss": torch.empty(1, device=DEV), "counts": torch.empty(E, dtype=torch.int32, device=DEV),
         "prob_mean": torch.empty(E, device=DEV), "tokens": torch.empty(1, dtype=torch.int32, device=DEV)}
    ws = torch.empty(M.balance_workspace_bytes(T, E), dtype=torch.uint8, device=DEV)
    M.balance_loss(logits, ids, mask, coef, o["loss"], o["counts"], o["prob_mean"], o["tokens"], ws)
    assert M.read_device_status(ws) == M.OK
    return o


@pytest.mark.parametrize("E", [5, 9])
def test_error_of_the_means_does_not_grow_with_the_rows(E):
    """Equal rows, whose roundings all go one way: 1200 of them a lane.  Added up in FP32
    alone, the means were 1.0e-5 (E = 5) and 1.4e-5 (E = 9) off."""
    T = 1200 * 296 * 32
    logits = torch.zeros((T, E), device=DEV)
    ids = (torch.arange(T, device=DEV, dtype=torch.int32) * 7 % E).view(T, 1)
    o = balance(logits, ids, None, 0.5)
    assert int(o["tokens"]) == T
    assert torch.equal(o["counts"].long(), torch.bincount(ids.view(-1), minlength=E))
    err = (o["prob_mean"].double() * E - 1).abs().max()
    assert float(err) <= 113 * U, float(err)
    assert abs(float(o["loss"]) / 0.5 - 1) <= 113 * U


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", [(400003, 4, 2), (606208, 2, 1), (606209, 2, 1), (700000, 7, 3), (1300003, 65, 2)])
def test_many_rows_of_few_experts(T, E, k, masked):
    g = torch.Generator().manual_seed(T)
    logits = torch.randn((T, E), generator=g) * 3.0
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    mask = (torch.rand(T, generator=g) < 0.9) if masked else None
    r = ref.balance(logits, ids, None if mask is None else mask.to(torch.uint8), 0.02)
    o = balance(logits.to(DEV), ids.to(DEV), None if mask is None else mask.to(DEV), 0.02)
    S = float((logits.amax(1, keepdim=True) - logits).max())
    bound = (4.5 * S + 113) * U
    assert torch.equal(o["counts"].cpu().long(), r["counts"].long()) and int(o["tokens"]) == r["tokens"]
    got = o["prob_mean"].cpu().double()
    assert bool(((got - r["prob_mean"]).abs() <= bound * r["prob_mean"]).all())
    assert abs(float(o["loss"]) - r["loss"]) <= bound * abs(r["loss"])


@pytest.mark.parametrize("S", [1.0, 30.0, 60.0, 85.0, 120.0, 3.0e4])
@pytest.mark.parametrize("T,E,k", [(100, 256, 8), (1000, 60, 4)])
@pytest.mark.parametrize("renorm", [True, False])
def test_spread(T, E, k, renorm, S):
    """Logits from m - S to m, m itself large or small."""
    g = torch.Generator().manual_seed(int(S) + T)
    logits = -S * torch.rand((T, E), generator=g)
    logits[:, 0] = 0.0
    logits[:, 1] = -S
    logits += torch.tensor([-2.0, 0.0, 3.0, 40.0])[torch.arange(T) % 4].view(T, 1)
    S = float((logits.amax(1, keepdim=True).double() - logits.double()).max())
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    top = logits.gather(1, ids.long()).double()
    base = top if renorm else logits.double()
    w = (torch.exp(top - base.amax(1, keepdim=True)) / torch.exp(base - base.amax(1, keepdim=True)).sum(1, keepdim=True))
    w = w.float()
    r = ref.balance(logits, ids, None, 0.02)
    o = balance(logits.to(DEV), ids.to(DEV), None, 0.02)
    bound = (4.5 * S + 113) * U
    got = o["prob_mean"].cpu().double()
    assert bool(((got - r["prob_mean"]).abs() <= bound * r["prob_mean"] + TINY).all())
    assert abs(float(o["loss"]) - r["loss"]) <= bound * abs(r["loss"])
    dw = torch.randn((T, k), generator=g)
    dloss = torch.tensor([0.7])
    for parts in ((dw, None), (None, dloss), (dw, dloss)):
        d, size = ref.route_backward(logits, ids, w, parts[0], None, renorm, parts[1], 0.02, r["counts"], r["tokens"])
        out = torch.empty((T, E), device=DEV)
        M.route_backward(logits.to(DEV), ids.to(DEV), w.to(DEV), None if parts[0] is None else dw.to(DEV), None, renorm,
                         None if parts[1] is None else dloss.to(DEV), 0.02, o["counts"], o["tokens"], out)
        err = (out.cpu().double() - d).abs() - (9 * S + 93) * U * size - TINY * 8
        assert bool((err <= 0).all()), float(err.max())
