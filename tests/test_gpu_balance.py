"""The balance loss, its counts and the gradient of the router logits against
their formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24):
  - counts, tokens: exact;
  - a softmax value: the argument l - m rounds by |l - m| u, expf by 2 ulp (4 u),
    the row sum by 13 additions, the reciprocal and its product by 2 u more;
    the sums over a warp's rows and a block's warps add at most one u per row
    and warp.  With |l - m| <= 40 and at most 64 rows and 32 warps:
    relative 160 u < 1e-5;
  - dlogits: each term is a product of at most six rounded factors with such a
    softmax value: 1e-5 of the sum of the terms' magnitudes."""
import numpy as np
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expert_layer_dual_b200.moe as M

DEV = "cuda"
TOL = 1e-5


def make(T, E, k, seed, renorm=True, mask=None, weights=True, loss=True):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((T, E), generator=g) * 3.0
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32) if T else torch.zeros((0, k), dtype=torch.int32)
    base = logits.gather(1, ids.long()) if renorm else logits
    top = logits.gather(1, ids.long())
    w = (torch.exp(top - base.amax(1, keepdim=True)) / torch.exp(base - base.amax(1, keepdim=True))
         .sum(1, keepdim=True)) if T else torch.zeros((0, k))
    keep = None
    if mask is not None:
        keep = (torch.rand(T, generator=g) < mask).to(torch.uint8)
    dw = torch.randn((T, k), generator=g) if weights else None
    return {"logits": logits, "ids": ids, "w": w, "dw": dw, "mask": keep, "renorm": renorm,
            "dloss": torch.tensor([0.7]) if loss else None, "coef": 0.02}


def dev(t):
    return None if t is None else t.to(DEV)


def outputs(T, E):
    return {"loss": torch.full((1,), 9.0, device=DEV),
            "counts": torch.full((E,), 9, dtype=torch.int32, device=DEV),
            "prob_mean": torch.full((E,), 9.0, device=DEV),
            "tokens": torch.full((1,), 9, dtype=torch.int32, device=DEV),
            "dlogits": torch.full((T, E), 9.0, device=DEV),
            "ws": torch.empty(M.balance_workspace_bytes(T, E), dtype=torch.uint8, device=DEV)}


def run(c, o, stream=None):
    M.balance_loss(c["logits"], c["ids"], c["mask"], c["coef"], o["loss"], o["counts"], o["prob_mean"],
                   o["tokens"], o["ws"], stream)
    M.route_backward(c["logits"], c["ids"], c["w"], c["dw"], c["mask"], c["renorm"], c["dloss"],
                     c["coef"], o["counts"], o["tokens"], o["dlogits"], stream)


def check(c, o):
    r = ref.balance(c["logits"], c["ids"], c["mask"], c["coef"])
    assert np.array_equal(o["counts"].cpu().numpy(), r["counts"].numpy())
    assert int(o["tokens"].cpu()) == r["tokens"]
    got = o["prob_mean"].cpu().double()
    assert bool((abs(got - r["prob_mean"]) <= TOL * r["prob_mean"] + 1e-37).all())
    assert abs(float(o["loss"].cpu()) - r["loss"]) <= TOL * abs(r["loss"])
    d, size = ref.route_backward(c["logits"], c["ids"], c["w"], c["dw"], c["mask"], c["renorm"],
                                 c["dloss"], c["coef"], r["counts"], r["tokens"])
    err = (o["dlogits"].cpu().double() - d).abs()
    assert bool((err <= TOL * size + 1e-37).all()), float((err - TOL * size).max())


CASES = [
    dict(T=1, E=2, k=1), dict(T=1, E=256, k=8), dict(T=2, E=1, k=1), dict(T=7, E=8, k=8),
    dict(T=64, E=256, k=8), dict(T=100, E=60, k=4), dict(T=513, E=255, k=3), dict(T=511, E=33, k=5),
    dict(T=512, E=128, k=8), dict(T=2000, E=256, k=8), dict(T=3001, E=4, k=2), dict(T=5000, E=129, k=7),
    dict(T=20011, E=64, k=6), dict(T=4100, E=160, k=6), dict(T=9473, E=192, k=8), dict(T=9600, E=193, k=8),
    dict(T=129, E=130, k=2),
]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("mask", [None, 0.8, 0.0])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_against_formula(case, mask, renorm):
    c = make(seed=case["T"] * 31 + case["E"], renorm=renorm, mask=mask, **case)
    o = outputs(case["T"], case["E"])
    g = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    run(g, o)
    torch.cuda.synchronize()
    check(c, o)
    assert M.read_device_status(o["ws"]) == M.OK


@pytest.mark.parametrize("T,E,k", [(37, 256, 8), (5003, 60, 4), (9500, 129, 7)])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_in_place(T, E, k, renorm):
    """dlogits may be the logits' own buffer: the same bits as into another one."""
    c = {n: dev(v) if isinstance(v, torch.Tensor) else v for n, v in make(T, E, k, T, renorm, 0.8).items()}
    o = outputs(T, E)
    run(c, o)
    apart = o["dlogits"].clone()
    o["dlogits"] = c["logits"]
    run(c, o)
    assert torch.equal(c["logits"], apart)


@pytest.mark.parametrize("weights,loss", [(True, False), (False, True)])
@pytest.mark.parametrize("renorm", [True, False])
def test_one_part_alone(weights, loss, renorm):
    c = make(700, 96, 4, seed=5, renorm=renorm, weights=weights, loss=loss)
    o = outputs(700, 96)
    run({k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}, o)
    check(c, o)


@pytest.mark.parametrize("T", [40, 900])
def test_masked_rows_are_not_read(T):
    c = make(T, 40, 4, seed=11, mask=0.5)
    bad = c["mask"] == 0
    clean = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    o1 = outputs(T, 40)
    run(clean, o1)
    dirty = dict(clean)
    for name, val in (("logits", float("nan")), ("w", float("inf")), ("dw", float("nan"))):
        t = c[name].clone()
        t[bad] = val
        dirty[name] = t.to(DEV)
    ids = c["ids"].clone()
    ids[bad] = -7
    dirty["ids"] = ids.to(DEV)
    o2 = outputs(T, 40)
    run(dirty, o2)
    for k in ("loss", "counts", "prob_mean", "tokens", "dlogits"):
        assert torch.equal(o1[k], o2[k]), k
    assert M.read_device_status(o2["ws"]) == M.OK
    check(c, o2)


@pytest.mark.parametrize("T", [30, 1500])
def test_minus_infinity(T):
    c = make(T, 48, 4, seed=12, renorm=False)
    l = c["logits"]
    l[:, 5] = float("-inf")              # an expert that nobody may select
    l[3] = float("-inf")                 # a row that leaves nothing
    l[4] = torch.finfo(torch.float32).min
    c["w"][3] = 0.0
    c["w"][4] = 1.0 / 48
    o = outputs(T, 48)
    run({k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}, o)
    check(c, o)
    assert bool((o["dlogits"][3] == 0).all())


@pytest.mark.parametrize("T", [20, 3000])
def test_id_out_of_range_is_reported_and_skipped(T):
    c = make(T, 16, 3, seed=13)
    c["ids"][1, 0], c["ids"][2, 2] = -1, 16
    o = outputs(T, 16)
    run({k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}, o)
    check(c, o)
    assert M.read_device_status(o["ws"]) == M.DEVICE_BAD_INDEX


def test_same_expert_twice_in_a_row():
    c = make(50, 12, 3, seed=14)
    c["ids"][:, 1] = c["ids"][:, 0]
    o = outputs(50, 12)
    run({k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}, o)
    check(c, o)


def test_no_tokens():
    o = outputs(0, 32)
    c = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in make(0, 32, 2, seed=1).items()}
    run(c, o)
    assert float(o["loss"]) == 0.0 and int(o["tokens"]) == 0
    assert bool((o["counts"] == 0).all()) and bool((o["prob_mean"] == 0).all())


def test_gradient_in_place_and_repeatable():
    c = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in make(6000, 200, 6, seed=15).items()}
    a, b = outputs(6000, 200), outputs(6000, 200)
    run(c, a)
    run(c, b)
    for k in ("loss", "counts", "prob_mean", "tokens", "dlogits"):
        assert torch.equal(a[k], b[k]), k
    M.route_backward(c["logits"], c["ids"], c["w"], c["dw"], c["mask"], c["renorm"], c["dloss"],
                     c["coef"], a["counts"], a["tokens"], c["logits"])
    assert torch.equal(c["logits"], a["dlogits"])


@pytest.mark.parametrize("T", [96, 4000])
def test_graph_replay_on_another_stream(T):
    """Two captured graphs share one workspace; replayed in turn on a side
    stream with new inputs they give the eager bits."""
    cs = [{k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in make(T, 64, 4, seed=s, mask=0.9).items()}
          for s in (1, 2, 3)]
    os_ = [outputs(T, 64) for _ in cs]
    os_[1]["ws"] = os_[0]["ws"]
    want = outputs(T, 64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(st):
        run(cs[0], os_[0], st)
        for i in (0, 1):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                run(cs[i], os_[i], st)
            graphs.append(g)
        for k in ("logits", "ids", "w", "dw", "mask"):
            cs[0][k].copy_(cs[2][k])
        graphs[1].replay()
        graphs[0].replay()
    torch.cuda.current_stream().wait_stream(st)
    run(cs[2], want)
    torch.cuda.synchronize()
    for k in ("loss", "counts", "prob_mean", "tokens", "dlogits"):
        assert torch.equal(os_[0][k], want[k]), k
    run(cs[1], want)
    for k in ("loss", "counts", "prob_mean", "tokens", "dlogits"):
        assert torch.equal(os_[1][k], want[k]), k


def test_gradient_against_differences_of_the_loss():
    """Central differences of the library's own loss along a direction.  The
    counts are constants of the gradient, so the ids stay fixed.  The step h
    leaves a third-order term of at most h^2 |v|^3 relative, and the two losses
    round by TOL each: both are counted."""
    T, E, k, h = 200, 32, 4, 0.25
    c = make(T, E, k, seed=21, weights=False)
    g = {n: dev(v) if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    g["coef"] = 1.0
    o = outputs(T, E)
    run(g, o)
    d = o["dlogits"].cpu().double()
    v = torch.sign(d)                    # the steepest direction: no cancellation
    ends = []
    for sgn in (1, -1):
        moved = dict(g, logits=(c["logits"] + sgn * h * v.float()).to(DEV))
        e = outputs(T, E)
        M.balance_loss(moved["logits"], moved["ids"], None, 1.0, e["loss"], e["counts"], e["prob_mean"],
                       e["tokens"], e["ws"])
        ends.append(float(e["loss"]))
    slope = (ends[0] - ends[1]) / (2 * h)
    want = float((d * v).sum()) / 0.7    # dloss is 0.7 in the gradient
    rounding = TOL * (abs(ends[0]) + abs(ends[1])) / (2 * h)
    assert abs(slope - want) <= rounding + h * h * abs(want)
