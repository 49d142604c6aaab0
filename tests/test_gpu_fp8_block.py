"""The FP8 block-128 product, its gradients and the token-block quantiser against
their formulas in 64 bits on the codes' values.

Tolerances: codes and scales exact (FP32 decides them on both sides); a product
within train_ref.product_bound of the exact sum plus half a step of the output
type (train_ref.HALF_STEP)."""
import numpy as np
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expert_layer_dual_b200.moe as M

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def randn(shape, seed, scale=1.0, outliers=True):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale
    if outliers:
        x[..., :: 37] *= 30.0
    return x.to(torch.bfloat16)


def offsets_of(sizes, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]) + first, dtype=torch.int32)


def workspace():
    return torch.empty(256, dtype=torch.uint8, device=DEV)


def check_rows(got, want, size, blocks, dtype):
    got = got.double()
    bound = ref.product_bound(size, blocks) + ref.HALF_STEP[dtype] * want.abs() + 2.0 ** -25 * (dtype == torch.float16)
    err = (got - want).abs()
    assert bool((err <= bound).all()), (float((err - bound).max()), float(err.max()))


# sizes around every tile boundary: one row, a part of a tile, whole tiles, one row more
DENSE = [(1, 128, 128), (1, 640, 2048), (2, 256, 384), (7, 1152, 256), (16, 512, 640), (17, 128, 1024),
         (33, 384, 512), (63, 256, 896), (64, 2048, 128), (65, 768, 256), (100, 384, 384), (128, 128, 256),
         (129, 256, 128), (200, 640, 640), (255, 256, 256), (256, 512, 512), (257, 384, 1152),
         (300, 1280, 256), (513, 256, 2176), (700, 896, 128), (1025, 512, 384)]
# shapes whose 64 x 128 tiles take twice the waves of the 128 x 256 ones, so that the
# products take the latter (forward: by N; input: the same with N and K exchanged)
WIDE = [(1, 37120, 128), (63, 37120, 256), (130, 12800, 384), (255, 9728, 128), (257, 6400, 640), (600, 4736, 256),
        (1500, 2176, 512), (1920, 2048, 128)]
# (rows of each group, first row, rows behind the last group, N, K)
GROUPED = [([5], 0, 0, 256, 128), ([0, 3, 0], 0, 0, 128, 256), ([1] * 9, 2, 5, 256, 256),
           ([130, 0, 1, 256, 77], 0, 0, 384, 256), ([0, 0], 0, 40, 128, 128), ([300, 20, 500], 7, 9, 256, 640),
           ([64, 64, 63, 65], 0, 0, 512, 384), ([3] * 256, 0, 0, 128, 128), ([0] * 100 + [400] + [0] * 60, 1, 1, 256, 256),
           ([2, 700, 5, 0, 31, 16, 1], 3, 0, 640, 384), ([1100, 900], 0, 0, 384, 512)]


def make_groups(sizes, first, behind):
    rows = first + int(np.sum(sizes)) + behind
    return rows, offsets_of(sizes, first)


def product(op, rows, N, K, G, off, dtype, seed, stream=None):
    """Runs the product on codes made on the CPU: (output on the CPU with a
    sentinel behind unwritten rows, exact, magnitudes, covered)."""
    a_cols, o_cols = (K, N) if op == "forward" else (N, K)
    aq, a_s = ref.quantise_rows(randn((rows, a_cols), seed))
    wq, ws = ref.quantise_weights(randn((G, N, K), seed + 1, 0.1))
    out = torch.full((rows, o_cols), 7.0, dtype=dtype, device=DEV)
    w = workspace()
    f = M.gemm_fp8 if op == "forward" else M.gemm_fp8_dgrad
    f(aq.to(DEV), a_s.to(DEV), (wq if off is not None else wq[0]).to(DEV),
      (ws if off is not None else ws[0]).to(DEV), None if off is None else off.to(DEV), out, w, stream)
    torch.cuda.synchronize()
    assert M.read_device_status(w) == M.OK
    want, size, covered = ref.grouped(ref.rows64(aq, a_s), ref.weights64(wq, ws), off, rows, op == "forward")
    return out.cpu(), want, size, covered


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("op", ["forward", "input"])
@pytest.mark.parametrize("shape", DENSE, ids=lambda s: "x".join(map(str, s)))
def test_dense(shape, op, dtype):
    rows, N, K = shape
    got, want, size, _ = product(op, rows, N, K, 1, None, TYPES[dtype], rows + N)
    check_rows(got, want, size, (K if op == "forward" else N) // 128, TYPES[dtype])


def takes_wide_tiles(rows, cols, groups=1, sms=148):
    """The library's rule, for shapes that have to reach the wide tiles."""
    avg = -(-rows // groups)
    each = rows if groups == 1 else avg + avg // 2
    few, wide = groups * -(-each // 64) * (cols // 128), groups * -(-each // 128) * -(-cols // 256)
    return not -(-few // sms) < 2 * -(-wide // sms)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("op", ["forward", "input"])
@pytest.mark.parametrize("shape", WIDE, ids=lambda s: "x".join(map(str, s)))
def test_dense_wide(shape, op, dtype):
    rows, cols, inner = shape
    assert takes_wide_tiles(rows, cols)
    N, K = (cols, inner) if op == "forward" else (inner, cols)
    got, want, size, _ = product(op, rows, N, K, 1, None, TYPES[dtype], rows)
    check_rows(got, want, size, inner // 128, TYPES[dtype])


# groups for the wide tiles: empty ones, single rows, tiles filled to the row and one
# over, a first row and rows behind
WIDE_GROUPED = [([0, 300, 1, 0, 128, 129, 127, 700, 0], 5, 3, 5120, 256), ([256] * 6, 0, 0, 3840, 128),
                ([1] * 40 + [900], 0, 7, 5120, 256), ([64] * 30, 0, 0, 1280, 384)]


@pytest.mark.parametrize("op", ["forward", "input"])
@pytest.mark.parametrize("case", range(len(WIDE_GROUPED)))
def test_grouped_wide(case, op):
    sizes, first, behind, cols, inner = WIDE_GROUPED[case]
    rows, off = make_groups(sizes, first, behind)
    assert takes_wide_tiles(rows, cols, len(sizes))
    N, K = (cols, inner) if op == "forward" else (inner, cols)
    for dtype in (torch.bfloat16, torch.float32):
        got, want, size, covered = product(op, rows, N, K, len(sizes), off, dtype, case)
        check_rows(got[covered], want[covered], size[covered], inner // 128, dtype)
        assert bool((got[~covered] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["forward", "input"])
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped(case, op, dtype):
    sizes, first, behind, N, K = GROUPED[case]
    rows, off = make_groups(sizes, first, behind)
    got, want, size, covered = product(op, rows, N, K, len(sizes), off, TYPES[dtype], case)
    check_rows(got[covered], want[covered], size[covered], (K if op == "forward" else N) // 128, TYPES[dtype])
    assert bool((got[~covered] == 7.0).all())


@pytest.mark.parametrize("cols", [128, 384, 1024])
@pytest.mark.parametrize("case", [None] + list(range(len(GROUPED))))
def test_token_quantiser_exact(case, cols):
    if case is None:
        rows, off, G = 333, None, 1
    else:
        sizes, first, behind, _, _ = GROUPED[case]
        rows, off = make_groups(sizes, first, behind)
        G = len(sizes)
    x = randn((rows, cols), 3 * cols)
    x[:, 5] = 0
    R = M.fp8_token_rows(rows, G)
    q = torch.full((cols, R), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((R // 128, cols), -1.0, device=DEV)
    M.quantize_fp8_tokens(x.to(DEV), None if off is None else off.to(DEV), q, s)
    wq, ws, used = ref.quantise_tokens(x, off, R)
    q, s = q.cpu(), s.cpu()
    assert torch.equal(q[:, : used * 128], wq[:, : used * 128])
    assert torch.equal(s[:used], ws[:used])
    assert bool((q[:, used * 128:] == 0x55).all()) and bool((s[used:] == -1.0).all())


def weight_gradient(rows, N, K, G, off, accumulate, seed):
    dy, x = randn((rows, N), seed, 1e-3), randn((rows, K), seed + 1)
    R = M.fp8_token_rows(rows, G)
    offd = None if off is None else off.to(DEV)
    ops = []
    for t in (dy, x):
        # what lies behind the groups' blocks is never read: poison it
        q = torch.full((t.shape[1], R), 0x7F, dtype=torch.uint8, device=DEV)
        s = torch.full((R // 128, t.shape[1]), float("nan"), device=DEV)
        M.quantize_fp8_tokens(t.to(DEV), offd, q, s)
        ops += [q, s]
    start = randn((G, N, K), seed + 2, outliers=False).float()
    dw = (start if off is not None else start[0]).to(DEV)
    w = workspace()
    M.gemm_fp8_wgrad(*ops, offd, rows, dw, accumulate, w)
    torch.cuda.synchronize()
    assert M.read_device_status(w) == M.OK
    want, size = ref.weight_gradient(ops[0].cpu(), ops[1].cpu(), ops[2].cpu(), ops[3].cpu(), off, rows)
    if accumulate:
        want, size = want + start.double(), size + start.double().abs()
    return dw.cpu().reshape(G, N, K), want, size


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("shape", DENSE, ids=lambda s: "x".join(map(str, s)))
def test_weight_gradient_dense(shape, accumulate):
    rows, N, K = shape
    got, want, size = weight_gradient(rows, N, K, 1, None, accumulate, rows)
    check_rows(got, want, size, (rows + 127) // 128, torch.float32)


# few tiles and long sums: rows, N, K, where a cluster of eight, four or two CTAs shares
# the blocks of a tile; blocks that do not divide evenly and CTAs left without one.
# (The cluster's sums round up to seven times more.)
SPLIT_SUMS = [(4096, 512, 512), (4097, 128, 128), (4993, 256, 384), (5001, 1024, 1024), (4200, 1024, 2048),
              (9345, 384, 640)]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("shape", SPLIT_SUMS, ids=lambda s: "x".join(map(str, s)))
def test_weight_gradient_of_long_sums(shape, accumulate):
    rows, N, K = shape
    got, want, size = weight_gradient(rows, N, K, 1, None, accumulate, rows)
    check_rows(got, want, size, (rows + 127) // 128 + 7, torch.float32)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("sizes", [[9000, 0, 300], [4100, 4095], [1, 0, 16500]], ids=str)
def test_weight_gradient_of_long_groups(sizes, accumulate):
    """Groups without rows keep what was there, or become zeros."""
    rows, off = make_groups(sizes, 2, 3)
    got, want, size = weight_gradient(rows, 256, 384, len(sizes), off, accumulate, rows)
    for g, n in enumerate(sizes):
        check_rows(got[g], want[g], size[g], (n + 127) // 128 + 7, torch.float32)
        if n == 0:
            assert torch.equal(got[g], want[g].float())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("op", ["forward", "input"])
@pytest.mark.parametrize("shape", [(1024, 2048, 6144), (1001, 2176, 6272), (700, 2432, 8192)],
                         ids=lambda s: "x".join(map(str, s)))
def test_dense_long_sums(shape, op, dtype):
    rows, cols, inner = shape
    assert takes_wide_tiles(rows, cols)
    N, K = (cols, inner) if op == "forward" else (inner, cols)
    got, want, size, _ = product(op, rows, N, K, 1, None, TYPES[dtype], rows)
    check_rows(got, want, size, inner // 128 + 1, TYPES[dtype])


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_weight_gradient_grouped(case, accumulate):
    sizes, first, behind, N, K = GROUPED[case]
    if len(sizes) > 100:
        N = K = 128
    rows, off = make_groups(sizes, first, behind)
    got, want, size = weight_gradient(rows, N, K, len(sizes), off, accumulate, case)
    check_rows(got, want, size, max(1, (max(sizes) + 127) // 128), torch.float32)


def test_no_rows():
    w = workspace()
    q = torch.empty((0, 128), dtype=torch.uint8, device=DEV)
    s = torch.empty((0, 1), device=DEV)
    wq, ws = ref.quantise_weights(randn((1, 128, 128), 1))
    out = torch.empty((0, 128), device=DEV)
    M.gemm_fp8(q, s, wq[0].to(DEV), ws[0].to(DEV), None, out, w)
    t = torch.empty((128, 0), dtype=torch.uint8, device=DEV)
    ts = torch.empty((0, 128), device=DEV)
    M.quantize_fp8_tokens(torch.empty((0, 128), dtype=torch.bfloat16, device=DEV), None, t, ts)
    dw = torch.ones((128, 128), device=DEV)
    M.gemm_fp8_wgrad(t, ts, t, ts, None, 0, dw, True, w)
    assert bool((dw == 1).all())
    M.gemm_fp8_wgrad(t, ts, t, ts, None, 0, dw, False, w)
    assert bool((dw == 0).all())


def test_offsets_out_of_order_touch_nothing_outside():
    """Offsets that no routing gives are clamped: a running maximum inside [0, M]."""
    rows, N, K = 90, 128, 128
    bad = torch.tensor([-5, 40, 20, 1000], dtype=torch.int32)
    good = torch.tensor([0, 40, 40, 90], dtype=torch.int32)
    aq, a_s = ref.quantise_rows(randn((rows, K), 1))
    wq, ws = ref.quantise_weights(randn((3, N, K), 2))
    outs = []
    for off in (bad, good):
        room = torch.full((rows + 64, N), 7.0, device=DEV)
        M.gemm_fp8(aq.to(DEV), a_s.to(DEV), wq.to(DEV), ws.to(DEV), off.to(DEV), room[:rows], workspace())
        assert bool((room[rows:] == 7.0).all())
        outs.append(room[:rows].clone())
    assert torch.equal(outs[0], outs[1])


def test_f16_saturates():
    rows, N, K = 3, 128, 256
    aq, a_s = ref.quantise_rows(torch.full((rows, K), 300.0).to(torch.bfloat16))
    wq, ws = ref.quantise_weights(torch.full((1, N, K), 2.0).to(torch.bfloat16))
    out = torch.empty((rows, N), dtype=torch.float16, device=DEV)
    M.gemm_fp8(aq.to(DEV), a_s.to(DEV), wq[0].to(DEV), ws[0].to(DEV), None, out, workspace())
    assert bool((out == 65504.0).all())


@pytest.mark.parametrize("shape", [(4, 256, 512), (400, 384, 256), (400, 12800, 256)])
def test_infinite_scale_stays_in_its_row(shape):
    """A NaN code or an infinite scale reaches its own row of y only."""
    rows, N, K = shape
    aq, a_s = ref.quantise_rows(randn((rows, K), 1))
    wq, ws = ref.quantise_weights(randn((1, N, K), 2))
    clean = torch.empty((rows, N), device=DEV)
    args = (wq[0].to(DEV), ws[0].to(DEV), None)
    M.gemm_fp8(aq.to(DEV), a_s.to(DEV), *args, clean, workspace())
    aq[1, 3] = 0x7F
    a_s[2, 1] = float("inf")
    dirty = torch.empty((rows, N), device=DEV)
    M.gemm_fp8(aq.to(DEV), a_s.to(DEV), *args, dirty, workspace())
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[1:3] = False
    assert torch.equal(clean[keep], dirty[keep])
    assert bool(torch.isnan(dirty[1]).all()) and not bool(torch.isfinite(dirty[2]).any())


def test_capture_and_replay_on_a_side_stream():
    """The whole step (quantise, product, both gradients) captured; two graphs with
    one workspace, replayed in turn with new inputs, give the eager bits."""
    rows, N, K, sizes = 500, 384, 256, [100, 0, 390, 10]
    off = offsets_of(sizes).to(DEV)
    G, R = len(sizes), M.fp8_token_rows(rows, len(sizes))
    wq, ws = [t.to(DEV) for t in ref.quantise_weights(randn((G, N, K), 9, 0.1))]
    shared = workspace()

    def state(seed):
        e = lambda *s, d=torch.uint8: torch.zeros(s, dtype=d, device=DEV)  # noqa: E731
        return {"x": randn((rows, K), seed).to(DEV), "dy": randn((rows, N), seed + 1).to(DEV),
                "xq": e(rows, K), "xs": e(rows, K // 128, d=torch.float32), "dq": e(rows, N),
                "ds": e(rows, N // 128, d=torch.float32), "xt": e(K, R), "xts": e(R // 128, K, d=torch.float32),
                "dt": e(N, R), "dts": e(R // 128, N, d=torch.float32), "y": e(rows, N, d=torch.bfloat16),
                "dx": e(rows, K, d=torch.bfloat16), "dw": e(G, N, K, d=torch.float32)}

    def step(s, w, stream=None):
        M.quantize_act_fp8(s["x"], s["xq"], s["xs"], stream)
        M.gemm_fp8(s["xq"], s["xs"], wq, ws, off, s["y"], w, stream)
        M.quantize_act_fp8(s["dy"], s["dq"], s["ds"], stream)
        M.gemm_fp8_dgrad(s["dq"], s["ds"], wq, ws, off, s["dx"], w, stream)
        M.quantize_fp8_tokens(s["dy"], off, s["dt"], s["dts"], stream)
        M.quantize_fp8_tokens(s["x"], off, s["xt"], s["xts"], stream)
        M.gemm_fp8_wgrad(s["dt"], s["dts"], s["xt"], s["xts"], off, rows, s["dw"], False, w, stream)

    a, b, fresh = state(1), state(3), state(5)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(st):
        step(a, shared, st)
        for s in (a, b):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                step(s, shared, st)
            graphs.append(g)
        a["x"].copy_(fresh["x"])
        a["dy"].copy_(fresh["dy"])
        graphs[1].replay()
        graphs[0].replay()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    step(fresh, workspace())
    eager_b = state(3)
    step(eager_b, workspace())
    torch.cuda.synchronize()
    for k in ("y", "dx", "dw"):
        assert torch.equal(a[k], fresh[k]) and torch.equal(b[k], eager_b[k]), k


# rows of each group, N, K: the persistent tiles and their bulk stores, and sums split
# over clusters
ACCUMULATED = [([700], 1024, 5120), ([0, 300, 129, 5], 512, 640), ([4500], 384, 640), ([40] * 30, 640, 768)]


@pytest.mark.parametrize("case", range(len(ACCUMULATED)))
def test_accumulation_in_a_row(case):
    """Weight gradients added into one buffer by launches that follow one another, eager
    and replayed: each adds the same bits with one rounding."""
    sizes, N, K = ACCUMULATED[case]
    rows, off = make_groups(sizes, 0, 0)
    G, R = len(sizes), M.fp8_token_rows(rows, len(sizes))
    off = off.to(DEV)
    ops = []
    for i, c in enumerate((N, K)):
        q = torch.zeros((c, R), dtype=torch.uint8, device=DEV)
        s = torch.zeros((R // 128, c), device=DEV)
        M.quantize_fp8_tokens(randn((rows, c), 11 + i).to(DEV), off, q, s)
        ops += [q, s]
    dw, w = torch.empty((G, N, K), device=DEV), workspace()
    M.gemm_fp8_wgrad(*ops, off, rows, dw, False, w)
    one = dw.clone()
    for _ in range(3):
        M.gemm_fp8_wgrad(*ops, off, rows, dw, True, w)
    want = ((one + one) + one) + one
    assert torch.equal(dw, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        for _ in range(2):
            M.gemm_fp8_wgrad(*ops, off, rows, dw, True, w)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for _ in range(4):
        want = want + one
    assert torch.equal(dw, want) and M.read_device_status(w) == M.OK


def test_two_streams_of_weight_gradients():
    """Split sums and persistent tiles in flight together, a workspace each."""
    shapes = [(4500, 384, 640), (600, 1024, 4096)]
    calls = []
    for i, (rows, N, K) in enumerate(shapes):
        R = M.fp8_token_rows(rows)
        ops = []
        for j, c in enumerate((N, K)):
            q = torch.zeros((c, R), dtype=torch.uint8, device=DEV)
            s = torch.zeros((R // 128, c), device=DEV)
            M.quantize_fp8_tokens(randn((rows, c), 5 * i + j).to(DEV), None, q, s)
            ops += [q, s]
        alone = torch.empty((N, K), device=DEV)
        M.gemm_fp8_wgrad(*ops, None, rows, alone, False, workspace())
        calls.append((ops, rows, alone, torch.empty_like(alone), workspace(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for ops, rows, _, out, w, st in calls:
            M.gemm_fp8_wgrad(*ops, None, rows, out, False, w, st)
    torch.cuda.synchronize()
    for _, _, alone, out, w, _ in calls:
        assert torch.equal(out, alone) and M.read_device_status(w) == M.OK


def test_two_streams_at_once():
    """Two products in flight on two streams (a workspace each) give the bits of one."""
    rows, N, K = 600, 640, 512
    aq, a_s = [t.to(DEV) for t in ref.quantise_rows(randn((rows, K), 1))]
    wq, ws = [t[0].to(DEV) for t in ref.quantise_weights(randn((1, N, K), 2))]
    outs = [torch.empty((rows, N), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    spaces = [workspace() for _ in range(3)]
    M.gemm_fp8(aq, a_s, wq, ws, None, outs[2], spaces[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i, st in enumerate(streams):
            M.gemm_fp8(aq, a_s, wq, ws, None, outs[i], spaces[i], st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])


def test_training_step_of_routed_experts():
    """The operators together, as a routed FP8 projection is trained: top-k and
    permute of the logits, x in the permuted order, the experts' product, the
    gradients of the rows, the expert weights and the router's logits."""
    T, E, k, N, K = 300, 12, 3, 256, 384
    g = torch.Generator().manual_seed(6)
    logits = torch.randn((T, E), generator=g) * 2
    x, dy = randn((T, K), 7), randn((T * k, N), 8, 1e-2)
    wq, ws = ref.quantise_weights(randn((E, N, K), 9, 0.1))
    d = {n: t.to(DEV) for n, t in (("l", logits), ("x", x), ("dy", dy), ("wq", wq), ("ws", ws))}
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)  # noqa: E731
    f32 = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    ids, w, counts, off, perm, inv = i32(T, k), f32(T, k), i32(E), i32(E + 1), i32(T * k), i32(T * k)
    M.route_topk(d["l"], k, True, ids, w)
    M.permute(ids, E, counts, off, perm, inv, u8(M.permute_workspace_bytes(T, E, k)))
    loss, bc, pm, tok, dl = f32(1), i32(E), f32(E), i32(1), f32(T, E)
    M.balance_loss(d["l"], ids, None, 0.01, loss, bc, pm, tok, u8(M.balance_workspace_bytes(T, E)))
    assert torch.equal(bc, counts)
    R = T * k
    xq, xs, y, sp = u8(R, K), f32(R, K // 128), torch.empty((R, N), dtype=torch.float16, device=DEV), workspace()
    M.quantize_act_fp8_permuted(d["x"], perm, k, 0, xq, xs)
    M.gemm_fp8(xq, xs, d["wq"], d["ws"], off, y, sp)
    dq, ds, dx = u8(R, N), f32(R, N // 128), f32(R, K)
    M.quantize_act_fp8(d["dy"], dq, ds)
    M.gemm_fp8_dgrad(dq, ds, d["wq"], d["ws"], off, dx, sp)
    rows = M.fp8_token_rows(R, E)
    dt, dts, xt, xts, dw = u8(N, rows), f32(rows // 128, N), u8(K, rows), f32(rows // 128, K), f32(E, N, K)
    xp = d["x"][(perm // k).long()].contiguous()
    M.quantize_fp8_tokens(d["dy"], off, dt, dts)
    M.quantize_fp8_tokens(xp, off, xt, xts)
    M.gemm_fp8_wgrad(dt, dts, xt, xts, off, R, dw, False, sp)
    # the gradient of w_j: <dy, y> of its row, then the router's logits
    dwts = (d["dy"].float() * y.float()).sum(1)[inv.long()].reshape(T, k).contiguous()
    one = torch.ones(1, device=DEV)
    M.route_backward(d["l"], ids, w, dwts, None, True, one, 0.01, bc, tok, dl)
    torch.cuda.synchronize()

    offc, idc = off.cpu(), ids.cpu()
    want = ref.balance(logits, idc, None, 0.01)
    assert abs(float(loss.cpu()) - want["loss"]) <= 1e-5 * want["loss"]
    W = ref.weights64(wq, ws)
    yw, size, _ = ref.grouped(ref.rows64(xq.cpu(), xs.cpu()), W, offc, R, True)
    check_rows(y.cpu(), yw, size, K // 128, torch.float16)
    rq, rs = ref.quantise_rows(x[(perm.cpu() // k).long()])
    assert torch.equal(rq, xq.cpu()) and torch.equal(rs, xs.cpu())
    dxw, size, _ = ref.grouped(ref.rows64(dq.cpu(), ds.cpu()), W, offc, R, False)
    check_rows(dx.cpu(), dxw, size, N // 128, torch.float32)
    dww, size = ref.weight_gradient(dt.cpu(), dts.cpu(), xt.cpu(), xts.cpu(), offc, R)
    check_rows(dw.cpu(), dww, size, int((counts.max() + 127) // 128), torch.float32)
    dlw, size = ref.route_backward(logits, idc, w.cpu(), dwts.cpu(), None, True, 1.0, 0.01, want["counts"], T)
    assert bool(((dl.cpu().double() - dlw).abs() <= 1e-5 * size + 1e-37).all())
    # the adjoint identities on the values the codes stand for: <dy, y> = <dx, x>
    lhs = float((ref.rows64(dq.cpu(), ds.cpu()) * yw).sum())
    rhs = float((dxw * ref.rows64(xq.cpu(), xs.cpu())).sum())
    assert abs(lhs - rhs) <= 1e-9 * float((dxw.abs() * ref.rows64(xq.cpu(), xs.cpu()).abs()).sum())


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -60, 2.0 ** 60, 2.0 ** -115, 2.0 ** 118, 3.0e-39])
def test_codes_of_every_bf16_value(scale):
    """Every finite bf16 pattern, scaled into a group whose largest magnitude is
    448 * scale or the pattern's own: the codes of both quantisers are the
    rounded FP32 quotients (ties, e4m3 subnormals and saturation among them)."""
    bits = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[torch.isfinite(v)].float()
    v = (v * scale).to(torch.bfloat16)
    v = v[torch.isfinite(v)]
    v = v[v.abs().float() <= 448.0 * scale] if scale >= 1.0 else v
    tops = torch.tensor([448.0, 1.0, 3.7, 100.0, 2.0 ** -7]) * scale
    rows = []
    for top in tops.tolist():
        w = v[v.abs().float() <= top]
        w = w[: w.numel() // 127 * 127].reshape(-1, 127)
        rows.append(torch.cat([torch.full((w.shape[0], 1), top).to(torch.bfloat16), w], 1))
    x = torch.cat(rows)                                   # groups of 128, the first value the largest
    q = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    s = torch.empty((x.shape[0], 1), device=DEV)
    M.quantize_act_fp8(x.to(DEV), q, s)
    wq, ws = ref.quantise_rows(x)
    assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu(), wq)
    xt = x[: x.shape[0] // 128 * 128].T.contiguous()      # the same groups along the tokens
    R = M.fp8_token_rows(128, 1)
    qt = torch.empty((xt.shape[1], R), dtype=torch.uint8, device=DEV)
    st = torch.empty((1, xt.shape[1]), device=DEV)
    M.quantize_fp8_tokens(xt.to(DEV), None, qt, st)
    n = xt.shape[1]
    assert torch.equal(qt.cpu(), wq[:n]) and torch.equal(st.cpu()[0], ws[:n, 0])


def test_scale_of_every_bf16_maximum():
    """s = fp32(amax) / 448 by the IEEE division for every positive finite bf16 amax."""
    top = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros((top.numel(), 128), dtype=torch.bfloat16)
    x[:, 77] = -top
    q = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    s = torch.empty((x.shape[0], 1), device=DEV)
    M.quantize_act_fp8(x.to(DEV), q, s)
    wq, ws = ref.quantise_rows(x)
    assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu(), wq)


@pytest.mark.parametrize("shape", [(5, 2176), (2900, 1408), (1200, 3328), (10700, 1408), (4500, 3328)],
                         ids=lambda s: "x".join(map(str, s)))
def test_row_quantiser_exact(shape):
    """One, two and four loads a warp, with rows that end inside a warp's columns, and
    nothing written behind the rows."""
    rows, cols = shape
    x = randn(shape, rows)
    x[:, 128:256] = 0
    q = torch.full((rows + 1, cols), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((rows + 1, cols // 128), -1.0, device=DEV)
    M.quantize_act_fp8(x.to(DEV), q[:rows], s[:rows])
    wq, ws = ref.quantise_rows(x)
    assert torch.equal(q[:rows].cpu(), wq) and torch.equal(s[:rows].cpu(), ws)
    assert bool((q[rows] == 0x55).all()) and bool((s[rows] == -1.0).all())


def test_codes_of_values_that_are_not_finite():
    """NaN and infinities in a group: the codes and scales are those of the quantiser
    of permuted rows (here in the rows' own order), which divides, and the same
    along the tokens."""
    bf = torch.bfloat16
    rows = []
    for special in ([float("nan")], [float("inf")], [-float("inf")], [float("nan"), -float("inf")],
                    [-0.0, float("nan")]):
        for n in (1, 5, 128):
            r = torch.linspace(-3, 3, 128).to(bf)
            v = torch.tensor(special).to(bf)
            r[:n] = v.repeat(128)[:n]
            rows += [r, (r.view(torch.int16) ^ -32768).view(bf)]   # the signs of NaN too
    x = torch.stack(rows)
    x = torch.cat([x, x[: 128 % x.shape[0]], x, x, x])[:128].contiguous()
    T = x.shape[0]
    q, pq, qt = (torch.empty((T, 128), dtype=torch.uint8, device=DEV) for _ in range(3))
    s, ps, st = (torch.empty((T, 1), device=DEV) for _ in range(3))
    M.quantize_act_fp8(x.to(DEV), q, s)
    M.quantize_act_fp8_permuted(x.to(DEV), torch.arange(T, dtype=torch.int32, device=DEV), 1, 0, pq, ps)
    assert torch.equal(q, pq) and torch.equal(s.view(torch.int32), ps.view(torch.int32))
    M.quantize_fp8_tokens(x.T.contiguous().to(DEV), None, qt, st.T)
    assert torch.equal(qt, pq) and torch.equal(st.view(torch.int32), ps.view(torch.int32))


def test_binding_refuses_what_is_not_the_calls():
    """Shapes, types, layouts and devices that do not fit raise ValueError before a
    launch; limits of the library come back as its status."""
    z = lambda *s, d=torch.uint8: torch.zeros(s, dtype=d, device=DEV)  # noqa: E731
    f32 = torch.float32
    good = dict(x_q=z(4, 256), x_s=z(4, 2, d=f32), w_q=z(128, 256), w_s=z(1, 2, d=f32), offsets=None,
                y=z(4, 128, d=f32), ws=z(256))
    M.gemm_fp8(*good.values())
    for change in ({"x_q": z(256, 4).T}, {"x_q": z(4, 128)}, {"x_q": z(4, 256, d=f32)}, {"x_s": z(4, 3, d=f32)},
                   {"x_s": z(2, 4, d=f32)}, {"x_s": z(4, 2, d=torch.float64)}, {"w_q": z(128, 256).cpu()},
                   {"w_s": z(2, 1, d=f32)}, {"y": z(4, 256, d=f32)}, {"y": z(4, 128, d=torch.int32)},
                   {"y": z(4, 256, d=f32)[:, ::2]}, {"offsets": z(2, d=torch.int64)},
                   {"offsets": z(3, d=torch.int32)}, {"w_q": z(2, 128, 256), "w_s": z(2, 1, 2, d=f32)},
                   {"ws": z(256).cpu()}, {"x_q": None}):
        with pytest.raises((ValueError, AttributeError)):
            M.gemm_fp8(*{**good, **change}.values())
    for change, code in (({"ws": z(128)}, M.WORKSPACE_TOO_SMALL),
                         ({"w_q": z(100, 256), "w_s": z(0, 2, d=f32), "y": z(4, 100, d=f32)}, M.UNSUPPORTED),
                         ({"x_q": z(4 * 256 + 8)[8:].view(4, 256)}, M.INVALID_ARG)):
        with pytest.raises(M.MoEError) as e:
            M.gemm_fp8(*{**good, **change}.values())
        assert e.value.code == code
    dw, t, ts = z(128, 256, d=f32), z(128, 128), z(1, 128, d=f32)
    xt, xts = z(256, 128), z(1, 256, d=f32)
    M.gemm_fp8_wgrad(t, ts, xt, xts, None, 5, dw, False, z(256))
    for bad in ((t, ts, xt, xts, None, 129, dw, False, z(256)), (xt, ts, xt, xts, None, 5, dw, False, z(256)),
                (t, ts, xt, xts, None, 5, dw.half(), False, z(256))):
        with pytest.raises(ValueError):
            M.gemm_fp8_wgrad(*bad)
    with pytest.raises(M.MoEError):
        M.gemm_fp8_wgrad(z(128, 0), z(0, 128, d=f32), z(256, 0), z(0, 256, d=f32), None, -1, dw, False, z(256))


def test_unaligned_outputs_and_scales():
    """16 bytes of alignment are enough for the outputs, 4 for the scales (the wide
    stores and copies fall back)."""
    def off_by(t, n):
        flat = torch.zeros(t.numel() + 64, dtype=t.dtype, device=DEV)
        v = flat[n: n + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    for rows, N, K in ((70, 256, 512), (600, 4736, 512)):
        aq, a_s = [t.to(DEV) for t in ref.quantise_rows(randn((rows, K), 1))]
        wq, ws = [t[0].to(DEV) for t in ref.quantise_weights(randn((1, N, K), 2, 0.1))]
        for dtype, step in ((torch.bfloat16, 8), (torch.float32, 4)):
            y = torch.empty((rows, N), dtype=dtype, device=DEV)
            M.gemm_fp8(aq, a_s, wq, ws, None, y, workspace())
            z = off_by(torch.zeros_like(y), step)
            assert z.data_ptr() % 32 == 16
            M.gemm_fp8(off_by(aq, 16), off_by(a_s, 1), off_by(wq, 16), off_by(ws, 3), None, z, workspace())
            assert torch.equal(y, z)
    R = M.fp8_token_rows(300, 1)
    ops = []
    for c, seed in ((256, 3), (384, 4)):
        q, s = torch.empty((c, R), dtype=torch.uint8, device=DEV), torch.empty((R // 128, c), device=DEV)
        M.quantize_fp8_tokens(randn((300, c), seed).to(DEV), None, q, s)
        ops += [q, s]
    dw = torch.empty((256, 384), device=DEV)
    M.gemm_fp8_wgrad(*ops, None, 300, dw, False, workspace())
    dz = off_by(dw * 0, 4)
    M.gemm_fp8_wgrad(ops[0], off_by(ops[1], 1), ops[2], off_by(ops[3], 2), None, 300, dz, False, workspace())
    assert torch.equal(dw, dz)


def test_first_calls_inside_a_capture():
    """A process whose first use of the products is inside a stream capture."""
    import subprocess
    import sys
    code = """
import torch, expert_layer_dual_b200.moe as M
d = "cuda"
z = lambda *s, t=torch.uint8: torch.full(s, 1, dtype=t, device=d)
f = torch.float32
a, s, w, ws, y, sp = z(40, 512), z(40, 4, t=f), z(256, 512), z(2, 4, t=f), z(40, 256, t=f), z(256)
big, bs, bw, bws, by = z(700, 256), z(700, 2, t=f), z(4736, 256), z(37, 2, t=f), z(700, 4736, t=f)
t, ts, dw = z(256, 128), z(1, 256, t=f), z(256, 256, t=f)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    M.gemm_fp8(a, s, w, ws, None, y, sp)
    M.gemm_fp8(big, bs, bw, bws, None, by, sp)
    M.gemm_fp8_wgrad(t, ts, t, ts, None, 100, dw, False, sp)
y.zero_(), by.zero_(), dw.zero_()
g.replay()
torch.cuda.synchronize()
v = 2.0 ** -9  # code 1 is the smallest e4m3 value
assert bool((y == 512 * v * v).all()) and bool((by == 256 * v * v).all()) and bool((dw == 128 * v * v).all())
print("fine")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
