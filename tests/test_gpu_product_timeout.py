"""The failure path of the FP8 block products: a bounded wait that runs out in one block
is reported, and leaves the output tiles that depend on that block as they were (also
those that a cluster of blocks shares), the context usable.  The wait is one that
nothing completes; it ends by its limit."""
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expert_layer_dual_b200.moe as M

DEV = "cuda"
LIMIT_US = 20000


def operands(op, rows, N, K, seed=3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    if op == 2:
        R = M.fp8_token_rows(rows, 1)
        ops = []
        for c in (N, K):
            q, s = torch.empty((c, R), dtype=torch.uint8, device=DEV), torch.empty((R // 128, c), device=DEV)
            M.quantize_fp8_tokens(r(rows, c).to(DEV), None, q, s)
            ops += [q, s]
        return ops, (N, K)
    a, a_s = ref.quantise_rows(r(rows, K if op == 0 else N))
    w, w_s = ref.quantise_weights(r(1, N, K))
    return [t.to(DEV) for t in (a, a_s, w[0], w_s[0])], (rows, N if op == 0 else K)


def product(op, ops, rows, out, ws, accumulate=False):
    if op == 2:
        M.gemm_fp8_wgrad(*ops, None, rows, out, accumulate, ws)
    else:
        (M.gemm_fp8 if op == 0 else M.gemm_fp8_dgrad)(*ops, None, out, ws)


# (op, rows, N, K, block that gives up, rows and columns of a tile): whole tiles, tiles
# shared by clusters (long sums), the few-row form in clusters and alone
CASES = [(0, 600, 4736, 256, 5, 128, 256), (1, 600, 256, 4736, 0, 128, 256), (2, 1000, 2048, 4096, 17, 128, 256),
         (0, 1024, 2048, 6144, 3, 128, 256), (1, 1024, 6144, 2048, 64, 128, 256), (2, 16384, 1024, 1024, 2, 128, 256),
         (2, 16384, 1024, 1024, 127, 128, 256), (0, 64, 4096, 2048, 9, 64, 128), (1, 33, 4096, 2048, 1, 64, 128),
         (0, 64, 18944, 256, 7, 64, 128)]


@pytest.mark.parametrize("case", [(c, False) for c in CASES] + [(c, True) for c in CASES if c[0] == 2],
                         ids=lambda c: "-".join(map(str, c[0])) + ("-accumulate" if c[1] else ""))
def test_timeout_leaves_the_tiles_it_concerns(case):
    (op, rows, N, K, block, bm, bn), accumulate = case
    ops, shape = operands(op, rows, N, K)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    before = torch.randn(shape, generator=torch.Generator().manual_seed(9)).to(DEV)
    want = before.clone()
    product(op, ops, rows, want, ws, accumulate)
    assert M.read_device_status(ws) == M.OK
    got = before.clone()
    M.selftest_product_timeout(op, *ops, rows, got, accumulate, block, LIMIT_US, ws)
    assert M.read_device_status(ws) == M.DEVICE_TIMEOUT
    # every tile is either what the product gives or what it was; few were left, one at least
    left = written = 0
    for i in range(0, shape[0], bm):
        for j in range(0, shape[1], bn):
            t = (slice(i, i + bm), slice(j, j + bn))
            same, done = torch.equal(got[t], before[t]), torch.equal(got[t], want[t])
            assert same or done, f"tile at {i}, {j} holds neither the result nor what it held"
            left += same
            written += done
    assert left >= 1 and written > left, (left, written)
    # the context is usable and the next call right
    product(op, ops, rows, before, ws, accumulate)
    assert M.read_device_status(ws) == M.OK and torch.equal(before, want)
