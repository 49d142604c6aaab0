"""The FP8 block products under conditions that the single-call tests do not make: as many
groups as the library takes, on every tile form, and first calls from several threads."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import train_ref as ref
from test_gpu_fp8_block import check_rows, make_groups, product, randn, takes_wide_tiles, workspace

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import expert_layer_dual_b200.moe as M

DEV = "cuda"


def sizes_of(groups, rows, seed):
    """A ragged split: some groups empty, some of one row, some past a tile."""
    rng = np.random.RandomState(seed)
    p = rng.pareto(1.2, groups) * (rng.rand(groups) < 0.8)
    return rng.multinomial(rows, p / p.sum())


@pytest.mark.parametrize("op", ["forward", "input"])
@pytest.mark.parametrize("groups,rows,cols,inner", [(256, 25600, 256, 128), (256, 16000, 512, 256), (255, 30001, 384, 128)])
def test_256_groups_on_wide_tiles(groups, rows, cols, inner, op):
    assert takes_wide_tiles(rows, cols, groups)
    total, off = make_groups(sizes_of(groups, rows, rows), 3, 5)
    N, K = (cols, inner) if op == "forward" else (inner, cols)
    got, want, size, covered = product(op, total, N, K, groups, off, torch.bfloat16, groups)
    check_rows(got[covered], want[covered], size[covered], inner // 128, torch.bfloat16)
    assert bool((got[~covered] == 7.0).all())


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows", [9000, 40])
def test_weight_gradient_of_256_groups(rows, accumulate):
    G, N, K = 256, 256, 128
    sizes = sizes_of(G, rows, rows)
    total, off = make_groups(sizes, 0, 0)
    dy, x = randn((total, N), 1), randn((total, K), 2)
    R = M.fp8_token_rows(total, G)
    ops = []
    for v in (dy, x):
        q, s = torch.empty((v.shape[1], R), dtype=torch.uint8, device=DEV), torch.empty((R // 128, v.shape[1]), device=DEV)
        M.quantize_fp8_tokens(v.to(DEV), off.to(DEV), q, s)
        ops += [q, s]
    before = torch.randn((G, N, K), generator=torch.Generator().manual_seed(3))
    out, ws = before.to(DEV), workspace()
    M.gemm_fp8_wgrad(*ops, off.to(DEV), total, out, accumulate, ws)
    assert M.read_device_status(ws) == M.OK
    out, q = out.cpu(), [t.cpu() for t in ops]
    block = 0
    for g in range(G):
        b = -(-int(sizes[g]) // 128)
        want = torch.zeros((N, K), dtype=torch.float64)
        size = torch.zeros_like(want)
        for i in range(block, block + b):
            a = q[0][:, 128 * i: 128 * i + 128].view(torch.float8_e4m3fn).double() * q[1][i].double()[:, None]
            c = q[2][:, 128 * i: 128 * i + 128].view(torch.float8_e4m3fn).double() * q[3][i].double()[:, None]
            want += a @ c.T
            size += a.abs() @ c.abs().T
        block += b
        if accumulate:
            want += before[g]
            size += before[g].abs()
        check_rows(out[g], want, size, b + 1, torch.float32)


def test_first_calls_from_several_threads():
    """A process whose first uses of the products are on four threads at once, each with a
    stream of its own: the set-up that each makes once per device is shared."""
    code = """
import threading, torch, expert_layer_dual_b200.moe as M
d = "cuda"
z = lambda *s, t=torch.uint8: torch.full(s, 1, dtype=t, device=d)
f = torch.float32
a, s, w, ws = z(40, 512), z(40, 4, t=f), z(256, 512), z(2, 4, t=f)
big, bs, bw, bws = z(700, 256), z(700, 2, t=f), z(4736, 256), z(37, 2, t=f)
t, ts = z(256, 128), z(1, 256, t=f)
lt, lts = z(256, 8192), z(64, 256, t=f)
outs = [[z(40, 256, t=f), z(700, 4736, t=f), z(40, 512, t=f), z(256, 256, t=f), z(256, 256, t=f)] for _ in range(4)]
sps = [z(256) for _ in range(4)]
da, das = z(40, 256), z(40, 2, t=f)
streams = [torch.cuda.Stream() for _ in range(4)]
torch.cuda.synchronize()
start, errors = threading.Barrier(4), []

def work(i):
    try:
        torch.cuda.set_device(0)
        st, sp, o = streams[i], sps[i], outs[i]
        start.wait()
        calls = [lambda: M.gemm_fp8(a, s, w, ws, None, o[0], sp, st), lambda: M.gemm_fp8(big, bs, bw, bws, None, o[1], sp, st),
                 lambda: M.gemm_fp8_dgrad(da, das, w, ws, None, o[2], sp, st),
                 lambda: M.gemm_fp8_wgrad(t, ts, t, ts, None, 100, o[3], False, sp, st),
                 lambda: M.gemm_fp8_wgrad(lt, lts, lt, lts, None, 8192, o[4], False, sp, st)]
        for c in range(len(calls)):
            calls[(c + i) % len(calls)]()
    except BaseException as e:
        errors.append(e)

ts_ = [threading.Thread(target=work, args=(i,)) for i in range(4)]
[x.start() for x in ts_], [x.join() for x in ts_]
assert not errors, errors
torch.cuda.synchronize()
v = 2.0 ** -9  # code 1 is the smallest e4m3 value
for o in outs:
    for y, n in zip(o, (512, 256, 256, 128, 8192)):
        assert bool((y == n * v * v).all()), (n, y)
print("fine")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
