"""Cases that measure the training-side operators of the MoE layer library.

Three operators, each in a plain form (elementary torch operations) and as the
library's entry points (``own``):

balance
    The load-balance loss of a router with its per-expert counts, and the
    gradient of the router logits: that of the loss plus that of the top-k
    weights.  With P = softmax(logits) over the E experts, c_e the number of
    assignments to expert e and n the number of tokens that count,
        f_e = E c_e / (k n),   loss = coef * sum_e f_e * (1/n) sum_t P[t][e],
        dlogits[t][e] = dloss coef / n * P[t][e] (f_e - sum_j f_j P[t][j])
                        + (the top-k softmax's gradient for dw).
product, product_dx, product_dw
    The FP8 e4m3 matrix product with one scale per block of 128, over all rows
    or over each expert's interval of rows, and its two gradients:
        y  = x W^T    x per 1x128 along K,   W [N][K] per 128x128
        dx = dy W     dy per 1x128 along N,  the same W
        dw = dy^T x   dy and x per 128 tokens of one column
    x and dy arrive in bf16 and are quantised in the call: s = fp32(amax)/448
    (1 for a block of zeros), q = e4m3 of fp32(v / s).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _balance(name, T, E, k, renorm=True, mask=0.0, skew=False, weights=True):
    return {"name": name, "op": "balance", "T": T, "E": E, "k": k, "renorm": renorm, "mask": mask,
            "skew": skew, "weights": weights}


def _product(name, op, M, N, K, G=0, out="bf16"):
    # G == 0: one weight matrix for all rows; G > 0: G experts, each with its interval of rows
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "G": G, "out": out}


def listed():
    return [
        # one decode-sized step of the 256-expert router
        _balance("balance_64", 64, 256, 8),
        # the skewed workload: Zipf-biased logits, eight experts never selected
        _balance("balance_skew_16384", 16384, 256, 8, skew=True),
        # padded batch, odd sizes, weights not renormalised
        _balance("balance_padded_10007", 10007, 60, 4, renorm=False, mask=0.15),
        # a long accumulated batch, the loss's own gradient alone
        _balance("balance_131072", 131072, 256, 8, mask=0.01, weights=False),
        # single token through an FP8 projection: the weight read bounds it
        _product("product_token", "product", 1, 6144, 2048),
        # a decode batch
        _product("product_64", "product", 64, 4096, 6144),
        # a prefill batch: the tensor cores bound it
        _product("product_8192", "product", 8192, 4096, 6144),
        # one rank's 32 experts, rows spread unevenly, rows as the combine reads them
        _product("product_experts", "product", 8192, 4096, 6144, G=32, out="f16"),
        # input gradient of the down projection
        _product("dx_4096", "product_dx", 4096, 6144, 2048),
        # small experts with ragged row counts, FP32 gradient
        _product("dx_experts", "product_dx", 3001, 1408, 640, G=16, out="f32"),
        # weight gradients: dense, and experts of which some get no row
        _product("dw_8192", "product_dw", 8192, 4096, 6144, out="f32"),
        _product("dw_experts", "product_dw", 5003, 2048, 1408, G=32, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["balance", "balance", "product", "product", "product_dx", "product_dw"])
    if op == "balance":
        E = rng.choice([rng.randint(2, 256), 256, 64])
        return {"op": op, "T": _log_int(rng, 1, 100000), "E": E, "k": rng.randint(1, min(8, E)),
                "renorm": rng.random() < 0.7, "mask": rng.choice([0.0, 0.0, 0.1, 0.9]),
                "skew": rng.random() < 0.4, "weights": rng.random() < 0.7}
    N, K = 128 * _log_int(rng, 1, 48), 128 * _log_int(rng, 1, 48)
    G = 0 if rng.random() < 0.5 else _log_int(rng, 1, 40)
    # at most the work of the largest listed product, and weights of at most 32 x 4096 x 6144
    M = _log_int(rng, 1, 8192)
    G = min(G, 32 * 4096 * 6144 // (N * K))
    out = "f32" if op == "product_dw" else rng.choice(["bf16", "bf16", "f16", "f32"])
    return {"op": op, "M": M, "N": N, "K": K, "G": G, "out": out}


def work(case):
    if case["op"] == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        nbytes = 2 * T * E * 4 + T * k * 4 + (2 * T * k * 4 if case["weights"] else 0)
        nbytes += (T if case["mask"] else 0) + 8 * E
        return {"bytes": nbytes, "flops": 10.0 * T * E}
    M, N, K, G = case["M"], case["N"], case["K"], max(1, case["G"])
    size = 4 if case["out"] == "f32" else 2
    scales = G * (N // BLOCK) * (K // BLOCK) * 4
    if case["op"] == "product":
        nbytes = 2 * M * K + min(G, M) * N * K + scales + size * M * N
    elif case["op"] == "product_dx":
        nbytes = 2 * M * N + min(G, M) * N * K + scales + size * M * K
    else:
        nbytes = 2 * M * (N + K) + size * G * N * K
    return {"bytes": nbytes, "flops": 2.0 * M * N * K}


# ------------------------------------------------------------------ inputs
def _group_rows(case, seed):
    """Rows of each expert: a Zipf-like split of M over G, in a shuffled order."""
    G, M = case["G"], case["M"]
    if not G:
        return None
    rng = np.random.RandomState(seed % (1 << 31))
    p = 1.0 / np.arange(1, G + 1) ** 0.7
    return rng.multinomial(M, rng.permutation(p / p.sum()))


def _quantised_weights(gen, G, N, K):
    """Weights as they stand in memory: e4m3 codes (bytes) and one scale per 128x128."""
    w = torch.randn((G, N // BLOCK, BLOCK, K // BLOCK, BLOCK), device="cuda", generator=gen,
                    dtype=torch.bfloat16)
    w *= K ** -0.5
    s = w.abs().amax(dim=(2, 4)).float() / 448.0
    q = torch.empty((G, N, K), dtype=torch.uint8, device="cuda")
    q.copy_((w / s[:, :, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            .view(torch.uint8).view(G, N, K))
    return q, s.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        logits = torch.randn((T, E), device="cuda", generator=gen)
        if case["skew"]:
            rank = torch.randperm(E, device="cuda", generator=gen).float() + 1.0
            bias = 0.38 * torch.log(rank ** -1.2 / (rank ** -1.2).sum())
            logits += torch.where(rank > E - E // 32, torch.full_like(bias, -1e4), bias)
        ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        top = logits.gather(1, ids.long())
        base = top if case["renorm"] else logits
        w = (torch.exp(top - base.amax(1, keepdim=True))
             / torch.exp(base - base.amax(1, keepdim=True)).sum(1, keepdim=True))
        dw = torch.randn((T, k), device="cuda", generator=gen) / T if case["weights"] else None
        mask = None
        if case["mask"]:
            mask = (torch.rand(T, device="cuda", generator=gen) >= case["mask"]).to(torch.uint8)
        return {"case": case, "logits": logits, "ids": ids, "w": w, "dw": dw, "mask": mask,
                "dloss": torch.ones(1, device="cuda"), "coef": 0.01,
                "loss": torch.empty(1, device="cuda"),
                "counts": torch.empty(E, dtype=torch.int32, device="cuda"),
                "prob_mean": torch.empty(E, device="cuda"),
                "tokens": torch.empty(1, dtype=torch.int32, device="cuda"),
                "dlogits": torch.empty_like(logits)}
    M, N, K, G = case["M"], case["N"], case["K"], max(1, case["G"])
    sizes = _group_rows(case, seed)
    state = {"case": case, "offsets": None, "group": None, "inside": None, "longest": M}
    if sizes is not None:
        ends = np.concatenate([[0], np.cumsum(sizes)])
        group = np.repeat(np.arange(G), sizes)
        state["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        state["group"] = torch.tensor(group, device="cuda")
        state["inside"] = torch.tensor(np.arange(M) - ends[group], device="cuda")
        state["longest"] = int(sizes.max())
    if case["op"] != "product":
        dy = torch.randn((M, N), device="cuda", generator=gen, dtype=torch.bfloat16) * 1e-3
        state["dy"] = dy
    if case["op"] != "product_dx":
        x = torch.randn((M, K), device="cuda", generator=gen, dtype=torch.bfloat16)
        x[:, :: max(1, K // 5)] *= 20.0  # a few channels stand out
        state["x"] = x
    if case["op"] == "product_dw":
        state["out"] = torch.empty((G, N, K), device="cuda")
    else:
        state["w_q"], state["w_s"] = _quantised_weights(gen, G, N, K)
        cols = N if case["op"] == "product" else K
        state["out"] = torch.empty((M, cols), dtype=DTYPES[case["out"]], device="cuda")
    return state


# ------------------------------------------------------------------ plain forms
def _softmax(l):
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_balance(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    keep = torch.ones(T, device="cuda") if s["mask"] is None else (s["mask"] != 0).float()
    P = _softmax(s["logits"]) * keep[:, None]
    ids = s["ids"].long()
    counts = torch.zeros(E, dtype=torch.int32, device="cuda").index_add_(
        0, ids.reshape(-1), keep.to(torch.int32).repeat_interleave(k))
    tokens = keep.to(torch.int32).sum(dtype=torch.int32).reshape(1)
    n = tokens.clamp(min=1).float()
    f = counts.double() * (E / (k * n.double()))
    prob_mean = (P.double().sum(0) / n).float()
    loss = s["coef"] * (f * prob_mean.double()).sum().float().reshape(1)
    # f - sum_j f_j P_j with f - 1 in the place of f (the P sum to 1): f is near 1, and 32 bits
    # would lose the difference
    f1 = (f - 1.0).float()
    d = (s["dloss"] * s["coef"] / n) * P * (f1 - (P * f1).sum(1, keepdim=True))
    if s["dw"] is not None:
        dw, w = s["dw"] * keep[:, None], s["w"]
        if c["renorm"]:
            d = d.scatter_add(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
        else:
            g = torch.zeros_like(P).scatter_add(1, ids, dw)
            d = d + P * (g - (w * dw).sum(1, keepdim=True))
    return {"loss": loss, "counts": counts, "prob_mean": prob_mean, "tokens": tokens, "dlogits": d}


def _scale(a):
    # a tensor divisor: a scalar one may become a product with its reciprocal, another rounding
    return torch.where(a == 0, 1.0, a / torch.full_like(a, 448.0))


def _e4m3(v, s):
    return (v / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()


def _through_fp8_rows(x):
    """x quantised per 1x128 of a row and taken back, in FP32."""
    b = x.float().view(x.shape[0], -1, BLOCK)
    a = b.abs().amax(2, keepdim=True)
    s = _scale(a)
    return (_e4m3(b, s) * s).view(x.shape)


def _through_fp8_tokens(x):
    """x [G][rows][C] quantised per 128 rows of a column and taken back, in FP32."""
    b = x.float().view(x.shape[0], -1, BLOCK, x.shape[2])
    a = b.abs().amax(2, keepdim=True)
    s = _scale(a)
    return (_e4m3(b, s) * s).view(x.shape)


def _weights(s):
    q, sc = s["w_q"], s["w_s"]
    G, N, K = q.shape
    v = q.view(torch.float8_e4m3fn).float().view(G, N // BLOCK, BLOCK, K // BLOCK, BLOCK)
    return (v * sc[:, :, None, :, None]).view(G, N, K)


def _spread(s, v, rows):
    """Rows [M][C] -> [G][rows][C], each expert's from its own start, zeros behind them."""
    G = max(1, s["case"]["G"])
    p = torch.zeros((G, rows, v.shape[1]), dtype=v.dtype, device=v.device)
    if s["group"] is None:
        p[0, : v.shape[0]] = v
    else:
        p[s["group"], s["inside"]] = v
    return p


def _plain_product(s):
    op = s["case"]["op"]
    if op == "product_dw":
        rows = -(-s["longest"] // BLOCK) * BLOCK
        dy = _through_fp8_tokens(_spread(s, s["dy"], rows))
        x = _through_fp8_tokens(_spread(s, s["x"], rows))
        return torch.bmm(dy.transpose(1, 2), x)
    a = _through_fp8_rows(s["x"] if op == "product" else s["dy"])
    W = _weights(s)
    W = W.transpose(1, 2) if op == "product" else W
    if s["group"] is None:
        return (a @ W[0]).to(s["out"].dtype)
    y = torch.bmm(_spread(s, a, s["longest"]), W)
    return y[s["group"], s["inside"]].to(s["out"].dtype)


# ------------------------------------------------------------------ the library's calls
def _own_balance(s):
    import expert_layer_dual_b200.moe as M
    c = s["case"]
    if "ws" not in s:  # kept by the program that calls it step after step
        s["ws"] = torch.empty(M.balance_workspace_bytes(c["T"], c["E"]), dtype=torch.uint8,
                              device="cuda")
    M.balance_loss(s["logits"], s["ids"], s["mask"], s["coef"], s["loss"], s["counts"],
                   s["prob_mean"], s["tokens"], s["ws"])
    M.route_backward(s["logits"], s["ids"], s["w"], s["dw"], s["mask"], c["renorm"], s["dloss"],
                     s["coef"], s["counts"], s["tokens"], s["dlogits"])
    return {k: s[k] for k in ("loss", "counts", "prob_mean", "tokens", "dlogits")}


def _own_product(s):
    import expert_layer_dual_b200.moe as M
    c = s["case"]
    m, N, K, G = c["M"], c["N"], c["K"], max(1, c["G"])

    def buffers(name, q_shape, s_shape):
        if name not in s:
            s[name] = (torch.empty(q_shape, dtype=torch.uint8, device="cuda"),
                       torch.empty(s_shape, dtype=torch.float32, device="cuda"))
        return s[name]

    if "ws" not in s:
        s["ws"] = torch.empty(256, dtype=torch.uint8, device="cuda")
    if c["op"] == "product_dw":
        rows = M.fp8_token_rows(m, G)
        dyt, dyt_s = buffers("dy_t", (N, rows), (rows // BLOCK, N))
        xt, xt_s = buffers("x_t", (K, rows), (rows // BLOCK, K))
        M.quantize_fp8_tokens(s["dy"], s["offsets"], dyt, dyt_s)
        M.quantize_fp8_tokens(s["x"], s["offsets"], xt, xt_s)
        M.gemm_fp8_wgrad(dyt, dyt_s, xt, xt_s, s["offsets"], m, s["out"], False, s["ws"])
        return s["out"]
    a = s["x"] if c["op"] == "product" else s["dy"]
    aq, a_s = buffers("a_q", a.shape, (m, a.shape[1] // BLOCK))
    M.quantize_act_fp8(a, aq, a_s)
    gemm = M.gemm_fp8 if c["op"] == "product" else M.gemm_fp8_dgrad
    gemm(aq, a_s, s["w_q"], s["w_s"], s["offsets"], s["out"], s["ws"])
    return s["out"]


def run(state):
    if state["case"]["op"] == "balance":
        return _own_balance(state) if own else _plain_balance(state)
    return _own_product(state) if own else _plain_product(state)


# ------------------------------------------------------------------ the definition in 64 bits
def _round_e4m3(v):
    """float32 -> the nearest e4m3 value (ties to even), limited to +-448, as float64."""
    v = v.double().clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(v / step) * step


def _blocks64(x, axis):
    """The values that x's e4m3 codes stand for, blocks of 128 along `axis` (the last block may be short)."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[axis], BLOCK):
        part = x.narrow(axis, at, min(BLOCK, x.shape[axis] - at)).float()
        scale = part.abs().amax(axis, keepdim=True)
        scale = torch.where(scale == 0, torch.ones_like(scale), torch.div(scale, torch.full_like(scale, 448.0)))
        out.narrow(axis, at, part.shape[axis]).copy_(_round_e4m3(part / scale) * scale.double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        E, k, coef = case["E"], case["k"], s["coef"]
        keep = torch.ones(case["T"], dtype=torch.bool, device="cuda") if s["mask"] is None \
            else s["mask"].bool()
        P = torch.softmax(s["logits"].double(), 1)
        ids = s["ids"].long()
        counts = torch.bincount(ids[keep].reshape(-1), minlength=E)
        n = int(keep.sum())
        f = counts.double() * E / (k * max(1, n))
        mean = P[keep].sum(0) / max(1, n)
        d = coef / max(1, n) * P * (f - (P @ f)[:, None])
        if s["dw"] is not None:
            top = P.gather(1, ids)
            w = top / top.sum(1, keepdim=True) if case["renorm"] else top
            dot = (w * s["dw"].double()).sum(1, keepdim=True)
            if case["renorm"]:
                d = d + torch.zeros_like(P).scatter_add(1, ids, w * (s["dw"].double() - dot))
            else:
                d = d - P * dot + torch.zeros_like(P).scatter_add(1, ids, w * s["dw"].double())
        return {"loss": (coef * (f * mean).sum()).reshape(1), "counts": counts.to(torch.int32),
                "prob_mean": mean, "tokens": torch.tensor([n], dtype=torch.int32),
                "dlogits": d * keep[:, None]}
    M, G = case["M"], max(1, case["G"])
    ends = [0, M] if s["offsets"] is None else s["offsets"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for g in range(G):
        a, b = ends[g], ends[g + 1]
        if a == b:
            continue
        if case["op"] == "product_dw":
            out[g] = _blocks64(s["dy"][a:b], 0).T @ _blocks64(s["x"][a:b], 0)
            continue
        W = s["w_q"][g].view(torch.float8_e4m3fn).double()
        W *= s["w_s"][g].double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
        if case["op"] == "product":
            out[a:b] = _blocks64(s["x"][a:b], 1) @ W.T
        else:
            out[a:b] = _blocks64(s["dy"][a:b], 1) @ W
    return out
