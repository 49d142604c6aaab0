"""The training-side operators in 64 bits, from their formulas (plain PyTorch
FP64 on the CPU, nothing of the library): the balance loss with its counts and
the gradient of the router logits, and the FP8 block-128 product with its two
gradients.  Each float result comes with the sum of the magnitudes its terms
have, which the tests' rounding bounds are relative to."""
from __future__ import annotations

import torch


# ------------------------------------------------------------------ router
def softmax64(logits):
    """Row softmax; a row without any finite logit gives zeros."""
    l = logits.double()
    m = l.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(l - m)
    s = e.sum(1, keepdim=True)
    return torch.where(s > 0, e / s.clamp(min=1e-300), torch.zeros_like(e))


def balance(logits, ids, mask, coef):
    T, E = logits.shape
    k = ids.shape[1]
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    P = softmax64(logits[keep])
    flat = ids[keep].reshape(-1).long()
    flat = flat[(flat >= 0) & (flat < E)]
    counts = torch.bincount(flat, minlength=E)
    n = int(keep.sum())
    mean = P.sum(0) / max(n, 1)
    f = counts.double() * E / (k * max(n, 1))
    return {"loss": coef * float((f * mean).sum()), "counts": counts, "prob_mean": mean, "tokens": n}


def route_backward(logits, ids, w, dw, mask, renorm, dloss, coef, counts, n):
    """(dlogits, the sum of the magnitudes of each element's terms)."""
    T, E = logits.shape
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    P = torch.zeros((T, E), dtype=torch.float64)
    P[keep] = softmax64(logits[keep])
    d = torch.zeros_like(P)
    size = torch.zeros_like(P)
    if dw is not None:
        w64, dw64 = w.double(), dw.double()
        dot = (w64 * dw64).sum(1, keepdim=True)
        adot = (w64 * dw64.abs()).sum(1, keepdim=True)
        for j in range(ids.shape[1]):
            ok = (ids[:, j] >= 0) & (ids[:, j] < E)
            r = torch.nonzero(ok).reshape(-1)
            c = ids[ok, j].long()
            if renorm:
                d.index_put_((r, c), (w64[:, j: j + 1] * (dw64[:, j: j + 1] - dot))[ok, 0], accumulate=True)
                size.index_put_((r, c), (w64[:, j: j + 1] * (dw64[:, j: j + 1].abs() + adot))[ok, 0],
                                accumulate=True)
            else:
                d.index_put_((r, c), P[r, c] * dw64[ok, j], accumulate=True)
                size.index_put_((r, c), P[r, c] * dw64[ok, j].abs(), accumulate=True)
        if not renorm:
            d -= P * dot
            size += P * adot
    if dloss is not None and n > 0:
        f1 = counts.double() * E / (ids.shape[1] * n) - 1.0
        c = float(dloss) * coef / n
        d += c * P * (f1 - (P @ f1)[:, None])
        size += abs(c) * P * (f1.abs() + (P @ f1.abs())[:, None])
    d[~keep] = 0.0
    size[~keep] = 0.0
    return d, size


# ------------------------------------------------------------------ FP8 blocks
def quantise(v):
    """v [..., 128, ...] grouped along dim 1: (codes as float8, scale) with the
    scale and the quotient in FP32, as the format's rule says."""
    a = v.float().abs().amax(1, keepdim=True)
    s = torch.where(a == 0, torch.ones_like(a), a / torch.full_like(a, 448.0))
    return (v.float() / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s


def quantise_rows(x):
    """x [M, C] -> codes [M, C] (uint8), scales [M, C/128]."""
    M, C = x.shape
    q, s = quantise(x.reshape(M * (C // 128), 128, 1))
    return q.view(torch.uint8).reshape(M, C), s.reshape(M, C // 128)


def quantise_weights(w):
    """w [G, N, K] -> codes (uint8), scales [G, N/128, K/128]."""
    G, N, K = w.shape
    b = w.reshape(G, N // 128, 128, K // 128, 128).permute(0, 1, 3, 2, 4)
    q, s = quantise(b.reshape(-1, 128 * 128, 1))
    q = q.view(torch.uint8).reshape(G, N // 128, K // 128, 128, 128).permute(0, 1, 3, 2, 4)
    return q.reshape(G, N, K).contiguous(), s.reshape(G, N // 128, K // 128)


def quantise_tokens(x, offsets, R):
    """x [M, C] -> (codes [C, R], scales [R/128, C], number of blocks in use)."""
    M, C = x.shape
    q = torch.zeros((C, R), dtype=torch.uint8)
    s = torch.zeros((R // 128, C))
    b = 0
    ends = [0, M] if offsets is None else offsets.tolist()
    for lo, hi in zip(ends[:-1], ends[1:]):
        for r in range(lo, hi, 128):
            part = torch.zeros((128, C))
            part[: min(128, hi - r)] = x[r: min(r + 128, hi)].float()
            qq, ss = quantise(part.T.reshape(C, 128, 1))
            q[:, b * 128: (b + 1) * 128] = qq.view(torch.uint8).reshape(C, 128)
            s[b] = ss.reshape(C)
            b += 1
    return q, s, b


def values(q):
    return q.view(torch.float8_e4m3fn).double()


def rows64(q, s):
    return values(q) * s.double().repeat_interleave(128, 1)


def weights64(q, s):
    return values(q) * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)


def grouped(a64, w64, offsets, M, transpose):
    """a [M, .] times each group's matrix: (result, sum of magnitudes, rows covered)."""
    ends = [0, M] if offsets is None else offsets.tolist()
    cols = w64.shape[1] if transpose else w64.shape[2]
    out = torch.zeros((M, cols), dtype=torch.float64)
    size = torch.zeros_like(out)
    covered = torch.zeros(M, dtype=torch.bool)
    for g, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        W = w64[g].T if transpose else w64[g]
        out[lo:hi] = a64[lo:hi] @ W
        size[lo:hi] = a64[lo:hi].abs() @ W.abs()
        covered[lo:hi] = True
    return out, size, covered


def weight_gradient(dyt, dyts, xt, xts, offsets, M):
    """dw [G, N, K] and its sums of magnitudes from the token-block operands."""
    ends = [0, M] if offsets is None else offsets.tolist()
    a = values(dyt) * dyts.double().T.repeat_interleave(128, 1)
    b = values(xt) * xts.double().T.repeat_interleave(128, 1)
    out, size, at = [], [], 0
    for lo, hi in zip(ends[:-1], ends[1:]):
        n = (hi - lo + 127) // 128 * 128
        out.append(a[:, at: at + n] @ b[:, at: at + n].T)
        size.append(a[:, at: at + n].abs() @ b[:, at: at + n].abs().T)
        at += n
    return torch.stack(out), torch.stack(size)


def product_bound(size, blocks):
    """How far an FP32-accumulated block product may be from the exact sum.  The
    products of two e4m3 values are exact in FP32.  Each of a block's 128
    additions loses at most one unit in the last place (2^-23, truncation
    allowed for) of a partial sum that the block's magnitudes bound; the scale
    product, its product with the sum and the addition over blocks round once
    per block (2^-24 each)."""
    return size * (128 * 2.0 ** -23 + (blocks + 3) * 2.0 ** -24)


HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
