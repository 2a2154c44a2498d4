"""Error bounds of the attention operators, from their arithmetic.

u is half a step of a type (relative): 2^-24 for fp32, 2^-8 for bf16.  A dot
product of n terms accumulated in fp32 is off by at most (n + 2) 2^-24 times the
sum of the terms' magnitudes.  Scores are such dot products of exact inputs, so a
probability is off by the factor exp(e) with e the score's error plus that of lse;
in bf16 it is rounded once more (u) before its product with v, dS likewise before
its products, and every output is rounded once to the type.  An exponential below
2^-126 (TINY) underflows to zero, so each probability may also be off by that much.
"""

import numpy as np
import torch

from oracle import attn_oracle as ora

F32, BF16 = torch.float32, torch.bfloat16
U24 = 2.0 ** -24
TINY = 2.0 ** -126
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def heads(x, H):
    """[T,HK,D] repeated to [H,T,D]."""
    return np.repeat(x.transpose(1, 0, 2), H // x.shape[1], axis=0)


def fwd_bounds(q, k, v, dtype, scale, causal=True, window=0, q_len=None, kv_len=None):
    """(o, lse, bound of o, bound of lse) of attn_forward in `dtype`."""
    o, lse = ora.attn_forward(q, k, v, scale, causal, window, q_len, kv_len)
    bo, bl = np.zeros(o.shape), np.zeros(lse.shape)
    B, Tq, H, D = q.shape
    for b, (ql, kl) in enumerate(zip(ora._lens(q_len, B, Tq), ora._lens(kv_len, B, k.shape[1]))):
        seen = ora.visible(ql, kl, causal, window)
        K, V = heads(k[b, :kl], H), heads(v[b, :kl], H)
        for h in range(H):
            P, _ = ora._softmax(scale * q[b, :ql, h] @ K[h].T, seen)
            e = score_error(q[b, :ql, h], K[h], scale, seen)
            n = kl + 64
            mass = P @ np.abs(V[h])
            under = TINY * np.abs(V[h]).sum(0)
            rel = np.expm1(2 * e)[:, None] + (2 * n + 8) * U24 + (U[dtype] if dtype == BF16 else 4 * U24)
            off = rel * mass + under
            bo[b, :ql, h] = off + U[dtype] * (np.abs(o[b, :ql, h]) + off)
            z = lse[b, h, :ql]
            bl[b, h, :ql] = e + (n + 8) * U24 + 4 * U24 * np.abs(np.where(np.isfinite(z), z, 0.0))
    return o, lse, bo, bl


def score_error(q, k, scale, seen):
    """Largest error of a visible score of each row, in units of the exponent: the
    dot product's, and four roundings (scale, log2 e, the fused subtraction, the
    maximum) of numbers of the score's size."""
    a = scale * (np.abs(q) @ np.abs(k).T)
    e = (q.shape[1] + 2 + 4 + 2) * U24 * np.where(seen, a, 0.0)
    return e.max(1, initial=0.0)


def bwd_bounds(q, k, v, dout, dtype, scale, causal=True, window=0, q_len=None, kv_len=None):
    """((dq, dk, dv), their bounds) of attn_backward from the operator's own o and lse."""
    grads = ora.attn_backward(q, k, v, dout, scale, causal, window, q_len, kv_len)
    o, lse, bo, bl = fwd_bounds(q, k, v, dtype, scale, causal, window, q_len, kv_len)
    out = [np.zeros(g.shape) for g in grads]
    B, Tq, H, D = q.shape
    u = U[dtype] if dtype == BF16 else 0.0
    for b, (ql, kl) in enumerate(zip(ora._lens(q_len, B, Tq), ora._lens(kv_len, B, k.shape[1]))):
        seen = ora.visible(ql, kl, causal, window)
        for h in range(H):
            g = h * k.shape[2] // H
            qh, kh, vh, do = q[b, :ql, h], k[b, :kl, g], v[b, :kl, g], dout[b, :ql, h]
            P, z = ora._softmax(scale * qh @ kh.T, seen)
            rel = np.expm1(score_error(qh, kh, scale, seen) + bl[b, h, :ql])[:, None] + 8 * U24
            dP = do @ vh.T
            de = (P * dP).sum(1, keepdims=True)
            e_dp = (D + 2) * U24 * (np.abs(do) @ np.abs(vh).T)
            e_de = ((np.abs(do) * (bo[b, :ql, h] + (D + 2) * U24 * np.abs(o[b, :ql, h]))).sum(1, keepdims=True))
            dS = P * (dP - de)
            e_ds = TINY * (1 + np.abs(dP - de) + e_dp + e_de) + P * (e_dp + e_de) * (1 + rel) + rel * np.abs(dS) + 4 * U24 * np.abs(dS)
            e_ds += u * (np.abs(dS) + e_ds)
            e_p = (rel + u * (1 + rel)) * P + TINY
            nq, nk = (ql + 66) * U24 * H // k.shape[2], (kl + 66) * U24
            aS = np.abs(dS) + e_ds
            out[0][b, :ql, h] += scale * (e_ds @ np.abs(kh) + nk * (aS @ np.abs(kh)))
            out[1][b, :kl, g] += scale * (e_ds.T @ np.abs(qh) + nq * (aS.T @ np.abs(qh)))
            out[2][b, :kl, g] += e_p.T @ np.abs(do) + nq * ((P + e_p).T @ np.abs(do))
    bounds = [x + (U[dtype] + 2 * U24) * (np.abs(g) + x) for x, g in zip(out, grads)]
    return grads, bounds


def check(got, want, bound, what):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fin = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fin), f"{what}: finite in different places"
    assert np.array_equal(got[~fin], want[~fin], equal_nan=True), f"{what}: non-finite values differ"
    bound = np.broadcast_to(bound, want.shape)
    over = np.abs(np.where(fin, got, 0) - np.where(fin, want, 0)) - bound - 1e-38
    worst = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert worst is None or over[worst] <= 0, f"{what}: {got[worst]} instead of {want[worst]} at {worst} (bound {bound[worst]:.3g})"
