"""fp64 oracle of the softmax-attention operators, written from their formulas and
independent of the package: rotary positions, attention forward and backward, the
8-bit paged cache and the attention over it.  NumPy, token by token where that is
the plainest form.
"""

import math

import numpy as np


# ------------------------------------------------------------------ rotary

def rotary_freqs(rot, base=10000.0, scaling="none", factor=1.0, trained=0, beta_fast=32.0, beta_slow=1.0):
    """(inverse frequencies, scale): base^(-2i/rot), scaled for longer contexts."""
    out, scale = [], 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            # index at which a channel turns n times in the trained length
            idx = lambda n: rot / (2.0 * math.log(base)) * math.log(trained / (2.0 * math.pi * n))  # noqa: E731
            lo, hi = max(math.floor(idx(beta_fast)), 0), min(math.ceil(idx(beta_slow)), rot - 1)
            keep = 1.0 - min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = f * keep + f / factor * (1.0 - keep)
        out.append(f)
    if scaling == "yarn":
        scale = 0.1 * math.log(factor) + 1.0
    return np.array(out), scale


def rotary(x, positions, freqs, scale=1.0, interleaved=False, inverse=False):
    """x [B,T,H,D]; positions [B,T]; pairs (2i, 2i+1) or (i, i + rot/2) turned by positions * freqs."""
    rot = 2 * len(freqs)
    y = x.copy()
    first = np.arange(rot // 2) * 2 if interleaved else np.arange(rot // 2)
    second = first + 1 if interleaved else first + rot // 2
    ang = positions[:, :, None, None].astype(np.float64) * freqs
    c, s = np.cos(ang) * scale, np.sin(ang) * scale * (-1.0 if inverse else 1.0)
    u, w = x[..., first], x[..., second]
    y[..., first] = c * u - s * w
    y[..., second] = s * u + c * w
    return y


# ------------------------------------------------------------------ attention

def visible(ql, kl, causal, window):
    """[ql, kl] truth values: query i stands at key position i + kl - ql."""
    p = np.arange(ql)[:, None] + kl - ql
    j = np.arange(kl)[None]
    m = np.ones((ql, kl), bool)
    if causal:
        m &= j <= p
    if window:
        m &= j > p - window
    return m


def _softmax(x, seen):
    """Row softmax over the visible entries: (P, lse); rows without any give 0 and -inf."""
    x = np.where(seen, x, -np.inf)
    m = x.max(1, initial=-np.inf)
    with np.errstate(divide="ignore"):
        e = np.exp(x - np.where(np.isfinite(m), m, 0.0)[:, None])
        s = e.sum(1)
        return e / np.where(s > 0, s, 1.0)[:, None], np.where(np.isfinite(m), m, 0.0) + np.log(s)


def _lens(x, B, full):
    return [full] * B if x is None else [min(max(int(n), 0), full) for n in x]


def attn_forward(q, k, v, scale, causal=True, window=0, q_len=None, kv_len=None):
    """q [B,Tq,H,D]; k, v [B,Tk,HK,D] -> o [B,Tq,H,D], lse [B,H,Tq]."""
    B, Tq, H, D = q.shape
    Tk, HK = k.shape[1:3]
    o, lse = np.zeros(q.shape), np.full((B, H, Tq), -np.inf)
    for b, (ql, kl) in enumerate(zip(_lens(q_len, B, Tq), _lens(kv_len, B, Tk))):
        seen = visible(ql, kl, causal, window)
        for h in range(H):
            kh, vh = k[b, :kl, h * HK // H], v[b, :kl, h * HK // H]
            P, z = _softmax(scale * q[b, :ql, h] @ kh.T, seen)
            o[b, :ql, h], lse[b, h, :ql] = P @ vh, z
    return o, lse


def attn_backward(q, k, v, dout, scale, causal=True, window=0, q_len=None, kv_len=None):
    """Gradients of sum(dout * o): dq, dk, dv."""
    B, Tq, H, D = q.shape
    Tk, HK = k.shape[1:3]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b, (ql, kl) in enumerate(zip(_lens(q_len, B, Tq), _lens(kv_len, B, Tk))):
        seen = visible(ql, kl, causal, window)
        for h in range(H):
            g = h * HK // H
            qh, kh, vh, do = q[b, :ql, h], k[b, :kl, g], v[b, :kl, g], dout[b, :ql, h]
            P, _ = _softmax(scale * qh @ kh.T, seen)
            dP = do @ vh.T
            dS = P * (dP - (P * dP).sum(1, keepdims=True))
            dq[b, :ql, h] = scale * dS @ kh
            dk[b, :kl, g] += scale * dS.T @ qh
            dv[b, :kl, g] += P.T @ do
    return dq, dk, dv


# ------------------------------------------------------------------ the 8-bit cache

def e4m3(x):
    """Nearest value of 1 sign, 4 exponent (bias 7) and 3 mantissa bits, ties to even, saturating at 448."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, np.clip(x, -448.0, 448.0)))
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -60))), -6.0)
    step = 2.0 ** (e - 3.0)
    return np.where(np.isnan(x), np.nan, np.sign(x) * np.rint(a / step) * step)


def e4m3_value(code):
    """Value of 8-bit codes."""
    c = np.asarray(code).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where((c & 127) == 127, np.nan, np.where(c & 128, -v, v))


def page_scale(values):
    """Smallest power of two s >= 2^-100 with |x| <= 448 s over the finite values."""
    a = np.abs(values[np.isfinite(values)])
    top = a.max(initial=0.0)
    s = 2.0 ** -100
    if top > 448.0 * s:
        s = 2.0 ** math.ceil(math.log2(top / 448.0) - 1e-9)
        while top > 448.0 * s:
            s *= 2.0
        while top <= 448.0 * (s / 2.0):
            s /= 2.0
    return min(s, 2.0 ** 120)


class Cache:
    """Stored values (as multiples of the page's scale) of one kind, K or V:
    val [n_pages,HK,page,D], scale [n_pages,HK]."""

    def __init__(self, n_pages, HK, page, D):
        self.val = np.zeros((n_pages, HK, page, D))
        self.scale = np.ones((n_pages, HK))
        self.page = page

    def append(self, x, table, cache_len, new_len=None):
        """x [B,T,HK,D] behind the cache_len[b] tokens of each sequence."""
        B, T, HK, D = x.shape
        for b in range(B):
            first = max(int(cache_len[b]), 0)
            n = T if new_len is None else min(max(int(new_len[b]), 0), T)
            for p in range(first // self.page, -(-(first + n) // self.page)):
                lo, hi = max(first, p * self.page), min(first + n, (p + 1) * self.page)
                if lo >= hi or p >= table.shape[1] or not 0 <= table[b, p] < len(self.val):
                    continue
                pg, old = table[b, p], lo - p * self.page
                for h in range(HK):
                    new = x[b, lo - first:hi - first, h]
                    s = page_scale(new)
                    if old:
                        was = self.scale[pg, h]
                        s = max(s, was) if was == was else s      # a page never written may hold anything
                        if s > was:
                            self.val[pg, h, :old] = e4m3(self.val[pg, h, :old] * (was / s))
                    self.val[pg, h, old:hi - p * self.page] = e4m3(new / s)
                    self.scale[pg, h] = s

    def tokens(self, table_row, n):
        """The first n cached tokens of a sequence: values [n,HK,D] and which of them have a page."""
        HK, D = self.val.shape[1], self.val.shape[3]
        out, have = np.zeros((n, HK, D)), np.zeros(n, bool)
        for j in range(n):
            p = j // self.page
            if p < len(table_row) and 0 <= table_row[p] < len(self.val):
                pg = table_row[p]
                out[j] = self.val[pg, :, j % self.page] * self.scale[pg][:, None]
                have[j] = True
        return out, have


def attn_step(q, K, V, table, cache_len, scale, new_len=None, window=0):
    """q [B,Tq,H,D] over the caches K, V: query i at position cache_len[b] + i."""
    B, Tq, H, D = q.shape
    o = np.zeros(q.shape)
    for b in range(B):
        first = max(int(cache_len[b]), 0)
        nq = Tq if new_len is None else min(max(int(new_len[b]), 0), Tq)
        n = min(first + nq, table.shape[1] * K.page)
        k, have = K.tokens(table[b], n)
        v, _ = V.tokens(table[b], n)
        HK = k.shape[1]
        p, j = first + np.arange(nq)[:, None], np.arange(n)[None]
        seen = (j <= p) & have[None]
        if window:
            seen &= j > p - window
        for h in range(H):
            kh, vh = k[:, h * HK // H], v[:, h * HK // H]
            P, _ = _softmax(scale * q[b, :nq, h] @ kh.T, seen)
            o[b, :nq, h] = P @ vh
    return o
