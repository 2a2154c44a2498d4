"""CPU oracle of the operators that continue one prompt several times: pages of the 8-bit
cache, attention with a common prefix, selection over beams and vocabulary, states that
follow their parents.  One sequence after another, in fp64, written from the contract in
include/kda.h before the kernels.
"""

from __future__ import annotations

import numpy as np

from oracle import attn_oracle


def _names(e, n_pages):
    return 0 <= e < n_pages


# ------------------------------------------------------------------ pages

def fork(table, cache_len, parent, refs, page, keep=False):
    """(table_out, len_out, refs) of R requests; parent [R,K_out]."""
    table, parent, refs = np.asarray(table), np.asarray(parent), np.array(refs)
    R, K_out = parent.shape
    K_in, width = len(table) // max(R, 1), table.shape[1]
    out, lens = np.full((R * K_out, width), -1, np.int32), np.zeros(R * K_out, np.int32)
    for r in range(R):
        for c in range(K_out):
            p = parent[r, c]
            if not 0 <= p < K_in:
                continue
            n = max(int(cache_len[r * K_in + p]), 0)
            lens[r * K_out + c] = n
            used = min(-(-n // page), width)
            out[r * K_out + c, :used] = table[r * K_in + p, :used]
    for e in out[out >= 0]:
        if e < len(refs):
            refs[e] += 1
    if not keep:
        for e in table[table >= 0]:
            if e < len(refs):
                refs[e] -= 1
    return out, lens, refs


def reserve(table, cache_len, refs, T, page, new_len=None):
    """(table, refs, src, dst, info) after room was made for new_len[b] tokens."""
    table, refs = np.array(table), np.array(refs)
    B, width = table.shape
    free = [p for p in range(len(refs)) if refs[p] == 0]
    src, dst, lacking = np.full(B, -1, np.int32), np.full(B, -1, np.int32), 0
    for b in range(B):
        n = max(int(cache_len[b]), 0)
        new = T if new_len is None else min(max(int(new_len[b]), 0), T)
        for j in range(n // page, -(-(n + new) // page) if new else 0):
            if j >= width:
                break
            e, older = table[b, j], j == n // page and n % page != 0
            if _names(e, len(refs)):
                if refs[e] <= 1:
                    continue
                refs[e] -= 1
            elif older:
                continue
            at = free.pop(0) if free else -1
            table[b, j] = at
            if at < 0:
                lacking += 1
                continue
            refs[at] = 1
            if older:
                src[b], dst[b] = e, at
    return table, refs, src, dst, np.array([lacking, len(free)], np.int32)


def free(table, refs, page, keep_from=None, keep_to=None):
    """(table, refs) without the pages that hold no token of [keep_from, keep_to)."""
    table, refs = np.array(table), np.array(refs)
    for b in range(table.shape[0]):
        lo = 0 if keep_from is None else int(keep_from[b])
        hi = 0 if keep_to is None else int(keep_to[b])
        for j in range(table.shape[1]):
            if max(lo, j * page) < min(hi, (j + 1) * page):
                continue
            if _names(table[b, j], len(refs)):
                refs[table[b, j]] -= 1
            table[b, j] = -1
    return table, refs


def compact(table, refs):
    """(table, refs, remap, pairs of (from, to))."""
    table, refs = np.array(table), np.asarray(refs)
    used = [p for p in range(len(refs)) if refs[p] != 0]
    holes = [p for p in range(len(used)) if refs[p] == 0]
    remap = np.full(len(refs), -1, np.int32)
    pairs = []
    for p in used:
        remap[p] = p
        if p >= len(used):
            remap[p] = holes.pop(0)
            pairs.append((p, int(remap[p])))
    new_refs = np.zeros(len(refs), np.int32)
    for p in used:
        new_refs[remap[p]] = refs[p]
    for at in np.ndindex(table.shape):
        if _names(table[at], len(refs)):
            table[at] = remap[table[at]]
    return table, new_refs, remap, pairs


# ------------------------------------------------------------------ attention

def attn_shared(q, K, V, table, cache_len, group_first, prefix_len, scale, new_len=None, window=0):
    """attn_oracle.attn_step where the whole pages of the first prefix_len[g] tokens of a
    group's sequences are those that its first sequence's row names."""
    B, Tq, H, D = q.shape
    o = np.zeros(q.shape)
    cap = table.shape[1] * K.page
    for b in range(B):
        lead, prefix = b, 0
        for g in range(len(prefix_len)):
            if group_first[g] <= b < group_first[g + 1]:
                lead, prefix = int(group_first[g]), min(max(int(prefix_len[g]), 0), cap) // K.page * K.page
        first = max(int(cache_len[b]), 0)
        nq = Tq if new_len is None else min(max(int(new_len[b]), 0), Tq)
        n = min(first + nq, cap)
        (k0, have0), (k1, have1) = K.tokens(table[lead], n), K.tokens(table[b], n)
        v0, v1 = V.tokens(table[lead], n)[0], V.tokens(table[b], n)[0]
        common = np.arange(n) < prefix
        k, v = np.where(common[:, None, None], k0, k1), np.where(common[:, None, None], v0, v1)
        have = np.where(common, have0, have1)
        HK = k.shape[1]
        p, j = first + np.arange(nq)[:, None], np.arange(n)[None]
        seen = (j <= p) & have[None]
        if window:
            seen &= j > p - window
        for h in range(H):
            P, _ = attn_oracle._softmax(scale * q[b, :nq, h] @ k[:, h * HK // H].T, seen)
            o[b, :nq, h] = P @ v[:, h * HK // H]
    return o


# ------------------------------------------------------------------ beams

def beam_select(logits, scores, M, done=None, end=-1):
    """(scores [R,M], parent, token [R,M])."""
    logits = np.asarray(logits, np.float64)
    scores, done = (None if a is None else np.asarray(a) for a in (scores, done))
    R, K, V = logits.shape
    out, parent, token = np.full((R, M), -np.inf), np.full((R, M), -1, np.int32), np.full((R, M), -1, np.int32)
    for r in range(R):
        s, b, w, l = [], [], [], []
        for k in range(K):
            score = 0.0 if scores is None else float(scores[r, k])
            if not np.isfinite(score):
                continue
            if done is not None and done[r, k]:
                s.append(np.array([score])), b.append(np.array([k])), w.append(np.array([end])), l.append(np.zeros(1))
                continue
            x = logits[r, k]
            if np.isnan(x).any() or np.isposinf(x).any():
                continue
            at = np.flatnonzero(x > -np.inf)
            if len(at) == 0:
                continue
            top = x.max()
            y = score + (x[at] - (top + np.log(np.exp(x[at] - top).sum())))
            fits = np.abs(y) < 2.0 ** 128 - 2.0 ** 103      # what fp32 rounds to -infinity is none
            s.append(y[fits]), b.append(np.full(fits.sum(), k)), w.append(at[fits]), l.append(x[at[fits]])
        if not s:
            continue
        s, b, w, l = np.concatenate(s), np.concatenate(b), np.concatenate(w), np.concatenate(l)
        order = np.lexsort((w, -l, b, -s))[:M]      # a beam's logits decide where rounded scores do not
        n = len(order)
        out[r, :n], parent[r, :n], token[r, :n] = s[order], b[order], w[order]
    return out, parent, token


def state_reorder(state, parent):
    parent = np.asarray(parent)
    R, K_out = parent.shape
    rows = np.asarray(state)
    K_in = len(rows) // max(R, 1)
    out = np.zeros((R * K_out, *rows.shape[1:]), rows.dtype)
    for r in range(R):
        for c in range(K_out):
            if 0 <= parent[r, c] < K_in:
                out[r * K_out + c] = rows[r * K_in + parent[r, c]]
    return out
