"""GPU parity of softmax attention, forward and backward, with the fp64 oracle, at
the sizes, lengths, masks and strides where tiles end; bounds in tests/attn_check.py."""

import numpy as np
import pytest
import torch

from gated_delta_rule_82_amd import kda
from oracle import attn_oracle as ora
from tests.attn_check import BF16, F32, bwd_bounds, check, fwd_bounds, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    kda.load()
    yield
    torch.cuda.synchronize()


def draw(B, Tq, Tk, H, HK, D, dtype, seed, packed=False):
    g = torch.Generator().manual_seed(seed)
    if packed and Tq == Tk:
        x = torch.randn(B, Tq, H + 2 * HK, D, generator=g).to(dtype).cuda()
        q, k, v = x[:, :, :H], x[:, :, H:H + HK], x[:, :, H + HK:]
    else:
        q, k, v = (torch.randn(B, t, h, D, generator=g).to(dtype).cuda() for t, h in ((Tq, H), (Tk, HK), (Tk, HK)))
    return q, k, v, torch.randn(B, Tq, H, D, generator=g).to(dtype).cuda()


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def run_both(q, k, v, do, dtype, what="", scale=None, ql=None, kl=None, poison=False, **kw):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    lens = dict(q_len=ints(ql), kv_len=ints(kl))
    ref = [np64(x) for x in (q, k, v, do)]
    if poison:  # what lies past the lengths is never read
        q, k, v, do = (x.clone() for x in (q, k, v, do))
        for b in range(q.shape[0]):
            for x, n in ((q, ql), (do, ql), (k, kl), (v, kl)):
                if n is not None:
                    x[b, max(n[b], 0):] = float("nan")
    o, lse = kda.attn_fwd(q, k, v, scale=scale, **lens, **kw)
    torch.cuda.synchronize()
    wo, wl, bo, bl = fwd_bounds(*ref[:3], dtype, scale, q_len=ql, kv_len=kl, **kw)
    check(o, wo, bo, f"{what} o")
    check(lse, wl, bl, f"{what} lse")
    if poison:
        o, lse = o.clone(), lse.clone()
        for b in range(q.shape[0]):
            if ql is not None:
                o[b, max(ql[b], 0):] = float("nan")
                lse[b, :, max(ql[b], 0):] = float("nan")
    g = kda.attn_bwd(q, k, v, o, lse, do, scale=scale, **lens, **kw)
    torch.cuda.synchronize()
    grads, bounds = bwd_bounds(*ref, dtype, scale, q_len=ql, kv_len=kl, **kw)
    for n, w, b in zip(("dq", "dk", "dv"), grads, bounds):
        check(g[n], w, b, f"{what} {n}")


SIZES = [(1, 1, 1, 1, 1), (2, 1, 37, 4, 2), (1, 33, 33, 3, 3), (2, 65, 64, 2, 1), (1, 64, 129, 8, 2), (3, 20, 7, 5, 1),
         (1, 200, 200, 2, 2)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("B,Tq,Tk,H,HK", SIZES)
def test_attn_matches_oracle(dtype, D, B, Tq, Tk, H, HK):
    x = draw(B, Tq, Tk, H, HK, D, dtype, 100 * D + Tq, packed=True)
    for causal, window in ((True, 0), (False, 0), (True, 5), (False, 40)):
        run_both(*x, dtype, f"causal {causal} window {window}", causal=causal, window=window)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 17)])
def test_attn_lengths(dtype, causal, window):
    B, T = 6, 150
    x = draw(B, T, T, 4, 2, 64, dtype, 7, packed=True)
    run_both(*x, dtype, "equal lengths", ql=[150, 1, 0, 64, 65, 127], kl=[150, 1, 0, 64, 65, 127], poison=True,
             causal=causal, window=window)
    # no key at all, fewer keys than queries, out of range (clamped)
    run_both(*x, dtype, "unequal lengths", ql=[150, 10, 3, 70, 200, 128], kl=[3, 0, 150, 65, 150, -4], poison=True,
             causal=causal, window=window)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq,H,HK", [(1, 8, 2), (3, 4, 4), (16, 8, 1), (40, 6, 2)])
def test_attn_split_key_axis(dtype, Tq, H, HK):
    """Few rows over a long key axis: several workgroups and a join."""
    B, Tk = 2, 2600
    assert kda.attn_fwd_workspace_bytes(B, Tq, Tk, H, HK, 64, dtype) > 0
    q, k, v, _ = draw(B, Tq, Tk, H, HK, 64, dtype, Tq)
    for kw, ql, kl in ((dict(causal=True, window=0), None, None), (dict(causal=False, window=0), [Tq, Tq], [2600, 9]),
                       (dict(causal=True, window=700), [Tq, Tq // 2], [2600, 1300])):
        o, lse = kda.attn_fwd(q, k, v, q_len=ints(ql), kv_len=ints(kl), **kw)
        torch.cuda.synchronize()
        wo, wl, bo, bl = fwd_bounds(np64(q), np64(k), np64(v), dtype, 64 ** -0.5, q_len=ql, kv_len=kl, **kw)
        check(o, wo, bo, f"o {kw}")
        check(lse, wl, bl, f"lse {kw}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,H,HK,T", [(128, 16, 16, 150), (64, 32, 16, 97), (16, 48, 16, 130), (128, 16, 16, 420), (32, 16, 16, 513)])
def test_attn_enough_heads_to_fill_the_card(dtype, D, H, HK, T):
    """Grids of at least 256 workgroups: the forms with whole tiles of keys and rows."""
    x = draw(16, T, T, H, HK, D, dtype, D, packed=True)
    n = [T - 9 * b for b in range(16)]
    for kw, lens in ((dict(causal=True, window=0), {}), (dict(causal=True, window=40), dict(ql=n, kl=n))):
        run_both(*x, dtype, f"D {D} {kw}", **lens, **kw)


@pytest.mark.parametrize("D,H,HK,Tq,Tk", [(128, 48, 16, 90, 333), (64, 16, 16, 300, 70), (32, 32, 16, 1, 260)])
def test_attn_full_grids_of_unequal_lengths(D, H, HK, Tq, Tk):
    """The same with shared heads, more or fewer keys than queries, and empty sequences among them."""
    x = draw(16, Tq, Tk, H, HK, D, BF16, D + 1)
    ql = [Tq, 0, 1, Tq // 2] * 4
    kl = [Tk, Tk, 1, 0, Tk // 3, Tk, 65, 64] * 2
    for kw in (dict(causal=True, window=0), dict(causal=True, window=33), dict(causal=False, window=0)):
        run_both(*x, BF16, f"D {D} {kw}", ql=[min(n, Tq) for n in ql], kl=[min(n, Tk) for n in kl], **kw)


def run_heads(q, k, v, do, picks, ql, kl, what, **kw):
    """Both directions on the whole batch; the oracle on the (sequence, key/value head) pairs of `picks`."""
    D, G = q.shape[-1], q.shape[2] // k.shape[2]
    scale = D ** -0.5
    lens = dict(q_len=ints(ql), kv_len=ints(kl))
    o, lse = kda.attn_fwd(q, k, v, scale=scale, **lens, **kw)
    g = kda.attn_bwd(q, k, v, o, lse, do, scale=scale, **lens, **kw)
    torch.cuda.synchronize()
    for b, h in picks:
        qs, ks = (slice(b, b + 1), slice(None), slice(h * G, (h + 1) * G)), (slice(b, b + 1), slice(None), slice(h, h + 1))
        x = [np64(t[s]) for t, s in ((q, qs), (k, ks), (v, ks), (do, qs))]
        one = dict(q_len=None if ql is None else [ql[b]], kv_len=None if kl is None else [kl[b]], **kw)
        wo, wl, bo, bl = fwd_bounds(*x[:3], BF16, scale, **one)
        check(o[qs], wo, bo, f"{what} {b} {h} o")
        check(lse[b:b + 1, h * G:(h + 1) * G], wl, bl, f"{what} {b} {h} lse")
        grads, bounds = bwd_bounds(*x, BF16, scale, **one)
        for n, w, bound, s in zip(("dq", "dk", "dv"), grads, bounds, (qs, ks, ks)):
            check(g[n][s], w, bound, f"{what} {b} {h} {n}")


@pytest.mark.parametrize("D,B,Tq,Tk,H,HK,kw,ql,kl", [
    (128, 2, 4100, 4100, 16, 8, dict(causal=True, window=0), None, None),
    (128, 2, 4130, 4200, 16, 8, dict(causal=True, window=4099), [4130, 4001], [4200, 4200]),
    (128, 4, 700, 700, 64, 64, dict(causal=False, window=0), [700, 0, 33, 690], [700, 650, 700, 0]),
    (128, 2, 2111, 1000, 16, 16, dict(causal=False, window=0), [2111, 1990], [1000, 961]),
    (128, 2, 2111, 1000, 32, 16, dict(causal=True, window=2060), [2111, 5], [30, 1000]),
    (64, 4, 520, 777, 64, 64, dict(causal=False, window=600), [520, 300, 1, 257], [777, 700, 777, 64]),
    (64, 2, 2100, 2100, 16, 16, dict(causal=True, window=0), [2100, 2050], [2100, 2060]),
    (64, 3, 2100, 2100, 12, 3, dict(causal=True, window=0), [1031, 2050, 2100], [1040, 2060, 2100]),
    (64, 2, 2100, 2100, 32, 8, dict(causal=True, window=1500), [2100, 1999], [2100, 2010]),
    (128, 2, 2052, 2052, 16, 16, dict(causal=True, window=0), [2052, 2050], [2052, 2049]),
    (128, 4, 4100, 4099, 16, 4, dict(causal=True, window=0), [4100, 2000, 777, 3001], [4099, 2500, 777, 3000]),
])
def test_attn_long_sequences_that_fill_the_card(D, B, Tq, Tk, H, HK, kw, ql, kl):
    x = draw(B, Tq, Tk, H, HK, D, BF16, D + Tq, packed=True)
    run_heads(*x, [(b, b * (HK - 1) // max(B - 1, 1)) for b in range(B)], ql, kl, f"D {D} {kw}", **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 30.0])
def test_attn_scales(dtype, scale):
    """From nearly uniform rows to one key per row; large scores on both sides of zero."""
    q, k, v, do = draw(1, 70, 70, 2, 2, 32, dtype, 11)
    run_both(q, k, v, do, dtype, f"scale {scale}", scale=scale, causal=True, window=0)


@pytest.mark.parametrize("cut", [1, 13, 40])
def test_attn_bwd_over_parts_of_the_keys(cut):
    """Key axis in two calls with the whole's o and lse, short parts (whose row values come from
    their keys where these are all there is) and longer ones."""
    q, k, v, do = draw(2, 50, 70, 4, 2, 64, F32, 22)
    o, lse = kda.attn_fwd(q, k, v, causal=False)
    parts = [kda.attn_bwd(q, k[:, s].contiguous(), v[:, s].contiguous(), o, lse, do, causal=False)
             for s in (slice(0, cut), slice(cut, 70))]
    torch.cuda.synchronize()
    grads, bounds = bwd_bounds(*[np64(x) for x in (q, k, v, do)], F32, 64 ** -0.5, causal=False, window=0)
    # each part's terms are among the whole's: its error is within the whole's bound
    check(parts[0]["dq"] + parts[1]["dq"], grads[0], 2 * bounds[0], "dq")
    for i, n in ((1, "dk"), (2, "dv")):
        check(torch.cat([p[n] for p in parts], 1), grads[i], bounds[i], n)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attn_gradients_of_rows_with_few_keys_are_as_precise_as_others(dtype):
    """dS nearly vanishes where a row sees two or three keys; its error is measured against the gradients,
    not against the terms that cancel.  bf16: a rounding of dS and one of the result, each eps / 2 / sqrt(3)
    in the mean square at most (uniform up to half a step of a value's binade), 0.82 eps / 2 together.  fp32:
    a dozen roundings (the chains of q.k and dout.v, lse, the exponential, the sums)."""
    most = 1.0 if dtype is BF16 else 12.0
    for T, window in ((2, 0), (3, 0), (40, 2), (300, 3), (200, 0)):
        q, k, v, do = draw(4, T, T, 8, 4, 64, dtype, 23 + T)
        o, lse = kda.attn_fwd(q, k, v, window=window)
        g = kda.attn_bwd(q, k, v, o, lse, do, window=window)
        torch.cuda.synchronize()
        grads, _ = bwd_bounds(*[np64(x) for x in (q, k, v, do)], dtype, 64 ** -0.5, causal=True, window=window)
        for n, w in zip(("dq", "dk", "dv"), grads):
            e = np.linalg.norm(np64(g[n]) - w) / np.linalg.norm(w)
            assert e < most * torch.finfo(dtype).eps / 2, (T, window, n, e)


def peaked(n, rest, dtype, seed):
    """70 keys whose first n hold all but about `rest` of every row's mass; the others' values are thirty
    times as large, so that what they add to delta shows."""
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(2, t, h, 64, generator=g) for t, h in ((24, 4), (70, 2), (70, 2), (24, 4)))
    q, k = 0.3 * q, 0.3 * k
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[:, :n, :, 0] = float(np.log((70 - n) / (n * rest)))
    v[:, n:] *= 30.0
    return [x.to(dtype).cuda() for x in (q, k, v, do)]


def part_terms(q, k, v, do, keys, scale, dtype):
    """The gradients' terms of some of the keys in 64 bits, and the size of their error.  Sums of exact
    products are off by a dozen fp32 roundings of the products' size in the mean square (their signs are
    random), an exponential by as many of 1 + |score|; o, and with it delta, in bf16 by its own rounding and
    that of the probabilities; dS and every result is rounded to the type once."""
    r, u = 12 * 2.0 ** -24, torch.finfo(dtype).eps / 2
    out = [[np.zeros(q.shape), np.zeros(k[:, keys].shape), np.zeros(k[:, keys].shape)] for _ in range(2)]
    least, G = 1.0, q.shape[2] // k.shape[2]
    for b in range(q.shape[0]):
        for h in range(q.shape[2]):
            qh, kh, vh, dh = q[b, :, h], k[b, :, h // G], v[b, :, h // G], do[b, :, h]
            x = scale * qh @ kh.T
            P = np.exp(x - x.max(1, keepdims=True))
            P /= P.sum(1, keepdims=True)
            dP = dh @ vh.T
            delta = (P * dP).sum(1, keepdims=True)
            e_delta = (r + (2 * u if dtype is BF16 else 0)) * np.linalg.norm(dh * (P @ np.abs(vh)), axis=1, keepdims=True)
            P, dP, kh, vh = P[:, keys], dP[:, keys], kh[keys], vh[keys]
            least = min(least, 1 - P.sum(1).max())
            dS = P * (dP - delta)
            rel = r * (1 + np.abs(x).max()) + (u if dtype is BF16 else 0)
            e_dS = P * (e_delta + r * np.linalg.norm(dh[:, None] * vh, axis=2)) + rel * np.abs(dS)
            for i, (to, w, y) in enumerate(((out[0], dS, None), (out[1], e_dS, np.abs))):
                f = (lambda z: z) if y is None else y
                to[0][b, :, h] = scale * w @ f(kh)
                to[1][b, :, h // G] += scale * w.T @ f(qh)
                to[2][b, :, h // G] += (P if i == 0 else rel * P).T @ f(dh)
    return out[0], [e + u * np.abs(w) for w, e in zip(*out)], least


@pytest.mark.parametrize("dtype,rest", [(F32, 3e-3), (F32, 1e-4), (F32, 1e-5), (F32, 1e-6), (BF16, 3e-3), (BF16, 1e-3)])
@pytest.mark.parametrize("n", [1, 4, 32])
def test_attn_bwd_over_a_part_with_nearly_all_of_the_mass(dtype, rest, n):
    """A few keys that nearly every query attends to, in a call of their own: their gradients are what the
    other keys leave of them, however little that is."""
    q, k, v, do = peaked(n, rest, dtype, n)
    o, lse = kda.attn_fwd(q, k, v, causal=False, scale=0.125)
    for keys in (slice(0, n), slice(n, 70)):
        g = kda.attn_bwd(q, k[:, keys].contiguous(), v[:, keys].contiguous(), o, lse, do, causal=False, scale=0.125)
        torch.cuda.synchronize()
        want, size, least = part_terms(*[np64(x) for x in (q, k, v, do)], keys, 0.125, dtype)
        assert keys.start or 0 < least < 2 * rest
        for name, w, e in zip(("dq", "dk", "dv"), want, size):
            off = np.linalg.norm(np64(g[name]) - w)
            assert off <= np.linalg.norm(e), (keys, name, off, np.linalg.norm(e), np.linalg.norm(w))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attn_gradients_of_few_keys_that_a_window_calls_whole(dtype):
    """A window, however long, says that the keys are all there: without a causal mask too rows of few keys
    are then as precise as others (bounds as in the test of precision above)."""
    most = 1.0 if dtype is BF16 else 12.0
    for Tq, Tk, window in ((1, 1, 1), (7, 2, 40), (30, 3, 100), (60, 31, 2 ** 20)):
        q, _, _, do = draw(4, Tq, Tq, 8, 4, 64, dtype, 31 + Tq)
        _, k, v, _ = draw(4, Tk, Tk, 8, 4, 64, dtype, 32 + Tk)
        kw = dict(causal=False, window=window)
        o, lse = kda.attn_fwd(q, k, v, **kw)
        g = kda.attn_bwd(q, k, v, o, lse, do, **kw)
        torch.cuda.synchronize()
        grads = ora.attn_backward(*[np64(x) for x in (q, k, v, do)], 64 ** -0.5, **kw)
        for name, w in zip(("dq", "dk", "dv"), grads):
            if Tk == 1 and name != "dv":
                assert not g[name].any(), name
                continue
            e = np.linalg.norm(np64(g[name]) - w) / np.linalg.norm(w)
            assert e < most * torch.finfo(dtype).eps / 2, (Tq, Tk, name, e)


def test_attn_one_key_has_no_gradient_of_its_score():
    q, k, v, do = draw(3, 1, 1, 4, 2, 64, BF16, 24)
    o, lse = kda.attn_fwd(q, k, v)
    g = kda.attn_bwd(q, k, v, o, lse, do)
    assert not g["dq"].any() and not g["dk"].any()


def test_attn_smallest_scale():
    """Uniform rows: the gradients of v are means of dout, the others vanish."""
    q, k, v, do = draw(1, 70, 70, 2, 2, 64, BF16, 21)
    run_both(q, k, v, do, BF16, "scale 2^-64", scale=2.0 ** -64, causal=True, window=0)


def test_attn_equal_rows_and_large_magnitudes():
    q, k, v, do = draw(1, 40, 40, 2, 1, 64, BF16, 12)
    k.zero_()
    run_both(q, k, v, do, BF16, "zero keys", causal=True, window=0)
    q, k, v, do = draw(1, 40, 40, 2, 1, 64, F32, 13)
    run_both(q * 1e-20, k, v * 1e15, do, F32, "tiny queries", causal=False, window=0)


def test_attn_nan_and_infinity_reach_only_the_rows_that_see_them():
    q, k, v, _ = draw(1, 300, 300, 1, 1, 64, F32, 14)
    k[0, 200, 0, 3] = float("nan")
    o, lse = kda.attn_fwd(q, k, v, causal=True)
    torch.cuda.synchronize()
    bad = torch.isnan(o[0, :, 0]).any(-1)
    assert bool(bad[200:].all()) and not bool(bad[:200].any())
    assert bool(torch.isnan(lse[0, 0, 200:]).all()) and bool(torch.isfinite(lse[0, 0, :200]).all())
    # the same through the split key axis
    o, lse = kda.attn_fwd(q[:, -1:], torch.cat([k] * 6, 1), torch.cat([v] * 6, 1), causal=True)
    assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attn_writes_its_outputs_only(dtype):
    B, Tq, Tk, H, HK, D = 2, 37, 50, 4, 2, 64
    q, k, v, do = draw(B, Tq, Tk, H, HK, D, dtype, 15)
    big = torch.full((B * Tq * H * D + 512,), 7.0, dtype=dtype, device="cuda")
    o = big[256:-256].view(B, Tq, H, D)
    lbig = torch.full((B * H * Tq + 64,), 7.0, device="cuda")
    lse = lbig[32:-32].view(B, H, Tq)
    kda.attn_fwd(q, k, v, o=o, lse=lse)
    torch.cuda.synchronize()
    assert bool((big[:256] == 7).all()) and bool((big[-256:] == 7).all())
    assert bool((lbig[:32] == 7).all()) and bool((lbig[-32:] == 7).all())


@pytest.mark.parametrize("dtype,B,Tq,Tk,H,HK,D,kw", [
    (F32, 2, 37, 50, 4, 2, 64, dict(causal=1)), (F32, 1, 131, 45, 6, 3, 128, dict(causal=0)), (F32, 1, 9, 21, 2, 2, 16, dict(window=5)),
    (BF16, 2, 37, 50, 4, 2, 64, dict(causal=1)), (BF16, 1, 45, 131, 6, 3, 128, dict(window=70)), (BF16, 3, 7, 5, 4, 1, 32, dict(causal=0)),
    (BF16, 16, 300, 333, 16, 16, 64, dict(causal=1)), (BF16, 2, 2111, 1001, 16, 16, 128, dict(causal=0)),
])
def test_attn_bwd_writes_its_outputs_and_workspace_only(dtype, B, Tq, Tk, H, HK, D, kw):
    """The C entry with room around every output and a workspace of just the bytes asked for."""
    lib = kda.load()
    q, k, v, do = draw(B, Tq, Tk, H, HK, D, dtype, 25)
    kw = dict(causal=0, window=0) | kw
    o, lse = kda.attn_fwd(q, k, v, **kw)
    dt = 1 if dtype is BF16 else 0
    need = lib.kda_attn_bwd_workspace(B, Tq, Tk, H, HK, D, dt)
    e = q.element_size()
    sizes = [B * Tq * H * D * e, B * Tk * HK * D * e, B * Tk * HK * D * e, need]
    room = [torch.full((n + 8192,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes]
    at = [x.data_ptr() + 4096 for x in room]
    st = lib.kda_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, o.data_ptr(), lse.data_ptr(), do.data_ptr(), *at[:3],
                          B, Tq, Tk, H, HK, D, 0, 0, 0, D ** -0.5, kw["causal"], kw["window"], dt, at[3], need,
                          torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    want = kda.attn_bwd(q, k, v, o, lse, do, **kw)
    for x, n, name in zip(room, sizes, ("dq", "dk", "dv", None)):
        assert bool((x[:4096] == 0x5A).all()) and bool((x[4096 + n:] == 0x5A).all()), name
        if name:
            assert torch.equal(x[4096:4096 + n].view(dtype), want[name].view(-1)), name


@pytest.mark.parametrize("dtype,T,H,D", [(F32, 150, 2, 64), (BF16, 150, 2, 32), (BF16, 300, 2, 128)])
def test_attn_rows_the_largest_stride_apart(dtype, T, H, D):
    """q, k and v in rows of 2^23 elements: the last row of a tile of 128 lies almost 2^32 bytes behind its first."""
    x = torch.empty(1, T, 2 ** 23, dtype=dtype, device="cuda")
    part = lambda i: x[:, :, 2 ** 20 * i:2 ** 20 * i + H * D].unflatten(2, (H, D))  # noqa: E731
    c = draw(1, T, T, H, H, D, dtype, 26)
    far = [part(i) for i in range(3)]
    for y, z in zip(far, c):
        y.copy_(z)
    for kw in (dict(causal=True), dict(causal=False), dict(causal=True, window=40)):
        o, lse = kda.attn_fwd(*far, **kw)
        g = kda.attn_bwd(*far, o, lse, c[3], **kw)
        wo, wl = kda.attn_fwd(*c[:3], **kw)
        w = kda.attn_bwd(*c[:3], wo, wl, c[3], **kw)
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(lse, wl) and all(torch.equal(g[n], w[n]) for n in w), kw


def test_attn_bwd_repeats_bit_for_bit():
    q, k, v, do = draw(2, 260, 260, 8, 2, 128, BF16, 16)
    o, lse = kda.attn_fwd(q, k, v)
    a = kda.attn_bwd(q, k, v, o, lse, do)
    for _ in range(3):
        b = kda.attn_bwd(q, k, v, o, lse, do)
        torch.cuda.synchronize()
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_attn_gradient_against_differences():
    """The derivative along a direction, from differences of the fp64 forward, against
    the operator's gradients: the gradients' own bounds plus the difference's h^2 term
    (third derivatives of these sums are below 1e3 at this size)."""
    q, k, v, do = draw(1, 24, 30, 4, 2, 16, F32, 17)
    kw = dict(causal=True, window=9, q_len=[20], kv_len=[27])
    o, lse = kda.attn_fwd(q, k, v, causal=True, window=9, q_len=ints([20]), kv_len=ints([27]))
    g = kda.attn_bwd(q, k, v, o, lse, do, causal=True, window=9, q_len=ints([20]), kv_len=ints([27]))
    ref = [np64(x) for x in (q, k, v, do)]
    _, bounds = bwd_bounds(*ref, F32, 0.25, **kw)
    rng, h = np.random.default_rng(0), 1e-4
    for i, n in enumerate(("dq", "dk", "dv")):
        d = rng.standard_normal(ref[i].shape)
        at = lambda s: (ora.attn_forward(*[x + s * d if j == i else x for j, x in enumerate(ref[:3])], 0.25, **kw)[0] * ref[3]).sum()  # noqa: E731
        diff = (at(h) - at(-h)) / (2 * h)
        assert abs(diff - (np64(g[n]) * d).sum()) <= (bounds[i] * np.abs(d)).sum() + 1e3 * h * h, n


def test_attn_streams_and_two_calls_at_once():
    xs = [draw(1, 128, 1500, 8, 2, 64, BF16, s) for s in (21, 22)]
    want = [kda.attn_fwd(*x[:3]) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for s, x in zip(streams, xs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([kda.attn_fwd(*x[:3]) for _ in range(4)])
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for o, lse in many:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


def test_attn_captured_and_replayed():
    q, k, v, do = draw(2, 100, 100, 4, 2, 64, BF16, 23)
    qs, ks, vs, _ = draw(1, 4, 2048, 8, 2, 64, BF16, 24)   # the split form
    step = lambda: (kda.attn_fwd(q, k, v), kda.attn_fwd(qs, ks, vs))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        (o, lse), _ = step()
        kda.attn_bwd(q, k, v, o, lse, do)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (o, lse), (o2, lse2) = step()
        g = kda.attn_bwd(q, k, v, o, lse, do)
    for i in range(3):
        for x in (q, k, v, do, qs, ks, vs):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(30 + i)).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        (wo, wl), (wo2, wl2) = step()
        wg = kda.attn_bwd(q, k, v, wo, wl, do)
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(lse, wl) and torch.equal(o2, wo2) and torch.equal(lse2, wl2)
        assert all(torch.equal(g[n], wg[n]) for n in g)


def test_attn_empty():
    for B, Tq, Tk in ((0, 3, 3), (2, 0, 3), (2, 3, 0)):
        q, k, v, do = draw(B, Tq, Tk, 2, 1, 32, F32, 1)
        o, lse = kda.attn_fwd(q, k, v)
        g = kda.attn_bwd(q, k, v, o, lse, do)
        torch.cuda.synchronize()
        assert bool((o == 0).all()) and bool((lse == float("-inf")).all())
        assert all(bool((x == 0).all()) for x in g.values())


def test_attn_rows_past_32_bit_offsets():
    """Keys whose byte offset in the tensor passes 2^32: the last sequence of a long cache."""
    B, Tk, HK, D = 5, 524288, 8, 128
    k = torch.zeros(B, Tk, HK, D, dtype=BF16, device="cuda")
    v = torch.zeros(B, Tk, HK, D, dtype=BF16, device="cuda")
    q = torch.randn(B, 1, HK, D, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    n = [64, 64, 64, 64, Tk]
    k[4, -8:] = torch.randn(8, HK, D, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    v[4, -8:] = torch.randn(8, HK, D, generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    o, lse = kda.attn_fwd(q, k, v, kv_len=ints(n), window=8)
    torch.cuda.synchronize()
    wo, wl, bo, bl = fwd_bounds(np64(q[4:]), np64(k[4:, -8:]), np64(v[4:, -8:]), BF16, D ** -0.5)
    check(o[4:], wo, bo, "o")
    check(lse[4:], wl, bl, "lse")


def test_attn_refusals():
    q, k, v, do = draw(2, 8, 8, 4, 2, 32, BF16, 1)
    o, lse = kda.attn_fwd(q, k, v)
    with pytest.raises(TypeError):
        kda.attn_fwd(q.half(), k.half(), v.half())
    with pytest.raises(TypeError):
        kda.attn_fwd(q, k.float(), v)
    with pytest.raises(ValueError):
        kda.attn_fwd(q, k, v[:, :4])
    with pytest.raises(ValueError):
        kda.attn_fwd(q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2))
    with pytest.raises(ValueError):
        kda.attn_fwd(q, k, v, kv_len=ints([1, 2, 3]))
    with pytest.raises(TypeError):
        kda.attn_fwd(q, k, v, kv_len=torch.ones(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.attn_fwd(q[:, :, :3], k, v)            # three query heads over two
    for s in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(kda.KDAError):
            kda.attn_fwd(q, k, v, scale=s)
    with pytest.raises(kda.KDAError):
        kda.attn_fwd(q, k, v, window=-1)
    with pytest.raises(kda.KDAError):
        kda.attn_fwd(q, k, v, o=q)                 # the output over an input
    with pytest.raises(ValueError):
        kda.attn_bwd(q, k, v, o, lse, do[:, :4])
    with pytest.raises(kda.KDAError):
        kda.attn_fwd(*(x[..., :24].contiguous() for x in (q, k, v)))
