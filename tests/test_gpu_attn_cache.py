"""GPU parity of the 8-bit cache: appended codes and scales equal the oracle's bit for
bit (the scales are powers of two), and the attention over the cache is within the
bounds of tests/attn_check.py of the oracle over the stored values."""

import numpy as np
import pytest
import torch

from gated_delta_rule_82_amd import kda
from oracle import attn_oracle as ora
from tests.attn_check import BF16, F32, U, bwd_bounds, check, fwd_bounds, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    kda.load()
    yield
    torch.cuda.synchronize()


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


class Pair:
    """The library's cache and the oracle's, filled side by side."""

    def __init__(self, n_pages, HK, D, page, seed=0):
        self.dev = kda.new_cache(n_pages, HK, D, page)
        g = torch.Generator().manual_seed(seed)
        for c in self.dev[:2]:   # what an unused page holds may be anything, NaN codes among it
            c.copy_(torch.randint(0, 256, c.shape, generator=g, dtype=torch.uint8))
        for s in self.dev[2:]:
            s.fill_(float("nan"))
        self.raw = [x.clone() for x in self.dev]
        self.K, self.V = ora.Cache(n_pages, HK, page, D), ora.Cache(n_pages, HK, page, D)
        self.K.val[:], self.V.val[:] = (ora.e4m3_value(x.cpu().numpy()) for x in (self.raw[0], self.raw[1].transpose(-1, -2)))
        self.K.scale[:] = self.V.scale[:] = np.nan
        self.written = np.zeros((n_pages, page), bool)

    def append(self, k, v, table, cache_len, new_len=None):
        kda.cache_append(k, v, *self.dev, table, ints(cache_len), ints(new_len))
        torch.cuda.synchronize()
        t = table.cpu().numpy()
        self.K.append(np64(k), t, cache_len, new_len)
        self.V.append(np64(v), t, cache_len, new_len)
        for b in range(k.shape[0]):
            n = k.shape[1] if new_len is None else min(max(new_len[b], 0), k.shape[1])
            for j in range(max(cache_len[b], 0), max(cache_len[b], 0) + n):
                p = j // self.K.page
                if p < t.shape[1] and 0 <= t[b, p] < len(self.written):
                    self.written[t[b, p], j % self.K.page] = True

    def check(self):
        kc, vc, ks, vs = self.dev
        w = self.written[:, None, :, None]
        for codes, raw, scale, c in ((kc, self.raw[0], ks, self.K), (vc.transpose(-1, -2), self.raw[1].transpose(-1, -2), vs, self.V)):
            got = ora.e4m3_value(codes.cpu().numpy())
            assert np.array_equal(np.where(w, got, 0), np.where(w, c.val, 0), equal_nan=True)
            assert np.array_equal(np.where(w, 0, codes.cpu().numpy()), np.where(w, 0, raw.cpu().numpy()))  # left as it was
            used = self.written.any(1)
            assert np.array_equal(scale.cpu().numpy()[used], c.scale[used])
            assert bool(torch.isnan(scale.cpu()[torch.from_numpy(~used)]).all())


def tables(B, max_pages, seed, spare=2):
    g = torch.Generator().manual_seed(seed)
    n = B * max_pages + spare
    return torch.randperm(n, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32).cuda(), n


def kv(B, T, HK, D, dtype, seed, packed=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, 2 * HK, D, generator=g) * torch.exp2(torch.randint(-3, 4, (B, T, 1, 1), generator=g).float())
    x = x.to(dtype).cuda()
    k, v = x[:, :, :HK], x[:, :, HK:]
    return (k, v) if packed else (k.contiguous(), v.contiguous())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D,HK", [(16, 3), (32, 1), (64, 2), (128, 2)])
def test_append_matches_oracle(dtype, page, D, HK):
    B, mp = 3, 4
    table, n = tables(B, mp, page)
    c = Pair(n, HK, D, page)
    at = [0, 0, 0]
    for i, (T, new) in enumerate([(page + 3, None), (1, None), (2 * page - 7, [2 * page - 7, 5, 0]), (1, [1, 1, 1]), (3, [9, -1, 2])]):
        k, v = kv(B, T, HK, D, dtype, 10 * i + D, packed=i % 2 == 0)
        c.append(k, v, table, at, new)
        c.check()
        at = [a + (T if new is None else min(max(x, 0), T)) for a, x in zip(at, new or [0] * B)]


def test_append_special_values():
    """Zeros, subnormal results, infinities and NaN, and a page whose scale grows by a lot."""
    table, n = tables(1, 2, 1)
    c = Pair(n, 1, 16, 16)
    x = torch.zeros(1, 4, 1, 16)
    c.append(x.cuda(), x.cuda(), table, [0])
    c.check()
    x[0, 0, 0, :8] = torch.tensor([1e-3, -2e-3, 3e-5, float("inf"), float("-inf"), float("nan"), 2.0, 1e-9])
    c.append(x.cuda(), (x * 7).cuda(), table, [4])
    c.check()
    x[0, 1, 0, 0], x[0, 0, 0, 6] = 3e4, 1e38
    c.append(x.cuda(), x.cuda(), table, [8])
    c.check()
    c.append(x.cuda() * 1e-30, x.cuda() * 0, table, [14])   # over a page's end
    c.check()


def test_append_drops_tokens_without_a_page():
    table, n = tables(3, 2, 5)
    table[0, 1], table[1, 0] = -1, n
    c = Pair(n, 2, 32, 16)
    k, v = kv(3, 40, 2, 32, BF16, 3)
    c.append(k, v, table, [0, 0, 10])      # also past the table's end
    c.append(k, v, table, [-7, 30, 1000])
    c.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page,D,H,HK,Tq", [(16, 16, 4, 2, 1), (32, 32, 3, 3, 2), (64, 64, 8, 1, 1), (128, 128, 8, 2, 5),
                                            (64, 128, 2, 2, 40), (16, 64, 12, 2, 3)])
@pytest.mark.parametrize("window", [0, 50])
def test_step_matches_oracle(dtype, page, D, H, HK, Tq, window):
    lens = [0, 1, 15, 16, 63, 64, 200, 777]
    B, mp = len(lens), -(-(777 + Tq) // page)
    table, n = tables(B, mp, D + page)
    c = Pair(n, HK, D, page)
    k, v = kv(B, 777, HK, D, dtype, 1)
    c.append(k, v, table, [0] * B, lens)
    k, v = kv(B, Tq, HK, D, dtype, 2)
    new = [Tq, Tq, 0, 1, Tq, Tq, max(Tq - 1, 0), Tq]
    c.append(k, v, table, lens, new)
    q = torch.randn(B, Tq, H, D, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    for b in range(B):
        q[b, new[b]:] = float("nan")       # rows past the newest token are not read
    o = kda.attn_step(q, *c.dev, table, ints(lens), ints(new), window=window)
    torch.cuda.synchronize()
    compare_step(o, q, c, table, lens, new, window, dtype)


def compare_step(o, q, c, table, lens, new, window, dtype):
    B, Tq, H, D = q.shape
    t = table.cpu().numpy()
    qn = np.nan_to_num(np64(q))
    want = ora.attn_step(qn, c.K, c.V, t, lens, D ** -0.5, new, window)
    bound = np.zeros(want.shape)
    for b in range(B):
        n = min(lens[b] + new[b], t.shape[1] * c.K.page)
        if new[b] == 0 or n == 0:
            continue
        K, have = c.K.tokens(t[b], n)
        V, _ = c.V.tokens(t[b], n)
        if not have.all() or n < lens[b] + new[b]:
            bound[b] = 0.05 * np.abs(V).max()
            continue
        _, _, bo, _ = fwd_bounds(qn[b:b + 1, :new[b]], K[None], V[None], dtype, D ** -0.5, True, window)
        bound[b, :new[b]] = bo[0]
    check(o, want, bound, "o")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step_splits_a_long_cache(dtype):
    B, Tq, H, HK, D, page, n0 = 2, 2, 8, 2, 64, 64, 5000
    assert kda.attn_step_workspace_bytes(B, Tq, H, HK, D, 80 * page) > 0
    table, n = tables(B, 80, 3)
    c = Pair(n, HK, D, page)
    lens = [n0, 321]
    k, v = kv(B, n0 + Tq, HK, D, dtype, 5)
    c.append(k, v, table, [0, 0], [x + Tq for x in lens])
    q = torch.randn(B, Tq, H, D, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()
    for window in (0, 1000):
        o = kda.attn_step(q, *c.dev, table, ints(lens), window=window)
        torch.cuda.synchronize()
        compare_step(o, q, c, table, lens, [Tq, Tq], window, dtype)


def test_step_without_pages():
    """Missing pages hide their tokens; a sequence with none, or none in its window, gets zeros."""
    table, n = tables(4, 3, 7)
    c = Pair(n, 2, 32, 16)
    k, v = kv(4, 40, 2, 32, F32, 8)
    c.append(k, v, table, [0] * 4)
    table[0, 1] = -1
    table[1, :] = n
    table[2, 2] = 1 << 30
    q = torch.randn(4, 1, 4, 32, generator=torch.Generator().manual_seed(9)).cuda()
    lens = [39, 39, 39, 39]
    for window in (0, 8):
        o = kda.attn_step(q, *c.dev, table, ints(lens), window=window)
        torch.cuda.synchronize()
        t = table.cpu().numpy()
        want = ora.attn_step(np64(q), c.K, c.V, t, lens, 32 ** -0.5, None, window)
        assert np.all(want[1] == 0) and (window == 0 or np.all(want[2] == 0))
        # the stored values are below 64 and a row's bound as in fwd_bounds is below 1e-5 of them
        check(o, want, 64 * 1e-5, f"window {window}")
    # a length past the table: the tokens that the table has are seen
    o = kda.attn_step(q, *c.dev, table, ints([1000, 0, 1 << 30, 100]))
    torch.cuda.synchronize()
    want = ora.attn_step(np64(q), c.K, c.V, table.cpu().numpy(), [1000, 0, 1 << 20, 100], 32 ** -0.5)
    check(o[:3], want[:3], 64 * 1e-5, "past the table")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 3])
def test_step_window_past_the_end_of_the_table(dtype, T):
    """Queries whose position lies past the table's last token: a window counts from there, also one as
    long as the table or longer."""
    page, mp, H, HK, D = 16, 6, 4, 2, 64
    cap = page * mp
    lens = [cap - 2, cap + 9, cap + 60, cap + 94, cap + 95, cap + 96, 2 * cap, (1 << 31) - 1]
    table, n = tables(len(lens), mp, 21)
    c = Pair(n, HK, D, page)
    k, v = kv(len(lens), cap, HK, D, dtype, 4)
    c.append(k, v, table, [0] * len(lens))
    q = torch.randn(len(lens), T, H, D, generator=torch.Generator().manual_seed(7)).to(dtype).cuda()
    kn, vn = ([x.tokens(table.cpu().numpy()[b], cap)[0] for b in range(len(lens))] for x in (c.K, c.V))
    for window in (0, cap - 1, cap, cap + 1, cap + 64, 3 * cap, (1 << 31) - 1):
        o = kda.attn_step(q, *c.dev, table, ints(lens), window=window)
        torch.cuda.synchronize()
        for b, first in enumerate(lens):
            want = np.zeros((T, H, D))
            bound = np.zeros((T, H, D))
            for t in range(T):
                lo = max(first + t - window + 1, 0) if window else 0
                hi = min(first + t + 1, cap)
                if lo < hi:  # one row over the keys it sees
                    bo = fwd_bounds(np64(q[b:b + 1, t:t + 1]), kn[b][None, lo:hi], vn[b][None, lo:hi], dtype, D ** -0.5, False)
                    want[t], bound[t] = bo[0][0, 0], bo[2][0, 0]
            check(o[b], want, bound, f"window {window} at {first}")


def test_shared_pages_are_read_by_several_sequences():
    page, D, HK = 32, 64, 2
    c = Pair(8, HK, D, page)
    t = torch.tensor([[3, 5, 0], [3, 5, 1], [3, 5, 2]], dtype=torch.int32, device="cuda")
    k, v = kv(1, 64, HK, D, BF16, 1)
    c.append(k, v, t[:1], [0])
    k, v = kv(3, 1, HK, D, BF16, 2)
    c.append(k, v, t, [64] * 3)
    q = torch.randn(3, 1, 4, D, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    o = kda.attn_step(q, *c.dev, t, ints([64] * 3))
    torch.cuda.synchronize()
    compare_step(o, q, c, t, [64] * 3, [1] * 3, 0, BF16)


def test_cache_captured_and_replayed():
    """A decode step (rotary, append, attention) captured once and replayed as the lengths advance."""
    B, H, HK, D, page, mp = 3, 8, 2, 64, 16, 80
    table, n = tables(B, mp, 11)
    c, e = Pair(n, HK, D, page), Pair(n, HK, D, page)
    lens = ints([0, 5, 37])
    for x in (c, e):
        k, v = kv(B, 64, HK, D, BF16, 1)
        kda.cache_append(k, v, *x.dev, table, ints([0] * 3), lens)
    x = torch.randn(B, 1, H + 2 * HK, D).to(BF16).cuda()
    f, s = kda.rotary_freqs(32, scaling="yarn", factor=4.0, trained=64)

    def step(dev):
        q, k = kda.rotary(x[:, :, :H], x[:, :, H:H + HK], f, lens.view(B, 1), scale=s)
        kda.cache_append(k, x[:, :, H + HK:], *dev, table, lens)
        return kda.attn_step(q, *dev, table, lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c.dev)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(c.dev)
    for i in range(20):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(50 + i)).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        want = step(e.dev)
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        lens += 1


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [4096, 262144])
def test_last_token_of_a_packed_prompt(dtype, T):
    """The first decode step takes the last token where the prompt's projection holds it: sequences lie
    25 million and 1.6 billion elements apart.  The same calls on contiguous copies give the same bits."""
    B, H, HK, D, page, mp = 2, 40, 4, 128, 16, 80
    x = torch.empty(B, T, H + 2 * HK, D, dtype=dtype, device="cuda")
    x[:, -1:] = torch.randn(B, 1, H + 2 * HK, D, generator=torch.Generator().manual_seed(5)).to(dtype)
    parts = lambda y: (y[:, -1:, :H], y[:, -1:, H:H + HK], y[:, -1:, H + HK:])  # noqa: E731
    f, s = kda.rotary_freqs(64, scaling="yarn", factor=4.0, trained=64)
    pos = torch.full((B, 1), 1000, dtype=torch.int32, device="cuda")
    table, n = tables(B, mp, 11)
    k0, v0 = kv(B, 1200, HK, D, dtype, 1)

    def step(q, k, v, in_place):
        dev = kda.new_cache(n, HK, D, page)
        kda.cache_append(k0, v0, *dev, table, ints([0, 0]))
        q, k = kda.rotary(q, k, f, pos, scale=s, **(dict(q_out=q, k_out=k) if in_place else {}))
        kda.cache_append(k, v, *dev, table, ints([1200, 17]))
        o = kda.attn_step(q, *dev, table, ints([1200, 17]))
        o2, lse2 = kda.attn_fwd(q, k0, v0)
        torch.cuda.synchronize()
        return q.clone(), k.clone(), o, o2, lse2

    want = step(*(y.contiguous() for y in parts(x)), False)
    for in_place in (False, True):
        for got, w in zip(step(*parts(x), in_place), want):
            assert torch.equal(got, w)


def test_training_chain():
    """Rotary, attention and both backward passes over a packed projection, as a layer runs them, in fp32:
    the oracle's chain in 64 bits; the rotation adds 12 * 2^-24 of a pair to q, k and to the gradients, well
    inside four times the backward's own bounds plus 1e-5 of the largest gradient."""
    B, T, H, HK, D = 2, 75, 4, 2, 32
    x = torch.randn(B, T, H + 2 * HK, D, generator=torch.Generator().manual_seed(1)).cuda()
    do = torch.randn(B, T, H, D, generator=torch.Generator().manual_seed(2)).cuda()
    f, s = kda.rotary_freqs(16, scaling="ntk", factor=2.0)
    pos = torch.arange(T, dtype=torch.int32).expand(B, T)
    n = ints([75, 40])
    q, k, v = x[:, :, :H], x[:, :, H:H + HK], x[:, :, H + HK:]
    qr, kr = kda.rotary(q, k, f, scale=s, interleaved=True)
    o, lse = kda.attn_fwd(qr, kr, v, q_len=n, kv_len=n)
    g = kda.attn_bwd(qr, kr, v, o, lse, do, q_len=n, kv_len=n)
    dq, dk = kda.rotary(g["dq"], g["dk"], f, scale=s, interleaved=True, inverse=True)
    torch.cuda.synchronize()
    r = lambda y, inv=False: ora.rotary(y, pos.numpy(), np64(f), s, True, inv)  # noqa: E731
    ref = (r(np64(q)), r(np64(k)), np64(v))
    kw = dict(q_len=[75, 40], kv_len=[75, 40])
    (wq, wk, wv), bounds = bwd_bounds(*ref, np64(do), F32, D ** -0.5, **kw)
    check(o, ora.attn_forward(*ref, D ** -0.5, **kw)[0], 1e-5 * 4, "o")
    for got, w, b in ((dq, r(wq, True), bounds[0]), (dk, r(wk, True), bounds[1]), (g["dv"], wv, bounds[2])):
        check(got, w, 4 * b.max() + 1e-5 * np.abs(w).max(), "gradient")


def test_cache_refusals():
    dev = kda.new_cache(4, 2, 32, 16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), ints([0, 0])
    k, v = kv(2, 1, 2, 32, BF16, 1)
    q = k.repeat_interleave(2, 2)
    with pytest.raises(ValueError):
        kda.cache_append(k[:, :, :1], v[:, :, :1], *dev, table, lens)
    with pytest.raises(TypeError):
        kda.cache_append(k, v, *dev, table.long(), lens)
    with pytest.raises(ValueError):
        kda.cache_append(k, v, *dev, table[:1], lens)
    with pytest.raises(ValueError):
        kda.attn_step(q, dev[1], dev[0], dev[2], dev[3], table, lens)   # k and v pages exchanged
    with pytest.raises(kda.KDAError):
        kda.attn_step(q[:, :, :3], *dev, table, lens)
    with pytest.raises(kda.KDAError):
        kda.attn_step(q, *dev, table, lens, scale=0.0)
    with pytest.raises(kda.KDAError):
        kda.attn_step(q, *kda.new_cache(4, 2, 32, 48), table, lens)
