"""GPU parity of the attention with a common prefix: within the bounds of
tests/attn_check.py of the oracle over the stored values, as the decode step is, at
groups, prefixes and masks where it can go wrong."""

import numpy as np
import pytest
import torch

from gated_delta_rule_82_amd import kda
from oracle import branch_oracle as ora
from tests.attn_check import BF16, F32, check, np64
from tests.test_gpu_attn_cache import Pair, compare_step, ints, kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    kda.load()
    yield
    torch.cuda.synchronize()


class Batch:
    """Groups of sequences filled side by side in the library's cache and the oracle's: the
    prefix into the first one's pages, the page in which it ends copied for the others, and
    everybody's own tokens behind it.  Sequences of no group have a prefix of 0."""

    def __init__(self, sizes, prefixes, own, HK, D, page, Tq, dtype, seed=0, before=0):
        self.first = [before]
        for n in sizes:
            self.first.append(self.first[-1] + n)
        B = self.first[-1] + before
        self.B, self.prefix = B, prefixes
        pre = [0] * before + [p for n, p in zip(sizes, prefixes) for _ in range(n)] + [0] * before
        own = [own[b % len(own)] for b in range(B)]
        self.lens = [p + n for p, n in zip(pre, own)]
        width = -(-(max(self.lens) + Tq) // page)
        n_pages = B * width + 3
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))[:B * width].view(B, width)
        lead = list(range(B))
        for g, n in enumerate(sizes):
            for b in range(self.first[g], self.first[g + 1]):
                lead[b] = self.first[g]
                order[b, :prefixes[g] // page] = order[lead[b], :prefixes[g] // page]
        self.table = order.to(torch.int32).cuda()
        c = self.cache = Pair(n_pages, HK, D, page, seed)
        k, v = kv(B, max(pre) or 1, HK, D, dtype, seed + 1)
        c.append(k, v, self.table, [0] * B, [p if lead[b] == b else 0 for b, p in enumerate(pre)])
        src, dst = [], []
        for b, p in enumerate(pre):
            if lead[b] != b and p % page:
                src.append(int(order[lead[b], p // page]))
                dst.append(int(order[b, p // page]))
        if src:
            kda.cache_copy(*c.dev, ints(src), ints(dst))
            for x in (c.K, c.V):
                x.val[dst], x.scale[dst] = x.val[src], x.scale[src]
            c.written[dst] = c.written[src]
        k, v = kv(B, max(own) + Tq, HK, D, dtype, seed + 2)
        c.append(k, v, self.table, pre, [n + Tq for n in own])

    def groups(self):
        return ints(self.first), ints(self.prefix)


def queries(B, Tq, H, D, dtype, seed=3):
    return torch.randn(B, Tq, H, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def run(x, q, new=None, window=0, **kw):
    o = kda.attn_shared(q, *x.cache.dev, x.table, ints(x.lens), *x.groups(), ints(new), window=window, **kw)
    torch.cuda.synchronize()
    Tq = q.shape[1]
    compare_step(o, q, x.cache, x.table, x.lens, [Tq] * x.B if new is None else new, window, q.dtype)
    return o


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page,D,H,HK,Tq", [(16, 16, 4, 2, 1), (32, 32, 3, 3, 2), (64, 64, 8, 1, 1), (128, 128, 8, 2, 3), (16, 128, 2, 2, 9),
                                            (64, 128, 32, 8, 1)])
@pytest.mark.parametrize("window", [0, 60])
def test_groups(dtype, page, D, H, HK, Tq, window):
    """Groups of one to nine sequences (one empty) with prefixes of 0 to 333 tokens, and sequences of none."""
    x = Batch([3, 1, 0, 9, 2, 4], [130, 64, 50, 333, 0, 1], [5, 0, 40, 17], HK, D, page, Tq, dtype, seed=D + page, before=1)
    run(x, queries(x.B, Tq, H, D, dtype), window=window)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("N,G,Tq", [(1, 1, 1), (5, 3, 1), (16, 4, 1), (33, 4, 1), (11, 4, 3), (70, 1, 2), (40, 8, 1)])
def test_rows_of_a_group(dtype, D, N, G, Tq):
    """Tiles of rows: less than one, several, and a last one that is not full."""
    x = Batch([N], [200], [3, 11, 0, 30], 2, D, 16, Tq, dtype, seed=N)
    run(x, queries(x.B, Tq, 2 * G, D, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("prefix", [1, 15, 16, 63, 64, 65, 128, 1000, 4097])
@pytest.mark.parametrize("N,H", [(3, 2), (20, 16)])
def test_prefix_lengths(dtype, prefix, N, H):
    """Prefixes around a block of keys and a page, and long ones whose parts are joined."""
    x = Batch([N, 2], [prefix, prefix], [0, 1, 70], 2, 64, 64, 1, dtype, seed=prefix)
    run(x, queries(x.B, 1, H, 64, dtype))
    if prefix > 60:
        run(x, queries(x.B, 1, H, 64, dtype), window=50)          # some see nothing of the prefix
        run(x, queries(x.B, 1, H, 64, dtype), window=prefix - 20)


def test_new_lengths():
    """Padded queries are not read and give zeros; a sequence without any, a group without any."""
    x = Batch([3, 2], [100, 40], [8, 3], 2, 32, 16, 4, F32)
    q = queries(5, 4, 4, 32, F32)
    new = [4, 0, 2, 0, 0]
    for b in range(5):
        q[b, new[b]:] = float("nan")
    o = run(x, q, new)
    assert all(bool((o[b, new[b]:] == 0).all()) for b in range(5))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lengths_below_the_prefix(dtype):
    """A prefix that says more than a sequence has: it sees its own length."""
    x = Batch([4, 3], [200, 90], [20, 0], 2, 64, 16, 2, dtype)
    x.lens = [200, 30, 0, 199, 5, 90, 89]
    run(x, queries(7, 2, 4, 64, dtype))
    x.prefix = [1 << 30, 90]                      # clamped to the table; all read the first one's row
    o = kda.attn_shared(queries(7, 2, 4, 64, dtype), *x.cache.dev, x.table, ints(x.lens), *x.groups())
    torch.cuda.synchronize()
    want = ora.attn_shared(np64(queries(7, 2, 4, 64, dtype)), x.cache.K, x.cache.V, x.table.cpu().numpy(), x.lens, x.first, x.prefix, 0.125)
    assert np.abs(np64(o) - want).max() <= (0.05 if dtype == BF16 else 1e-5) * np.abs(want).max()


def test_the_prefix_is_read_through_the_first_row():
    """Other rows' entries below the prefix are not looked at, but for the page in which it ends."""
    x = Batch([3], [100], [20], 2, 32, 16, 1, F32)
    q = queries(3, 1, 4, 32, F32)
    want = kda.attn_shared(q, *x.cache.dev, x.table, ints(x.lens), *x.groups())
    x.table[1:, :6] = -1
    got = kda.attn_shared(q, *x.cache.dev, x.table, ints(x.lens), *x.groups())
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_missing_pages():
    x = Batch([3, 2], [100, 64], [20], 2, 32, 16, 1, F32)
    t = x.table
    t[0, 2] = -1                  # of the prefix: hidden from the whole group
    t[1, 7] = 1 << 30             # of one sequence's own
    t[3:, :] = -1                 # a group without anything
    q = queries(5, 1, 4, 32, F32)
    o = kda.attn_shared(q, *x.cache.dev, t, ints(x.lens), *x.groups())
    torch.cuda.synchronize()
    want = ora.attn_shared(np64(q), x.cache.K, x.cache.V, t.cpu().numpy(), x.lens, x.first, x.prefix, 32 ** -0.5)
    assert np.all(want[3:] == 0)
    check(o, want, 64 * 1e-5, "missing pages")    # values below 64; a row's bound is below 1e-5 of them


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [2, 12, 40])
def test_scales_that_are_no_powers_of_two(dtype, N):
    """A cache that somebody else filled: a code stands for itself times any scale."""
    x = Batch([N], [200], [3, 40], 2, 64, 16, 1, dtype, seed=N)
    c = x.cache
    g = torch.Generator().manual_seed(N)
    for dev, o in ((c.dev[2], c.K), (c.dev[3], c.V)):
        f = 1.0 + torch.rand(dev.shape, generator=g).cuda()
        f[torch.rand(dev.shape, generator=g).cuda() < 0.5] = 1.0
        dev.mul_(f)
        o.scale[:] = np64(dev)
    run(x, queries(N, 1, 8, 64, dtype))


def test_groups_that_are_none():
    """No groups, groups outside the batch: the decode step."""
    x = Batch([4], [50], [20, 3], 2, 32, 16, 1, F32)
    q = queries(4, 1, 4, 32, F32)
    want = ora.attn_shared(np64(q), x.cache.K, x.cache.V, x.table.cpu().numpy(), x.lens, [0], [], 32 ** -0.5)
    for first, prefix in (([0], []), ([0, 0], [50]), ([4, 9], [50]), ([-3, 0, 0], [50, 50]), ([7, 2, 1], [10, 10])):
        o = kda.attn_shared(q, *x.cache.dev, x.table, ints(x.lens), ints(first), ints(prefix))
        torch.cuda.synchronize()
        check(o, want, 64 * 1e-5, str(first))


def test_many_groups():
    """More groups than a wave looks at together."""
    x = Batch([1, 2, 0] * 50, [20, 35, 7] * 50, [2, 9], 1, 16, 16, 1, BF16)
    run(x, queries(x.B, 1, 2, 16, BF16))


@pytest.mark.parametrize("at", [0, 255, 256, 4095, 4999])
def test_a_group_far_down(at):
    """Empty groups before and behind the one that there is."""
    x = Batch([0] * at + [5] + [0] * (4999 - at), [16] * at + [100] + [16] * (4999 - at), [20, 3], 2, 32, 16, 1, BF16, before=1)
    run(x, queries(7, 1, 4, 32, BF16))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_packed_queries(dtype):
    """The queries of a packed projection, read where they lie; a workspace of the caller's."""
    x = Batch([6], [90], [20, 3], 2, 64, 16, 2, dtype)
    p = queries(6, 2, 4 + 4, 64, dtype)
    ws = torch.empty(kda.attn_shared_workspace_bytes(6, 2, 4, 2, 64, 1, x.table.shape[1] * 16), dtype=torch.uint8, device="cuda")
    a = run(x, p[:, :, :4], workspace=ws)
    b = run(x, p[:, :, :4].contiguous())
    assert torch.equal(a, b)


def test_values_of_keys_that_nobody_sees():
    """What the first sequence has from the page on in which the prefix ends is not the group's: NaN codes
    there, in the same 64 keys as the last common ones, reach only itself."""
    x = Batch([3], [40], [30], 1, 32, 16, 1, F32)
    q = queries(3, 1, 2, 32, F32)
    want = kda.attn_shared(q, *x.cache.dev, x.table, ints(x.lens), *x.groups())
    for pg in x.table[0, 2:4].tolist():
        x.cache.dev[0][pg] = 0x7f
        x.cache.dev[1][pg] = 0x7f
    got = kda.attn_shared(q, *x.cache.dev, x.table, ints(x.lens), *x.groups())
    torch.cuda.synchronize()
    assert torch.equal(got[1:], want[1:]) and bool(torch.isnan(got[0]).all())


def test_captured_and_replayed():
    """Prefixes, groups and lengths change between replays of one graph."""
    x = Batch([4, 3], [150, 60], [30, 3], 2, 64, 16, 1, BF16)
    q, lens = queries(7, 1, 8, 64, BF16), ints(x.lens)
    first, prefix = x.groups()
    call = lambda: kda.attn_shared(q, *x.cache.dev, x.table, lens, first, prefix)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call()
    for i, (f, p) in enumerate((([0, 4, 7], [150, 60]), ([0, 4, 7], [16, 0]), ([0, 2, 4], [149, 150]), ([0, 0, 7], [9, 0]))):
        q.copy_(queries(7, 1, 8, 64, BF16, 50 + i))
        first.copy_(ints(f)), prefix.copy_(ints(p))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, call())
        torch.cuda.synchronize()
        compare_step(o, q, x.cache, x.table, x.lens, [1] * 7, 0, BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_as_the_decode_step(dtype):
    """The same rows with and without groups: within both bounds of each other, and the same bits every time."""
    x = Batch([20, 12], [700, 300], [50, 10, 0], 2, 128, 64, 1, dtype)
    q = queries(32, 1, 8, 128, dtype)
    a = run(x, q)
    b = kda.attn_step(q, *x.cache.dev, x.table, ints(x.lens))
    torch.cuda.synchronize()
    compare_step(b, q, x.cache, x.table, x.lens, [1] * 32, 0, dtype)
    assert all(torch.equal(a, run(x, q)) for _ in range(2))


def test_refusals():
    x = Batch([2], [20], [4], 2, 32, 16, 1, BF16)
    q, lens = queries(2, 1, 4, 32, BF16), ints(x.lens)
    first, prefix = x.groups()
    with pytest.raises(ValueError):
        kda.attn_shared(q, *x.cache.dev, x.table, lens, first[:1], prefix)
    with pytest.raises(TypeError):
        kda.attn_shared(q, *x.cache.dev, x.table, lens, first, prefix.long())
    with pytest.raises(kda.KDAError):
        kda.attn_shared(q[:, :, :3], *x.cache.dev, x.table, lens, first, prefix)
    with pytest.raises(kda.KDAError):
        kda.attn_shared(q, *x.cache.dev, x.table, lens, first, prefix, scale=0.0)
    with pytest.raises(ValueError):
        kda.attn_shared(q, *x.cache.dev, x.table, lens, first, prefix, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(kda.KDAError):
        kda.attn_shared(q, *x.cache.dev, x.table, lens, first, prefix, o=q)
    with pytest.raises(kda.KDAError):          # more groups than are looked through
        kda.attn_shared(q, *x.cache.dev, x.table, lens, ints([0] * ((1 << 16) + 2)), ints([0] * ((1 << 16) + 1)))
