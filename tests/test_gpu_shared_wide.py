"""GPU parity of the attention with a common prefix on tiles of 64 and 128 rows, which are
taken where groups have more than 32 rows and tables room for many keys: the tables here
are wider than their sequences need, by entries that nobody has."""

import numpy as np
import pytest
import torch

from gated_delta_rule_82_amd import kda
from oracle import branch_oracle as ora
from tests.attn_check import BF16, check, np64
from tests.test_gpu_attn_cache import compare_step, ints
from tests.test_gpu_shared import Batch, queries, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    kda.load()
    yield
    torch.cuda.synchronize()


def roomy(x, tokens=1 << 18):
    """The batch with a table of so many tokens."""
    B, n = x.table.shape
    more = torch.full((B, max(0, tokens // x.cache.K.page - n)), -1, dtype=torch.int32, device="cuda")
    x.table = torch.cat((x.table, more), 1).contiguous()
    return x


def rounding(x):
    """Of an output and of the probabilities behind it to eight bits, for two results: 2^-8 each of the largest value."""
    c = x.cache.V
    v = np.abs(c.val) * c.scale[:, :, None, None]
    return 4 * 2.0 ** -8 * np.nanmax(np.where(x.cache.written[:, None, :, None], v, 0.0))


@pytest.mark.parametrize("page,D,H,HK,Tq", [(16, 32, 24, 2, 1), (32, 64, 12, 1, 1), (64, 64, 16, 1, 2), (128, 128, 32, 2, 3), (16, 128, 16, 1, 1),
                                            (64, 128, 32, 2, 1), (128, 32, 24, 1, 1)])
@pytest.mark.parametrize("window", [0, 60])
def test_groups(page, D, H, HK, Tq, window):
    """Groups of one to nine sequences (one empty) with prefixes of 0 to 333 tokens, and sequences of none;
    42 to 168 rows a group on average."""
    x = roomy(Batch([3, 1, 0, 9, 2, 4], [130, 64, 50, 333, 0, 1], [5, 0, 40, 17], HK, D, page, Tq, BF16, seed=D + page, before=1))
    run(x, queries(x.B, Tq, H, D, BF16), window=window)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("N,G,Tq", [(33, 1, 1), (16, 3, 1), (16, 4, 1), (65, 1, 1), (33, 4, 1), (11, 4, 3), (70, 1, 2), (40, 8, 1)])
def test_rows_of_a_group(D, N, G, Tq):
    """Tiles of rows: one that is not full, one that is, several."""
    x = roomy(Batch([N], [200], [3, 11, 0, 30], 2, D, 16, Tq, BF16, seed=N))
    run(x, queries(x.B, Tq, 2 * G, D, BF16))


@pytest.mark.parametrize("prefix", [1, 15, 16, 64, 65, 127, 128, 129, 1000, 4097])
@pytest.mark.parametrize("N", [8, 20])
def test_prefix_lengths(prefix, N):
    """Prefixes around a step of keys and a page, each part one step at most."""
    x = roomy(Batch([N, 2], [prefix, prefix], [0, 1, 70], 2, 64, 64, 1, BF16, seed=prefix))
    run(x, queries(x.B, 1, 16, 64, BF16))
    if prefix > 60:
        run(x, queries(x.B, 1, 16, 64, BF16), window=50)
        run(x, queries(x.B, 1, 16, 64, BF16), window=prefix - 20)


def long_prefixes(sizes, prefixes, own, HK, G, D, page, room, windows):
    """Codes and scales at random, as long as these prefixes need; a token each, against softmax in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(D + page)
    rand = lambda *n: torch.randint(0, 256, n, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    first = [0]
    for n in sizes:
        first.append(first[-1] + n)
    B, lens, rows, used = first[-1], [], [], 0
    for n, p in zip(sizes, prefixes):
        common = list(range(used, used + p // page))
        used += len(common)
        for _ in range(n):
            lens.append(p + own[len(lens) % len(own)])
            more = -(-(lens[-1] + 1) // page) - len(common)
            rows.append(common + list(range(used, used + more)))
            used += more
    order = torch.randperm(used, generator=torch.Generator().manual_seed(page)).tolist()
    table = torch.full((B, room // page), -1, dtype=torch.int32)
    for b, r in enumerate(rows):
        table[b, :len(r)] = torch.tensor([order[i] for i in r], dtype=torch.int32)
    table = table.cuda()
    k, v = rand(used, HK, page, D), rand(used, HK, D, page)
    for c in (k, v):
        c[(c & 0x7f) == 0x7f] = 0x11                # no NaN; values below 448 2^-8
    ks, vs = (torch.ldexp(torch.ones(used, HK, device="cuda"), rand(used, HK).int() % 3 - 10) for _ in range(2))
    q = torch.randn(B, 1, HK * G, D, generator=g, device="cuda").to(BF16)
    for window in windows:
        o = kda.attn_shared(q, k, v, ks, vs, table, ints(lens), ints(first), ints(prefixes), window=window)
        torch.cuda.synchronize()
        for b in range(B):
            if b - first[max(i for i in range(len(sizes)) if first[i] <= b)] not in (0, 1, 32):
                continue
            pages = table[b, :len(rows[b])].long()
            lo = max(0, lens[b] - window + 1) if window else 0
            K = (k[pages].view(torch.float8_e4m3fn).double() * ks[pages].double()[:, :, None, None]).permute(1, 0, 2, 3).reshape(HK, -1, D)
            V = (v[pages].view(torch.float8_e4m3fn).double() * vs[pages].double()[:, :, None, None]).permute(1, 0, 3, 2).reshape(HK, -1, D)
            K, V = K[:, lo:lens[b] + 1], V[:, lo:lens[b] + 1]
            x = q[b, 0].double().view(HK, G, 1, D)
            prob = torch.softmax((x * K[:, None]).sum(-1) * D ** -0.5 if G * K.shape[1] * D * HK < 1 << 24 else
                                 torch.matmul(x[:, :, 0], K.transpose(1, 2).contiguous()) * D ** -0.5, -1)
            want = torch.matmul(prob, V).view(HK * G, D)
            # a probability and the output, each rounded to eight bits: 2^-8 of the largest value
            far = (o[b, 0].double() - want).abs().max()
            assert bool(torch.isfinite(o[b]).all()) and float(far) <= 2 * 2.0 ** -8 * float(V.abs().max()), (b, window, float(far))


@pytest.mark.parametrize("N", [34, 66])
@pytest.mark.parametrize("D,page", [(32, 16), (32, 64), (64, 32), (128, 128)])
def test_parts_of_many_steps(N, D, page):
    """Two parts a prefix: none, one, several and sixteen steps each."""
    long_prefixes([N] * 4, [4100, 150, 1664, 700], [0, 9], 32, 1, D, page, 6400, (0, 1500))


@pytest.mark.parametrize("D,page", [(32, 64), (64, 16)])
def test_a_part_of_more_steps_than_page_numbers_held(D, page):
    """One part: its page numbers are taken 8192 keys at a time."""
    long_prefixes([33] + [0] * 63, [16500] + [0] * 63, [3, 40], 4, 64, D, page, 20480, (0, 16000))


def test_new_lengths():
    """Padded queries are not read and give zeros; a sequence without any, a group without any."""
    x = roomy(Batch([30, 20], [100, 40], [8, 3], 2, 32, 16, 4, BF16))
    q = queries(50, 4, 4, 32, BF16)
    new = [(4, 0, 2)[b % 3] if b < 30 else 0 for b in range(50)]
    for b in range(50):
        q[b, new[b]:] = float("nan")
    o = run(x, q, new)
    assert all(bool((o[b, new[b]:] == 0).all()) for b in range(50))


def test_lengths_below_the_prefix():
    x = roomy(Batch([24, 13], [200, 90], [20, 0], 2, 64, 16, 2, BF16))
    x.lens = [(200, 30, 0, 199, 5, 90)[b % 6] if b < 24 else 90 - b % 3 for b in range(37)]
    run(x, queries(37, 2, 4, 64, BF16))


def test_missing_pages():
    x = roomy(Batch([30, 20], [100, 64], [20], 2, 32, 16, 1, BF16))
    t = x.table
    t[0, 2] = -1                  # of the prefix: hidden from the whole group
    t[1, 7] = 1 << 30             # of one sequence's own
    t[30:, :] = -1                # a group without anything
    q = queries(50, 1, 8, 32, BF16)
    o = kda.attn_shared(q, *x.cache.dev, t, ints(x.lens), *x.groups())
    torch.cuda.synchronize()
    want = ora.attn_shared(np64(q), x.cache.K, x.cache.V, t.cpu().numpy(), x.lens, x.first, x.prefix, 32 ** -0.5)
    assert np.all(want[30:] == 0)
    check(o, want, rounding(x), "missing pages")


@pytest.mark.parametrize("N,D", [(12, 64), (40, 64), (12, 128), (40, 32)])
def test_scales_that_are_no_powers_of_two(N, D):
    x = roomy(Batch([N], [200], [3, 40], 2, D, 16, 1, BF16, seed=N))
    c = x.cache
    g = torch.Generator().manual_seed(N)
    for dev, o in ((c.dev[2], c.K), (c.dev[3], c.V)):
        f = 1.0 + torch.rand(dev.shape, generator=g).cuda()
        f[torch.rand(dev.shape, generator=g).cuda() < 0.5] = 1.0
        dev.mul_(f)
        o.scale[:] = np64(dev)
    run(x, queries(N, 1, 8, D, BF16))


def test_values_of_keys_that_nobody_sees():
    """NaN codes behind the prefix, in the step of its last keys, and in a page behind a window."""
    x = roomy(Batch([40], [40], [30], 1, 32, 16, 1, BF16))
    q = queries(40, 1, 2, 32, BF16)
    want = kda.attn_shared(q, *x.cache.dev, x.table, ints(x.lens), *x.groups())
    for pg in x.table[0, 2:4].tolist():
        x.cache.dev[0][pg] = 0x7f
        x.cache.dev[1][pg] = 0x7f
    got = kda.attn_shared(q, *x.cache.dev, x.table, ints(x.lens), *x.groups())
    torch.cuda.synchronize()
    assert torch.equal(got[1:], want[1:]) and bool(torch.isnan(got[0]).all())


def test_captured_and_replayed():
    x = roomy(Batch([40, 30], [150, 60], [30, 3], 2, 64, 16, 1, BF16))
    q, lens = queries(70, 1, 8, 64, BF16), ints(x.lens)
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
    for i, (f, p) in enumerate((([0, 40, 70], [150, 60]), ([0, 40, 70], [16, 0]), ([0, 20, 40], [149, 150]), ([0, 0, 70], [9, 0]))):
        q.copy_(queries(70, 1, 8, 64, BF16, 50 + i))
        first.copy_(ints(f)), prefix.copy_(ints(p))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, call())
        torch.cuda.synchronize()
        compare_step(o, q, x.cache, x.table, x.lens, [1] * 70, 0, BF16)
