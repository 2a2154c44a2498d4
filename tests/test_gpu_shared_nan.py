"""NaN codes of v at cached tokens that a query does not see: they may reach it from the same 64
tokens, whatever its neighbours in a group or a packed tile see."""

import pytest
import torch

from gated_delta_rule_82_amd import kda
from tests.attn_check import BF16, F32
from tests.test_gpu_attn_cache import ints

pytestmark = pytest.mark.gpu

CHANNEL = 5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    kda.load()
    yield
    torch.cuda.synchronize()


def cache(n_pages, HK, D, page, seed):
    """Codes at random without NaN, scales 2^-10 .. 2^-8."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *n: torch.randint(0, 256, n, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    k, v = rand(n_pages, HK, page, D), rand(n_pages, HK, D, page)
    for c in (k, v):
        c[(c & 0x7f) == 0x7f] = 0x11
    ks, vs = (torch.ldexp(torch.ones(n_pages, HK, device="cuda"), rand(n_pages, HK).int() % 3 - 10) for _ in range(2))
    return k, v, ks, vs


def planted(call, v, page_number, offset, heads, sees, spared):
    """With a NaN code in one channel of head 0: rows (sequence, token) of `sees` get it there and nowhere else,
    those of `spared` are as before, bit for bit."""
    want = call()
    v[page_number, 0, CHANNEL, offset] = 0xff
    got = call()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(want).all()) and sees and spared
    for b, t in sees:
        bad = torch.isnan(got[b, t, :heads])
        assert bool(bad[:, CHANNEL].all()) and int(bad.sum()) == heads, (b, t)
    for b, t in spared:
        assert torch.equal(got[b, t], want[b, t]), (b, t)
    assert torch.equal(got[:, :, heads:], want[:, :, heads:])


@pytest.mark.parametrize("window", [0, 600])
@pytest.mark.parametrize("dtype,N,G,room", [(F32, 6, 2, 0), (F32, 13, 2, 0), (BF16, 6, 2, 0), (BF16, 13, 2, 0), (BF16, 40, 1, 1 << 14),
                                            (BF16, 40, 2, 1 << 14), (BF16, 70, 2, 1 << 14)])
@pytest.mark.parametrize("D,page", [(32, 16), (64, 64), (128, 32), (128, 128)])
def test_shared(window, dtype, N, G, room, D, page):
    """Sequences of a group that end before a key of the prefix, or whose window has passed it.  Groups enough to fill
    the card, so that a wave takes several blocks of keys; the first one's keys are planted."""
    HK, R, prefix, at = 8, 33, 1024, 450
    lens = [(1024, 1300, 1040, 1200)[b % 4] if window else (1024, 100, 380, 1100, 447)[b % 5] for b in range(N)]
    width, common = -(-1400 // page), prefix // page
    own = common * 2 + torch.arange(R * N * (width - common), dtype=torch.int32).view(R * N, -1)
    table = torch.full((R * N, max(width, room // page)), -1, dtype=torch.int32)
    table[:, :common] = torch.arange(common)
    table[:N, :common] += common
    table[:, common:width] = own
    k, v, ks, vs = cache(common * 2 + own.numel(), HK, D, page, D + N)
    q = torch.randn(R * N, 1, HK * G, D, generator=torch.Generator().manual_seed(N)).to(dtype).cuda()
    args = (table.cuda(), ints(lens * R), ints([N * i for i in range(R + 1)]), ints([prefix] * R))
    call = lambda: kda.attn_shared(q, k, v, ks, vs, *args, window=window)  # noqa: E731
    first = [x - window + 1 if window else 0 for x in lens]
    sees = [(b, 0) for b in range(N) if first[b] <= at <= lens[b]]
    spared = [(b, 0) for b in range(N) if first[b] > at // 64 * 64 + 63 or lens[b] < at // 64 * 64]
    planted(call, v, int(table[0, at // page]), at % page, G, sees, spared + [(b, 0) for b in range(N, R * N)])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("at,window", [(62, 240), (320, 0), (320, 240)])
@pytest.mark.parametrize("D", [16, 64])
def test_tokens_of_a_sequence(dtype, shared, at, window, D):
    """New tokens of one sequence, packed in tiles, whose windows begin and whose positions end in different blocks."""
    B, Tq, H, page, before = 300, 30, 8, 32, 300
    table = torch.arange(B * 11, dtype=torch.int32, device="cuda").view(B, 11)
    k, v, ks, vs = cache(B * 11, H, D, page, D)
    q = torch.randn(B, Tq, H, D, generator=torch.Generator().manual_seed(at)).to(dtype).cuda()
    lens = ints([before] * B)
    if shared:
        first, prefix = ints(list(range(B + 1))), ints([0] * B)
        call = lambda: kda.attn_shared(q, k, v, ks, vs, table, lens, first, prefix, window=window)  # noqa: E731
    else:
        call = lambda: kda.attn_step(q, k, v, ks, vs, table, lens, window=window)  # noqa: E731
    block, sees, spared = at // 64 * 64, [], [(b, t) for b in (0, B - 1) for t in range(Tq)]
    for t in range(Tq):
        lo, hi = max(0, before + t - window + 1) if window else 0, before + t
        if lo <= at <= hi:
            sees.append((1, t))
        elif lo > block + 63 or hi < block:
            spared.append((1, t))
    assert len(spared) > 2 * Tq
    planted(call, v, int(table[1, at // page]), at % page, 1, sees, spared)
