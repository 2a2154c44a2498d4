"""Host validation of the softmax-attention entry points (no GPU: a rejected call
makes no HIP call), their workspace sizes, and the rotary frequencies, which are
computed on the host."""

import ctypes
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_82_amd import kda
from oracle import attn_oracle as ora

NULL, SHAPE, ALIGN, DTYPE, WORKSPACE, SCALE = 1, 2, 3, 4, 6, 9


@pytest.fixture(scope="module")
def lib():
    return kda.load()


def addr(i):
    """Distinct aligned fake device addresses, 4 GiB apart (never dereferenced)."""
    return 0x10000 + (i << 32)


def call(fn, defaults, **kw):
    args = dict(defaults)
    unknown = set(kw) - set(args)
    assert not unknown, unknown
    args.update(kw)
    return fn(*args.values())


# ------------------------------------------------------------------ rotary frequencies

@pytest.mark.parametrize("rot", [2, 16, 62, 128])
@pytest.mark.parametrize("kw", [{}, dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0, base=500000.0),
                                dict(scaling="yarn", factor=4.0, trained=4096), dict(scaling="yarn", factor=1.0, trained=1),
                                dict(scaling="yarn", factor=32.0, trained=8192, beta_fast=16.0, beta_slow=2.0, base=1e6)])
def test_rotary_freqs(rot, kw):
    f, s = kda.rotary_freqs(rot, device="cpu", **kw)
    fr, sr = ora.rotary_freqs(rot, **kw)
    assert np.allclose(f.numpy(), fr, rtol=1e-14, atol=0) and abs(s - sr) <= 2.0 ** -24 * sr


def test_rotary_freqs_refusals(lib):
    buf = (ctypes.c_double * 64)()
    d = dict(out=ctypes.addressof(buf), scale=None, rot=16, base=1e4, kind=0, factor=1.0, trained=0, fast=32.0, slow=1.0)
    f = lambda **kw: call(lib.kda_rotary_freqs, d, **kw)  # noqa: E731
    assert f() == 0
    for rot in (0, 3, -2, 130):
        assert f(rot=rot) == SHAPE
    assert f(kind=4) == SHAPE and f(kind=-1) == SHAPE and f(kind=3, trained=0) == SHAPE
    for base in (1.0, 0.0, math.inf, math.nan):
        assert f(base=base) == SCALE
    assert f(kind=1, factor=0.5) == SCALE and f(kind=2, factor=math.nan) == SCALE
    assert f(kind=3, trained=4096, fast=1.0, slow=1.0) == SCALE and f(kind=3, trained=4096, slow=0.0) == SCALE
    assert f(out=None) == NULL
    with pytest.raises(KeyError):
        kda.rotary_freqs(16, scaling="other", device="cpu")


# ------------------------------------------------------------------ refusals

ROTARY = dict(q=addr(1), k=addr(2), qo=addr(3), ko=addr(4), pos=addr(5), freq=addr(6), B=2, T=8, H=4, HK=2, D=64, rot=32,
              ldq=0, ldk=0, ldqo=0, ldko=0, scale=1.0, mode=0, dt=1, stream=None)


def test_rotary_refusals(lib):
    f = lambda **kw: call(lib.kda_rotary, ROTARY, **kw)  # noqa: E731
    assert f(dt=2) == DTYPE and f(mode=4) == DTYPE
    for bad in (dict(D=48), dict(D=256), dict(rot=66), dict(rot=0), dict(rot=7), dict(B=-1), dict(T=-1), dict(H=-1),
                dict(HK=-1), dict(T=2 ** 31 - 1), dict(B=2 ** 24, T=2 ** 20), dict(ldq=255), dict(ldq=-256),
                dict(ldko=100)):
        assert f(**bad) == SHAPE, bad
    assert f(ldq=257) == ALIGN and f(q=addr(1) + 8) == ALIGN and f(pos=addr(5) + 4) == ALIGN
    assert f(q=None) == NULL and f(qo=None) == NULL and f(ko=None) == NULL and f(freq=None) == NULL
    for s in (math.nan, math.inf):
        assert f(scale=s) == SCALE
    # overlaps: a shifted view, the other input, each other, the positions; another stride in place
    assert f(qo=addr(1) + 64) == SHAPE and f(qo=addr(2)) == SHAPE and f(ko=addr(3)) == SHAPE and f(ko=addr(5)) == SHAPE
    assert f(qo=addr(1), ldqo=512) == SHAPE
    # nothing to do
    assert f(B=0) == 0 and f(T=0) == 0 and f(H=0, k=None) == 0


ATTN = dict(q=addr(1), k=addr(2), v=addr(3), ql=addr(4), kl=addr(5), o=addr(6), lse=addr(7), B=2, Tq=8, Tk=16, H=4, HK=2, D=64,
            ldq=0, ldk=0, ldv=0, scale=0.125, causal=1, window=0, dt=1, ws=None, ws_bytes=0, stream=None)
BWD = dict(q=addr(1), k=addr(2), v=addr(3), ql=addr(4), kl=addr(5), o=addr(6), lse=addr(7), do=addr(8), dq=addr(9), dk=addr(10),
           dv=addr(11), B=2, Tq=8, Tk=16, H=4, HK=2, D=64, ldq=0, ldk=0, ldv=0, scale=0.125, causal=1, window=0, dt=1,
           ws=addr(12), ws_bytes=1 << 20, stream=None)
BAD_SIZES = [dict(D=48), dict(D=256), dict(D=0), dict(B=-1), dict(Tq=-1), dict(Tk=-1), dict(H=-4), dict(HK=-2), dict(HK=3),
             dict(HK=0), dict(window=-1), dict(Tq=2 ** 31 - 1), dict(Tk=2 ** 31 - 1), dict(B=2 ** 22, Tq=4096),
             dict(B=2 ** 22, Tk=4096), dict(H=2 ** 22, HK=1, Tq=2 ** 12), dict(ldq=128), dict(ldk=64), dict(ldv=-128)]


def test_attn_bwd_refuses_more_row_pieces_than_a_grid_holds(lib):
    big = dict(B=1, Tq=2 ** 20, Tk=1, H=160, HK=160, D=128, dt=0, ws_bytes=1 << 40, causal=0)
    assert call(lib.kda_attn_bwd, BWD, **big) == SHAPE
    assert lib.kda_attn_bwd_workspace(1, 2 ** 20, 1, 160, 160, 128, 0) == 0
    assert lib.kda_attn_bwd_workspace(1, 2 ** 20, 1, 100, 100, 128, 0) > 0


def test_attn_refuses_scales_whose_inverse_overflows_the_statistics(lib):
    for f, args in ((lib.kda_attn_fwd, ATTN), (lib.kda_attn_bwd, BWD)):
        assert call(f, args, scale=1e-37) == SCALE and call(f, args, scale=2.0 ** -65) == SCALE
        assert call(f, args, scale=2.0 ** -64, B=0) == 0


def test_attn_step_takes_long_caches(lib):
    """The cache's length bounds no grid: 256 sequences of up to 2^20 tokens."""
    assert lib.kda_attn_step_workspace(256, 1, 32, 8, 128, 2 ** 20) == 0      # enough workgroups without a split
    assert lib.kda_attn_step_workspace(1, 1, 32, 8, 128, 2 ** 20) > 0


def test_attn_fwd_refusals(lib):
    f = lambda **kw: call(lib.kda_attn_fwd, ATTN, **kw)  # noqa: E731
    assert f(dt=9) == DTYPE
    for bad in BAD_SIZES:
        assert f(**bad) == SHAPE, bad
    assert f(ldk=132) == ALIGN and f(k=addr(2) + 2) == ALIGN and f(lse=addr(7) + 4) == ALIGN and f(ql=addr(4) + 4) == ALIGN
    for n in ("q", "k", "v", "o"):
        assert f(**{n: None}) == NULL
    for s in (0.0, -1.0, math.nan, math.inf, 3e38):
        assert f(scale=s) == SCALE, s
    for n in ("q", "k", "v", "ql", "kl", "lse"):
        assert f(o=ATTN[n]) == SHAPE, n
    assert f(lse=addr(1)) == SHAPE
    # the parts of one packed projection do not overlap each other, an output inside it does
    packed = dict(q=addr(1), k=addr(1) + 512, v=addr(1) + 768, ldq=512, ldk=512, ldv=512, Tk=8)
    assert f(o=addr(1) + 256, **packed) == SHAPE
    # few rows over many keys need a workspace
    need = lib.kda_attn_fwd_workspace(1, 1, 65536, 8, 2, 128, 1)
    big = dict(B=1, Tq=1, Tk=65536, H=8, HK=2, D=128)
    assert need > 0 and f(**big) == WORKSPACE and f(ws=addr(20) + 16, ws_bytes=need, **big) == WORKSPACE
    assert f(ws=addr(20), ws_bytes=need - 1, **big) == WORKSPACE
    assert f(ws=addr(6), ws_bytes=need, **big) == SHAPE           # the workspace over o
    assert f(B=0) == 0 and f(H=0, HK=0) == 0 and f(Tq=0) == 0


def test_attn_bwd_refusals(lib):
    f = lambda **kw: call(lib.kda_attn_bwd, BWD, **kw)  # noqa: E731
    assert f(dt=-1) == DTYPE
    for bad in BAD_SIZES:
        assert f(**bad) == SHAPE, bad
    for n in ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv"):
        assert f(**{n: None}) == NULL, n
        assert f(**{n: BWD[n] + 8}) == ALIGN, n
    for n in ("q", "k", "v", "o", "lse", "do", "ql", "kl", "ws"):
        for g in ("dq", "dk", "dv"):
            assert f(**{g: BWD[n]}) == SHAPE, (g, n)
    assert f(dq=addr(10)) == SHAPE and f(dv=addr(10)) == SHAPE
    need = lib.kda_attn_bwd_workspace(2, 8, 16, 4, 2, 64, 1)
    assert need >= 2 * 4 * 8 * 8
    assert f(ws=None) == WORKSPACE and f(ws_bytes=need - 1) == WORKSPACE and f(ws=addr(12) + 128) == WORKSPACE
    for s in (0.0, math.nan):
        assert f(scale=s) == SCALE
    assert f(B=0) == 0 and f(Tq=0, Tk=0) == 0


APPEND = dict(k=addr(1), v=addr(2), kc=addr(3), vc=addr(4), ks=addr(5), vs=addr(6), table=addr(7), cl=addr(8), nl=addr(9),
              n_pages=8, max_pages=4, B=2, T=5, HK=2, D=64, page=32, ldk=0, ldv=0, dt=1, stream=None)
STEP = dict(q=addr(1), kc=addr(3), vc=addr(4), ks=addr(5), vs=addr(6), table=addr(7), cl=addr(8), nl=addr(9), o=addr(10),
            n_pages=8, max_pages=4, B=2, Tq=1, H=4, HK=2, D=64, page=32, ldq=0, scale=0.125, window=0, dt=1, ws=None,
            ws_bytes=0, stream=None)


def test_cache_append_refusals(lib):
    f = lambda **kw: call(lib.kda_cache_append, APPEND, **kw)  # noqa: E731
    assert f(dt=3) == DTYPE
    for bad in (dict(D=48), dict(page=0), dict(page=8), dict(page=48), dict(page=256), dict(n_pages=-1), dict(max_pages=-1),
                dict(B=-1), dict(T=-1), dict(HK=-1), dict(n_pages=2 ** 30, HK=2), dict(max_pages=2 ** 30), dict(B=2 ** 23),
                dict(T=2 ** 30, page=16), dict(ldk=64), dict(ldv=-1)):
        assert f(**bad) == SHAPE, bad
    for n in ("k", "v", "kc", "vc", "ks", "vs", "table", "cl"):
        assert f(**{n: None}) == NULL, n
        assert f(**{n: APPEND[n] + 4}) == ALIGN, n
    assert f(nl=addr(9) + 4) == ALIGN
    for out in ("kc", "vc", "ks", "vs"):
        for n in ("k", "v", "table", "cl", "nl"):
            assert f(**{out: APPEND[n]}) == SHAPE, (out, n)
    assert f(kc=addr(4)) == SHAPE and f(vs=addr(5)) == SHAPE
    assert f(B=0) == 0 and f(T=0) == 0 and f(HK=0) == 0 and f(n_pages=0) == 0 and f(max_pages=0) == 0


def test_attn_step_refusals(lib):
    f = lambda **kw: call(lib.kda_attn_step, STEP, **kw)  # noqa: E731
    assert f(dt=7) == DTYPE
    for bad in (dict(D=48), dict(page=24), dict(n_pages=-1), dict(max_pages=-1), dict(B=-1), dict(Tq=-1), dict(H=3),
                dict(HK=0), dict(HK=-1), dict(window=-2), dict(n_pages=2 ** 30), dict(max_pages=2 ** 26), dict(ldq=8)):
        assert f(**bad) == SHAPE, bad
    for n in ("q", "kc", "vc", "ks", "vs", "table", "cl", "o"):
        assert f(**{n: None}) == NULL, n
        assert f(**{n: STEP[n] + 4}) == ALIGN, n
    for n in ("q", "kc", "vc", "ks", "vs", "table", "cl", "nl"):
        assert f(o=STEP[n]) == SHAPE, n
    for s in (0.0, -0.5, math.inf):
        assert f(scale=s) == SCALE
    need = lib.kda_attn_step_workspace(2, 1, 4, 2, 64, 2048 * 32)
    assert need > 0 and f(max_pages=2048) == WORKSPACE and f(max_pages=2048, ws=addr(11), ws_bytes=need - 1) == WORKSPACE
    assert f(B=0) == 0 and f(Tq=0) == 0


def test_workspace_sizes(lib):
    for bad in ((1, 1, 65536, 3, 2, 128, 1), (1, 1, 65536, 8, 2, 96, 1), (-1, 1, 65536, 8, 2, 128, 1), (1, 1, 65536, 8, 2, 128, 5)):
        assert lib.kda_attn_fwd_workspace(*bad) == 0 and lib.kda_attn_bwd_workspace(*bad) == 0
    assert lib.kda_attn_fwd_workspace(4, 4096, 4096, 16, 4, 128, 1) == 0          # enough rows to fill the card
    assert lib.kda_attn_step_workspace(256, 1, 32, 8, 128, 65536) == 0
    assert lib.kda_attn_step_workspace(1, 1, 8, 3, 128, 65536) == 0
    # two floats for each query, a head's padded to 64
    assert lib.kda_attn_bwd_workspace(2, 33, 50, 4, 2, 64, 1) == 2 * 4 * 64 * 8


# ------------------------------------------------------------------ the binding's integers

class OnDevice:
    """What the binding asks of a device tensor; nothing lies behind it."""

    is_cuda = True

    def __init__(self, shape, stride):
        self.shape, self._stride = shape, stride

    def numel(self):
        return math.prod(self.shape)

    def stride(self):
        return self._stride

    def is_contiguous(self):
        B, T, H, D = self.shape
        return self._stride == (T * H * D, H * D, D, 1)

    def data_ptr(self):
        return addr(1)


def test_strides_and_sizes_past_32_bits_are_refused():
    """The last token of [B, 2^20, 32, 128] lies 2^32 elements from the next sequence's: 0 in 32 bits."""
    for ld in (2 ** 32, 2 ** 32 + 4096, 2 ** 31, 2 ** 40):
        with pytest.raises(ValueError, match="apart"):
            kda._rows("q", OnDevice((4, 1, 32, 128), (ld, 4096, 128, 1)))
        with pytest.raises(ValueError, match="apart"):
            kda._rows("q", OnDevice((1, 4, 32, 128), (4 * ld, ld, 128, 1)))
    assert kda._rows("q", OnDevice((4, 1, 32, 128), (2 ** 20, 4096, 128, 1))) == (addr(1), 2 ** 20)
    for shape in ((1, 2 ** 32, 1, 16), (2 ** 32 + 2, 1, 1, 16), (1, 1, 2 ** 31, 16)):
        B, T, H, D = shape
        with pytest.raises(ValueError, match="q has"):
            kda._rows("q", OnDevice(shape, (T * H * D, H * D, D, 1)))
    meta = lambda *n, dtype=torch.int32: torch.empty(n, dtype=dtype, device="meta")  # noqa: E731
    kc, ks = meta(2, 1, 16, 16, dtype=torch.uint8), meta(2, 1, dtype=torch.float32)
    with pytest.raises(ValueError, match="block_table"):
        kda._cache_shapes(kc, kc, ks, ks, meta(1, 2 ** 32), meta(1), None, 1, 16, kc.device)
    assert kda._cache_shapes(kc, kc, ks, ks, meta(1, 8), meta(1), None, 1, 16, kc.device) == (2, 1, 16, 8)


def test_windows_past_32_bits_are_refused():
    """2^32 would arrive as no window at all."""
    x = torch.empty(1, 2, 2, 32, dtype=torch.bfloat16, device="meta")
    lse, n = torch.empty(1, 2, 2, device="meta"), torch.empty(1, dtype=torch.int32, device="meta")
    kc, vc, ks = (torch.empty(s, dtype=t, device="meta") for s, t in
                  (((2, 2, 16, 32), torch.uint8), ((2, 2, 32, 16), torch.uint8), ((2, 2), torch.float32)))
    table = torch.empty(1, 2, dtype=torch.int32, device="meta")
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 32):
        for call_ in (lambda: kda.attn_fwd(x, x, x, window=window), lambda: kda.attn_bwd(x, x, x, x, lse, x, window=window),
                      lambda: kda.attn_step(x, kc, vc, ks, ks, table, n, window=window)):
            with pytest.raises(ValueError, match="window"):
                call_()
    for kw in (dict(rot=2 ** 32 + 16), dict(rot=16, scaling="yarn", factor=2.0, trained=2 ** 32 + 64)):
        with pytest.raises(ValueError, match="32 bits"):
            kda.rotary_freqs(device="cpu", **kw)


def test_strides_of_tiles_are_bounded(lib):
    """Rows that are copied as tiles are addressed with 32-bit offsets: 2^23 elements between them at most."""
    far = 2 ** 23 + 8
    for n in ("ldk", "ldv"):
        assert call(lib.kda_attn_fwd, ATTN, **{n: far}) == SHAPE
    for n in ("ldq", "ldk", "ldv"):
        assert call(lib.kda_attn_bwd, BWD, **{n: far}) == SHAPE
    # elsewhere any multiple of 16 bytes passes the check (the next one refuses these calls)
    assert call(lib.kda_attn_fwd, ATTN, ldq=far, o=None) == NULL
    assert call(lib.kda_attn_step, STEP, ldq=far, o=None) == NULL
    for n in ("ldk", "ldv"):
        assert call(lib.kda_cache_append, APPEND, **{n: far}, kc=None) == NULL
    for n in ("ldq", "ldk", "ldqo", "ldko"):
        assert call(lib.kda_rotary, ROTARY, **{n: 2 ** 31 - 8}, freq=None) == NULL
        assert call(lib.kda_rotary, ROTARY, **{n: 2 ** 31 - 1}, freq=None) == ALIGN


def test_workspaces_of_another_device_are_refused():
    """Kernels would write through them; whether they are large enough does not matter."""
    given = torch.empty(256, dtype=torch.uint8, device="meta")
    for need in (0, 256, 512):
        for dev in ("cuda:0", "cuda:1", "cpu"):
            with pytest.raises(ValueError, match="workspace is on meta"):
                kda._workspace(need, given, torch.device(dev))
    # on the right one: used where it is large enough, as many bytes as it has
    assert kda._workspace(256, given, given.device) is given and kda._workspace(0, given, given.device) is given
    assert kda._workspace(1024, torch.empty(256, device="meta"), given.device).dtype is torch.float32
    assert kda._workspace(512, given, given.device).numel() == 512
    assert kda._workspace(0, None, given.device) is None
