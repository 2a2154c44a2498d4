"""Host validation of the operators that continue one prompt several times (no GPU: a
rejected call makes no HIP call), their workspace sizes and the binding's checks."""

import pytest
import torch

from gated_delta_rule_82_amd import kda
from tests.test_attn_abi_cpu import addr, call

NULL, SHAPE, ALIGN, DTYPE, WORKSPACE, SCALE = 1, 2, 3, 4, 6, 9


@pytest.fixture(scope="module")
def lib():
    return kda.load()


FORK = dict(table=addr(1), cl=addr(2), parent=addr(3), table_out=addr(4), len_out=addr(5), refs=addr(6), R=2, K_in=2, K_out=3,
            max_pages=4, n_pages=8, page=16, keep=0, stream=None)
RESERVE = dict(table=addr(1), refs=addr(2), cl=addr(3), nl=addr(4), src=addr(5), dst=addr(6), info=addr(7), B=2, T=1, max_pages=4,
               n_pages=8, page=16, stream=None)
FREE = dict(table=addr(1), refs=addr(2), lo=addr(3), hi=addr(4), B=2, max_pages=4, n_pages=8, page=16, stream=None)
COMPACT = dict(table=addr(1), refs=addr(2), table_out=addr(3), refs_out=addr(4), remap=addr(5), src=addr(6), dst=addr(7),
               info=addr(8), B=2, max_pages=4, n_pages=8, stream=None)
COPY = dict(k=addr(1), v=addr(2), ks=addr(3), vs=addr(4), kt=addr(5), vt=addr(6), kst=addr(7), vst=addr(8), src=addr(9),
            dst=addr(10), count=addr(11), n=3, n_src=8, n_dst=9, HK=2, D=64, page=32, stream=None)


def test_fork_refusals(lib):
    f = lambda **kw: call(lib.kda_cache_fork, FORK, **kw)  # noqa: E731
    for bad in (dict(page=0), dict(page=24), dict(page=256), dict(R=-1), dict(K_in=-1), dict(K_in=1025), dict(K_out=1025),
                dict(max_pages=-1), dict(n_pages=-1), dict(n_pages=2 ** 30 + 1), dict(R=2 ** 30), dict(max_pages=2 ** 29),
                dict(R=2 ** 22, K_in=1024, max_pages=0)):
        assert f(**bad) == SHAPE, bad
    for n in ("table", "cl", "parent", "table_out", "len_out", "refs"):
        assert f(**{n: None}) == NULL, n
        assert f(**{n: FORK[n] + 4}) == ALIGN, n
    for out in ("table_out", "len_out", "refs"):
        for n in set(FORK) & {"table", "cl", "parent", "table_out", "len_out", "refs"} - {out}:
            assert f(**{out: FORK[n]}) == SHAPE, (out, n)
    assert f(R=0) == 0 and f(K_in=0, K_out=0) == 0


def test_reserve_refusals(lib):
    f = lambda **kw: call(lib.kda_cache_reserve, RESERVE, **kw)  # noqa: E731
    for bad in (dict(page=8), dict(T=-1), dict(B=-1), dict(B=2 ** 30), dict(B=2 ** 28, max_pages=4), dict(max_pages=-1),
                dict(n_pages=-1), dict(T=2 ** 31 - 1, B=16)):
        assert f(**bad) == SHAPE, bad
    for n in ("table", "refs", "cl", "src", "dst", "info"):
        assert f(**{n: None}) == NULL, n
        assert f(**{n: RESERVE[n] + 8}) == ALIGN, n
    assert f(nl=addr(4) + 4) == ALIGN
    for out in ("table", "refs", "src", "dst", "info"):
        for n in {"table", "refs", "cl", "nl", "src", "dst", "info"} - {out}:
            assert f(**{out: RESERVE[n]}) == SHAPE, (out, n)


def test_free_refusals(lib):
    f = lambda **kw: call(lib.kda_cache_free, FREE, **kw)  # noqa: E731
    for bad in (dict(page=1), dict(B=-1), dict(max_pages=-1), dict(n_pages=-1), dict(B=2 ** 29)):
        assert f(**bad) == SHAPE, bad
    for n in ("table", "refs"):
        assert f(**{n: None}) == NULL and f(**{n: FREE[n] + 4}) == ALIGN
        for m in {"table", "refs", "lo", "hi"} - {n}:
            assert f(**{n: FREE[m]}) == SHAPE
    assert f(lo=addr(3) + 4) == ALIGN and f(hi=addr(4) + 4) == ALIGN
    assert f(B=0) == 0 and f(max_pages=0) == 0


def test_compact_refusals(lib):
    f = lambda **kw: call(lib.kda_cache_compact, COMPACT, **kw)  # noqa: E731
    for bad in (dict(B=-1), dict(max_pages=-1), dict(n_pages=-1), dict(n_pages=2 ** 30 + 1), dict(B=2 ** 29)):
        assert f(**bad) == SHAPE, bad
    names = {"table", "refs", "table_out", "refs_out", "remap", "src", "dst", "info"}
    for n in names:
        assert f(**{n: None}) == NULL and f(**{n: COMPACT[n] + 4}) == ALIGN
    for out in names - {"table", "refs"}:
        for n in names - {out}:
            if (out, n) not in (("table_out", "table"), ("refs_out", "refs")):    # in place
                assert f(**{out: COMPACT[n]}) == SHAPE, (out, n)
    assert f(table_out=addr(1) + 16) == SHAPE and f(refs_out=addr(2) + 16) == SHAPE


def test_copy_refusals(lib):
    f = lambda **kw: call(lib.kda_cache_copy, COPY, **kw)  # noqa: E731
    for bad in (dict(D=48), dict(page=48), dict(HK=-1), dict(n=-1), dict(n_src=-1), dict(n_dst=-1), dict(n_src=2 ** 30),
                dict(n_src=1, n_dst=1, HK=2 ** 20)):
        assert f(**bad) == SHAPE, bad
    names = ("k", "v", "ks", "vs", "kt", "vt", "kst", "vst", "src", "dst")
    for n in names:
        assert f(**{n: None}) == NULL and f(**{n: COPY[n] + 8}) == ALIGN
    assert f(count=addr(11) + 4) == ALIGN
    for out in ("kt", "vt", "kst", "vst"):
        for n in (set(names) | {"count"}) - {out}:
            assert f(**{out: COPY[n]}) == SHAPE, (out, n)
    # the same cache by all four pointers, of the same size
    one = dict(kt=addr(1), vt=addr(2), kst=addr(3), vst=addr(4))
    assert f(**one) == SHAPE and f(**one, n_dst=8, src=addr(1)) == SHAPE
    assert f(n=0) == 0 and f(n_src=0) == 0 and f(n_dst=0) == 0 and f(HK=0) == 0


SHARED = dict(q=addr(1), kc=addr(3), vc=addr(4), ks=addr(5), vs=addr(6), table=addr(7), cl=addr(8), nl=addr(9), gf=addr(10),
              pl=addr(11), o=addr(12), n_groups=2, n_pages=8, max_pages=4, B=2, Tq=1, H=4, HK=2, D=64, page=32, ldq=0, scale=0.125,
              window=0, dt=1, ws=addr(13), ws_bytes=1 << 30, stream=None)


def test_shared_refusals(lib):
    f = lambda **kw: call(lib.kda_attn_shared, SHARED, **kw)  # noqa: E731
    assert f(dt=7) == DTYPE
    for bad in (dict(D=48), dict(page=24), dict(n_pages=-1), dict(max_pages=-1), dict(B=-1), dict(Tq=-1), dict(H=3), dict(HK=0),
                dict(HK=-1), dict(window=-2), dict(n_pages=2 ** 30), dict(max_pages=2 ** 26), dict(ldq=8), dict(n_groups=-1),
                dict(n_groups=2 ** 24), dict(B=2 ** 20, Tq=1024, H=1, HK=1)):
        assert f(**bad) == SHAPE, bad
    for n in ("q", "kc", "vc", "ks", "vs", "table", "cl", "gf", "pl", "o"):
        assert f(**{n: None}) == NULL, n
        assert f(**{n: SHARED[n] + 4}) == ALIGN, n
    assert f(nl=addr(9) + 4) == ALIGN
    for n in ("q", "kc", "vc", "ks", "vs", "table", "cl", "nl", "gf", "pl", "ws"):
        assert f(o=SHARED[n]) == SHAPE, n
        if n != "ws":
            assert f(ws=SHARED[n]) == SHAPE, n
    for s in (0.0, -0.5, float("inf")):
        assert f(scale=s) == SCALE
    need = lib.kda_attn_shared_workspace(2, 1, 4, 2, 64, 2, 4 * 32)
    assert need > 0 and f(ws_bytes=need - 1) == WORKSPACE and f(ws=None) == WORKSPACE and f(ws=addr(13) + 16) == WORKSPACE
    assert f(B=0) == 0 and f(Tq=0) == 0 and f(H=0, HK=0) == 0


def test_shared_workspace(lib):
    ws = lib.kda_attn_shared_workspace
    for bad in ((2, 1, 4, 3, 64, 1, 64), (2, 1, 4, 2, 96, 1, 64), (-1, 1, 4, 2, 64, 1, 64), (2, 1, 4, 2, 64, -1, 64),
                (2, 1, 4, 2, 64, 1, -64)):
        assert ws(*bad) == 0
    # a part for the prefixes and one for the own keys at least: output, maximum and sum
    assert ws(2, 1, 4, 2, 64, 1, 64) == 2 * 8 * 64 * 4 + 256
    assert ws(256, 1, 32, 8, 128, 1, 2 ** 20) > 0


REORDER = dict(state=addr(1), out=addr(2), parent=addr(3), R=2, K_in=3, K_out=4, row_bytes=64, stream=None)


def test_reorder_refusals(lib):
    f = lambda **kw: call(lib.kda_state_reorder, REORDER, **kw)  # noqa: E731
    for bad in (dict(R=-1), dict(K_in=-1), dict(K_out=-1), dict(R=2 ** 24), dict(K_out=2 ** 24), dict(row_bytes=2 ** 41),
                dict(row_bytes=2 ** 40), dict(out=addr(1)), dict(out=addr(1) + 64), dict(out=addr(3)),
                dict(out=addr(1), K_in=65, K_out=65), dict(out=addr(1), K_in=4, R=2 ** 14, row_bytes=2 ** 22)):
        assert f(**bad) == SHAPE, bad
    assert f(row_bytes=24) == ALIGN
    for n in ("state", "out", "parent"):
        assert f(**{n: None}) == NULL and f(**{n: REORDER[n] + 8}) == ALIGN
    assert f(R=0) == 0 and f(K_out=0) == 0 and f(row_bytes=0) == 0


SELECT = dict(logits=addr(1), scores=addr(2), done=addr(3), scores_out=addr(4), parent=addr(5), token=addr(6), R=2, K=3, V=100,
              M=4, ld=0, end=5, dt=1, ws=addr(7), ws_bytes=1 << 30, stream=None)


def test_select_refusals(lib):
    f = lambda **kw: call(lib.kda_beam_select, SELECT, **kw)  # noqa: E731
    assert f(dt=2) == DTYPE
    for bad in (dict(R=-1), dict(K=0), dict(K=65), dict(V=0), dict(V=-1), dict(V=2 ** 30 + 1), dict(M=0), dict(M=65), dict(ld=99),
                dict(ld=-1), dict(end=-1), dict(end=100), dict(R=2 ** 18)):
        assert f(**bad) == SHAPE, bad
    for n in ("logits", "scores_out", "parent", "token"):
        assert f(**{n: None}) == NULL, n
    for n in ("logits", "scores", "done", "scores_out", "parent", "token"):
        assert f(**{n: SELECT[n] + 4}) == ALIGN, n
    for out in ("scores_out", "parent", "token"):
        for n in {"logits", "scores", "done", "scores_out", "parent", "token", "ws"} - {out}:
            assert f(**{out: SELECT[n]}) == SHAPE, (out, n)
    for n in ("logits", "scores", "done"):
        assert f(ws=SELECT[n]) == SHAPE
    need = lib.kda_beam_select_workspace(2, 3, 100, 4, 1)
    assert need > 0 and f(ws_bytes=need - 1) == WORKSPACE and f(ws=None) == WORKSPACE and f(ws=addr(7) + 64) == WORKSPACE
    assert f(R=0) == 0 and f(R=0, done=None, end=-1) == 0


def test_select_workspace(lib):
    ws = lib.kda_beam_select_workspace
    for bad in ((1, 0, 10, 1, 1), (1, 1, 0, 1, 1), (1, 1, 10, 65, 1), (-1, 1, 10, 1, 1), (1, 1, 10, 1, 9)):
        assert ws(*bad) == 0
    for R, K, V, M, dt in ((1, 1, 1, 1, 0), (64, 8, 131072, 16, 1), (1, 64, 2 ** 30, 64, 0), (1, 4, 32000, 8, 0)):
        assert ws(R, K, V, M, dt) >= R * K * (16 + 8 * M)


# ------------------------------------------------------------------ the binding

def meta(*n, dtype=torch.int32):
    return torch.empty(n, dtype=dtype, device="meta")


def test_binding_checks_shapes():
    t, n, refs = meta(4, 6), meta(4), meta(9)
    for bad in (lambda: kda.cache_fork(t, n, meta(3, 2), refs, page=16), lambda: kda.cache_fork(t, n, meta(8), refs, page=16),
                lambda: kda.cache_fork(t, meta(5), meta(2, 2), refs, page=16), lambda: kda.cache_fork(meta(4), n, meta(2, 2), refs, page=16),
                lambda: kda.cache_fork(t, n, meta(2, 2), refs, page=16, table_out=meta(4, 5)),
                lambda: kda.cache_fork(t, n, meta(0, 2), refs, page=16),
                lambda: kda.cache_reserve(t, meta(3), refs, page=16), lambda: kda.cache_reserve(t, n, refs, page=16, info=meta(3)),
                lambda: kda.cache_free(t, refs, meta(5), page=16), lambda: kda.cache_compact(t, meta(3, 3)),
                lambda: kda.cache_compact(t, refs, refs_out=meta(8)), lambda: kda.state_reorder(meta(5, 4), meta(2, 2)),
                lambda: kda.state_reorder(meta(4, 4), meta(4)), lambda: kda.beam_select(meta(2, 3, dtype=torch.float32)),
                lambda: kda.beam_select(meta(2, 3, 4, dtype=torch.float32))):     # not on a device
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: kda.cache_free(t, meta(9, dtype=torch.int64), page=16), lambda: kda.cache_reserve(t, n.float(), refs, page=16),
                lambda: kda.state_reorder(meta(4, 4), meta(2, 2, dtype=torch.int64))):
        with pytest.raises(TypeError):
            bad()


def test_integers_past_32_bits_are_refused():
    t, n, refs = meta(4, 6), meta(4), meta(9)
    with pytest.raises(ValueError, match="32 bits"):
        kda.cache_reserve(t, n, refs, T=2 ** 32 + 1, page=16, src=meta(4), dst=meta(4), info=meta(2))
    with pytest.raises(ValueError, match="32 bits"):
        kda.cache_free(meta(1, 2 ** 32), refs, page=16)
    with pytest.raises(ValueError, match="32 bits"):
        kda.cache_free(t, meta(2 ** 32), page=16)
    for bad in (lambda: kda.cache_fork(t, n, meta(2, 2), refs, page=2 ** 32 + 16), lambda: kda.cache_reserve(t, n, refs, page=2 ** 32 + 16),
                lambda: kda.cache_free(t, refs, page=2 ** 32 + 16), lambda: kda.beam_select(meta(2, 3, 4, dtype=torch.float32), M=2 ** 32 + 1),
                lambda: kda.beam_select(meta(2, 3, 4, dtype=torch.float32), end=2 ** 32)):
        with pytest.raises(ValueError, match="32 bits"):
            bad()
