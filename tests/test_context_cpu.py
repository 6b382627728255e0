"""The operators of long contexts without a GPU: their float64 definitions (oracle/paged.py) against hand-derived
values, and every refusal of the entry points that comes before any device work."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import paged as od
from test_decode_cpu import CACHE_FAULTS, P, _cache, _on, made_up_addresses, two_gpus  # noqa: F401 (a fixture)


@pytest.fixture(scope="module")
def b():
    import bit_weight_gemm_int2_amd as m
    m.lib()
    return m


# ------------------------------------------------------------ the definitions ---

def test_norm_by_hand():
    y = od.norm(np.array([[3.0, 4.0, 0.0, 0.0]]), np.array([1.0, 2.0, 3.0, 4.0]), 0.0)
    assert np.allclose(y, [[3 / 2.5, 2 * 4 / 2.5, 0, 0]])     # the mean square is 25 / 4
    assert (od.norm(np.zeros((2, 4)), np.ones(4), 0.0) == 0).all()
    assert np.allclose(od.norm(np.ones((1, 4)), np.ones(4), 3.0), 0.5)


def test_frequencies_by_hand():
    f, m = od.frequencies(64, 10000.0)
    assert m == 1 and f[0] == 1 and f[16] == pytest.approx(0.01) and len(f) == 32
    g, _ = od.frequencies(64, 10000.0, "linear", 4.0)
    assert np.allclose(g, f / 4)
    # ntk leaves the fastest frequency and divides the slowest by the factor
    g, _ = od.frequencies(64, 10000.0, "ntk", 4.0)
    assert g[0] == 1 and g[31] == pytest.approx(f[31] / 4)
    for kind in ("yarn", "wavelength"):
        g, m = od.frequencies(64, 10000.0, kind, 8.0, 2048, 1.0, 32.0)
        turns = 2048 * f / (2 * math.pi)
        assert m == (pytest.approx(0.1 * math.log(8) + 1) if kind == "yarn" else 1)
        assert np.allclose(g[0], f[0]) and np.allclose(g[-1], f[-1] / 8)      # many turns stay, few are divided
        assert (g <= f * (1 + 1e-12)).all() and (g >= f / 8 * (1 - 1e-12)).all()
        between = (g < f * 0.999) & (g > f / 8 * 1.001)
        assert between.any() and (turns[between] > 0.5).all() and (turns[between] < 50).all()
    # half of the way between low and high: half of the frequency is divided
    f1 = 2 * math.pi * 16.5 / 2048
    base = f1 ** (-64.0 / 10)                                  # the frequency of dimension 5
    g, _ = od.frequencies(64, base, "wavelength", 8.0, 2048, 1.0, 32.0)
    assert g[5] == pytest.approx(f1 * (0.5 + 0.5 / 8))


def test_attention_with_first_tokens_by_hand():
    g = np.random.default_rng(3)
    v, vs = g.standard_normal((9, 1, 4)), np.ones((9, 1))
    q = g.standard_normal((2, 1, 4))
    out, lse, _, _ = od.attention(q, np.zeros((9, 1, 4)), v, vs, 7, 0.5, True, 2, 3)   # equal scores: means
    assert np.allclose(out[0, 0], v[[0, 1, 2, 6, 7], 0].mean(0)) and np.allclose(out[1, 0], v[[0, 1, 2, 7, 8], 0].mean(0))
    assert np.allclose(lse, math.log(5))
    early, _, _, _ = od.attention(q, np.zeros((9, 1, 4)), v, vs, 1, 0.5, True, 1, 3)   # first tokens after a query stay hidden
    assert np.allclose(early[0, 0], v[:2, 0].mean(0))


def test_remap_by_hand():
    table = np.array([[5, 2, 7, -1], [5, 3, -1, -1]])
    # two sequences of 40 and 20 tokens in pages of 16 with a common first page
    new, L, pairs, counts = od.remap(table, [40, 20], 9, 16)
    assert new.tolist() == [[5, 2, 7, -1], [5, 3, -1, -1]] and pairs == [] and counts == [0, 4, 0, 0]
    # the first one forked: the second of its rows copies the last page to the lowest free one
    new, L, pairs, counts = od.remap(table, [40, 20], 9, 16, rows=[0, 0])
    assert new.tolist() == [[5, 2, 7, -1], [5, 2, 0, -1]] and pairs == [(7, 0)] and counts == [1, 4, 0, 0]
    # room of 9 tokens: 40 + 9 need a fourth page; an empty sequence gets its first
    new, L, pairs, counts = od.remap(table, [40, 20], 9, 16, rows=[0, -1], room=[9, 1])
    assert new.tolist() == [[5, 2, 7, 0], [1, -1, -1, -1]] and L.tolist() == [40, 0] and counts == [0, 5, 0, 0]
    # trimmed to 32 tokens by a narrower table: page 7 is free again, page 2 is whole
    new, L, pairs, counts = od.remap(table, [40, 20], 9, 16, rows=[0], width=2)
    assert new.tolist() == [[5, 2]] and L.tolist() == [32]
    # a window of 10: 40 - 10 = 30, so tokens 0 .. 30 are out of sight, but token 31 of the second page is seen
    assert od.remap(table, [40, 20], 9, 16, rows=[0], window=10)[0].tolist() == [[-1, 2, 7, -1]]
    assert od.remap(table, [40, 20], 9, 16, rows=[0], window=9)[0].tolist() == [[-1, -1, 7, -1]]
    assert od.remap(table, [40, 20], 9, 16, rows=[0], window=9, sinks=1)[0].tolist() == [[5, -1, 7, -1]]
    # compact: three pages in use become 0 .. 2; 5 and 7 move to 0 and 1
    new, L, pairs, counts = od.remap(table, [40, 20], 9, 16, rows=[0], compact=True)
    assert new.tolist() == [[0, 2, 1, -1]] and pairs == [(5, 0), (7, 1)] and counts == [2, 3, 0, 2]
    # no page left: the copy and the room find none
    new, L, pairs, counts = od.remap(table, [40, 20], 8, 16, rows=[0, 0, 0, 0, 1, 0], room=[0, 0, 9, 0, 0, 0])
    assert new[1:4, 2:].tolist() == [[0, -1], [1, 4], [6, -1]] and new[4].tolist() == [5, 3, -1, -1]
    assert new[5].tolist() == [5, 2, -1, -1] and counts == [3, 8, 1, 0]


# ------------------------------------------------------------------- refusals ---

@made_up_addresses
def test_kv_append_norm_refusals(b):
    Q = P + (8 << 32)
    good = dict(q=Q + 2048, qo=P + (9 << 32), qn=P + (12 << 32), kn=P + (13 << 32), nd=b.BF16, eps=1e-6, bad=None, T=40)

    def call(**kw):
        a = dict(good, **kw)
        return b.lib().lowbit_kv_append_norm(
            _cache(b), P + (4 << 32), 10, P + (5 << 32), P + (6 << 32), 3, a["T"], 20, b.BF16, Q, 1536, 128, Q + 1024, 1536, 128,
            a["q"], 1536, 128, 4, a["qo"], 512, 128, P + (10 << 32), P + (11 << 32), 128, 500, 0, a["qn"], a["kn"], a["nd"],
            a["eps"], a["bad"], None)

    assert call() == b.ERR_DEVICE                             # every check passes; there is no GPU here
    assert call(qn=None) == b.ERR_DEVICE and call(kn=None) == b.ERR_DEVICE and call(eps=0.0) == b.ERR_DEVICE
    assert call(qn=None, kn=None, nd=b.NONE) == b.ERR_DEVICE
    assert call(qn=None, q=None, qo=None) == b.ERR_DEVICE
    assert call(T=0, q=None, qo=None) == b.OK                 # no tokens: empty arrays may have no address
    for kw, want in ((dict(q=None, qo=None), "NULL"), (dict(qn=None, kn=None), "NULL"), (dict(nd=b.NONE), "DTYPE"),
                     (dict(nd=17), "DTYPE"), (dict(eps=-1.0), "SHAPE"), (dict(eps=float("nan")), "SHAPE"),
                     (dict(eps=float("inf")), "SHAPE"), (dict(kn=P + 8 + (13 << 32)), "ALIGN"),
                     (dict(qn=P + (1 << 32)), "OVERLAP"), (dict(kn=P + (9 << 32)), "OVERLAP"),
                     (dict(bad=P + (12 << 32)), "OVERLAP")):
        assert call(**kw) == getattr(b, "ERR_" + want), kw


@made_up_addresses
def test_attention_sinks_refusals(b):
    good = dict(cache=_cache(b), st=P + (6 << 32), T=3, mx=1, ml=1600, dt=b.F16, q=P + (8 << 32), hq=8, o=P + (9 << 32),
                win=100, sinks=4, ws=P + (10 << 32), wsb=1 << 30)

    def call(**kw):
        a = dict(good, **kw)
        return b.lib().lowbit_attention_sinks(a["cache"], P + (4 << 32), 100, P + (5 << 32), a["st"], 3, a["T"], a["mx"],
                                              a["ml"], a["dt"], a["q"], 1024, 128, a["hq"], a["o"], 1024, 128, None, 0.1, 1,
                                              a["win"], a["sinks"], a["ws"], a["wsb"], None)

    assert call() == b.ERR_DEVICE and call(sinks=1 << 40) == b.ERR_DEVICE and call(win=0) == b.ERR_DEVICE
    assert call(T=0, q=None, o=None) == b.OK
    for kw, want in ((dict(sinks=-1), "SHAPE"), (dict(win=-1), "SHAPE"), (dict(hq=6), "SHAPE"), (dict(q=None), "NULL"),
                     (dict(dt=b.F32), "DTYPE"), (dict(o=P + (8 << 32)), "OVERLAP"), (dict(ws=P + (1 << 32)), "OVERLAP")):
        assert call(**kw) == getattr(b, "ERR_" + want), kw
    for kw, want in CACHE_FAULTS:
        assert call(cache=_cache(b, **kw)) == getattr(b, "ERR_" + want), kw
    f, g = b.lib().lowbit_attention_workspace_bytes, b.lib().lowbit_attention_sinks_workspace_bytes
    for win in (0, 100, 5000):
        assert g(1, 1, 1, 100000, 32, 8, 128, 1, win, 0) == f(1, 1, 1, 100000, 32, 8, 128, win)
    assert g(1, 1, 1, 100000, 32, 8, 128, 1, 0, 50) == f(1, 1, 1, 100000, 32, 8, 128, 0)
    assert g(1, 1, 1, 100000, 32, 8, 128, 1, 5000, 100000) >= g(1, 1, 1, 100000, 32, 8, 128, 1, 5000, 4) > 0
    assert g(1, 1, 1, 100000, 32, 8, 128, 1, 5000, -1) == 0


@made_up_addresses
def test_norm_rotate_refusals(b):
    Q = P + (8 << 32)
    good = dict(dt=b.BF16, T=40, D=128, q=Q, qts=1536, qhs=128, hq=4, qo=P + (9 << 32), ots=512, ohs=128, k=Q + 1024, kts=1536,
                khs=128, hk=4, ko=P + (7 << 32), kots=512, kohs=128, qn=P + (12 << 32), kn=P + (13 << 32), nd=b.F32, eps=1e-6,
                cos=P + (10 << 32), sin=P + (11 << 32), rot=128, rows=500, pos=None, bad=None)

    def call(**kw):
        a = dict(good, **kw)
        return b.lib().lowbit_norm_rotate(a["dt"], a["T"], a["D"], a["q"], a["qts"], a["qhs"], a["hq"], a["qo"], a["ots"],
                                          a["ohs"], a["k"], a["kts"], a["khs"], a["hk"], a["ko"], a["kots"], a["kohs"], a["qn"],
                                          a["kn"], a["nd"], a["eps"], a["cos"], a["sin"], a["rot"], a["rows"], a["pos"], 0,
                                          a["bad"], None)

    assert call() == b.ERR_DEVICE
    assert call(k=None, ko=None, kn=None) == b.ERR_DEVICE and call(qn=None, kn=None, nd=b.NONE) == b.ERR_DEVICE
    assert call(cos=None, sin=None, rot=0) == b.ERR_DEVICE and call(pos=P) == b.ERR_DEVICE
    assert call(qo=Q, ots=1536, ko=Q + 1024, kots=1536) == b.ERR_DEVICE          # both in place
    assert call(T=0, q=None, qo=None, k=None, ko=None) == b.OK
    for kw, want in ((dict(dt=b.NONE), "DTYPE"), (dict(nd=5), "DTYPE"), (dict(D=96), "SHAPE"), (dict(T=-1), "SHAPE"),
                     (dict(hq=0), "SHAPE"), (dict(hk=70000), "SHAPE"), (dict(rot=48), "SHAPE"), (dict(rot=160), "SHAPE"),
                     (dict(rows=0), "SHAPE"), (dict(eps=-1e-9), "SHAPE"), (dict(ots=384), "SHAPE"), (dict(qts=-8), "SHAPE"),
                     (dict(q=None), "NULL"), (dict(qo=None), "NULL"), (dict(ko=None), "NULL"), (dict(k=None), "NULL"),
                     (dict(k=None, ko=None), "NULL"), (dict(cos=None), "NULL"), (dict(rot=0), "NULL"),
                     (dict(cos=None, sin=None, rot=0, pos=P), "NULL"), (dict(cos=None, sin=None, rot=0, qn=None, kn=None, nd=3), "NULL"),
                     (dict(qn=None, kn=None), "NULL"), (dict(q=Q + 8), "ALIGN"), (dict(qts=1540), "ALIGN"),
                     (dict(qn=P + 4 + (12 << 32)), "ALIGN"), (dict(pos=P + 2), "ALIGN"), (dict(bad=P + 1), "ALIGN"),
                     (dict(qo=Q, ots=2048), "OVERLAP"), (dict(qo=Q + 1024, ots=1536), "OVERLAP"), (dict(ko=Q, kots=1536), "OVERLAP"),
                     (dict(ko=P + (9 << 32)), "OVERLAP"), (dict(pos=P + (9 << 32)), "OVERLAP"), (dict(bad=Q), "OVERLAP"),
                     (dict(kn=P + (7 << 32)), "OVERLAP"), (dict(cos=P + (9 << 32)), "OVERLAP")):
        assert call(**kw) == getattr(b, "ERR_" + want), kw


@made_up_addresses
def test_rope_tables_refusals(b):
    good = dict(cos=P, sin=P + (1 << 32), n=1000, rot=128, first=0, base=1e4, kind=3, factor=4.0, orig=4096.0, low=1.0,
                high=32.0, mag=0.0)

    def call(**kw):
        a = dict(good, **kw)
        return b.lib().lowbit_rope_tables(a["cos"], a["sin"], a["n"], a["rot"], a["first"], a["base"], a["kind"], a["factor"],
                                          a["orig"], a["low"], a["high"], a["mag"], None)

    nan, inf = float("nan"), float("inf")
    for kind in range(5):
        assert call(kind=kind) == b.ERR_DEVICE
    assert call(kind=0, factor=0.0, orig=0.0, low=0.0, high=0.0) == b.ERR_DEVICE      # not read
    assert call(kind=1, orig=nan, low=nan) == b.ERR_DEVICE and call(n=1, first=(1 << 31) - 1) == b.ERR_DEVICE
    assert call(n=0, cos=None, sin=None) == b.OK
    for kw, want in ((dict(kind=5), "DTYPE"), (dict(kind=-1), "DTYPE"), (dict(n=-1), "SHAPE"), (dict(first=-1), "SHAPE"),
                     (dict(first=1 << 31), "SHAPE"), (dict(rot=0), "SHAPE"), (dict(rot=48), "SHAPE"), (dict(rot=288), "SHAPE"),
                     (dict(base=1.0), "SHAPE"), (dict(base=nan), "SHAPE"), (dict(base=inf), "SHAPE"), (dict(factor=0.5), "SHAPE"),
                     (dict(factor=nan), "SHAPE"), (dict(orig=0.0), "SHAPE"), (dict(low=0.0), "SHAPE"), (dict(high=1.0), "SHAPE"),
                     (dict(high=nan), "SHAPE"), (dict(mag=-1.0), "SHAPE"), (dict(mag=nan), "SHAPE"), (dict(cos=None), "NULL"),
                     (dict(sin=P + 8 + (1 << 32)), "ALIGN"), (dict(sin=P + 4096), "OVERLAP"), (dict(sin=P), "OVERLAP")):
        assert call(**kw) == getattr(b, "ERR_" + want), kw


@made_up_addresses
def test_page_call_refusals(b):
    L = b.lib()
    A = [P + (i << 32) for i in range(20)]
    good = dict(table=A[0], width=20, lens=A[1], batch=6, pages=500, page=16, rows=A[2], room=A[3], n=4, win=0, sinks=0, comp=0,
                new=A[4], wide=22, nl=A[5], src=A[6], dst=A[7], pairs=4, counts=A[8], ws=A[9], wsb=1 << 20)

    def call(**kw):
        a = dict(good, **kw)
        return L.lowbit_kv_remap(a["table"], a["width"], a["lens"], a["batch"], a["pages"], a["page"], a["rows"], a["room"],
                                 a["n"], a["win"], a["sinks"], a["comp"], a["new"], a["wide"], a["nl"], a["src"], a["dst"],
                                 a["pairs"], a["counts"], a["ws"], a["wsb"], None)

    assert call() == b.ERR_DEVICE and call(rows=None, room=None, n=6, pairs=6) == b.ERR_DEVICE
    assert call(batch=0, table=None, lens=None) == b.ERR_DEVICE                     # nothing old: new sequences alone
    for rows in (A[2], None):                                 # all end; an empty array may have no address
        assert call(n=0, new=None, nl=None, src=None, dst=None, pairs=0, rows=rows) == b.ERR_DEVICE
    assert call(comp=1, pairs=84) == b.ERR_DEVICE
    for kw, want in ((dict(page=48), "SHAPE"), (dict(pages=0), "SHAPE"), (dict(batch=-1), "SHAPE"), (dict(n=70000), "SHAPE"),
                     (dict(wide=1 << 30), "SHAPE"), (dict(win=-1), "SHAPE"), (dict(sinks=-1), "SHAPE"), (dict(pairs=3), "SHAPE"),
                     (dict(comp=1, pairs=83), "SHAPE"), (dict(rows=None), "SHAPE"), (dict(table=None), "NULL"),
                     (dict(lens=None), "NULL"), (dict(new=None), "NULL"), (dict(nl=None), "NULL"), (dict(src=None), "NULL"),
                     (dict(counts=None), "NULL"), (dict(room=P + 2), "ALIGN"), (dict(ws=A[9] + 128), "ALIGN"),
                     (dict(ws=None), "WORKSPACE"), (dict(wsb=256), "WORKSPACE"), (dict(new=A[0]), "OVERLAP"),
                     (dict(nl=A[1]), "OVERLAP"), (dict(dst=A[6] + 12), "OVERLAP"), (dict(ws=A[4]), "OVERLAP"),
                     (dict(counts=A[3]), "OVERLAP")):
        assert call(**kw) == getattr(b, "ERR_" + want), kw
    assert L.lowbit_kv_remap_pairs(20, 4, 500, 0) == 4 and L.lowbit_kv_remap_pairs(20, 4, 500, 1) == 84
    assert L.lowbit_kv_remap_pairs(200, 4, 500, 1) == 254 and L.lowbit_kv_remap_pairs(20, 4, 0, 0) == -1
    assert L.lowbit_kv_remap_workspace_bytes(4, 500) > 0 and L.lowbit_kv_remap_workspace_bytes(4, 0) == 0

    def copy(**kw):
        a = dict(dict(cache=_cache(b), src=A[6], dst=A[7], pairs=10, count=None), **kw)
        return L.lowbit_kv_copy_pages(a["cache"], a["src"], a["dst"], a["pairs"], a["count"], None)

    assert copy() == b.ERR_DEVICE and copy(count=A[8]) == b.ERR_DEVICE and copy(pairs=0, src=None, dst=None) == b.OK
    for kw, want in ((dict(src=None), "NULL"), (dict(dst=None), "NULL"), (dict(pairs=-1), "SHAPE"), (dict(src=A[6] + 1), "ALIGN"),
                     (dict(src=P), "OVERLAP"), (dict(count=P + (2 << 32)), "OVERLAP"), (dict(cache=_cache(b, v=P + 4096)), "OVERLAP")):
        assert copy(**kw) == getattr(b, "ERR_" + want), kw
    for kw, want in CACHE_FAULTS:
        assert copy(cache=_cache(b, **kw)) == getattr(b, "ERR_" + want), kw


# ------------------------------------------------------------------- devices ---

def _calls(gpu, **other):
    """Calls of the operators with every operand on `gpu`, but those named in `other`."""
    def t(name, shape, dtype):
        return _on(other.get(name, gpu), shape, dtype)
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16

    def cache(b):
        return b.KVCache(*(t("cache", (3, 2, 16, 64), torch.uint8) for _ in range(2)),
                         *(t("cache", (3, 2), f32) for _ in range(2)))

    rows = lambda n, h=2: t(n, (4, h, 64), bf)  # noqa: E731
    where = lambda: (_on(gpu, (1, 3), i32), _on(gpu, (2,), i32), _on(gpu, (1,), i32))  # noqa: E731
    turn = lambda: dict(cos=t("cos", (48, 32), f32), sin=t("sin", (48, 32), f32))  # noqa: E731
    return dict(
        append=lambda b: b.kv_append(_on(gpu, (4, 2, 64), bf), _on(gpu, (4, 2, 64), bf), cache(b), *where(), 4,
                                     q=_on(gpu, (4, 4, 64), bf), q_norm=t("q_norm", (64,), f32), k_norm=t("k_norm", (64,), f32)),
        turn=lambda b: b.norm_rotate(rows("q", 4), rows("k"), t("q_norm", (64,), bf), t("k_norm", (64,), bf), **turn(),
                                     positions=t("positions", (4,), i32), q_out=rows("q_out", 4), k_out=rows("k_out"),
                                     bad_count=t("bad", (1,), i32)),
        tables=lambda b: b.rope_tables(48, 64, out=(t("cos", (48, 32), f32), t("sin", (48, 32), f32))),
        attend=lambda b: b.attention(rows("q", 4), cache(b), *where(), 4, 4, window=3, sinks=2),
        copy=lambda b: b.kv_copy_pages(cache(b), t("src", (5,), i32), t("dst", (5,), i32), t("count", (4,), i32)))


@pytest.mark.parametrize("gpu", [0, 1])
def test_calls_run_on_their_operands_device(b, two_gpus, gpu):  # noqa: F811
    for call in _calls(gpu).values():
        call(b)
    made = {name: (device, args[-1]) for name, device, args in two_gpus.log}
    assert {d for d, _ in made.values()} == {gpu} and two_gpus.now == 0 and len(made) == 6
    assert all(q == 1000 + gpu for name, (_, q) in made.items() if "workspace" not in name)


@pytest.mark.parametrize("call,names", [
    ("append", ("q_norm", "k_norm")), ("attend", ("q",)), ("tables", ("sin",)),
    ("turn", ("k", "q_norm", "k_norm", "cos", "sin", "positions", "q_out", "k_out", "bad")),
    ("copy", ("src", "dst", "count"))])
def test_operands_of_another_device_are_refused(b, two_gpus, call, names):  # noqa: F811
    for name in names:
        for wrong in (1, -1):                                 # another GPU, the host
            with pytest.raises(ValueError, match="must be on"):
                _calls(0, **{name: wrong})[call](b)
    with pytest.raises(ValueError, match="must be on a GPU"):
        _calls(-1)[call](b)
    assert not [n for n, _, _ in two_gpus.log if "workspace" not in n]


def test_remap_operands(b, two_gpus):  # noqa: F811
    i32 = torch.int32
    cache = b.KVCache(_on(0, (3, 2, 16, 64), torch.uint8), _on(0, (3, 2, 16, 64), torch.uint8),
                      _on(0, (3, 2), torch.float32), _on(0, (3, 2), torch.float32))
    good = dict(block_table=_on(0, (2, 3), i32), lens=_on(0, (2,), i32), rows=_on(0, (5,), i32), room=_on(0, (5,), i32))
    for name, shape in (("block_table", (6,)), ("lens", (3,)), ("rows", (5, 1)), ("room", (4,))):
        with pytest.raises(ValueError):
            b.kv_remap(**dict(good, **{name: _on(0, shape, i32)}), cache=cache)
        with pytest.raises(ValueError, match="must be on"):
            b.kv_remap(**dict(good, **{name: _on(1, good[name].shape, i32)}), cache=cache)
        with pytest.raises(ValueError, match="int32"):
            b.kv_remap(**dict(good, **{name: _on(0, good[name].shape, torch.int64)}), cache=cache)
    assert not two_gpus.log


def test_python_refusals(b):
    with pytest.raises(ValueError, match="scaling"):
        b.rope_tables(10, 64, scaling="cubic")
    with pytest.raises(ValueError, match="GPU"):
        b.rope_tables(10, 64, device="cpu")
    x = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        b.norm_rotate(x, q_norm=torch.ones(64))


def test_python_refusals_of_shapes(b, two_gpus):  # noqa: F811
    bf, f32 = torch.bfloat16, torch.float32
    q, k, w = _on(0, (4, 4, 64), bf), _on(0, (4, 2, 64), bf), _on(0, (64,), f32)
    turn = dict(cos=_on(0, (9, 32), f32), sin=_on(0, (9, 32), f32))
    for kw, what in ((dict(q_norm=_on(0, (32,), f32)), "one type"), (dict(q_norm=w, k=k, k_norm=_on(0, (64,), bf)), "one type"),
                     (dict(k_norm=w), "without k"), (dict(), "neither"), (dict(positions=_on(0, (4,), torch.int32), q_norm=w), "without cos"),
                     (dict(turn, positions=_on(0, (4,), torch.int64)), "int32"), (dict(turn, positions=_on(0, (3,), torch.int32)), "int32"),
                     (dict(cos=turn["cos"]), "go together"), (dict(turn, k=_on(0, (3, 2, 64), bf)), "k must be"),
                     (dict(turn, k=_on(0, (4, 2, 64), f32)), "k must be"), (dict(turn, bad_count=_on(0, (2,), torch.int32)), "bad_count")):
        with pytest.raises(ValueError, match=what):
            b.norm_rotate(q, **kw)
    assert not two_gpus.log


def test_struct_and_signatures_hold_the_new_calls(b):
    names = {n for n, _, _ in b.SIGNATURES}
    for n in ("lowbit_kv_append_norm", "lowbit_norm_rotate", "lowbit_rope_tables", "lowbit_kv_remap", "lowbit_kv_copy_pages",
              "lowbit_attention_sinks"):
        assert n in names and isinstance(getattr(b.lib(), n), ctypes._CFuncPtr)


def test_attention_plan(b):
    """The test hook that names the kernels of a call agrees with the workspace that the call asks for; without a GPU it
    plans for 256 CUs. (Refusals need no GPU.)"""
    L = b.lib()
    for batch, tokens, new, length, hq, h, d, causal, window, sinks in (
            (1, 1, 1, 300, 8, 2, 128, 1, 0, 0), (4, 4, 1, 9000, 8, 1, 64, 1, 0, 0), (1, 90, 90, 4500, 1, 1, 256, 0, 0, 0),
            (1, 4096, 4096, 20000, 32, 8, 128, 1, 2500, 70), (48, 48, 1, 16000, 40, 8, 128, 1, 4096, 20),
            (24, 24, 1, 16000, 16, 4, 256, 1, 4000, 4), (1, 2000, 2000, 20000, 32, 8, 128, 1, 2500, 0)):
        plan = b.attention_plan(batch, tokens, new, length, hq, h, d, causal, window, sinks)
        assert plan.tile == (16 if new * hq // h <= 80 else plan.tile) and plan.tile in (16, 128, 256)
        assert plan.part_tokens % 128 == 0 and plan.parts * plan.part_tokens >= min(length, window + sinks if window else length)
        assert plan.join == (0 if plan.parts == 1 else 1 if plan.parts <= min(8, 1024 // d) and tokens * hq >= 512 else 2)
        need = (L.lowbit_attention_sinks_workspace_bytes(batch, tokens, new, length, hq, h, d, causal, window, sinks) if sinks else
                L.lowbit_attention_workspace_bytes(batch, tokens, new, length, hq, h, d, window))
        assert need == (plan.parts * tokens * hq * (d + 2) * 4 if plan.parts > 1 else 0)
    plan = (ctypes.c_int32 * 4)()
    call = L.lowbit_debug_attention_plan
    good = (1, 1, 1, 300, 8, 2, 128, 1, 0, 0)
    assert call(*good, plan) == b.OK and call(*good, None) == b.ERR_NULL
    for at, value in ((0, 0), (0, 65536), (1, 0), (1, 1 << 31), (2, 0), (3, -1), (3, (1 << 30) + 1), (4, 1), (4, 65537), (5, 0), (6, 96),
                      (6, 0), (8, -1), (9, -1)):
        assert call(*good[:at], value, *good[at + 1:], plan) == b.ERR_SHAPE, (at, value)
    with pytest.raises(b.LowbitError):
        b.attention_plan(0, 1, 1, 300, 8, 2, 128)


@pytest.mark.parametrize("window,parts", [(4000, 4), (1000, 3)])
def test_plan_of_few_rows_knows_which_join_heads_of_256_take(b, window, parts):
    """Where 5 parts with a workgroup a row to join and 3 or 4 joined by rows come out nearly alike, the dearer join counts
    (48 sequences of 16 heads; on 256 CUs)."""
    plan = b.attention_plan(48, 48, 1, 4 * window, 16, 1, 256, True, window, 4)
    assert plan.join == 1 and plan.parts == parts
