"""The decoding operators without a GPU: the float64 definitions (oracle/paged.py)
against hand-derived values and closed forms, and every refusal of the entry
points that comes before any device work."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged as od

made_up_addresses = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                       reason="made-up device addresses; CPU-only checks")
P = 1 << 40


@pytest.fixture(scope="module")
def b():
    import bit_weight_gemm_int2_amd as m
    m.lib()
    return m


# ------------------------------------------------------------ the definitions ---

def test_block_layout_by_hand():
    # keys, D = 64: token 17 is token 1 of the second tile of 16; d = 35 is byte 3 of piece 2
    assert od.k_place(17, 35, 64) == 16 * 64 + 2 * 256 + 16 + 3
    # values, D = 64: token 6 is token 2 of the second quad
    assert od.v_place(6, 35, 64) == 256 + 4 * 35 + 2
    for page, D in ((16, 64), (64, 128), (256, 256)):
        t, d = np.meshgrid(np.arange(page), np.arange(D), indexing="ij")
        for place in (od.k_place, od.v_place):
            assert np.array_equal(np.sort(place(t, d, D).ravel()), np.arange(page * D))   # a permutation


@pytest.mark.parametrize("which", ["k", "v"])
def test_block_round_trip(which):
    codes = np.random.default_rng(1).integers(-127, 128, (32, 64))
    assert np.array_equal(od.block_codes(od.block_bytes(codes, which), which, 32, 64), codes)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_a_rotation(inter):
    x = np.random.default_rng(2).standard_normal((3, 2, 64))
    a = np.arange(10)[:, None] * 0.3 ** np.arange(16)
    y = od.rotate(x, np.array([0, 1, 7]), np.cos(a), np.sin(a), inter)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[:, :, 32:], x[:, :, 32:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-14)
    # turned back by the opposite angle
    assert np.allclose(od.rotate(y, np.array([0, 1, 7]), np.cos(a), -np.sin(a), inter), x, atol=1e-14)
    # one pair by hand: a quarter turn takes (x, y) to (-y, x)
    q = od.rotate(x[:1], np.array([0]), np.zeros((1, 16)), np.ones((1, 16)), inter)
    i, j = (4, 5) if inter else (2, 18)
    assert q[0, 0, i] == -x[0, 0, j] and q[0, 0, j] == x[0, 0, i]


def test_append_block_by_hand():
    codes, scale = od.append_block(np.zeros((16, 64), dtype=np.int64), 5.0, 0, np.full((1, 64), 12.7))
    assert scale == pytest.approx(0.1) and (codes[0] == 127).all() and (codes[1:] == 0).all()
    codes[0, 0] = 63
    twice, s2 = od.append_block(codes, scale, 1, np.full((2, 64), -25.4))     # twice the scale: codes halve
    assert s2 == pytest.approx(0.2)
    assert twice[0, 0] == 32 and (twice[0, 1:] == 64).all() and (twice[1:3] == -127).all()   # 31.5 and 63.5 to even
    same, s3 = od.append_block(twice, s2, 3, np.full((1, 64), 0.2))
    assert s3 == s2 and np.array_equal(same[:3], twice[:3]) and (same[3] == 1).all()


def test_attention_closed_forms():
    g = np.random.default_rng(3)
    v, vs = g.standard_normal((6, 1, 4)), np.ones((6, 1))
    q = g.standard_normal((2, 2, 4))
    out, lse, _, _ = od.attention(q, np.zeros((6, 1, 4)), v, vs, 4, 0.5, True, 0)   # equal scores: means
    assert np.allclose(out[0, 0], v[:5, 0].mean(0)) and np.allclose(out[1, 1], v[:, 0].mean(0))
    assert np.allclose(lse, np.log([[5, 5], [6, 6]]))
    one, l1, _, _ = od.attention(q, g.standard_normal((6, 1, 4)), v, vs, 4, 0.5, True, 1)   # only itself
    assert np.allclose(one[:, 0], v[4:, 0])
    none, ln, _, _ = od.attention(q, np.zeros((6, 1, 4)), v, vs, -3, 0.5, True, 0)
    assert (none == 0).all() and np.isneginf(ln).all()


# ------------------------------------------------------------------- refusals ---

@made_up_addresses
def test_gemv_int4_refusals(b):
    L = b.lib()
    good = dict(X=P, xd=b.BF16, M=4, K=256, ldx=256, W=P + (1 << 30), S=P + (2 << 30), Z=P + (3 << 30), group=128,
                N=64, bias=None, bd=b.NONE, Y=P + (4 << 30), yd=b.F32, ldy=64, act=0)

    def call(**kw):
        a = dict(good, **kw)
        return L.lowbit_gemv_int4(a["X"], a["xd"], a["M"], a["K"], a["ldx"], a["W"], a["S"], a["Z"], a["group"],
                                  a["N"], a["bias"], a["bd"], a["Y"], a["yd"], a["ldy"], a["act"], None)

    assert call() == b.ERR_DEVICE                             # every check passes; there is no GPU here
    for kw, want in ((dict(M=17), b.ERR_SHAPE), (dict(M=0), b.ERR_SHAPE), (dict(K=200), b.ERR_SHAPE),
                     (dict(Z=None), b.ERR_NULL), (dict(S=None), b.ERR_NULL), (dict(Z=P + (3 << 30) + 1), b.ERR_ALIGN),
                     (dict(X=P + 8), b.ERR_ALIGN), (dict(xd=b.F32), b.ERR_DTYPE), (dict(act=7), b.ERR_DTYPE),
                     (dict(group=64), b.ERR_GROUP), (dict(ldx=128), b.ERR_SHAPE), (dict(ldy=60), b.ERR_SHAPE),
                     (dict(N=1 << 25, ldy=1 << 25), b.ERR_SHAPE), (dict(bd=b.F16), b.ERR_NULL),
                     (dict(Y=P + (3 << 30)), b.ERR_OVERLAP), (dict(Y=P + (1 << 30)), b.ERR_OVERLAP),
                     (dict(Y=P), b.ERR_OVERLAP)):
        assert call(**kw) == want, kw


def _cache(b, **kw):
    a = dict(k=P, v=P + (1 << 32), ks=P + (2 << 32), vs=P + (3 << 32), pages=100, heads=4, page=16, d=128)
    a.update(kw)
    return ctypes.byref(b._CacheStruct(a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["heads"], a["page"], a["d"]))


CACHE_FAULTS = [(dict(k=None), "NULL"), (dict(vs=None), "NULL"), (dict(pages=0), "SHAPE"), (dict(heads=0), "SHAPE"),
                (dict(heads=5000), "SHAPE"), (dict(pages=1 << 30), "SHAPE"), (dict(page=48), "SHAPE"),
                (dict(page=512), "SHAPE"), (dict(d=96), "SHAPE"), (dict(k=P + 8), "ALIGN"), (dict(ks=P + 2), "ALIGN")]


@made_up_addresses
def test_kv_append_and_read_refusals(b):
    L = b.lib()
    T = 40
    Q = P + (8 << 32)
    good = dict(cache=_cache(b), table=P + (4 << 32), width=10, cu=P + (5 << 32), st=P + (6 << 32), batch=3, T=T, mx=20,
                dt=b.BF16, k=Q, kts=1536, khs=128, v=Q + 1024, vts=1536, vhs=128, q=Q + 2048, qts=1536, qhs=128, hq=4,
                qo=P + (9 << 32), ots=512, ohs=128, cos=P + (10 << 32), sin=P + (11 << 32), rot=128, rows=500, bad=None)

    def call(**kw):
        a = dict(good, **kw)
        return L.lowbit_kv_append(a["cache"], a["table"], a["width"], a["cu"], a["st"], a["batch"], a["T"], a["mx"],
                                  a["dt"], a["k"], a["kts"], a["khs"], a["v"], a["vts"], a["vhs"], a["q"], a["qts"],
                                  a["qhs"], a["hq"], a["qo"], a["ots"], a["ohs"], a["cos"], a["sin"], a["rot"],
                                  a["rows"], 0, a["bad"], None)

    assert call() == b.ERR_DEVICE
    assert call(qo=Q + 2048, ots=1536) == b.ERR_DEVICE        # the queries in place, between the keys and values
    assert call(q=None, qo=None) == b.ERR_DEVICE and call(rot=0, cos=None, sin=None) == b.ERR_DEVICE
    assert call(T=0, k=None, v=None, q=None, qo=None) == b.OK
    assert call(T=0, k=None, v=None, q=None, qo=None, batch=0, mx=0) == b.OK
    for kw, want in ((dict(table=None), "NULL"), (dict(cu=None), "NULL"), (dict(k=None), "NULL"), (dict(qo=None), "NULL"),
                     (dict(cos=None), "NULL"), (dict(rot=0), "NULL"), (dict(dt=b.NONE), "DTYPE"), (dict(batch=0), "SHAPE"),
                     (dict(batch=70000), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(mx=0), "SHAPE"), (dict(rot=48), "SHAPE"),
                     (dict(rot=160), "SHAPE"), (dict(rows=0), "SHAPE"), (dict(hq=0), "SHAPE"), (dict(kts=-8), "SHAPE"),
                     (dict(kts=1540), "ALIGN"), (dict(k=Q + 8), "ALIGN"), (dict(cos=P + 4 + (10 << 32)), "ALIGN"),
                     (dict(cu=P + 2 + (5 << 32)), "ALIGN"), (dict(ots=384), "SHAPE"), (dict(ohs=64), "SHAPE"),
                     (dict(qo=P), "OVERLAP"), (dict(k=P), "OVERLAP"), (dict(q=P + (2 << 32)), "OVERLAP"),
                     (dict(qo=Q, ots=1536), "OVERLAP"), (dict(qo=Q + 2048 - 256, ots=1536), "OVERLAP"),
                     (dict(qo=Q + 2048, ots=2048), "OVERLAP"), (dict(bad=P + 64), "OVERLAP"),
                     (dict(table=P + (3 << 32)), "OVERLAP"), (dict(cache=_cache(b, v=P + 4096)), "OVERLAP")):
        assert call(**kw) == getattr(b, "ERR_" + want), kw
    for kw, want in CACHE_FAULTS:
        assert call(cache=_cache(b, **kw)) == getattr(b, "ERR_" + want), kw
    assert call(cache=None) == b.ERR_NULL

    def read(**kw):
        a = dict(good, k=Q, kts=512, khs=128, v=P + (9 << 32), vts=512, vhs=128)
        a.update(kw)
        return L.lowbit_kv_read(a["cache"], a["table"], a["width"], a["cu"], a["st"], a["batch"], a["T"], a["mx"], a["dt"],
                                a["k"], a["kts"], a["khs"], a["v"], a["vts"], a["vhs"], None)

    assert read() == b.ERR_DEVICE and read(T=0, k=None, v=None) == b.OK
    assert read(kts=1024, v=Q + 1024, vts=1024) == b.ERR_DEVICE   # keys and values of a token side by side
    for kw, want in ((dict(k=None), "NULL"), (dict(khs=120), "SHAPE"), (dict(kts=256), "SHAPE"), (dict(dt=9), "DTYPE"),
                     (dict(v=Q), "OVERLAP"), (dict(v=Q + 1008), "OVERLAP"), (dict(k=P), "OVERLAP"),
                     (dict(cu=P + (9 << 32)), "OVERLAP")):
        assert read(**kw) == getattr(b, "ERR_" + want), kw


@made_up_addresses
def test_attention_refusals(b):
    L = b.lib()
    good = dict(cache=_cache(b), table=P + (4 << 32), width=100, cu=P + (5 << 32), st=P + (6 << 32), batch=3, T=3, mx=1,
                ml=1600, dt=b.F16, q=P + (8 << 32), qts=1024, qhs=128, hq=8, o=P + (9 << 32), ots=1024, ohs=128, lse=None,
                win=0, ws=P + (10 << 32), wsb=1 << 30)

    def call(**kw):
        a = dict(good, **kw)
        return L.lowbit_attention(a["cache"], a["table"], a["width"], a["cu"], a["st"], a["batch"], a["T"], a["mx"],
                                  a["ml"], a["dt"], a["q"], a["qts"], a["qhs"], a["hq"], a["o"], a["ots"], a["ohs"],
                                  a["lse"], 0.1, 1, a["win"], a["ws"], a["wsb"], None)

    assert call() == b.ERR_DEVICE
    assert call(T=0, q=None, o=None) == b.OK
    for kw, want in ((dict(dt=b.F32), "DTYPE"), (dict(hq=6), "SHAPE"), (dict(hq=0), "SHAPE"), (dict(ml=-1), "SHAPE"),
                     (dict(ml=(1 << 30) + 1), "SHAPE"), (dict(win=-1), "SHAPE"), (dict(q=None), "NULL"),
                     (dict(o=None), "NULL"), (dict(st=None), "NULL"), (dict(qts=1020), "ALIGN"),
                     (dict(q=P + 2 + (8 << 32)), "ALIGN"), (dict(lse=P + 1), "ALIGN"), (dict(ots=512), "SHAPE"),
                     (dict(T=1 << 20, mx=1 << 30, hq=256), "SHAPE"),
                     (dict(o=P + (8 << 32)), "OVERLAP"), (dict(o=P + (1 << 32)), "OVERLAP"),
                     (dict(lse=P + (9 << 32)), "OVERLAP"), (dict(ws=P + (8 << 32)), "OVERLAP"),
                     (dict(ws=P + (2 << 32)), "OVERLAP"), (dict(lse=P + (10 << 32)), "OVERLAP")):
        assert call(**kw) == getattr(b, "ERR_" + want), kw
    for kw, want in CACHE_FAULTS:
        assert call(cache=_cache(b, **kw)) == getattr(b, "ERR_" + want), kw


def test_attention_workspace_query(b):
    f = b.lib().lowbit_attention_workspace_bytes
    assert f(0, 1, 1, 100, 8, 8, 128, 0) == 0 and f(1, 0, 1, 100, 8, 8, 128, 0) == 0
    assert f(4, 4, 1, 0, 8, 8, 128, 0) == 0                  # nothing cached: one part
    few = f(1, 1, 1, 100000, 32, 8, 128, 0)
    assert few % (32 * 130 * 4) == 0 and few // (32 * 130 * 4) >= 25   # parts of at most 4096 tokens
    assert f(1, 1, 1, 100000, 32, 8, 128, 200) < few          # a window needs fewer parts
    assert f(64, 64 * 512, 512, 4096, 32, 8, 128, 0) == 0     # prompts that fill the GPU are not split


@made_up_addresses
def test_an_empty_batch_needs_no_addresses(b):
    """No sequences and no tokens: the arrays are empty, and an empty array's address may be null."""
    L, none = b.lib(), (None, 7, None, None, 0, 0, 0)
    assert L.lowbit_kv_append(_cache(b), *none, b.BF16, None, 512, 128, None, 512, 128, None, 0, 0, 0, None, 0, 0, None,
                              None, 0, 0, 0, None, None) == b.OK
    assert L.lowbit_kv_read(_cache(b), *none, b.F32, None, 512, 128, None, 512, 128, None) == b.OK
    assert L.lowbit_attention(_cache(b), *none, 0, b.F16, None, 1024, 128, 8, None, 1024, 128, None, 0.1, 1, 0, None, 0,
                              None) == b.OK
    some = (None, 7, None, None, 0, 3, 3)                     # tokens of no sequence
    assert L.lowbit_kv_read(_cache(b), *some, b.F32, P, 512, 128, P, 512, 128, None) == b.ERR_NULL
    for i in range(3):                                        # sequences without their arrays
        ptr = [P + (4 << 32), P + (5 << 32), P + (6 << 32)]
        ptr[i] = None
        assert L.lowbit_kv_read(_cache(b), ptr[0], 7, ptr[1], ptr[2], 2, 0, 0, b.F32, None, 512, 128, None, 512, 128,
                                None) == b.ERR_NULL


def test_python_refusals(b):
    cpu = torch.zeros((2, 1, 16, 64), dtype=torch.uint8)
    s = torch.zeros((2, 1))
    with pytest.raises(ValueError):
        b.KVCache(cpu, cpu, s, s)                             # not on a GPU
    with pytest.raises(ValueError):
        b.KVCache(cpu[0], cpu, s, s)
    with pytest.raises(ValueError):
        b.KVCache(cpu, cpu, s[:1], s)
    with pytest.raises(ValueError):
        b.gemv_int4(torch.zeros(1, 128), torch.zeros((4, 64), dtype=torch.uint8), s, s)


def test_a_workspace_is_one_dense_block(b):
    """One byte expanded to 4096, and every other byte of a block, are not 4096 bytes to write to."""
    for t in (torch.empty(1, dtype=torch.uint8).expand(4096), torch.empty(8192, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            b._given_workspace(t, 4096, "a call")
    with pytest.raises(ValueError, match="GPU"):
        b._given_workspace(torch.empty(4096, dtype=torch.uint8), 4096, "a call")


# ------------------------------------------------------------------- devices ---

class On(torch.Tensor):
    """A host tensor that says it is on GPU `gpu` (the checks go by get_device)."""

    def get_device(self):
        return self.gpu


def _on(gpu, shape, dtype):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.gpu = gpu
    return t


class Library:
    """Stands in for the library: notes the device that is current in each call."""

    def __init__(self, log):
        self.log = log

    def __getattr__(self, name):
        return lambda *args: self.log.append((name, self.now, args)) or 0


@pytest.fixture
def two_gpus(b, monkeypatch):
    lib = Library([])
    lib.now = 0

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.was, lib.now = lib.now, self.index

        def __exit__(self, *exc):
            lib.now = self.was

    monkeypatch.setattr(b, "lib", lambda: lib)
    monkeypatch.setattr(b, "_new", lambda shape, dtype, like, stream: _on(like.gpu, shape, dtype))
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: lib.now, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    return lib


def _operands(gpu, **other):
    """Calls of the four operators with every operand on `gpu`, but those named in `other`."""
    def t(name, shape, dtype):
        return _on(other.get(name, gpu), shape, dtype)
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16

    def cache(b):
        return b.KVCache(t("k_cache", (3, 2, 16, 64), torch.uint8), t("v_cache", (3, 2, 16, 64), torch.uint8),
                         t("k_scale", (3, 2), f32), t("v_scale", (3, 2), f32))

    def where():
        return t("block_table", (1, 3), i32), t("cu", (2,), i32), t("starts", (1,), i32)

    rows = lambda n, h=2: t(n, (4, h, 64), bf)  # noqa: E731
    return dict(
        gemv=lambda b: b.gemv_int4(t("x", (2, 128), bf), t("packed", (8, 64), torch.uint8), t("scales", (8, 1), torch.float16),
                                   t("zeros", (8, 1), torch.float16), bias=t("bias", (8,), f32), out=t("out", (2, 8), bf)),
        append=lambda b: b.kv_append(rows("k"), rows("v"), cache(b), *where(), 4, q=rows("q", 4), cos=t("cos", (48, 32), f32),
                                     sin=t("sin", (48, 32), f32), q_out=rows("q_out", 4), bad_count=t("bad", (2,), i32)),
        read=lambda b: b.kv_read(cache(b), *where(), 4, 4, bf, out=(rows("k_out"), rows("v_out"))),
        attend=lambda b: b.attention(rows("q", 4), cache(b), *where(), 4, 4, out=rows("out", 4), return_lse=True))


@pytest.mark.parametrize("gpu", [0, 1])
def test_calls_run_on_their_operands_device(b, two_gpus, gpu):
    for call in _operands(gpu).values():
        call(b)
    made = {name: (device, args[-1]) for name, device, args in two_gpus.log}
    assert {d for d, _ in made.values()} == {gpu} and two_gpus.now == 0 and len(made) == 5
    assert all(q == 1000 + gpu for name, (_, q) in made.items() if "workspace" not in name)   # that device's current stream


@pytest.mark.parametrize("call,names", [
    ("gemv", ("x", "packed", "scales", "zeros", "bias", "out")),
    ("append", ("k", "v", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "cu", "starts", "q", "cos", "sin",
                "q_out", "bad")),
    ("read", ("k_cache", "v_scale", "block_table", "cu", "starts", "k_out", "v_out")),
    ("attend", ("q", "k_cache", "v_scale", "block_table", "cu", "starts", "out"))])
def test_operands_of_another_device_are_refused(b, two_gpus, call, names):
    for name in names:
        for wrong in (1, -1):                                 # another GPU, the host
            with pytest.raises(ValueError, match="must be on"):
                _operands(0, **{name: wrong})[call](b)
    with pytest.raises(ValueError, match="must be on a GPU"):
        _operands(-1)[call](b)
    assert not two_gpus.log


def test_a_cache_keeps_its_tensors(b, two_gpus):
    """The calls go by the addresses taken when the cache was made: assigning a larger tensor would leave them behind."""
    ts = [_on(0, shape, dt) for shape, dt in (((3, 2, 16, 64), torch.uint8),) * 2 + (((3, 2), torch.float32),) * 2]
    cache = b.KVCache(*ts)
    assert all(getattr(cache, n) is t for n, t in zip(("k", "v", "k_scale", "v_scale"), ts))
    for n in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(cache, n, _on(0, (6, 2, 16, 64), torch.uint8))
    assert cache.struct.k == ts[0].data_ptr() and cache.struct.v_scale == ts[3].data_ptr()


def test_a_stream_of_another_device_is_refused(b, two_gpus):
    class Stream:
        device_index, cuda_stream = 1, 77

    assert b._queue(Stream, 1) == 77
    with pytest.raises(ValueError, match="stream"):
        b._queue(Stream, 0)
