"""GPU parity of the decoding operators against float64 NumPy definitions
(oracle/paged.py): 4-bit products of 1 .. 16 rows, appending to and reading the
8-bit paged cache, and attention over it.

Tolerances, from the contracts of include/lowbit.h:
* 4-bit products: 1e-3 sum|x w| + 1e-5 + 2^-19 (16 + max|z|) sum|x s| (+ half an
  output ulp).
* append: a stored value is within 0.5001 scale of the rotated input (0.5 from the
  rounding to a code, the rest FP32 rounding of the rotation and the quotient:
  a few 2^-24 of 127 steps), older values that followed a grown scale within half
  of the new one more. Scales within 2^-20 relatively (FP32 rotation of the
  largest value: three roundings of terms up to sqrt 2 of it, and one division).
* read: exact scale * code, rounded once to the output type.
* attention: |d| <= 2^-10 sum p |v| / sum p + 2^-25 tokens 127 max(p v_scale) / sum p
  + half an output ulp. FP16 probabilities p v_scale / max are within 2^-11
  relatively, or 2^-25 below FP16's normal range; queries are scaled exactly and
  BF16 ones fit FP16's 11 bits; FP32 score rounding adds about 2^-23 |q| |k| scale
  (< 2^-13 in these tests) to each exponent, inside the other half of 2^-10.
* lse: 2^-14 absolute plus 2^-22 relative, FP32 scores, exponent and logarithm."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from oracle import paged as od
from gpu_util import TORCH_DT, banner, dev_bits, to_host64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import bit_weight_gemm_int2_amd as b
    b.lib()
    return b


def _f16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float16).view(np.int16)).cuda().view(torch.float16)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _half_ulp(y, dtype):
    if dtype == torch.float32:
        return 0.0
    bits, low = (8, -133) if dtype == torch.bfloat16 else (11, -24)
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -140)))
    return 0.5 * 2.0 ** np.maximum(e - bits + 1, low)


# ------------------------------------------------- 4-bit products of few rows ---

def _gemv_check(lb, lin, act=None, x=None, out=None, bias=True):
    q = torch.from_numpy(np.ascontiguousarray(lin.q)).cuda()
    x = dev_bits(lin.x, lin.x_dtype) if x is None else x
    b = _f16(lin.bias) if bias and lin.bias is not None else None
    y = lb.gemv_int4(x, lb.pack_int4(q), _f16(lin.scales), _f16(lin.zeros), bias=b,
                     out_dtype=TORCH_DT[lin.y_dtype], activation=act, out=out)
    torch.cuda.synchronize()
    Y = to_host64(y)
    hb = lin.bias if bias else None
    A = oracle.linear_int4(lin.x, lin.x_dtype, lin.q, lin.scales, lin.zeros, hb)
    Mg = oracle.magnitude_int4(lin.x, lin.x_dtype, lin.q, lin.scales, lin.zeros, hb)
    ax = np.abs(oracle.decode(lin.x, lin.x_dtype))
    s = np.repeat(np.abs(lin.scales.astype(np.float64)), oracle.GROUP, axis=1)
    extra = 2.0 ** -19 * (16.0 + np.abs(lin.zeros.astype(np.float64)).max(axis=1))[None, :] * (ax @ s.T)
    if act == "gelu":
        A, Mg, extra = oracle.gelu(A), 1.13 * Mg, 1.13 * extra
    bnd = oracle.bound(A, Mg, lin.y_dtype, Y) + extra
    d = np.abs(Y - A)
    assert (d <= bnd).all(), f"{lin.name}: {int((~(d <= bnd)).sum())} outside, worst {float(np.max(d / bnd)):.3g}"
    return y


GEMV = [(1, 16, 128), (1, 1, 128), (1, 33, 256), (2, 17, 384), (3, 200, 640), (5, 1000, 1152), (7, 31, 4096),
        (8, 520, 4224), (9, 64, 8192), (12, 100, 8320), (16, 16, 128), (16, 513, 2560), (15, 16400, 256),
        (16, 9000, 1280), (4, 48, 16512)]


@pytest.mark.parametrize("M,N,K", GEMV)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gemv_int4_shapes(lb, M, N, K, dt):
    banner(f"gemv int4 {dt} {M}x{N}x{K}")
    lin = wl.make_int4_linear(f"gv_{M}x{N}x{K}", M, N, K, dt, seed=M * 11 + N + K, with_bias=(M % 2 == 1))
    _gemv_check(lb, lin, act="gelu" if M % 3 == 0 else None)


def test_gemv_int4_every_row_count_and_output_type(lb):
    for M in range(1, 17):
        lin = wl.make_int4_linear(f"gv_m{M}", M, 70, 384, "bf16" if M % 2 else "f16", seed=300 + M, with_bias=True)
        lin.y_dtype = ("f32", "f16", "bf16")[M % 3]
        banner(f"gemv int4 rows {M} -> {lin.y_dtype}")
        _gemv_check(lb, lin)


def test_gemv_int4_strided_rows_and_output(lb):
    banner("gemv int4 strided x and out")
    lin = wl.make_int4_linear("gv_str", 6, 90, 512, "bf16", seed=77, with_bias=True)
    wide = torch.full((6, 520), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :512] = dev_bits(lin.x, "bf16")
    out = torch.full((6, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    _gemv_check(lb, lin, x=wide[:, :512], out=out[:, :90])
    assert (out[:, 90:] == 7.0).all()


def test_gemv_int4_zero_points_far_from_the_codes(lb):
    banner("gemv int4 far zero points")
    lin = wl.make_int4_linear("gv_z", 4, 100, 640, "f16", seed=78, with_bias=False)
    lin.zeros = (lin.zeros.astype(np.float32) * 100).astype(np.float16)
    lin.zeros[3] = 0
    lin.zeros[4] = -30000
    lin.scales[5] = 0
    _gemv_check(lb, lin)


def test_gemv_int4_agrees_with_gemm_int4_and_repeats_bit_for_bit(lb):
    banner("gemv int4 twice, and on another stream")
    lin = wl.make_int4_linear("gv_rep", 16, 3000, 2560, "bf16", seed=79, with_bias=True)
    y = _gemv_check(lb, lin)
    s = torch.cuda.Stream()
    q = lb.pack_int4(torch.from_numpy(np.ascontiguousarray(lin.q)).cuda())
    args = (dev_bits(lin.x, "bf16"), q, _f16(lin.scales), _f16(lin.zeros))
    torch.cuda.synchronize()
    z = lb.gemv_int4(*args, bias=_f16(lin.bias), stream=s)
    s.synchronize()
    assert torch.equal(y, z)


def test_gemv_int4_keeps_nonfinite_rows_apart(lb):
    banner("gemv int4 with a NaN row and an infinite row")
    lin = wl.make_int4_linear("gv_nan", 5, 64, 256, "f16", seed=80, with_bias=False)
    clean = _gemv_check(lb, lin)
    x = dev_bits(lin.x, "f16")
    x[1, 7], x[3, 200] = float("nan"), float("inf")
    q = lb.pack_int4(torch.from_numpy(np.ascontiguousarray(lin.q)).cuda())
    y = lb.gemv_int4(x, q, _f16(lin.scales), _f16(lin.zeros))
    assert torch.equal(y[[0, 2, 4]], clean[[0, 2, 4]])
    assert not torch.isfinite(y[[1, 3]]).any()


# ------------------------------------------------------------ the paged cache ---

class Paged:
    """Sequences of given lengths over a shuffled page table, on host and device."""

    def __init__(self, lens, H, page, D, seed, spare=3, scale=(0.5, 1.5)):
        g = np.random.default_rng(seed)
        self.H, self.page, self.D, self.lens = H, page, D, np.asarray(lens)
        self.width = max(1, int(-(-self.lens.max() // page))) if len(lens) else 1
        B = len(lens)
        self.pages = B * self.width + spare
        self.table = g.permutation(self.pages)[:B * self.width].reshape(B, self.width).astype(np.int32)
        shape = (self.pages, H, page, D)
        self.k, self.v = (np.clip(np.rint(g.standard_normal(shape) * 36), -127, 127).astype(np.int64) + 128
                          for _ in range(2))
        self.k, self.v = self.k.astype(np.uint8), self.v.astype(np.uint8)
        self.ks, self.vs = (((scale[0] + (scale[1] - scale[0]) * g.random((self.pages, H))) * (3.5 / 127))
                            .astype(np.float32) for _ in range(2))

    def cache(self, lb):
        return lb.KVCache(*(torch.from_numpy(a).cuda() for a in (self.k, self.v, self.ks, self.vs)))


def _values(g, shape, dt):
    bits = oracle.encode(g.standard_normal(shape), dt) if dt != "f32" else None
    if dt == "f32":
        a = g.standard_normal(shape).astype(np.float32)
        return torch.from_numpy(a).cuda(), a.astype(np.float64)
    return dev_bits(bits, dt), oracle.decode(bits, dt)


def _rope(positions, rot, base=10000.0):
    a = np.arange(positions)[:, None] * base ** (-np.arange(rot // 2) / max(1, rot // 2))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


APPEND = [  # starts, new, H, Hq, page, D, rot, interleaved, dtype
    ([0], [1], 1, 1, 16, 64, 64, False, "bf16"),
    ([15, 16, 17], [1, 1, 1], 2, 6, 16, 64, 32, True, "f16"),
    ([0, 5, 100], [37, 0, 3], 2, 2, 32, 128, 128, False, "bf16"),
    ([63, 64, 1], [2, 64, 200], 3, 3, 64, 128, 64, True, "f32"),
    ([7], [300], 2, 10, 128, 256, 256, False, "f16"),
    ([250, 3], [9, 258], 1, 8, 256, 64, 0, False, "bf16"),
    ([2, 0, 0, 40], [6, 7, 33, 24], 8, 32, 64, 128, 96, True, "bf16"),
    ([10, 1000], [5, 1], 4, 4, 16, 256, 32, False, "f16"),
]


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
def test_kv_append(lb, case):
    starts, new, H, Hq, page, D, rot, inter, dt = case
    banner(f"append {case}")
    g = np.random.default_rng(1000 + len(starts) + D + page)
    lens = np.asarray(starts) + np.asarray(new)
    P = Paged(lens, H, page, D, seed=5)
    cache, T = P.cache(lb), int(sum(new))
    # operands are slices of a fused projection: strides apart from the shape
    x, hx = _values(g, (T, Hq + 2 * H, D), dt)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    cu = np.concatenate([[0], np.cumsum(new)])
    cos, sin = _rope(int(lens.max()), rot)
    bad = torch.zeros(2, dtype=torch.int32, device="cuda")
    dev = [torch.from_numpy(a).cuda() for a in (cos, sin)] if rot else [None, None]
    qo = lb.kv_append(k, v, cache, _i32(P.table), _i32(cu), _i32(starts), max(new), q=q, cos=dev[0], sin=dev[1],
                      interleaved=inter, bad_count=bad)
    torch.cuda.synchronize()
    assert bad.tolist() == [0, 0]
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, new)]).astype(int)
    turn = (lambda a: od.rotate(a, pos, cos, sin, inter)) if rot else (lambda a: a)
    want_q = turn(hx[:, :Hq])
    d = np.abs(to_host64(qo) - want_q)
    big = np.abs(hx[:, :Hq]).max()
    assert (d <= _half_ulp(want_q, qo.dtype) * 1.001 + 2.0 ** -22 * big).all()
    got = {n: [t.cpu().numpy() for t in ts] for n, ts in dict(k=(cache.k, cache.k_scale), v=(cache.v, cache.v_scale)).items()}
    start = dict(k=(P.k, P.ks), v=(P.v, P.vs))
    dense = dict(k=turn(hx[:, Hq:Hq + H]), v=hx[:, Hq + H:])
    touched = set()
    for b, (s0, n) in enumerate(zip(starts, new)):
        for slot in range(s0 // page, (s0 + n - 1) // page + 1 if n else s0 // page):
            p, lo, hi = P.table[b, slot], max(s0, slot * page), min(s0 + n, (slot + 1) * page)
            touched.add(int(p))
            for name in "kv":
                for h in range(H):
                    first = lo - slot * page
                    was = od.block_codes(start[name][0][p, h], name, page, D)
                    now = od.block_codes(got[name][0][p, h], name, page, D)
                    rows = dense[name][cu[b] + lo - s0:cu[b] + hi - s0, h]
                    codes, want = od.append_block(was, start[name][1][p, h], first, rows)
                    scale = float(got[name][1][p, h])
                    assert abs(scale - want) <= 2.0 ** -20 * want
                    n_new = hi - lo
                    assert (np.abs(now[first:first + n_new] * scale - rows) <= 0.5001 * scale).all()
                    old, kept = float(start[name][1][p, h]), now[:first]
                    if scale == old:
                        assert np.array_equal(kept, was[:first])
                    else:
                        assert (np.abs(kept * scale - was[:first] * old) <= 0.5001 * scale).all()
                    assert np.array_equal(now[first + n_new:], was[first + n_new:])   # later tokens stay
    rest = [p for p in range(P.pages) if p not in touched]
    for name in "kv":
        assert np.array_equal(got[name][0][rest], start[name][0][rest])
        assert np.array_equal(got[name][1][rest], start[name][1][rest])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("page,D", [(16, 128), (64, 64), (256, 256)])
def test_kv_read_is_exact(lb, dt, page, D):
    banner(f"read {dt} page {page} D {D}")
    lens, starts = [1, 300, 0, 70], [0, 37, 0, 69]
    P = Paged(lens, 2, page, D, seed=9)
    n = np.asarray(lens) - starts
    cu = np.concatenate([[0], np.cumsum(n)])
    P.table[1, 0] = P.pages + 7                                # no page: zeros there
    k, v = lb.kv_read(P.cache(lb), _i32(P.table), _i32(cu), _i32(starts), int(cu[-1]), int(n.max()), TORCH_DT[dt])
    for name, t, codes, sc in (("k", k, P.k, P.ks), ("v", v, P.v, P.vs)):
        for b in range(4):
            want = np.nan_to_num(od.cache_rows(codes, sc, P.table[b], name, starts[b], lens[b]))
            have = to_host64(t[int(cu[b]):int(cu[b + 1])])
            want = want.astype(np.float32).astype(np.float64)   # one FP32 product, then the output's rounding
            want = want if dt == "f32" else oracle.decode(oracle.encode(want, dt), dt)
            assert np.array_equal(have, want)


def test_append_one_by_one_equals_the_definition_and_read_gives_it_back(lb):
    """A block filled token by token, with growing values: every growth may cost
    older tokens half a step of the scale then; the sum over the growths bounds it."""
    banner("append 64 tokens one by one")
    H, D, page = 2, 128, 64
    g = np.random.default_rng(3)
    x = (g.standard_normal((64, H, D)) * (1 + np.arange(64))[:, None, None]).astype(np.float32)
    cache = lb.new_kv_cache(2, H, page, D)
    table, cu = _i32([[1]]), _i32([0, 1])
    t = torch.from_numpy(x).cuda()
    slack = np.zeros((64, H))
    scale = np.zeros(H)
    for i in range(64):
        lb.kv_append(t[i:i + 1], t[i:i + 1], cache, table, cu, _i32([i]), 1)
        now = cache.k_scale[1].cpu().numpy().astype(np.float64)
        grown = now > scale
        slack[:i, grown] += 0.5001 * now[grown]
        slack[i] = 0.5001 * now
        scale = now
    k, v = lb.kv_read(cache, table, _i32([0, 64]), _i32([0]), 64, 64, torch.float32)
    for y in (k, v):
        assert (np.abs(to_host64(y) - x) <= slack[:, :, None] + 1e-6).all()


def test_append_nonfinite_zero_and_tiny_values(lb):
    banner("append NaN, infinities, zeros, tiny values")
    H, D, page = 1, 64, 16
    x = torch.zeros((32, H, D), dtype=torch.float32, device="cuda")
    x[3, 0, 5], x[4, 0, 6], x[5, 0, 7], x[6, 0, 8] = float("nan"), float("inf"), -float("inf"), 2.0
    x[16:] = 1e-36                                            # below 127 * 2^-100: becomes zero
    cache = lb.new_kv_cache(3, H, page, D)
    bad = torch.zeros(2, dtype=torch.int32, device="cuda")
    lb.kv_append(x, x, cache, _i32([[2, 0]]), _i32([0, 32]), _i32([0]), 32, bad_count=bad)
    assert bad.tolist() == [6, 0]                              # three keys and three values
    k, v = lb.kv_read(cache, _i32([[2, 0]]), _i32([0, 32]), _i32([0]), 32, 32, torch.float32)
    for y in (k, v):
        want = torch.zeros_like(x)
        want[6, 0, 8] = 2.0
        assert (y - want).abs().max() <= 4e-7             # three FP32 roundings of 2
    assert cache.k_scale[0, 0] == 0 and cache.v_scale[0, 0] == 0


def test_append_leaves_out_tokens_without_page_or_position(lb):
    banner("append without page / position")
    H, D, page = 2, 64, 16
    x = torch.randn((40, H, D), device="cuda").half()
    cache = lb.new_kv_cache(3, H, page, D)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    bad = torch.zeros(2, dtype=torch.int32, device="cuda")
    # 40 tokens: page 0 exists, page 1 is -1, the third slot is past the table
    lb.kv_append(x, x, cache, _i32([[1, -1]]), _i32([0, 40]), _i32([0]), 40, bad_count=bad)
    assert bad.tolist() == [0, 24]
    for t, o in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
        assert torch.equal(t[[0, 2]], o[[0, 2]])
    cos, sin = (torch.from_numpy(a).cuda() for a in _rope(10, 32))
    bad.zero_()
    lb.kv_append(x[:14], x[:14], cache, _i32([[0]]), _i32([0, 14]), _i32([0]), 14, cos=cos, sin=sin, bad_count=bad)
    assert bad.tolist() == [0, 4]
    assert (cache.k[0].cpu().view(H, -1)[:, [od.k_place(12, 3, D)]] == 0).all()


def test_append_in_place_queries_and_on_another_stream(lb):
    banner("append: q in place, another stream")
    P = Paged([50, 20], 2, 32, 128, seed=6)
    g = np.random.default_rng(8)
    x, _ = _values(g, (9, 8, 128), "bf16")
    cos, sin = (torch.from_numpy(a).cuda() for a in _rope(64, 128))
    args = lambda y, c: (y[:, 4:6], y[:, 6:], c, _i32(P.table), _i32([0, 5, 9]), _i32([45, 16]), 5)  # noqa: E731
    a, b, s = P.cache(lb), P.cache(lb), torch.cuda.Stream()
    want = lb.kv_append(*args(x, a), q=x[:, :4], cos=cos, sin=sin)
    y = x.clone()
    second = args(y, b)
    torch.cuda.synchronize()
    out = lb.kv_append(*second, q=y[:, :4], cos=cos, sin=sin, q_out=y[:, :4], stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)


# ------------------------------------------------------------------ attention ---

def _attend(lb, lens, new, H, Hq, page, D, dt, seed=0, causal=True, window=0, scale=None, qmul=1.0, kv=None, hole=None,
            width=None, max_len=None, strided=False):
    P = kv or Paged(lens, H, page, D, seed=seed)
    if hole is not None:
        P.table[hole[0], hole[1]] = hole[2]
    g = np.random.default_rng(seed + 1)
    T = int(sum(new))
    q, hq = _values(g, (T, Hq + 1, D) if strided else (T, Hq, D), dt)
    q, hq = q[:, :Hq] * qmul, hq[:, :Hq] * qmul
    hq = to_host64(q.contiguous())
    if strided:
        q = torch.cat([q, q], 2)[:, :, :D]
    cu = np.concatenate([[0], np.cumsum(new)])
    table = P.table if width is None else P.table[:, :width]
    out, lse = lb.attention(q, P.cache(lb), _i32(table), _i32(cu), _i32(lens), max(1, max(new)),
                            int(max(lens)) if max_len is None else max_len, scale=scale, causal=causal, window=window,
                            return_lse=True)
    torch.cuda.synchronize()
    O, E = to_host64(out), to_host64(lse)
    for b, (L, n) in enumerate(zip(lens, new)):
        L = min(L, table.shape[1] * page)
        k = od.cache_rows(P.k, P.ks, table[b], "k", 0, L)
        v = od.cache_rows(P.v, P.vs, table[b], "v", 0, L)
        rows = slice(int(cu[b]), int(cu[b + 1]))
        at = np.where((table[b] >= 0) & (table[b] < P.pages), table[b], 0)[np.arange(L) // page]
        want, we, mag, peak = od.attention(hq[rows], k, np.nan_to_num(v), P.vs[at].astype(np.float64), L - n,
                                           D ** -0.5 if scale is None else scale, causal, window)
        d = np.abs(O[rows] - want)
        bound = 2.0 ** -10 * mag + 2.0 ** -25 * peak + _half_ulp(np.maximum(np.abs(want), np.abs(O[rows])), out.dtype)
        assert (d <= bound).all(), f"sequence {b}: worst {np.max(d / np.maximum(bound, 1e-30)):.3g}"
        empty = np.isneginf(we)
        assert np.array_equal(empty, np.isneginf(E[rows]))
        assert (O[rows][empty] == 0).all()
        assert (np.abs(E[rows][~empty] - we[~empty]) <= 2.0 ** -14 + 2.0 ** -22 * np.abs(we[~empty])).all()
    return out


ATTEND = [  # lens, new, H, Hq, page, D, dtype, causal, window
    ([1], [1], 1, 1, 16, 64, "bf16", True, 0),
    ([1, 2, 15, 16, 17, 31, 33], [1] * 7, 2, 2, 16, 128, "f16", True, 0),
    ([0, 5, 0], [1, 1, 0], 1, 3, 32, 64, "bf16", True, 0),            # a sequence with nothing cached
    ([300, 64, 65], [1, 1, 1], 2, 10, 64, 128, "bf16", True, 0),
    ([1500, 700], [1, 1], 2, 16, 16, 128, "f16", True, 0),            # parts that are joined
    ([1300, 257], [3, 5], 2, 8, 32, 256, "bf16", True, 0),
    ([900], [1], 1, 5, 128, 256, "f16", True, 100),
    ([2, 3], [5, 6], 1, 2, 16, 64, "f16", True, 0),                   # more queries than tokens: some see nothing
    ([700, 40], [2, 4], 2, 6, 64, 64, "bf16", False, 0),
    ([1000, 600], [16, 3], 1, 2, 256, 128, "bf16", True, 17),
    ([130], [130], 2, 4, 16, 128, "bf16", True, 0),                   # prompts
    ([64, 1, 65, 129], [64, 1, 65, 129], 1, 3, 64, 64, "f16", True, 0),
    ([500, 333], [77, 200], 2, 10, 32, 128, "f16", True, 0),          # chunks over a cached prefix
    ([400], [150], 1, 2, 128, 256, "bf16", True, 64),
    ([300, 90], [90, 90], 2, 2, 16, 64, "bf16", False, 0),
    ([60], [100], 1, 4, 16, 128, "f16", True, 0),                     # first queries at negative positions
    ([3000], [40], 1, 1, 16, 128, "bf16", True, 0),                   # few row tiles: the context is split
    ([2500], [40], 1, 2, 64, 64, "f16", True, 1500),
    ([200], [64], 1, 1, 16, 64, "f16", True, 10),                     # rows whose first tile holds one to four tokens
    ([200], [64], 1, 1, 32, 128, "bf16", True, 3),
    ([200], [16], 1, 1, 16, 128, "bf16", True, 3),
    ([4500], [33], 1, 1, 16, 256, "f16", False, 0),                   # more pages than one segment holds
]


@pytest.mark.parametrize("case", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
def test_attention(lb, case):
    lens, new, H, Hq, page, D, dt, causal, window = case
    banner(f"attention {case}")
    _attend(lb, lens, new, H, Hq, page, D, dt, seed=len(lens) + D, causal=causal, window=window,
            strided=(D == 128))


@pytest.mark.parametrize("new", [1, 40])
def test_attention_missing_pages_and_clipped_lengths(lb, new):
    banner(f"attention with holes, new {new}")
    _attend(lb, [200, 100], [new, new], 2, 4, 16, 128, "bf16", seed=20, hole=(0, 3, -1))
    _attend(lb, [200, 100], [new, new], 2, 4, 16, 128, "bf16", seed=21, hole=(1, 0, 10 ** 6))
    # a table shorter than the lengths: they count as what it holds
    _attend(lb, [200, 100], [new, new], 2, 4, 16, 128, "bf16", seed=23, width=9)
    # every page missing: zeros
    P = Paged([40], 1, 16, 64, seed=22)
    P.table[:] = -1
    _attend(lb, [40], [new], 1, 2, 16, 64, "f16", kv=P)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_block_scales_far_apart(lb, new):
    """Value scales over ten orders of magnitude, zero scales (all-zero blocks)
    and peaked scores; unused tokens of pages hold anything."""
    banner(f"attention scales apart, new {new}")
    P = Paged([260], 1, 16, 128, seed=30)
    g = np.random.default_rng(31)
    P.vs[:] = (10.0 ** g.uniform(-9, 1, P.vs.shape)).astype(np.float32)
    P.vs[P.table[0, 4]] = 0
    P.v[P.table[0, 4]] = 128
    P.ks[P.table[0, 5]] = 0
    _attend(lb, [260], [new], 1, 4, 16, 128, "f16", kv=P, seed=32)
    P.vs[:] = 0
    P.v[:] = 128
    out = _attend(lb, [260], [new], 1, 4, 16, 128, "f16", kv=P, seed=33)
    assert (out == 0).all()


@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("dt,qmul", [("bf16", 2.0 ** 60), ("bf16", 2.0 ** -60), ("f16", 200.0), ("f16", 2.0 ** -20)])
def test_attention_query_ranges(lb, new, dt, qmul):
    """Queries far from 1 with the softmax scale that undoes it."""
    banner(f"attention {dt} queries x {qmul}, new {new}")
    _attend(lb, [150], [new], 2, 4, 32, 64, dt, seed=40, qmul=qmul, scale=float(0.125 / qmul))


@pytest.mark.parametrize("new", [1, 50])
def test_attention_nonfinite_queries_stay_in_their_rows(lb, new):
    banner(f"attention NaN rows, new {new}")
    P = Paged([200], 1, 16, 128, seed=50)
    q = torch.randn((new, 4, 128), device="cuda").half()
    args = (P.cache(lb), _i32(P.table), _i32([0, new]), _i32([200]), new, 200)
    clean = lb.attention(q, *args)
    q[0, 1, 3] = float("nan")
    y = lb.attention(q, *args)
    assert torch.isnan(y[0, 1]).all()
    y[0, 1] = clean[0, 1]
    assert torch.equal(y, clean)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_masked_tokens_hold_anything(lb, new):
    """Codes behind the length, scales (NaN) of pages that are not used, and
    entries of the table behind the last page do not matter."""
    banner(f"attention garbage, new {new}")
    P = Paged([70, 33], 1, 16, 64, seed=60)
    q = torch.randn((2 * new, 2, 64), device="cuda").half()
    call = lambda P: lb.attention(q, P.cache(lb), _i32(P.table), _i32([0, new, 2 * new]), _i32([70, 33]), new, 70)  # noqa: E731
    clean = call(P)
    used = set(P.table[0, :5]) | set(P.table[1, :3])
    for p in range(P.pages):
        if p not in used:
            P.ks[p], P.vs[p], P.k[p], P.v[p] = np.nan, np.inf, 255, 0
    P.table[1, 3:] = -5
    tail = [t for t in range(33 % 16, 16)]
    d = np.arange(64)
    for t in tail:
        P.k[P.table[1, 2], 0].reshape(-1)[od.k_place(t, d, 64)] = 255
        P.v[P.table[1, 2], 0].reshape(-1)[od.v_place(t, d, 64)] = 0
    assert torch.equal(call(P), clean)


def test_attention_cache_beyond_4_gib(lb):
    """Blocks whose byte offsets pass 2^32 (and 2^31) are reached by every operator."""
    banner("cache of 4.6 GB")
    H, page, D, pages = 2, 256, 256, 36000
    cache = lb.new_kv_cache(pages, H, page, D)
    small = lb.new_kv_cache(4, H, page, D)
    x = torch.randn((300, H, D), device="cuda").bfloat16()
    q = torch.randn((300, 4, D), device="cuda").bfloat16()
    got = []
    for c, table in ((cache, [[35999, 17000]]), (small, [[1, 2]])):
        args = (_i32(table), _i32([0, 300]))
        lb.kv_append(x, x, c, *args, _i32([0]), 300)
        got.append([*lb.kv_read(c, *args, _i32([0]), 300, 300), lb.attention(q, c, *args, _i32([300]), 300, 300),
                    lb.attention(q[:1], c, _i32(table), _i32([0, 1]), _i32([300]), 1, 300)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_decoding_in_a_graph(lb):
    """Append, attention (context split, so with workspace and join) and a 4-bit
    product under capture; every replay against the eager result, with the cache put
    back and other work between them."""
    banner("graph of append + attention + gemv")
    P = Paged([2000, 900], 2, 16, 128, seed=70)
    g = np.random.default_rng(71)
    x, _ = _values(g, (2, 12, 128), "bf16")
    lin = wl.make_int4_linear("gv_g", 2, 300, 1024, "bf16", seed=72, with_bias=False)
    w = lb.pack_int4(torch.from_numpy(np.ascontiguousarray(lin.q)).cuda())
    sc, ze = _f16(lin.scales), _f16(lin.zeros)
    cos, sin = (torch.from_numpy(a).cuda() for a in _rope(2000, 128))
    table, cu, starts, lens = _i32(P.table), _i32([0, 1, 2]), _i32([1999, 899]), _i32([2000, 900])
    cache, clean = P.cache(lb), P.cache(lb)

    def put_back():
        for a, b in ((cache.k, clean.k), (cache.v, clean.v), (cache.k_scale, clean.k_scale), (cache.v_scale, clean.v_scale)):
            a.copy_(b)

    def step():
        q = lb.kv_append(x[:, 8:10], x[:, 10:], cache, table, cu, starts, 1, q=x[:, :8], cos=cos, sin=sin)
        y = lb.attention(q, cache, table, cu, lens, 1, 2000)
        return q, y, lb.gemv_int4(y.view(2, 1024), w, sc, ze)

    eager = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        put_back()
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for _ in range(4):
        put_back()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, eager):
            assert torch.equal(a, b)
        put_back()
        for a, b in zip(step(), eager):
            assert torch.equal(a, b)


def test_example_decodes_like_the_definition(lb, capsys, monkeypatch):
    """The example program on a small model: prompts of different lengths, then
    tokens one by one; its last step against float64 (2 % a layer: four bf16
    roundings of 2^-9 and an 8-bit cache of 1/127 steps a layer, relative to the
    logits' norm)."""
    banner("example: small decoder")
    import importlib.util
    import os
    import sys
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "text_decode.py")
    spec = importlib.util.spec_from_file_location("text_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(sys, "argv", ["text_decode", "--layers", "2", "--hidden", "256", "--q-heads", "6", "--kv-heads", "2",
                                      "--head-dim", "64", "--mlp", "384", "--vocab", "500", "--page", "16", "--batch", "3",
                                      "--prompt", "37", "--tokens", "9", "--check"])
    m.main()
    assert "relative difference" in capsys.readouterr().out


def test_attention_long_prompt_in_256_row_tiles(lb):
    """A prompt chunk long enough for 256 rows a workgroup, over more pages than
    one segment holds, against float64 on sampled queries (keys and values read
    back from the cache, exact in FP32)."""
    banner("attention: 2100 queries of 64 heads over 9000 tokens")
    H, Hq, D, page, L, n = 8, 64, 128, 16, 9000, 2100
    P = Paged([L], H, page, D, seed=90)
    cache, table = P.cache(lb), _i32(P.table)
    q, _ = _values(np.random.default_rng(91), (n, Hq, D), "bf16")
    out = lb.attention(q, cache, table, _i32([0, n]), _i32([L]), n, L)
    k, v = lb.kv_read(cache, table, _i32([0, L]), _i32([0]), L, L, torch.float32)
    k, v = k.double(), v.double()
    vs = torch.from_numpy(P.vs[P.table[0][np.arange(L) // page]]).cuda().double()
    rows = [0, 1, 31, 32, 63, 64, 1000, 1027, 2047, 2048, 2098, 2099]
    for i in rows:
        for h in (0, 7, 8, 29, 63):
            seen, g = L - n + i + 1, h // (Hq // H)
            s = (k[:seen, g] @ q[i, h].double()) * D ** -0.5
            e = torch.exp(s - s.max())
            want, mag = (e @ v[:seen, g]) / e.sum(), (e @ v[:seen, g].abs()) / e.sum()
            peak = 127 * seen * (e * vs[:seen, g]).max() / e.sum()
            d = (out[i, h].double() - want).abs()
            half = torch.from_numpy(np.asarray(_half_ulp(np.maximum(want.abs().cpu().numpy(), np.abs(to_host64(out[i, h]))),
                                                         out.dtype))).cuda()
            assert (d <= 2.0 ** -10 * mag + 2.0 ** -25 * peak + half).all(), (i, h)
