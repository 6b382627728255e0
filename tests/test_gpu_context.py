"""GPU parity of the operators of long contexts against float64 definitions
(oracle/paged.py): attention with a window and first tokens that stay visible,
norms of heads with rotation (into the cache and dense), rotary tables, and
tables of pages with the copies they ask for.

Tolerances, from the contracts of include/lowbit.h:
* attention: as in test_gpu_decode.py, 2^-10 sum p |v| / sum p + 2^-25 tokens 127
  max(p v_scale) / sum p + half an output ulp, over the tokens that are seen.
* norm and rotation: a normalised value takes three FP32 roundings (the root's,
  and two products: 3 * 2^-24), the rotation two more on two terms of up to the
  row's largest normalised value a each: sqrt 2 * 5 * 2^-24 a < 2^-21 a (times the
  tables' magnitude); plus half an output ulp.
* append: scales within 2^-20 relatively (10 * 2^-24 of the largest rotated value,
  which is at least a / sqrt 2, and one division), stored values within 0.5001 scale.
* tables: m (2^-21 + 2^-50 position).
* pages: equal."""
import numpy as np
import pytest
import torch

import oracle
from oracle import paged as od
from gpu_util import TORCH_DT, banner, to_host64
from test_gpu_decode import Paged, _half_ulp, _i32, _rope, _values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import bit_weight_gemm_int2_amd as b
    b.lib()
    return b


# --------------------------------------------------- attention with a window ---

def _check_attention(P, table, hq, O, E, lens, new, cu, D, dtype, causal, window, sinks):
    for b, (L, n) in enumerate(zip(lens, new)):
        L = min(L, table.shape[1] * P.page)
        k = od.cache_rows(P.k, P.ks, table[b], "k", 0, L)
        v = od.cache_rows(P.v, P.vs, table[b], "v", 0, L)
        rows = slice(int(cu[b]), int(cu[b + 1]))
        at = np.where((table[b] >= 0) & (table[b] < P.pages), table[b], 0)[np.arange(L) // P.page]
        want, we, mag, peak = od.attention(hq[rows], k, np.nan_to_num(v), P.vs[at].astype(np.float64), L - n, D ** -0.5, causal,
                                           window, sinks)
        d = np.abs(O[rows] - want)
        bound = 2.0 ** -10 * mag + 2.0 ** -25 * peak + _half_ulp(np.maximum(np.abs(want), np.abs(O[rows])), dtype)
        assert (d <= bound).all(), f"sequence {b}: worst {np.max(d / np.maximum(bound, 1e-30)):.3g}"
        empty = np.isneginf(we)
        assert np.array_equal(empty, np.isneginf(E[rows])) and (O[rows][empty] == 0).all()
        assert (np.abs(E[rows][~empty] - we[~empty]) <= 2.0 ** -14 + 2.0 ** -22 * np.abs(we[~empty])).all()


def _attend(lb, lens, new, H, Hq, page, D, dt, window, sinks, causal=True, seed=0, change=None):
    P = Paged(lens, H, page, D, seed=seed)
    if change:
        change(P)
    T = int(sum(new))
    q, hq = _values(np.random.default_rng(seed + 1), (T, Hq, D), dt)
    cu = np.concatenate([[0], np.cumsum(new)])
    out, lse = lb.attention(q, P.cache(lb), _i32(P.table), _i32(cu), _i32(lens), max(1, max(new)), int(max(lens)), causal=causal,
                            window=window, sinks=sinks, return_lse=True)
    torch.cuda.synchronize()
    _check_attention(P, P.table, hq, to_host64(out), to_host64(lse), lens, new, cu, D, out.dtype, causal, window, sinks)
    return out


ATTEND = [  # lens, new, H, Hq, page, D, dtype, window, sinks
    ([300], [1], 1, 1, 16, 64, "bf16", 40, 4),
    ([300, 70, 5, 44, 45], [1] * 5, 2, 6, 16, 128, "f16", 40, 4),       # with and without a gap
    ([500, 0, 130], [1, 0, 1], 2, 16, 64, 128, "bf16", 100, 17),        # head and window in one page
    ([900], [1], 1, 4, 128, 256, "f16", 1, 1),                          # only itself and the first
    ([900], [1], 2, 2, 256, 64, "bf16", 33, 300),                       # more first tokens than window
    ([200], [1], 1, 2, 32, 128, "f16", 50, 10 ** 9),                    # all of them
    ([6000, 2500], [1, 1], 2, 8, 16, 128, "bf16", 3000, 100),           # in parts, one of which holds the gap
    ([3000], [1], 1, 5, 32, 64, "f16", 500, 1400),                      # parts before and behind the gap
    ([700, 400], [5, 3], 2, 6, 64, 128, "bf16", 90, 20),                # queries with windows of their own
    ([600], [16], 1, 5, 16, 128, "f16", 17, 16),                        # 80 rows in tiles of 16
    ([20, 3], [20, 7], 1, 2, 16, 64, "f16", 5, 2),                      # more queries than tokens
    ([130], [130], 2, 4, 16, 128, "bf16", 30, 3),                       # prompts
    ([700, 333], [300, 200], 2, 10, 32, 128, "f16", 64, 40),
    ([900], [200], 1, 2, 256, 256, "bf16", 100, 70),
    ([500, 64], [500, 64], 1, 3, 64, 64, "f16", 1, 1),
    ([2500], [100], 1, 2, 16, 64, "bf16", 600, 1000),
    ([7000], [90], 1, 1, 16, 128, "f16", 5000, 333),                    # more pages than one segment, in parts
    ([6200], [130], 8, 64, 16, 64, "bf16", 4500, 100),                  # two segments, the first with the gap
]


@pytest.mark.parametrize("case", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
def test_attention_sinks(lb, case):
    lens, new, H, Hq, page, D, dt, window, sinks = case
    banner(f"attention with first tokens {case}")
    _attend(lb, lens, new, H, Hq, page, D, dt, window, sinks, seed=len(lens) + D)


@pytest.mark.parametrize("new", [2, 60])
def test_attention_sinks_not_causal(lb, new):
    banner(f"attention with first tokens, not causal, new {new}")
    _attend(lb, [400, 90], [new, new], 2, 4, 32, 128, "bf16", 30, 9, causal=False, seed=3)


@pytest.mark.parametrize("new", [1, 60])
def test_attention_sinks_leaves_the_gap_alone(lb, new):
    """Pages between the first tokens and the window have gone back to the pool
    (no entry, NaN scales), page 1 of the head has none, and a head that is all
    missing leaves the window alone."""
    banner(f"attention with freed pages, new {new}")
    lens, window, sinks, page = [1000, 300], 128, 40, 16

    def freed(P):
        for b, L in enumerate(lens):
            first = (L - new - window + 1) // page
            for s in range(3, first):
                p = P.table[b, s]
                P.ks[p], P.vs[p], P.k[p], P.v[p] = np.nan, np.inf, 255, 0
                P.table[b, s] = -1 if s % 2 else P.pages + 3
        P.table[0, 1] = -1

    a = _attend(lb, lens, [new, new], 2, 4, page, 64, "f16", window, sinks, seed=5, change=freed)

    def no_head(P):
        freed(P)
        P.table[:, :3] = -1

    b = _attend(lb, lens, [new, new], 2, 4, page, 64, "f16", window, sinks, seed=5, change=no_head)
    assert not torch.equal(a, b)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_sinks_beside_the_plain_calls(lb, new):
    """No first tokens, or no window: the same bits as without them; a first
    token alone beside a window that holds the rest: the tokens of no window, in
    parts of its own (each result is within its bound of the definition)."""
    banner(f"attention: sinks 0, window 0, new {new}")
    P = Paged([700, 30], 2, 32, 128, seed=8)
    q, hq = _values(np.random.default_rng(9), (new + 1, 8, 128), "bf16")
    args = (q, P.cache(lb), _i32(P.table), _i32([0, new, new + 1]), _i32([700, 30]), new, 700)
    assert torch.equal(lb.attention(*args, window=100, sinks=0), lb.attention(*args, window=100))
    assert torch.equal(lb.attention(*args, window=0, sinks=9), lb.attention(*args))
    for kw in (dict(window=699, sinks=1), dict()):
        out, lse = lb.attention(*args, **kw, return_lse=True)
        _check_attention(P, P.table, hq, to_host64(out), to_host64(lse), [700, 30], [new, 1], [0, new, new + 1], 128, out.dtype,
                         True, 0, 0)


def test_attention_sinks_long_prompt_in_256_row_tiles(lb):
    """Tiles of 256 rows over more pages than one segment holds, against float64 on sampled queries."""
    banner("attention: 2100 queries of 64 heads, window of 8300 and 50 first tokens of 12000")
    H, Hq, D, page, L, n, window, sinks = 8, 64, 128, 16, 12000, 2100, 8300, 50
    P = Paged([L], H, page, D, seed=90)
    cache, table = P.cache(lb), _i32(P.table)
    q, _ = _values(np.random.default_rng(91), (n, Hq, D), "bf16")
    out = lb.attention(q, cache, table, _i32([0, n]), _i32([L]), n, L, window=window, sinks=sinks)
    k, v = lb.kv_read(cache, table, _i32([0, L]), _i32([0]), L, L, torch.float32)
    k, v = k.double(), v.double()
    vs = torch.from_numpy(P.vs[P.table[0][np.arange(L) // page]]).cuda().double()
    for i in [0, 1, 31, 32, 63, 64, 1000, 1027, 2047, 2048, 2098, 2099]:
        pos = L - n + i
        seen = torch.cat([torch.arange(sinks), torch.arange(max(sinks, pos - window + 1), pos + 1)]).cuda()
        for h in (0, 7, 8, 29, 63):
            g = h // (Hq // H)
            s = (k[seen, g] @ q[i, h].double()) * D ** -0.5
            e = torch.exp(s - s.max())
            want, mag = (e @ v[seen, g]) / e.sum(), (e @ v[seen, g].abs()) / e.sum()
            peak = 127 * len(seen) * (e * vs[seen, g]).max() / e.sum()
            half = torch.from_numpy(np.asarray(_half_ulp(np.maximum(want.abs().cpu().numpy(), np.abs(to_host64(out[i, h]))),
                                                         out.dtype))).cuda()
            assert ((out[i, h].double() - want).abs() <= 2.0 ** -10 * mag + 2.0 ** -25 * peak + half).all(), (i, h)


JOIN = [  # lens, new, H, Hq, page, D, dtype, window, sinks: few parts of many rows
    ([3000 - 17 * i for i in range(60)], [1] * 60, 1, 16, 16, 128, "bf16", 2500, 20),
    ([900, 4000], [300, 250], 1, 2, 64, 64, "f16", 3000, 50),
    ([4000, 20], [300, 20], 1, 2, 64, 256, "bf16", 3000, 50),
    ([3000], [700], 1, 4, 32, 128, "f16", 2000, 50),
]


@pytest.mark.parametrize("case", JOIN, ids=[str(i) for i in range(len(JOIN))])
def test_attention_sinks_joined_by_rows(lb, case):
    lens, new, H, Hq, page, D, dt, window, sinks = case
    banner(f"attention, join by rows: {len(lens)} sequences, heads of {D}")
    B, T = len(lens), sum(new)
    need = lb.lib().lowbit_attention_sinks_workspace_bytes(B, T, max(new), max(lens), Hq, H, D, 1, window, sinks)
    assert 2 <= need // (T * Hq * (D + 2) * 4) <= 8           # parts
    _attend(lb, lens, new, H, Hq, page, D, dt, window, sinks, seed=77)


def test_attention_sinks_leaves_rows_of_no_sequence(lb):
    banner("attention with first tokens, padded batch")
    P = Paged([4000, 500], 1, 16, 64, seed=12)
    q, _ = _values(np.random.default_rng(13), (8, 2, 64), "f16")
    out = torch.full_like(q, 7.0)
    lb.attention(q, P.cache(lb), _i32(P.table), _i32([2, 3, 5]), _i32([4000, 500]), 2, 4000, window=2500, sinks=60, out=out)
    assert (out[[0, 1, 5, 6, 7]] == 7.0).all() and not (out[2:5] == 7.0).any()


# ------------------------------------------------------- norms and rotation ---

def _weights(g, D, dt):
    w, hw = _values(g, (D,), dt)
    return (1 + w.float() / 4).to(w.dtype), to_host64((1 + w.float() / 4).to(w.dtype))


TURN = [  # T, Hq, Hk, D, rot, interleaved, dtype, weights' dtype, rows
    (1, 1, 0, 64, 64, False, "bf16", "bf16", 0),
    (5, 3, 1, 64, 32, True, "f16", "f32", 0),
    (33, 32, 8, 128, 128, False, "bf16", "f32", 500),
    (17, 5, 5, 128, 96, False, "f32", "f16", 40),
    (40, 24, 24, 128, 128, True, "bf16", "bf16", 0),
    (7, 2, 1, 256, 256, False, "f16", "f16", 9),
    (300, 1, 7, 256, 32, True, "f32", "bf16", 1000),
    (64, 6, 2, 128, 0, False, "bf16", "bf16", 0),                 # a norm alone
]


@pytest.mark.parametrize("case", TURN, ids=[str(i) for i in range(len(TURN))])
def test_norm_rotate(lb, case):
    T, Hq, Hk, D, rot, inter, dt, wdt, rows = case
    banner(f"norm and rotation {case}")
    g = np.random.default_rng(T + D)
    x, hx = _values(g, (T, Hq + 2 * Hk + 1, D), dt)              # slices of a fused projection, with more behind them
    x, hx = x * 3, hx * 3
    hx = to_host64(x)
    (wq, hwq), (wk, hwk) = _weights(g, D, wdt), _weights(g, D, wdt)
    cos, sin = _rope(max(rows, T), rot) if rot else (None, None)
    dev = [None, None] if not rot else [torch.from_numpy(a).cuda() for a in (cos, sin)]
    pos = g.integers(0, rows, T) if rows else np.arange(T)
    for norm_q, norm_k in ((True, True), (False, True), (True, False)):
        if not Hk and norm_k:
            norm_k = False
        if not rot and not (norm_q and norm_k):
            continue
        got = lb.norm_rotate(x[:, :Hq], x[:, Hq:Hq + Hk] if Hk else None, wq if norm_q else None, wk if norm_k else None,
                             cos=dev[0], sin=dev[1], positions=_i32(pos) if rows else None, eps=1e-5, interleaved=inter)
        for y, rows_in, w, on in zip((got,) if not Hk else got, (hx[:, :Hq], hx[:, Hq:Hq + Hk]), (hwq, hwk), (norm_q, norm_k)):
            n = od.norm(rows_in, w, np.float64(np.float32(1e-5))) if on else rows_in
            want = od.rotate(n, pos, cos, sin, inter) if rot else n
            big = np.abs(n).max(-1, keepdims=True)
            assert (np.abs(to_host64(y) - want) <= 2.0 ** -21 * big + 1.001 * _half_ulp(want, y.dtype)).all()


def test_norm_rotate_head_major_and_in_place(lb):
    banner("norm and rotation: head-major operands, in place, another stream")
    g = np.random.default_rng(4)
    x, _ = _values(g, (12, 50, 128), "bf16")                     # [heads, tokens, D]
    (wq, _), (wk, _) = _weights(g, 128, "bf16"), _weights(g, 128, "bf16")
    cos, sin = (torch.from_numpy(a).cuda() for a in _rope(50, 128))
    q, k = x[:8].transpose(0, 1), x[8:].transpose(0, 1)
    want = lb.norm_rotate(q, k, wq, wk, cos, sin)
    plain = lb.norm_rotate(q.contiguous(), k.contiguous(), wq, wk, cos, sin)
    assert all(torch.equal(a, b) for a, b in zip(want, plain))
    y, s = x.clone(), torch.cuda.Stream()
    q, k = y[:8].transpose(0, 1), y[8:].transpose(0, 1)
    torch.cuda.synchronize()
    lb.norm_rotate(q, k, wq, wk, cos, sin, q_out=q, k_out=k, stream=s)
    s.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_norm_rotate_positions_outside_the_tables(lb):
    banner("norm and rotation: positions outside the tables")
    x = torch.randn((6, 3, 64), device="cuda").half()
    cos, sin = (torch.from_numpy(a).cuda() for a in _rope(10, 64))
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.ones(64, device="cuda")
    q, k = lb.norm_rotate(x, x[:, :1], w, w, cos, sin, positions=_i32([0, -1, 9, 10, 2 ** 31 - 1, 3]), bad_count=bad)
    assert bad.item() == 3 and (q[[1, 3, 4]] == 0).all() and (k[[1, 3, 4]] == 0).all()
    assert torch.equal(q[[0, 2, 5]], lb.norm_rotate(x[[0, 2, 5]], None, w, None, cos, sin, positions=_i32([0, 9, 3])))
    # more tokens than rows: those behind have no position
    bad.zero_()
    z = lb.norm_rotate(x, cos=cos[:4].contiguous(), sin=sin[:4].contiguous(), bad_count=bad)
    assert bad.item() == 2 and (z[4:] == 0).all() and torch.equal(z[:1], x[:1])


def test_norm_of_huge_tiny_zero_and_nonfinite_rows(lb):
    """Squares that FP32 cannot hold; rows of zeros; NaN and infinity stay in their rows."""
    banner("norm of rows out of FP32's squares")
    x = torch.randn((8, 1, 128), device="cuda")
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -100
    x[3] = 0
    x[4, 0, 7], x[5, 0, 9] = float("nan"), float("inf")
    x[6] *= 3.0e38 / x[6].abs().max()
    w = torch.full((128,), 2.0, device="cuda")
    y = to_host64(lb.norm_rotate(x, q_norm=w, eps=0.0))[:, 0]
    h = x.double().cpu().numpy()[:, 0]
    rows = [0, 1, 2, 3, 6, 7]
    want = od.norm(h[rows], 2.0, 0.0)
    # a root below FP32's normal numbers (row 6: 1 / 1e38) is within 2^-22 of itself
    assert (np.abs(y[rows] - want) <= 2.0 ** -21 * np.abs(want).max(-1, keepdims=True)).all()
    assert np.isnan(y[4]).all() and np.isnan(y[5, 9]) and (np.delete(y[5], 9) == 0).all()
    # with eps the tiny row is its ratio to the root of eps
    y = to_host64(lb.norm_rotate(x, q_norm=w, eps=1e-6))[2, 0]
    assert np.allclose(y, h[2] * 2 / np.sqrt(np.float64(np.float32(1e-6))), rtol=2.0 ** -21, atol=0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_norm_of_subnormal_rows(lb, dt):
    """Rows whose root mean square has no FP32 inverse: without eps they have a norm like any others."""
    banner(f"norm of subnormal rows {dt}")
    g = np.random.default_rng(11)
    h = g.standard_normal((6, 1, 128)) * 2.0 ** -126
    h[1] *= 2.0 ** -6
    h[2] *= 2.0 ** -120                                          # all 0 but where it is moved up below
    h[2, 0, 5], h[2, 0, 77] = 2.0 ** -133, -2.0 ** -132          # BF16's smallest value, and twice that
    h[3] *= 2.0 ** 20                                            # a mean just above 2^-252 x 2^40
    h[4] *= 2.0 ** 1                                             # a mean around 2^-250
    x = torch.from_numpy(h).to(dt).cuda()
    h = to_host64(x)
    w = torch.full((128,), 2.0, device="cuda")
    got, same = lb.norm_rotate(x, x, q_norm=w, eps=0.0)
    want = od.norm(h, 2.0, 0.0)
    big = np.abs(want).max(-1, keepdims=True)
    assert (big[[0, 1, 2, 3, 4]] > 1).all()
    assert (np.abs(to_host64(got) - want) <= 2.0 ** -21 * big + 1.001 * _half_ulp(want, got.dtype)).all()
    assert torch.equal(same, x)                                  # keys without a norm stay as they are
    # and in the append: the same norm, then the same codes
    a, b = (lb.new_kv_cache(1, 1, 16, 128) for _ in range(2))
    where = (_i32([[0]]), _i32([0, 6]), _i32([0]), 6)
    lb.kv_append(x, x, a, *where, k_norm=w, eps=0.0)
    y = lb.norm_rotate(x.float(), q_norm=w, eps=0.0)
    lb.kv_append(y, x.float(), b, *where)
    assert torch.equal(a.k, b.k) and torch.equal(a.k_scale, b.k_scale)


def test_rows_of_many_tokens_and_heads(lb):
    """The most heads that a call takes, and one head of many tokens."""
    banner("norm of 65536 heads, and of 300000 tokens")
    w = torch.ones(64, device="cuda")
    for shape in ((3, 65536, 64), (300000, 1, 64)):
        x = torch.randn(shape, device="cuda").bfloat16()
        y = lb.norm_rotate(x, q_norm=w)
        z = x.double()
        z = z / (z.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        assert ((y.double() - z).abs() <= z.abs() * 1.01 * 2.0 ** -8 + 2.0 ** -19).all()


def test_calls_without_tokens(lb):
    banner("append with norms, norm and rotation, attention: no tokens")
    x, w = torch.empty((0, 2, 64), device="cuda").half(), torch.ones(64, device="cuda").half()
    cache = lb.new_kv_cache(2, 2, 16, 64)
    cos, sin = lb.rope_tables(10, 64)
    for batch in (0, 3):
        where = (_i32(np.zeros((batch, 1))), _i32(np.zeros(batch + 1)), _i32(np.zeros(batch)))
        q = lb.kv_append(x, x, cache, *where, 1, q=x, cos=cos, sin=sin, q_norm=w, k_norm=w)
        assert q.shape == x.shape
        assert lb.attention(q, cache, *where, 1, 10, window=5, sinks=2).shape == x.shape
    q, k = lb.norm_rotate(x, x, w, w, cos, sin)
    assert q.shape == k.shape == x.shape


def test_norm_rotate_in_more_than_one_launch(lb):
    """More units than one launch takes: 8200 tokens of 65536 heads."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GiB of free GPU memory")
    banner("norm and rotation: 8200 tokens of 65536 heads")
    x = torch.randn((1, 65536, 64), device="cuda").half().expand(8200, -1, -1)     # one token's rows, read again for each
    w = torch.ones(64, device="cuda").half()
    cos, sin = lb.rope_tables(8200, 64)
    y = lb.norm_rotate(x, q_norm=w, cos=cos, sin=sin)
    at = [0, 1, 8190, 8191, 8192, 8193, 8199]
    assert torch.equal(y[at], lb.norm_rotate(x[at], q_norm=w, cos=cos, sin=sin, positions=_i32(at)))
    del y
    torch.cuda.empty_cache()


APPEND = [  # starts, new, H, Hq, page, D, rot, interleaved, dtype, weights' dtype
    ([0], [1], 1, 1, 16, 64, 64, False, "bf16", "bf16"),
    ([15, 16, 17], [1, 1, 1], 2, 6, 16, 64, 32, True, "f16", "f32"),
    ([0, 5, 100], [37, 0, 3], 2, 2, 32, 128, 128, False, "bf16", "f16"),
    ([63, 64, 1], [2, 64, 200], 3, 3, 64, 128, 64, True, "f32", "f32"),
    ([7], [300], 2, 10, 128, 256, 256, False, "f16", "f16"),
    ([250, 3], [9, 258], 1, 8, 256, 64, 0, False, "bf16", "bf16"),
]


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
def test_kv_append_with_norms(lb, case):
    starts, new, H, Hq, page, D, rot, inter, dt, wdt = case
    banner(f"append with norms {case}")
    g = np.random.default_rng(2000 + len(starts) + D + page)
    lens = np.asarray(starts) + np.asarray(new)
    P = Paged(lens, H, page, D, seed=5)
    T = int(sum(new))
    x, hx = _values(g, (T, Hq + 2 * H, D), dt)
    (wq, hwq), (wk, hwk) = _weights(g, D, wdt), _weights(g, D, wdt)
    cu = np.concatenate([[0], np.cumsum(new)])
    cos, sin = _rope(int(lens.max()), rot)
    dev = [torch.from_numpy(a).cuda() for a in (cos, sin)] if rot else [None, None]
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, new)]).astype(int)
    eps = np.float64(np.float32(1e-6))
    for norm_q, norm_k in ((wq, wk), (None, wk), (wq, None)):
        cache = P.cache(lb)
        bad = torch.zeros(2, dtype=torch.int32, device="cuda")
        qo = lb.kv_append(x[:, Hq:Hq + H], x[:, Hq + H:], cache, _i32(P.table), _i32(cu), _i32(starts), max(new), q=x[:, :Hq],
                          cos=dev[0], sin=dev[1], interleaved=inter, bad_count=bad, q_norm=norm_q, k_norm=norm_k)
        assert bad.tolist() == [0, 0]
        turn = (lambda a: od.rotate(a, pos, cos, sin, inter)) if rot else (lambda a: a)
        n = od.norm(hx[:, :Hq], hwq, eps) if norm_q is not None else hx[:, :Hq]
        want = turn(n)
        big = np.abs(n).max(-1, keepdims=True)
        assert (np.abs(to_host64(qo) - want) <= 2.0 ** -21 * big + 1.001 * _half_ulp(want, qo.dtype)).all()
        keys = turn(od.norm(hx[:, Hq:Hq + H], hwk, eps) if norm_k is not None else hx[:, Hq:Hq + H])
        got = {m: [t.cpu().numpy() for t in ts] for m, ts in dict(k=(cache.k, cache.k_scale), v=(cache.v, cache.v_scale)).items()}
        start, dense = dict(k=(P.k, P.ks), v=(P.v, P.vs)), dict(k=keys, v=hx[:, Hq + H:])
        for b, (s0, m) in enumerate(zip(starts, new)):
            for slot in range(s0 // page, (s0 + m - 1) // page + 1 if m else s0 // page):
                p, lo, hi = P.table[b, slot], max(s0, slot * page), min(s0 + m, (slot + 1) * page)
                for name in "kv":
                    for h in range(H):
                        first, many = lo - slot * page, hi - lo
                        was = od.block_codes(start[name][0][p, h], name, page, D)
                        now = od.block_codes(got[name][0][p, h], name, page, D)
                        rows = dense[name][cu[b] + lo - s0:cu[b] + hi - s0, h]
                        _, want = od.append_block(was, start[name][1][p, h], first, rows)
                        scale, old = float(got[name][1][p, h]), float(start[name][1][p, h])
                        assert abs(scale - want) <= 2.0 ** -20 * want
                        assert (np.abs(now[first:first + many] * scale - rows) <= 0.5001 * scale).all()
                        assert (np.abs(now[:first] * scale - was[:first] * old) <= (0 if scale == old else 0.5001 * scale)).all()
                        assert np.array_equal(now[first + many:], was[first + many:])


def test_append_with_norms_is_the_dense_norm_then_append(lb):
    """The same codes and queries as norm_rotate in FP32 first, then a plain append of its result."""
    banner("append with norms against norm_rotate and append")
    g = np.random.default_rng(6)
    x, _ = _values(g, (90, 8, 128), "f32")
    (wq, _), (wk, _) = _weights(g, 128, "f32"), _weights(g, 128, "f32")
    cos, sin = (torch.from_numpy(a).cuda() for a in _rope(100, 64))
    a, b = (lb.new_kv_cache(4, 2, 64, 128) for _ in range(2))
    where = (_i32([[2, 1]]), _i32([0, 90]), _i32([10]), 90)
    q = lb.kv_append(x[:, 4:6], x[:, 6:], a, *where, q=x[:, :4], cos=cos, sin=sin, q_norm=wq, k_norm=wk)
    q2, k2 = lb.norm_rotate(x[:, :4], x[:, 4:6], wq, wk, cos, sin, positions=_i32(np.arange(10, 100)))
    lb.kv_append(k2, x[:, 6:], b, *where)
    assert torch.equal(q, q2)
    for s, t in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert torch.equal(s, t)


def test_append_with_norms_nonfinite_rows_and_missing_places(lb):
    banner("append with norms: NaN, infinity, no page, no position")
    x = torch.randn((40, 2, 64), device="cuda").half()
    x[3, 0, 5], x[4, 1, 6] = float("nan"), float("inf")
    cos, sin = (torch.from_numpy(a).cuda() for a in _rope(36, 64))
    w = torch.ones(64, device="cuda").half()
    cache = lb.new_kv_cache(3, 2, 16, 64)
    bad = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = lb.kv_append(x, torch.zeros_like(x), cache, _i32([[2, -1, 0]]), _i32([0, 40]), _i32([0]), 40, q=x, cos=cos, sin=sin,
                     bad_count=bad, q_norm=w, k_norm=w)
    # the NaN's row (64), the infinity and its partner of the rotation (2); 16 tokens without a page, 4 without a position
    assert bad.tolist() == [66, 20] and (q[36:] == 0).all()
    k, _ = lb.kv_read(cache, _i32([[2, -1, 0]]), _i32([0, 36]), _i32([0]), 36, 36, torch.float32)
    assert (k[3, 0] == 0).all() and (k[4, 1] == 0).all() and (k[16:32] == 0).all() and torch.isfinite(k).all()
    assert (k[5] != 0).any() and (k[32:] != 0).any()


# ------------------------------------------------------------------- tables ---

TABLES = [  # positions, rot, first, base, scaling
    (1, 32, 0, 1e4, dict()),
    (1000, 64, 0, 1e4, dict()),
    (777, 96, 100000, 5e5, dict(scaling="linear", factor=3.0)),
    (300, 128, 5000, 1e6, dict(scaling="ntk", factor=8.0)),
    (2000, 128, 30000, 1e6, dict(scaling="yarn", factor=4.0, original=32768, low=1.0, high=32.0)),
    (50, 256, 7, 1e4, dict(scaling="yarn", factor=16.0, original=100, low=1.0, high=32.0)),
    (400, 64, 1000, 5e5, dict(scaling="wavelength", factor=8.0, original=8192, low=1.0, high=4.0)),
    (64, 32, 2 ** 24, 1e4, dict(scaling="linear", factor=1.0, magnitude=0.7)),
    (100, 64, 2 ** 31 - 100, 1e4, dict()),
]


@pytest.mark.parametrize("case", TABLES, ids=[str(i) for i in range(len(TABLES))])
def test_rope_tables(lb, case):
    n, rot, first, base, kw = case
    banner(f"rotary tables {case}")
    cos, sin = lb.rope_tables(n, rot, base=base, first=first, **kw)
    assert cos.shape == sin.shape == (n, rot // 2) and cos.dtype == torch.float32
    f, m = od.frequencies(rot, base, **{a: v for a, v in kw.items() if a != "magnitude"})
    m = kw.get("magnitude", m)
    pos = np.arange(first, first + n)
    bound = m * (2.0 ** -21 + 2.0 ** -50 * pos[:, None])
    a = _reduced(pos, f)
    assert (np.abs(to_host64(cos) - m * np.cos(a.astype(np.float64))) <= bound).all()
    assert (np.abs(to_host64(sin) - m * np.sin(a.astype(np.float64))) <= bound).all()


def _reduced(pos, f):
    """pos * f without whole turns, in long double with 2 pi from its decimal digits: off by 2^-64 of the angle."""
    two_pi = np.longdouble("6.283185307179586476925286766559")
    a = pos[:, None].astype(np.longdouble) * f.astype(np.longdouble)
    return a - np.rint(a / two_pi) * two_pi


def test_rope_tables_out_and_stream(lb):
    banner("rotary tables into given tensors, on another stream; rows by offset; none")
    s = torch.cuda.Stream()
    big = lb.rope_tables(500, 64, base=5e5, scaling="wavelength", factor=8.0, original=8192, low=1.0, high=4.0)
    out = tuple(torch.empty((40, 32), device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    got = lb.rope_tables(40, 64, base=5e5, scaling="wavelength", factor=8.0, original=8192, low=1.0, high=4.0, first=300, out=out,
                         stream=s)
    s.synchronize()
    assert got[0] is out[0] and all(torch.equal(a, b[300:340]) for a, b in zip(got, big))
    assert lb.rope_tables(0, 64)[0].shape == (0, 32)


# -------------------------------------------------------------------- pages ---

class Pool:
    """A cache whose bytes and scales name their page, so that every copy shows."""

    def __init__(self, lb, pages, page, H=2, D=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.cache = lb.KVCache(*(torch.randint(0, 256, (pages, H, page, D), generator=g, device="cuda", dtype=torch.uint8)
                                  for _ in range(2)),
                                *(torch.rand((pages, H), generator=g, device="cuda") for _ in range(2)))

    def arrays(self):
        c = self.cache
        return [t.cpu().numpy().copy() for t in (c.k, c.v, c.k_scale, c.v_scale)]


def _remap_check(lb, table, lens, pages, page, rows=None, room=None, cache=None, **kw):
    table, lens = np.asarray(table, dtype=np.int32), np.asarray(lens, dtype=np.int32)
    want, L, pairs, counts = od.remap(table, lens, pages, page, rows=rows, room=room, **kw)
    pool = Pool(lb, pages, page) if cache is None else cache
    before = pool.arrays()
    plan = lb.kv_remap(_i32(table), _i32(lens), pool.cache, rows=None if rows is None else _i32(rows),
                       room=None if room is None else _i32(room), **kw)
    assert plan.counts.tolist() == counts
    assert np.array_equal(plan.table.cpu().numpy(), want) and np.array_equal(plan.lens.cpu().numpy(), L)
    src, dst = plan.src.tolist(), plan.dst.tolist()
    assert list(zip(src, dst))[:len(pairs)] == pairs and set(src[len(pairs):] + dst[len(pairs):]) <= {-1}
    # what the contract promises of the pairs: no destination twice, or a source, or kept by a new sequence before
    assert len({d for _, d in pairs}) == len(pairs) and not {d for _, d in pairs} & {s for s, _ in pairs}
    lb.kv_copy_pages(pool.cache, plan.src, plan.dst, plan.counts)
    for a, b in zip(before, pool.arrays()):
        for s, d in pairs:
            a[d] = a[s]
        assert np.array_equal(a, b)
    return plan


def _random_tables(g, B, W, pages, page, shared, junk):
    """Ragged sequences with common first pages, some entries that are no page."""
    lens = g.integers(0, W * page + 1, B)
    perm = g.permutation(pages)
    table = np.full((B, W), -1, dtype=np.int64)
    at = 0
    for b in range(B):
        n = -(-int(lens[b]) // page)
        n = min(n, max(0, pages - at))
        table[b, :n] = perm[at:at + n]
        at += n
    if B:
        prefix = max(0, min(shared, int(lens[0]) // page))
        for b in range(1, B):
            m = min(prefix, int(lens[b]) // page)
            table[b, :m] = table[0, :m]
    hit = g.random((B, W)) < junk
    table[hit] = g.choice([-1, -7, pages, 2 ** 31 - 1], int(hit.sum()))
    return table, lens


@pytest.mark.parametrize("seed", range(24))
def test_kv_remap(lb, seed):
    g = np.random.default_rng(seed)
    page = int(g.choice([16, 32, 64, 128, 256]))
    B, W = int(g.integers(1, 40)), int(g.integers(1, 12))
    pages = int(g.integers(max(1, B * W // 2), 2 * B * W + 4))
    table, lens = _random_tables(g, B, W, pages, page, int(g.integers(0, W)), 0.05 if seed % 3 == 0 else 0.0)
    if seed % 4 == 1:
        lens = lens + g.choice([-5 * page, 0, 3 * W * page], B)  # negative ones, and ones past the table
    R = int(g.integers(1, 60))
    rows = g.integers(-1 if seed % 2 else 0, B + (seed % 2), R)
    room = None if seed % 5 == 0 else g.integers(-3, 4 * page, R)
    window = 0 if seed % 3 == 1 else int(g.integers(1, W * page))
    kw = dict(window=window, sinks=int(g.integers(0, 3 * page)), compact=bool(seed % 2), width=None if seed % 7 else W + 3)
    banner(f"remap {B} x {W} of {pages} pages of {page} to {R} rows, {kw}")
    _remap_check(lb, table, lens, pages, page, rows=rows, room=room, **kw)


def test_kv_remap_by_default_keeps_everything(lb):
    banner("remap: identity, narrower and wider tables")
    g = np.random.default_rng(50)
    table, lens = _random_tables(g, 9, 8, 100, 16, 0, 0.0)
    plan = _remap_check(lb, table, lens, 100, 16)
    kept = np.where(np.arange(8)[None] < -(-lens // 16)[:, None], table, -1)
    assert np.array_equal(plan.table.cpu().numpy(), kept) and plan.counts.tolist()[0] == 0
    for width in (1, 3, 8, 20):
        _remap_check(lb, table, lens, 100, 16, width=width, room=np.full(9, 40))
    _remap_check(lb, table, lens, 100, 16, window=2 ** 40, sinks=2 ** 40)


@pytest.mark.parametrize("compact", [False, True])
def test_kv_remap_of_large_tables(lb, compact):
    """Tables and pools at the end of what one workgroup takes, and beyond: the steps as launches of their own."""
    banner(f"remap of 300 x 100, compact {compact}")
    g = np.random.default_rng(60)
    table, lens = _random_tables(g, 300, 100, 40000, 16, 20, 0.01)
    rows = np.concatenate([g.permutation(300)[:170], g.integers(0, 300, 30), [-1, 300]])
    _remap_check(lb, table, lens, 40000, 16, rows=rows, room=g.integers(0, 90, len(rows)), window=900, sinks=40, compact=compact,
                 width=110)
    # few rows over a pool of more pages than one workgroup takes; with all rows the free pages run out
    _remap_check(lb, table[:3], lens[:3], 70000, 16, rows=np.array([2, 2, 0]), room=np.array([50, 0, 7]), compact=compact)
    table, lens = _random_tables(g, 300, 100, 17000, 16, 0, 0.0)
    _remap_check(lb, table, lens, 17000, 16, rows=g.integers(0, 300, 2000), room=np.full(2000, 200), compact=compact)
    # more slots than one workgroup takes, with common pages, a window and entries that are no page
    table, lens = _random_tables(g, 300, 100, 40000, 16, 20, 0.01)
    rows = g.integers(-1, 301, 900)
    _remap_check(lb, table, lens, 40000, 16, rows=rows, room=g.integers(-9, 90, 900), window=900, sinks=40, compact=compact,
                 width=110)
    # more pages than its sets hold
    _remap_check(lb, table[:50], lens[:50], 170000, 16, rows=rows[:60], room=g.integers(0, 90, 60), window=500, compact=compact,
                 cache=Pool(lb, 170000, 16, 1))


def test_kv_remap_of_nothing(lb):
    banner("remap: no old sequences, no new ones, tables without a slot")
    _remap_check(lb, np.zeros((0, 4)), np.zeros(0), 10, 16, rows=np.array([-1, 0, 5]), room=np.array([17, 0, 33]))
    for compact in (False, True):
        for pages in (10, 3000, 100000):                          # all sequences end
            _remap_check(lb, np.array([[3, 1]]), [20], pages, 16, rows=np.zeros(0, dtype=int), compact=compact)
    _remap_check(lb, np.array([[3, 1]]), [20], 10, 16, rows=np.array([0]), width=0, room=np.array([5]))
    _remap_check(lb, np.zeros((2, 0)), [7, 0], 10, 16, room=np.array([5, 5]), width=2)
    _remap_check(lb, np.array([[0]]), [16], 1, 16, rows=np.array([0, 0]), room=np.array([1, 1]), width=2)   # no page left


def test_kv_remap_from_several_threads_and_streams(lb):
    """Four host threads with streams of their own, each with its own tables; every result as alone."""
    banner("remap from four threads")
    import threading
    g = np.random.default_rng(80)
    jobs, got, errors = [], [None] * 4, []
    for i in range(4):
        table, lens = _random_tables(g, 20 + 90 * i, 30, 30000, 16, 5, 0.01)
        rows, room = g.integers(-1, len(lens), 50), g.integers(0, 40, 50)
        jobs.append((table, lens, rows, room, bool(i % 2)))
    pool = Pool(lb, 30000, 16, 1)
    args = [(_i32(t), _i32(n), pool.cache, _i32(r), _i32(m)) for t, n, r, m, _ in jobs]
    torch.cuda.synchronize()

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got[i] = lb.kv_remap(*args[i], window=100, sinks=20, compact=jobs[i][4], stream=s)
            s.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for (table, lens, rows, room, compact), plan in zip(jobs, got):
        want, L, pairs, counts = od.remap(table, lens, 30000, 16, rows=rows, room=room, window=100, sinks=20, compact=compact)
        assert plan.counts.tolist() == counts and np.array_equal(plan.table.cpu().numpy(), want)
        assert list(zip(plan.src.tolist(), plan.dst.tolist()))[:len(pairs)] == pairs and plan.lens.tolist() == L.tolist()


def test_kv_copy_pages_lists(lb):
    banner("copy pages: counts, entries that are no page, large pages, a pair twice")
    for pages, page, H, D in ((7, 16, 1, 64), (9, 256, 3, 256), (40, 64, 8, 128)):
        pool = Pool(lb, pages, page, H, D)
        for src, dst, count in (([0, 1, -1, pages, 2, 3, 3], [4, 5, 6, 6, -3, pages, 3], None), ([0, 1], [6, 5], 1), ([2, 1], [6, 5], 0),
                                ([0, 1], [6, 5], -4), ([0, 2], [6, 5], 100), ([3, 3], [4, 4], None)):
            before = pool.arrays()
            lb.kv_copy_pages(pool.cache, _i32(src), _i32(dst), None if count is None else _i32([count]))
            n = len(src) if count is None else max(0, min(count, len(src)))
            for a, b in zip(before, pool.arrays()):
                for s, d in list(zip(src, dst))[:n]:
                    if 0 <= s < pages and 0 <= d < pages:
                        a[d] = a[s]
                assert np.array_equal(a, b)
    lb.kv_copy_pages(pool.cache, _i32([]), _i32([]))


def test_kv_copy_pages_beyond_4_gib(lb):
    banner("copy pages of a cache of 4.6 GB")
    cache = lb.new_kv_cache(36000, 2, 256, 256)
    cache.k[35999] = 7
    cache.v[35999] = 9
    cache.k[3] = 5
    cache.k_scale[35999] = 2.5
    lb.kv_copy_pages(cache, _i32([35999, 3]), _i32([17000, 35998]))
    assert (cache.k[17000] == 7).all() and (cache.v[17000] == 9).all() and (cache.k_scale[17000] == 2.5).all()
    assert (cache.k[35998] == 5).all() and int((cache.k == 7).sum()) == 2 * 2 * 256 * 256


# ----------------------------------------------------------------- together ---

def _step(lb, x, cache, table, cu, starts, lens, tables, w, window, sinks, most):
    q = lb.kv_append(x[:, 4:6], x[:, 6:], cache, table, cu, starts, 1, q=x[:, :4], cos=tables[0], sin=tables[1], q_norm=w, k_norm=w)
    return lb.attention(q, cache, table, cu, lens, 1, most, window=window, sinks=sinks)


def test_forked_sequences_decode_as_if_each_had_its_own_cache(lb):
    """A prompt, forked into three answers that go on with tokens of their own,
    reordered, compacted and slid along a window: every step's attention equals
    that of caches in which each sequence has its own pages from the start."""
    banner("prompt, fork, window, compact, reorder")
    page, D, window, sinks, W, steps = 16, 64, 60, 5, 12, 45
    g = torch.Generator(device="cuda").manual_seed(3)
    tables = lb.rope_tables(W * page, D, base=5e5, scaling="yarn", factor=2.0, original=100)
    w = 1 + torch.randn(D, generator=g, device="cuda") / 8
    prompt = torch.randn((70, 8, D), generator=g, device="cuda").bfloat16()
    shared, own = lb.new_kv_cache(60, 2, page, D), [lb.new_kv_cache(W, 2, page, D) for _ in range(3)]
    flat = _i32(np.arange(W)[None])

    def fill(cache, table):
        lb.kv_append(prompt[:, 4:6], prompt[:, 6:], cache, table, _i32([0, 70]), _i32([0]), 70, cos=tables[0], sin=tables[1], k_norm=w)

    plan = lb.kv_remap(torch.full((0, W), -1, dtype=torch.int32, device="cuda"), _i32([]), shared, rows=_i32([-1]), room=_i32([70]))
    fill(shared, plan.table)
    for c in own:
        fill(c, flat)
    table, lens = plan.table, _i32([70])
    order = [0, 1, 2]                                         # the own cache of each row
    rows = _i32([0, 0, 0])
    used = []
    for step in range(steps):
        plan = lb.kv_remap(table, lens, shared, rows=rows, room=_i32([1, 1, 1]), window=window, sinks=sinks, compact=step % 10 == 7)
        lb.kv_copy_pages(shared, plan.src, plan.dst, plan.counts)
        assert int(plan.counts[2]) == 0
        used.append(int(plan.counts[1]))
        table, at = plan.table, plan.lens
        lens = at + 1
        x = torch.randn((3, 8, D), generator=g, device="cuda").bfloat16()
        most = 71 + step
        y = _step(lb, x, shared, table, _i32([0, 1, 2, 3]), at, lens, tables, w, window, sinks, most)
        for r in range(3):
            z = _step(lb, x[r:r + 1], own[order[r]], flat, _i32([0, 1]), _i32([70 + step]), _i32([71 + step]), tables, w, window,
                      sinks, most)
            assert torch.equal(y[r:r + 1], z), (step, r)
        perm = [1, 2, 0] if step % 3 == 1 else [0, 1, 2]
        rows, order = _i32(perm), [order[i] for i in perm]
    # the pages that the window passed have gone back: 5 first tokens and 60 of each sequence in at most 1 + 5 pages each
    assert used[-1] <= 3 * 6 and max(used) <= 5 + 3 * 6


def test_together_in_a_graph(lb):
    """Remap, copy, append with norms, attention with first tokens, dense rows and
    tables under capture; every replay against the eager result, with the cache
    put back and other work between them."""
    banner("graph of the operators of long contexts")
    page, D, W = 16, 64, 200
    P = Paged([2900, 1500], 2, page, D, seed=70, spare=400)
    x, _ = _values(np.random.default_rng(71), (3, 8, D), "bf16")
    cache, clean = P.cache(lb), P.cache(lb)
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    old, lens, rows, room = _i32(P.table), _i32([2900, 1500]), _i32([0, 0, 1]), _i32([1, 1, 1])
    cu, pos = _i32([0, 1, 2, 3]), _i32([2900, 2900, 1500])

    def put_back():
        for a, b in ((cache.k, clean.k), (cache.v, clean.v), (cache.k_scale, clean.k_scale), (cache.v_scale, clean.v_scale)):
            a.copy_(b)

    def step():
        tables = lb.rope_tables(W * page, D, base=1e6, scaling="ntk", factor=2.0)
        plan = lb.kv_remap(old, lens, cache, rows=rows, room=room, window=2000, sinks=4)
        lb.kv_copy_pages(cache, plan.src, plan.dst, plan.counts)
        y = _step(lb, x, cache, plan.table, cu, plan.lens, plan.lens + 1, tables, w, 2000, 4, W * page)
        turned = lb.norm_rotate(x[:, :4], x[:, 4:6], w, w, *tables, positions=pos)
        return (*plan, y, *turned, *tables, cache.k.clone(), cache.k_scale.clone())

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
        assert all(torch.equal(a, b) for a, b in zip(res, eager))
        put_back()
        assert all(torch.equal(a, b) for a, b in zip(step(), eager))


@pytest.mark.parametrize("flags", [["--window", "16", "--sinks", "3", "--answers", "3", "--head-norms", "--scaling", "yarn"],
                                   ["--answers", "2", "--scaling", "wavelength", "--tokens", "1"],
                                   ["--head-norms", "--scaling", "ntk", "--window", "5"]])
def test_example_with_windows_norms_and_answers(lb, capsys, monkeypatch, flags):
    """The example program on a small model against float64: 2 % a layer, as in
    test_gpu_decode.py (the norm of a head adds one rounding, of the weights none)."""
    banner(f"example: {flags}")
    import importlib.util
    import os
    import sys
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "text_decode.py")
    spec = importlib.util.spec_from_file_location("text_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(sys, "argv", ["text_decode", "--layers", "2", "--hidden", "256", "--q-heads", "6", "--kv-heads", "2",
                                      "--head-dim", "64", "--mlp", "384", "--vocab", "500", "--page", "16", "--batch", "2",
                                      "--prompt", "37", "--tokens", "9", "--check", *flags])
    m.main()
    assert "relative difference" in capsys.readouterr().out
