"""The decoding operators on paths and inputs that the tests of test_gpu_decode.py
do not reach: definitions, tolerances and helpers as there unless a test says
otherwise."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from oracle import paged as od
from gpu_util import TORCH_DT, banner, dev_bits, to_host64
from test_gpu_decode import Paged, _attend, _f16, _gemv_check, _half_ulp, _i32, _rope, _values, lb  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ appending ---

def _append_both(lb, cache, rows, start, dt):
    t = torch.from_numpy(rows).cuda().to(TORCH_DT[dt])
    lb.kv_append(t, t, cache, _i32([[0]]), _i32([0, len(rows)]), _i32([start]), len(rows))
    torch.cuda.synchronize()


def _codes_and_scale(cache, page, D):
    return [(od.block_codes(c.cpu().numpy()[0, 0], n, page, D), np.float32(s.cpu().numpy()[0, 0]))
            for n, c, s in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale))]


@pytest.mark.parametrize("m", [1, 3, 7, 13, 41, 61, 83])
def test_append_ties_go_to_even(lb, m):
    """A block whose largest magnitude is 127 m has the scale m exactly, and the
    values (n + 1/2) m lie on ties, in FP32 as in the definition: no tolerance.
    Older codes that follow a scale grown to 2 m or to 82 lie on ties too."""
    banner(f"append ties, scale {m}")
    page, D = 16, 64
    n = np.arange(-127, 127) + 0.5
    rows = np.zeros((8, 1, D), dtype=np.float32)
    rows.reshape(-1)[:len(n)] = n * m
    rows[7, 0, 63] = 127 * m
    cache = lb.new_kv_cache(1, 1, page, D)
    _append_both(lb, cache, rows, 0, "f32")
    want = np.rint(rows[:, 0].astype(np.float64) / m).astype(np.int64)
    for codes, scale in _codes_and_scale(cache, page, D):
        assert scale == m and np.array_equal(codes[:8], want)
    top = 2 * m if m < 41 else 82
    if top < m:
        return
    _append_both(lb, cache, np.full((1, 1, D), 127 * top, dtype=np.float32), 8, "f32")
    want = np.rint(want.astype(np.float32) * (np.float32(m) / np.float32(top))).astype(np.int64)
    for codes, scale in _codes_and_scale(cache, page, D):
        assert scale == max(m, top) and np.array_equal(codes[:8], want) and (codes[8] == 127).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page,D", [(16, 64), (64, 128), (256, 256)])
def test_append_is_the_fp32_definition_bit_for_bit(lb, page, D, dt):
    """Without rotation: scale = a / 127, codes rint(r / scale), older codes
    rint(c (s_old / s)), each quotient rounded once in FP32."""
    banner(f"append against FP32 arithmetic, page {page}, D {D}, {dt}")
    g = np.random.default_rng(page + D)
    cache = lb.new_kv_cache(1, 1, page, D)
    f = np.float32
    codes, scale = np.zeros((page, D), dtype=np.int64), f(0)
    at = 0
    for n, size in ((page // 2 - 1, 1.0), (3, 0.5), (2, 1.7), (page // 4, 40.0)):
        rows = (g.standard_normal((n, 1, D)) * size).astype(np.float32)
        rows = torch.from_numpy(rows).to(TORCH_DT[dt]).float().numpy()
        _append_both(lb, cache, rows, at, dt)
        new = max(scale, f(np.abs(rows).max()) / f(127))
        if at and new != scale:
            codes[:at] = np.rint(codes[:at].astype(f) * (scale / new))
        codes[at:at + n] = np.clip(np.rint(rows[:, 0] / new), -127, 127)
        at, scale = at + n, new
        for have, s in _codes_and_scale(cache, page, D):
            assert s == scale and np.array_equal(have[:at], codes[:at])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_queries_without_a_position_become_zeros(lb, dt, in_place):
    """Tables of 20 positions: tokens 20 .. 39 have none, the last page no token with one."""
    banner(f"append, queries past the tables, {dt}, in place {in_place}")
    H, Hq, page, D = 2, 5, 16, 64
    g = np.random.default_rng(90)
    x, _ = _values(g, (40, Hq + 2 * H, D), dt)
    cos, sin = (torch.from_numpy(a).cuda() for a in _rope(40, D))
    res = []
    for rows in (40, 20):
        y, cache = x.clone(), lb.new_kv_cache(3, H, page, D)
        q = y[:, :Hq] if in_place else x[:, :Hq]
        out = q if in_place else torch.full((40, Hq, D), 7.0, dtype=x.dtype, device="cuda")
        bad = torch.zeros(2, dtype=torch.int32, device="cuda")
        lb.kv_append(x[:, Hq:Hq + H], x[:, Hq + H:], cache, _i32([[2, 0, 1]]), _i32([0, 40]), _i32([0]), 40, q=q,
                     cos=cos[:rows].contiguous(), sin=sin[:rows].contiguous(), q_out=out, bad_count=bad)
        assert bad.tolist() == [0, 40 - rows]
        assert torch.equal(y[:, Hq:], x[:, Hq:])
        res.append((out.clone(), cache))
    (full, c0), (cut, c1) = res
    assert torch.equal(cut[:20], full[:20]) and (cut[20:] == 0).all() and (full[20:] != 0).any()
    assert torch.equal(c0.k[2], c1.k[2]) and torch.equal(c0.v[2], c1.v[2])
    assert (c1.k[1] == 0).all() and (c1.v[1] == 0).all()                   # the last page stays as it was


@pytest.mark.parametrize("width", [0, 5])
def test_an_empty_batch_gives_empty_results(lb, width):
    """A scheduler's step without sequences: every array is empty."""
    banner(f"empty batch, table width {width}")
    cache = lb.new_kv_cache(3, 2, 16, 64)
    x = torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    e = [torch.empty(shape, dtype=torch.int32, device="cuda") for shape in ((0, width), (0,))]
    cu = _i32([0])
    cos, sin = (torch.from_numpy(a).cuda() for a in _rope(20, 64))
    q = lb.kv_append(x[:, 4:6], x[:, 6:], cache, e[0], cu, e[1], 0, q=x[:, :4], cos=cos, sin=sin)
    k, v = lb.kv_read(cache, e[0], cu, e[1], 0, 0)
    y, lse = lb.attention(x[:, :4], cache, e[0], cu, e[1], 0, 0, return_lse=True)
    assert q.shape == y.shape == (0, 4, 64) and k.shape == v.shape == (0, 2, 64) and lse.shape == (0, 4)


# ------------------------------------------------------------------ attention ---

def _sinks(L, Hq, n, seed):
    """Queries and a cache of which every 32nd token takes nearly all of the softmax
    and has the value 0: what is left of the others, about 2^-24.6 each, is the result."""
    P = Paged([L], 1, 16, 128, seed=seed)
    g = np.random.default_rng(seed + 1)
    q = g.standard_normal((n, Hq, 128))
    q[:, :, 0] = 8
    q = oracle.encode(q, "bf16")
    codes = [od.block_codes(P.k[p, 0], "k", 16, 128) for p in range(P.pages)]
    for p in range(P.pages):
        codes[p][:, 0] = 0
    for t in range(0, L, 32):                                  # the first token of every other page
        p = P.table[0, t // 16]
        codes[p][:] = 0
        codes[p][0, 0] = 127
        P.ks[p] = 17.3 / (128 ** -0.5 * 8 * 127)
        v = od.block_codes(P.v[p, 0], "v", 16, 128)
        v[0] = 0
        P.v[p, 0] = od.block_bytes(v, "v").reshape(16, 128)
    for p in range(P.pages):
        P.k[p, 0] = od.block_bytes(codes[p], "k").reshape(16, 128)
    return P, dev_bits(q, "bf16"), oracle.decode(q, "bf16")


@pytest.mark.parametrize("n", [1, 30])
def test_attention_keeps_what_sinks_leave(lb, n):
    """Scores of 17.3 against normal ones: the other tokens' probabilities are
    2^-24.6 e^s of a sink's, and all of the result. Relative 2-norm error: the BF16
    output's rounding is at most 2^-9; FP16 probabilities above their normal range
    add 2^-12 (independent roundings of at most 2^-11), and 2^-9.6 if no more than
    seven powers of two lift a sink's above 1 (steps of 2^-31 of it). Together below 2^-8."""
    banner(f"attention with sinks, {n} queries")
    L, Hq = 4000, 4
    P, q, hq = _sinks(L, Hq, n, 95)
    out, lse = lb.attention(q, P.cache(lb), _i32(P.table), _i32([0, n]), _i32([L]), n, L, return_lse=True)
    k, v = (od.cache_rows(*a, 0, L) for a in ((P.k, P.ks, P.table[0], "k"), (P.v, P.vs, P.table[0], "v")))
    vs = P.vs[P.table[0][np.arange(L) // 16]].astype(np.float64)
    want, we, _, _ = od.attention(hq, k, v, vs, L - n, 128 ** -0.5, True, 0)
    O = to_host64(out)
    off = np.linalg.norm(O - want, axis=2) / np.linalg.norm(want, axis=2)
    print(f"relative error {off.max():.3g}")
    assert (np.abs(to_host64(lse) - we) <= 2.0 ** -14 + 2.0 ** -22 * np.abs(we)).all()
    assert off.max() <= 2.0 ** -8


@pytest.mark.parametrize("n", [1, 50])
@pytest.mark.parametrize("power", [125, 126, 127, -120, -126])
def test_attention_bf16_queries_at_the_ends_of_the_range(lb, n, power):
    """Rows whose largest magnitude is 2^power .. 2^(power + 1), with key scales and
    the softmax scale that bring the scores back to order 1 (each a normal number)."""
    banner(f"attention, bf16 queries of 2^{power}, {n} queries")
    P = Paged([150], 2, 32, 64, seed=100)
    half = 20 if power > 0 else -20
    P.ks[:] = P.ks * np.float32(2.0 ** -half)
    g = np.random.default_rng(101)
    q = g.uniform(-1, 1, (n, 4, 64))
    q[:, :, 7] = 1.5                                           # the row's largest: 1.5 2^power
    q = oracle.encode(q * 2.0 ** power, "bf16")
    hq, scale = oracle.decode(q, "bf16"), 0.125 * 2.0 ** (half - power)
    out, lse = lb.attention(dev_bits(q, "bf16"), P.cache(lb), _i32(P.table), _i32([0, n]), _i32([150]), n, 150,
                            scale=scale, return_lse=True)
    k, v = (od.cache_rows(*a, 0, 150) for a in ((P.k, P.ks, P.table[0], "k"), (P.v, P.vs, P.table[0], "v")))
    vs = P.vs[P.table[0][np.arange(150) // 32]].astype(np.float64)
    want, we, mag, peak = od.attention(hq, k, v, vs, 150 - n, scale, True, 0)
    O = to_host64(out)
    bound = 2.0 ** -10 * mag + 2.0 ** -25 * peak + _half_ulp(np.maximum(np.abs(want), np.abs(O)), out.dtype)
    assert (np.abs(O - want) <= bound).all()
    assert (np.abs(to_host64(lse) - we) <= 2.0 ** -14 + 2.0 ** -22 * np.abs(we)).all()


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("power", [-64, -30, 0, 30, 40])
def test_attention_all_zero_blocks_keep_their_weight(lb, n, power):
    """Equal scores over one block of values and one whose scale is 0: the mean of
    all 32 tokens, whatever the other block's scale. Probabilities are equal powers
    of two or their neighbours: 2^-10 sum p |v| / sum p and half an output ulp."""
    banner(f"attention, zero block beside scale 2^{power}, {n} queries")
    P = Paged([32], 1, 16, 64, seed=96)
    P.k[:] = 128
    a, b = P.table[0]
    P.vs[a], P.vs[b] = 2.0 ** power, 0
    P.v[b] = 128
    q, _ = _values(np.random.default_rng(97), (n, 1, 64), "bf16")
    out, lse = lb.attention(q, P.cache(lb), _i32(P.table), _i32([0, n]), _i32([32]), n, 32, causal=False,
                            return_lse=True)
    v = od.block_codes(P.v[a, 0], "v", 16, 64) * 2.0 ** power
    want = np.broadcast_to(v.sum(0) / 32, (n, 1, 64))
    O = to_host64(out)
    bound = 2.0 ** -10 * np.abs(v).sum(0) / 32 + _half_ulp(np.maximum(np.abs(want), np.abs(O)), out.dtype)
    assert (np.abs(O - want) <= bound).all()
    assert (np.abs(to_host64(lse) - np.log(32)) <= 2.0 ** -14).all()


@pytest.mark.parametrize("n", [1, 100])
def test_attention_value_scales_a_hundred_powers_apart(lb, n):
    """Equal scores over blocks of scale 2^-60 and 2^40: each token has 1/32 of the sum."""
    banner(f"attention, value scales 2^100 apart, {n} queries")
    P = Paged([32], 1, 16, 64, seed=98)
    P.k[:] = 128
    a, b = P.table[0]
    P.vs[a], P.vs[b] = 2.0 ** 40, 2.0 ** -60
    q, _ = _values(np.random.default_rng(99), (n, 1, 64), "bf16")
    out, lse = lb.attention(q, P.cache(lb), _i32(P.table), _i32([0, n]), _i32([32]), n, 32, causal=False,
                            return_lse=True)
    v = od.block_codes(P.v[a, 0], "v", 16, 64) * 2.0 ** 40
    O = to_host64(out)
    want = np.broadcast_to(v.sum(0) / 32, (n, 1, 64))
    bound = 2.0 ** -10 * (np.abs(v).sum(0) + 1) / 32 + _half_ulp(np.maximum(np.abs(want), np.abs(O)), out.dtype)
    assert (np.abs(O - want) <= bound).all()
    assert (np.abs(to_host64(lse) - np.log(32)) <= 2.0 ** -14).all()


def test_attention_workspaces(lb):
    """A given workspace of just the bytes needed works; a strided or expanded one that
    counts as many elements, and a smaller one, are refused."""
    banner("attention workspaces")
    P, n, L = Paged([3000], 1, 16, 64, seed=102), 2, 3000
    q, _ = _values(np.random.default_rng(103), (n, 2, 64), "f16")
    need = lb.lib().lowbit_attention_workspace_bytes(1, n, n, L, 2, 1, 64, 0)
    assert need
    call = lambda ws: lb.attention(q, P.cache(lb), _i32(P.table), _i32([0, n]), _i32([L]), n, L, workspace=ws)  # noqa: E731
    assert torch.equal(call(torch.empty(need, dtype=torch.uint8, device="cuda")), call(None))
    one = torch.empty(1, dtype=torch.uint8, device="cuda")
    for ws in (one.expand(need), torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2], one):
        with pytest.raises(ValueError, match="workspace"):
            call(ws)


@pytest.mark.parametrize("n,H,Hq", [(1, 2, 4), (100, 1, 2)])
@pytest.mark.parametrize("L", [200, 3000])
def test_attention_leaves_rows_of_no_sequence_alone(lb, n, H, Hq, L):
    """Rows before and behind those that cu_tokens covers (a batch padded to a fixed
    size) stay as they are, whether or not the context is split; a split's workspace
    holds NaN beforehand."""
    banner(f"attention, padded batch, {n} queries over {L}")
    P = Paged([L], H, 16, 64, seed=104)
    T = n + 12
    q, _ = _values(np.random.default_rng(105), (T, Hq, 64), "bf16")
    need = lb.lib().lowbit_attention_workspace_bytes(1, T, n, L, Hq, H, 64, 0)
    assert (need > 0) == (L > 2000)
    out = torch.full((T, Hq, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((max(1, need // 4),), float("nan"), device="cuda")
    cache, table, lens = P.cache(lb), _i32(P.table), _i32([L])
    lb.attention(q, cache, table, _i32([5, 5 + n]), lens, n, L, out=out, workspace=ws)
    want = lb.attention(q[5:5 + n], cache, table, _i32([0, n]), lens, n, L)
    assert (out[:5] == 7).all() and (out[5 + n:] == 7).all()
    assert torch.isfinite(want).all() and torch.allclose(out[5:5 + n].float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -7)


def test_attention_joins_more_rows_than_one_grid_dimension_holds(lb):
    """65535 sequences of 260 heads, 17 million rows (a launch's first dimension holds
    2^24 workgroups of 256 threads), split by a bound of 5000 tokens: all see the same
    three tokens and ask the same."""
    banner("attention: 17 million rows in two parts")
    B, H, Hq, D = 65535, 4, 260, 64
    P = Paged([3], H, 16, D, seed=106)
    cache, one = P.cache(lb), _values(np.random.default_rng(107), (1, Hq, D), "f16")[0]
    want = lb.attention(one, cache, _i32(P.table), _i32([0, 1]), _i32([3]), 1, 3)
    table = _i32(P.table).expand(B, 1).contiguous()
    assert lb.lib().lowbit_attention_workspace_bytes(B, B, 1, 5000, Hq, H, D, 0) == 2 * B * Hq * (D + 2) * 4
    out = lb.attention(one.expand(B, Hq, D), cache, table, torch.arange(B + 1, dtype=torch.int32, device="cuda"),
                       torch.full((B,), 3, dtype=torch.int32, device="cuda"), 1, 5000)
    assert torch.equal(out, want.expand(B, Hq, D))


@pytest.mark.parametrize("new", [[1, 1], [50, 70]])
def test_head_major_operands_give_the_same_bits(lb, new):
    """Every dense operand as [heads, tokens, head_dim] in memory, queries, keys and
    values in one block, against the token-major layout."""
    banner(f"head-major operands, {new} new tokens")
    H, Hq, D, page, past = 2, 6, 128, 32, [37, 100]
    lens = [p + n for p, n in zip(past, new)]
    P, T = Paged(lens, H, page, D, seed=108), sum(new)
    x, _ = _values(np.random.default_rng(109), (T, Hq + 2 * H, D), "bf16")
    cos, sin = (torch.from_numpy(a).cuda() for a in _rope(max(lens), D))
    at = (_i32(P.table), _i32([0, new[0], T]))
    res = []
    for swap in (False, True):
        order = (lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)) if swap else (lambda t: t)
        y, cache = order(x), P.cache(lb)
        out = [order(torch.full((T, h, D), 7.0, dtype=x.dtype, device="cuda")) for h in (Hq, Hq, H, H)]
        q = lb.kv_append(y[:, Hq:Hq + H], y[:, Hq + H:], cache, *at, _i32(past), max(new), q=y[:, :Hq], cos=cos, sin=sin,
                         q_out=out[0])
        o = lb.attention(q, cache, *at, _i32(lens), max(new), max(lens), out=out[1])
        k, v = lb.kv_read(cache, *at, _i32(past), T, max(new), out=(out[2], out[3]))
        assert q is out[0] and o is out[1] and q.is_contiguous() != swap
        res.append([q, o, k, v, cache.k, cache.v, cache.k_scale, cache.v_scale])
    for a, b in zip(*res):
        assert torch.equal(a, b)


# -------------------------------------- the many-row kernel (over 80 rows a head) ---

def _parts(lb, lens, new, H, Hq, D, window=0):
    """Parts that the call's context is split into (1: no workspace)."""
    T = sum(new)
    need = lb.lib().lowbit_attention_workspace_bytes(len(lens), T, max(new), max(lens), Hq, H, D, window)
    assert need % (T * Hq * (D + 2) * 4) == 0
    return max(1, need // (T * Hq * (D + 2) * 4))


MANY = [  # lens, new, H, Hq, page, D, dtype, causal, window, parts
    ([3000], [100], 1, 1, 16, 128, "bf16", True, 0, 2),
    ([3000, 1100], [100, 90], 1, 1, 64, 64, "f16", True, 0, 2),       # the second part of a shorter sequence is empty
    ([6000], [100], 1, 2, 64, 64, "f16", True, 3000, 3),
    ([4500], [100], 1, 1, 16, 256, "f16", False, 0, 4),
    ([4500], [45], 1, 2, 128, 256, "bf16", True, 0, 4),
    ([2200], [2200], 1, 1, 32, 64, "bf16", True, 0, 2),               # later parts that early rows do not see
    ([2100, 40], [30, 40], 1, 3, 16, 128, "f16", True, 0, 2),
    ([2500], [90], 1, 1, 16, 128, "bf16", False, 2300, 2),
    ([200], [100], 1, 1, 16, 64, "f16", True, 10, 1),                 # windows of part of a tile
    ([200], [100], 1, 1, 32, 128, "bf16", True, 3, 1),
    ([200], [100], 1, 2, 16, 256, "bf16", True, 1, 1),
    ([300], [90], 1, 1, 256, 128, "f16", False, 20, 1),
    ([60], [100], 1, 2, 16, 64, "bf16", True, 0, 1),                  # queries before the first token
    ([0, 70], [90, 70], 1, 2, 16, 128, "f16", True, 0, 1),            # nothing cached
]


@pytest.mark.parametrize("case", MANY, ids=[str(i) for i in range(len(MANY))])
def test_attention_many_rows(lb, case):
    lens, new, H, Hq, page, D, dt, causal, window, parts = case
    banner(f"attention, many rows {case}")
    assert max(new) * (Hq // H) > 80 and _parts(lb, lens, new, H, Hq, D, window) == parts
    _attend(lb, lens, new, H, Hq, page, D, dt, seed=200 + len(lens) + D, causal=causal, window=window, strided=(D == 128))


@pytest.mark.parametrize("lens,page", [((200, 100), 16), ((2500, 1200), 64)])
def test_attention_many_rows_missing_pages_and_short_tables(lb, lens, page):
    banner(f"attention, many rows with holes, {lens}")
    lens, new = list(lens), [90, 90]
    assert _parts(lb, lens, new, 2, 4, 128) == (2 if lens[0] > 2000 else 1)
    _attend(lb, lens, new, 2, 4, page, 128, "bf16", seed=220, hole=(0, 3, -1))
    _attend(lb, lens, new, 2, 4, page, 128, "bf16", seed=221, hole=(1, 0, 10 ** 6))
    # a table shorter than the lengths: they count as what it holds
    _attend(lb, lens, new, 2, 4, page, 128, "bf16", seed=223, width=lens[0] // page - 3)
    P = Paged(lens, 2, page, 128, seed=224)                    # every page missing: zeros
    P.table[:] = -1
    assert (_attend(lb, lens, new, 2, 4, page, 128, "f16", kv=P) == 0).all()


@pytest.mark.parametrize("lens,page", [((170, 133), 16), ((2500, 2133), 64)])
def test_attention_many_rows_masked_tokens_hold_anything(lb, lens, page):
    """As for few rows, one part and two: codes behind the length, scales of pages
    that are not used and entries of the table behind the last page do not matter,
    nor does what a missing page's stand-in (page 0) holds."""
    banner(f"attention, many rows, garbage, {lens}")
    n, H, D = 90, 1, 64
    P = Paged(list(lens), H, page, D, seed=230, spare=6)
    P.table[P.table == 0] = min(set(range(1, P.pages)) - set(P.table.ravel()))   # page 0 is nobody's
    P.table[0, 1] = -1
    q = torch.randn((2 * n, 2, D), device="cuda").half()
    call = lambda: lb.attention(q, P.cache(lb), _i32(P.table), _i32([0, n, 2 * n]), _i32(list(lens)), n, max(lens))  # noqa: E731
    clean = call()
    used = [set(P.table[b, :-(-lens[b] // page)]) for b in range(2)]
    for p in range(P.pages):
        if p not in used[0] | used[1]:
            P.ks[p], P.vs[p], P.k[p], P.v[p] = np.nan, np.nan, 255, 0
    P.table[1, -(-lens[1] // page):] = -5
    d = np.arange(D)
    for b in range(2):
        last = P.table[b, (lens[b] - 1) // page]
        for t in range(lens[b] % page, page):
            P.k[last, 0].reshape(-1)[od.k_place(t, d, D)] = 255
            P.v[last, 0].reshape(-1)[od.v_place(t, d, D)] = 0
    again = call()
    assert torch.isfinite(clean).all() and torch.equal(again, clean)


def test_attention_many_rows_several_segments_of_pages(lb):
    """Four waves a workgroup over more pages than one segment holds (4096 tokens in
    pages of 16), the context in one part: sampled rows against float64."""
    banner("attention: 530 queries of 64 heads of 64 over 5000 tokens")
    H, Hq, D, page, L, n = 8, 64, 64, 16, 5000, 530
    assert _parts(lb, [L], [n], H, Hq, D) == 1
    P = Paged([L], H, page, D, seed=240)
    cache, table = P.cache(lb), _i32(P.table)
    q, hq = _values(np.random.default_rng(241), (n, Hq, D), "f16")
    out = lb.attention(q, cache, table, _i32([0, n]), _i32([L]), n, L)
    k, v = (t.double().cpu().numpy() for t in lb.kv_read(cache, table, _i32([0, L]), _i32([0]), L, L, torch.float32))
    vs = P.vs[P.table[0][np.arange(L) // page]].astype(np.float64)
    O = to_host64(out)
    for i in (0, 15, 16, 31, 300, 528, 529):
        for h in (0, 8, 33, 63):
            kv = h // (Hq // H)
            want, _, mag, peak = od.attention(hq[i:i + 1, h:h + 1], k[:, kv:kv + 1], v[:, kv:kv + 1], vs[:, kv:kv + 1],
                                              L - n + i, D ** -0.5, True, 0)
            bound = 2.0 ** -10 * mag + 2.0 ** -25 * peak + _half_ulp(np.maximum(np.abs(want), np.abs(O[i, h])), out.dtype)
            assert (np.abs(O[i, h] - want) <= bound).all(), (i, h)


def test_gemv_int4_and_gemm_int4_agree(lb):
    """The two entry points on the same operands differ by no more than both
    contracts' bounds together (the larger kernel's adds 2^-19 (128 + max|z|) sum|x s|
    where this one has 16)."""
    banner("gemv int4 against gemm int4")
    for M, dt in ((1, "bf16"), (7, "f16"), (16, "bf16")):
        lin = wl.make_int4_linear(f"gv_gm_{M}", M, 3000, 2560, dt, seed=250 + M, with_bias=True)
        y = to_host64(_gemv_check(lb, lin))
        q = lb.pack_int4(torch.from_numpy(np.ascontiguousarray(lin.q)).cuda())
        z = to_host64(lb.gemm_int4(dev_bits(lin.x, dt), q, _f16(lin.scales), _f16(lin.zeros), bias=_f16(lin.bias),
                                   out_dtype=TORCH_DT[lin.y_dtype]))
        A = oracle.linear_int4(lin.x, dt, lin.q, lin.scales, lin.zeros, lin.bias)
        Mg = oracle.magnitude_int4(lin.x, dt, lin.q, lin.scales, lin.zeros, lin.bias)
        s = np.repeat(np.abs(lin.scales.astype(np.float64)), oracle.GROUP, axis=1)
        terms = np.abs(oracle.decode(lin.x, dt)) @ s.T
        zmax = np.abs(lin.zeros.astype(np.float64)).max(axis=1)[None, :]
        bound = (oracle.bound(A, Mg, lin.y_dtype, y) + oracle.bound(A, Mg, lin.y_dtype, z)
                 + 2.0 ** -19 * (144.0 + 2 * zmax) * terms)
        assert (np.abs(y - z) <= bound).all()
