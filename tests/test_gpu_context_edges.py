"""The operators of long contexts where the cases of test_gpu_context.py do not
reach, against the float64 definitions of oracle/paged.py with the tolerances
derived there."""
import numpy as np
import pytest
import torch

from oracle import paged as od
from gpu_util import banner, to_host64
from test_gpu_decode import _i32, _values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import bit_weight_gemm_int2_amd as b
    b.lib()
    return b


# ------------------------------------------------- attention by the shape of its plan ---

class Long:
    """Sequences in a cache made on the GPU, with pages in no order."""

    def __init__(self, lb, lens, H, page, D, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.page, self.D = lens, page, D
        width = -(-max(lens) // page)
        pages = len(lens) * width + 3
        k, v = ((torch.randn((pages, H, page, D), generator=g, device="cuda") * 36).round_().clamp_(-127, 127).add_(128)
                .to(torch.uint8) for _ in range(2))
        ks, vs = ((0.5 + torch.rand((pages, H), generator=g, device="cuda")) * (3.5 / 127) for _ in range(2))
        self.cache = lb.KVCache(k, v, ks, vs)
        self.table = torch.randperm(pages, generator=g, device="cuda")[:len(lens) * width].to(torch.int32).view(len(lens), width)

    def rows(self, lb, b):
        """Keys and values [L, H, D] and value scales [L, H] of sequence b, float64."""
        L = self.lens[b]
        k, v = lb.kv_read(self.cache, self.table[b:b + 1].contiguous(), _i32([0, L]), _i32([0]), L, L, torch.float32)
        vs = self.cache.v_scale[self.table[b].long()[torch.arange(L, device="cuda") // self.page]]
        return k.double(), v.double(), vs.double()


def _half(y, dtype):
    """Half a unit in the last place of y."""
    bits, low = (8, -133) if dtype == torch.bfloat16 else (11, -24)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -140)))
    return 0.5 * torch.exp2((e - bits + 1).clamp(min=low))


def _check(lb, P, q, out, lse, cu, causal, window, sinks):
    """Every row against float64 on the GPU: 2^-10 sum p |v| / sum p + 2^-25 tokens 127 max(p v_scale) / sum p + half an
    output ulp, and the log of the sum within 2^-14 + 2^-22 of itself."""
    H, group = P.cache.kv_heads, q.shape[1] // P.cache.kv_heads
    for b in range(len(P.lens)):
        L, n = P.lens[b], cu[b + 1] - cu[b]
        if not n or not L:
            assert (out[cu[b]:cu[b + 1]] == 0).all() and torch.isneginf(lse[cu[b]:cu[b + 1]]).all()
            continue
        k, v, vs = P.rows(lb, b)
        pos = L - n + torch.arange(n, device="cuda").repeat_interleave(group)[:, None]
        j = torch.arange(L, device="cuda")[None]
        seen = (j <= pos) if causal else (j >= 0).expand(n * group, L)
        if window:
            seen = seen & ((j > pos - window) | (j < sinks))
        for h in range(H):
            rows = (slice(cu[b], cu[b + 1]), slice(h * group, (h + 1) * group))
            s = q[rows].double().reshape(-1, P.D) @ k[:, h].t().contiguous() * P.D ** -0.5
            s.masked_fill_(~seen, -torch.inf)
            top = s.amax(-1, keepdim=True)
            e = torch.exp(s - torch.where(top > -torch.inf, top, 0.0))
            total = e.sum(-1, keepdim=True)
            safe = torch.where(total > 0, total, 1.0)
            want, mag = (e @ v[:, h].contiguous()) / safe, (e @ v[:, h].abs().contiguous()) / safe
            peak = 127 * seen.sum(-1, keepdim=True) * (e * vs[:, h]).amax(-1, keepdim=True) / safe
            got = out[rows].double().reshape(-1, P.D)
            bound = 2.0 ** -10 * mag + 2.0 ** -25 * peak + _half(torch.maximum(want.abs(), got.abs()), out.dtype)
            assert ((got - want).abs() <= bound).all(), (b, h, ((got - want).abs() / bound.clamp(min=1e-30)).max().item())
            want, got = (top + torch.log(total)).flatten(), lse[rows].double().flatten()
            none = total.flatten() == 0
            assert torch.isneginf(got[none]).all()
            assert ((got - want).abs()[~none] <= 2.0 ** -14 + 2.0 ** -22 * want.abs()[~none]).all()


PLANS = [  # lens, new, H, Hq, page, D, dtype, window, sinks, (rows of a tile, parts, join), more tokens a part than a segment of pages holds
    # 256-row tiles over several segments
    ([12000], [1900], 8, 64, 16, 128, "bf16", 8300, 50, (256, 1, 0), True),
    ([9000, 7777], [2048, 1000], 8, 64, 32, 128, "f16", 5000, 333, (256, 1, 0), False),
    # 128-row tiles over two segments, the first with the gap
    ([6200], [130], 8, 512, 16, 64, "bf16", 4500, 100, (128, 1, 0), True),
    # 16-row tiles in parts: several tiles a sequence and head, and heads of 256
    ([4000 - 300 * i for i in range(8)], [16] * 8, 1, 5, 16, 128, "bf16", 2500, 20, (16, 6, 1), False),
    ([5000, 3100, 40], [10, 9, 10], 1, 8, 64, 64, "f16", 3000, 33, (16, 13, 2), False),
    ([3000, 1900], [80, 41], 1, 1, 16, 256, "f16", 2000, 40, (16, 9, 2), False),
    ([8000 - 200 * i for i in range(24)], [1] * 24, 4, 16, 32, 256, "bf16", 4000, 4, (16, 8, 2), False),
    ([9000, 6100, 6000, 100, 5], [1] * 5, 1, 2, 16, 256, "f16", 6000, 100, (16, 24, 2), False),
]


@pytest.mark.parametrize("case", PLANS, ids=[str(i) for i in range(len(PLANS))])
def test_attention_sinks_by_plan(lb, case):
    """Shapes that are planned as stated (on 256 CUs), each row against float64."""
    lens, new, H, Hq, page, D, dt, window, sinks, plan, segments = case
    banner(f"attention with first tokens as planned {case}")
    T, cu = sum(new), [0, *np.cumsum(new).tolist()]
    got = lb.attention_plan(len(lens), T, max(new), max(lens), Hq, H, D, True, window, sinks)
    assert (got.tile, got.parts, got.join) == plan
    assert (got.part_tokens > 256 * page) == segments          # of pages that the LDS holds at a time
    P = Long(lb, lens, H, page, D, seed=D + page)
    q = 6 * _values(np.random.default_rng(T), (T, Hq, D), dt)[0]    # a few tokens rule each row: one too many or too few shows
    out, lse = lb.attention(q, P.cache, P.table, _i32(cu), _i32(lens), max(new), max(lens), window=window, sinks=sinks,
                            return_lse=True)
    _check(lb, P, q, out, lse, cu, True, window, sinks)


JOINS = [  # lens, new, H, Hq, D, window, sinks, parts
    ([2500], [90], 1, 1, 64, 0, 0, 2),
    ([9000], [90], 1, 1, 64, 0, 0, 8),
    ([3000], [90], 1, 2, 64, 2500, 30, 5),
    ([3400], [90], 1, 1, 128, 0, 0, 3),
    ([7800], [90], 1, 1, 128, 0, 0, 7),
    ([3000], [90], 1, 2, 128, 2500, 30, 5),
    ([2500], [90], 1, 1, 256, 0, 0, 2),
    ([4500], [90], 1, 1, 256, 0, 0, 4),
    ([1400, 1000, 900, 10, 0, 600, 904, 1399], [1] * 8, 1, 4, 256, 900, 4, 4),
]


@pytest.mark.parametrize("case", JOINS, ids=[str(i) for i in range(len(JOINS))])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_the_two_joins_give_the_same_bits(lb, case, dt):
    """The same queries in a batch of fewer than 512 rows, whose parts one workgroup a row
    joins, and padded to more with rows of no sequence, where groups of threads do."""
    lens, new, H, Hq, D, window, sinks, parts = case
    banner(f"the two joins of {parts} parts, heads of {D}, {case} {dt}")
    T, B, most, longest = sum(new), len(lens), max(new), max(lens)
    more = T + 600 // Hq
    a, b = (lb.attention_plan(B, t, most, longest, Hq, H, D, True, window, sinks) for t in (T, more))
    assert a[:3] == b[:3] and a.parts == parts and (a.join, b.join) == (2, 1) and T * Hq < 512 <= more * Hq
    P, cu = Long(lb, lens, H, 16, D, seed=parts), [0, *np.cumsum(new).tolist()]
    q, _ = _values(np.random.default_rng(D + parts), (more, Hq, D), dt)
    call = lambda x: lb.attention(x, P.cache, P.table, _i32(cu), _i32(lens), most, longest, window=window, sinks=sinks,  # noqa: E731
                                  return_lse=True)
    (out, lse), (wide, wide_lse) = call(q[:T].contiguous()), call(q)
    assert torch.equal(out, wide[:T]) and torch.equal(lse, wide_lse[:T])
    _check(lb, P, q, out, lse, cu, True, window, sinks)


def test_the_join_by_rows_of_heads_of_256(lb):
    """Parts of two ragged sequences, joined by rows; the second one's later parts hold nothing."""
    lens, new, window, sinks = [2500, 20], [300, 20], 1500, 50
    banner("join by rows, heads of 256")
    assert lb.attention_plan(2, 320, 300, 2500, 2, 1, 256, True, window, sinks)[1:] == (3, 640, 1)
    P, cu = Long(lb, lens, 1, 16, 256, seed=21), [0, 300, 320]
    for dt in ("bf16", "f16"):
        q, _ = _values(np.random.default_rng(22), (320, 2, 256), dt)
        out, lse = lb.attention(q, P.cache, P.table, _i32(cu), _i32(lens), 300, 2500, window=window, sinks=sinks, return_lse=True)
        _check(lb, P, q, out, lse, cu, True, window, sinks)


BIG = [  # rows of the batch, queries, length, (parts, join): more than a launch's first dimension holds
    (2 ** 22 + 100, 60, 1500, (6, 2)),        # more parts than the join by rows takes: both dimensions of the other one
    (2 ** 24 + 100, 100, 2500, (2, 2)),       # more rows than the join by rows takes
]


@pytest.mark.parametrize("rows,n,L,plan", BIG, ids=["parts", "rows"])
def test_joins_of_more_rows_than_one_grid_dimension_holds(lb, rows, n, L, plan):
    """One sequence's queries at the end of a batch of rows of no sequence (which stay as they
    are): the same bits as without them."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB of free GPU memory")
    banner(f"join of {rows} rows of 256 in {plan[0]} parts")
    P = Long(lb, [L], 1, 16, 256, seed=31)
    assert lb.attention_plan(1, rows, n, L, 1, 1, 256)[1::2] == plan
    x, _ = _values(np.random.default_rng(32), (n, 1, 256), "bf16")
    q = torch.zeros((rows, 1, 256), dtype=torch.bfloat16, device="cuda")
    q[-n:] = x
    out = torch.full((rows, 1, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    lb.attention(q, P.cache, P.table, _i32([rows - n, rows]), _i32([L]), n, L, out=out)
    want, lse = lb.attention(x, P.cache, P.table, _i32([0, n]), _i32([L]), n, L, return_lse=True)
    assert torch.equal(out[-n:], want) and (out[:-n] == 7.0).all()
    _check(lb, P, x, want, lse, [0, n], True, 0, 0)
    del q, out
    torch.cuda.empty_cache()


# ------------------------------------------------- norms at the end of the range ---

HUGE = [  # |x|, weights of the halves, cos, sin: with a subnormal factor 1 / |x| 1.017 to 1.019 of the bound
    ("0x1.fdb0c6p+127", "0x1.c17d86p-1", "0x1.c0298cp-1", "0x1.6e638ap-1", "0x1.65a2b6p-1"),
    ("0x1.f38c3ep+127", "0x1.c04a9ap-1", "0x1.c0128cp-1", "0x1.5a3918p-1", "0x1.793118p-1"),
    ("0x1.fd171ap+127", "0x1.c0f11ep-1", "0x1.c03890p-1", "0x1.5c5f1ep-1", "0x1.773518p-1"),
]


@pytest.mark.parametrize("case", HUGE, ids=["0", "1", "2"])
@pytest.mark.parametrize("way", ["dense", "append"])
def test_norm_and_rotation_of_rows_beyond_2_to_126(lb, case, way):
    """Rows whose root mean square has a subnormal FP32 inverse, of 22 bits: rotated, they
    too are within 2^-21 of the row's largest normalised value (the rows here are the ones
    that a model of the FP32 steps found farthest off with such an inverse)."""
    banner(f"norm and rotation of huge rows, {way}, {case}")
    x, w0, w1, c, s = (np.float32(float.fromhex(v)) for v in case)
    D, half = 64, 32
    rows = np.concatenate([np.full(half, x), np.full(half, -x)]).astype(np.float32)
    w = np.concatenate([np.full(half, w0), np.full(half, w1)]).astype(np.float32)
    cos, sin = (np.full((1, half), v, dtype=np.float32) for v in (c, s))
    q, wt, ct, st = (torch.from_numpy(a).cuda() for a in (rows.reshape(1, 1, D), w, cos, sin))
    if way == "dense":
        got = lb.norm_rotate(q, q_norm=wt, cos=ct, sin=st, eps=0.0)
    else:
        zero = torch.zeros((1, 1, D), device="cuda")
        got = lb.kv_append(zero, zero, lb.new_kv_cache(1, 1, 16, D), _i32([[0]]), _i32([0, 1]), _i32([0]), 1, q=q, cos=ct, sin=st,
                           q_norm=wt, eps=0.0)
    n = od.norm(rows.reshape(1, 1, D), w.astype(np.float64), 0.0)
    want = od.rotate(n, np.zeros(1, dtype=int), cos, sin, False)
    assert (np.abs(to_host64(got) - want) <= 2.0 ** -21 * np.abs(n).max()).all()


# -------------------------------------------------------------------------- pages ---

@pytest.mark.parametrize("stream", [False, True])
def test_kept_page_plans_hold_their_results_only(lb, stream):
    """A table is kept as long as its sequences live: its memory does not grow with the pool
    (the workspace takes 8 bytes a page, 0.8 MB here)."""
    banner(f"memory of a page plan, stream {stream}")
    cache = lb.new_kv_cache(100000, 1, 16, 64)
    table = _i32(np.arange(12).reshape(3, 4))
    s = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    for compact in (False, True):
        plan = lb.kv_remap(table, _i32([64, 30, 50]), cache, rows=_i32([0, 0, 2, 1]), room=_i32([1, 1, 1, 1]), width=5, compact=compact,
                           stream=s)
        torch.cuda.synchronize()
        assert plan.counts.tolist() == [0, 12, 0, 0] and plan.table[0].tolist() == [0, 1, 2, 3, 6] and plan.table[1, 4] == 7
        words = sum(t.numel() for t in plan)
        assert all(t.untyped_storage().nbytes() <= 4 * words for t in plan)


# ------------------------------------------------------------------ the example ---

def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "text_decode.py")
    spec = importlib.util.spec_from_file_location("text_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_says_when_its_pool_runs_out(lb):
    """Two prompts of 20 tokens and 14 more in pages of 16 need six pages, in two answers
    each ten (the prompts' first pages are shared): enough pages pass, fewer raise, and the
    model goes on with shorter sequences after that."""
    banner("example: a pool with too few pages")
    m = _example()
    prompts = [list(range(20)), list(range(5, 25))]
    for pages, answers, ok in ((6, 1, True), (5, 1, False), (10, 2, True), (6, 2, False)):
        model = m.Model(1, 128, 2, 1, 64, 128, 64, 16, pages, 48)
        if ok:
            seqs, _, _ = m.generate(model, prompts, 15, 3, answers)
            assert [len(s) for s in seqs] == [35] * (2 * answers)
        else:
            with pytest.raises(RuntimeError, match="ran out of pages"):
                m.generate(model, prompts, 15, 3, answers)
            assert len(m.generate(model, [prompts[0][:3]], 2, 3)[0]) == 1
