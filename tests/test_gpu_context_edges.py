"""The operators of long contexts where the cases of test_gpu_context.py do not
reach, against the float64 definitions of oracle/paged.py with the tolerances
derived there."""
import numpy as np
import pytest
import torch

from oracle import paged as od
from gpu_util import banner, to_host64
from test_gpu_decode import _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lb():
    import bit_weight_gemm_int2_amd as b
    b.lib()
    return b


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
