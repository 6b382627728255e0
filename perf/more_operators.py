"""Cases that measure the operators of long contexts: attention with a sliding window and first tokens that stay
visible, norms of queries and keys for each head with the rotation by position (on the way into the 8-bit paged cache,
and dense), tables of rotary positions scaled for long contexts, and the pages of the cache (forking, freeing,
compacting, copying).

The shapes are those of the 4-bit text encoder that this repository already benchmarks (32 query and 8 key/value heads
of 128), of the 4608 tokens of its image step, and generic ones around them."""
import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1.0e-6


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one token of one conversation that has outgrown its window: latency
        dict(name="attend 1 x 1000+4", op="attend", B=1, new=1, ctx=30000, Hq=32, H=8, D=128, page=64, window=1000,
             sinks=4, x="bf16"),
        # one token of each of 48 ragged conversations, small pages
        dict(name="attend 48 x 4096+20", op="attend", B=48, new=1, ctx=16000, Hq=40, H=8, D=128, page=16, window=4096,
             sinks=20, x="f16"),
        # a chunk of a long prompt, every query with its own window
        dict(name="attend chunk 4096, 2500+70", op="attend", B=1, new=4096, ctx=20000, Hq=32, H=8, D=128, page=128,
             window=2500, sinks=70, x="bf16"),
        # one token of one sequence into the cache: the smallest append
        dict(name="append 1 token", op="append", B=1, new=1, past=300, Hq=32, H=8, D=128, page=64, rot=128, inter=False,
             x="bf16", w="bf16"),
        # ragged prompts that start inside a page, part of each head rotated
        dict(name="append prompts 6x2500", op="append", B=6, new=2500, past=777, Hq=32, H=8, D=128, page=64, rot=64,
             inter=False, x="bf16", w="f32"),
        # the queries and keys of sixteen drafted tokens at positions of their own
        dict(name="turn 16 x 32+8", op="turn", T=16, Hq=32, H=8, D=128, rot=128, inter=False, rows=9000, x="f16", w="f16"),
        # the image and text tokens of one block of an image step, a table row a token
        dict(name="turn 4608 x 24+24", op="turn", T=4608, Hq=24, H=24, D=128, rot=128, inter=True, rows=0, x="bf16",
             w="bf16"),
        # tables of a short context, frequencies divided by bands
        dict(name="tables 1000 x 64", op="tables", n=1000, rot=64, base=5.0e5, kind="wavelength", factor=8.0,
             original=8192, low=1.0, high=4.0, first=100000),
        # tables of a long one, as serving makes them once for all layers
        dict(name="tables 131072 x 128", op="tables", n=131072, rot=128, base=1.0e6, kind="yarn", factor=4.0,
             original=32768, low=1.0, high=32.0, first=0),
        # four answers to one prompt
        dict(name="pages fork 1 to 4", op="pages", B=1, R=4, ctx=1000, shared=0, pool=400, H=8, D=128, page=64, room=1,
             window=0, sinks=0, compact=False),
        # a step of a beam search over 64 rows with common prefixes, in small pages, old ones out of the window
        dict(name="pages beams 64", op="pages", B=64, R=64, ctx=5000, shared=1500, pool=20000, H=4, D=64, page=16, room=3,
             window=3500, sinks=8, compact=False),
        # a third of 300 sequences have ended: the others' pages move to the front of the pool
        dict(name="pages compact 200 of 300", op="pages", B=300, R=200, ctx=2500, shared=0, pool=9000, H=8, D=128, page=64,
             room=64, window=0, sinks=0, compact=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "turn", "tables", "pages"])
    x = rng.choice(["bf16", "f16"])
    H, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    Hq = H * rng.choice([1, 2, 3, 4, 5, 8])
    rot = rng.choice([D, D, D // 2])
    if op == "attend":
        while True:
            prompt = rng.random() < 0.4
            B = _log(rng, 1, 4 if prompt else 48)
            new = _log(rng, 17, 4096) if prompt else rng.choice([1, 1, 1, 2, 5])
            window, sinks = _log(rng, 30, 8000), rng.choice([1, 4, 16, 17, 64, 200])
            ctx = max(new, _log(rng, window, 30000))
            pairs = float(B) * new * min(ctx, window + sinks)
            if 4.0 * pairs * Hq * D < 1.6e11 and 4.0 * B * ctx * max(2 * H * D, 2 * Hq * new) < 1.0e10:
                break
        return dict(op=op, B=B, new=new, ctx=ctx, Hq=Hq, H=H, D=D, page=page, window=window, sinks=sinks, x=x)
    if op == "append":
        many = rng.random() < 0.5
        return dict(op=op, B=_log(rng, 1, 6 if many else 64), new=_log(rng, 2, 2500) if many else 1, past=_log(rng, 1, 4000),
                    Hq=min(Hq, 32), H=H, D=min(D, 128), page=page, rot=min(rot, 128), inter=rng.random() < 0.4, x=x,
                    w=rng.choice([x, "f32"]))
    if op == "turn":
        x = rng.choice(["bf16", "f16", "f32"])
        return dict(op=op, T=_log(rng, 1, 4608), Hq=min(Hq, 24), H=H, D=min(D, 128), rot=rng.choice([min(rot, 128), 32]),
                    inter=rng.random() < 0.5, rows=rng.choice([0, 5000]), x=x, w=rng.choice([x, "f32"]))
    if op == "tables":
        kind = rng.choice(["none", "linear", "ntk", "yarn", "wavelength"])
        rot = rng.choice([32, 64, 96, 128])
        return dict(op=op, n=_log(rng, 100, 131072), rot=rot, base=rng.choice([1.0e4, 5.0e5, 1.0e6]), kind=kind,
                    factor=1.0 if kind == "none" else rng.choice([2.0, 4.0, 10.5]), original=rng.choice([4096, 8192, 32768]),
                    low=1.0, high=rng.choice([4.0, 32.0]), first=rng.choice([0, 0, 77, 500000]))
    R = _log(rng, 1, 200)
    B = rng.choice([max(1, R // 4), R, R + R // 2])
    ctx = _log(rng, 20, 4000)
    H, D = rng.choice([1, 2, 4]), min(D, 128)
    pool = _log(rng, 1.3, 3) + 1 + B * (ctx // page + 1) + R * 6
    return dict(op=op, B=B, R=R, ctx=ctx, shared=rng.choice([0, ctx // 3]), pool=pool, H=H, D=D, page=page,
                room=rng.choice([0, 1, 5, 70]), window=rng.choice([0, 0, max(1, ctx // 2)]), sinks=rng.choice([0, 4, 100]),
                compact=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs ---

def _lengths(case):
    """Per sequence: (tokens in the cache before, new tokens), ragged, the same for every seed."""
    r = np.random.RandomState(53 + case["B"])
    B, n = case["B"], case.get("new", 0)
    if case["op"] == "attend":
        new = np.full(B, n) if n <= 8 else np.maximum(1, (n * (0.6 + 0.4 * r.rand(B))).astype(int))
        new[0] = n
        total = np.maximum(new, (case["ctx"] * (0.25 + 0.75 * r.rand(B))).astype(int))
        total[0] = case["ctx"]
        past = total - new
    elif case["op"] == "append":
        new = np.full(B, n) if n == 1 else np.maximum(1, (n * (0.5 + 0.5 * r.rand(B))).astype(int))
        new[0] = n
        past = np.maximum(0, (case["past"] * (0.3 + 0.7 * r.rand(B))).astype(int))
        past[0] = case["past"]
    else:
        past = np.maximum(1, (case["ctx"] * (0.3 + 0.7 * r.rand(B))).astype(int))
        past[0] = case["ctx"]
        new = np.zeros(B, dtype=int)
    return past.astype(np.int64), new.astype(np.int64)


def _cache(case, g, pages):
    """A cache that is in use: codes of normal values, scales of blocks of slightly different size."""
    H, page, D = case["H"], case["page"], case["D"]
    k, v = ((torch.randn((pages, H, page, D), generator=g, device="cuda") * 36).round_().clamp_(-127, 127).add_(128)
            .to(torch.uint8) for _ in range(2))
    ks, vs = ((0.5 + torch.rand((pages, H), generator=g, device="cuda")) * (3.5 / 127) for _ in range(2))
    return dict(k_cache=k, v_cache=v, k_scale=ks, v_scale=vs)


def _i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _norm_weight(case, g, D):
    return (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(DT[case["w"]])


def _angles(g, n, half):
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 1.0e6 ** (
        -torch.arange(half, device="cuda", dtype=torch.float64) / half)
    a = a + 6.28 * torch.rand((1, half), generator=g, device="cuda", dtype=torch.float64)
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    op = case["op"]
    if op == "tables":
        # a case's settings are its input; another seed begins at another position
        st["first"] = case["first"] + seed % 1009
        return st
    if op == "turn":
        T, Hq, H, D = case["T"], case["Hq"], case["H"], case["D"]
        # one projection's output holds queries, keys and values of a token side by side
        qkv = (2 * torch.randn((T, Hq + 2 * H, D), generator=g, device="cuda")).to(DT[case["x"]])
        st.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H], q_norm=_norm_weight(case, g, D), k_norm=_norm_weight(case, g, D))
        st["cos"], st["sin"] = _angles(g, case["rows"] or T, case["rot"] // 2)
        st["positions"] = (torch.randint(0, case["rows"], (T,), generator=g, device="cuda").to(torch.int32)
                           if case["rows"] else None)
        return st
    past, new = _lengths(case)
    page, H, D, B = case["page"], case["H"], case["D"], case["B"]
    if op == "pages":
        r = np.random.RandomState(71 + case["R"])
        # every old sequence goes on, or a draw of them where there are more or fewer new ones
        R = case["R"]
        rows = np.sort(r.choice(B, R, replace=False)) if R <= B and not case["shared"] else r.randint(0, B, R)
        room = r.randint(0, case["room"] + 1, R)
        room[0] = case["room"]
        width = int(-(-(past.max() + case["room"]) // page))
        perm = torch.randperm(case["pool"], generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        slots = torch.arange(width, device="cuda")[None, :]
        has = slots < torch.from_numpy(-(-past // page)).cuda()[:, None]
        table[has] = perm[: int(has.sum())]
        if case["shared"]:  # whole pages of a common prefix, those of the first sequence
            common = (slots < case["shared"] // page) & (slots < torch.from_numpy(past // page).cuda()[:, None])
            table = torch.where(common, table[:1], table)
        st.update(_cache(case, g, case["pool"]))
        st.update(table=table, lens=_i32(past), rows=_i32(rows), room=_i32(room))
        return st
    Hq = case["Hq"]
    total = past + new
    width = int(-(-total.max() // page))
    pages = B * width + 3
    st.update(_cache(case, g, pages))
    T = int(new.sum())
    cu = np.concatenate([[0], np.cumsum(new)])
    st.update(table=torch.randperm(pages, generator=g, device="cuda")[: B * width].to(torch.int32).view(B, width),
              cu=_i32(cu), T=T, max_new=int(new.max()), max_len=int(total.max()), total=_i32(total), past=_i32(past))
    # what the plain form indexes with: the sequence and the place of every new token
    seq = np.repeat(np.arange(B), new)
    st["seq"], st["pos"] = (torch.from_numpy(a).cuda() for a in (seq, np.arange(T) - cu[seq] + past[seq]))
    if op == "append":
        qkv = (2 * torch.randn((T, Hq + 2 * H, D), generator=g, device="cuda")).to(DT[case["x"]])
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        st.update(q_norm=_norm_weight(case, g, D), k_norm=_norm_weight(case, g, D))
        st["cos"], st["sin"] = _angles(g, int(total.max()), case["rot"] // 2)
        # the blocks that the append changes are read back from their first token on
        first = past // page * page
        n = total - first
        cur = np.concatenate([[0], np.cumsum(n)])
        s2 = np.repeat(np.arange(B), n)
        st.update(first=_i32(first), cu_read=_i32(cur), T_read=int(n.sum()), max_read=int(n.max()))
        st["seq_read"], st["pos_read"] = (torch.from_numpy(a).cuda() for a in (s2, np.arange(len(s2)) - cur[s2] + first[s2]))
    else:
        st["q"] = (torch.randn((T, Hq, D), generator=g, device="cuda") * 1.5).to(DT[case["x"]])
    return st


# ------------------------------------------------------------- plain forms ---

def _rows(codes, which):
    """The cache's blocks [pages, heads, page, D] as tokens [pages, page, heads, D]: keys are kept in 16-byte pieces
    of 16 tokens each ([page/16][D/16][16][16]), values in quads of tokens ([page/4][D][4])."""
    p, h, t, d = codes.shape
    if which == "k":
        c = codes.view(p, h, t // 16, d // 16, 16, 16).permute(0, 2, 4, 1, 3, 5)
    else:
        c = codes.view(p, h, t // 4, d, 4).permute(0, 2, 4, 1, 3)
    return c.reshape(p, t, h, d)


def _blocks(rows, which):
    """The inverse of _rows."""
    p, t, h, d = rows.shape
    if which == "k":
        c = rows.view(p, t // 16, 16, h, d // 16, 16).permute(0, 3, 1, 4, 2, 5)
    else:
        c = rows.view(p, t // 4, 4, h, d).permute(0, 3, 1, 4, 2)
    return c.reshape(p, h, t, d)


def _norm(x, w):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, cos, sin, inter):
    half = cos.shape[-1]
    if inter:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., 2 * half:]], -1)


def _plain_turn(s):
    case = s["case"]
    cos, sin = (s[n] if s["positions"] is None else s[n][s["positions"].long()] for n in ("cos", "sin"))
    return dict((n, _rotate(_norm(s[n], s[n + "_norm"]), cos[:, None], sin[:, None], case["inter"]).to(DT[case["x"]]))
                for n in ("q", "k"))


def _plain_append(s):
    case = s["case"]
    page = case["page"]
    cos, sin = s["cos"][s["pos"]][:, None], s["sin"][s["pos"]][:, None]
    q, k = (_rotate(_norm(s[n], s[n + "_norm"]), cos, sin, case["inter"]) for n in ("q", "k"))
    ids, slot = s["table"][s["seq"], s["pos"] // page].long(), s["pos"] % page
    out = [q.to(DT[case["x"]])]
    for name, new in (("k", k), ("v", s["v"].float())):  # the two halves of the cache
        codes, scale = s[name + "_cache"], s[name + "_scale"]
        touched, at = torch.unique(ids, return_inverse=True)
        top = torch.zeros((touched.numel(), case["H"]), device=new.device).scatter_reduce_(
            0, at[:, None].expand(-1, case["H"]), new.abs().amax(-1), "amax")
        kept = torch.full((touched.numel(),), page, device=new.device, dtype=torch.int64).scatter_reduce_(0, at, slot, "amin")
        before = torch.where((kept > 0)[:, None], scale[touched], torch.zeros_like(top))
        after = torch.maximum(before, top / 127)
        safe = torch.where(after > 0, after, torch.ones_like(after))
        rows = _rows(codes[touched], name).float() - 128
        old = torch.arange(page, device=new.device)[None, :] < kept[:, None]
        moved = torch.round(rows * (before / safe)[:, None, :, None])
        rows = torch.where(old[:, :, None, None], moved, rows)
        rows[at, slot] = torch.round(new / safe[at][..., None]).clamp(-127, 127)
        codes[touched] = _blocks((rows + 128).to(torch.uint8), name)
        scale[touched] = after
    ids, slot = s["table"][s["seq_read"], s["pos_read"] // page].long(), s["pos_read"] % page
    for name in ("k", "v"):
        t, at = torch.unique(ids, return_inverse=True)
        vals = (_rows(s[name + "_cache"][t], name).float() - 128) * s[name + "_scale"][t][:, None, :, None]
        out.append(vals[at, slot].to(DT[case["x"]]))
    return dict(q=out[0], k=out[1], v=out[2])


def _plain_attend(s):
    case = s["case"]
    H, Hq, D, B = case["H"], case["Hq"], case["D"], case["B"]
    L, n, rep = s["max_len"], s["max_new"], Hq // H
    K, V = ((_rows(s[c + "_cache"][s["table"].flatten().long()], c).float() - 128)
            .mul_(s[c + "_scale"][s["table"].flatten().long()][:, None, :, None])
            .view(B, -1, H, D)[:, :L].transpose(1, 2) for c in ("k", "v"))
    # queries padded to [B, H, n * rep, D]
    first = s["cu"][:-1].long()
    before = s["total"].long() - (s["cu"][1:].long() - first)
    at = s["pos"] - before[s["seq"]]
    q = torch.zeros((B, n, H, rep, D), device="cuda")
    q[s["seq"], at] = s["q"].float().view(-1, H, rep, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, H, n * rep, D)
    S = torch.matmul(q, K.transpose(2, 3).contiguous()) * D ** -0.5
    i = (before[:, None] + torch.arange(n, device="cuda")[None, :])[:, :, None]
    j = torch.arange(L, device="cuda")[None, None, :]
    seen = (j < s["total"][:, None, None]) & (j <= i) & ((j > i - case["window"]) | (j < case["sinks"]))
    S.view(B, H, n, rep, L).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = S.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    P = S.sub_(m).exp_()
    total = P.sum(-1, keepdim=True)
    o = torch.matmul(P, V.contiguous()) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(B, H, n, rep, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    return o[s["seq"], at].to(DT[case["x"]])


def _plain_tables(s):
    """Angles in 64 bits: at position 100000 a 32-bit product is off by thousandths of a radian."""
    c = s["case"]
    rot, base, kind = c["rot"], c["base"], c["kind"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    if kind == "ntk":
        base = base * c["factor"] ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    magnitude = 1.0
    if kind == "linear":
        f = f / c["factor"]
    elif kind == "yarn":
        lo, hi = (rot * math.log(c["original"] / (2 * math.pi * t)) / (2 * math.log(base)) for t in (c["high"], c["low"]))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / c["factor"] * ramp
        magnitude = 0.1 * math.log(c["factor"]) + 1
    elif kind == "wavelength":
        turns = c["original"] * f / (2 * math.pi)
        keep = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        f = f * keep + f / c["factor"] * (1 - keep)
    a = torch.arange(s["first"], s["first"] + c["n"], device="cuda", dtype=torch.float64)[:, None] * f
    return dict(cos=(a.cos() * magnitude).float(), sin=(a.sin() * magnitude).float())


def _plain_pages(s):
    c = s["case"]
    page, pages = c["page"], c["pool"]
    table, rows = s["table"].long(), s["rows"].long()
    R, W = rows.numel(), table.shape[1]
    goes = (rows >= 0) & (rows < table.shape[0])
    r = torch.where(goes, rows, torch.zeros_like(rows))
    L = torch.where(goes, s["lens"].long()[r].clamp(0, W * page), torch.zeros_like(rows))
    slot = torch.arange(W, device="cuda")[None, :]
    ids, L1 = table[r], L[:, None]
    kept = (ids >= 0) & (ids < pages) & (slot * page < L1)
    part = (slot == L1 // page) & (L1 % page != 0)          # the slot that the next token goes to
    if c["window"]:
        last = torch.minimum((slot + 1) * page, L1) - 1
        kept &= part | (slot * page < c["sinks"]) | (last > L1 - c["window"])
    safe = torch.where(kept, ids, torch.full_like(ids, pages))
    used, whole = (torch.zeros(pages + 1, dtype=torch.bool, device="cuda") for _ in range(2))
    used[safe.flatten()] = True
    whole[torch.where(part, torch.full_like(ids, pages), safe).flatten()] = True
    used[pages] = whole[pages] = False
    c_of = torch.arange(R, device="cuda")[:, None].expand(R, W)
    owner = torch.full((pages + 1,), R, device="cuda", dtype=torch.int64).scatter_reduce_(
        0, torch.where(part, safe, torch.full_like(ids, pages)).flatten(), c_of.flatten(), "amin")
    copied = kept & part & (whole[safe] | (owner[safe] != c_of))
    more = (slot >= -(-L1 // page)) & (slot < -(-(L1 + s["room"].long()[:, None].clamp(min=0)) // page))
    wants = copied | more
    nth = wants.flatten().long().cumsum(0).view(R, W) - 1
    kept_n, free = used.long().sum(), torch.nonzero(~used[:pages]).flatten()
    need = wants.long().sum()
    fresh = torch.minimum(need, torch.tensor(free.numel(), device="cuda"))
    n = kept_n + fresh
    to = torch.arange(pages + 1, device="cuda")
    moves = torch.zeros((0,), dtype=torch.int64, device="cuda")
    if c["compact"]:
        moves = torch.nonzero(used & (to >= n)).flatten()
        to[moves] = free[:moves.numel()]
        free = free[moves.numel():]
    free = torch.cat([free, torch.full((1,), -1, device="cuda", dtype=torch.int64)])
    taken = torch.where(nth < fresh, free[nth.clamp(0, free.numel() - 1)], torch.full_like(nth, -1))
    new = torch.where(wants, taken, torch.where(kept, to[safe], torch.full_like(ids, -1)))
    pair = copied & (taken >= 0)
    src = torch.cat([moves, ids[pair]])
    dst = torch.cat([to[moves], taken[pair]])
    room = R + (min(pages // 2, R * W) if c["compact"] else 0)
    pad = torch.full((room - src.numel(),), -1, device="cuda", dtype=torch.int64)
    for name in ("k", "v"):
        s[name + "_cache"][dst] = s[name + "_cache"][src]
        s[name + "_scale"][dst] = s[name + "_scale"][src]
    counts = torch.stack([torch.tensor(src.numel(), device="cuda"), n, need - fresh, torch.tensor(moves.numel(), device="cuda")])
    i32 = torch.int32
    return dict(table=new.to(i32), lens=L.to(i32), src=torch.cat([src, pad]).to(i32), dst=torch.cat([dst, pad]).to(i32),
                counts=counts.to(i32), k=s["k_cache"], v=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])


# ------------------------------------------------------------------ a pass ---

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "turn": _plain_turn, "tables": _plain_tables,
                "pages": _plain_pages}[op](s)
    import bit_weight_gemm_int2_amd as lb
    if op == "turn":
        q, k = lb.norm_rotate(s["q"], s["k"], q_norm=s["q_norm"], k_norm=s["k_norm"], cos=s["cos"], sin=s["sin"],
                              positions=s["positions"], eps=EPS, interleaved=case["inter"])
        return dict(q=q, k=k)
    if op == "tables":
        cos, sin = lb.rope_tables(case["n"], case["rot"], base=case["base"], scaling=None if case["kind"] == "none" else case["kind"],
                                  factor=case["factor"], original=case["original"], low=case["low"], high=case["high"],
                                  first=s["first"])
        return dict(cos=cos, sin=sin)
    cache = lb.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if op == "append":
        q = lb.kv_append(s["k"], s["v"], cache, s["table"], s["cu"], s["past"], s["max_new"], q=s["q"], cos=s["cos"],
                         sin=s["sin"], interleaved=case["inter"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        k, v = lb.kv_read(cache, s["table"], s["cu_read"], s["first"], s["T_read"], s["max_read"], DT[case["x"]])
        return dict(q=q, k=k, v=v)
    if op == "pages":
        plan = lb.kv_remap(s["table"], s["lens"], cache, rows=s["rows"], room=s["room"], window=case["window"],
                           sinks=case["sinks"], compact=case["compact"])
        lb.kv_copy_pages(cache, plan.src, plan.dst, count=plan.counts)
        return dict(table=plan.table, lens=plan.lens, src=plan.src, dst=plan.dst, counts=plan.counts, k=cache.k, v=cache.v,
                    k_scale=cache.k_scale, v_scale=cache.v_scale)
    return lb.attention(s["q"], cache, s["table"], s["cu"], s["total"], s["max_new"], s["max_len"], window=case["window"],
                        sinks=case["sinks"])


def work(case):
    op = case["op"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if op == "tables":
        return {"bytes": 4 * case["n"] * case["rot"], "flops": 2.0 * case["n"] * case["rot"]}
    if op == "turn":
        T, heads, D = case["T"], case["Hq"] + case["H"], case["D"]
        return {"bytes": 2 * size[case["x"]] * T * heads * D + 4 * T * case["rot"] + 2 * size[case["w"]] * D,
                "flops": T * heads * (4.0 * D + 3.0 * case["rot"])}
    past, new = _lengths(case)
    H, D, page = case["H"], case["D"], case["page"]
    if op == "pages":
        # the pairs of a state of this case, which no seed changes in number, from the tables alone
        got = _plan(case, past, *_shapes(case, past))
        return {"bytes": 4 * (2 * got["table"].size + 2 * got["lens"].size) + int(got["counts"][0]) * (4 * H * page * D + 16 * H),
                "flops": 0}
    Hq, T = case["Hq"], int(new.sum())
    if op == "append":
        read = int((past + new - past // page * page).sum())
        return {"bytes": 2 * T * Hq * D + 4 * T * case["rot"] + 2 * T * (Hq + 2 * H) * D + 2 * T * H * D + 2 * read * H * D * 3
                + 2 * size[case["w"]] * D, "flops": T * (Hq + H) * (4.0 * D + 3.0 * case["rot"])}
    seen = pairs = 0
    w, sinks = case["window"], case["sinks"]
    for p, n in zip(past.tolist(), new.tolist()):
        a = np.arange(p + 1, p + n + 1)
        pairs += int(np.minimum(a, w + np.minimum(sinks, np.maximum(a - w, 0))).sum())
        seen += min(p + n, w + n - 1 + sinks)
    return {"bytes": 2 * seen * H * D + 8 * (seen // page + 1) * H + 4 * T * Hq * D, "flops": 4.0 * pairs * Hq * D}


# ----------------------------------------------------- by definition, 64 bits ---

def _shapes(case, past):
    """A table like prepare's with pages in order, the sequences that go on, and room."""
    s = {}
    r = np.random.RandomState(71 + case["R"])
    B, R, page = case["B"], case["R"], case["page"]
    s["rows"] = np.sort(r.choice(B, R, replace=False)) if R <= B and not case["shared"] else r.randint(0, B, R)
    s["room"] = r.randint(0, case["room"] + 1, R)
    s["room"][0] = case["room"]
    width = int(-(-(past.max() + case["room"]) // page))
    perm = np.random.RandomState(3).permutation(case["pool"])
    table, at = np.full((B, width), -1), 0
    for b in range(B):
        n = -(-int(past[b]) // page)
        table[b, :n] = perm[at:at + n]
        at += n
    for b in range(1, B):
        n = min(case["shared"], int(past[b])) // page
        table[b, :n] = table[0, :n]
    return table, s["rows"], s["room"]


def _plan(case, lens, table, rows, room):
    """One row and slot after the other: what each new sequence keeps, then copies and new pages from the lowest free ones."""
    page, pages, window, sinks = case["page"], case["pool"], case["window"], case["sinks"]
    R, W = len(rows), table.shape[1]
    new, L, refs, first = np.full((R, W), -1, dtype=np.int64), np.zeros(R, dtype=np.int64), {}, {}
    for c in range(R):
        if not 0 <= rows[c] < len(lens):
            continue
        L[c] = min(max(int(lens[rows[c]]), 0), W * page)
        for t in range(0, int(L[c]), page):
            p, end = int(table[rows[c], t // page]), min(t + page, int(L[c]))
            whole = end == t + page
            if not 0 <= p < pages or (window and whole and t >= sinks and end - 1 <= L[c] - window):
                continue
            new[c, t // page] = p
            refs[p] = refs.get(p, False) or whole
            if not whole:
                first.setdefault(p, c)
    free = iter([p for p in range(pages) if p not in refs])
    wants = []
    for c in range(R):
        for s in range(W):
            begin = s * page
            if begin < L[c] < begin + page:
                p = int(new[c, s])
                if p >= 0 and (refs[p] or first[p] != c):
                    wants.append((c, s, p))
            elif L[c] <= begin < L[c] + max(0, int(room[c])):
                wants.append((c, s, -1))
    fresh = min(len(wants), pages - len(refs))
    n = len(refs) + fresh
    src, dst, to = [], [], {}
    if case["compact"]:
        for p in sorted(refs):
            if p >= n:
                to[p] = next(free)
                src.append(p)
                dst.append(to[p])
    moves = len(src)
    for (c, s), p in np.ndenumerate(new.copy()):
        if int(p) in to:
            new[c, s] = to[int(p)]
    for c, s, p in wants:
        q = next(free, -1) if fresh > 0 else -1
        fresh -= 1
        new[c, s] = q
        if p >= 0 and q >= 0:
            src.append(p)
            dst.append(q)
    return dict(table=new, lens=L, src=np.array(src, dtype=np.int64), dst=np.array(dst, dtype=np.int64),
                counts=np.array([len(src), n, len(wants) - (n - len(refs)), moves]))


def _turn64(x, w, cos, sin, inter):
    """Norm and rotation of rows [T, heads, D] with the angles' [T, half]."""
    x = x.double()
    y = x * w.double() / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    i = torch.arange(cos.shape[-1], device="cuda")
    lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + cos.shape[-1])
    c, s = cos.double()[:, None], sin.double()[:, None]
    r = y.clone()
    r[..., lo], r[..., hi] = y[..., lo] * c - y[..., hi] * s, y[..., lo] * s + y[..., hi] * c
    return r


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "tables":
        rot, base, out = case["rot"], case["base"], {}
        pos = np.arange(s["first"], s["first"] + case["n"], dtype=np.float64)
        cos, sin = np.empty((case["n"], rot // 2)), np.empty((case["n"], rot // 2))
        big = 1.0
        for i in range(rot // 2):
            f = 1.0 / base ** (2.0 * i / rot)
            if case["kind"] == "linear":
                f /= case["factor"]
            elif case["kind"] == "ntk":
                f = 1.0 / (base * case["factor"] ** (rot / (rot - 2.0))) ** (2.0 * i / rot)
            elif case["kind"] == "wavelength":
                length = 2 * math.pi / f
                if length > case["original"] / case["low"]:
                    f /= case["factor"]
                elif length >= case["original"] / case["high"]:
                    t = (case["original"] / length - case["low"]) / (case["high"] - case["low"])
                    f = (1 - t) * f / case["factor"] + t * f
            elif case["kind"] == "yarn":
                def dim(turns):
                    return rot * math.log(case["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
                lo, hi = max(math.floor(dim(case["high"])), 0), min(math.ceil(dim(case["low"])), rot - 1)
                t = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
                f = f / case["factor"] * t + f * (1 - t)
                big = 1.0 + 0.1 * math.log(case["factor"])
            cos[:, i], sin[:, i] = big * np.cos(pos * f), big * np.sin(pos * f)
        return dict(cos=cos, sin=sin)
    if op == "turn":
        at = torch.arange(case["T"], device="cuda") if s["positions"] is None else s["positions"].long()
        return {n: _turn64(s[n], s[n + "_norm"], s["cos"][at], s["sin"][at], case["inter"]) for n in ("q", "k")}
    if op == "pages":
        got = _plan(case, s["lens"].cpu().numpy(), *(s[n].cpu().numpy() for n in ("table", "rows", "room")))
        out = dict(table=got["table"], lens=got["lens"], src=None, dst=None, counts=got["counts"], k=None, v=None)
        for n in ("k_scale", "v_scale"):
            before = s[n].cpu().double().numpy()
            out[n] = before.copy()
            out[n][got["dst"]] = before[got["src"]]
        return out
    past, new = _lengths(case)
    table, page, H, Hq, D = s["table"].cpu().numpy(), case["page"], case["H"], case["Hq"], case["D"]
    cu = np.concatenate([[0], np.cumsum(new)])

    def scales(name, ids):
        return s[name + "_scale"][torch.from_numpy(np.ascontiguousarray(ids)).cuda().long()].double()

    if op == "append":
        got = {"q": [], "k": [], "v": []}
        t, d = (a.reshape(-1) for a in np.meshgrid(np.arange(page), np.arange(D), indexing="ij"))
        place = dict(k=(t // 16) * 16 * D + (d // 16) * 256 + (t % 16) * 16 + d % 16, v=(t // 4) * 4 * D + d * 4 + t % 4)
        for b, (p, n) in enumerate(zip(past.tolist(), new.tolist())):
            a, pos = slice(int(cu[b]), int(cu[b]) + n), torch.arange(p, p + n, device="cuda")
            got["q"].append(_turn64(s["q"][a], s["q_norm"], s["cos"][pos], s["sin"][pos], case["inter"]))
            lo, hi = p // page, (p + n - 1) // page
            ids = table[b, lo:hi + 1]
            for name in ("k", "v"):
                fresh = (_turn64(s["k"][a], s["k_norm"], s["cos"][pos], s["sin"][pos], case["inter"]) if name == "k"
                         else s["v"][a].double())
                full = torch.zeros(((hi - lo + 1) * page, H, D), dtype=torch.float64, device="cuda")
                at = p - lo * page
                full[at:at + n] = fresh
                blocks = full.view(-1, page, H, D)
                old = scales(name, ids)
                before = torch.zeros_like(old)
                if at:
                    before[0] = old[0]
                after = torch.maximum(before, blocks.abs().amax((1, 3)) / 127)
                unit = torch.where(after > 0, after, 1.0)[:, None, :, None]
                codes = torch.round(blocks / unit).clamp(-127, 127)
                if at:
                    was = s[name + "_cache"][int(ids[0])].reshape(H, page * D)[:, torch.from_numpy(place[name]).cuda()]
                    was = was.view(H, page, D).transpose(0, 1)[:at].double() - 128
                    codes[0, :at] = torch.round(was * (before[0] / unit[0, 0, :, 0])[None, :, None])
                got[name].append((codes * after[:, None, :, None]).reshape(-1, H, D)[:at + n])
        return {n: torch.cat(v) for n, v in got.items()}
    out = torch.zeros((s["T"], Hq, D), dtype=torch.float64, device="cuda")
    rep, w, sinks = Hq // H, case["window"], case["sinks"]
    for b, (p, n) in enumerate(zip(past.tolist(), new.tolist())):
        L = p + n
        ids = table[b, : -(-L // page)]
        for h in range(H):
            kk, vv = ((s[c + "_cache"][torch.from_numpy(ids).cuda().long(), h]) for c in ("k", "v"))
            kk = kk.view(-1, page // 16, D // 16, 16, 16).transpose(2, 3).reshape(-1, page, D).double() - 128
            vv = vv.view(-1, page // 4, D, 4).transpose(2, 3).reshape(-1, page, D).double() - 128
            kk = (kk * scales("k", ids)[:, h, None, None]).view(-1, D)[:L]
            vv = (vv * scales("v", ids)[:, h, None, None]).view(-1, D)[:L]
            q = s["q"][int(cu[b]):int(cu[b]) + n, h * rep:(h + 1) * rep].double()
            for a in range(0, n, 512):
                x = q[a:a + 512].reshape(-1, D) @ kk.t().contiguous() / math.sqrt(D)
                i = (p + a + torch.arange(x.shape[0] // rep, device="cuda")).repeat_interleave(rep)[:, None]
                j = torch.arange(L, device="cuda")[None]
                hide = (j > i) | ((j <= i - w) & (j >= sinks))
                x = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ vv
                out[int(cu[b]) + a:int(cu[b]) + min(n, a + 512), h * rep:(h + 1) * rep] = x.view(-1, rep, D)
    return out
