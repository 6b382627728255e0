"""A small decoder with 4-bit weights and an 8-bit paged cache, prompt then token by token.

Random weights of the text encoder's layer shape (hidden size, heads and MLP can be made smaller). One step is, per
layer: norm, fused q|k|v linear, rotation + append to the cache, attention over it, output linear, norm, fused gate|up
linear, gated MLP, down linear; then the output vocabulary. Prompts run the same step with gemm_int4 in place of
gemv_int4. With --check the step is compared with the same arithmetic in float64 on the CPU (cache in 8 bits apart).

The pages come from one pool: every step makes room for its tokens, and lets go of pages that a --window has passed.
--answers continues each prompt in several ways that share its pages, and --head-norms normalises the heads of queries
and keys before their rotation, whose tables --scaling stretches.

    python examples/text_decode.py --layers 4 --prompt 200 --tokens 32 --check
    python examples/text_decode.py --prompt 300 --window 128 --sinks 4 --head-norms --scaling yarn --answers 3 --check
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_gemm_int2_amd as lb  # noqa: E402


class Linear4:
    """Random 4-bit weights [n, k], packed."""

    def __init__(self, n, k, gen):
        self.codes = torch.randint(0, 16, (n, k), generator=gen, device="cuda", dtype=torch.uint8)
        self.packed = lb.pack_int4(self.codes)
        self.scales = (torch.rand((n, k // 128), generator=gen, device="cuda") * 0.2 + 0.9).mul_(0.2 / k ** 0.5).half()
        self.zeros = (7.5 + 0.5 * torch.randn((n, k // 128), generator=gen, device="cuda")).half()

    def __call__(self, x):
        call = lb.gemv_int4 if x.shape[0] <= 16 else lb.gemm_int4
        return call(x, self.packed, self.scales, self.zeros)

    def dense(self):
        s, z = (t.double().repeat_interleave(128, 1) for t in (self.scales, self.zeros))
        return ((self.codes.double() - z) * s).cpu()


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Model:
    def __init__(self, layers, hidden, q_heads, kv_heads, head_dim, mlp, vocab, page, pages, positions, seed=0,
                 head_norms=False, window=0, sinks=0, scaling=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.h, self.d = q_heads, kv_heads, head_dim
        self.window, self.sinks = window, sinks
        self.missing = torch.zeros(1, dtype=torch.int32, device="cuda")  # pages that the pool did not have
        self.embed = torch.randn((vocab, hidden), generator=g, device="cuda").bfloat16()
        self.layers = [dict(qkv=Linear4((q_heads + 2 * kv_heads) * head_dim, hidden, g),
                            o=Linear4(hidden, q_heads * head_dim, g), up=Linear4(2 * mlp, hidden, g),
                            down=Linear4(hidden, mlp, g), cache=lb.new_kv_cache(pages, kv_heads, page, head_dim))
                       for _ in range(layers)]
        self.head = Linear4(vocab, hidden, g)
        for w in self.layers:  # weights of the heads' norms, or none
            w["q_norm"], w["k_norm"] = ((1 + torch.randn(head_dim, generator=g, device="cuda") / 8).bfloat16() if head_norms
                                        else None for _ in range(2))
        self.cos, self.sin = lb.rope_tables(positions, head_dim, base=1e6, scaling=scaling, factor=4.0 if scaling else 1.0,
                                            original=max(1, positions // 4), low=1.0, high=32.0)

    def forward(self, tokens, table, cu, starts, lens, max_new, max_len):
        """Logits of every token; the cache grows by them."""
        x = self.embed[tokens]
        for w in self.layers:
            qkv = w["qkv"](norm(x)).view(-1, self.hq + 2 * self.h, self.d)
            q, k, v = qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.h], qkv[:, self.hq + self.h:]
            q = lb.kv_append(k, v, w["cache"], table, cu, starts, max_new, q=q, cos=self.cos, sin=self.sin,
                             q_norm=w["q_norm"], k_norm=w["k_norm"])
            y = lb.attention(q, w["cache"], table, cu, lens, max_new, max_len, window=self.window, sinks=self.sinks)
            x = x + w["o"](y.view(len(tokens), -1))
            gate, up = w["up"](norm(x)).chunk(2, -1)
            x = x + w["down"](torch.nn.functional.silu(gate) * up)
        return self.head(norm(x))

    def pages_for(self, table, lens, rows, room):
        """A table for the sequences that go on, with room for their next tokens; copies what it asks for. Tokens whose page the
        pool does not have are lost: counted on the GPU, which a step does not wait for."""
        plan = lb.kv_remap(table, lens, self.layers[0]["cache"], rows=rows, room=room, window=self.window, sinks=self.sinks)
        for w in self.layers:
            lb.kv_copy_pages(w["cache"], plan.src, plan.dst, plan.counts)
        self.missing += plan.counts[2]
        return plan.table, plan.lens

    def reference(self, tokens):
        """Logits of one sequence in float64 on the CPU, from the definition."""
        x = self.embed[tokens].double().cpu()
        n, half = len(tokens), self.d // 2
        c, s = self.cos[:n].double().cpu()[:, None], self.sin[:n].double().cpu()[:, None]

        def nrm(t):
            return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)

        def turn(t, weight):
            if weight is not None:
                t = nrm(t) * weight.double().cpu()
            a, b = t[..., :half], t[..., half:]
            return torch.cat([a * c - b * s, a * s + b * c], -1)

        i, j = torch.arange(n)[:, None], torch.arange(n)[None, :]
        hidden = j > i
        if self.window:
            hidden |= (j <= i - self.window) & (j >= self.sinks)
        for w in self.layers:
            qkv = (nrm(x) @ w["qkv"].dense().t()).view(n, -1, self.d)
            q, k = turn(qkv[:, :self.hq], w["q_norm"]), turn(qkv[:, self.hq:self.hq + self.h], w["k_norm"])
            v = qkv[:, self.hq + self.h:]
            k, v = (t.repeat_interleave(self.hq // self.h, 1) for t in (k, v))
            a = torch.einsum("ihd,jhd->hij", q, k) * self.d ** -0.5
            a = a.masked_fill(hidden, -torch.inf).softmax(-1)
            x = x + torch.einsum("hij,jhd->ihd", a, v).reshape(n, -1) @ w["o"].dense().t()
            gate, up = (nrm(x) @ w["up"].dense().t()).chunk(2, -1)
            x = x + (torch.nn.functional.silu(gate) * up) @ w["down"].dense().t()
        return nrm(x) @ self.head.dense().t()


def generate(model, prompts, steps, width, answers=1):
    """Greedy continuations of a batch of prompts (lists of token numbers): `answers` of each, which differ in their first
    token (the likeliest ones). Returns the sequences, the last step's logits and the seconds a step took. A pool with too few
    pages is an error, found at the end."""
    model.missing.zero_()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, most = [len(p) for p in prompts], max(len(p) for p in prompts)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    table, starts = model.pages_for(i32([]).view(0, width), i32([]), i32([-1] * len(prompts)), i32(lens))
    first = model.forward(torch.tensor(sum(prompts, []), device="cuda"), table, i32(cu), starts, i32(lens), most, most)
    logits = first[i32(cu[1:]).long() - 1]
    out = [logits.topk(answers, -1).indices.flatten()]
    pos, rows = i32(lens), i32([b for b in range(len(prompts)) for _ in range(answers)])
    n = len(rows)
    cu, one, same = i32(list(range(n + 1))), i32([1] * n), i32(list(range(n)))
    torch.cuda.synchronize()
    t = time.perf_counter()
    for s in range(steps - 1):
        table, pos = model.pages_for(table, pos, rows, one)
        rows = same
        logits = model.forward(out[-1], table, cu, pos, pos + 1, 1, most + s + 1)
        pos = pos + 1
        out.append(logits.argmax(-1))
    torch.cuda.synchronize()
    took = (time.perf_counter() - t) / max(1, steps - 1)
    if int(model.missing):
        raise RuntimeError(f"the pool ran out of pages: {int(model.missing)} that the sequences needed were missing")
    tails = torch.stack(out, 1).tolist()
    return [prompts[i // answers] + t for i, t in enumerate(tails)], logits, took


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("layers", 4), ("hidden", 2560), ("q-heads", 32), ("kv-heads", 8), ("head-dim", 128),
                        ("mlp", 9728), ("vocab", 32768), ("page", 64), ("batch", 2), ("prompt", 200), ("tokens", 32)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--answers", type=int, default=1, help="continuations of each prompt")
    ap.add_argument("--window", type=int, default=0, help="tokens that a query sees (0: all)")
    ap.add_argument("--sinks", type=int, default=0, help="first tokens that it sees beside them")
    ap.add_argument("--head-norms", action="store_true", help="norms of the heads of queries and keys")
    ap.add_argument("--scaling", choices=("linear", "ntk", "yarn", "wavelength"), help="rotary positions for four times the length")
    ap.add_argument("--check", action="store_true", help="compare the last step with float64 on the CPU")
    a = ap.parse_args()
    width = -(-(a.prompt + a.tokens) // a.page)
    model = Model(a.layers, a.hidden, a.q_heads, a.kv_heads, a.head_dim, a.mlp, a.vocab, a.page, a.batch * a.answers * width,
                  a.prompt + a.tokens, head_norms=a.head_norms, window=a.window, sinks=a.sinks, scaling=a.scaling)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, a.vocab, (max(1, a.prompt - 7 * b),), generator=g).tolist() for b in range(a.batch)]
    seqs, logits, took = generate(model, prompts, a.tokens, width, a.answers)
    print(f"{len(seqs)} sequences, {a.layers} layers, prompt of {a.prompt}, {a.tokens} tokens: {took * 1e6:.0f} us a step")
    if a.check:
        off = 0.0
        for i in range(a.answers):
            # with one token the logits are those of the prompts' ends
            want = model.reference(torch.tensor(seqs[i][:-1]))[-1]
            off = max(off, float((logits[i if a.tokens > 1 else 0].double().cpu() - want).norm() / want.norm()))
        print(f"last logits against float64: relative difference {off:.4f}")
        # bf16 activations through 4 roundings a layer and 8-bit keys and values (steps of 1/127 of a block's largest)
        assert off < 0.02 * a.layers, off


if __name__ == "__main__":
    main()
