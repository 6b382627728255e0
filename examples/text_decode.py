"""A small decoder with 4-bit weights and an 8-bit paged cache, prompt then token by token.

Random weights of the text encoder's layer shape (hidden size, heads and MLP can be made smaller). One step is, per
layer: norm, fused q|k|v linear, rotation + append to the cache, attention over it, output linear, norm, fused gate|up
linear, gated MLP, down linear; then the output vocabulary. Prompts run the same step with gemm_int4 in place of
gemv_int4. With --check the step is compared with the same arithmetic in float64 on the CPU (cache in 8 bits apart).

    python examples/text_decode.py --layers 4 --prompt 200 --tokens 32 --check
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
    def __init__(self, layers, hidden, q_heads, kv_heads, head_dim, mlp, vocab, page, pages, positions, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.h, self.d = q_heads, kv_heads, head_dim
        self.embed = torch.randn((vocab, hidden), generator=g, device="cuda").bfloat16()
        self.layers = [dict(qkv=Linear4((q_heads + 2 * kv_heads) * head_dim, hidden, g),
                            o=Linear4(hidden, q_heads * head_dim, g), up=Linear4(2 * mlp, hidden, g),
                            down=Linear4(hidden, mlp, g), cache=lb.new_kv_cache(pages, kv_heads, page, head_dim))
                       for _ in range(layers)]
        self.head = Linear4(vocab, hidden, g)
        f = 1e6 ** (-torch.arange(head_dim // 2, device="cuda", dtype=torch.float64) / (head_dim // 2))
        a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
        self.cos, self.sin = a.cos().float(), a.sin().float()

    def forward(self, tokens, table, cu, starts, lens, max_new, max_len):
        """Logits of every token; the cache grows by them."""
        x = self.embed[tokens]
        for w in self.layers:
            qkv = w["qkv"](norm(x)).view(-1, self.hq + 2 * self.h, self.d)
            q, k, v = qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.h], qkv[:, self.hq + self.h:]
            q = lb.kv_append(k, v, w["cache"], table, cu, starts, max_new, q=q, cos=self.cos, sin=self.sin)
            y = lb.attention(q, w["cache"], table, cu, lens, max_new, max_len)
            x = x + w["o"](y.view(len(tokens), -1))
            gate, up = w["up"](norm(x)).chunk(2, -1)
            x = x + w["down"](torch.nn.functional.silu(gate) * up)
        return self.head(norm(x))

    def reference(self, tokens):
        """Logits of one sequence in float64 on the CPU, from the definition."""
        x = self.embed[tokens].double().cpu()
        n, half = len(tokens), self.d // 2
        c, s = self.cos[:n].double().cpu()[:, None], self.sin[:n].double().cpu()[:, None]

        def nrm(t):
            return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)

        def turn(t):
            a, b = t[..., :half], t[..., half:]
            return torch.cat([a * c - b * s, a * s + b * c], -1)

        for w in self.layers:
            qkv = (nrm(x) @ w["qkv"].dense().t()).view(n, -1, self.d)
            q, k, v = turn(qkv[:, :self.hq]), turn(qkv[:, self.hq:self.hq + self.h]), qkv[:, self.hq + self.h:]
            k, v = (t.repeat_interleave(self.hq // self.h, 1) for t in (k, v))
            a = torch.einsum("ihd,jhd->hij", q, k) * self.d ** -0.5
            a = a.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), -torch.inf).softmax(-1)
            x = x + torch.einsum("hij,jhd->ihd", a, v).reshape(n, -1) @ w["o"].dense().t()
            gate, up = (nrm(x) @ w["up"].dense().t()).chunk(2, -1)
            x = x + (torch.nn.functional.silu(gate) * up) @ w["down"].dense().t()
        return nrm(x) @ self.head.dense().t()


def generate(model, prompts, steps, page, width):
    """Greedy continuation of a batch of prompts (lists of token numbers); returns the sequences, the last step's
    logits and the seconds a step took."""
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    batch, lens = len(prompts), [len(p) for p in prompts]
    table = torch.arange(batch * width, dtype=torch.int32, device="cuda").view(batch, width)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    first = model.forward(torch.tensor(sum(prompts, []), device="cuda"), table, i32(cu), i32([0] * batch), i32(lens),
                          max(lens), max(lens))
    logits = first[i32(cu[1:]).long() - 1]
    cu, pos, most = i32(list(range(batch + 1))), i32(lens), max(lens)
    out = [logits.argmax(-1)]
    torch.cuda.synchronize()
    t = time.perf_counter()
    for s in range(steps - 1):
        logits = model.forward(out[-1], table, cu, pos, pos + 1, 1, most + s + 1)
        pos = pos + 1
        out.append(logits.argmax(-1))
    torch.cuda.synchronize()
    took = (time.perf_counter() - t) / max(1, steps - 1)
    tails = torch.stack(out, 1).tolist()
    return [p + t for p, t in zip(prompts, tails)], logits, took


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("layers", 4), ("hidden", 2560), ("q-heads", 32), ("kv-heads", 8), ("head-dim", 128),
                        ("mlp", 9728), ("vocab", 32768), ("page", 64), ("batch", 2), ("prompt", 200), ("tokens", 32)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--check", action="store_true", help="compare the last step with float64 on the CPU")
    a = ap.parse_args()
    width = -(-(a.prompt + a.tokens) // a.page)
    model = Model(a.layers, a.hidden, a.q_heads, a.kv_heads, a.head_dim, a.mlp, a.vocab, a.page, a.batch * width,
                  a.prompt + a.tokens)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, a.vocab, (max(1, a.prompt - 7 * b),), generator=g).tolist() for b in range(a.batch)]
    seqs, logits, took = generate(model, prompts, a.tokens, a.page, width)
    print(f"{a.batch} sequences, {a.layers} layers, prompt of {a.prompt}, {a.tokens} tokens: {took * 1e6:.0f} us a step")
    if a.check:
        want = model.reference(torch.tensor(seqs[0][:-1]))[-1]
        off = float((logits[0].double().cpu() - want).norm() / want.norm())
        print(f"last logits against float64: relative difference {off:.4f}")
        # bf16 activations through 4 roundings a layer and 8-bit keys and values (steps of 1/127 of a block's largest)
        assert off < 0.02 * a.layers, off


if __name__ == "__main__":
    main()
