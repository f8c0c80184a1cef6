"""Speculative decoding with a small hyper-connected decoder: a tree of drafted tokens a step.

One step, for every sequence of the batch: the drafted tree's mask and positions (hc_tree_build); the
decoder over all nodes (hc_stack), whose attention sublayers turn the heads (hc_rope), store the keys and
values (hc_kv_write) and attend over the paged cache (hc_tree_attention); the logits (hc_exit_logits);
which drafts hold (hc_verify); and the accepted rows moved to where the sequence goes on (hc_kv_compact).
The decoder's weights are random, and its draft is a table of next tokens made from the embedding.

    python examples/speculative_decode.py [--cache bf16|fp8|int4] [--temperature X] [--tokens N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from hyper_connection_residual_call_gb300 import binding as B, inputs  # noqa: E402

# The drafted tree: the root is the token that the last step ended with; three guesses after it, two after the best, ...
PARENTS = [-1, 0, 0, 0, 1, 1, 2, 4, 4, 7]


class Decoder:
    """``layers`` layers of attention and a gated MLP around a residual of ``C`` streams of ``H`` elements."""

    def __init__(self, *, H=256, C=4, L=64, layers=2, q_heads=8, kv_heads=2, D=64, V=1024, max_pos=4096, seed=0):
        self.H, self.C, self.q_heads, self.kv_heads, self.D, self.V = H, C, q_heads, kv_heads, D, V
        g = torch.Generator(device="cuda").manual_seed(seed)
        draw = lambda rows, cols: (torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).bfloat16()  # noqa: E731
        self.hc = [tuple(inputs.make_hc_weights(H, C, L, seed, 2 * i + j).to("cuda") for j in range(2)) for i in range(layers)]
        self.final = inputs.make_hc_weights(H, C, L, seed, 2 * layers, with_inject=False).to("cuda")
        self.qkv = [draw((q_heads + 2 * kv_heads) * D, H) for _ in range(layers)]
        self.out = [draw(H, q_heads * D) for _ in range(layers)]
        self.up = [draw(4 * H, H) for _ in range(layers)]
        self.down = [draw(H, 2 * H) for _ in range(layers)]
        self.emb = torch.randn(V, H, generator=g, device="cuda").bfloat16()
        self.lm_head = draw(V, H)
        self.rope = B.rope_table(max_pos, D, 10000.0)

    def caches(self, kind, batch, max_len, page=16):
        """One paged cache a layer; the layers share a page table."""
        per = -(-max_len // page)
        table = torch.randperm(batch * per, device="cuda").int().view(batch, per)
        return [B.kv_cache(kind, batch * per, self.kv_heads, page, self.D, table) for _ in self.qkv]

    def logits(self, tokens, caches, ctx_len, positions, mask=None):
        """fp32 [batch, T, V] of the nodes ``tokens`` [batch, T], whose rows go to ctx_len .. ctx_len + T - 1."""
        b, t = tokens.shape
        hq, hk, d = self.q_heads, self.kv_heads, self.D

        def sublayer(layer, which, t0, mixed):
            if which == 1:
                gate, x = (mixed @ self.up[layer].T).chunk(2, -1)
                return (torch.nn.functional.silu(gate) * x) @ self.down[layer].T
            heads = (mixed @ self.qkv[layer].T).view(b, t, hq + 2 * hk, d)
            q, k, v = heads.split((hq, hk, hk), 2)  # views: the operators take strided rows
            q, k = B.hc_rope(q, k, positions, self.rope)
            B.hc_kv_write(k, v, caches[layer], ctx_len)
            out, _ = B.hc_tree_attention(q, caches[layer], ctx_len, mask=mask)
            return out.view(b * t, hq * d) @ self.out[layer].T

        _, raw = B.hc_stack(self.emb[tokens.long()].view(b * t, self.H), self.hc, self.final, sublayer, C=self.C)
        _, logits = B.hc_exit_logits(raw, self.final, self.lm_head, H=self.H, C=self.C)
        return logits.view(b, t, self.V)


def generate(model, prompt, n_tokens, *, kind="bf16", temperature=0.0, seed=0):
    """``n_tokens`` (or a few more) tokens after ``prompt`` [batch, length], which all sequences take whole.
    Returns (per sequence the new tokens, the caches, the context lengths, the steps taken)."""
    b, n = prompt.shape
    T = len(PARENTS)
    g = torch.Generator(device="cuda").manual_seed(seed)
    parents = torch.tensor(PARENTS, dtype=torch.int32, device="cuda")
    # the draft's distributions: one row a token
    draft = torch.softmax(model.emb.float() @ model.lm_head.float().T / max(temperature, 0.5), -1)
    best = draft.topk(3, -1).indices.int()
    nth = [PARENTS[:i].count(p) for i, p in enumerate(PARENTS)]
    temp = torch.full((b,), float(temperature), device="cuda")

    caches = model.caches(kind, b, n + n_tokens + 2 * T)
    ctx = torch.zeros(b, dtype=torch.int32, device="cuda")
    positions = torch.arange(n, dtype=torch.int32, device="cuda").repeat(b, 1)
    logits = model.logits(prompt, caches, ctx, positions)[:, -1:].contiguous()
    ctx = ctx + n

    def decide(logits, tokens, parents, probs):
        if temperature <= 0:
            return B.hc_verify(logits, tokens, parents)
        u = torch.rand(tokens.shape, generator=g, device="cuda")
        noise = torch.empty(b, model.V, device="cuda").exponential_(generator=g).clamp_min_(1e-30)
        return B.hc_verify(logits, tokens, parents, temp, draft_probs=probs, u=u, noise=noise)

    # the first token: a tree of a root alone
    tokens = prompt[:, -1:].contiguous()
    _, _, last = decide(logits, tokens, None, draft[tokens.long()])
    made = [[int(x)] for x in last]
    steps = 0
    while min(map(len, made)) < n_tokens:
        tokens = torch.empty(b, T, dtype=torch.int32, device="cuda")
        tokens[:, 0] = last
        for i, p in enumerate(PARENTS[1:], 1):
            if temperature <= 0:
                tokens[:, i] = best[tokens[:, p].long(), nth[i]]
            else:
                tokens[:, i] = torch.multinomial(draft[tokens[:, p].long()], 1, generator=g)[:, 0].int()
        mask, positions = B.hc_tree_build(parents, ctx)
        logits = model.logits(tokens, caches, ctx, positions, mask)
        accepted, path, last = decide(logits, tokens, parents, draft[tokens.long()])
        for cache in caches:
            new_ctx = B.hc_kv_compact(cache, ctx, path, accepted)
        steps += 1
        for i in range(b):
            if len(made[i]) < n_tokens:
                took = tokens[i, path[i, 1:1 + int(accepted[i])].long()]
                made[i] += took.tolist() + [int(last[i])]
                ctx[i] = new_ctx[i]
            else:  # done: it takes part without going on
                last[i] = tokens[i, 0]
    if B.device_status() != B.TS_OK:
        raise RuntimeError(B.ts_hc_last_error())
    return made, caches, ctx, steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--cache", choices=("bf16", "fp8", "int4"), default="fp8")
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--batch", type=int, default=4)
    a = ap.parse_args()
    model = Decoder()
    prompt = torch.randint(model.V, (a.batch, 40), generator=torch.Generator().manual_seed(1)).int().cuda()
    made, _, _, steps = generate(model, prompt, a.tokens, kind=a.cache, temperature=a.temperature)
    n = sum(map(len, made))
    print(f"{n} tokens of {a.batch} sequences in {steps} steps of {len(PARENTS)} nodes ({n / a.batch / steps:.2f} a step)")
    for row in made:
        print(*row[:16], "...")


if __name__ == "__main__":
    main()
