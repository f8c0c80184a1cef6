"""Cases for the operators of a speculative decoding step: rotary positions, a paged cache that is
quantised as it is written, attention for a tree of drafted tokens over that cache, and the
verification of the drafted tokens.

``run`` with ``own`` false computes each operator from elementary torch operations in 32 bits; with
``own`` true it makes the library's calls. ``exact`` computes the same results in 64 bits from the
operators' definitions.
"""
import math
import random

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One decoded token: every layer of a decoder turns its query and key heads once (2560 = 20 heads of 128).
        dict(name="rope one token", op="rope", tokens=1, q_heads=20, kv_heads=4, dim=128, rot=128,
             interleaved=False, inverse=False, max_pos=32768),
        # A prompt's chunks in a long context: interleaved pairs, half of each head turned.
        dict(name="rope long prompt", op="rope", tokens=16384, q_heads=32, kv_heads=8, dim=128, rot=64,
             interleaved=True, inverse=False, max_pos=131072),
        # The gradient of a batch's turn (the inverse rotation), an odd number of tokens.
        dict(name="rope gradient odd", op="rope", tokens=4099, q_heads=16, kv_heads=2, dim=64, rot=64,
             interleaved=False, inverse=True, max_pos=8192),
        # The keys and values of one step's drafted tokens go to a 4-bit cache and come back.
        dict(name="cache step int4", op="kv", kind="int4", group=64, batch=8, tokens=13, ctx=4000, kv_heads=4, dim=128,
             page=16),
        # A prompt's keys and values go to an 8-bit cache and come back for a later prompt with the same prefix.
        dict(name="cache prompt fp8", op="kv", kind="fp8", group=0, batch=4, tokens=8192, ctx=1000, kv_heads=8, dim=128,
             page=64),
        # One sequence, one token, a short context: the smallest call, where latency counts.
        dict(name="attention one token", op="attn", kind="bf16", group=0, batch=1, tokens=1, ctx=1000, q_heads=20,
             kv_heads=4, dim=128, page=16, tree=False),
        # A serving batch of ragged contexts, a chain of 8 drafted tokens each.
        dict(name="attention batch chain bf16", op="attn", kind="bf16", group=0, batch=32, tokens=8, ctx=6000,
             q_heads=32, kv_heads=8, dim=128, page=64, tree=False),
        # A tree of 16 drafted tokens over long 8-bit caches.
        dict(name="attention tree fp8 long", op="attn", kind="fp8", group=0, batch=4, tokens=16, ctx=65536,
             q_heads=32, kv_heads=8, dim=128, page=64, tree=True),
        # Very long 4-bit caches, few drafted tokens.
        dict(name="attention chain int4 long", op="attn", kind="int4", group=64, batch=2, tokens=3, ctx=131072,
             q_heads=32, kv_heads=8, dim=128, page=32, tree=False),
        # A wide tree over shared heads: products of 512 rows with every key.
        dict(name="attention wide tree bf16", op="attn", kind="bf16", group=0, batch=4, tokens=64, ctx=16384,
             q_heads=64, kv_heads=8, dim=128, page=64, tree=True),
        # One sequence's chain of four drafted tokens, the vocabulary of this library's own exit.
        dict(name="verify chain", op="verify", batch=1, tokens=5, vocab=32768, tree=False, greedy=False),
        # A serving batch of trees over a large odd vocabulary, some sequences greedy.
        dict(name="verify tree batch", op="verify", batch=16, tokens=26, vocab=128001, tree=True, greedy=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "kv", "attn", "attn", "verify"])
    if op == "rope":
        dim = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8])
        return dict(op="rope", tokens=_log(rng, 1, 16384), q_heads=kv * rng.choice([1, 4, 5, 8][:3 if kv == 8 else 4]),
                    kv_heads=kv, dim=dim, rot=rng.choice([dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.3, max_pos=rng.choice([8192, 32768, 131072]))
    if op == "kv":
        kind = rng.choice(["bf16", "fp8", "int4"])
        batch = _log(rng, 1, 32)
        return dict(op="kv", kind=kind, group=rng.choice([32, 64]) if kind == "int4" else 0, batch=batch,
                    tokens=_log(rng, 1, 32768 // batch), ctx=_log(rng, 1, 4000), kv_heads=rng.choice([1, 2, 4, 8]),
                    dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]))
    if op == "attn":
        kind = rng.choice(["bf16", "fp8", "int4"])
        kv = rng.choice([1, 2, 4, 8])
        batch = _log(rng, 1, 32)
        tokens = _log(rng, 1, 64)
        return dict(op="attn", kind=kind, group=rng.choice([32, 64]) if kind == "int4" else 0, batch=batch, tokens=tokens,
                    ctx=_log(rng, 100, min(131072, 200000 // batch, 16384 * 256 // (batch * tokens))),
                    q_heads=kv * rng.choice([1, 4, 5, 8]), kv_heads=kv, dim=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]), tree=rng.random() < 0.6)
    batch = _log(rng, 1, 48)
    tokens = _log(rng, 2, 26)
    return dict(op="verify", batch=batch, tokens=tokens, vocab=_log(rng, 1000, min(128001, 16 * 26 * 128001 // (batch * tokens))),
                tree=rng.random() < 0.6, greedy=rng.random() < 0.25)


def _lengths(case):
    """The sequences' context lengths, longest last: from half of ctx up to ctx (one sequence has all of it)."""
    b, n = case["batch"], case["ctx"]
    return [n if b == 1 else n // 2 + (n - n // 2) * i // (b - 1) for i in range(b)]


def _row_bytes(case):
    """Bytes that one token and head of the cache takes, keys or values."""
    d = case["dim"]
    return {"bf16": 2 * d, "fp8": d + 1, "int4": d // 2 + (4 * d // case["group"] if case["group"] else 0)}[case["kind"]]


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        return dict(bytes=n * case["dim"] * 4 + case["tokens"] * (case["rot"] * 4 + 4), flops=3 * n * case["rot"])
    if case["op"] == "kv":  # bf16 in, codes out; codes in, bf16 out
        n = 2 * case["batch"] * case["tokens"] * case["kv_heads"]
        return dict(bytes=n * (4 * case["dim"] + 2 * _row_bytes(case)), flops=4 * n * case["dim"])
    if case["op"] == "attn":
        t, hq = case["tokens"], case["q_heads"]
        keys = sum(x + t for x in _lengths(case))
        return dict(bytes=keys * case["kv_heads"] * 2 * _row_bytes(case) + case["batch"] * t * hq * (4 * case["dim"] + 4),
                    flops=4 * keys * t * hq * case["dim"])
    # A walk visits the root's row at least; a sampled one reads a draft row where it rejects (most walks end with a
    # rejection) and the noise. What further rows it visits is up to the data.
    rows = 1 if case["greedy"] else 3
    return dict(bytes=case["batch"] * case["vocab"] * 4 * rows, flops=case["batch"] * case["vocab"] * 4 * rows)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).bfloat16()


def _power(e):
    """2**e in 32 bits for whole e, from its bits: exact, which exp2 need not be."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x, kind, group):
    """Codes, scales and biases of rows x [..., D] (32 bits)."""
    if kind == "bf16":
        return x.bfloat16(), None, None
    if kind == "fp8":
        fine = torch.isfinite(x)
        amax = torch.where(fine, x.abs(), 0.0).amax(-1)
        m, e = torch.frexp(amax)
        e = torch.where(m <= 0.875, e - 9, e - 8)  # the smallest e with amax <= 448 * 2**e
        e = torch.where(amax > 0, e, -117).clamp(min=-117)
        byte = torch.where(fine.all(-1), e + 127, 255).to(torch.uint8)
        codes = (x * _power(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        return codes, byte, None
    y = x.unflatten(-1, (-1, group))
    lo, hi = y.amin(-1), y.amax(-1)
    s = ((hi - lo) / 15).clamp(max=65504).half()
    b = lo.clamp(-65504, 65504).half()
    sf = s.float()[..., None]
    q = torch.where(sf > 0, torch.round((y - b.float()[..., None]) / sf), 0.0).clamp(0, 15).to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), s, b


def _dequantise(codes, s, b, kind, group):
    """The values (32 bits) that the codes stand for."""
    if kind == "bf16":
        return codes.float()
    if kind == "fp8":
        scale = torch.where(s == 255, float("nan"), _power(s.int() - 127))
        return codes.view(torch.float8_e4m3fn).float() * scale[..., None]
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, group))
    return (q * s.float()[..., None] + b.float()[..., None]).flatten(-2)


def _pages(case, seed):
    """The page table [B][max_pages] (a random order of the pool's pages) and the pool's number of pages."""
    per = -(-(case["ctx"] + case["tokens"]) // case["page"])
    n = per * case["batch"] + 3
    g = torch.Generator().manual_seed(seed + 5)
    return torch.randperm(n, generator=g)[:per * case["batch"]].view(case["batch"], per).int().to(DEV), n


def _parents(case, seed):
    """[B][T] int32: a chain, or a random tree (node 0 is the root)."""
    r = random.Random(seed * 31 + 7)
    rows = []
    for _ in range(case["batch"]):
        p = [-1]
        for i in range(1, case["tokens"]):
            p.append(i - 1 if not case["tree"] or r.random() < 0.4 else r.randrange(i if r.random() < 0.5 else min(i, 4)))
        rows.append(p)
    return rows


def _ancestors(rows):
    """Per sequence, the nodes that each node sees: itself and what is above it."""
    out = []
    for p in rows:
        seen = []
        for i, q in enumerate(p):
            seen.append((seen[q] if q >= 0 else frozenset()) | {i})
        out.append(seen)
    return out


def _mask_words(rows):
    t = len(rows[0])
    words = [[[sum(1 << (j & 31) for j in seen if j >> 5 == w) for w in range(-(-t // 32))] for seen in seq]
             for seq in _ancestors(rows)]
    m = torch.tensor(words, dtype=torch.int64)
    return torch.where(m >= 1 << 31, m - (1 << 32), m).int().to(DEV)


def _table(rot, max_pos):
    """cos and sin [max_pos][rot/2][2]: base 10000, the lowest quarter of the frequencies slowed by 4 as for a long context."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    f = 10000.0 ** (-2 * i / rot) / torch.where(i >= rot * 3 / 8, 4.0, 1.0)
    a = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.stack((a.cos(), a.sin()), -1).float()


def prepare(case, seed):
    g = _gen(seed)
    c = case
    s = dict(case=case)
    if c["op"] == "rope":
        # query, key and value heads lie side by side in one projection's output
        hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
        x = _randn(g, c["tokens"], hq + 2 * hk, d)
        s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hk]
        first = int(torch.randint(0, max(1, c["max_pos"] - c["tokens"]), (1,), generator=g, device=DEV))
        s["pos"] = ((torch.arange(c["tokens"], device=DEV) + first) % c["max_pos"]).int()
        s["table"] = _table(c["rot"], c["max_pos"])
        return s
    if c["op"] == "verify":
        b, t, v = c["batch"], c["tokens"], c["vocab"]
        rows = _parents(c, seed)
        logits = torch.randn(b, t, v, generator=g, device=DEV) * 2.5
        s["logits"] = logits
        s["parents"] = torch.tensor(rows, dtype=torch.int32, device=DEV)
        at = torch.arange(b, device=DEV)
        par = s["parents"].long()
        if c["greedy"]:
            temp = torch.zeros(b, device=DEV)
        else:
            temp = torch.tensor([(0.7, 1.0, 1.0, 0.0)[i % 4] if b > 1 else 0.8 for i in range(b)], device=DEV)
        s["temp"] = temp
        t1 = torch.where(temp > 0, temp, 1.0)
        # The draft's logits are the target's with some noise; a node's children are drawn from the draft at the node.
        draft = logits + torch.randn(b, t, v, generator=g, device=DEV) * 0.8
        draft = torch.softmax(draft / t1[:, None, None], -1)
        tokens = torch.zeros(b, t, dtype=torch.int32, device=DEV)
        for i in range(1, t):
            e = torch.empty(b, v, device=DEV).exponential_(generator=g)
            drawn = (draft[at, par[:, i]] / e).argmax(-1)
            best = logits[at, par[:, i]].argmax(-1)
            easy = torch.rand(b, generator=g, device=DEV) < 0.6
            tokens[:, i] = torch.where((temp <= 0) & easy, best, drawn).int()
        s["tokens"] = tokens
        s["draft"] = None if c["greedy"] else draft
        s["u"] = None if c["greedy"] else torch.rand(b, t, generator=g, device=DEV)
        s["noise"] = None if c["greedy"] else torch.empty(b, v, device=DEV).exponential_(generator=g).clamp(min=1e-12)
        return s
    # a paged cache
    hk, d, p = c["kv_heads"], c["dim"], c["page"]
    s["pages"], n = _pages(c, seed)
    order = random.Random(seed).sample(range(c["batch"]), c["batch"])
    lens = _lengths(c)
    s["ctx"] = torch.tensor([lens[i] for i in order], dtype=torch.int32, device=DEV)
    for name in ("k", "v"):
        codes, scales, biases = [], [], []
        step = max(1, (1 << 26) // (hk * p * d))
        for lo in range(0, n, step):
            m = min(step, n - lo)
            x = torch.randn(m, hk, p, d, generator=g, device=DEV) if c["op"] == "attn" else torch.zeros(m, hk, p, d, device=DEV)
            a, sc, bi = _quantise(x.bfloat16().float(), c["kind"], c["group"])
            codes.append(a)
            scales.append(sc)
            biases.append(bi)
        s[name + "_pool"] = torch.cat(codes)
        s[name + "_scale"] = torch.cat(scales) if scales[0] is not None else None
        s[name + "_bias"] = torch.cat(biases) if biases[0] is not None else None
    if c["op"] == "kv":
        s["k"] = _randn(g, c["batch"], c["tokens"], hk, d)
        s["v"] = _randn(g, c["batch"], c["tokens"], hk, d, scale=0.3)
    else:
        s["q"] = _randn(g, c["batch"], c["tokens"], c["q_heads"], d, scale=2.0)
        s["mask"] = _mask_words(_parents(c, seed)) if c["tree"] else None
        s["scale"] = d ** -0.5
    if own:  # the handle that a program keeps beside its cache's tensors
        from hyper_connection_residual_call_gb300 import binding as B
        s["cache"] = B.KVCache(c["kind"], s["k_pool"], s["v_pool"], s["pages"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                               k_bias=s["k_bias"], v_bias=s["v_bias"], group=c["group"])
        if c["op"] == "attn":
            s["ws"] = B.tree_attention_workspace(c["batch"], c["tokens"], c["q_heads"], s["cache"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        from hyper_connection_residual_call_gb300 import binding as B
        if c["op"] == "rope":
            return B.hc_rope(s["q"], s["k"], s["pos"], s["table"], interleaved=c["interleaved"], inverse=c["inverse"])
        if c["op"] == "kv":
            B.hc_kv_write(s["k"], s["v"], s["cache"], s["ctx"])
            return B.hc_kv_read(s["cache"], s["ctx"], c["tokens"])
        if c["op"] == "attn":
            return B.hc_tree_attention(s["q"], s["cache"], s["ctx"], mask=s["mask"], scale=s["scale"], ws=s["ws"])
        return B.hc_verify(s["logits"], s["tokens"], s["parents"], s["temp"], draft_probs=s["draft"], u=s["u"],
                           noise=s["noise"])
    return {"rope": _plain_rope, "kv": _plain_kv, "attn": _plain_attn, "verify": _plain_verify}[c["op"]](s)


def _plain_rope(s):
    c = s["case"]
    cs = s["table"][s["pos"].long()][:, None]  # [N][1][rot/2][2]
    cos, sin = cs[..., 0], cs[..., 1]
    if c["inverse"]:
        sin = -sin
    r = c["rot"]

    def turn(x):
        y = x.float()
        if c["interleaved"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            z = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:r]
            z = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((z, y[..., r:]), -1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _slots(s, n):
    """Page and place within it of the n positions from each sequence's context length on: [B][n] each."""
    at = s["ctx"].long()[:, None] + torch.arange(n, device=s["ctx"].device)
    p = s["case"]["page"]
    return s["pages"].long().gather(1, at // p), at % p


def _plain_kv(s):
    c = s["case"]
    page, place = _slots(s, c["tokens"])
    out = []
    for name in ("k", "v"):
        for pool, x in zip((s[name + "_pool"], s[name + "_scale"], s[name + "_bias"]),
                           _quantise(s[name].float(), c["kind"], c["group"])):
            if pool is not None:
                pool[page, :, place] = x
        back = [None if pool is None else pool[page, :, place]
                for pool in (s[name + "_pool"], s[name + "_scale"], s[name + "_bias"])]
        out.append(_dequantise(*back, c["kind"], c["group"]).bfloat16())
    return tuple(out)


def _plain_attn(s):
    c = s["case"]
    b, t, hq, hk, d = c["batch"], c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
    pages = s["pages"].long()

    def rows(name):  # [B][Hk][L][D]
        parts = [None if s[name + x] is None else s[name + x][pages].transpose(1, 2).flatten(2, 3)
                 for x in ("_pool", "_scale", "_bias")]
        return _dequantise(*parts, c["kind"], c["group"])

    k, v = rows("k"), rows("v")
    at = torch.arange(k.shape[2], device=k.device)
    node = at - s["ctx"].long()[:, None]  # [B][L]: which drafted token a key is, negative in the context
    if s["mask"] is None:
        sees = node[:, None] <= torch.arange(t, device=k.device)[:, None]
    else:
        n = node.clamp(0, t - 1)
        word = s["mask"].long().gather(2, (n >> 5)[:, None].expand(-1, t, -1))
        sees = (((word >> (n & 31)[:, None]) & 1) > 0) & (node < t)[:, None] | (node < 0)[:, None]  # [B][T][L]
    q = s["q"].float().view(b, t, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    x = (q @ k.transpose(2, 3)).view(b, hk, t, hq // hk, -1) * s["scale"]
    x = torch.where(sees[:, None, :, None], x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    x = (x - m).exp()
    z = x.sum(-1, keepdim=True)
    out = ((x / z).flatten(2, 3) @ v).view(b, hk, t, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(b, t, hq, d)
    lse = (m + z.log())[..., 0].permute(0, 2, 1, 3).reshape(b, t, hq)
    return out.bfloat16(), lse


def _plain_verify(s):
    c = s["case"]
    logits, tokens, parents, temp = s["logits"], s["tokens"].long(), s["parents"].long(), s["temp"]
    b, t, v = logits.shape
    at = torch.arange(b, device=logits.device)
    greedy = temp <= 0
    t1 = torch.where(greedy, 1.0, temp)[:, None]
    m = logits.amax(-1)
    ids = torch.arange(v, device=logits.device)

    def first_best(x):
        return torch.where(x == x.amax(-1, keepdim=True), ids, v).amin(-1)

    cur = torch.zeros(b, dtype=torch.long, device=logits.device)
    count = torch.zeros_like(cur)
    path = torch.full((b, t), -1, dtype=torch.int32, device=logits.device)
    path[:, 0] = 0
    taken = torch.zeros(b, device=logits.device)  # how much of the draft was subtracted
    left = torch.ones(b, device=logits.device)  # the sum of what is left of the target

    def probs(cur):
        x = ((logits[at, cur] - m[at, cur][:, None]) / t1).exp()
        return x / x.sum(-1, keepdim=True)

    p = probs(cur)
    best = first_best(logits[at, cur])
    for i in range(1, t):  # a node's children come after it, in their order
        here = parents[:, i] == cur
        x = tokens[:, i]
        if c["greedy"]:
            ok = here & (x == best)
        else:
            q = s["draft"][at, cur]
            r = (p[at, x] - taken * q[at, x]).clamp(min=0)
            ok = here & torch.where(greedy, x == best, s["u"][:, i] * left * q[at, x] < r)
            no = here & ~ok
            less = taken + left
            rest = (p - less[:, None] * q).clamp(min=0).sum(-1)
            taken = torch.where(ok, 0.0, torch.where(no, less, taken))
            left = torch.where(ok, 1.0, torch.where(no, rest, left))
        cur = torch.where(ok, i, cur)
        count = count + ok
        path[at, count] = torch.where(ok, i, path[at, count].long()).int()
        p = probs(cur)
        best = first_best(logits[at, cur])
    if c["greedy"]:
        return count.int(), path, best.int()
    r = torch.where(taken[:, None] > 0, (p - taken[:, None] * s["draft"][at, cur]).clamp(min=0), p)
    r = torch.where(left[:, None] > 0, r, p)
    return count.int(), path, torch.where(greedy, best, first_best(r / s["noise"])).int()


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "kv": _exact_kv, "attn": _exact_attn, "verify": _exact_verify}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    r, inter = c["rot"], c["interleaved"]
    half = torch.arange(r // 2, device=DEV)
    i0, i1 = (2 * half, 2 * half + 1) if inter else (half, half + r // 2)
    z = torch.view_as_complex(s["table"].double()[s["pos"].long()])[:, None]
    z = z.conj() if c["inverse"] else z
    out = []
    for x in (s["q"], s["k"]):
        y = x.double()
        w = torch.complex(y[..., i0], y[..., i1]) * z
        y = y.clone()
        y[..., i0], y[..., i1] = w.real, w.imag
        out.append(y)
    return tuple(out)


def _two_to(e):
    """2**e in 64 bits for whole e (held in 64 bits): exact, which pow need not be."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _values64(x, kind, group):
    """What rows x (64 bits) come back as."""
    if kind == "bf16":
        return x
    if kind == "fp8":
        top = x.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(top / 448)).clamp(min=-117)
        e = torch.where(448 * _two_to(e - 1) >= top, e - 1, e).clamp(min=-117)
        e = torch.where(448 * _two_to(e) < top, e + 1, e)
        y = x / _two_to(e)
        ulp = _two_to((torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4).double())  # three bits after the first
        return torch.round(y / ulp) * ulp * _two_to(e)
    y = x.view(*x.shape[:-1], -1, group)
    b = y.amin(-1, keepdim=True)
    s = ((y.amax(-1, keepdim=True) - b) / 15).half().double()
    b = b.half().double()
    q = torch.round((y - b) / torch.where(s > 0, s, 1.0)).clamp(0, 15) * (s > 0)
    return (q * s + b).view(x.shape)


def _exact_kv(s):
    c = s["case"]
    return tuple(_values64(s[n].double(), c["kind"], c["group"]) for n in ("k", "v"))


def _exact_attn(s):
    c = s["case"]
    b, t, hq, hk, d, p = c["batch"], c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    g = hq // hk
    out = torch.empty(b, t, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(b, t, hq, dtype=torch.float64, device=DEV)

    def rows(name, i, h, n):
        ids = s["pages"][i, :-(-n // p)].long()
        x = s[name + "_pool"][ids, h].reshape(-1, s[name + "_pool"].shape[-1])[:n]
        if c["kind"] == "bf16":
            return x.double()
        sc = s[name + "_scale"][ids, h]
        if c["kind"] == "fp8":
            return x.view(torch.float8_e4m3fn).double() * _two_to(sc.reshape(-1, 1)[:n].long() - 127)
        sc = sc.reshape(-1, d // c["group"])[:n].double().repeat_interleave(c["group"], 1)
        bi = s[name + "_bias"][ids, h].reshape(-1, d // c["group"])[:n].double().repeat_interleave(c["group"], 1)
        q = torch.empty(n, d, dtype=torch.float64, device=DEV)
        q[:, 0::2], q[:, 1::2] = (x & 15).double(), (x >> 4).double()
        return q * sc + bi

    for i, ctx in enumerate(s["ctx"].tolist()):
        n = ctx + t
        hide = torch.zeros(t, n, dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            hide[:, ctx:] = torch.ones(t, t, dtype=torch.bool, device=DEV).triu(1)
        else:
            words = s["mask"][i].tolist()
            hide[:, ctx:] = torch.tensor([[not (words[r][j // 32] >> (j % 32)) & 1 for j in range(t)] for r in range(t)], device=DEV)
        for h in range(hk):
            x = torch.einsum("tgd,nd->tgn", s["q"][i, :, h * g:(h + 1) * g].double(), rows("k", i, h, n)) * s["scale"]
            x.masked_fill_(hide[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            out[i, :, h * g:(h + 1) * g] = torch.einsum("tgn,nd->tgd", (x - z[..., None]).exp(), rows("v", i, h, n))
            lse[i, :, h * g:(h + 1) * g] = z
    return out, lse


def _exact_verify(s):
    counts, paths, nexts = [], [], []
    parents, tokens = s["parents"].tolist(), s["tokens"].tolist()
    for i, temp in enumerate(s["temp"].tolist()):
        def target(node):
            x = s["logits"][i, node].double()
            if temp <= 0:
                y = torch.zeros_like(x)
                y[int((x == x.max()).nonzero()[0])] = 1
                return y
            return torch.softmax(x / temp, -1)

        path, r = [0], target(0)
        child = 1
        while child < len(parents[i]):
            if parents[i][child] == path[-1]:
                x = tokens[i][child]
                if temp <= 0:
                    ok = float(r[x]) > 0
                else:
                    q = s["draft"][i, path[-1]].double()
                    ok = float(s["u"][i, child]) * float(q[x]) < float(r[x])
                if ok:
                    path.append(child)
                    r = target(child)
                elif temp > 0:
                    rest = (r - q).clamp(min=0)
                    if float(rest.sum()) > 0:
                        r = rest / rest.sum()
            child += 1
        y = r if temp <= 0 else r / s["noise"][i].double()
        counts.append(len(path) - 1)
        paths.append(path + [-1] * (len(parents[i]) - len(path)))
        nexts.append(int((y == y.max()).nonzero()[0]))
    return (torch.tensor(counts, dtype=torch.int32), torch.tensor(paths, dtype=torch.int32), torch.tensor(nexts, dtype=torch.int32))
