"""Cases for the operators of a prompt's pass through a decoder and of the token after it: the norms of query and
key heads with their rotary positions, causal attention over packed prompts, the gated delta rule (a prompt in
chunks, a few tokens at a time), and the log probabilities of given tokens.

``run`` with ``own`` false computes each operator from elementary torch operations in 32 bits (long sums in 64);
with ``own`` true it makes the library's calls. ``exact`` computes the same results in 64 bits from the operators'
definitions.
"""
import math
import random

import torch

own = False
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One decoded token: every attention layer norms and turns its heads once (2560 = 20 heads of 128).
        dict(name="norm rope one token", op="rope", tokens=1, q_heads=20, kv_heads=4, dim=128, rot=128,
             interleaved=False, max_pos=32768),
        # A long prompt, an odd number of tokens: interleaved pairs, half of each head turned.
        dict(name="norm rope long prompt", op="rope", tokens=16381, q_heads=32, kv_heads=8, dim=128, rot=64,
             interleaved=True, max_pos=131072),
        # Many short prompts packed into one call (questions, a classifier's batch): most shorter than a tile.
        dict(name="attention short prompts", op="attn", seqs=48, longest=200, q_heads=16, kv_heads=2, dim=64),
        # A serving batch of ragged prompts.
        dict(name="attention batch", op="attn", seqs=8, longest=2048, q_heads=32, kv_heads=8, dim=128),
        # One long document.
        dict(name="attention long prompt", op="attn", seqs=1, longest=16384, q_heads=32, kv_heads=8, dim=128),
        # One sequence, one token: the smallest call, where latency counts.
        dict(name="delta one token", op="step", batch=1, tokens=1, k_heads=16, v_heads=32, dim=128, ragged=False),
        # A serving batch, a chain of drafted tokens each; sequences take part with one to four of them.
        dict(name="delta batch drafts", op="step", batch=64, tokens=4, k_heads=16, v_heads=32, dim=128, ragged=True),
        # A serving batch of ragged prompts that go on from a state, smaller heads.
        dict(name="delta batch prompts", op="delta", seqs=24, longest=1500, k_heads=8, v_heads=8, dim=64),
        # One long document.
        dict(name="delta long prompt", op="delta", seqs=1, longest=8192, k_heads=16, v_heads=32, dim=128),
        # One decoded token's log probability with its five best alternatives, the vocabulary of this library's own
        # exit, a part of it ruled out.
        dict(name="logprobs one row", op="logp", rows=1, vocab=32768, given=1, top=5, kind="fp32", ruled_out=0.3),
        # A prompt's tokens scored, with twenty alternatives each, over a large odd vocabulary.
        dict(name="logprobs prompt", op="logp", rows=2048, vocab=128001, given=1, top=20, kind="fp32", ruled_out=0.0),
        # Eight choices scored at every place, and the entropy; 16-bit logits, an odd vocabulary.
        dict(name="logprobs choices bf16", op="logp", rows=4099, vocab=65537, given=8, top=0, kind="bf16", ruled_out=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "step", "delta", "delta", "logp"])
    if op == "rope":
        dim, kv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 16381), q_heads=kv * rng.choice([1, 4, 5, 8][:3 if kv == 8 else 4]),
                    kv_heads=kv, dim=dim, rot=rng.choice([dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.5,
                    max_pos=rng.choice([32768, 131072]))
    if op == "attn":
        kv, seqs = rng.choice([1, 2, 4, 8]), _log(rng, 1, 48)
        return dict(op=op, seqs=seqs, longest=_log(rng, 1, int(16384 / seqs ** 0.5)), q_heads=kv * rng.choice([1, 3, 4]),
                    kv_heads=kv, dim=rng.choice([64, 128]))
    if op == "step":
        k = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, batch=_log(rng, 1, 64), tokens=rng.choice([1, 1, 2, 3, 4]), k_heads=k, v_heads=k * rng.choice([1, 2]),
                    dim=rng.choice([64, 128]), ragged=rng.random() < 0.5)
    if op == "delta":
        k, seqs = rng.choice([1, 2, 4, 8, 16]), _log(rng, 1, 24)
        return dict(op=op, seqs=seqs, longest=_log(rng, 1, 8192 // seqs), k_heads=k, v_heads=k * rng.choice([1, 2]),
                    dim=rng.choice([64, 128]))
    rows = _log(rng, 1, 4099)
    return dict(op=op, rows=rows, vocab=_log(rng, 1000, min(128001, 2048 * 128001 // rows)), given=rng.choice([1, 1, 2, 8]),
                top=rng.choice([0, 1, 5, 20]), kind=rng.choice(["fp32", "bf16"]), ruled_out=rng.choice([0.0, 0.3]))


def _lengths(case):
    """The prompts' lengths: one has all of ``longest``, the others from an eighth of it up, the shortest first."""
    s, n = case["seqs"], case["longest"]
    return [n if s == 1 else max(1, n // 8 + (n - n // 8) * i // (s - 1)) for i in range(s)]


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * (c["q_heads"] + c["kv_heads"])
        return dict(bytes=n * c["dim"] * 4 + c["tokens"] * (c["rot"] * 4 + 4) + 4 * c["dim"], flops=n * (4 * c["dim"] + 3 * c["rot"]))
    if c["op"] == "attn":
        lens = _lengths(c)
        return dict(bytes=sum(lens) * (4 * c["dim"] * (c["q_heads"] + c["kv_heads"]) + 4 * c["q_heads"]),
                    flops=sum(4 * (n * (n + 1) // 2) * c["q_heads"] * c["dim"] for n in lens))
    if c["op"] in ("step", "delta"):
        d, hk, hv = c["dim"], c["k_heads"], c["v_heads"]
        seqs = c["batch"] if c["op"] == "step" else c["seqs"]
        tokens = sum(_counts(c)) if c["op"] == "step" else sum(_lengths(c))
        # a token: q and k, v and the result, decay and beta; a sequence: its state in and out. Three products of a
        # vector with the state each token, and the state's decay.
        return dict(bytes=tokens * (4 * d * (hk + hv) + 8 * hv) + seqs * hv * d * d * 8, flops=tokens * hv * 7 * d * d)
    size = 4 if c["kind"] == "fp32" else 2
    return dict(bytes=c["rows"] * (c["vocab"] * size + 8 * c["given"] + 8 * c["top"] + 4), flops=c["rows"] * c["vocab"] * 4)


def _counts(case):
    """How many of its tokens each sequence of a step takes."""
    t = case["tokens"]
    return [1 + (i * 7 + 3) % t if case["ragged"] else t for i in range(case["batch"])]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)
    return g


def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).bfloat16()


def _table(rot, max_pos):
    """cos and sin [max_pos][rot/2][2], base 10000."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    a = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (-2 * i / rot)
    return torch.stack((a.cos(), a.sin()), -1).float()


def _starts(case, seed):
    """The prompts' lengths in an order of their own, and the packed rows where they start, [S + 1]."""
    lens = _lengths(case)
    random.Random(seed * 13 + 1).shuffle(lens)
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return lens, torch.tensor(at, dtype=torch.int32, device=DEV)


def _gates(g, hv, *lead):
    """Log decays and betas as a gated layer makes them: -A softplus(a + b) with A in [1, 16] a head, sigmoid(x)."""
    rate = torch.rand(hv, generator=g, device=DEV) * 15 + 1
    bias = torch.log(torch.expm1(torch.exp(torch.rand(hv, generator=g, device=DEV) * math.log(100.0) + math.log(1e-3))))
    decay = -rate * torch.nn.functional.softplus(torch.randn(*lead, hv, generator=g, device=DEV) * 0.5 + bias)
    return decay.float(), torch.sigmoid(torch.randn(*lead, hv, generator=g, device=DEV))


def prepare(case, seed):
    g = _gen(seed)
    c = case
    s = dict(case=case)
    if c["op"] == "rope":
        # query, key and value heads lie side by side in one projection's output
        hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
        x = _randn(g, c["tokens"], hq + 2 * hk, d, scale=1.7)
        s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hk]
        s["qw"], s["kw"] = ((1 + 0.3 * torch.randn(d, generator=g, device=DEV)).bfloat16() for _ in range(2))
        first = int(torch.randint(0, max(1, c["max_pos"] - c["tokens"]), (1,), generator=g, device=DEV))
        s["pos"] = ((torch.arange(c["tokens"], device=DEV) + first) % c["max_pos"]).int()
        s["table"] = _table(c["rot"], c["max_pos"])
        return s
    if c["op"] == "attn":
        hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
        s["lens"], s["starts"] = _starts(c, seed)
        n = sum(s["lens"])
        s["q"] = _randn(g, n, hq, d, scale=1.5)
        kv = _randn(g, n, 2 * hk, d)
        s["k"], s["v"] = kv[:, :hk], kv[:, hk:]
        return s
    if c["op"] in ("step", "delta"):
        hk, hv, d = c["k_heads"], c["v_heads"], c["dim"]
        if c["op"] == "step":
            lead, seqs = (c["batch"], c["tokens"]), c["batch"]
            counts = _counts(c)
            random.Random(seed * 13 + 1).shuffle(counts)
            s["counts"] = torch.tensor(counts, dtype=torch.int32, device=DEV) if c["ragged"] else None
            s["out"] = torch.zeros(*lead, hv, d, dtype=torch.bfloat16, device=DEV)  # tokens past a count stay as they are
        else:
            s["lens"], s["starts"] = _starts(c, seed)
            lead, seqs = (sum(s["lens"]),), c["seqs"]
        x = _randn(g, *lead, 2 * hk + hv, d)
        s["q"], s["k"], s["v"] = x[..., :hk, :], x[..., hk:2 * hk, :], x[..., 2 * hk:, :]
        s["decay"], s["beta"] = _gates(g, hv, *lead)
        s["state"] = torch.randn(seqs, hv, d, d, generator=g, device=DEV) * 0.1
        s["state_out"] = torch.empty_like(s["state"])
        if own and c["op"] == "delta":
            from hyper_connection_residual_call_gb300 import binding as B
            s["ws"] = B.delta_prompt_workspace(lead[0], seqs, hk, hv, d, device=DEV)
        return s
    rows, v = c["rows"], c["vocab"]
    # a few words stand out, as a trained model's do: the scores' spread differs from row to row
    spread = torch.rand(rows, 1, generator=g, device=DEV) * 4 + 0.5
    x = torch.randn(rows, v, generator=g, device=DEV) * spread
    s["tokens"] = torch.randint(0, v, (rows, c["given"]), generator=g, device=DEV, dtype=torch.int32)
    if c["ruled_out"]:
        out = torch.rand(rows, v, generator=g, device=DEV) < c["ruled_out"]
        out[:, v // 2] = False
        x = x.masked_fill_(out, float("-inf"))
    s["logits"] = x if c["kind"] == "fp32" else x.bfloat16()
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        from hyper_connection_residual_call_gb300 import binding as B
        if c["op"] == "rope":
            return B.hc_qk_norm_rope(s["q"], s["k"], s["pos"], s["table"], s["qw"], s["kw"], eps=EPS, interleaved=c["interleaved"])
        if c["op"] == "attn":
            return B.hc_prompt_attention(s["q"], s["k"], s["v"], s["starts"])
        if c["op"] == "step":
            return B.hc_delta_step(s["q"], s["k"], s["v"], s["decay"], s["beta"], s["state"], counts=s["counts"], norm_eps=EPS,
                                   out=s["out"], state_out=s["state_out"])
        if c["op"] == "delta":
            return B.hc_delta_prompt(s["q"], s["k"], s["v"], s["decay"], s["beta"], s["state"], s["starts"], norm_eps=EPS,
                                     state_out=s["state_out"], ws=s["ws"])
        return tuple(x for x in B.hc_logprobs(s["logits"], s["tokens"], top=c["top"]) if x is not None)
    return {"rope": _plain_rope, "attn": _plain_attn, "step": _plain_step, "delta": _plain_delta, "logp": _plain_logp}[c["op"]](s)


def _plain_rope(s):
    c = s["case"]
    cs = s["table"][s["pos"].long()][:, None]  # [N][1][rot/2][2]
    cos, sin = cs[..., 0], cs[..., 1]
    r = c["rot"]

    def turn(x, w):
        y = x.float()
        y = y / ((y * y).mean(-1, keepdim=True) + EPS).sqrt() * w.float()
        if c["interleaved"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            z = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:r]
            z = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((z, y[..., r:]), -1).to(x.dtype)

    return turn(s["q"], s["qw"]), turn(s["k"], s["kw"])


def _plain_attn(s):
    c = s["case"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
    at = 0
    for n in s["lens"]:
        q = s["q"][at:at + n].float().transpose(0, 1).unflatten(0, (hk, hq // hk))  # [Hk][G][n][D]
        k, v = (s[x][at:at + n].float().transpose(0, 1)[:, None] for x in "kv")
        for lo in range(0, n, 2048):  # the scores of 2048 rows at a time
            hi = min(n, lo + 2048)
            x = q[:, :, lo:hi] @ k[:, :, :hi].transpose(2, 3) * d ** -0.5
            sees = torch.arange(hi, device=x.device) <= torch.arange(lo, hi, device=x.device)[:, None]
            x = torch.where(sees, x, float("-inf"))
            m = x.amax(-1, keepdim=True)
            x = (x - m).exp()
            z = x.sum(-1, keepdim=True)
            out[at + lo:at + hi] = (x @ v[:, :, :hi] / z).flatten(0, 1).transpose(0, 1).to(out.dtype)
            lse[at + lo:at + hi] = (m + z.log())[..., 0].flatten(0, 1).transpose(0, 1)
        at += n
    return out, lse


def _plain_delta_rows(q, k, v, decay, beta, state, counts):
    """The recurrence over [B, T] tokens, of which a sequence takes its ``counts``; 32 bits. Returns (out, state)."""
    b, t, hv, d = v.shape

    def heads(x):  # a value head's key head; rows of length one
        x = x.float().repeat_interleave(hv // x.shape[2], 2)
        return x / ((x * x).sum(-1, keepdim=True) + EPS).sqrt()

    q, k, v = heads(q) * d ** -0.5, heads(k), v.float()
    on = torch.arange(t, device=v.device) < counts[:, None]
    keep = torch.where(on[..., None], decay, 0.0).exp()[..., None, None]  # a token that is not taken changes nothing
    beta = torch.where(on[..., None], beta, 0.0)[..., None]
    out = torch.empty_like(v)
    for i in range(t):
        state = state * keep[:, i]
        u = (v[:, i] - (k[:, i, :, None] @ state)[:, :, 0]) * beta[:, i]
        state = state + k[:, i, :, :, None] * u[:, :, None]
        out[:, i] = (q[:, i, :, None] @ state)[:, :, 0]
    return out.bfloat16(), state


def _plain_step(s):
    c = s["case"]
    counts = s["counts"] if s["counts"] is not None else torch.full((c["batch"],), c["tokens"], device=DEV)
    out, state = _plain_delta_rows(s["q"], s["k"], s["v"], s["decay"], s["beta"], s["state"], counts)
    on = torch.arange(c["tokens"], device=out.device) < counts[:, None]
    return torch.where(on[..., None, None], out, s["out"]), state


def _plain_delta(s):
    lens = torch.tensor(s["lens"], device=DEV)
    at = torch.arange(max(s["lens"]), device=DEV)
    rows = (s["starts"][:-1].long()[:, None] + at).clamp(max=sum(s["lens"]) - 1)  # padded to the longest
    out, state = _plain_delta_rows(*(s[x][rows] for x in ("q", "k", "v", "decay", "beta")), s["state"], lens)
    return out[at < lens[:, None]], state


def _plain_logp(s):
    c = s["case"]
    logits, tokens = s["logits"], s["tokens"].long()
    ids = torch.arange(c["vocab"], device=logits.device)
    step = max(1, (1 << 26) // c["vocab"])  # rows at a time
    parts = []
    for lo in range(0, c["rows"], step):
        x = logits[lo:lo + step].float()
        y = x - x.amax(-1, keepdim=True)
        e = y.exp()
        z = e.sum(-1, keepdim=True, dtype=torch.float64)
        log_z = z.log()
        entropy = log_z - torch.where(e > 0, y * e, 0.0).sum(-1, keepdim=True, dtype=torch.float64) / z
        part = [(y.gather(1, tokens[lo:lo + step]).double() - log_z).float(), entropy[:, 0].float()]
        if c["top"]:
            best = []
            left = x.clone()
            free = torch.ones_like(x, dtype=torch.bool)
            for _ in range(c["top"]):
                m = left.amax(-1, keepdim=True)
                i = torch.where((left == m) & free, ids, c["vocab"]).amin(-1, keepdim=True)
                best.append(i)
                left.scatter_(1, i, float("-inf"))
                free.scatter_(1, i, False)
            best = torch.cat(best, 1)
            part += [best.int(), (y.gather(1, best).double() - log_z).float()]
        parts.append(part)
    return tuple(torch.cat(x) for x in zip(*parts))


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "step": _exact_step, "delta": _exact_delta, "logp": _exact_logp}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    r = c["rot"]
    half = torch.arange(r // 2, device=DEV)
    i0, i1 = (2 * half, 2 * half + 1) if c["interleaved"] else (half, half + r // 2)
    z = torch.view_as_complex(s["table"].double()[s["pos"].long()])[:, None]
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.double()
        y = y * (torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / c["dim"] + EPS) ** -0.5 * w.double()
        t = torch.complex(y[..., i0], y[..., i1]) * z
        y[..., i0], y[..., i1] = t.real, t.imag
        out.append(y)
    return tuple(out)


def _exact_attn(s):
    c = s["case"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for first, last in zip(s["starts"].tolist()[:-1], s["starts"].tolist()[1:]):
        for h in range(hq):
            k, v = (s[x][first:last, h * hk // hq].double() for x in "kv")
            for lo in range(first, last, 4096):
                n = min(last, lo + 4096)
                x = torch.einsum("td,nd->tn", s["q"][lo:n, h].double(), k[:n - first]) / math.sqrt(d)
                x.masked_fill_(torch.ones(x.shape, dtype=torch.bool, device=DEV).triu_(lo - first + 1), -math.inf)
                z = torch.logsumexp(x, -1)
                out[lo:n, h] = (x - z[:, None]).exp_() @ v[:n - first]
                lse[lo:n, h] = z
    return out, lse


def _exact_chunks(q, k, v, decay, beta, state):
    """One sequence's tokens [T] from ``state`` [Hv][D][D], 64 at a time, each chunk's updates from one triangular system."""
    t, hv, d = v.shape
    g = hv // q.shape[1]
    unit = lambda x: (x / (x.square().sum(-1, keepdim=True) + EPS).sqrt()).repeat_interleave(g, 1).transpose(0, 1)  # noqa: E731
    q, k = unit(q.double()) / math.sqrt(d), unit(k.double())  # [Hv][T][D]
    v, decay, beta = v.double().transpose(0, 1), decay.double().T, beta.double().T
    outs = []
    for lo in range(0, t, 64):
        sl = slice(lo, min(t, lo + 64))
        qc, kc, vc, b = q[:, sl], k[:, sl], v[:, sl], beta[:, sl, None]
        total = decay[:, sl].cumsum(-1)
        apart = (total[:, :, None] - total[:, None]).tril().exp().tril()
        system = (kc @ kc.transpose(1, 2) * apart).tril(-1) * b
        right = b * (vc - total.exp()[..., None] * (kc @ state))
        u = torch.linalg.solve_triangular(system, right, upper=False, unitriangular=True)
        outs.append(total.exp()[..., None] * (qc @ state) + (qc @ kc.transpose(1, 2) * apart) @ u)
        state = total[:, -1, None, None].exp() * state + (kc * (total[:, -1:] - total).exp()[..., None]).transpose(1, 2) @ u
    return torch.cat(outs, 1).transpose(0, 1), state


def _exact_step(s):
    c = s["case"]
    out, state = s["out"].double(), s["state"].double()
    for i, n in enumerate(s["counts"].tolist() if s["counts"] is not None else [c["tokens"]] * c["batch"]):
        out[i, :n], state[i] = _exact_chunks(*(s[x][i, :n] for x in ("q", "k", "v", "decay", "beta")), state[i])
    return out, state


def _exact_delta(s):
    out, state = torch.empty(s["v"].shape, dtype=torch.float64, device=DEV), s["state"].double()
    at = s["starts"].tolist()
    for i, (lo, hi) in enumerate(zip(at[:-1], at[1:])):
        out[lo:hi], state[i] = _exact_chunks(*(s[x][lo:hi] for x in ("q", "k", "v", "decay", "beta")), state[i])
    return out, state


def _exact_logp(s):
    c = s["case"]
    step = max(1, (1 << 25) // c["vocab"])
    parts = []
    for lo in range(0, c["rows"], step):
        x = torch.log_softmax(s["logits"][lo:lo + step].double(), -1)
        part = [x.gather(1, s["tokens"][lo:lo + step].long()), -torch.xlogy(x.exp(), x.exp()).sum(-1)]
        if c["top"]:
            order = torch.sort(s["logits"][lo:lo + step].float(), dim=-1, descending=True, stable=True).indices[:, :c["top"]]
            part += [order.int(), x.gather(1, order)]
        parts.append(part)
    return tuple(torch.cat(x) for x in zip(*parts))
