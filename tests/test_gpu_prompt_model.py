"""The operators of a prompt's pass and of the tokens after it together, as a decoder runs them in hc_stack's
sublayers: packed prompts (head norms with rotary positions, attention, the delta rule in chunks), then drafted
tokens over the cache and the states, and the log probabilities of what was taken. And each operator captured
into a graph, on another stream, beside another call of itself, and its refusals in Python."""
import pytest
import torch

from gpu_common import require_gpu
from hyper_connection_residual_call_gb300 import binding as B, inputs

pytestmark = pytest.mark.gpu

H, C, L, V = 256, 4, 64, 512
HQ, HK, DH = 8, 2, 64      # attention's heads
DK, DV, DD = 2, 4, 64      # the delta rule's
KINDS = ("delta", "attention", "delta", "attention")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    B.device_status()


class Decoder:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        draw = lambda rows, cols: (torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).bfloat16()  # noqa: E731
        n = len(KINDS)
        self.hc = [tuple(inputs.make_hc_weights(H, C, L, seed, 2 * i + j).to("cuda") for j in range(2)) for i in range(n)]
        self.final = inputs.make_hc_weights(H, C, L, seed, 2 * n, with_inject=False).to("cuda")
        self.proj = [draw((HQ + 2 * HK) * DH if kind == "attention" else (2 * DK + DV) * DD + 2 * DV, H) for kind in KINDS]
        self.out = [draw(H, HQ * DH if kind == "attention" else DV * DD) for kind in KINDS]
        self.norms = [(1 + 0.1 * torch.randn(2, DH, generator=g, device="cuda")).bfloat16() for _ in KINDS]
        self.up, self.down = [draw(4 * H, H) for _ in KINDS], [draw(H, 2 * H) for _ in KINDS]
        self.emb, self.lm_head = torch.randn(V, H, generator=g, device="cuda").bfloat16(), draw(V, H)
        self.rope = B.rope_table(1024, DH, 10000.0)

    def cache(self, batch, max_len, page=16):
        per = -(-max_len // page)
        table = torch.arange(batch * per, device="cuda").int().view(batch, per).flip(0).contiguous()
        return [B.kv_cache("bf16", batch * per, HK, page, DH, table) if kind == "attention" else
                torch.zeros(batch, DV, DD, DD, device="cuda") for kind in KINDS]

    def run(self, tokens, attention, delta):
        """fp32 logits of ``tokens`` (any shape), with the given forms of the two sublayers."""
        lead = tokens.shape

        def sublayer(layer, which, t0, mixed):
            if which == 1:
                gate, x = (mixed @ self.up[layer].T).chunk(2, -1)
                return (torch.nn.functional.silu(gate) * x) @ self.down[layer].T
            x = mixed @ self.proj[layer].T
            if KINDS[layer] == "attention":
                q, k, v = x.view(*lead, HQ + 2 * HK, DH).split((HQ, HK, HK), -2)
                out = attention(layer, q, k, v)
            else:
                heads, gates = x.split(((2 * DK + DV) * DD, 2 * DV), -1)
                q, k, v = heads.unflatten(-1, (-1, DD)).view(*lead, -1, DD).split((DK, DK, DV), -2)
                gates = gates.float().view(*lead, 2, DV)
                out = delta(layer, q, k, v, -torch.nn.functional.softplus(gates[..., 0, :]), torch.sigmoid(gates[..., 1, :]))
            return out.reshape(-1, self.out[layer].shape[1]) @ self.out[layer].T

        _, raw = B.hc_stack(self.emb[tokens.long()].view(-1, H), self.hc, self.final, sublayer, C=C)
        _, logits = B.hc_exit_logits(raw, self.final, self.lm_head, H=H, C=C)
        return logits.view(*lead, V)

    def prompts(self, tokens, starts, positions, memory, padded=None):
        """The packed prompts' logits [N, V]. ``memory``: caches and states, taken up to the prompts' ends;
        ``padded`` [B, T]: each sequence's rows, and behind them any."""
        zero = None if padded is None else torch.zeros(padded.shape[0], dtype=torch.int32, device="cuda")

        def attention(layer, q, k, v):
            q, k = B.hc_qk_norm_rope(q, k, positions, self.rope, self.norms[layer][0], self.norms[layer][1])
            if padded is not None:  # what lies behind a sequence is overwritten by its next tokens
                B.hc_kv_write(k[padded], v[padded], memory[layer], zero)
            return B.hc_prompt_attention(q, k, v, starts)[0]

        def delta(layer, q, k, v, decay, beta):
            return B.hc_delta_prompt(q, k, v, decay, beta, memory[layer], starts)[0]

        return self.run(tokens, attention, delta)

    def drafts(self, tokens, ctx, memory):
        """Logits [B, T, V] of a chain of tokens after ctx, and a function that moves the states on by counts."""
        B_, T = tokens.shape
        positions = ctx[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")
        taken = []

        def attention(layer, q, k, v):
            q, k = B.hc_qk_norm_rope(q, k, positions, self.rope, self.norms[layer][0], self.norms[layer][1])
            B.hc_kv_write(k, v, memory[layer], ctx)
            return B.hc_tree_attention(q, memory[layer], ctx)[0]

        def delta(layer, *args):
            taken.append((args, memory[layer]))
            return B.hc_delta_step(*args, memory[layer], state_out=torch.empty_like(memory[layer]))[0]

        def accept(counts):
            for args, state in taken:
                B.hc_delta_step(*args, state, counts=counts)

        return self.run(tokens, attention, delta), accept


@pytest.fixture(scope="module")
def model(_gpu):
    return Decoder()


def packed(lens):
    starts = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int()
    positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])
    return starts.cuda(), positions.cuda()


def test_tokens_after_packed_prompts(model):
    """Prompts in one pass, then drafted chains of which some tokens are taken, against one packed pass over the
    whole sequences. The two passes differ by the roundings of bf16 activations: some 70 in a row, each off by
    2^-9 / sqrt(3) of its value on the whole, 0.01 of a logit's standard deviation of about 1, and the largest of
    the 10^4 logits compared by 4.5 times that. A layer can double it, so 0.15 is allowed; a token missed or a
    state of another step changes logits by their standard deviation."""
    lens, T = [70, 1, 130, 5], 3
    counts = [[1, 3, 2, 1], [3, 1, 3, 2], [2, 2, 1, 3]]  # tokens of the chain that are taken, step by step
    rng = torch.Generator().manual_seed(7)
    whole = [torch.randint(V, (n + sum(c[i] for c in counts) + T,), generator=rng).int() for i, n in enumerate(lens)]

    starts, positions = packed(lens)
    padded = torch.tensor([[min(int(starts[i]) + t, sum(lens) - 1) for t in range(max(lens))] for i in range(len(lens))]).cuda()
    memory = model.cache(len(lens), max(map(len, whole)) + T)
    tokens = torch.cat([w[:n] for w, n in zip(whole, lens)]).cuda()
    first = model.prompts(tokens, starts, positions, memory, padded)
    got = [[first[int(starts[i]):int(starts[i]) + n]] for i, n in enumerate(lens)]
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for c in counts:
        # only the tokens taken are the sequence's; those behind them are others, and leave nothing behind
        chain = torch.stack([torch.cat([w[int(n):int(n) + k], (w[int(n) + k:int(n) + T] + 1) % V]) for w, n, k in zip(whole, ctx.cpu(), c)]).cuda()
        logits, accept = model.drafts(chain.int(), ctx, memory)
        counts_d = torch.tensor(c, dtype=torch.int32, device="cuda")
        accept(counts_d)
        for i, k in enumerate(c):
            got[i].append(logits[i, :k])
        ctx = ctx + counts_d

    whole = [w[:int(n)] for w, n in zip(whole, ctx.cpu())]
    starts2, positions2 = packed([len(w) for w in whole])
    fresh = model.cache(len(lens), max(map(len, whole)))
    everything = torch.cat(whole).cuda()
    want = model.prompts(everything, starts2, positions2, fresh)
    got = torch.cat([torch.cat(g) for g in got])
    assert float(want.std()) > 0.3
    assert float((got - want).abs().max()) <= 0.15
    for kind, a, z in zip(KINDS, memory, fresh):
        if kind == "delta":  # the states, up to the same roundings
            assert float((a - z).abs().max()) <= 0.15 * float(z.abs().max())
    # what the next tokens' probabilities were: the logits' difference twice, in the token's and in the sum's
    after = everything.roll(-1).view(-1, 1).contiguous()
    for x, y in zip(B.hc_logprobs(got, after, top=4)[:2], B.hc_logprobs(want, after, top=4)[:2]):
        assert float((x - y).abs().max()) <= 0.3 * max(1.0, float(y.abs().max()) / 4)
    lp = torch.log_softmax(got.double(), -1)
    ids, top = B.hc_logprobs(got, None, top=4)[2:]
    assert torch.equal(ids.long(), lp.topk(4, -1).indices)
    assert float((top.double() - lp.topk(4, -1).values).abs().max()) <= 1e-5
    assert B.device_status() == B.TS_OK


def test_a_captured_pass_is_the_eager_one(model):
    lens = [40, 0, 129, 3]
    starts, positions = packed(lens)
    tokens = torch.randint(V, (sum(lens),), generator=torch.Generator().manual_seed(1)).int().cuda()
    memory = model.cache(len(lens), 8)
    eager = model.prompts(tokens, starts, positions, memory)
    states = [m.clone() for m in memory if isinstance(m, torch.Tensor)]
    graph = torch.cuda.CUDAGraph()
    for m in memory:
        if isinstance(m, torch.Tensor):
            m.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        replayed = model.prompts(tokens, starts, positions, memory)
        lp, entropy, ids, top = B.hc_logprobs(replayed, tokens.view(-1, 1), top=3)
    for _ in range(2):
        for m in memory:
            if isinstance(m, torch.Tensor):
                m.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(replayed, eager)
        for a, z in zip((m for m in memory if isinstance(m, torch.Tensor)), states):
            assert torch.equal(a, z)
    # other lengths, in the same buffers: what is captured reads them at replay
    starts2, positions2 = packed([3, 100, 9, 60])
    starts.copy_(starts2)
    positions.copy_(positions2)
    for m in memory:
        if isinstance(m, torch.Tensor):
            m.zero_()
    graph.replay()
    want = model.prompts(tokens, starts2, positions2, model.cache(4, 8))
    assert torch.equal(replayed, want)
    for a, z in zip((lp, entropy, ids, top), B.hc_logprobs(want, tokens.view(-1, 1), top=3)):
        assert torch.equal(a, z)
    assert B.device_status() == B.TS_OK


def calls():
    """Each operator on inputs of its own: name -> a function of no arguments that returns its results."""
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n, lens = 333, [200, 0, 100, 33]
    starts, positions = packed(lens)
    table = B.rope_table(512, 64, 10000.0)
    q, k, v = r(n, 6, 64).bfloat16(), r(n, 2, 64).bfloat16(), r(n, 2, 64).bfloat16()
    w = r(2, 64).bfloat16()
    dq, dk, dv = r(n, 2, 128).bfloat16(), r(n, 2, 128).bfloat16(), r(n, 4, 128).bfloat16()
    decay, beta = -r(n, 4).abs(), torch.sigmoid(r(n, 4))
    state = r(4, 4, 128, 128)
    logits, chosen = r(n, 5000), torch.randint(5000, (n, 2), generator=g, device="cuda", dtype=torch.int32)
    step = [x[:12].view(4, 3, *x.shape[1:]) for x in (dq, dk, dv, decay, beta)]
    return {
        "norms": lambda s=None: B.hc_qk_norm_rope(q, k, positions, table, w[0], w[1], stream=s),
        "attention": lambda s=None: B.hc_prompt_attention(q, k, v, starts, stream=s),
        "delta step": lambda s=None: B.hc_delta_step(*step, state, state_out=torch.empty_like(state), stream=s),
        "delta prompt": lambda s=None: B.hc_delta_prompt(dq, dk, dv, decay, beta, state, starts, state_out=torch.empty_like(state), stream=s),
        "log probabilities": lambda s=None: B.hc_logprobs(logits, chosen, top=8, stream=s),
        "one row's": lambda s=None: B.hc_logprobs(logits[:1], chosen[:1], top=8, stream=s),
    }


@pytest.mark.parametrize("name", list(("norms", "attention", "delta step", "delta prompt", "log probabilities", "one row's")))
def test_streams_and_graphs(name):
    """The same bits on a stream that is given, on one that is current, in a graph's replay, and from two calls of
    it at once, each with results and workspace of its own."""
    call = calls()[name]
    want = call()
    same = lambda got: all(torch.equal(a, z) for a, z in zip(got, want))  # noqa: E731
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got = call(one)
    one.synchronize()
    assert same(got)
    with torch.cuda.stream(two):
        got = call()
    two.synchronize()
    assert same(got)
    many = [call(s) for _ in range(4) for s in (one, two)]
    torch.cuda.synchronize()
    assert all(map(same, many))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
        again = call()
    for _ in range(2):
        for x in (*got, *again):
            if x is not None:
                x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got) and same(again)
    assert B.device_status() == B.TS_OK


def refusals():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    f, i = torch.float32, torch.int32
    q, k, v, starts = z(8, 4, 64), z(8, 2, 64), z(8, 2, 64), z(3, dt=i)
    pos, table, w = z(8, dt=i), B.rope_table(16, 64, 10000.0), z(64)
    gate, state = z(8, 2, dt=f), z(2, 2, 64, 64, dt=f)
    step = (z(2, 4, 2, 64), z(2, 4, 2, 64), z(2, 4, 2, 64), z(2, 4, 2, dt=f), z(2, 4, 2, dt=f), state)
    dp = (k, k.clone(), v, gate, gate.clone(), state, starts)
    x = z(4, 100, dt=f)

    def swap(args, at, new):
        return (*args[:at], new, *args[at + 1:])

    yield "norms: fp32 q", lambda: B.hc_qk_norm_rope(q.float(), k, pos, table, w, w)
    yield "norms: k of other rows", lambda: B.hc_qk_norm_rope(q, k[:7], pos, table, w, w)
    yield "norms: k's weight missing", lambda: B.hc_qk_norm_rope(q, k, pos, table, w)
    yield "norms: weight of another size", lambda: B.hc_qk_norm_rope(q, k, pos, table, z(32), w)
    yield "norms: 64-bit positions", lambda: B.hc_qk_norm_rope(q, k, pos.long(), table, w, w)
    yield "norms: positions of other tokens", lambda: B.hc_qk_norm_rope(q, k, pos[:7].contiguous(), table, w, w)
    yield "norms: a CPU tensor", lambda: B.hc_qk_norm_rope(q, k, pos, table, w.cpu(), w)
    yield "norms: results of another size", lambda: B.hc_qk_norm_rope(q, k, pos, table, w, w, q_out=z(8, 4, 32))
    yield "attention: heads that do not divide", lambda: B.hc_prompt_attention(z(8, 3, 64), k, v, starts)
    yield "attention: D of 96", lambda: B.hc_prompt_attention(z(8, 4, 96), z(8, 2, 96), z(8, 2, 96), starts)
    yield "attention: v of other heads", lambda: B.hc_prompt_attention(q, k, z(8, 1, 64), starts)
    yield "attention: fp16", lambda: B.hc_prompt_attention(q.half(), k.half(), v.half(), starts)
    yield "attention: starts of two dimensions", lambda: B.hc_prompt_attention(q, k, v, starts.view(1, 3))
    yield "attention: starts on the CPU", lambda: B.hc_prompt_attention(q, k, v, starts.cpu())
    yield "attention: elements with a stride", lambda: B.hc_prompt_attention(z(8, 4, 128)[..., ::2], k, v, starts)
    yield "attention: out of another type", lambda: B.hc_prompt_attention(q, k, v, starts, out=z(8, 4, 64, dt=f))
    yield "attention: out over q", lambda: B.hc_prompt_attention(q, k, v, starts, out=q)
    yield "attention: scale of NaN", lambda: B.hc_prompt_attention(q, k, v, starts, scale=float("nan"))
    for name, fn, args in (("step", B.hc_delta_step, step), ("prompt", B.hc_delta_prompt, dp)):
        a0 = args[0]
        yield f"delta {name}: k of another shape", lambda fn=fn, args=args, a0=a0: fn(*swap(args, 1, a0[..., :1, :]))
        yield f"delta {name}: bf16 gates", lambda fn=fn, args=args: fn(*swap(args, 3, args[3].bfloat16()))
        yield f"delta {name}: a state of another head count", lambda fn=fn, args=args: fn(*swap(args, 5, z(2, 1, 64, 64, dt=f)))
        yield f"delta {name}: bf16 state", lambda fn=fn, args=args: fn(*swap(args, 5, state.bfloat16()))
        yield f"delta {name}: out over v", lambda fn=fn, args=args: fn(*args, out=args[2])
        yield f"delta {name}: eps of NaN", lambda fn=fn, args=args: fn(*args, norm_eps=float("nan"))
        both = z(3, 2, 64, 64, dt=f)
        yield f"delta {name}: state_out a row beside state", lambda fn=fn, args=args, both=both: fn(*swap(args, 5, both[:2]), state_out=both[1:])
    yield "delta step: counts of another batch", lambda: B.hc_delta_step(*step, counts=z(3, dt=i))
    yield "delta prompt: a workspace too small", lambda: B.hc_delta_prompt(*dp, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    yield "log probabilities: fp16", lambda: B.hc_logprobs(x.half())
    yield "log probabilities: a CPU tensor", lambda: B.hc_logprobs(x.cpu())
    yield "log probabilities: 33 alternatives", lambda: B.hc_logprobs(x, top=33)
    yield "log probabilities: more alternatives than words", lambda: B.hc_logprobs(x[:, :3], top=4)
    yield "log probabilities: transposed", lambda: B.hc_logprobs(x.T)
    yield "log probabilities: 64-bit tokens", lambda: B.hc_logprobs(x, z(4, 1, dt=torch.int64))
    yield "log probabilities: tokens of other rows", lambda: B.hc_logprobs(x, z(3, 1, dt=i))


def test_refusals():
    for what, call in refusals():
        with pytest.raises(B.HCError):
            call()
            pytest.fail(f"{what} was taken")
    torch.cuda.synchronize()
    assert B.device_status() == B.TS_OK


def shifted(t):
    """``t``'s elements at an address that is a multiple of 16 bytes and not of 32."""
    flat = torch.empty(t.numel() + 16 // t.element_size(), dtype=t.dtype, device=t.device)
    got = flat[16 // t.element_size():].view(t.shape)
    assert got.data_ptr() % 32 == 16
    return got.copy_(t)


@pytest.mark.parametrize("d", [64, 128])
def test_addresses_on_16_bytes(d):
    """Inputs, outputs and states need lie on 16 bytes only: the same bits as where they lie on more."""
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n = 150
    starts, positions = packed([90, 60])
    q, k, v, w = r(n, 4, d).bfloat16(), r(n, 2, d).bfloat16(), r(n, 2, d).bfloat16(), r(d).bfloat16()
    table, decay, beta, state = B.rope_table(256, d, 10000.0), -r(n, 2).abs(), torch.sigmoid(r(n, 2)), r(2, 2, d, d)
    S = shifted
    want = B.hc_prompt_attention(q, k, v, starts)
    got = B.hc_prompt_attention(S(q), S(k), S(v), starts, out=S(torch.zeros_like(q)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want = B.hc_qk_norm_rope(q, k, positions, table, w, w)
    got = B.hc_qk_norm_rope(S(q), S(k), positions, S(table), S(w), S(w), q_out=S(torch.zeros_like(q)), k_out=S(torch.zeros_like(k)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    args = (k, q[:, :2], v, decay, beta, state, starts)
    want = B.hc_delta_prompt(*args, state_out=torch.zeros_like(state))
    got = B.hc_delta_prompt(*map(S, args[:6]), starts, out=S(torch.zeros_like(v)), state_out=S(torch.zeros_like(state)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    args = [x[:8].reshape(2, 4, *x.shape[1:]) for x in args[:5]] + [state]
    want = B.hc_delta_step(*args, state_out=torch.zeros_like(state))
    got = B.hc_delta_step(*map(S, args), out=S(torch.zeros_like(args[2])), state_out=S(torch.zeros_like(state)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert B.device_status() == B.TS_OK


def far_apart(t, stride):
    """``t``'s rows ``stride`` elements apart."""
    flat = torch.empty((t.shape[0] - 1) * stride + t[0].numel(), dtype=t.dtype, device=t.device)
    view = flat.as_strided(t.shape, (stride, *t.stride()[1:]))
    return view.copy_(t)


def test_offsets_past_32_bits():
    """Rows so far apart that elements' offsets do not fit 32 bits: the same bits as side by side."""
    g = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n, far = 5, (1 << 30) + 8  # up to 8.6 GB
    starts, positions = packed([3, 2])
    q, k = r(n, 4, 64).bfloat16(), r(n, 2, 64).bfloat16()
    w, table, decay, beta, state = r(64).bfloat16(), B.rope_table(64, 64, 10000.0), -r(n, 2).abs(), torch.sigmoid(r(n, 2)), r(2, 2, 64, 64)
    q_far, k_far = far_apart(q, far), far_apart(k, far)
    for got, want in ((B.hc_qk_norm_rope(q_far, k_far, positions, table, w, w), B.hc_qk_norm_rope(q, k, positions, table, w, w)),
                      (B.hc_prompt_attention(q_far, k_far, k, starts), B.hc_prompt_attention(q, k, k, starts)),
                      (B.hc_prompt_attention(q, k, k_far, starts), B.hc_prompt_attention(q, k, k, starts))):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del q_far
    out_far = far_apart(torch.zeros_like(q), far)
    B.hc_qk_norm_rope(q, None, positions, table, w, q_out=out_far)
    assert torch.equal(out_far, B.hc_qk_norm_rope(q, None, positions, table, w)[0])
    del out_far
    for args in ((k_far, k, k), (k, k_far, k), (k, k, k_far)):
        apart = lambda: dict(state_out=torch.zeros_like(state))  # noqa: E731
        for got, want in ((B.hc_delta_prompt(*args, decay, beta, state, starts, **apart()), B.hc_delta_prompt(k, k, k, decay, beta, state, starts, **apart())),
                          (B.hc_delta_step(*(x.unsqueeze(0) for x in (*args, decay, beta)), state[:1].contiguous(), state_out=torch.zeros_like(state[:1])),
                           B.hc_delta_step(*(x.unsqueeze(0) for x in (k, k, k, decay, beta)), state[:1].contiguous(), state_out=torch.zeros_like(state[:1])))):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del k_far, args
    x, chosen = r(n, 3000), torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    for got, want in zip(B.hc_logprobs(far_apart(x, (1 << 30) + 4), chosen, top=5), B.hc_logprobs(x, chosen, top=5)):
        assert torch.equal(got, want)
    assert B.device_status() == B.TS_OK


def test_many_sequences_and_heads():
    """The most sequences, most of them empty, and many heads."""
    s = 65535
    lens = torch.zeros(s, dtype=torch.int32)
    lens[[0, 17, 300, 40000, s - 1]] = torch.tensor([3, 70, 1, 130, 2], dtype=torch.int32)
    starts = torch.cat([torch.zeros(1, dtype=torch.int32), lens.cumsum(0).int()]).cuda()
    few, _ = packed([3, 70, 1, 130, 2])
    g = torch.Generator(device="cuda").manual_seed(8)
    n = int(lens.sum())
    q, k, v = (torch.randn(n, h, 64, generator=g, device="cuda").bfloat16() for h in (2, 1, 1))
    for got, want in zip(B.hc_prompt_attention(q, k, v, starts), B.hc_prompt_attention(q, k, v, few)):
        assert torch.equal(got, want)
    decay, beta = -torch.rand(n, 1, generator=g, device="cuda"), torch.rand(n, 1, generator=g, device="cuda")
    state = torch.zeros(s, 1, 64, 64, device="cuda")
    some = torch.zeros(5, 1, 64, 64, device="cuda")
    got, want = B.hc_delta_prompt(k, k, v, decay, beta, state, starts)[0], B.hc_delta_prompt(k, k, v, decay, beta, some, few)[0]
    assert torch.equal(got, want)
    assert torch.equal(state[[0, 17, 300, 40000, s - 1]], some)
    state[[0, 17, 300, 40000, s - 1]] = 0
    assert not state.any()
    # 1024 heads
    q, k = torch.randn(9, 1024, 64, generator=g, device="cuda").bfloat16(), torch.randn(9, 1024, 64, generator=g, device="cuda").bfloat16()
    at, _ = packed([9])
    wide = B.hc_prompt_attention(q, k, k, at)
    for h in (0, 511, 1023):
        one = B.hc_prompt_attention(*(x[:, h:h + 1].contiguous() for x in (q, k, k)), at)
        assert torch.equal(wide[0][:, h], one[0][:, 0]) and torch.equal(wide[1][:, h], one[1][:, 0])
    assert B.device_status() == B.TS_OK
