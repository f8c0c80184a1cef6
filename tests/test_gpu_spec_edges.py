"""GPU tests of the speculative decoding step's operators at the ends of their ranges: the largest finite
values, logits without a distribution, refused paths, very small weights, and the sizes at which a kernel
takes another path. Tolerances are test_gpu_spec's, with what a test adds to them derived beside it."""
import numpy as np
import pytest
import torch

import spec_reference as R
from gpu_common import require_gpu
from hyper_connection_residual_call_gb300 import binding as B
from test_gpu_spec import TREE, U16, U32, check_verify, gen, make_cache, randn, random_tree, run_attention, verify_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    B.device_status()


def bf16_bits(*bits):
    return torch.tensor(np.array(bits, np.uint16).view(np.int16)).cuda().view(torch.bfloat16)


def zeros(n=1):
    return torch.zeros(n, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ the cache's largest finite values

@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_largest_finite_values_saturate(group):
    """The lowest and the highest finite bf16, each beside ordinary elements and both in one group."""
    g = gen(40)
    cache = make_cache(g, "int4", 1, 16, 1, 16, 128, group)
    x = randn(g, 1, 6, 1, 128)
    low, high, next_low = bf16_bits(0xFF7F, 0x7F7F, 0xFF7E)
    x[0, 0, 0, 5], x[0, 1, 0, 70], x[0, 2, 0, 3] = low, high, next_low
    x[0, 3, 0, 9], x[0, 3, 0, 10] = low, high
    x[0, 4], x[0, 5] = low, high
    B.hc_kv_write(x, x, cache, zeros())
    want = R.stored(R.f64(x), "int4", group)
    assert np.isfinite(want).all()
    for got in B.hc_kv_read(cache, zeros(), 6):
        assert (np.abs(R.f64(got) - want) <= U16 * np.abs(want) + 1e-6).all()
    out, lse = B.hc_tree_attention(x[:, :1] * 0, cache, zeros() + 5)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    assert B.device_status() == B.TS_OK


FP8_LARGEST = (0x7F7F, 0xFF7F, 0x7F78, 0xFF78, 0x7F77, 0x7F61)  # +-(2 - 2^-7) 2^127, +-1.9375 2^127, and below it


def test_fp8_largest_finite_values_read_back_finite():
    """With a scale of 2^120 the code 256 would be 2^128: such an element is stored as 240 2^120."""
    g = gen(41)
    cache = make_cache(g, "fp8", 1, 16, 1, 16, 128)
    x = randn(g, 1, 8, 1, 128, scale=1e37)
    for i, v in enumerate(bf16_bits(*FP8_LARGEST)):
        x[0, i, 0, 7 * i + 1] = v
    x[0, 6] = bf16_bits(0xFF7F)[0]
    B.hc_kv_write(x, x, cache, zeros())
    x64 = R.f64(x)
    want = np.stack([R.fp8_row(r)[2] for r in x64.reshape(-1, 128)]).reshape(x64.shape)
    want = np.clip(want, -240 * 2.0 ** 120, 240 * 2.0 ** 120)
    for got in B.hc_kv_read(cache, zeros(), 8):
        assert np.array_equal(R.f64(got), want)
    assert (np.abs(want - x64) <= 2.0 ** -4 * np.abs(x64) + 2.0 ** 110).all()  # half a spacing of e4m3, also where it is held back
    assert B.device_status() == B.TS_OK


@pytest.mark.parametrize("hq", [2, 4, 8, 16])
def test_fp8_largest_values_of_unseen_nodes_do_not_reach_a_row(hq):
    """24, 48, 96 and 192 rows: a node's largest finite values are no infinities to the rows that do not see it."""
    g = gen(42)
    t, ctx, d = 12, 150, 128
    cache = make_cache(g, "fp8", 1, ctx + t, 1, 32, d)
    k, v = randn(g, 1, ctx + t, 1, d), randn(g, 1, ctx + t, 1, d)
    see = R.sees(TREE)
    mask = R.words(see)[None].cuda()
    q = randn(g, 1, t, hq, d)
    B.hc_kv_write(k, v, cache, zeros())
    out, lse = B.hc_tree_attention(q, cache, zeros() + ctx, mask=mask)
    largest = bf16_bits(*FP8_LARGEST)
    v[0, ctx + 5, 0, :6], v[0, ctx + 9, 0, 60:66] = largest, largest
    B.hc_kv_write(k, v, cache, zeros())
    out2, lse2 = B.hc_tree_attention(q, cache, zeros() + ctx, mask=mask)
    clean = torch.from_numpy(~(see[:, 5] | see[:, 9])).cuda()
    assert torch.equal(out2[:, clean], out[:, clean]) and torch.equal(lse2, lse)
    assert B.device_status() == B.TS_OK


# ------------------------------------------------------------------ logits without a distribution

def accepting_chain(v, t=4, seed=43):
    """Logits, tokens and the rest of a call whose chain of drafts holds at every node, greedy and sampled."""
    g = gen(seed)
    logits = torch.randn(1, t, v, generator=g, device="cuda")
    tokens = torch.zeros(1, t, dtype=torch.int32, device="cuda")
    tokens[0, 1:] = logits[0, :-1].argmax(-1).int()
    draft = torch.softmax(logits.double(), -1).float()
    rest = dict(draft_probs=draft, u=torch.zeros(1, t, device="cuda"), noise=torch.ones(1, v, device="cuda"))
    return logits, tokens, rest


def verify_both(logits, tokens, rest, sampled):
    if sampled:
        return B.hc_verify(logits, tokens, None, torch.ones(1, device="cuda"), **rest)
    return B.hc_verify(logits, tokens)


@pytest.mark.parametrize("v", [1, 50, 5000, 40001, 160000])
@pytest.mark.parametrize("node", [0, 2, 3])
@pytest.mark.parametrize("sampled", [False, True])
def test_verify_records_a_nan(v, node, sampled):
    """A NaN in a row that the walk reaches ends it there: recorded, and the next token is 0."""
    logits, tokens, rest = accepting_chain(v)
    for at in sorted({0, v // 2, v - 1}):
        bad = logits.clone()
        bad[0, node, at] = float("nan")
        n, path, nxt = verify_both(bad, tokens, rest, sampled)
        assert B.device_status() == B.TS_ERR_INVALID_ARG
        assert n.tolist() == [node] and path[0].tolist() == list(range(node + 1)) + [-1] * (3 - node) and nxt.tolist() == [0]


@pytest.mark.parametrize("sampled", [False, True])
def test_verify_records_a_nan_among_ruled_out_words(sampled):
    """160000 words over 8 CTAs: a thread that has nothing but -infinity before the NaN, which lies past what it keeps in registers."""
    logits, tokens, rest = accepting_chain(160000)
    logits[0, 0] = float("-inf")
    logits[0, 0, 7], logits[0, 0, 16384 + 5] = 1.0, float("nan")
    n, _, nxt = verify_both(logits, tokens, rest, sampled)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    assert n.tolist() == [0] and nxt.tolist() == [0]


def test_verify_infinities():
    """An infinite logit has no softmax (recorded) but an argmax; a row that is all -infinity has no softmax."""
    logits, tokens, rest = accepting_chain(3000)
    for value, all_of_it in ((float("inf"), False), (float("-inf"), True)):
        bad = logits.clone()
        bad[0, 1, slice(None) if all_of_it else 17] = value
        n, path, nxt = verify_both(bad, tokens, rest, True)
        assert B.device_status() == B.TS_ERR_INVALID_ARG
        assert n.tolist() == [1] and path[0].tolist() == [0, 1, -1, -1] and nxt.tolist() == [0]
        if not all_of_it:
            n, _, nxt = verify_both(bad, tokens, rest, False)
            assert n.tolist() == [1] and nxt.tolist() == [17]
            assert B.device_status() == B.TS_OK


@pytest.mark.parametrize("sampled", [False, True])
def test_verify_does_not_look_at_rows_off_the_walk(sampled):
    logits, tokens, rest = accepting_chain(3000)
    parents = torch.tensor([-1, 0, 0, 1], dtype=torch.int32, device="cuda")
    tokens[0, 3] = logits[0, 1].argmax().int()
    logits[0, 2] = float("nan")
    kw = dict(rest) if sampled else {}
    n, path, _ = B.hc_verify(logits, tokens, parents, torch.ones(1, device="cuda") if sampled else None, **kw)
    assert n.tolist() == [2] and path[0].tolist() == [0, 1, 3, -1]
    assert B.device_status() == B.TS_OK


# ------------------------------------------------------------------ compaction of a refused path

@pytest.mark.parametrize("kind,group", [("bf16", 0), ("fp8", 0), ("int4", 32)])
def test_compact_counts_what_it_moved(kind, group):
    """A path that is refused at a step: the rows before it are moved, and new_len counts those."""
    g = gen(44)
    b, t, heads, page, d = 6, 8, 2, 16, 64
    cache = make_cache(g, kind, b, 64, heads, page, d, group or 64)
    lens = torch.tensor([0, 9, 12, 3, 5, 10], dtype=torch.int32, device="cuda")
    B.hc_kv_write(randn(g, b, t, heads, d), randn(g, b, t, heads, d), cache, lens)
    k0, v0 = B.hc_kv_read(cache, lens, t)
    table = cache.tensors[2]
    was = table[2, 1].clone()
    table[2, 1] = -1  # positions 16 .. 31 of sequence 2, its nodes 4 and on
    paths = [[0, 3, 2], [0, 2, 9], [0, 2, 3, 5], [0, 2, 4, 7], [0, 1, 3], [0, 0]]
    moved = [1, 1, 2, 3, 0, 0]  # steps that hold
    path = torch.full((b, t), -1, dtype=torch.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = torch.tensor(p)
    n = torch.tensor([2, 2, 3, 3, 9, 1], dtype=torch.int32, device="cuda")  # sequence 4: more than there are nodes
    new = B.hc_kv_compact(cache, lens, path.cuda(), n)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    want = [int(c) + m + 1 for c, m in zip(lens.tolist(), moved)]
    want[4] = 5  # nothing is known of its path
    assert new.tolist() == want
    table[2, 1] = was
    k1, v1 = B.hc_kv_read(cache, lens, t)
    for i, (p, m) in enumerate(zip(paths, moved)):
        source = list(range(t))
        source[:m + 1] = p[:m + 1]
        for a, z in ((k0, k1), (v0, v1)):
            assert torch.equal(z[i], a[i, torch.tensor(source, device="cuda")])
    assert B.device_status() == B.TS_OK


# ------------------------------------------------------------------ very small weights

@pytest.mark.parametrize("heads,g,batch", [(608, 1, 4), (152, 72, 2)])
def test_int4_weights_far_below_the_largest(heads, g, batch):
    """Few-row and wide blocks with several items a CTA: keys of weight 1 with values of 0, and 8192 of weight
    2^-25.4 with values of 1, which are all of the result. A weight is held in fp16 as 2^6 of itself or more
    (relative to the largest), with a spacing of at most 2^-24 where it is subnormal, so that it is off by
    2^-31 at most, beside the 2^-11 that the bound has: 2^-31 sum|v| / Z more."""
    d, page, n = 64, 64, 8192
    table = torch.ones(batch, n // page, dtype=torch.int32, device="cuda")
    table[:, :4] = 0  # both streams of the wide kernel and every warp of the other have a large weight
    cache = B.kv_cache("int4", 2, heads, page, d, table, group=64)
    k = torch.full((1, 2 * page, heads, d), -17.625, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    k[:, :page:16], v[:, :page:16] = 0.0, 0.0
    B.hc_kv_write(k, v, B.KVCache("int4", *cache.tensors[:2], torch.arange(2, dtype=torch.int32, device="cuda")[None],
                                  k_scale=cache.tensors[3], v_scale=cache.tensors[4], k_bias=cache.tensors[5], v_bias=cache.tensors[6],
                                  group=64), zeros())
    q = torch.full((batch, 1, heads * g, d), 0.125, dtype=torch.bfloat16, device="cuda")
    out, lse = B.hc_tree_attention(q, cache, zeros(batch) + (n - 1), scale=0.125)
    small, large = n - 16, 16
    mass = small * np.exp(-17.625)
    z = large + mass
    want, reach = mass / z, 0.125 * 0.125 * 17.625 * d
    delta = (d + 8) * U32 * reach
    tol = (1.5 * U16 + 4 * delta + 64 * U32) * want + U16 * want + U32 + 2.0 ** -31 * small / z
    assert float(np.abs(R.f64(out) - want).max()) <= tol, (float(out.min()), float(out.max()), want, tol)
    assert float(np.abs(R.f64(lse) - np.log(z)).max()) <= 2 * delta + 64 * U32 * (1 + np.log(z))
    assert B.device_status() == B.TS_OK


# ------------------------------------------------------------------ other paths of the kernels

@pytest.mark.parametrize("kind,group", [("bf16", 0), ("fp8", 0), ("int4", 64)])
@pytest.mark.parametrize("page", [128, 256, 1024])
@pytest.mark.parametrize("d,hq,t", [(64, 4, 2), (128, 4, 12), (128, 8, 12), (128, 8, 24), (256, 2, 5)])
def test_attention_large_pages(kind, group, page, d, hq, t):
    """Pages of a tile's keys and more: lengths around a page's end, a page that ends inside a tile's rows."""
    run_attention(45, kind, group, d, hq, 1, page, [0, page - 1, page, page + 3, 1500], t, [random_tree(np.random.default_rng(t), t)] * 5)


@pytest.mark.parametrize("kind,group", [("bf16", 0), ("fp8", 0), ("int4", 32)])
@pytest.mark.parametrize("d,hq,hk,t", [(128, 1, 1, 65), (128, 1, 1, 100), (64, 2, 1, 97), (128, 2, 1, 130), (256, 1, 1, 70)])
def test_attention_masks_of_many_words(kind, group, d, hq, hk, t):
    """Mask rows of three to five words, in blocks of 64, 128 and 256 rows; nodes that reach over several tiles."""
    rng = np.random.default_rng(t)
    run_attention(46, kind, group, d, hq, hk, 16, [0, 1, 127, 350], t, [random_tree(rng, t) for _ in range(4)])


@pytest.mark.parametrize("kind,group", [("bf16", 0), ("fp8", 0), ("int4", 64)])
@pytest.mark.parametrize("hq,t", [(1, 140), (2, 300)])
def test_attention_of_a_prompt(kind, group, hq, t):
    """A chain of several tiles of nodes."""
    run_attention(47, kind, group, 128, hq, 1, 64, [0, 77], t)


@pytest.mark.parametrize("t,v,tree", [(1024, 60, True), (1025, 60, False), (1500, 300, True), (4096, 20, True)])
def test_verify_many_nodes(t, v, tree):
    """More nodes than a block keeps in shared memory."""
    args = verify_inputs(t, 2, t, v, tree, [0.9, 0.0], agree=0.3)
    logits, tokens, parents, temp, draft, u, noise = (torch.from_numpy(x).cuda() for x in args)
    check_verify(args, B.hc_verify(logits, tokens, parents, temp, draft_probs=draft, u=u, noise=noise))
    if not tree:
        check_verify(args, B.hc_verify(logits, tokens, None, temp, draft_probs=draft, u=u, noise=noise), chain=True)
    check_verify(args, B.hc_verify(logits, tokens, parents), greedy=True)
    assert B.device_status() == B.TS_OK


# ------------------------------------------------------------------ dependent launches

@pytest.mark.parametrize("kind,hq", [("bf16", 2), ("fp8", 4), ("int4", 8), ("bf16", 16)])
def test_steps_back_to_back_read_what_the_step_before_wrote(kind, hq):
    """Steps whose masks, positions, lengths, rows and table lie in the same buffers and change each time, with
    nothing between the launches, against the same steps with the GPU waited for after each call."""
    g = gen(48)
    b, t, hk, d, steps = 3, 12, 1, 128, 40
    rng = np.random.default_rng(48)
    parents = torch.tensor(np.array([[random_tree(rng, t) for _ in range(b)] for _ in range(steps)]), dtype=torch.int32, device="cuda")
    q, k, v = randn(g, steps, b, t, hq, d), randn(g, steps, b, t, hk, d), randn(g, steps, b, t, hk, d)
    path = torch.full((b, t), -1, dtype=torch.int32, device="cuda")
    path[:, :3] = torch.tensor([0, 2, 5], dtype=torch.int32)
    count = torch.tensor([2, 1, 0], dtype=torch.int32, device="cuda")

    def run(wait):
        after = torch.cuda.synchronize if wait else lambda: None
        cache = make_cache(gen(49), kind, b, 4 * steps + t, hk, 16, d, 64)
        lens = [zeros(b), zeros(b)]
        mask, pos = torch.zeros(b, t, 1, dtype=torch.int32, device="cuda"), torch.zeros(b, t, dtype=torch.int32, device="cuda")
        table = torch.zeros(4 * steps + 2 * t, d // 2, 2, device="cuda")
        qo, ko = torch.empty_like(q[0]), torch.empty_like(k[0])
        outs = torch.empty(steps, b, t, hq, d, dtype=torch.bfloat16, device="cuda")
        ws = B.tree_attention_workspace(b, t, hq, cache)
        lse = torch.empty(b, t, hq, device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):
            now, then = lens[i % 2], lens[(i + 1) % 2]
            assert B.ts_hc_rope_table(table.data_ptr(), table.shape[0], d, 1000.0 + i, None, torch.cuda.current_stream().cuda_stream) == B.TS_OK
            after()
            B.hc_tree_build(parents[i], now, mask=mask, positions=pos)
            after()
            B.hc_rope(q[i], k[i], pos.view(-1), table, q_out=qo, k_out=ko)
            after()
            B.hc_kv_write(ko, v[i], cache, now)
            after()
            B.hc_tree_attention(qo, cache, now, mask=mask, out=outs[i], lse=lse, ws=ws)
            after()
            B.hc_kv_compact(cache, now, path, count, new_len=then)
            after()
        torch.cuda.synchronize()
        return outs, lens[steps % 2].clone()

    want, want_len = run(True)
    assert want_len.tolist() == [3 * steps, 2 * steps, steps]
    for _ in range(5):
        got, got_len = run(False)
        assert torch.equal(got, want) and torch.equal(got_len, want_len)
    assert B.device_status() == B.TS_OK
