"""GPU tests of the speculative decoding step's operators through the binding and the C ABI, against
64-bit implementations (spec_reference).

Tolerances, from the number formats (unit roundoffs: u16 = 2^-8 of bf16, 8 bits of significand; u32 = 2^-24):
  rotary      |err| <= u16 |y| + 4 u32 (|x0| + |x1|): two products and a sum in fp32, one rounding
  cache       codes, scales and biases are equal; bf16 and FP8 rows read back exactly, INT4's
              q * scale + bias with one fp32 rounding and one to bf16
  attention   the scores are off by at most d = (D + 8) u32 max_j scale sum|q||k| (a sum of D products in
              fp32; the 8 for the scale, the maximum and the exponential), so that each weight is off by a
              factor of 1 + 2 d; P is rounded to 16 bits (u16 of p |v|), the result to bf16 (u16 of |out|);
              an INT4 value to fp16 (2^-11 |v| < u16/8): with A = sum p |v|
                |err| <= (u16 (1 + 1/2) + 4 d + 64 u32) A + u16 |out| + 2^-24,  lse: 2 d + 64 u32 (1 + |lse|)
  verification  whole numbers, equal; the inputs' decisions are asserted to be 1e-4 apart, far above
              the fp32 error of a sum of V probabilities (V u32)
"""
import numpy as np
import pytest
import torch

import spec_reference as R
from gpu_common import require_gpu
from hyper_connection_residual_call_gb300 import binding as B

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    B.device_status()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


# ------------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("kind,kw", [
    ("plain", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
    ("by_parts", dict(factor=16.0, original=4096.0, fast=32.0, slow=1.0)),
])
@pytest.mark.parametrize("rot", [2, 20, 64, 128])
def test_rope_table(kind, kw, rot):
    if kind == "ntk" and rot == 2:
        pytest.skip("refused")
    n, theta, mag = 1500, 10000.0, 1.25
    names = dict(plain=B.TS_ROPE_PLAIN, linear=B.TS_ROPE_LINEAR, ntk=B.TS_ROPE_NTK, by_parts=B.TS_ROPE_BY_PARTS)
    sc = B.TsHcRopeScaling(names[kind], kw.get("factor", 1.0), kw.get("original", 1.0), kw.get("fast", 2.0), kw.get("slow", 1.0), mag)
    t = R.f64(B.rope_table(n, rot, theta, scaling=sc))
    a = np.arange(n)[:, None] * R.rope_frequencies(rot, theta, kind, **kw)
    want = mag * np.stack([np.cos(a), np.sin(a)], -1)
    assert np.abs(t - want).max() <= mag * U32 * 1.01 + 1e-9


def test_rope_table_far_positions():
    n = 1 << 20
    t = B.rope_table(n, 8, 1e6)
    at = np.array([n - 1, n - 12345, 777777])
    a = at[:, None] * R.rope_frequencies(8, 1e6)
    assert np.abs(R.f64(t[torch.from_numpy(at)]) - np.stack([np.cos(a), np.sin(a)], -1)).max() <= U32 * 1.01 + 1e-9


def check_rope(y, x, pos, table, interleaved, inverse):
    want = R.rope(R.f64(x), pos.tolist(), R.f64(table), interleaved, inverse)
    size = np.abs(R.f64(x))
    half = table.shape[1]
    both = np.zeros_like(size)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        both[..., a] = both[..., b] = size[..., a] + size[..., b]
    assert (np.abs(R.f64(y) - want) <= U16 * np.abs(want) + 4 * U32 * both).all()
    assert np.array_equal(R.f64(y)[..., 2 * half:], R.f64(x)[..., 2 * half:])


@pytest.mark.parametrize("n,hq,hk,d,rot", [(1, 20, 4, 128, 128), (3, 4, 1, 64, 32), (7, 5, 5, 80, 20), (130, 3, 2, 256, 64),
                                           (2, 1, 0, 8, 6), (2500, 16, 4, 128, 64), (33, 2, 1, 48, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(n, hq, hk, d, rot, interleaved, inverse):
    g = gen(n + d)
    table = B.rope_table(4096, rot, 10000.0)
    x = randn(g, n, hq + 2 * hk + 1, d)  # a projection's output with more in it than the heads that turn
    q, k = x[:, :hq], x[:, hq:hq + hk] if hk else None
    pos = torch.randint(0, 4096, (n,), generator=g, device="cuda").int()
    before = x.clone()
    qo, ko = B.hc_rope(q, k, pos, table, interleaved=interleaved, inverse=inverse)
    assert torch.equal(x, before)
    some = slice(0, 40)
    check_rope(qo[some], q[some], pos[some], table, interleaved, inverse)
    if hk:
        check_rope(ko[some], k[some], pos[some], table, interleaved, inverse)
    # in place: the same bits, and nothing beside the heads changes
    B.hc_rope(q, k, pos, table, interleaved=interleaved, inverse=inverse, q_out=q, k_out=k)
    assert torch.equal(q, qo) and (not hk or torch.equal(k, ko))
    assert torch.equal(x[:, hq + hk:], before[:, hq + hk:])
    assert B.device_status() == B.TS_OK


def test_rope_gradient():
    """The operator is linear: column j of its matrix is its value at e_j (and the difference quotient in
    that direction); the inverse's matrix is the transpose."""
    d, rot = 32, 24
    table = B.rope_table(512, rot, 100.0)
    pos = torch.full((d,), 333, dtype=torch.int32, device="cuda")
    eye = torch.eye(d, device="cuda").bfloat16().view(d, 1, d)
    for inter in (False, True):
        col, _ = B.hc_rope(eye, None, pos, table, interleaved=inter)
        row, _ = B.hc_rope(eye, None, pos, table, interleaved=inter, inverse=True)
        assert torch.equal(col.view(d, d).T, row.view(d, d))
        g = gen(5)
        x, step = randn(g, 1, 1, d), randn(g, 1, 1, d)
        f = lambda t: R.f64(B.hc_rope(t, None, pos[:1], table, interleaved=inter)[0]).ravel()  # noqa: E731
        up = x + step
        # f(x + h) - f(x) = J h: three results rounded to bf16 (u16 of each), on inputs that are exact
        h = R.f64(up).ravel() - R.f64(x).ravel()
        want = R.f64(col).reshape(d, d).T @ h
        bound = U16 * (np.abs(f(up)) + np.abs(f(x))) + U16 * (np.abs(R.f64(col).reshape(d, d).T) @ np.abs(h)) + 1e-6
        assert (np.abs(f(up) - f(x) - want) <= bound).all()


def test_rope_bad_position_is_recorded():
    table = B.rope_table(16, 32, 10000.0)
    q = randn(gen(1), 3, 2, 32)
    for bad in (16, -1):
        pos = torch.tensor([3, bad, 5], dtype=torch.int32, device="cuda")
        y, _ = B.hc_rope(q, None, pos, table)
        assert B.device_status() == B.TS_ERR_INVALID_ARG
        assert torch.count_nonzero(y[1]) == 0
        check_rope(y[::2], q[::2], pos[::2], table, False, False)


# ------------------------------------------------------------------ the cache

def pages_for(g, batch, per, spare=2):
    n = batch * per + spare
    return torch.randperm(n, generator=torch.Generator().manual_seed(int(g.initial_seed()) + 3))[:batch * per].view(batch, per).int().cuda(), n


def make_cache(g, kind, batch, length, heads, page, d, group=64):
    table, n = pages_for(g, batch, -(-length // page))
    return B.kv_cache(kind, n, heads, page, d, table, group=min(group, d))


def spread(g, *shape):
    """Rows of very different sizes, some of them zero, some with elements that fall between two codes."""
    x = torch.randn(*shape, generator=g, device="cuda")
    size = torch.exp2(torch.randint(-20, 20, shape[:-1], generator=g, device="cuda").float())[..., None]
    x = (x * size).bfloat16()
    x[..., 0, :] = 0
    x[..., 0, :, :] = (x[..., 0, :, :].float().sign() * torch.randint(0, 60, x[..., 0, :, :].shape, generator=g, device="cuda") * 0.125).bfloat16()
    return x


KINDS = [("bf16", 0), ("fp8", 0), ("int4", 32), ("int4", 64), ("int4", 128)]


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("d,heads,page,batch,t,ctx", [(64, 3, 16, 2, 5, 14), (128, 2, 32, 3, 1, 0), (256, 1, 16, 1, 40, 7),
                                                      (128, 5, 64, 2, 33, 63)])
def test_cache_write_and_read(kind, group, d, heads, page, batch, t, ctx):
    if group > d:
        pytest.skip("a group is at most a row")
    g = gen(d + t)
    cache = make_cache(g, kind, batch, ctx + t + batch, heads, page, d, group or 64)
    lens = torch.tensor([ctx + i for i in range(batch)], dtype=torch.int32, device="cuda")
    # slices of one projection's output
    x = torch.cat((spread(g, batch, t, heads, d), randn(g, batch, t, heads, d, scale=0.3), randn(g, batch, t, 1, d)), 2)
    k, v = x[:, :, :heads], x[:, :, heads:2 * heads]
    before = [None if y is None else y.clone() for y in cache.tensors]
    B.hc_kv_write(k, v, cache, lens)
    ko, vo = B.hc_kv_read(cache, lens, t)
    for got, src in ((ko, k), (vo, v)):
        want = R.stored(R.f64(src), kind, group)
        if kind == "int4":
            assert (np.abs(R.f64(got) - want) <= U16 * np.abs(want) + 2 * U32 * (np.abs(want) + 1e-30) + 1e-38).all()
        else:
            assert np.array_equal(R.f64(got), want)
    # the codes themselves, and nothing else in the pools
    touched = torch.zeros(cache.tensors[0].shape[0], page, dtype=torch.bool)
    table = cache.tensors[2].cpu()
    for b in range(batch):
        for i in range(t):
            pos = ctx + b + i
            touched[table[b, pos // page], pos % page] = True
    for now, was in zip(cache.tensors, before):
        if now is not None and now.dim() >= 3:
            same = (now == was) | (now != now)
            same = same.flatten(3).all(-1) if same.dim() == 4 else same
            assert bool((same.all(1).cpu() | touched).all())
    if kind != "bf16":
        names = [("k", 0, 3, 5), ("v", 1, 4, 6)]
        for (name, at, sc, bi), src in zip(names, (k, v)):
            for b in range(batch):
                for i in (0, t - 1):
                    pos = ctx + b + i
                    page_id, place = int(table[b, pos // page]), pos % page
                    row = R.f64(src[b, i, heads - 1])
                    codes = cache.tensors[at][page_id, heads - 1, place].cpu().numpy()
                    if kind == "fp8":
                        want, byte, _ = R.fp8_row(row)
                        assert byte == int(cache.tensors[sc][page_id, heads - 1, place])
                        assert np.array_equal(R.E4M3[codes], R.E4M3[want])
                    else:
                        want, s, bias, _ = R.int4_row(row, group)
                        assert np.array_equal(np.stack([codes & 15, codes >> 4], -1).ravel(), want)
                        assert np.array_equal(cache.tensors[sc][page_id, heads - 1, place].cpu().numpy(), s)
                        assert np.array_equal(cache.tensors[bi][page_id, heads - 1, place].cpu().numpy(), bias)
    assert B.device_status() == B.TS_OK


@pytest.mark.parametrize("kind", ["fp8", "int4"])
def test_cache_marks_infinities_and_nans(kind):
    g = gen(9)
    cache = make_cache(g, kind, 1, 16, 2, 16, 64, 32)
    k, v = randn(g, 1, 4, 2, 64), randn(g, 1, 4, 2, 64)
    k[0, 1, 0, 40], k[0, 2, 1, 3], v[0, 3, 0, 63] = float("inf"), float("nan"), float("-inf")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.hc_kv_write(k, v, cache, start)
    for got, src in zip(B.hc_kv_read(cache, start, 4), (k, v)):
        want = R.stored(R.f64(src), kind, 32)
        assert np.array_equal(np.isnan(R.f64(got)), np.isnan(want))
        fine = np.isfinite(want)
        assert (np.abs(R.f64(got) - want)[fine] <= U16 * np.abs(want)[fine] + 1e-6).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_cache_extremes(kind):
    """The largest and smallest bf16 rows: FP8 scales at both ends, INT4 kept inside fp16."""
    g = gen(10)
    cache = make_cache(g, kind, 1, 16, 1, 16, 64, 32)
    x = torch.zeros(1, 6, 1, 64, device="cuda")
    x[0, 0], x[0, 1], x[0, 2], x[0, 3], x[0, 4] = 3e38, 1e-38, 2.0 ** -130, 1.0, 60000.0
    x[0, 3, 0, ::2] = -1.0
    x[0, 4, 0, 0] = -60000.0
    x = x.bfloat16()
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.hc_kv_write(x, x, cache, start)
    want = R.stored(R.f64(x), kind, 32)
    got = R.f64(B.hc_kv_read(cache, start, 6)[0])
    if kind == "int4":
        assert (np.abs(got - want) <= U16 * np.abs(want) + 1e-38).all()
    else:
        assert np.array_equal(got, want)


def test_cache_refuses_places_outside(kind="fp8"):
    g = gen(11)
    cache = make_cache(g, kind, 2, 32, 1, 16, 64)
    cache.tensors[2][1, 0] = cache.tensors[0].shape[0]  # not a page
    k = randn(g, 2, 4, 1, 64)
    lens = torch.tensor([30, 3], dtype=torch.int32, device="cuda")
    before = cache.tensors[0].clone()
    B.hc_kv_write(k, k, cache, lens)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    now = cache.tensors[0]
    changed = (now != before).flatten(1).any(1).nonzero().ravel().tolist()
    assert changed == [int(cache.tensors[2][0, 1])]  # positions 30 and 31 of sequence 0, nothing else
    ko, _ = B.hc_kv_read(cache, lens, 4)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    assert torch.count_nonzero(ko[0, 2:]) == 0 and torch.count_nonzero(ko[1]) == 0
    assert np.array_equal(R.f64(ko[0, :2]), R.stored(R.f64(k[0, :2]), kind))
    B.hc_kv_write(k, k, cache, torch.tensor([-1, -5], dtype=torch.int32, device="cuda"))
    assert B.device_status() == B.TS_ERR_INVALID_ARG


@pytest.mark.parametrize("kind,group", [("bf16", 0), ("fp8", 0), ("int4", 32)])
@pytest.mark.parametrize("d", [64, 256])
def test_compact(kind, group, d):
    g = gen(12)
    b, t, heads, page = 4, 40, 2, 16
    cache = make_cache(g, kind, b, 30 + t, heads, page, d, group or 64)
    lens = torch.tensor([0, 9, 30, 17], dtype=torch.int32, device="cuda")
    B.hc_kv_write(randn(g, b, t, heads, d), randn(g, b, t, heads, d), cache, lens)
    k0, v0 = B.hc_kv_read(cache, lens, t)
    paths = [[0], [0, 1, 2, 3], [0, 2, 5, 6, 39], [0] + list(range(2, 40))]
    path = torch.full((b, t), -1, dtype=torch.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = torch.tensor(p)
    n = torch.tensor([len(p) - 1 for p in paths], dtype=torch.int32, device="cuda")
    new = B.hc_kv_compact(cache, lens, path.cuda(), n)
    k1, v1 = B.hc_kv_read(cache, lens, t)
    for i, p in enumerate(paths):
        for was, now in ((k0, k1), (v0, v1)):
            assert torch.equal(now[i, :len(p)], was[i, torch.tensor(p, device="cuda")])
            untouched = list(range(len(p), t))
            assert torch.equal(now[i, untouched], was[i, untouched])
    assert new.tolist() == [int(x) + len(p) for x, p in zip(lens.tolist(), paths)]
    assert B.device_status() == B.TS_OK
    # a path that does not ascend is recorded and not followed past that
    path[0, :3] = torch.tensor([0, 3, 2])
    B.hc_kv_compact(cache, lens, path.cuda(), torch.tensor([2, 0, 0, 0], dtype=torch.int32, device="cuda"))
    assert B.device_status() == B.TS_ERR_INVALID_ARG


# ------------------------------------------------------------------ trees

TREE = [-1, 0, 0, 1, 1, 2, 3, -1, 6, 8, 7, 5]


@pytest.mark.parametrize("parents", [[-1], [0, 0], TREE, [-1] + list(range(69)), [-1] + [0] * 40])
def test_tree_build(parents):
    p = torch.tensor([parents, parents], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([100, 7], dtype=torch.int32, device="cuda")
    mask, pos = B.hc_tree_build(p, ctx)
    want = R.words(R.sees(parents))
    depth = torch.tensor(R.depths(parents))
    for b in range(2):
        assert torch.equal(mask[b].cpu(), want)
        assert torch.equal(pos[b].cpu().long(), depth + int(ctx[b]))
    shared, pos2 = B.hc_tree_build(p[0].contiguous(), batch=2)
    assert torch.equal(shared, mask) and torch.equal(pos2[0].cpu().long(), depth)
    assert B.device_status() == B.TS_OK


def test_tree_build_bad_parent_is_recorded():
    p = torch.tensor([[-1, 0, 2, 9]], dtype=torch.int32, device="cuda")
    mask, _ = B.hc_tree_build(p)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    assert mask.ravel().tolist() == [1, 3, 0, 0]


# ------------------------------------------------------------------ tree attention

def check_attention(out, lse, q, cache, lens, see, scale, keys):
    """keys(b, n): the stored rows [n, Hk, D] x 2 that sequence b's positions hold, 64 bits."""
    out, lse = R.f64(out), R.f64(lse)
    for b, ctx in enumerate(lens):
        k, v = keys(b, ctx + q.shape[1])
        want, want_lse, weight, reach = R.attention(R.f64(q[b]), k, v, ctx, see[b], scale)
        d = (q.shape[-1] + 8) * U32 * reach
        tol = (1.5 * U16 + 4 * d[..., None] + 64 * U32) * weight + U16 * np.abs(want) + U32
        assert np.isfinite(out[b]).all()
        err = np.abs(out[b] - want)
        assert (err <= tol).all(), (b, float((err / tol).max()))
        empty = np.isinf(want_lse)
        assert np.array_equal(np.isneginf(lse[b]), empty)
        err = np.abs(lse[b] - want_lse)[~empty]
        lim = (2 * d + 64 * U32 * (1 + np.abs(want_lse)))[~empty]
        assert (err <= lim).all(), (b, float((err / lim).max()))


def run_attention(seed, kind, group, d, hq, hk, page, lens, t, parents=None, shared=False, cut=None, q_scale=2.0):
    g = gen(seed)
    b = len(lens)
    cache = make_cache(g, kind, b, max(lens) + t, hk, page, d, group or 64)
    total = max(lens) + t
    start = torch.zeros(b, dtype=torch.int32, device="cuda")
    B.hc_kv_write(randn(g, b, total, hk, d), randn(g, b, total, hk, d), cache, start)
    k, v = B.hc_kv_read(cache, start, total)
    if kind == "int4":  # the values that the codes stand for, not their bf16 roundings
        k, v = exact_int4(cache, total)
    else:
        k, v = R.f64(k), R.f64(v)
    q = randn(g, b, t, hq + 3, d, scale=q_scale)[:, :, :hq]
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if parents is None:
        see, mask = [np.tril(np.ones((t, t), bool))] * b, None
    else:
        see = [R.sees(p) for p in parents]
        mask = torch.stack([R.words(m) for m in see]).cuda()
        if shared:
            mask = mask[0]
    out, lse = B.hc_tree_attention(q, cache, ctx, mask=mask, scale=d ** -0.5)
    check_attention(out, lse, q, cache, lens, see, d ** -0.5, lambda i, n: (k[i, :n], v[i, :n]))
    assert B.device_status() == B.TS_OK
    return q, cache, ctx, mask, out, lse


def exact_int4(cache, total):
    kp, vp, table, ks, vs, kb, vb = cache.tensors
    at = torch.arange(total, device="cuda")
    page, place = table.long()[:, at // cache.page_size], at % cache.page_size
    res = []
    for pool, s, bias in ((kp, ks, kb), (vp, vs, vb)):
        codes = pool[page, :, place[None].expand_as(page)]
        x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
        sc = s[page, :, place[None].expand_as(page)].double().repeat_interleave(cache.group, -1)
        bi = bias[page, :, place[None].expand_as(page)].double().repeat_interleave(cache.group, -1)
        res.append(R.f64(x * sc + bi))
    return res


def random_tree(rng, t):
    return [-1] + [int(rng.integers(max(0, i - 5), i)) for i in range(1, t)]


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("d,hq,hk,page,lens,t", [
    (128, 20, 4, 16, [5], 1),                 # one token, a few keys
    (64, 4, 4, 16, [0, 1, 15, 16, 17], 1),    # heads not shared; contexts around a page's end
    (128, 8, 1, 32, [0, 63, 64, 200], 2),     # 16 rows
    (64, 10, 2, 64, [130, 3], 7),             # 35 rows, an odd group
    (256, 6, 2, 16, [77, 260], 5),
    (128, 16, 2, 128, [500, 129, 1], 24),     # 192 rows
    (64, 8, 1, 16, [333], 33),                # 264 rows
])
def test_attention_chain(kind, group, d, hq, hk, page, lens, t):
    if group > d:
        pytest.skip("a group is at most a row")
    run_attention(1, kind, group, d, hq, hk, page, lens, t)


@pytest.mark.parametrize("kind,group", [("bf16", 0), ("fp8", 0), ("int4", 64)])
@pytest.mark.parametrize("d,hq,hk,page,lens,t", [
    (128, 4, 1, 16, [0, 100, 31], 12), (64, 32, 2, 32, [250, 7], 40), (256, 4, 4, 64, [64], 70), (128, 8, 2, 64, [1000, 3], 64),
])
@pytest.mark.parametrize("shared", [False, True])
def test_attention_tree(kind, group, d, hq, hk, page, lens, t, shared):
    rng = np.random.default_rng(t)
    parents = [random_tree(rng, t) for _ in lens]
    if t == 12:
        parents = [list(TREE) for _ in lens]  # with absent nodes, whose rows see only the context (nothing at 0)
    if shared:
        parents = [parents[0]] * len(lens)
    run_attention(2, kind, group, d, hq, hk, page, lens, t, parents, shared)


@pytest.mark.parametrize("kind,group", [("bf16", 0), ("fp8", 0), ("int4", 32)])
@pytest.mark.parametrize("hq,t", [(4, 1), (8, 16)])
def test_attention_long_and_ragged(kind, group, hq, t):
    run_attention(3, kind, group, 128, hq, 2, 64, [9000, 1, 4097, 640], t)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_attention_many_sequences(kind):
    """More sequences than a block has threads, and more items than CTAs."""
    rng = np.random.default_rng(0)
    run_attention(4, kind, 32, 64, 4, 2, 16, rng.integers(0, 90, 300).tolist(), 3)


def test_attention_peaked_scores():
    """Scores of some hundreds, rising and falling along the context: the running maximum moves often."""
    run_attention(5, "bf16", 0, 128, 8, 2, 16, [700, 90], 6, q_scale=60.0)


def test_attention_empty_rows():
    g = gen(6)
    cache = make_cache(g, "bf16", 2, 64, 2, 16, 64)
    k = randn(g, 2, 40, 2, 64)
    lens = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    B.hc_kv_write(k, k, cache, lens)
    mask = torch.zeros(2, 40, 2, dtype=torch.int32, device="cuda")
    mask[1, 3, 0] = 8  # one row sees one node
    out, lse = B.hc_tree_attention(randn(g, 2, 40, 4, 64), cache, lens, mask=mask)
    assert torch.count_nonzero(out[0]) == 0 and bool(torch.isneginf(lse[0]).all())
    assert torch.equal(out[1, 3, 0], k[1, 3, 0]) and torch.equal(out[1, 3, 3], k[1, 3, 1])
    rest = [i for i in range(40) if i != 3]
    assert torch.count_nonzero(out[1, rest]) == 0 and bool(torch.isneginf(lse[1, rest]).all())


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("hq", [2, 16, 32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_unseen_infinities_and_nans_do_not_reach_a_row(kind, hq, bad):
    """Bad keys and values in nodes: the rows that do not see them keep their bits, those that do get NaN or
    an infinity where the formula has them; bad rows past the end change nothing."""
    g = gen(7)
    t, ctx, d = 12, 21, 64
    cache = make_cache(g, kind, 1, 64, 2, 16, d, 32)
    k, v = randn(g, 1, ctx + t + 9, 2, d), randn(g, 1, ctx + t + 9, 2, d)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = zero + ctx
    q = randn(g, 1, t, hq, d)
    see = R.sees(TREE)
    mask = R.words(see)[None].cuda()
    B.hc_kv_write(k, v, cache, zero)
    out, lse = B.hc_tree_attention(q, cache, lens, mask=mask)
    assert bool(torch.isfinite(out).all())
    k2, v2 = k.clone(), v.clone()
    k2[0, ctx + 4, :, 5], v2[0, ctx + 5, :, 7], v2[0, ctx + 9, 1, 50] = bad, bad, bad
    k2[0, ctx + t:], v2[0, ctx + t:] = bad, bad
    B.hc_kv_write(k2, v2, cache, zero)
    out2, lse2 = B.hc_tree_attention(q, cache, lens, mask=mask)
    hit = see[:, 4] | see[:, 5] | see[:, 9]
    clean = torch.from_numpy(~hit).cuda()
    assert torch.equal(out2[0, clean], out[0, clean]) and torch.equal(lse2[0, clean], lse[0, clean])
    saw = torch.from_numpy(see[:, 5]).cuda()
    assert not bool(torch.isfinite(out2[0, saw][..., 7]).any())
    if kind == "bf16":  # the other elements of a value's row stay as they were
        one = [i for i in range(t) if see[i, 5] and not see[i, 4] and not see[i, 9]]
        keep = [i for i in range(d) if i != 7]
        assert torch.equal(out2[0, one][..., keep], out[0, one][..., keep])
        value = out2[0, one][..., 7]
        assert bool((torch.isnan(value) if bad != bad else value == bad).all())
    assert B.device_status() == B.TS_OK


def test_attention_nan_in_the_context_is_seen():
    g = gen(8)
    cache = make_cache(g, "bf16", 2, 64, 1, 16, 64)
    k, v = randn(g, 2, 40, 1, 64), randn(g, 2, 40, 1, 64)
    v[0, 3, 0, 9] = float("nan")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    B.hc_kv_write(k, v, cache, zero)
    out, _ = B.hc_tree_attention(randn(g, 2, 2, 4, 64), cache, zero + 38)
    assert bool(torch.isnan(out[0, :, :, 9]).all()) and bool(torch.isfinite(out[1]).all())
    assert bool(torch.isfinite(out[0][..., :9]).all())


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_attention_is_deterministic_and_replays(kind):
    """The same bits on every run, on another stream, and from a captured graph with other lengths."""
    q, cache, ctx, mask, out, lse = run_attention(20, kind, 64, 128, 16, 2, 16, [900, 2100, 40], 16,
                                                  [random_tree(np.random.default_rng(1), 16)] * 3)
    again = B.hc_tree_attention(q, cache, ctx, mask=mask, scale=128 ** -0.5)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = B.hc_tree_attention(q, cache, ctx, mask=mask, scale=128 ** -0.5, stream=side)
    side.synchronize()
    assert torch.equal(other[0], out) and torch.equal(other[1], lse)
    ws = B.tree_attention_workspace(3, 16, 16, cache)
    o, l = torch.empty_like(out), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.hc_tree_attention(q, cache, ctx, mask=mask, scale=128 ** -0.5, out=o, lse=l, ws=ws)
    lens = ctx.clone()
    ctx.copy_(torch.tensor([3, 700, 1500], dtype=torch.int32))
    fresh = B.hc_tree_attention(q, cache, ctx.clone(), mask=mask, scale=128 ** -0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, fresh[0]) and torch.equal(l, fresh[1])
    ctx.copy_(lens)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hk,t", [(3, 1, 11), (8, 2, 12), (4, 1, 16), (13, 1, 5), (8, 1, 12), (16, 1, 8), (43, 1, 3), (8, 1, 32)])
def test_attention_wide_blocks(kind, hq, hk, t):
    """33 to 256 rows a key head: contexts around a tile's end, items that are cut and whole ones, odd groups."""
    run_attention(22, kind, 0, 128, hq, hk, 16, [0, 1, 127, 128, 129, 300, 1025, 2600], t, [random_tree(np.random.default_rng(t), t)] * 8)


def test_attention_fp8_query_of_wide_range():
    """Up to 64 rows the query meets the codes as two e4m3 parts: an element is off by at most 2^-17.8 of its
    row's largest (half of the second part's least spacing, 2^-10, of a largest element of more than 224), so
    that a score is off by 2^-17.8 max|q| scale sum|k| more."""
    g = gen(23)
    t, ctx, d = 12, 300, 128
    cache = make_cache(g, "fp8", 1, ctx + t, 1, 16, d)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.hc_kv_write(randn(g, 1, ctx + t, 1, d), randn(g, 1, ctx + t, 1, d), cache, zero)
    k, v = (R.f64(x[0]) for x in B.hc_kv_read(cache, zero, ctx + t))
    q = randn(g, 1, t, 4, d)
    q[..., 7] *= 64.0
    q[:, 1] *= 2.0 ** -60
    q[:, 2] *= 2.0 ** 20
    q[:, 3] = 0
    q[:, 4, :, 1:] = 0
    see = np.tril(np.ones((t, t), bool))
    out, lse = B.hc_tree_attention(q, cache, zero + ctx, scale=d ** -0.5)
    out, lse, q64 = R.f64(out[0]), R.f64(lse[0]), R.f64(q[0])
    want, want_lse, weight, reach = R.attention(q64, k, v, ctx, see, d ** -0.5)
    delta = (d + 8) * U32 * reach + 2.0 ** -17.8 * np.abs(q64).max(-1) * d ** -0.5 * np.abs(k).sum(-1).max()
    assert (np.abs(out - want) <= (1.5 * U16 + np.expm1(np.minimum(2 * delta, 600.0))[..., None] * 2 + 64 * U32) * weight + U16 * np.abs(want) + U32).all()
    assert (np.abs(lse - want_lse) <= 2 * delta + 64 * U32 * (1 + np.abs(want_lse))).all()
    # a NaN or an infinity in a row of the query reaches that row alone
    bad = q.clone()
    bad[0, 5, 2, 100], bad[0, 6, 1, 3] = float("nan"), float("inf")
    out2, lse2 = B.hc_tree_attention(bad, cache, zero + ctx, scale=d ** -0.5)
    assert bool(torch.isnan(out2[0, 5, 2]).all()) and bool(torch.isnan(lse2[0, 5, 2])) and not bool(torch.isfinite(out2[0, 6, 1]).any())
    rest = torch.ones(t, 4, dtype=torch.bool, device="cuda")
    rest[5, 2] = rest[6, 1] = False
    again = B.hc_tree_attention(q, cache, zero + ctx, scale=d ** -0.5)
    assert torch.equal(out2[0][rest], again[0][0][rest]) and torch.equal(lse2[0][rest], again[1][0][rest])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("hq", [4, 8, 16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_wide_blocks_keep_unseen_infinities_out(kind, hq, bad):
    """Bad nodes, a bad row behind the last one, and rows that see nothing at all: 48, 96 and 192 rows."""
    g = gen(24)
    t, d = 12, 128
    lens = torch.tensor([150, 0], dtype=torch.int32, device="cuda")
    zero = torch.zeros_like(lens)
    cache = make_cache(g, kind, 2, 200, 1, 32, d)
    k, v = randn(g, 2, 170, 1, d), randn(g, 2, 170, 1, d)
    see = R.sees(TREE)
    see[7:9] = False  # in the second sequence these rows see nothing
    mask = R.words(see)[None].expand(2, -1, -1).contiguous().cuda()
    q = randn(g, 2, t, hq, d)
    B.hc_kv_write(k, v, cache, zero)
    out, lse = B.hc_tree_attention(q, cache, lens, mask=mask)
    assert bool(torch.isfinite(out).all())
    assert torch.count_nonzero(out[1, 7:9]) == 0 and bool(torch.isneginf(lse[1, 7:9]).all())
    for i, n in enumerate((150, 0)):
        k[i, n + 4, 0, 5], v[i, n + 5, 0, 7] = bad, bad
        k[i, n + t:], v[i, n + t:] = bad, bad
    B.hc_kv_write(k, v, cache, zero)
    out2, lse2 = B.hc_tree_attention(q, cache, lens, mask=mask)
    clean = torch.from_numpy(~(see[:, 4] | see[:, 5])).cuda()
    assert torch.equal(out2[:, clean], out[:, clean]) and torch.equal(lse2[:, clean], lse[:, clean])
    saw = torch.from_numpy(see[:, 5]).cuda()
    assert not bool(torch.isfinite(out2[:, saw][..., 7]).any())
    assert B.device_status() == B.TS_OK


@pytest.mark.parametrize("kind,hq", [("bf16", 4), ("bf16", 16), ("fp8", 4), ("fp8", 8), ("fp8", 16)])
def test_attention_wide_blocks_many_times(kind, hq):
    """64, 128 and 256 rows, several items a block, 200 times: no wait runs out and every run has the same bits."""
    g = gen(25)
    b, t, ctx = 24, 16, 1800
    cache = make_cache(g, kind, b, ctx + t, 2, 64, 128)
    zero = torch.zeros(b, dtype=torch.int32, device="cuda")
    B.hc_kv_write(randn(g, b, ctx + t, 2, 128), randn(g, b, ctx + t, 2, 128), cache, zero)
    q, lens = randn(g, b, t, 2 * hq, 128), zero + ctx - 37 * torch.arange(b, device="cuda", dtype=torch.int32)
    out, lse = B.hc_tree_attention(q, cache, lens)
    o, l = torch.empty_like(out), torch.empty_like(lse)
    ws = B.tree_attention_workspace(b, t, 2 * hq, cache)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        B.hc_tree_attention(q, cache, lens, out=o, lse=l, ws=ws)
        differ += (o != out).sum() + (l != lse).sum()
    assert int(differ) == 0
    assert B.device_status() == B.TS_OK


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("hq,hk,t", [(3, 1, 11), (4, 1, 16), (8, 1, 12), (16, 1, 8), (43, 1, 3), (8, 2, 64)])
def test_attention_wide_blocks_int4(group, hq, hk, t):
    """A key as two bf16 parts is off by at most 2^-18 of itself, 64 u32, which the bound's D u32 for a sum in
    fp32 (of some ten steps) covers."""
    run_attention(26, "int4", group, 128, hq, hk, 16, [0, 1, 127, 128, 129, 300, 1025, 2600], t, [random_tree(np.random.default_rng(t), t)] * 8)


@pytest.mark.parametrize("kind,group", [("bf16", 0), ("fp8", 0), ("int4", 32), ("int4", 64)])
@pytest.mark.parametrize("hq,t", [(4, 9), (8, 9), (8, 17), (12, 30)])
def test_attention_wide_blocks_of_64(kind, group, hq, t):
    """36 to 360 rows of 64 elements."""
    run_attention(28, kind, group, 64, hq, 1, 32, [0, 1, 127, 128, 129, 300, 1025, 2600], t, [random_tree(np.random.default_rng(t), t)] * 8)


@pytest.mark.parametrize("hq", [4, 8, 16])
def test_attention_wide_blocks_int4_unseen_and_many_times(hq):
    """Unseen bad nodes change nothing; rows past the end neither; 100 runs have the same bits and no wait runs out."""
    g = gen(27)
    t, d = 12, 128
    lens = torch.tensor([1500, 150, 0], dtype=torch.int32, device="cuda")
    zero = torch.zeros_like(lens)
    cache = make_cache(g, "int4", 3, 1600, 1, 32, d, 32)
    k, v = randn(g, 3, 1530, 1, d), randn(g, 3, 1530, 1, d)
    see = R.sees(TREE)
    mask = R.words(see)[None].expand(3, -1, -1).contiguous().cuda()
    q = randn(g, 3, t, hq, d)
    B.hc_kv_write(k, v, cache, zero)
    out, lse = B.hc_tree_attention(q, cache, lens, mask=mask)
    assert bool(torch.isfinite(out).all())
    for i, n in enumerate(lens.tolist()):
        k[i, n + 4, 0, 5], v[i, n + 5, 0, 7] = float("nan"), float("nan")
        k[i, n + t:], v[i, n + t:] = float("nan"), float("nan")
    B.hc_kv_write(k, v, cache, zero)
    clean = torch.from_numpy(~(see[:, 4] | see[:, 5])).cuda()
    saw = torch.from_numpy(see[:, 5]).cuda()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        out2, lse2 = B.hc_tree_attention(q, cache, lens, mask=mask)
        differ += (out2[:, clean] != out[:, clean]).sum() + (lse2[:, clean] != lse[:, clean]).sum()
    assert int(differ) == 0
    assert not bool(torch.isfinite(out2[:, saw][..., 7]).any())
    assert B.device_status() == B.TS_OK


def test_attention_pages_past_2_to_31_elements():
    """A pool of more than 2^31 elements, the sequence at its end."""
    d, heads, page = 128, 8, 64
    n = (1 << 31) // (d * heads * page) + 40
    table = (torch.arange(20, dtype=torch.int32, device="cuda")[None] + n - 20).contiguous()
    g = gen(21)
    k_pool, v_pool = (torch.empty(n, heads, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = B.KVCache("bf16", k_pool, v_pool, table)
    total, t = 1200, 4
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = randn(g, 1, total, heads, d), randn(g, 1, total, heads, d)
    B.hc_kv_write(k, v, cache, zero)
    ko, vo = B.hc_kv_read(cache, zero, total)
    assert torch.equal(ko, k) and torch.equal(vo, v)
    q = randn(g, 1, t, 16, d)
    out, lse = B.hc_tree_attention(q, cache, zero + (total - t))
    check_attention(out, lse, q, cache, [total - t], [np.tril(np.ones((t, t), bool))], d ** -0.5,
                    lambda i, m: (R.f64(k[i, :m]), R.f64(v[i, :m])))


def test_attention_records_bad_lengths_and_pages():
    g = gen(22)
    cache = make_cache(g, "bf16", 2, 32, 1, 16, 64)
    k = randn(g, 2, 32, 1, 64)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    B.hc_kv_write(k, k, cache, zero)
    q = randn(g, 2, 3, 2, 64)
    for lens in ([30, 5], [-4, 5], [1 << 30, 5], [5, -2 ** 31]):
        out, _ = B.hc_tree_attention(q, cache, torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert bool(torch.isfinite(out).all())
        assert B.device_status() == B.TS_ERR_INVALID_ARG
    cache.tensors[2][0, 1] = -1
    out, _ = B.hc_tree_attention(q, cache, zero + 25)
    assert bool(torch.isfinite(out).all())
    assert B.device_status() == B.TS_ERR_INVALID_ARG


# ------------------------------------------------------------------ verification

def verify_inputs(seed, b, t, v, tree, temps, agree=0.8):
    rng = np.random.default_rng(seed)
    logits = rng.normal(size=(b, t, v)).astype(np.float32) * 2.5
    temp = np.array([temps[i % len(temps)] for i in range(b)], np.float32)
    x = logits.astype(np.float64) + rng.normal(size=(b, t, v)) * agree
    x = x / np.where(temp > 0, temp, 1)[:, None, None]
    x = np.exp(x - x.max(-1, keepdims=True))
    draft = (x / x.sum(-1, keepdims=True)).astype(np.float32)
    parents = np.zeros((b, t), np.int32)
    tokens = np.zeros((b, t), np.int32)
    for i in range(b):
        p = random_tree(rng, t) if tree else [-1] + list(range(t - 1))
        parents[i] = p
        for j in range(1, t):
            tokens[i, j] = rng.choice(v, p=draft[i, p[j]].astype(np.float64) / draft[i, p[j]].astype(np.float64).sum())
            if temp[i] <= 0 and rng.random() < 0.6:
                tokens[i, j] = logits[i, p[j]].argmax()
    u = rng.random((b, t)).astype(np.float32)
    noise = rng.exponential(size=(b, v)).astype(np.float32) + np.float32(1e-12)
    return logits, tokens, parents, temp, draft, u, noise


def check_verify(args, got, greedy=False, chain=False):
    logits, tokens, parents, temp, draft, u, noise = args
    n, path, nxt = (x.cpu().numpy() for x in got)
    for i in range(len(tokens)):
        d64 = lambda x: x[i].astype(np.float64)  # noqa: E731
        want = R.verify(d64(logits), tokens[i], None if chain else parents[i], 0.0 if greedy else float(temp[i]),
                        None if greedy else d64(draft), None if greedy else d64(u), None if greedy else d64(noise))
        if want[3] < 1e-4:
            continue  # a decision too near to call: not what this test is about
        assert n[i] == want[0] and path[i].tolist() == want[1] + [-1] * (len(tokens[i]) - len(want[1])) and nxt[i] == want[2], i


@pytest.mark.parametrize("b,t,v", [(1, 1, 1000), (1, 5, 32768), (3, 9, 50), (40, 6, 1), (7, 40, 2049), (160, 4, 501), (20, 5, 70001)])
@pytest.mark.parametrize("tree", [False, True])
def test_verify(b, t, v, tree):
    args = verify_inputs(b + t, b, t, v, tree, [0.7, 1.0, 0.0, 1.3])
    logits, tokens, parents, temp, draft, u, noise = (torch.from_numpy(x).cuda() for x in args)
    got = B.hc_verify(logits, tokens, parents, temp, draft_probs=draft, u=u, noise=noise)
    check_verify(args, got)
    if not tree:
        check_verify(args, B.hc_verify(logits, tokens, None, temp, draft_probs=draft, u=u, noise=noise), chain=True)
    check_verify(args, B.hc_verify(logits, tokens, parents), greedy=True)
    again = B.hc_verify(logits, tokens, parents, temp, draft_probs=draft, u=u, noise=noise)
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    assert B.device_status() == B.TS_OK


def test_verify_ties_and_masked_vocabulary():
    """Equal logits: the lowest index; tokens ruled out by -infinity are never taken."""
    v, t = 5000, 3
    logits = torch.full((2, t, v), -1.0, device="cuda")
    logits[:, :, 4001] = logits[:, :, 77] = 3.0
    tokens = torch.tensor([[0, 77, 77], [0, 4001, 77]], dtype=torch.int32, device="cuda")
    n, path, nxt = B.hc_verify(logits, tokens)
    assert n.tolist() == [2, 0] and nxt.tolist() == [77, 77] and path.tolist() == [[0, 1, 2], [0, -1, -1]]
    logits = torch.full((64, 1, v), float("-inf"), device="cuda")
    logits[:, 0, 123], logits[:, 0, 4321] = 0.0, 1.0
    one = torch.ones(64, device="cuda")
    noise = torch.empty(64, v, device="cuda").exponential_(generator=gen(1)).clamp(min=1e-12)
    draft = torch.full((64, 1, v), 1.0 / v, device="cuda")
    _, _, nxt = B.hc_verify(logits, torch.zeros(64, 1, dtype=torch.int32, device="cuda"), None, one, draft_probs=draft,
                            u=torch.zeros(64, 1, device="cuda"), noise=noise)
    assert set(nxt.tolist()) == {123, 4321}


def test_verify_draft_equal_to_target_accepts_everything():
    b, t, v = 8, 6, 3000
    logits = torch.randn(b, t, v, generator=gen(2), device="cuda")
    draft = torch.softmax(logits.double(), -1).float()
    tokens = torch.zeros(b, t, dtype=torch.int32, device="cuda")
    for i in range(1, t):
        tokens[:, i] = (draft[:, i - 1] / torch.empty(b, v, device="cuda").exponential_(generator=gen(i))).argmax(-1).int()
    u = torch.full((b, t), 0.999, device="cuda")
    n, _, _ = B.hc_verify(logits, tokens, None, torch.ones(b, device="cuda"), draft_probs=draft, u=u,
                          noise=torch.ones(b, v, device="cuda"))
    assert n.tolist() == [t - 1] * b


def test_verify_bad_token_is_recorded():
    logits = torch.randn(1, 3, 100, generator=gen(3), device="cuda")
    best = logits.argmax(-1)[0].tolist()
    tokens = torch.tensor([[0, 100, best[0]]], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[-1, 0, 0]], dtype=torch.int32, device="cuda")
    n, path, nxt = B.hc_verify(logits, tokens, parents)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    assert n.tolist() == [1] and path.tolist() == [[0, 2, -1]] and nxt.tolist() == [best[2]]


@pytest.mark.parametrize("children", [1, 3])
def test_verify_keeps_the_targets_distribution(children):
    """The first token that comes out, accepted or sampled, is distributed as the target: over n draws each
    frequency is within 5 sqrt(p (1 - p) / n) of p."""
    n, v, t = 40000, 7, 1 + children
    g = gen(4)
    row = torch.tensor([1.0, 0.2, -0.5, 2.0, 0.0, -3.0, 0.7], device="cuda")
    q = torch.softmax(torch.tensor([0.0, 1.5, 0.5, 0.3, -1.0, 0.0, 0.1], device="cuda"), 0)
    logits, draft = row.expand(n, t, v).contiguous(), q.expand(n, t, v).contiguous()
    tokens = torch.multinomial(q, n * t, replacement=True, generator=g).view(n, t).int()
    parents = torch.tensor([-1] + [0] * children, dtype=torch.int32, device="cuda")
    u = torch.rand(n, t, generator=g, device="cuda")
    noise = torch.empty(n, v, device="cuda").exponential_(generator=g).clamp(min=1e-12)
    count, path, nxt = B.hc_verify(logits, tokens, parents, torch.full((n,), 1.1, device="cuda"), draft_probs=draft, u=u, noise=noise)
    first = torch.where(count > 0, tokens.gather(1, path[:, 1:2].long().clamp(min=0))[:, 0], nxt)
    freq = torch.bincount(first.long(), minlength=v).double() / n
    p = torch.softmax(row.double() / 1.1, 0)
    assert bool(((freq - p).abs() <= 5 * (p * (1 - p) / n).sqrt()).all()), (freq.tolist(), p.tolist())
