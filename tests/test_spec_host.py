"""Refusals and no-ops of the speculative decoding step's entry points: every call here fails argument
validation or has nothing to do, so no CUDA call is made. And the tests' own 64-bit reference, against
closed forms and torch."""
import ctypes

import numpy as np
import pytest
import torch

import spec_reference as R
from hyper_connection_residual_call_gb300 import binding as B
from hyper_connection_residual_call_gb300.build import build

FAKE = 0x10000  # an aligned address that is never dereferenced: validation fails first
INVALID, UNSUPPORTED, WORKSPACE = B.TS_ERR_INVALID_ARG, B.TS_ERR_UNSUPPORTED, B.TS_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return B.library()


def refused(st, status, needle):
    assert st == status, B.ts_hc_last_error()
    assert needle in B.ts_hc_last_error()


def cache(**kw):
    c = B.TsHcKvCache(B.TS_KV_INT4, 64, 16, 4, 128, 10, 100, *([FAKE] * 7))
    for name, v in kw.items():
        setattr(c, name, v)
    return c


@pytest.mark.parametrize("kw,status,needle", [
    (dict(type=3), INVALID, "cache.type = 3"), (dict(type=-1), INVALID, "cache.type"),
    (dict(head_dim=96), UNSUPPORTED, "head_dim = 96"), (dict(head_dim=64, group=128), UNSUPPORTED, "group = 128"),
    (dict(group=16), UNSUPPORTED, "group = 16"), (dict(page_size=24), INVALID, "page_size = 24"),
    (dict(page_size=8), INVALID, "page_size = 8"), (dict(page_size=2048), INVALID, "page_size"),
    (dict(n_kv_heads=0), INVALID, "n_kv_heads = 0"), (dict(max_pages=0), INVALID, "max_pages = 0"),
    (dict(max_pages=1 << 27), INVALID, "max_pages"), (dict(n_pages=0), INVALID, "n_pages = 0"), (dict(n_pages=1 << 31), INVALID, "n_pages"),
    (dict(k=None), INVALID, "cache.k is NULL"), (dict(v=FAKE + 8), INVALID, "cache.v is not 16-byte aligned"),
    (dict(k_scales=None), INVALID, "cache.k_scales"), (dict(v_scales=None), INVALID, "cache.v_scales"),
    (dict(k_biases=None), INVALID, "cache.k_biases"), (dict(v_biases=FAKE + 2), INVALID, "cache.v_biases"),
    (dict(page_table=None), INVALID, "cache.page_table"),
])
def test_every_call_checks_the_cache(kw, status, needle):
    c = cache(**kw)
    refused(B.ts_hc_kv_write(FAKE, 512, FAKE, 512, c, FAKE, 1, 1, None), status, needle)
    refused(B.ts_hc_kv_read(c, FAKE, FAKE, FAKE, 1, 1, None), status, needle)
    refused(B.ts_hc_kv_compact(c, FAKE, FAKE, FAKE, None, 1, 1, None), status, needle)
    refused(B.ts_hc_tree_attention(FAKE, 1024, c, FAKE, None, 0, FAKE, None, 1, 1, 8, 1.0, FAKE, 1 << 30, None), status, needle)
    refused(B.ts_hc_kv_write(FAKE, 512, FAKE, 512, None, FAKE, 1, 1, None), INVALID, "cache is NULL")


def rope(**kw):
    a = dict(q=FAKE, sq=512, k=FAKE + (1 << 20), sk=256, pos=FAKE, table=FAKE, max_pos=100, qo=FAKE + (2 << 20), sqo=512,
             ko=FAKE + (3 << 20), sko=256, N=2, hq=4, hk=2, D=128, rot=64)
    a.update(kw)
    return B.ts_hc_rope(a["q"], a["sq"], a["k"], a["sk"], a["pos"], a["table"], a["max_pos"], a["qo"], a["sqo"], a["ko"], a["sko"], a["N"],
                        a["hq"], a["hk"], a["D"], a["rot"], 0, 0, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(q=None), INVALID, "q is NULL"), (dict(q=FAKE + 2), INVALID, "q is not 16-byte"), (dict(qo=None), INVALID, "q_out is NULL"),
    (dict(k=None), INVALID, "k is NULL"), (dict(ko=None), INVALID, "k_out is NULL"), (dict(pos=None), INVALID, "positions"),
    (dict(table=None), INVALID, "table"), (dict(N=-1), INVALID, "N = -1"), (dict(hq=0), INVALID, "q_heads = 0"),
    (dict(hk=-1), INVALID, "k_heads"), (dict(D=12), INVALID, "D = 12"), (dict(rot=63), INVALID, "rot = 63"), (dict(rot=130), INVALID, "rot = 130"),
    (dict(rot=0), INVALID, "rot = 0"), (dict(max_pos=0), INVALID, "max_pos"), (dict(sq=500), INVALID, "q_stride = 500"),
    (dict(sqo=516), INVALID, "q_out_stride"), (dict(sk=248), INVALID, "k_stride"), (dict(sko=0), INVALID, "k_out_stride"),
    (dict(qo=FAKE, sqo=520), INVALID, "q_out is q"), (dict(qo=FAKE + 1024), INVALID, "q_out overlaps q"),
    (dict(qo=FAKE + (1 << 20)), INVALID, "q_out overlaps k"), (dict(ko=FAKE), INVALID, "k_out overlaps q"),
    (dict(ko=FAKE + (2 << 20)), INVALID, "q_out overlaps k_out"), (dict(N=1 << 28), UNSUPPORTED, "split"),
])
def test_rope_refuses(kw, status, needle):
    refused(rope(**kw), status, needle)


def test_rope_table_refuses():
    def table(t=FAKE, n=10, rot=64, theta=1e4, **sc):
        s = dict(type=B.TS_ROPE_PLAIN, factor=2.0, original_positions=100.0, beta_fast=32.0, beta_slow=1.0, magnitude=1.0)
        s.update(sc)
        return B.ts_hc_rope_table(t, n, rot, theta, B.TsHcRopeScaling(**s), None)

    nan = float("nan")
    for kw, needle in ((dict(t=None), "table"), (dict(n=-1), "max_pos"), (dict(rot=3), "rot = 3"), (dict(theta=1.0), "theta"),
                       (dict(theta=nan), "theta"), (dict(type=4), "scaling.type"), (dict(magnitude=0.0), "magnitude"),
                       (dict(type=1, factor=0.0), "factor"), (dict(type=2, rot=2), "rot = 2"), (dict(type=3, beta_fast=1.0), "beta_fast"),
                       (dict(type=3, original_positions=0.0), "original_positions"), (dict(type=3, beta_slow=nan), "beta_slow")):
        refused(table(**kw), INVALID, needle)
    assert table(t=None, n=0) == B.TS_OK


def test_cache_calls_refuse():
    c = cache()
    w = lambda **kw: B.ts_hc_kv_write(*{**dict(k=FAKE, sk=512, v=FAKE, sv=512, c=c, n=FAKE, B=1, T=1, s=None), **kw}.values())  # noqa: E731
    for kw, needle in ((dict(k=None), "k is NULL"), (dict(v=FAKE + 2), "v is not"), (dict(sk=504), "k_stride"), (dict(sv=515), "v_stride"),
                       (dict(n=None), "ctx_len"), (dict(B=-1), "B = -1"), (dict(T=-1), "T = -1"), (dict(B=65536), "B = 65536")):
        refused(w(**kw), INVALID, needle)
    refused(w(B=60000, T=60000), UNSUPPORTED, "split")
    r = lambda **kw: B.ts_hc_kv_read(*{**dict(c=c, s=FAKE, k=FAKE, v=FAKE, B=1, n=1, st=None), **kw}.values())  # noqa: E731
    for kw, needle in ((dict(s=None), "start"), (dict(k=None), "k_out"), (dict(v=FAKE + 4), "v_out"), (dict(n=-2), "n = -2")):
        refused(r(**kw), INVALID, needle)
    m = lambda **kw: B.ts_hc_kv_compact(*{**dict(c=c, n=FAKE, p=FAKE, a=FAKE, new=None, B=2, T=3, s=None), **kw}.values())  # noqa: E731
    for kw, needle in ((dict(n=None), "ctx_len"), (dict(p=None), "path"), (dict(a=None), "n_accepted"), (dict(new=FAKE + 4), "new_len overlaps"),
                       (dict(T=4097), "T = 4097")):
        refused(m(**kw), INVALID, needle)


def test_tree_build_refuses():
    t = lambda **kw: B.ts_hc_tree_build(*{**dict(p=FAKE, sp=4, c=None, m=FAKE, pos=FAKE, B=2, T=4, s=None), **kw}.values())  # noqa: E731
    for kw, needle in ((dict(p=None), "parents"), (dict(sp=3), "parents_stride"), (dict(m=None, pos=None), "both NULL"), (dict(m=FAKE + 1), "mask"),
                       (dict(c=FAKE + 2), "ctx_len"), (dict(T=5000), "T = 5000")):
        refused(t(**kw), INVALID, needle)


def attention(**kw):
    a = dict(q=FAKE, sq=1024, c=cache(), n=FAKE, m=FAKE, sm=0, o=FAKE, l=FAKE, B=2, T=40, h=8, s=0.1, ws=FAKE, b=1 << 30, st=None)
    a.update(kw)
    return B.ts_hc_tree_attention(*a.values())


@pytest.mark.parametrize("kw,status,needle", [
    (dict(q=None), INVALID, "q is NULL"), (dict(sq=1016), INVALID, "q_stride"), (dict(n=None), INVALID, "ctx_len"),
    (dict(m=FAKE + 2), INVALID, "mask"), (dict(sm=79), INVALID, "mask_stride = 79"), (dict(o=None), INVALID, "out is NULL"),
    (dict(o=FAKE + 8), INVALID, "out is not"), (dict(l=FAKE + 2), INVALID, "lse"), (dict(h=6), INVALID, "q_heads = 6"), (dict(h=0), INVALID, "q_heads"),
    (dict(s=float("nan")), INVALID, "scale"), (dict(s=float("inf")), INVALID, "scale"), (dict(ws=None), WORKSPACE, "workspace of 0 bytes"),
    (dict(b=100), WORKSPACE, "workspace of 100 bytes"), (dict(ws=FAKE + 16), INVALID, "workspace"), (dict(T=-1), INVALID, "T = -1"),
    (dict(T=4096, h=4 * 16), UNSUPPORTED, "32768 rows"), (dict(B=-3), INVALID, "B = -3"),
])
def test_attention_refuses(kw, status, needle):
    refused(attention(**kw), status, needle)


def test_attention_workspace():
    assert B.ts_hc_tree_attention_workspace_bytes(1, 1, 7, cache()) == 0  # not a multiple of the key heads
    few, many = (B.ts_hc_tree_attention_workspace_bytes(1, t, 8, cache()) for t in (1, 64))
    assert 0 < few <= many
    assert B.ts_hc_tree_attention_workspace_bytes(64, 1, 8, cache()) >= few


def verify(**kw):
    a = dict(l=FAKE, d=FAKE, t=FAKE, p=FAKE, sp=0, temp=FAKE, u=FAKE, n=FAKE, na=FAKE, path=FAKE, nt=FAKE, B=1, T=4, V=100, s=None)
    a.update(kw)
    return B.ts_hc_verify(*a.values())


@pytest.mark.parametrize("kw,needle", [
    (dict(l=None), "logits"), (dict(t=None), "tokens"), (dict(d=None), "given together"), (dict(u=None), "given together"),
    (dict(n=None), "given together"), (dict(temp=None), "temperature"), (dict(sp=3), "parents_stride"), (dict(p=FAKE + 1), "parents"),
    (dict(na=None), "n_accepted"), (dict(path=None), "path"), (dict(nt=None), "next_token"), (dict(V=0), "V = 0"), (dict(V=1 << 30), "V ="),
    (dict(T=-1), "T = -1"), (dict(B=70000), "B = 70000"),
])
def test_verify_refuses(kw, needle):
    refused(verify(**kw), INVALID, needle)


def test_nothing_to_do_is_a_noop():
    c = B.TsHcKvCache(B.TS_KV_BF16, 0, 16, 1, 64, 1, 1, *([None] * 7))  # pointers are not examined
    for st in (B.ts_hc_rope(None, 0, None, 0, None, None, 1, None, 0, None, 0, 0, 1, 0, 64, 64, 0, 0, None),
               B.ts_hc_kv_write(None, 0, None, 0, c, None, 0, 5, None), B.ts_hc_kv_write(None, 0, None, 0, c, None, 5, 0, None),
               B.ts_hc_kv_read(c, None, None, None, 3, 0, None), B.ts_hc_kv_compact(c, None, None, None, None, 0, 1, None),
               B.ts_hc_tree_build(None, 0, None, None, None, 1, 0, None),
               B.ts_hc_tree_attention(None, 0, c, None, None, 0, None, None, 0, 4, 2, 1.0, None, 0, None),
               B.ts_hc_verify(None, None, None, None, 0, None, None, None, None, None, None, 4, 0, 10, None)):
        assert st == B.TS_OK and B.ts_hc_last_error() == ""


def test_binding_refuses_what_is_not_on_the_gpu():
    t = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: B.hc_rope(t, None, table, torch.zeros(4, 4, 2)), lambda: B.KVCache("bf16", t, t, table),
                 lambda: B.KVCache("fp16", t, t, table), lambda: B.hc_tree_build(table),
                 lambda: B.hc_verify(torch.zeros(1, 1, 4), table)):
        with pytest.raises(B.HCError):
            call()


# ---- the reference itself

def test_reference_e4m3_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(R.E4M3, codes.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    x = np.random.default_rng(0).normal(size=4096)
    x[:16] = np.arange(16) * 0.0625 + 448 - 16  # ties among the largest codes
    codes, byte, vals = R.fp8_row(x)
    s = 2.0 ** (byte - 127)
    assert 224 * s < np.abs(x).max() <= 448 * s
    assert np.array_equal(vals, torch.from_numpy(x / s).float().to(torch.float8_e4m3fn).double().numpy() * s)


def test_reference_attention_is_torchs():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(3, 4, 64)), rng.normal(size=(8, 2, 64)), rng.normal(size=(8, 2, 64))
    see = R.sees([-1, 0, 0])
    out, lse, _, _ = R.attention(q, k, v, 5, see, 0.2)
    mask = np.concatenate([np.ones((3, 5), bool), see], 1)
    tt = lambda x: torch.from_numpy(x).transpose(0, 1)  # noqa: E731
    want = torch.nn.functional.scaled_dot_product_attention(tt(q)[None], tt(k).repeat_interleave(2, 0)[None], tt(v).repeat_interleave(2, 0)[None],
                                                            attn_mask=torch.from_numpy(mask), scale=0.2)[0]
    assert np.abs(out - want.transpose(0, 1).numpy()).max() < 1e-12
    assert lse.shape == (3, 4)


def test_reference_verification_keeps_the_distribution():
    rng = np.random.default_rng(2)
    row, q = np.array([[0.3, 1.0, -1.0]] * 2), np.array([[0.2, 0.3, 0.5]] * 2)
    p = np.exp(row[0]) / np.exp(row[0]).sum()
    n, seen = 20000, np.zeros(3)
    for _ in range(n):
        tok = [0, rng.choice(3, p=q[0])]
        c, path, nxt, _ = R.verify(row, tok, None, 1.0, q, rng.random(2), rng.exponential(size=3))
        seen[tok[1] if c else nxt] += 1
    assert (np.abs(seen / n - p) <= 5 * np.sqrt(p * (1 - p) / n)).all()
    assert ctypes.sizeof(B.TsHcKvCache) == 88
