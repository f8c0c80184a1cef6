"""Refusals and no-ops of the prompt operators' entry points: every call here fails argument validation or has
nothing to do, so no CUDA call is made. And the tests' own 64-bit reference, against closed forms and torch."""
import numpy as np
import pytest
import torch

import prompt_reference as P
from hyper_connection_residual_call_gb300 import binding as B
from hyper_connection_residual_call_gb300.build import build

MB = 1 << 20
FAKE = 0x10000000  # an aligned address that is never dereferenced: validation fails first
INVALID, UNSUPPORTED, WORKSPACE = B.TS_ERR_INVALID_ARG, B.TS_ERR_UNSUPPORTED, B.TS_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return B.library()


def refused(st, status, needle):
    assert st == status, B.ts_hc_last_error()
    assert needle in B.ts_hc_last_error()


def norm_rope(**kw):
    a = dict(q=FAKE, sq=512, k=FAKE + MB, sk=256, pos=FAKE + 2 * MB, table=FAKE + 3 * MB, max_pos=100, qw=FAKE + 4 * MB, kw=FAKE + 5 * MB,
             eps=1e-6, qo=FAKE + 6 * MB, sqo=512, ko=FAKE + 7 * MB, sko=256, N=2, hq=4, hk=2, D=128, rot=64)
    a.update(kw)
    return B.ts_hc_qk_norm_rope(a["q"], a["sq"], a["k"], a["sk"], a["pos"], a["table"], a["max_pos"], a["qw"], a["kw"], a["eps"], a["qo"],
                                a["sqo"], a["ko"], a["sko"], a["N"], a["hq"], a["hk"], a["D"], a["rot"], 0, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(N=-1), INVALID, "N = -1"), (dict(hq=0), INVALID, "q_heads = 0"), (dict(hk=-1), INVALID, "k_heads"),
    (dict(D=100), INVALID, "D = 100"), (dict(D=0), INVALID, "D = 0"), (dict(D=1032), INVALID, "D = 1032"),
    (dict(rot=3), INVALID, "rot = 3"), (dict(rot=130), INVALID, "rot = 130"), (dict(max_pos=0), INVALID, "max_pos = 0"),
    (dict(eps=0.0), INVALID, "eps = 0"), (dict(eps=-1.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"),
    (dict(eps=float("inf")), INVALID, "eps"), (dict(q=None), INVALID, "q is NULL"), (dict(q=FAKE + 8), INVALID, "q is not 16-byte"),
    (dict(k=None), INVALID, "k is NULL"), (dict(qw=None), INVALID, "q_norm_w is NULL"), (dict(kw=FAKE + 2), INVALID, "k_norm_w"),
    (dict(pos=None), INVALID, "positions"), (dict(table=FAKE + 4), INVALID, "table"), (dict(sq=504), INVALID, "q_stride = 504"),
    (dict(sk=260), INVALID, "k_stride = 260"), (dict(sqo=8), INVALID, "q_out_stride"), (dict(sko=8), INVALID, "k_out_stride"),
    (dict(qo=FAKE + 64), INVALID, "q_out overlaps q"), (dict(qo=FAKE, sqo=1024), INVALID, "q_out is q but"),
    (dict(ko=FAKE + 7 * MB, k=FAKE + 7 * MB, sko=512), INVALID, "k_out is k but"), (dict(ko=FAKE + 6 * MB), INVALID, "q_out overlaps k_out"),
    (dict(qo=FAKE + MB), INVALID, "q_out overlaps k"), (dict(ko=FAKE), INVALID, "k_out overlaps q"),
    (dict(qw=FAKE + 6 * MB), INVALID, "an output overlaps"), (dict(pos=FAKE + 7 * MB), INVALID, "an output overlaps"),
    (dict(table=FAKE + 6 * MB), INVALID, "an output overlaps"),
    (dict(N=1 << 27, q=FAKE, sq=1 << 12), UNSUPPORTED, "too many for one call"),
])
def test_norm_rope_refusals(kw, status, needle):
    refused(norm_rope(**kw), status, needle)


def attention(**kw):
    a = dict(q=FAKE, sq=512, k=FAKE + MB, sk=256, v=FAKE + 2 * MB, sv=256, starts=FAKE + 3 * MB, out=FAKE + 4 * MB, lse=FAKE + 5 * MB, N=10, S=2,
             hq=4, hk=2, D=128, scale=1.0)
    a.update(kw)
    return B.ts_hc_prompt_attention(a["q"], a["sq"], a["k"], a["sk"], a["v"], a["sv"], a["starts"], a["out"], a["lse"], a["N"], a["S"], a["hq"],
                                    a["hk"], a["D"], a["scale"], None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(N=-1), INVALID, "N = -1"), (dict(S=-1), INVALID, "S = -1"), (dict(S=65536), INVALID, "S = 65536"), (dict(hq=0), INVALID, "q_heads = 0"),
    (dict(hk=0), INVALID, "kv_heads = 0"), (dict(hq=5), INVALID, "q_heads = 5 must be a multiple"), (dict(D=256), UNSUPPORTED, "D = 256"),
    (dict(D=80), UNSUPPORTED, "D = 80"), (dict(scale=0.0), INVALID, "scale = 0"), (dict(scale=-1.0), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"), (dict(scale=float("nan")), INVALID, "scale"), (dict(q=None), INVALID, "q is NULL"),
    (dict(k=FAKE + 8), INVALID, "k is not"), (dict(v=None), INVALID, "v is NULL"), (dict(sq=511), INVALID, "q_stride"),
    (dict(sk=128), INVALID, "k_stride = 128"), (dict(sv=260), INVALID, "v_stride = 260"), (dict(starts=None), INVALID, "starts"),
    (dict(out=FAKE + 4 * MB + 2), INVALID, "out is not"), (dict(lse=FAKE + 1), INVALID, "lse"), (dict(out=FAKE), INVALID, "out overlaps q"),
    (dict(out=FAKE + MB), INVALID, "out overlaps k"), (dict(out=FAKE + 2 * MB), INVALID, "out overlaps v"),
])
def test_attention_refusals(kw, status, needle):
    refused(attention(**kw), status, needle)


def step(**kw):
    a = dict(q=FAKE, sq=256, k=FAKE + MB, sk=256, v=FAKE + 2 * MB, sv=512, decay=FAKE + 3 * MB, beta=FAKE + 4 * MB, counts=FAKE + 5 * MB,
             si=FAKE + 6 * MB, so=FAKE + 8 * MB, out=FAKE + 10 * MB, B=2, T=3, hk=2, hv=4, D=128, scale=1.0, eps=1e-6)
    a.update(kw)
    return B.ts_hc_delta_step(a["q"], a["sq"], a["k"], a["sk"], a["v"], a["sv"], a["decay"], a["beta"], a["counts"], a["si"], a["so"],
                              a["out"], a["B"], a["T"], a["hk"], a["hv"], a["D"], a["scale"], a["eps"], None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(B=-1), INVALID, "B = -1"), (dict(B=65536), INVALID, "B = 65536"), (dict(T=4097), INVALID, "T = 4097"),
    (dict(hk=0), INVALID, "k_heads = 0"), (dict(hv=5), INVALID, "v_heads = 5 must be a multiple"), (dict(hv=0), INVALID, "v_heads = 0"),
    (dict(D=256), UNSUPPORTED, "D = 256"), (dict(D=96), UNSUPPORTED, "D = 96"), (dict(scale=float("nan")), INVALID, "scale"),
    (dict(eps=float("inf")), INVALID, "norm_eps"), (dict(q=None), INVALID, "q is NULL"), (dict(k=FAKE + 2), INVALID, "k is not"),
    (dict(v=None), INVALID, "v is NULL"), (dict(sq=128), INVALID, "q_stride = 128"), (dict(sk=257), INVALID, "k_stride = 257"),
    (dict(sv=256), INVALID, "v_stride = 256"), (dict(decay=None), INVALID, "decay"), (dict(beta=FAKE + 2), INVALID, "beta"),
    (dict(out=None), INVALID, "out is NULL"), (dict(counts=FAKE + 1), INVALID, "counts"), (dict(si=None), INVALID, "state_in"),
    (dict(so=FAKE + 4), INVALID, "state_out"), (dict(so=FAKE + 6 * MB + 64), INVALID, "state_out overlaps state_in"),
    (dict(out=FAKE), INVALID, "out overlaps q"), (dict(out=FAKE + MB), INVALID, "out overlaps k"),
    (dict(out=FAKE + 2 * MB), INVALID, "out overlaps v"), (dict(out=FAKE + 3 * MB), INVALID, "out overlaps decay"),
    (dict(out=FAKE + 6 * MB), INVALID, "out overlaps the states"),
])
def test_delta_step_refusals(kw, status, needle):
    refused(step(**kw), status, needle)


def prompt(**kw):
    a = dict(q=FAKE, sq=256, k=FAKE + MB, sk=256, v=FAKE + 2 * MB, sv=512, decay=FAKE + 3 * MB, beta=FAKE + 4 * MB, starts=FAKE + 5 * MB,
             si=FAKE + 6 * MB, so=FAKE + 8 * MB, out=FAKE + 10 * MB, N=100, S=3, hk=2, hv=4, D=128, scale=1.0, eps=1e-6, ws=FAKE + 16 * MB,
             n=1 << 30)
    a.update(kw)
    return B.ts_hc_delta_prompt(a["q"], a["sq"], a["k"], a["sk"], a["v"], a["sv"], a["decay"], a["beta"], a["starts"], a["si"], a["so"],
                                a["out"], a["N"], a["S"], a["hk"], a["hv"], a["D"], a["scale"], a["eps"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(N=-1), INVALID, "N = -1"), (dict(S=65536), INVALID, "S = 65536"), (dict(hk=3), INVALID, "v_heads = 4 must be a multiple"),
    (dict(D=32), UNSUPPORTED, "D = 32"), (dict(scale=float("inf")), INVALID, "scale"), (dict(eps=float("nan")), INVALID, "norm_eps"),
    (dict(q=None), INVALID, "q is NULL"), (dict(sk=8), INVALID, "k_stride = 8"), (dict(sv=511), INVALID, "v_stride"),
    (dict(beta=None), INVALID, "beta"), (dict(starts=None), INVALID, "starts"), (dict(si=FAKE + 4), INVALID, "state_in"),
    (dict(so=FAKE + 6 * MB + 16), INVALID, "state_out overlaps state_in"), (dict(out=FAKE + 2 * MB), INVALID, "out overlaps v"),
    (dict(out=FAKE + 8 * MB), INVALID, "out overlaps the states"), (dict(ws=None), WORKSPACE, "needed"), (dict(n=1000), WORKSPACE, "1000 bytes given"),
    (dict(ws=FAKE + 16 * MB + 64), INVALID, "workspace"),
])
def test_delta_prompt_refusals(kw, status, needle):
    refused(prompt(**kw), status, needle)


def test_delta_prompt_workspace():
    of = B.ts_hc_delta_prompt_workspace_bytes
    one = of(64, 0, 1, 1, 128)
    assert of(64, 0, 1, 1, 64) < one and of(100, 3, 1, 1, 128) == 4 * one and of(100, 3, 5, 5, 128) == 20 * one
    assert of(100, 3, 2, 5, 128) == 0 and "v_heads = 5" in B.ts_hc_last_error()
    assert of(1 << 30, 65535, 64, 64, 128) == ((1 << 24) + 65535) * 64 * one  # past 32 bits


def logprobs(**kw):
    a = dict(logits=FAKE, type=B.TS_LOGITS_FP32, stride=1000, tokens=FAKE + MB, logp=FAKE + 2 * MB, entropy=FAKE + 3 * MB, ids=FAKE + 4 * MB,
             best=FAKE + 5 * MB, N=4, V=1000, J=2, top=3)
    a.update(kw)
    return B.ts_hc_logprobs(a["logits"], a["type"], a["stride"], a["tokens"], a["logp"], a["entropy"], a["ids"], a["best"], a["N"], a["V"],
                            a["J"], a["top"], None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(N=-1), INVALID, "N = -1"), (dict(V=0), INVALID, "V = 0"), (dict(V=1 << 30), INVALID, "V = "), (dict(J=-1), INVALID, "J = -1"),
    (dict(top=33), INVALID, "top = 33"), (dict(top=-1), INVALID, "top = -1"), (dict(V=8, stride=8, top=9), INVALID, "top = 9"),
    (dict(type=2), INVALID, "logits_type = 2"), (dict(logits=None), INVALID, "logits is NULL"), (dict(logits=FAKE + 2), INVALID, "logits is not"),
    (dict(stride=999), INVALID, "logits_stride = 999"), (dict(tokens=None), INVALID, "tokens"), (dict(logp=None), INVALID, "logp"),
    (dict(entropy=FAKE + 2), INVALID, "entropy"), (dict(ids=None), INVALID, "top_ids"), (dict(best=None), INVALID, "top_logp"),
    (dict(J=0, entropy=None, top=0), INVALID, "nothing is asked for"), (dict(logp=FAKE + 8), INVALID, "logp overlaps logits"),
    (dict(logp=FAKE + MB), INVALID, "logp overlaps tokens"), (dict(ids=FAKE + 5 * MB), INVALID, "top_ids overlaps top_logp"),
    (dict(entropy=FAKE + 2 * MB), INVALID, "logp overlaps entropy"),
])
def test_logprobs_refusals(kw, status, needle):
    refused(logprobs(**kw), status, needle)


def test_nothing_to_do():
    assert norm_rope(N=0, q=None, qo=None) == B.TS_OK
    assert attention(N=0, q=None) == B.TS_OK
    assert attention(S=0, q=None) == B.TS_OK
    assert step(B=0, q=None) == B.TS_OK
    assert step(T=0, q=None, out=None) == B.TS_OK
    assert prompt(N=0, q=None, ws=None) == B.TS_OK
    assert prompt(S=0, q=None, ws=None) == B.TS_OK
    assert logprobs(N=0, logits=None) == B.TS_OK


# ------------------------------------------------------------------ the reference itself

def test_reference_delta_is_the_least_squares_step():
    """With beta 1, no decay and a key of norm 1, the state's answer to the key is the value."""
    r = np.random.default_rng(0)
    k = r.normal(size=(1, 1, 64))
    k /= np.linalg.norm(k)
    v = r.normal(size=(1, 1, 64))
    out, S, _ = P.delta(k, k, v, np.zeros((1, 1)), np.ones((1, 1)), r.normal(size=(1, 64, 64)), 1.0, None)
    assert np.allclose(S[0].T @ k[0, 0], v[0, 0]) and np.allclose(out[0, 0], v[0, 0])


def test_reference_norm_rope_keeps_lengths():
    r = np.random.default_rng(1)
    x, angle = r.normal(size=(3, 2, 16)), r.normal(size=(5, 8))
    n, y = P.norm_rope(x, np.ones(16), 1e-12, [0, 4, 2], np.stack([np.cos(angle), np.sin(angle)], -1), True)
    assert np.allclose((n * n).mean(-1), 1) and np.allclose((y * y).sum(-1), (n * n).sum(-1))


def test_reference_logprobs_match_torch():
    x = torch.randn(50, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    lp, h, _, _, order = P.logprobs(x.numpy())
    want = torch.log_softmax(x, 0)
    assert np.allclose(lp, want) and np.isclose(h, -(want.exp() * want).sum()) and order[0] == int(x.argmax())


# ------------------------------------------------------------------ outputs over what else a call reads or writes

@pytest.mark.parametrize("kw,needle", [
    (dict(starts=FAKE + 4 * MB), "out overlaps starts"), (dict(lse=FAKE + 4 * MB), "out overlaps lse"), (dict(lse=FAKE + 64), "lse overlaps q"),
    (dict(lse=FAKE + MB), "lse overlaps k"), (dict(lse=FAKE + 2 * MB), "lse overlaps v"), (dict(lse=FAKE + 3 * MB, starts=FAKE + 3 * MB), "lse overlaps starts"),
])
def test_attention_outputs_apart(kw, needle):
    refused(attention(**kw), INVALID, needle)


@pytest.mark.parametrize("kw,needle", [
    (dict(so=FAKE), "state_out overlaps q"), (dict(so=FAKE + MB), "state_out overlaps k"), (dict(so=FAKE + 2 * MB), "state_out overlaps v"),
    (dict(so=FAKE + 3 * MB), "state_out overlaps decay"), (dict(so=FAKE + 4 * MB), "state_out overlaps beta"),
    (dict(so=FAKE + 5 * MB), "state_out overlaps counts"), (dict(counts=FAKE + 10 * MB), "out overlaps counts"),
])
def test_delta_step_outputs_apart(kw, needle):
    refused(step(**kw), INVALID, needle)


@pytest.mark.parametrize("kw,needle", [
    (dict(so=FAKE), "state_out overlaps q"), (dict(so=FAKE + 5 * MB), "state_out overlaps starts"), (dict(starts=FAKE + 10 * MB), "out overlaps starts"),
    (dict(ws=FAKE), "workspace overlaps q"), (dict(ws=FAKE + 2 * MB + 256), "workspace overlaps v"), (dict(ws=FAKE + 6 * MB), "workspace overlaps state_in"),
    (dict(ws=FAKE + 8 * MB + 512), "state_out overlaps workspace"), (dict(ws=FAKE + 10 * MB), "out overlaps workspace"),
    (dict(ws=FAKE + 4 * MB), "workspace overlaps beta"),
])
def test_delta_prompt_outputs_apart(kw, needle):
    refused(prompt(**kw), INVALID, needle)
