"""Token scores and embedding rows without a GPU: the oracle's gradients
against differences of its values, and every refusal of the entry points."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import scores

INVALID = 1


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("masked", [0, 3])
def test_row_gradient_matches_differences(seed, masked):
    """Central differences in fp64: truncation h^2/6 |f'''| and rounding
    |f| 2^-53 / h are both below 1e-9 for h = 1e-5 and values below 10."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 2, size=17)
    x[rng.choice(17, masked, replace=False)] = -np.inf
    t = int(np.flatnonzero(x > -np.inf)[seed])
    gl, gh = rng.normal(size=2)
    want = scores.row_scores_grad(x, t, gl, gh)
    h = 1e-5
    for v in range(17):
        if x[v] == -np.inf:
            assert want[v] == 0.0
            continue
        f = []
        for step in (h, -h):
            y = x.copy()
            y[v] += step
            r = scores.row_scores(y, t)
            f.append(gl * r["logprob"] + gh * r["entropy"])
        assert abs((f[0] - f[1]) / (2 * h) - want[v]) < 1e-8


def test_embed_gradient_is_the_transpose():
    """<embed(table), dout> = <table, embed_grad(dout)>, to fp64 rounding of 60 products."""
    rng = np.random.default_rng(0)
    table, dout = rng.normal(size=(9, 4)), rng.normal(size=(15, 4))
    tokens = rng.integers(-1, 9, size=15)
    left = (scores.embed(table, tokens, 0.7) * dout).sum()
    right = (table * scores.embed_grad(dout, tokens, 0.7, None, 9)).sum()
    assert abs(left - right) < 1e-12


def test_row_scores_of_masked_rows():
    empty = scores.row_scores(np.full(5, -np.inf), 2, 3)
    assert empty["logprob"] == -np.inf and empty["entropy"] == 0 and empty["s"] == 0
    assert list(empty["top_tokens"]) == [-1, -1, -1]
    low = scores.row_scores(np.full(8, -3e38), 2, 2)
    assert abs(low["logprob"] + np.log(8)) < 1e-12 and list(low["top_tokens"]) == [0, 1]


FAKE = 4096      # never dereferenced: validation fails first
WS = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_semi_b200 import binding
    return binding.lib


def _logprobs(lib, **kw):
    a = dict(logits=FAKE, dtype=0, n_rows=8, stride=1000, row_start=FAKE, tokens=FAKE, B=2, C=3, V=1000, k=5,
             logprob=FAKE, entropy=FAKE, stats=FAKE, top=FAKE, top_lp=FAKE, ws=FAKE, ws_bytes=WS)
    a.update(kw)
    return lib.dspark_logprobs(a["logits"], a["dtype"], a["n_rows"], a["stride"], a["row_start"], a["tokens"], a["B"],
                               a["C"], a["V"], a["k"], a["logprob"], a["entropy"], a["stats"], a["top"], a["top_lp"],
                               a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=FAKE + 4), dict(tokens=None), dict(tokens=FAKE + 4), dict(logprob=None),
    dict(entropy=FAKE + 4), dict(stats=FAKE + 8), dict(row_start=FAKE + 8), dict(top=None), dict(top_lp=None),
    dict(ws=None), dict(ws_bytes=16), dict(dtype=2), dict(dtype=-1), dict(B=-1), dict(C=-1), dict(V=0),
    dict(V=(1 << 24) + 1, stride=1 << 25), dict(stride=999), dict(stride=1 << 33), dict(n_rows=-1), dict(n_rows=1 << 32, stride=1 << 32), dict(k=33),
    dict(k=-1), dict(B=1 << 13, C=(1 << 11) + 1)])
def test_logprobs_refuses(lib, bad):
    assert _logprobs(lib, **bad) == INVALID


def test_logprobs_of_nothing(lib):
    assert _logprobs(lib, B=0, logits=None, tokens=None, logprob=None) == 0
    assert _logprobs(lib, C=0) == 0
    assert _logprobs(lib, B=0, V=0) == INVALID


def _grad(lib, **kw):
    a = dict(logits=FAKE, dtype=0, stride=1000, tokens=FAKE, stats=FAKE, entropy=FAKE, g=FAKE, gh=FAKE, N=4, V=1000,
             d=2 * FAKE, gstride=1000, ws=FAKE, ws_bytes=WS)
    a.update(kw)
    return lib.dspark_logprobs_grad(a["logits"], a["dtype"], a["stride"], a["tokens"], a["stats"], a["entropy"],
                                    a["g"], a["gh"], a["N"], a["V"], a["d"], a["gstride"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=FAKE + 2), dict(tokens=None), dict(stats=None), dict(stats=FAKE + 4),
    dict(entropy=None), dict(entropy=FAKE + 4), dict(g=None), dict(gh=FAKE + 4), dict(d=None), dict(d=FAKE + 8),
    dict(dtype=3), dict(N=-1), dict(N=(1 << 24) + 1), dict(V=0), dict(stride=10), dict(gstride=10),
    dict(gstride=1 << 33), dict(d=FAKE, gstride=1001), dict(ws=None), dict(ws_bytes=0)])
def test_logprobs_grad_refuses(lib, bad):
    assert _grad(lib, **bad) == INVALID


def test_logprobs_grad_of_nothing(lib):
    assert _grad(lib, N=0, logits=None, d=None) == 0


def _embed(lib, **kw):
    a = dict(table=FAKE, td=1, tokens=FAKE, n=4, V=100, r=64, out=FAKE, od=0, ws=FAKE, ws_bytes=WS)
    a.update(kw)
    return lib.dspark_embed(a["table"], a["td"], a["tokens"], a["n"], a["V"], a["r"], 1.0, a["out"], a["od"], a["ws"],
                            a["ws_bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(table=None), dict(table=FAKE + 2), dict(tokens=None), dict(tokens=FAKE + 4), dict(out=None),
    dict(out=FAKE + 8), dict(td=2), dict(od=-1), dict(n=-1), dict(n=(1 << 24) + 1), dict(V=0), dict(V=(1 << 24) + 1),
    dict(r=0), dict(r=8193), dict(ws=None), dict(ws_bytes=100)])
def test_embed_refuses(lib, bad):
    assert _embed(lib, **bad) == INVALID


def test_embed_of_nothing(lib):
    assert _embed(lib, n=0, tokens=None, out=None) == 0


def _embed_grad(lib, **kw):
    a = dict(dout=FAKE, dd=1, tokens=FAKE, n=4, V=100, r=64, acc=0, d=FAKE, td=0, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return lib.dspark_embed_grad(a["dout"], a["dd"], a["tokens"], a["n"], a["V"], a["r"], 1.0, a["acc"], a["d"],
                                 a["td"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(dout=None), dict(dout=FAKE + 2), dict(tokens=None), dict(tokens=FAKE + 4), dict(d=None), dict(d=FAKE + 8),
    dict(dd=2), dict(td=9), dict(acc=2), dict(acc=-1), dict(n=-1), dict(n=(1 << 24) + 1), dict(V=0),
    dict(V=(1 << 24) + 1), dict(r=0), dict(r=8193), dict(ws=None), dict(ws_bytes=100)])
def test_embed_grad_refuses(lib, bad):
    assert _embed_grad(lib, **bad) == INVALID


def test_embed_grad_workspace(lib):
    f = lib.dspark_embed_grad_workspace_bytes
    assert f(0, 1, 1) > 0 and f(1 << 24, 1 << 24, 8192) > 0
    for n, V, r in ((-1, 10, 10), (10, 0, 10), (10, 10, 0), (10, 10, 8193), ((1 << 24) + 1, 10, 10)):
        assert f(n, V, r) == 0
    need = f(100000, 1000, 64)
    assert _embed_grad(lib, n=100000, V=1000, ws_bytes=need - 1) == INVALID


def test_binding_refuses_before_any_call():
    """Types, shapes and devices, on CPU tensors (the library computes on the GPU only)."""
    from speculative_decoding_semi_b200 import binding as b
    f, i = torch.zeros(4, 8), torch.zeros(2, 2, dtype=torch.int32)
    ws = torch.zeros(8192, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        b.dspark_logprobs(f, i, f, None, None, None, None, ws)
    with pytest.raises(TypeError):
        b.dspark_logprobs(f.half(), i, f, None, None, None, None, ws)
    with pytest.raises(TypeError):
        b.dspark_logprobs_grad(f, i, f, None, f, None, f.bfloat16(), ws)
    with pytest.raises(ValueError):
        b.dspark_embed(f, i, 1.0, f, ws)
    with pytest.raises(ValueError):
        b.dspark_embed_grad(f, i, 1.0, f, ws)
    with pytest.raises(b.DSparkError):
        b.dspark_embed_grad_workspace_bytes(4, 0, 4)
