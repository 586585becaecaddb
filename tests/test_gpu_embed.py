"""dspark_embed and dspark_embed_grad against the fp64 oracle.

Tolerances: a lookup is one fp32 product rounded to the output's type. A
gradient of c terms is an fp32 sum in some order, at most c - 1 roundings of
partial sums that are below the sum of magnitudes, one rounding for the scale
and its product each, one for the addition to the table and one of its type."""
import numpy as np
import pytest
import torch

from oracle import scores

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _binding():
    from speculative_decoding_semi_b200 import binding
    return binding


def _ws(n, V, r):
    b = _binding()
    ws = torch.empty(b.dspark_embed_grad_workspace_bytes(n, V, r), dtype=torch.uint8, device="cuda")
    b.dspark_workspace_init(ws)
    return ws


def _array(shape, dtype, rng):
    t = torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(DT[dtype])
    return t.cuda(), t.double().numpy()


TYPES = [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")]


@pytest.mark.parametrize("ti,to", TYPES)
@pytest.mark.parametrize("n,V,r", [(1, 1, 1), (5, 9, 3), (70, 100, 8), (33, 50, 20), (200, 1000, 100), (64, 5000, 256),
                                   (1000, 300, 129), (300, 700, 1000), (100, 64, 4096), (9, 20, 8192), (4001, 90, 64)])
def test_embed(n, V, r, ti, to):
    b = _binding()
    rng = np.random.default_rng(n + V + r)
    table, held = _array((V, r), ti, rng)
    tokens = rng.integers(-1, V, size=n).astype(np.int32)
    tokens[-1] = V - 1
    scale = 1.7
    out = torch.full((n, r), 7.0, dtype=DT[to], device="cuda")
    ws = _ws(0, 1, 1)
    b.dspark_embed(table, torch.from_numpy(tokens).cuda(), scale, out, ws)
    assert b.dspark_read_device_error(ws)[0] == 0
    want = scores.embed(held, tokens, float(np.float32(scale)))
    eps = torch.finfo(DT[to]).eps / 2
    tol = np.abs(want) * (U + eps * (1 + U)) + 1e-45
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)


def test_embed_far_rows_and_bad_tokens():
    """Rows past 2^31 elements of the table (4.4 GB of bf16, of which two rows are written); bad ids give zeros."""
    b = _binding()
    V, r = 270000, 8192
    table = torch.empty(V, r, dtype=torch.bfloat16, device="cuda")
    table[V - 1], table[0] = 3.0, 2.0
    tokens = torch.tensor([V - 1, 0, V, -1, -3], dtype=torch.int32, device="cuda")
    out = torch.full((5, r), 7.0, device="cuda")
    ws = _ws(0, 1, 1)
    b.dspark_embed(table, tokens, 0.5, out, ws)
    st, detail = b.dspark_read_device_error(ws)
    assert st == 5 and detail in (0x70000002, 0x70000004)
    assert torch.all(out[0] == 1.5) and torch.all(out[1] == 1.0) and torch.all(out[2:] == 0)


def _tokens(kind, n, V, rng):
    if kind == "distinct":
        return rng.permutation(max(n, V))[:n].astype(np.int32) % V
    if kind == "same":
        return np.full(n, V // 2, dtype=np.int32)
    if kind == "none":
        return np.full(n, -1, dtype=np.int32)
    if kind == "zipf":
        t = np.minimum((V ** rng.random(n)).astype(np.int64) - 1, V - 1).astype(np.int32)
        t[rng.random(n) < 0.1] = -1
        return t
    if kind == "ends":
        return np.where(rng.random(n) < 0.5, 0, V - 1).astype(np.int32)
    return rng.integers(0, V, size=n).astype(np.int32)


def _reference(dout, tokens, scale, before, V):
    """Sums and sums of magnitudes in fp64 (np.add.at in the items' order)."""
    g = np.zeros((V, dout.shape[1])) if before is None else before.copy()
    mag, count = np.zeros_like(g), np.zeros(V)
    ok = tokens >= 0
    np.add.at(g, tokens[ok], scale * dout[ok])
    np.add.at(mag, tokens[ok], np.abs(scale * dout[ok]))
    np.add.at(count, tokens[ok], 1)
    return g, mag, count


def _check_grad(kind, n, V, r, ti, to, accumulate, seed=0):
    b = _binding()
    rng = np.random.default_rng(seed + n + V + r)
    dout, held = _array((n, r), ti, rng)
    tokens = _tokens(kind, n, V, rng)
    dtable, before = _array((V, r), to, rng)
    scale = float(np.float32(0.3))
    ws = _ws(n, V, r)
    got = dtable.clone()
    t = torch.from_numpy(tokens).cuda()
    b.dspark_embed_grad(dout, t, scale, got, ws, accumulate=accumulate)
    assert b.dspark_read_device_error(ws)[0] == 0
    again = dtable.clone()
    b.dspark_embed_grad(dout, t, scale, again, ws, accumulate=accumulate)
    assert torch.equal(got, again)                     # the same bits each time
    want, mag, count = _reference(held, tokens, scale, before if accumulate else None, V)
    eps = torch.finfo(DT[to]).eps / 2
    tol = mag * (count[:, None] + 2) * U * 1.01 + (np.abs(want) + mag) * (U if accumulate else 0)
    tol = tol + (np.abs(want) + tol) * eps + 1e-45
    g = got.double().cpu().numpy()
    if accumulate:
        same = count == 0
        assert np.array_equal(g[same], before[same])   # rows without a token are left as they were
        tol[same] = 0
        g[same] = want[same]
    bad = np.abs(g - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], g[bad][:5], want[bad][:5], tol[bad][:5])


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("ti,to", TYPES)
@pytest.mark.parametrize("n,V,r", [(1, 1, 1), (2, 3, 5), (31, 7, 8), (100, 1000, 100), (512, 50257, 64), (513, 300, 256),
                                   (1500, 4000, 33), (2500, 40, 200), (9000, 20000, 48), (300, 500, 4096)])
def test_embed_grad_sizes(n, V, r, ti, to, accumulate):
    _check_grad("uniform", n, V, r, ti, to, accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["distinct", "same", "none", "zipf", "ends"])
@pytest.mark.parametrize("n,V,r", [(40, 64, 16), (700, 5000, 264), (3000, 70000, 40), (20011, 3001, 72)])
def test_embed_grad_distributions(kind, n, V, r, accumulate):
    _check_grad(kind, n, V, r, "bf16", "f32", accumulate)
    _check_grad(kind, n, V, r, "f32", "bf16", accumulate, seed=1)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["same", "zipf"])
@pytest.mark.parametrize("n,V,r", [(900, 50, 515), (1024, 3000, 500), (1025, 200, 500), (512, 40, 2050), (256, 30, 2052)])
def test_embed_grad_slabs(kind, n, V, r, accumulate):
    """Rows that several CTAs share, the last with a part of its slabs."""
    _check_grad(kind, n, V, r, "f32", "f32", accumulate)
    _check_grad(kind, n, V, r, "bf16", "bf16", accumulate, seed=1)


@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_large(accumulate):
    _check_grad("zipf", 100003, 30011, 24, "f32", "f32", accumulate)
    _check_grad("zipf", 66000, 129280, 64, "bf16", "f32", accumulate)
    _check_grad("uniform", 5000, 1500007, 8, "bf16", "f32", accumulate)


def test_embed_grad_far_rows():
    """Table rows past 2^31 elements (9.7 GB of fp32; the rows looked at only)."""
    b = _binding()
    V, r, n = 300000, 8192, 6
    dtable = torch.empty(V, r, device="cuda")
    tokens = torch.tensor([V - 1, 0, V - 1, 262145, -1, V - 2], dtype=torch.int32, device="cuda")
    dout = torch.arange(1, n + 1, device="cuda", dtype=torch.float32)[:, None].expand(n, r).contiguous()
    ws = _ws(n, V, r)
    b.dspark_embed_grad(dout, tokens, 1.0, dtable, ws)
    assert torch.all(dtable[V - 1] == 4) and torch.all(dtable[0] == 2) and torch.all(dtable[262145] == 4)
    assert torch.all(dtable[V - 2] == 6) and torch.all(dtable[V - 3] == 0) and torch.all(dtable[1] == 0)
    b.dspark_embed_grad(dout, tokens, 1.0, dtable, ws, accumulate=True)
    assert torch.all(dtable[V - 1] == 8) and torch.all(dtable[262145] == 8) and torch.all(dtable[V - 3] == 0)


def test_embed_grad_no_items_and_bad_tokens():
    b = _binding()
    dtable = torch.full((50, 12), 7.0, device="cuda")
    none = torch.empty(0, 12, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    b.dspark_embed_grad(*none, 1.0, dtable, _ws(0, 50, 12), accumulate=True)
    assert torch.all(dtable == 7)
    b.dspark_embed_grad(*none, 1.0, dtable, _ws(0, 50, 12))
    assert torch.all(dtable == 0)
    for n in (4, 3000):
        tokens = torch.full((n,), 3, dtype=torch.int32, device="cuda")
        tokens[1], tokens[2] = 50, -2
        ws = _ws(n, 50, 12)
        b.dspark_embed_grad(torch.ones(n, 12, device="cuda"), tokens, 1.0, dtable, ws)
        st, detail = b.dspark_read_device_error(ws)
        assert st == 5 and detail in (0x70000001, 0x70000002)
        assert torch.all(dtable[3] == n - 2) and float(dtable.sum()) == 12 * (n - 2)


@pytest.mark.parametrize("n", [300, 6000])
def test_embed_grad_captured_and_on_a_side_stream(n):
    """Two graphs that share a workspace, replayed in turn with changed tokens, and a side stream."""
    b = _binding()
    V, r = 4001, 72
    rng = np.random.default_rng(n)
    dout, _ = _array((n, r), "bf16", rng)
    tokens = torch.zeros(n, dtype=torch.int32, device="cuda")
    ws = _ws(n, V, r)
    a, c = torch.zeros(V, r, device="cuda"), torch.zeros(V, r, device="cuda")
    b.dspark_embed_grad(dout, tokens, 1.0, a, ws)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        b.dspark_embed_grad(dout, tokens, 1.0, a, ws)
    with torch.cuda.graph(g2):
        b.dspark_embed_grad(dout, tokens, 0.5, c, ws, accumulate=True)
    total = torch.zeros(V, r, device="cuda")
    c.zero_()
    for seed in range(3):
        tokens.copy_(torch.from_numpy(_tokens("zipf", n, V, np.random.default_rng(seed))))
        g1.replay()
        g2.replay()
        want = torch.empty(V, r, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        b.dspark_embed_grad(dout, tokens, 1.0, want, ws, stream=s)
        b.dspark_embed_grad(dout, tokens, 0.5, total, ws, accumulate=True, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(a, want) and torch.equal(c, total)
    assert b.dspark_read_device_error(ws)[0] == 0


@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_of_the_most_items(accumulate):
    """2^24 items of three tokens and some left out, where an item's place and its token's row fill the sort's words;
    sums of whole numbers below 2^24 are exact in any order."""
    b = _binding()
    n, V = 1 << 24, 4
    i = torch.arange(n, dtype=torch.int32, device="cuda")
    tokens = (i % 3).int()
    tokens[::1001] = -1
    dout = (1 + (i & 1)).float()[:, None]
    dtable = torch.full((V, 1), 5.0, device="cuda")
    ws = _ws(n, V, 1)
    b.dspark_embed_grad(dout, tokens, 1.0, dtable, ws, accumulate=accumulate)
    assert b.dspark_read_device_error(ws)[0] == 0
    want = torch.zeros(V + 1, 1, dtype=torch.float64, device="cuda").index_add_(0, tokens.long() + 1, dout.double())[1:]
    assert float(want.max()) < 1 << 24
    assert torch.equal(dtable.double(), want + (5.0 if accumulate else 0.0))
