"""dspark_logprobs and dspark_logprobs_grad against the fp64 oracle.

Tolerances, in half steps of fp32 (u = 2^-24), derived from the definition:
y = (x - m) log2 e carries 3 roundings (the difference, the constant, the
product), so e^(x-m) is off by 3 u |x-m| plus 4 u for the exponential (PTX
ex2: 2^-22), and a sum of up to 64 fp32 terms by 63 u more. Weighted by p,
with E1 = E|x-m| and E2 = E|x-m|^2 under the row:
  s: relative 3 u E1 + 68 u;  ln s, logprob: that absolute, plus u |value|
  (the final rounding);
  T/S (entropy): (3 E2 + 72 E1) u, plus E1 times s's relative error.
"""
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


def _ws():
    b = _binding()
    ws = torch.empty(b.dspark_workspace_bytes(1, 1, 8, 1), dtype=torch.uint8, device="cuda")
    b.dspark_workspace_init(ws)
    return ws


def _rows(kind, n, V, rng):
    x = rng.normal(0, 2.5, size=(n, V)).astype(np.float32)
    if kind == "masked":            # one row with nothing left, one with one token, one with few, one lowest value
        x[rng.random((n, V)) < 0.5] = -np.inf
        x[0] = -np.inf
        if n > 1:
            x[1] = -np.inf
            x[1, V // 2] = 3.0
        if n > 2:
            x[2] = np.finfo(np.float32).min
        if n > 3:
            x[3, : V // 2] = np.finfo(np.float32).min
            x[3, V // 2:] = 0.25
    elif kind == "ties":            # few distinct values; -0 and 0; a constant row
        x = np.round(x).astype(np.float32)
        x[x == 0] = np.where(rng.random((x == 0).sum()) < 0.5, -0.0, 0.0)
        x[0] = 1.5
        if n > 1:
            x[1] = np.where(rng.random(V) < 0.5, -0.0, 0.0)
    elif kind == "sorted":          # the largest all in one place, at either end
        x = -np.sort(-x, axis=1)
        x[1::2] = x[1::2, ::-1]
    elif kind == "far":             # large offsets and a wide spread
        x = (x * 30 + rng.choice([-1e4, 0, 1e4], size=(n, 1))).astype(np.float32)
    elif kind == "peaked":
        x[np.arange(n), rng.integers(0, V, size=n)] = 60.0
    return x


def _device_rows(x, dtype, pad):
    """The rows with `pad` NaN columns behind each (never to be read), and what is held."""
    n, V = x.shape
    t = torch.full((n, V + pad), float("nan"), dtype=DT[dtype], device="cuda")
    t[:, :V] = torch.from_numpy(x).cuda().to(DT[dtype])
    return t[:, :V], t[:, :V].double().cpu().numpy()


def _run(logits, tokens, k, ws=None, row_start=None, stream=None, outs=None):
    b = _binding()
    B, C = tokens.shape
    if outs is None:
        outs = dict(lp=torch.full((B, C), 7.0, device="cuda"), H=torch.full((B, C), 7.0, device="cuda"),
                    st=torch.full((B, C, 2), 7.0, device="cuda"),
                    top=torch.full((B, C, k), 7, dtype=torch.int32, device="cuda") if k else None,
                    tlp=torch.full((B, C, k), 7.0, device="cuda") if k else None)
    ws = _ws() if ws is None else ws
    b.dspark_logprobs(logits, tokens, outs["lp"], outs["H"], outs["st"], outs["top"], outs["tlp"], ws,
                      row_start=row_start, stream=stream)
    return outs, ws


def _close(got, want, tol):
    if np.isnan(want) or np.isinf(want):
        return got == want or (np.isnan(got) and np.isnan(want))
    return abs(got - want) <= tol


def _check_item(o, at, ref, k):
    lp, H, st = float(o["lp"][at]), float(o["H"][at]), o["st"][at]
    rel = (3 * ref["mean1"] + 68) * U
    assert _close(lp, ref["logprob"], rel + U * abs(ref["logprob"]) + 1e-45), (at, lp, ref["logprob"])
    tol = rel + (3 * ref["mean2"] + 72 * ref["mean1"]) * U + ref["mean1"] * rel + U * abs(ref["entropy"])
    assert _close(H, ref["entropy"], tol), (at, H, ref["entropy"])
    assert _close(float(st[0]), ref["m"], 0.0), (at, st)
    assert _close(float(st[1]), ref["s"], (rel + U) * abs(ref["s"])), (at, st, ref["s"])
    if k:
        assert np.array_equal(o["top"][at], ref["top_tokens"]), (at, o["top"][at], ref["top_tokens"])
        for g, w in zip(o["tlp"][at], ref["top_logprobs"]):
            assert _close(float(g), w, rel + U * abs(w)), (at, g, w)


def _host(outs):
    return {n: (None if v is None else v.cpu().numpy()) for n, v in outs.items()}


def _check(logits, held, tokens, k, row_start=None, ws=None):
    outs, ws = _run(logits, torch.from_numpy(tokens).cuda(), k, ws,
                    None if row_start is None else torch.from_numpy(row_start).cuda())
    assert _binding().dspark_read_device_error(ws)[0] == 0
    o = _host(outs)
    B, C = tokens.shape
    for b in range(B):
        for c in range(C):
            row = (row_start[b] if row_start is not None else b * C) + c
            if tokens[b, c] < 0:
                assert o["lp"][b, c] == 0 and o["H"][b, c] == 0 and np.all(o["st"][b, c] == 0)
                if k:
                    assert np.all(o["top"][b, c] == -1) and np.all(o["tlp"][b, c] == -np.inf)
            else:
                _check_item(o, (b, c), scores.row_scores(held[row], tokens[b, c], k), k)


SIZES = [(1, 1), (3, 2), (5, 7), (4, 8), (4, 31), (4, 33), (3, 127), (3, 1000), (5, 1024), (4, 1025), (4, 4099),
         (3, 8192), (4, 20011), (40, 2049), (7, 50257), (2, 151936)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", SIZES)
def test_logprobs_sizes(n, V, dtype):
    rng = np.random.default_rng(n * 1000 + V)
    for pad, k in ((0, 5), (1, 32), (5, 0), (64, 1)):
        x, held = _device_rows(_rows("plain", n, V, rng), dtype, pad)
        tokens = rng.integers(0, V, size=(n, 1)).astype(np.int32)
        tokens[0, 0] = V - 1
        tokens[-1, 0] = 0
        _check(x, held, tokens, k)


@pytest.mark.parametrize("kind", ["masked", "ties", "sorted", "far", "peaked"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 700, 5003, 60000])
def test_logprobs_values(kind, dtype, V):
    rng = np.random.default_rng(V)
    x, held = _device_rows(_rows(kind, 6, V, rng), dtype, 3)
    for k in (1, 20, 32):
        _check(x, held, rng.integers(0, V, size=(6, 1)).astype(np.int32), k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 3001, 40000])
def test_logprobs_nan_and_inf(dtype, V):
    rng = np.random.default_rng(V)
    x = _rows("plain", 5, V, rng)
    x[0, V // 3] = np.nan
    x[1, V - 1] = np.inf
    x[2, 0] = np.nan
    x[2, 1:] = -np.inf
    x[3] = np.nan
    x, held = _device_rows(x, dtype, 0)
    _check(x, held, rng.integers(0, V, size=(5, 1)).astype(np.int32), 4)


def test_logprobs_packed_rows():
    """Rows as the scheduler packs them: items behind the emitted tokens are left out and their rows (behind the last
    one, or another request's) not read; two requests may point at the same row."""
    rng = np.random.default_rng(1)
    B, C, V = 9, 4, 5000
    n_out = rng.integers(1, C + 1, size=B)
    start = (np.cumsum(n_out) - n_out).astype(np.int64)
    start[4] = start[2]
    x, held = _device_rows(_rows("plain", int(n_out.sum()), V, rng), "f32", 0)
    tokens = rng.integers(0, V, size=(B, C)).astype(np.int32)
    n_out[4] = min(n_out[4], n_out[2])
    tokens[np.arange(C) >= n_out[:, None]] = -1
    _check(x, held, tokens, 3, row_start=start)


def test_logprobs_errors_are_recorded():
    b = _binding()
    x = torch.randn(4, 100, device="cuda")
    for tokens, start, item in (([[0], [100], [5], [5]], None, 1), ([[0], [1], [-2], [5]], None, 2),
                                ([[0], [1], [2], [5]], [0, 1, 2, 4], 3), ([[0], [1], [2], [5]], [-1, 1, 2, 3], 0)):
        t = torch.tensor(tokens, dtype=torch.int32, device="cuda")
        rs = None if start is None else torch.tensor(start, dtype=torch.int64, device="cuda")
        outs, ws = _run(x, t, 2, row_start=rs)
        assert b.dspark_read_device_error(ws) == (5, 0x70000000 | item)
        o = _host(outs)
        assert o["lp"][item, 0] == 0 and np.all(o["top"][item] == -1)       # as an item left out
        good = (item + 1) % 4
        assert o["lp"][good, 0] < 0


def test_logprobs_optional_outputs():
    b = _binding()
    x = torch.randn(6, 3000, device="cuda")
    t = torch.randint(0, 3000, (6, 1), dtype=torch.int32, device="cuda")
    full, ws = _run(x, t, 3)
    lp = torch.empty(6, 1, device="cuda")
    b.dspark_logprobs(x, t, lp, None, None, None, None, ws)
    assert torch.equal(lp, full["lp"])
    outs = {"lp": torch.empty(0, 3, device="cuda"), "H": None, "st": None, "top": None, "tlp": None}
    _run(x, torch.empty(0, 3, dtype=torch.int32, device="cuda"), 0, outs=outs)     # no items: no launch


def test_logprobs_many_short_rows():
    rng = np.random.default_rng(5)
    x, held = _device_rows(_rows("plain", 3000, 61, rng), "bf16", 3)
    _check(x, held, rng.integers(-1, 61, size=(1000, 3)).astype(np.int32), 2)


def test_logprobs_long_row():
    rng = np.random.default_rng(6)
    V = (1 << 21) + 3
    for dtype in ("f32", "bf16"):
        x, held = _device_rows(_rows("plain", 2, V, rng), dtype, 0)
        _check(x, held, np.array([[5], [V - 1]], dtype=np.int32), 32)


def test_logprobs_many_long_rows():
    """More rows than the GPU runs at once, each long."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1300, 70001, device="cuda", generator=gen)
    t = torch.randint(0, 70001, (1300, 1), dtype=torch.int32, device="cuda", generator=gen)
    outs, ws = _run(x, t, 4)
    o = _host(outs)
    for i in (0, 1, 147, 148, 296, 700, 1298, 1299):
        _check_item(o, (i, 0), scores.row_scores(x[i].cpu().numpy(), int(t[i, 0]), 4), 4)
    want = torch.log_softmax(x.double(), 1).gather(1, t.long())
    assert float((outs["lp"].double() - want).abs().max()) < 200 * U     # E1 < 12 here: 3 E1 + 68 + |value|


def test_logprobs_offsets_past_32_bits():
    """Rows whose offset in elements does not fit in 32 bits (6.1 GB of bf16 logits, of which two rows are written)."""
    V, n = 151936, 20000
    x = torch.empty(n, V, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(7)
    rows = _rows("plain", 2, V, rng)
    x[n - 2:] = torch.from_numpy(rows).cuda().bfloat16()
    held = x[n - 2:].double().cpu().numpy()
    tokens = torch.tensor([[11, V - 2]], dtype=torch.int32, device="cuda")
    outs, ws = _run(x, tokens, 3, row_start=torch.tensor([n - 2], device="cuda"))
    o = _host(outs)
    for c in range(2):
        _check_item(o, (0, c), scores.row_scores(held[c], int(tokens[0, c]), 3), 3)


def test_logprobs_same_bits_each_time_and_on_a_side_stream():
    rng = np.random.default_rng(8)
    x, _ = _device_rows(_rows("ties", 17, 30011, rng), "f32", 1)
    t = torch.randint(0, 30011, (17, 1), dtype=torch.int32, device="cuda")
    a, ws = _run(x, t, 32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c, _ = _run(x, t, 32, ws)
    d, _ = _run(x, t, 32, ws, stream=s)
    torch.cuda.synchronize()
    for name in a:
        assert torch.equal(a[name], c[name]) and torch.equal(a[name], d[name])


def test_logprobs_and_gradient_captured():
    """Two graphs on one workspace, replayed in turn on changed inputs."""
    b = _binding()
    V, n, k = 20001, 6, 5
    x, t = torch.randn(n, V, device="cuda"), torch.randint(0, V, (n, 1), dtype=torch.int32, device="cuda")
    g = torch.randn(n, device="cuda")
    d = torch.empty_like(x)
    outs, ws = _run(x, t, k)
    b.dspark_logprobs_grad(x, t, outs["st"], outs["H"], g, g, d, ws)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        _run(x, t, k, ws, outs=outs)
    with torch.cuda.graph(g2):
        b.dspark_logprobs_grad(x, t, outs["st"], outs["H"], g, g, d, ws)
    for seed in range(3):
        x.copy_(torch.from_numpy(_rows("plain", n, V, np.random.default_rng(seed))))
        t.copy_(torch.from_numpy(np.random.default_rng(seed).integers(0, V, size=(n, 1)).astype(np.int32)))
        g1.replay()
        g2.replay()
        fresh, _ = _run(x, t, k)
        d2 = torch.empty_like(x)
        b.dspark_logprobs_grad(x, t, fresh["st"], fresh["H"], g, g, d2, ws)
        for name in outs:
            assert torch.equal(outs[name], fresh[name])
        assert torch.equal(d, d2)


# ------------------------------------------------------------------ gradient

def _grad_tolerance(x, token, gl, gh, eps):
    """p = 2^y / s is off by 3 |x-m| + 4 (ex2) + 3 (s, its reciprocal, the product) half steps and ln p by
    3 |x-m| + |ln s| + |ln p| half steps; the bracket c0 + c1 y adds its own three roundings; the result one of
    its type. `3 |x-m| + 12` covers the relative part of both. An exponential below the least normal number,
    2^-126, is held as 0, which leaves out at most 2^-126 times the bracket (40 and more where |x-m| is 87)."""
    r = scores.row_scores(x, token)
    d = np.where(x > -np.inf, np.abs(x - r["m"]), 0.0)
    p = np.exp(-d) / r["s"]
    size = np.abs(gl) + np.abs(gh) * (d + abs(np.log(r["s"])) + abs(r["entropy"]))
    H_err = (3 * r["mean2"] + 75 * r["mean1"] + 70) * U * (1 + r["mean1"])      # the forward entropy's own error
    tol = p * (size * (6 * d + 16 + 70) * U + np.abs(gh) * H_err)               # 70: s from the forward call
    want = scores.row_scores_grad(x, token, gl, gh)
    return tol + (np.abs(want) + tol) * eps + 2.0 ** -126 * (1 + size), want


def _check_grad(kind, n, V, dtype, pad, gpad, entropy, rng, in_place=False):
    b = _binding()
    x, held = _device_rows(_rows(kind, n, V, rng), dtype, pad)
    tokens = rng.integers(0, V, size=n).astype(np.int32)
    tokens[n // 2] = -1
    t = torch.from_numpy(tokens).cuda()
    outs, ws = _run(x, t.clamp(min=0)[:, None].contiguous(), 0)
    gl = rng.normal(size=n).astype(np.float32)
    gh = rng.normal(size=n).astype(np.float32) if entropy else np.zeros(n, dtype=np.float32)
    buf = torch.full((n, V + gpad), 7.0, dtype=DT[dtype], device="cuda")
    d = x if in_place else buf[:, :V]
    b.dspark_logprobs_grad(x, t, outs["st"], outs["H"] if entropy else None, torch.from_numpy(gl).cuda(),
                           torch.from_numpy(gh).cuda() if entropy else None, d, ws)
    assert b.dspark_read_device_error(ws)[0] == 0
    if not in_place:
        assert torch.all(buf[:, V:] == 7.0)
    got = d.double().cpu().numpy()
    eps = torch.finfo(DT[dtype]).eps / 2
    for i in range(n):
        if tokens[i] < 0 or np.all(held[i] == -np.inf):
            assert np.all(got[i] == 0)
            continue
        tol, want = _grad_tolerance(held[i], tokens[i], float(gl[i]), float(gh[i]), eps)
        bad = np.abs(got[i] - want) > tol
        assert not bad.any(), (i, np.flatnonzero(bad)[:5], got[i][bad][:5], want[bad][:5], tol[bad][:5])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", SIZES)
def test_grad_sizes(n, V, dtype):
    rng = np.random.default_rng(n * 77 + V)
    for pad, gpad, entropy in ((0, 0, True), (1, 1, False), (3, 8, True), (8, 3, False)):
        _check_grad("plain", n, V, dtype, pad, gpad, entropy, rng)


@pytest.mark.parametrize("kind", ["masked", "far", "peaked"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("entropy", [False, True])
def test_grad_values(kind, dtype, entropy):
    rng = np.random.default_rng(9)
    for V in (11, 5003):
        _check_grad(kind, 6, V, dtype, 2, 2, entropy, rng)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grad_in_place(dtype):
    _check_grad("plain", 5, 10007, dtype, 1, 0, True, np.random.default_rng(2), in_place=True)


def test_grad_nan_rows_and_errors():
    b = _binding()
    x = torch.randn(4, 500, device="cuda")
    x[1, 3] = float("nan")
    x[2, 3] = float("inf")
    t = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
    outs, ws = _run(x, t[:, None].contiguous(), 0)
    g, d = torch.ones(4, device="cuda"), torch.empty_like(x)
    b.dspark_logprobs_grad(x, t, outs["st"], outs["H"], g, g, d, ws)
    assert torch.isnan(d[1:3]).all() and torch.isfinite(d[[0, 3]]).all()
    t[0], t[3] = -5, 500
    b.dspark_logprobs_grad(x, t, outs["st"], outs["H"], g, g, d, ws)
    st, detail = b.dspark_read_device_error(ws)
    assert st == 5 and detail in (0x70000000, 0x70000003)
    assert torch.all(d[0] == 0) and torch.all(d[3] == 0)


def test_grad_sums_to_nothing_and_matches_differences():
    """The gradient of a log probability sums to 0 over the row, and agrees with differences of the entry point's own
    values: a step of 2^-6 in one logit; truncation h^2/6 |f'''| <= 4.1e-5 |f'''|, |f'''| <= 1, and 2 * 150 u / 2h."""
    b = _binding()
    V = 97
    x = torch.randn(1, V, device="cuda")
    t = torch.tensor([[5]], dtype=torch.int32, device="cuda")
    outs, ws = _run(x, t, 0)
    one, d = torch.ones(1, device="cuda"), torch.empty_like(x)
    b.dspark_logprobs_grad(x, t, outs["st"], None, one, None, d, ws)
    assert abs(float(d.double().sum())) < V * 150 * U
    h = 2.0 ** -6
    for v in (0, 5, 50, 96):
        f = []
        for step in (h, -h):
            y = x.clone()
            y[0, v] += step
            f.append(float(_run(y, t, 0)[0]["lp"].double()[0, 0]))
        assert abs((f[0] - f[1]) / (2 * h) - float(d[0, v])) < 4.1e-5 + 300 * U / (2 * h)


@pytest.mark.parametrize("B,C", [(100, 5), (23, 17), (640, 4)])
def test_logprobs_short_and_idle_requests(B, C):
    """Requests of every length, idle ones among them (all their items left out), and a batch of nothing else."""
    rng = np.random.default_rng(B)
    x, held = _device_rows(_rows("plain", B * C, 700, rng), "f32", 4)
    tokens = rng.integers(0, 700, size=(B, C)).astype(np.int32)
    n_out = rng.integers(0, C + 1, size=B)
    tokens[np.arange(C) >= n_out[:, None]] = -1
    _check(x, held, tokens, 3)
    _check(x, held, np.full_like(tokens, -1), 3)


def test_calls_on_two_streams_at_once():
    """Each stream with a workspace of its own; the same bits as one after the other."""
    b = _binding()
    V, r, n = 30000, 256, 6000
    xs = [torch.randn(40, V, device="cuda") for _ in range(2)]
    ts = [torch.randint(0, V, (40, 1), dtype=torch.int32, device="cuda") for _ in range(2)]
    dout = [torch.randn(n, r, device="cuda") for _ in range(2)]
    tok = [torch.randint(0, V // 50, (n,), dtype=torch.int32, device="cuda") for _ in range(2)]
    want = [_run(x, t, 20)[0] for x, t in zip(xs, ts)]
    size = b.dspark_embed_grad_workspace_bytes(n, V, r)
    ws = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    grads = [torch.zeros(V, r, device="cuda") for _ in range(2)]
    for k in range(2):
        b.dspark_embed_grad(dout[k], tok[k], 0.5, grads[k], ws[k])
    want_grads = [g.clone() for g in grads]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[k].append(_run(xs[k], ts[k], 20, ws=ws[k])[0])
                grads[k].fill_(7.0)
                b.dspark_embed_grad(dout[k], tok[k], 0.5, grads[k], ws[k])
    torch.cuda.synchronize()
    for k in range(2):
        for o in outs[k]:
            for name in o:
                assert torch.equal(o[name], want[k][name])
        assert torch.equal(grads[k], want_grads[k])
        assert b.dspark_read_device_error(ws[k])[0] == 0


def _short_requests(B, C, V, rng):
    """Tokens [B,C] of requests of every length, idle ones among them, and where their packed rows start."""
    n_out = rng.integers(0, C + 1, size=B)
    n_out[:3] = 0, C, 2
    tokens = rng.integers(0, V, size=(B, C)).astype(np.int32)
    tokens[np.arange(C) >= n_out[:, None]] = -1
    return tokens, (np.cumsum(n_out) - n_out).astype(np.int64), int(n_out.sum())


@pytest.mark.parametrize("dtype,B,C,V", [("f32", 20, 5, 40000), ("bf16", 20, 5, 40001), ("f32", 64, 9, 16397)])
@pytest.mark.parametrize("k", [0, 20])
def test_logprobs_short_requests_of_long_rows(dtype, B, C, V, k):
    """Requests of several lengths whose rows are long enough to be shared by the CTAs of a cluster."""
    rng = np.random.default_rng(B + V)
    tokens, start, rows = _short_requests(B, C, V, rng)
    x, held = _device_rows(_rows("plain", rows, V, rng), dtype, 1)
    _check(x, held, tokens, k, row_start=start)


@pytest.mark.parametrize("dtype,V", [("f32", 40000), ("bf16", 40001)])
def test_logprobs_errors_among_long_rows(dtype, V):
    """A bad token, and a request whose second row lies behind the last: recorded (one of the two), treated as left
    out, and the other items are scored as without them."""
    b = _binding()
    rng = np.random.default_rng(V)
    B, C, k = 20, 5, 20
    tokens, start, rows = _short_requests(B, C, V, rng)
    x, held = _device_rows(_rows("plain", rows, V, rng), dtype, 0)
    tokens[1, 3] = V
    start[2] = rows - 1
    outs, ws = _run(x, torch.from_numpy(tokens).cuda(), k, row_start=torch.from_numpy(start).cuda())
    code, detail = b.dspark_read_device_error(ws)
    assert code == 5 and detail in (0x70000000 | (C + 3), 0x70000000 | (2 * C + 1))
    o = _host(outs)
    for i in range(B):
        for c in range(C):
            if tokens[i, c] < 0 or (i, c) in ((1, 3), (2, 1)):
                assert o["lp"][i, c] == 0 and o["H"][i, c] == 0 and np.all(o["st"][i, c] == 0)
                assert np.all(o["top"][i, c] == -1) and np.all(o["tlp"][i, c] == -np.inf)
            else:
                _check_item(o, (i, c), scores.row_scores(held[start[i] + c], tokens[i, c], k), k)
