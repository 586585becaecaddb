"""A round's scores and the head's gradient step, as a user runs them: draft,
schedule, verify, then the scores of the emitted tokens and the gradients of
the Markov factors, against the fp64 oracle.

Tolerances: scores as derived for dspark_logprobs (3 E1 + 68 half steps of
fp32 and the value's own rounding). The gradients are fp32 products of at most
V = 8192 terms: any order is off by at most V half steps of the sum of
magnitudes, and what enters them (dz, with its statistics) by 400 more.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import scores as oracle_scores

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _round(seed=21, B=8, K=4, V=8192, r=64, variant="a"):
    from speculative_decoding_semi_b200 import round as rnd
    w = synth.custom(1, B=B, K=K, V=V, r=r, n_prof=128)
    inp = synth.make_round(w, seed=seed)
    d = rnd.to_device(inp)
    return inp, d, rnd.RoundBuffers(B, K, V, r, variant=variant)


@pytest.mark.parametrize("variant", ["a", "b"])
@pytest.mark.parametrize("packed", [False, True])
def test_round_with_scores(variant, packed):
    from speculative_decoding_semi_b200 import dspark_read_device_error, round as rnd
    inp, d, bufs = _round(variant=variant)
    B, K, k = bufs.B, bufs.K, 7
    scores = rnd.TokenScores(B, K, top_k=k)
    if packed:
        rnd.draft(d, bufs)
        rnd.schedule(d, bufs)
        dense = d["target"].view(B, K + 1, -1)
        L = bufs.verify_len.tolist()
        target = torch.cat([dense[b, :L[b] + 1] for b in range(B)]).contiguous()
        rnd.verify(d, bufs, target=target, row_start=bufs.row_start)
        rnd.score(d, bufs, scores, target=target, row_start=bufs.row_start)
    else:
        rnd.run_round(d, bufs, scores=scores)
    assert dspark_read_device_error(bufs.workspace)[0] == 0
    tokens, n_out = bufs.out_tokens.cpu().numpy(), bufs.n_out.cpu().numpy()
    lp, H = scores.logprob.cpu().numpy(), scores.entropy.cpu().numpy()
    top, tlp = scores.top_tokens.cpu().numpy(), scores.top_logprobs.cpu().numpy()
    target = inp["target"].reshape(B, K + 1, -1)
    for b in range(B):
        for c in range(K + 1):
            if c >= n_out[b]:
                assert lp[b, c] == 0 and H[b, c] == 0 and np.all(top[b, c] == -1)
                continue
            ref = oracle_scores.row_scores(target[b, c], tokens[b, c], k)
            rel = (3 * ref["mean1"] + 68) * U
            assert abs(lp[b, c] - ref["logprob"]) <= rel + U * abs(ref["logprob"])
            tol = rel * (1 + ref["mean1"]) + (3 * ref["mean2"] + 72 * ref["mean1"]) * U + U * abs(ref["entropy"])
            assert abs(H[b, c] - ref["entropy"]) <= tol
            assert np.array_equal(top[b, c], ref["top_tokens"])
            assert np.all(np.abs(tlp[b, c] - ref["top_logprobs"]) <= rel + U * np.abs(ref["top_logprobs"]))


def test_round_with_scores_is_the_same_round():
    from speculative_decoding_semi_b200 import round as rnd
    _, d, one = _round()
    _, _, two = _round()
    rnd.run_round(d, one)
    rnd.run_round(d, two, scores=rnd.TokenScores(two.B, two.K, top_k=3))
    for name in ("draft_tokens", "q_tok", "lse_q", "z", "verify_len", "accepted", "out_tokens", "n_out"):
        assert torch.equal(getattr(one, name), getattr(two, name)), name


def _factors(inp):
    return tuple(torch.from_numpy(inp[n].view(np.int16)).view(torch.bfloat16).double() for n in ("A", "Bf"))


def _reference(inp, bufs, entropy_bonus):
    """Loss and gradients in fp64 from the definition, with the sums of magnitudes."""
    K = bufs.K
    A, Bf = _factors(inp)
    out, drafts = bufs.out_tokens.cpu().numpy(), bufs.draft_tokens.cpu().numpy()
    z = bufs.z.cpu().numpy().astype(np.float64)
    n = int((out[:, :K] >= 0).sum())
    loss, dA, dBf, mA, mB = 0.0, torch.zeros_like(A), torch.zeros_like(Bf), torch.zeros_like(A), torch.zeros_like(Bf)
    for b, i in np.argwhere(out[:, :K] >= 0):
        prev = int(inp["anchor"][b] if i == 0 else drafts[b, i - 1])
        r = oracle_scores.row_scores(z[b, i], out[b, i])
        loss -= (r["logprob"] + entropy_bonus * r["entropy"]) / n
        dz = torch.from_numpy(oracle_scores.row_scores_grad(z[b, i], out[b, i], -1.0 / n, -entropy_bonus / n))
        outer = A[prev][:, None] * dz[None, :]
        dA[prev] += Bf @ dz
        mA[prev] += Bf.abs() @ dz.abs()
        dBf += outer
        mB += outer.abs()
    return loss, dA, dBf, mA, mB


@pytest.mark.parametrize("entropy_bonus", [0.0, 0.1])
def test_head_gradients(entropy_bonus):
    from speculative_decoding_semi_b200 import dspark_read_device_error, head, round as rnd
    inp, d, bufs = _round()
    rnd.run_round(d, bufs)
    grads = head.HeadGradients(bufs.B, bufs.K, bufs.V, bufs.r)
    loss = head.head_gradients(d, bufs, grads, entropy_bonus=entropy_bonus)
    assert dspark_read_device_error(grads.workspace)[0] == 0
    want, dA, dBf, mA, mB = _reference(inp, bufs, entropy_bonus)
    assert abs(float(loss) - want) <= 400 * U * (1 + abs(want))
    tol = (bufs.V + 400) * U
    for got, ref, mag in ((grads.dA, dA, mA), (grads.dBf, dBf, mB)):
        err = (got.double().cpu() - ref).abs()
        assert bool((err <= tol * mag + 1e-30).all()), float((err / (mag + 1e-30)).max())
    once = grads.dA.clone(), grads.dBf.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    head.head_gradients(d, bufs, grads, entropy_bonus=entropy_bonus, accumulate=True, stream=s)
    torch.cuda.synchronize()
    for got, first, mag in ((grads.dA, once[0], mA), (grads.dBf, once[1], mB)):
        assert bool(((got - 2 * first).double().cpu().abs() <= 2 * tol * mag + 1e-30).all())


def test_head_gradient_matches_differences_of_the_loss():
    """Along the gradient's own direction D (|D| = 1): (L(A + hD) - L(A - hD)) / 2h = |dL/dA|, the loss in fp64 from
    the definition, so that only the truncation h^2/6 |L'''| (|L'''| < 1, h = 1e-3) and the gradient's own error
    remain."""
    from speculative_decoding_semi_b200 import head, round as rnd
    inp, d, bufs = _round()
    rnd.run_round(d, bufs)
    grads = head.HeadGradients(bufs.B, bufs.K, bufs.V, bufs.r)
    head.head_gradients(d, bufs, grads)
    g = grads.dA.double().cpu()
    norm = float(g.norm())
    A, Bf = _factors(inp)
    out, drafts = bufs.out_tokens.cpu(), bufs.draft_tokens.cpu()
    used = out[:, :bufs.K] >= 0
    prev = torch.cat([torch.from_numpy(inp["anchor"])[:, None], drafts[:, :-1]], 1)[used].long()
    base = torch.from_numpy(inp["base"]).double()[used]
    label = out[:, :bufs.K][used].long()

    def loss(A):
        return -torch.log_softmax(base + A[prev] @ Bf, 1).gather(1, label[:, None]).mean()

    h = 1e-3
    slope = float(loss(A + h * g / norm) - loss(A - h * g / norm)) / (2 * h)
    assert abs(slope - norm) <= 1e-6 + (bufs.V + 400) * U * norm


def test_head_gradients_refuses():
    from speculative_decoding_semi_b200 import head
    _, d, bufs = _round(variant="b")
    grads = head.HeadGradients(bufs.B, bufs.K, bufs.V, bufs.r)
    with pytest.raises(ValueError, match="variant"):
        head.head_gradients(d, bufs, grads)
    _, d, bufs = _round()
    with pytest.raises(ValueError, match="RNN"):
        head.head_gradients(dict(d, W=d["A"]), bufs, grads)
    with pytest.raises(ValueError, match="round of"):
        head.head_gradients(d, bufs, head.HeadGradients(bufs.B, bufs.K + 1, bufs.V, bufs.r))


def test_round_scores_and_gradients_in_one_graph():
    """The whole step captured once and replayed on other inputs."""
    from speculative_decoding_semi_b200 import head, round as rnd
    _, d, bufs = _round(seed=31)
    scores, grads = rnd.TokenScores(bufs.B, bufs.K, top_k=4), head.HeadGradients(bufs.B, bufs.K, bufs.V, bufs.r)

    def step():
        rnd.run_round(d, bufs, scores=scores)
        return head.head_gradients(d, bufs, grads)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = step()
    _, other, _ = _round(seed=32)
    for name, t in d.items():
        t.copy_(other[name])
    g.replay()
    torch.cuda.synchronize()
    got = float(loss), scores.logprob.clone(), scores.top_tokens.clone(), grads.dA.clone()
    want = float(step())
    assert abs(got[0] - want) <= 8 * U * abs(want)      # the same terms, summed by torch
    assert torch.equal(got[1], scores.logprob) and torch.equal(got[2], scores.top_tokens)
    # drows is a library product, whose order may differ between capture and eager: V half steps of its magnitudes
    assert float((got[3] - grads.dA).abs().max()) <= bufs.V * U * float(grads.dA.abs().max() + 1)


@pytest.mark.parametrize("legacy", [False, True])
def test_head_gradients_on_a_stream_handle(legacy):
    """`stream` as the integer handle that the entry points take; 0 is the legacy default stream."""
    from speculative_decoding_semi_b200 import head, round as rnd
    inp, d, bufs = _round()
    rnd.run_round(d, bufs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    grads = head.HeadGradients(bufs.B, bufs.K, bufs.V, bufs.r)
    torch.cuda.synchronize()
    before = torch.cuda.current_stream()
    loss = head.head_gradients(d, bufs, grads, stream=0 if legacy else s.cuda_stream)
    (torch.cuda.default_stream() if legacy else s).synchronize()
    assert torch.cuda.current_stream() == before
    want, dA, dBf, mA, mB = _reference(inp, bufs, 0.0)
    assert abs(float(loss) - want) <= 400 * U * (1 + abs(want))
    for got, ref, mag in ((grads.dA, dA, mA), (grads.dBf, dBf, mB)):
        assert bool(((got.double().cpu() - ref).abs() <= (bufs.V + 400) * U * mag + 1e-30).all())


def test_replayed_scores_and_gradients_match_the_definition():
    """The captured step on other inputs: its gradients by the bounds of an eager step (sums of magnitudes of each
    entry), its scores bit by bit."""
    from speculative_decoding_semi_b200 import head, round as rnd
    _, d, bufs = _round(seed=41)
    scores, grads = rnd.TokenScores(bufs.B, bufs.K, top_k=4), head.HeadGradients(bufs.B, bufs.K, bufs.V, bufs.r)

    def step():
        rnd.run_round(d, bufs, scores=scores)
        return head.head_gradients(d, bufs, grads, entropy_bonus=0.1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = step()
    inp, other, _ = _round(seed=42)
    for name, t in d.items():
        t.copy_(other[name])
    g.replay()
    torch.cuda.synchronize()
    want, dA, dBf, mA, mB = _reference(inp, bufs, 0.1)
    assert abs(float(loss) - want) <= 400 * U * (1 + abs(want))
    for got, ref, mag in ((grads.dA, dA, mA), (grads.dBf, dBf, mB)):
        assert bool(((got.double().cpu() - ref).abs() <= (bufs.V + 400) * U * mag + 1e-30).all())
    replayed = {n: getattr(scores, n).clone() for n in ("logprob", "entropy", "stats", "top_tokens", "top_logprobs")}
    step()
    torch.cuda.synchronize()
    for n, t in replayed.items():
        assert torch.equal(t, getattr(scores, n)), n
