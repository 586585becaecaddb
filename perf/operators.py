"""Workloads of the token-scoring and embedding operators, for measuring them.

Four operators: log probabilities of given tokens with entropy and the top
alternatives (`logprobs`), their gradient with respect to the logits
(`logprobs_grad`), embedding lookup with scaling (`embed`) and its gradient by
sorted tokens (`embed_grad`). With `own` false, `run` computes them in
elementary torch operations; with `own` true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user's stream, 16 drafts a round: the emitted tokens of one round, with the alternatives an API reply shows
        dict(name="reply_one_request", op="logprobs", B=1, C=17, V=151936, pad=0, dtype="f32", top_k=20, packed=True),
        # a round of 64 requests with 8 drafts: target rows packed by the scheduler, five alternatives
        dict(name="reply_round", op="logprobs", B=64, C=9, V=151936, pad=0, dtype="f32", top_k=5, packed=True),
        # scoring given texts (evaluation, policy training): one row a token, bf16 logits, no alternatives
        dict(name="score_texts", op="logprobs", B=4096, C=1, V=129280, pad=0, dtype="bf16", top_k=0, packed=False),
        # an odd vocabulary, so that rows start at any alignment; alternatives from bf16 logits, where ties are common
        dict(name="score_odd_vocabulary", op="logprobs", B=333, C=2, V=50257, pad=0, dtype="bf16", top_k=32,
             packed=False),
        # a tiny head: a few short rows, where a call costs its latency
        dict(name="grad_tiny", op="logprobs_grad", N=16, V=1024, pad=0, dtype="f32", entropy=True),
        # the draft's logits of one round of 64 requests with 8 drafts, emitted tokens as labels, entropy regularised
        dict(name="grad_round", op="logprobs_grad", N=512, V=151936, pad=0, dtype="f32", entropy=True),
        # a training batch in bf16 with an odd vocabulary in padded rows
        dict(name="grad_texts", op="logprobs_grad", N=3000, V=50257, pad=47, dtype="bf16", entropy=False),
        # the operand rows of one position of 64 requests
        dict(name="embed_position", op="embed", n=64, V=151936, r=256, dtype="bf16", out="bf16"),
        # the input rows of a training batch, scaled
        dict(name="embed_batch", op="embed", n=16384, V=129280, r=4096, dtype="bf16", out="f32"),
        # one round's head gradient added to the gradient so far: few rows touched
        dict(name="embed_grad_round", op="embed_grad", n=512, V=151936, r=256, dtype="f32", grad="f32",
             accumulate=True),
        # an odd batch over an odd vocabulary, the gradient written whole
        dict(name="embed_grad_odd", op="embed_grad", n=10007, V=50257, r=200, dtype="bf16", grad="f32",
             accumulate=False),
        # a large training batch: many rows a token, the gradient written whole in bf16
        dict(name="embed_grad_batch", op="embed_grad", n=65536, V=129280, r=1024, dtype="bf16", grad="bf16",
             accumulate=False),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "embed", "embed_grad"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "logprobs":
        V = _log_uniform(rng, 500, 260000)
        C = rng.choice([1, 1, 2, 5, 9, 17])
        most = max(1, 500_000_000 // (V * C * SIZE[dtype]))
        B = _log_uniform(rng, 1, max(1, min(4096, most)))
        return dict(op=op, B=B, C=C, V=V, pad=rng.choice([0, 0, 1, 64]), dtype=dtype,
                    top_k=rng.choice([0, 1, 5, 20, 32]), packed=rng.random() < 0.5)
    if op == "logprobs_grad":
        V = _log_uniform(rng, 500, 260000)
        most = max(1, 250_000_000 // (V * SIZE[dtype]))
        return dict(op=op, N=_log_uniform(rng, 1, max(1, min(4096, most))), V=V, pad=rng.choice([0, 0, 1, 64]),
                    dtype=dtype, entropy=rng.random() < 0.5)
    V = _log_uniform(rng, 1000, 150000)
    r = _log_uniform(rng, 32, 4096) if rng.random() < 0.3 else rng.choice([64, 128, 200, 256, 512, 1024, 2048, 4096])
    n = _log_uniform(rng, 1, max(1, min(65536, 50_000_000 // r)))
    if op == "embed":
        return dict(op=op, n=n, V=min(V, 800_000_000 // (4 * r)), r=r, dtype=dtype, out=rng.choice(["f32", "bf16"]))
    return dict(op=op, n=n, V=min(V, 300_000_000 // (4 * r)), r=r, dtype=dtype, grad=rng.choice(["f32", "bf16"]),
                accumulate=rng.random() < 0.5)


def _emitted(B, C):
    """Emitted tokens of each request of a round: 1 to C, the shorter more often; half the slots for C = 1 rows."""
    if C == 1:
        return np.ones(B, dtype=np.int64)
    return 1 + (np.arange(B) * 5 + 3) % C * ((np.arange(B) * 3 + 2) % C) // C


def _token_ranks(n, V):
    """How often each distinct token occurs: the quantiles of a Zipf-like law over V, so that counts go by n and V."""
    u = (np.arange(n) + 0.5) / n
    return np.minimum((V ** u - 1).astype(np.int64), V - 1)


def work(case):
    c = case
    if c["op"] == "logprobs":
        rows = int(_emitted(c["B"], c["C"]).sum())
        items = c["B"] * c["C"]
        return {"bytes": rows * c["V"] * SIZE[c["dtype"]] + items * (4 + 16 + 8 * c["top_k"]),
                "flops": 6 * rows * c["V"]}
    if c["op"] == "logprobs_grad":
        return {"bytes": 2 * c["N"] * c["V"] * SIZE[c["dtype"]] + c["N"] * (24 if c["entropy"] else 16),
                "flops": 6 * c["N"] * c["V"]}
    touched = len(np.unique(_token_ranks(c["n"], c["V"])))
    if c["op"] == "embed":
        return {"bytes": c["r"] * (touched * SIZE[c["dtype"]] + c["n"] * SIZE[c["out"]]) + 4 * c["n"],
                "flops": c["n"] * c["r"]}
    grad = 2 * touched if c["accumulate"] else c["V"]
    return {"bytes": c["r"] * (c["n"] * SIZE[c["dtype"]] + grad * SIZE[c["grad"]]) + 4 * c["n"],
            "flops": 2 * c["n"] * c["r"]}


# ----------------------------------------------------------------- inputs

def _logits(rows, V, pad, dtype, gen):
    """Rows of logits as a model gives them: N(0, s) with s of each row its own, some rows with a grammar's mask of -inf
    that leaves a few hundred tokens, or one token, or none."""
    ld = V + pad
    x = torch.empty(rows, ld, device=DEVICE, dtype=DTYPES[dtype])
    s = 0.5 + 3.5 * torch.rand(rows, 1, device=DEVICE, generator=gen)
    step = max(1, 250_000_000 // ld)
    for at in range(0, rows, step):
        part = torch.randn(min(step, rows - at), ld, device=DEVICE, generator=gen)
        x[at:at + step] = (part * s[at:at + step]).to(x.dtype)
    x = x[:, :V]
    if rows >= 8:
        keep = torch.rand(2, V, device=DEVICE, generator=gen) < min(1.0, 300 / V)
        x[1::8] = x[1::8].masked_fill(~keep[0], -math.inf)
        x[5] = x[5].masked_fill(~keep[1], -math.inf)
        x[3] = -math.inf
        x[3, 7 % V] = 1.5
        x[6] = -math.inf
    return x


def _allowed_tokens(x, gen):
    """A token for each row, one that the row's mask leaves where it can (the best of eight tries)."""
    rows, V = x.shape
    t = torch.randint(0, V, (rows, 8), device=DEVICE, generator=gen)
    return t.gather(1, x.gather(1, t).float().argmax(1, keepdim=True)).squeeze(1)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": c}
    if c["op"] == "logprobs":
        B, C, V, k = c["B"], c["C"], c["V"], c["top_k"]
        n_out = torch.from_numpy(rng.permutation(_emitted(B, C))).to(DEVICE)
        if c["packed"]:     # as the scheduler packs the target rows: only those that a request verifies
            start = torch.cumsum(n_out, 0) - n_out
            n_rows = int(n_out.sum())
        else:
            start, n_rows = torch.arange(B, device=DEVICE) * C, B * C
        s["logits"] = _logits(n_rows, V, c["pad"], c["dtype"], gen)
        slot = torch.arange(C, device=DEVICE)
        used = slot < n_out[:, None]
        rows = (start[:, None] + slot)[used]
        s["tokens"] = torch.full((B, C), -1, dtype=torch.int32, device=DEVICE)
        s["tokens"][used] = _allowed_tokens(s["logits"][rows], gen).int()
        s["row_start"] = start if c["packed"] else None
        outs = dict(logprob=torch.empty(B, C, device=DEVICE), entropy=torch.empty(B, C, device=DEVICE),
                    stats=torch.empty(B, C, 2, device=DEVICE))
        if k:
            outs["top_tokens"] = torch.empty(B, C, k, dtype=torch.int32, device=DEVICE)
            outs["top_logprobs"] = torch.empty(B, C, k, device=DEVICE)
        s["outs"] = outs
    elif c["op"] == "logprobs_grad":
        N, V = c["N"], c["V"]
        x = s["logits"] = _logits(N, V, c["pad"], c["dtype"], gen)
        tokens = _allowed_tokens(x, gen).int()
        tokens[4::9] = -1                       # positions behind the last label
        s["tokens"] = tokens
        m, sums, H = _row_stats(x.float())
        s["stats"] = torch.stack([m, sums], 1).contiguous()
        s["entropy"] = H if c["entropy"] else None
        s["g_logprob"] = torch.randn(N, device=DEVICE, generator=gen) / N
        s["g_entropy"] = 0.01 * torch.randn(N, device=DEVICE, generator=gen) / N if c["entropy"] else None
        s["dlogits"] = torch.empty(N, V + c["pad"], dtype=x.dtype, device=DEVICE)[:, :V]
    else:
        n, V, r = c["n"], c["V"], c["r"]
        names = rng.permutation(V)              # which token has which rank
        tokens = names[rng.permutation(_token_ranks(n, V))]
        s["tokens"] = torch.from_numpy(tokens.astype(np.int32)).to(DEVICE)
        s["scale"] = 1.0 / math.sqrt(r) if c["op"] == "embed_grad" else math.sqrt(r)
        if c["op"] == "embed":
            s["table"] = (0.02 * torch.randn(V, r, device=DEVICE, generator=gen)).to(DTYPES[c["dtype"]])
            s["out"] = torch.empty(n, r, dtype=DTYPES[c["out"]], device=DEVICE)
        else:
            s["dout"] = torch.randn(n, r, device=DEVICE, generator=gen).to(DTYPES[c["dtype"]])
            s["dtable"] = torch.randn(V, r, device=DEVICE, generator=gen).to(DTYPES[c["grad"]])
    if own:
        from speculative_decoding_semi_b200 import binding
        size = (binding.dspark_embed_grad_workspace_bytes(c["n"], c["V"], c["r"]) if c["op"] == "embed_grad" else
                binding.dspark_workspace_bytes(1, 1, 8, 1))
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEVICE)
        binding.dspark_workspace_init(s["workspace"])
    return s


# -------------------------------------------------------------------- run

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "logprobs":
        return _plain_logprobs(s, c)
    if c["op"] == "logprobs_grad":
        return _plain_logprobs_grad(s)
    if c["op"] == "embed":
        return (s["table"][s["tokens"]].float() * s["scale"]).to(s["out"].dtype)
    total = s["dtable"].float() if c["accumulate"] else torch.zeros_like(s["dtable"], dtype=torch.float32)
    total.index_add_(0, s["tokens"], s["dout"].float(), alpha=s["scale"])
    s["dtable"].copy_(total)
    return s["dtable"]


def _run_own(s, c):
    from speculative_decoding_semi_b200 import binding
    if c["op"] == "logprobs":
        o = s["outs"]
        binding.dspark_logprobs(s["logits"], s["tokens"], o["logprob"], o["entropy"], o["stats"],
                                o.get("top_tokens"), o.get("top_logprobs"), s["workspace"], row_start=s["row_start"])
        return o
    if c["op"] == "logprobs_grad":
        binding.dspark_logprobs_grad(s["logits"], s["tokens"], s["stats"], s["entropy"], s["g_logprob"],
                                     s["g_entropy"], s["dlogits"], s["workspace"])
        return s["dlogits"]
    if c["op"] == "embed":
        binding.dspark_embed(s["table"], s["tokens"], s["scale"], s["out"], s["workspace"])
        return s["out"]
    binding.dspark_embed_grad(s["dout"], s["tokens"], s["scale"], s["dtable"], s["workspace"],
                              accumulate=c["accumulate"])
    return s["dtable"]


def _row_stats(x):
    """Largest logit, sum of exponentials under it, and entropy of each row; -inf, 0 and 0 for a row with nothing left."""
    m = x.amax(1)
    y = x - torch.where(m == -math.inf, 0.0, m)[:, None]
    e = y.exp()
    sums = e.sum(1)
    tilted = e.mul_(y.clamp_(min=-1e4)).sum(1)
    return m, sums, torch.where(sums > 0, sums.log() - tilted / sums, 0.0)


def _plain_logprobs(s, c):
    B, C, V, k = c["B"], c["C"], c["V"], c["top_k"]
    tokens = s["tokens"].reshape(-1)
    used = tokens >= 0
    slot = torch.arange(C, device=DEVICE)
    start = s["row_start"] if s["row_start"] is not None else torch.arange(B, device=DEVICE) * C
    x = s["logits"][(start[:, None] + slot).reshape(-1)[used]].float()
    m, sums, H = _row_stats(x)
    x_t = x.gather(1, tokens[used].long()[:, None]).squeeze(1)
    lp = torch.where(x_t == -math.inf, x_t, x_t - m - sums.log())
    o = {"logprob": torch.zeros(B * C, device=DEVICE), "entropy": torch.zeros(B * C, device=DEVICE),
         "stats": torch.zeros(B * C, 2, device=DEVICE)}
    o["logprob"][used] = lp
    o["entropy"][used] = H
    o["stats"][used] = torch.stack([m, sums], 1)
    if k:
        # the order of the alternatives as one 64-bit number: the logit's order, then the lowest token
        bits = (x + 0.0).view(torch.int32)
        key = ((bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32) + torch.arange(V - 1, -1, -1, device=DEVICE)
        at = V - 1 - (key.topk(min(k, V), dim=1).values & 0xFFFFFFFF)
        x_at = x.gather(1, at)
        none = x_at == -math.inf
        o["top_tokens"] = torch.full((B * C, k), -1, dtype=torch.int32, device=DEVICE)
        o["top_logprobs"] = torch.full((B * C, k), -math.inf, device=DEVICE)
        rows = used.nonzero()
        to = torch.arange(min(k, V), device=DEVICE)
        o["top_tokens"][rows, to] = torch.where(none, -1, at).int()
        o["top_logprobs"][rows, to] = torch.where(none, -math.inf, x_at - m[:, None] - sums.log()[:, None])
    return {name: v.reshape(B, C, *v.shape[1:]) for name, v in o.items()}


def _plain_logprobs_grad(s):
    x = s["logits"].float()
    m, sums = s["stats"][:, :1], s["stats"][:, 1:]
    y = (x - torch.where(m == -math.inf, 0.0, m)).clamp_(min=-1e4)
    p = torch.where(sums > 0, y.exp() / sums, 0.0)
    lp = y - sums.log()
    g = torch.where(s["tokens"] >= 0, s["g_logprob"], 0.0)[:, None]
    d = p * -g
    if s["g_entropy"] is not None:
        gh = torch.where(s["tokens"] >= 0, s["g_entropy"], 0.0)[:, None]
        d -= torch.where(p > 0, gh * p * (lp + s["entropy"][:, None]), 0.0)
    t = s["tokens"].long().clamp(min=0)[:, None]
    d.scatter_add_(1, t, torch.where(x.gather(1, t) > -math.inf, g, 0.0))
    s["dlogits"].copy_(d)
    return s["dlogits"]


# ------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "embed":
        return s["table"].to(f64)[s["tokens"].long()] * s["scale"]
    if c["op"] == "embed_grad":
        d = s["dtable"].to(f64) * (1.0 if c["accumulate"] else 0.0)
        order = torch.argsort(s["tokens"].long(), stable=True)
        at = s["tokens"].long()[order]
        last = torch.ones_like(at, dtype=torch.bool)
        last[:-1] = at[1:] != at[:-1]
        for j in range(0, c["r"], 128):        # sums of each token's run, from running totals in 64 bits
            total = torch.cumsum(s["dout"][:, j:j + 128].to(f64)[order], 0)[last]
            total[1:] -= total[:-1].clone()
            d[at[last], j:j + 128] += total * s["scale"]
        return d
    if c["op"] == "logprobs_grad":
        d = torch.zeros(c["N"], c["V"], dtype=f64, device=DEVICE)
        for i in range(0, c["N"], 256):
            x = s["logits"][i:i + 256].to(f64)
            t = s["tokens"][i:i + 256].long()
            left = (x > -math.inf) & (t >= 0)[:, None]
            lp = torch.log_softmax(x, 1)
            p = torch.where(left, lp.exp(), 0.0)
            g = s["g_logprob"][i:i + 256].to(f64)[:, None]
            hit = torch.arange(c["V"], device=DEVICE) == t[:, None]
            v = torch.where(left, g * (hit.to(f64) - p), 0.0)
            if c["entropy"]:
                safe = torch.where(p > 0, lp, 0.0)
                H = -(p * safe).sum(1, keepdim=True)
                v -= s["g_entropy"][i:i + 256].to(f64)[:, None] * p * (safe + H)
            d[i:i + 256] = v
        return d
    B, C, k = c["B"], c["C"], c["top_k"]
    tokens = s["tokens"].cpu().numpy()
    start = s["row_start"].cpu().numpy() if s["row_start"] is not None else np.arange(B) * C
    o = {"logprob": torch.zeros(B, C, dtype=f64), "entropy": torch.zeros(B, C, dtype=f64),
         "stats": torch.zeros(B, C, 2, dtype=f64)}
    if k:
        o["top_logprobs"] = torch.full((B, C, k), -math.inf, dtype=f64)
    b, j = np.nonzero(tokens >= 0)
    for i in range(0, len(b), 256):
        bi, ji = b[i:i + 256], j[i:i + 256]
        x = s["logits"][torch.from_numpy(start[bi] + ji).to(DEVICE)].to(f64)
        top = x.topk(min(max(k, 1), c["V"]), dim=1).values
        lse = torch.logsumexp(x, 1)
        empty = top[:, 0] == -math.inf
        lp = torch.where(x > -math.inf, x - lse[:, None], -math.inf)
        p = lp.exp()
        o["logprob"][bi, ji] = lp.gather(1, s["tokens"][bi, ji].long()[:, None]).squeeze(1).cpu()
        o["entropy"][bi, ji] = -torch.where(p > 0, p * lp, 0.0).sum(1).cpu()
        sums = torch.where(empty, 0.0, torch.exp(lse - top[:, 0]))
        o["stats"][bi, ji] = torch.stack([top[:, 0], sums], 1).cpu()
        if k:
            o["top_logprobs"][bi, ji, :top.shape[1]] = torch.where(top > -math.inf, top - lse[:, None], -math.inf).cpu()
            o["top_tokens"] = None
    return o
