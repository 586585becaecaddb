"""Gradient of the Markov head's factors from a round's outcome.

QbitAI article "DSpark: ten concepts are enough", section "online drafter
calibration": the drafter corrects itself from the workload it sees. Where
dspark_calibrate moves the confidence temperatures, this moves the head: the
emitted tokens are the labels of the draft's positions. Position i of request b
has one if the drafts before it were all accepted (out_tokens[b,i] for
i < n_out[b]: an accepted draft, the token drawn at the first rejection, or the
bonus token where the verify length ends before K), and
  loss = -(1/n) sum log q_i(label) - (entropy_bonus/n) sum H(q_i)
over the n positions that have one, q_i = softmax(z_i), z_i = base_i + A[t_{i-1}] . Bf.
The log probabilities, their gradient dz, the rows of A and the gradient of A
by sorted tokens are the library's kernels; the two plain products
dBf = rows^T dz and drows = dz Bf^T are torch's.
"""
from __future__ import annotations

import torch

from .binding import (dspark_embed, dspark_embed_grad, dspark_embed_grad_workspace_bytes, dspark_logprobs,
                      dspark_logprobs_grad, dspark_workspace_init)
from .round import RoundBuffers


class HeadGradients:
    """Gradients of A [V,r] and Bf [r,V] (float32) and the buffers of a step on
    rounds of this shape; logprob [B,K] and entropy [B,K] of the labels (0
    where a position has none) are left for the caller."""

    def __init__(self, B: int, K: int, V: int, r: int, device="cuda"):
        f32 = torch.float32
        self.B, self.K, self.V, self.r = B, K, V, r
        self.dA = torch.zeros(V, r, dtype=f32, device=device)
        self.dBf = torch.zeros(r, V, dtype=f32, device=device)
        self.logprob = torch.empty(B, K, dtype=f32, device=device)
        self.entropy = torch.empty(B, K, dtype=f32, device=device)
        self.stats = torch.empty(B, K, 2, dtype=f32, device=device)
        self.dz = torch.empty(B * K, V, dtype=f32, device=device)
        self.rows = torch.empty(B * K, r, dtype=f32, device=device)
        self.workspace = torch.empty(dspark_embed_grad_workspace_bytes(B * K, V, r), dtype=torch.uint8, device=device)
        dspark_workspace_init(self.workspace)


def _torch_stream(stream, device) -> torch.cuda.Stream:
    """What the entry points take as `stream` (None: the current one, a torch stream, or a handle; 0 is the legacy
    default stream) as a torch stream."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if not isinstance(stream, int):
        return stream
    return torch.cuda.ExternalStream(stream, device=device) if stream != 0 else torch.cuda.default_stream(device)


def head_gradients(d: dict, bufs: RoundBuffers, grads: HeadGradients, anchor=None, entropy_bonus: float = 0.0,
                   accumulate: bool = False, stream=None) -> torch.Tensor:
    """The loss (a device scalar), with its gradients in grads.dA and grads.dBf
    (added to them with accumulate=True), from the round that `d` and `bufs`
    just ran; no host synchronisation. `anchor` as it was given to the draft
    (default d["anchor"]). Variant "a" of the round (the draft stored z) with
    the Markov head."""
    if bufs.variant != "a":
        raise ValueError("head_gradients reads the draft's z: run the round with variant 'a'")
    if d.get("W") is not None:
        raise ValueError("head_gradients is of the Markov head; this round ran the RNN head")
    B, K, V, r = grads.B, grads.K, grads.V, grads.r
    if (bufs.B, bufs.K, bufs.V, bufs.r) != (B, K, V, r):
        raise ValueError(f"a round of {(bufs.B, bufs.K, bufs.V, bufs.r)} for gradients of {(B, K, V, r)}")
    with torch.cuda.stream(_torch_stream(stream, grads.dA.device)):
        labels = bufs.out_tokens[:, :K].contiguous()
        used = labels >= 0
        n = used.sum().clamp(min=1)
        anchor = d["anchor"] if anchor is None else anchor
        previous = torch.cat([anchor[:, None], bufs.draft_tokens[:, :K - 1]], dim=1)
        previous = torch.where(used, previous, -1)
        z = bufs.z.view(B * K, V)
        dspark_logprobs(z, labels, grads.logprob, grads.entropy, grads.stats, None, None, grads.workspace)
        g = (-1.0 / n).expand(B, K).contiguous()
        gh = (-entropy_bonus / n).expand(B, K).contiguous() if entropy_bonus != 0.0 else None
        dspark_logprobs_grad(z, labels, grads.stats, grads.entropy if gh is not None else None, g, gh, grads.dz,
                             grads.workspace)
        dspark_embed(d["A"], previous, 1.0, grads.rows, grads.workspace)
        if accumulate:
            grads.dBf.addmm_(grads.rows.t(), grads.dz)
        else:
            torch.mm(grads.rows.t(), grads.dz, out=grads.dBf)
        drows = torch.mm(grads.dz, d["Bf"].float().t())
        dspark_embed_grad(drows, previous, 1.0, grads.dA, grads.workspace, accumulate=accumulate)
        return -(grads.logprob.sum() + entropy_bonus * grads.entropy.sum()) / n
