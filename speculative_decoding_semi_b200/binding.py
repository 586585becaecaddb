"""Thin ctypes binding of libdspark (argument marshalling only).

The functions carry the C names of include/dspark.h and take torch CUDA
tensors (for device memory) plus an optional torch.cuda.Stream; every step of
the computation runs in the library's kernels. If the library is missing the
import fails loudly: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdspark.so")

DSPARK_F32, DSPARK_BF16 = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "CUDA error",
          4: "device-wide wait timed out", 5: "device-side check failed"}


class DSparkError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: int | None = None):
        self.status = status
        self.detail = detail
        msg = f"{fn}: {STATUS.get(status, status)} (status {status})"
        if detail is not None:
            msg += f", detail 0x{detail:08x}"
        super().__init__(msg)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python speculative_decoding_semi_b200/build.py` "
            "(nvcc, sm_100a). There is no CPU fallback.")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, Z, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    lib.dspark_workspace_bytes.argtypes = [I, I, I, I]
    lib.dspark_workspace_bytes.restype = Z
    lib.dspark_workspace_init.argtypes = [P, Z, S]
    lib.dspark_workspace_init.restype = I
    lib.dspark_markov_draft.argtypes = [P, P, P, I, I, P, P, I, I, I, P, P, P, P, P, Z, S]
    lib.dspark_markov_draft.restype = I
    lib.dspark_rnn_draft.argtypes = [P, P, P, P, I, I, P, P, I, I, I, P, P, P, P, P, Z, S]
    lib.dspark_rnn_draft.restype = I
    lib.dspark_schedule.argtypes = [P, P, P, I, I, I, P, P, P, P, P, Z, S]
    lib.dspark_schedule.restype = I
    lib.dspark_verify.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, P, P, P, P, Z, S]
    lib.dspark_verify.restype = I
    lib.dspark_markov_draft_b.argtypes = [P, P, P, I, I, P, P, I, I, I, P, P, P, P, P, Z, S]
    lib.dspark_markov_draft_b.restype = I
    lib.dspark_rnn_draft_b.argtypes = [P, P, P, P, I, I, P, P, I, I, I, P, P, P, P, P, Z, S]
    lib.dspark_rnn_draft_b.restype = I
    lib.dspark_verify_b.argtypes = [P, P, P, P, P, I, P, P, P, P, P, P, I, I, I, P, P, P, P, Z, S]
    lib.dspark_verify_b.restype = I
    lib.dspark_read_device_error.argtypes = [P, S, ctypes.POINTER(ctypes.c_uint32)]
    lib.dspark_read_device_error.restype = I
    lib.dspark_schedule_static.argtypes = [P, P, P, I, I, I, P, P, P, P, S]
    lib.dspark_schedule_static.restype = I
    F = ctypes.c_float
    lib.dspark_calibrate.argtypes = [P, P, P, I, I, F, F, F, P, P, Z, S]
    lib.dspark_calibrate.restype = I
    lib.dspark_advance_anchor.argtypes = [P, P, I, I, P, P, Z, S]
    lib.dspark_advance_anchor.restype = I
    L = ctypes.c_int64
    lib.dspark_logprobs.argtypes = [P, I, L, L, P, P, I, I, I, I, P, P, P, P, P, P, Z, S]
    lib.dspark_logprobs.restype = I
    lib.dspark_logprobs_grad.argtypes = [P, I, L, P, P, P, P, P, I, I, P, L, P, Z, S]
    lib.dspark_logprobs_grad.restype = I
    lib.dspark_embed.argtypes = [P, I, P, I, I, I, F, P, I, P, Z, S]
    lib.dspark_embed.restype = I
    lib.dspark_embed_grad_workspace_bytes.argtypes = [I, I, I]
    lib.dspark_embed_grad_workspace_bytes.restype = Z
    lib.dspark_embed_grad.argtypes = [P, I, P, I, I, I, F, I, P, I, P, Z, S]
    lib.dspark_embed_grad.restype = I
    lib.dspark_set_wait_budget.argtypes = [P, ctypes.c_uint32, S]
    lib.dspark_set_wait_budget.restype = I
    lib.dspark_inject_stall.argtypes = [P, I, ctypes.c_uint32, S]
    lib.dspark_inject_stall.restype = I
    lib.dspark_status_string.argtypes = [I]
    lib.dspark_status_string.restype = ctypes.c_char_p
    return lib


lib = _load()


def _ptr(t: torch.Tensor | None, name: str, dtype=None, numel=None) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor (the library computes on the GPU only)")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != 0:
        raise DSparkError(fn, status)


def dspark_workspace_bytes(B: int, K: int, V: int, r: int) -> int:
    n = lib.dspark_workspace_bytes(B, K, V, r)
    if n == 0:
        raise DSparkError("dspark_workspace_bytes", 1)
    return int(n)


def dspark_workspace_init(workspace: torch.Tensor, stream=None) -> None:
    _check("dspark_workspace_init",
           lib.dspark_workspace_init(_ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream)))


def dspark_markov_draft(base_logits, A, Bf, anchor, u_draft, draft_tokens, q_tok, lse_q, z, workspace,
                        stream=None) -> None:
    B, K, V = base_logits.shape
    r = A.shape[1]
    if A.dtype == torch.bfloat16 and Bf.dtype == torch.bfloat16:
        dt = DSPARK_BF16
    elif A.dtype == torch.float32 and Bf.dtype == torch.float32:
        dt = DSPARK_F32
    else:
        raise TypeError("A and Bf must both be float32 or both bfloat16")
    st = lib.dspark_markov_draft(
        _ptr(base_logits, "base_logits", torch.float32), _ptr(A, "A", numel=V * r), _ptr(Bf, "Bf", numel=r * V),
        dt, r, _ptr(anchor, "anchor", torch.int32, B), _ptr(u_draft, "u_draft", torch.float32, B * K),
        B, K, V, _ptr(draft_tokens, "draft_tokens", torch.int32, B * K), _ptr(q_tok, "q_tok", torch.float32, B * K),
        _ptr(lse_q, "lse_q", torch.float64, B * K), _ptr(z, "z", torch.float32, B * K * V),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("dspark_markov_draft", st)


def dspark_rnn_draft(base_logits, A, W, Bf, anchor, u_draft, draft_tokens, q_tok, lse_q, z, workspace,
                     stream=None) -> None:
    """Draft with the RNN sequential head (W [r,r] bf16); bf16 factors only."""
    B, K, V = base_logits.shape
    r = A.shape[1]
    if not (A.dtype == Bf.dtype == W.dtype == torch.bfloat16):
        raise TypeError("the RNN head takes bf16 A, W and Bf")
    st = lib.dspark_rnn_draft(
        _ptr(base_logits, "base_logits", torch.float32), _ptr(A, "A", numel=V * r), _ptr(W, "W", numel=r * r),
        _ptr(Bf, "Bf", numel=r * V), DSPARK_BF16, r, _ptr(anchor, "anchor", torch.int32, B),
        _ptr(u_draft, "u_draft", torch.float32, B * K), B, K, V,
        _ptr(draft_tokens, "draft_tokens", torch.int32, B * K), _ptr(q_tok, "q_tok", torch.float32, B * K),
        _ptr(lse_q, "lse_q", torch.float64, B * K), _ptr(z, "z", torch.float32, B * K * V),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("dspark_rnn_draft", st)


def dspark_markov_draft_b(base_logits, A, Bf, anchor, u_draft, draft_tokens, q_tok, lse_q, op_rows, workspace,
                          stream=None) -> None:
    """Variant B of dspark_markov_draft: no z; op_rows [B,K,r] (bfloat16)
    receives the operand row of every position. bf16 factors only."""
    B, K, V = base_logits.shape
    r = A.shape[1]
    if not (A.dtype == Bf.dtype == torch.bfloat16):
        raise TypeError("variant B takes bf16 A and Bf")
    st = lib.dspark_markov_draft_b(
        _ptr(base_logits, "base_logits", torch.float32), _ptr(A, "A", numel=V * r), _ptr(Bf, "Bf", numel=r * V),
        DSPARK_BF16, r, _ptr(anchor, "anchor", torch.int32, B), _ptr(u_draft, "u_draft", torch.float32, B * K),
        B, K, V, _ptr(draft_tokens, "draft_tokens", torch.int32, B * K), _ptr(q_tok, "q_tok", torch.float32, B * K),
        _ptr(lse_q, "lse_q", torch.float64, B * K), _ptr(op_rows, "op_rows", torch.bfloat16, B * K * r),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("dspark_markov_draft_b", st)


def dspark_rnn_draft_b(base_logits, A, W, Bf, anchor, u_draft, draft_tokens, q_tok, lse_q, op_rows, workspace,
                       stream=None) -> None:
    """Variant B of dspark_rnn_draft (op_rows in place of z)."""
    B, K, V = base_logits.shape
    r = A.shape[1]
    if not (A.dtype == Bf.dtype == W.dtype == torch.bfloat16):
        raise TypeError("the RNN head takes bf16 A, W and Bf")
    st = lib.dspark_rnn_draft_b(
        _ptr(base_logits, "base_logits", torch.float32), _ptr(A, "A", numel=V * r), _ptr(W, "W", numel=r * r),
        _ptr(Bf, "Bf", numel=r * V), DSPARK_BF16, r, _ptr(anchor, "anchor", torch.int32, B),
        _ptr(u_draft, "u_draft", torch.float32, B * K), B, K, V,
        _ptr(draft_tokens, "draft_tokens", torch.int32, B * K), _ptr(q_tok, "q_tok", torch.float32, B * K),
        _ptr(lse_q, "lse_q", torch.float64, B * K), _ptr(op_rows, "op_rows", torch.bfloat16, B * K * r),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("dspark_rnn_draft_b", st)


def dspark_schedule(conf_logits, temps, profile_ms, verify_len, survival, row_start, n_tokens, workspace,
                    stream=None) -> None:
    B, K = conf_logits.shape
    st = lib.dspark_schedule(
        _ptr(conf_logits, "conf_logits", torch.float32), _ptr(temps, "temps", torch.float32, K),
        _ptr(profile_ms, "profile_ms", torch.float32), profile_ms.numel(), B, K,
        _ptr(verify_len, "verify_len", torch.int32, B), _ptr(survival, "survival", torch.float32, B * K),
        _ptr(row_start, "row_start", torch.int64, B), _ptr(n_tokens, "n_tokens", torch.int32, 1),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("dspark_schedule", st)


def dspark_schedule_static(conf_logits, temps, profile_ms, verify_len, survival, row_start, n_tokens,
                           stream=None) -> None:
    """dspark_schedule without a workspace (scratch in a static device array
    inside the library), for callers that cannot allocate device memory. Same
    outputs; B*K is limited to 16384; calls must not overlap on the GPU."""
    B, K = conf_logits.shape
    st = lib.dspark_schedule_static(
        _ptr(conf_logits, "conf_logits", torch.float32), _ptr(temps, "temps", torch.float32, K),
        _ptr(profile_ms, "profile_ms", torch.float32), profile_ms.numel(), B, K,
        _ptr(verify_len, "verify_len", torch.int32, B), _ptr(survival, "survival", torch.float32, B * K),
        _ptr(row_start, "row_start", torch.int64, B), _ptr(n_tokens, "n_tokens", torch.int32, 1),
        _stream(stream))
    _check("dspark_schedule_static", st)


def dspark_verify(target_logits, row_start, z, lse_q, q_tok, draft_tokens, verify_len, u_accept, u_resample,
                  accepted, out_tokens, n_out, workspace, stream=None) -> None:
    B, K, V = z.shape
    if target_logits.shape[-1] != V:
        raise ValueError("target_logits must have V columns")
    st = lib.dspark_verify(
        _ptr(target_logits, "target_logits", torch.float32), _ptr(row_start, "row_start", torch.int64, B),
        _ptr(z, "z", torch.float32), _ptr(lse_q, "lse_q", torch.float64, B * K),
        _ptr(q_tok, "q_tok", torch.float32, B * K), _ptr(draft_tokens, "draft_tokens", torch.int32, B * K),
        _ptr(verify_len, "verify_len", torch.int32, B), _ptr(u_accept, "u_accept", torch.float32, B * K),
        _ptr(u_resample, "u_resample", torch.float32, B), B, K, V,
        _ptr(accepted, "accepted", torch.int32, B), _ptr(out_tokens, "out_tokens", torch.int32, B * (K + 1)),
        _ptr(n_out, "n_out", torch.int32, B), _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
        _stream(stream))
    _check("dspark_verify", st)


def dspark_verify_b(target_logits, row_start, base_logits, op_rows, Bf, lse_q, q_tok, draft_tokens, verify_len,
                    u_accept, u_resample, accepted, out_tokens, n_out, workspace, stream=None) -> None:
    """Variant B of dspark_verify: the rejected row's z is recomputed from
    base_logits, op_rows [B,K,r] (bfloat16) and Bf [r,V] (bfloat16)."""
    B, K, V = base_logits.shape
    r = Bf.shape[0]
    if target_logits.shape[-1] != V:
        raise ValueError("target_logits must have V columns")
    st = lib.dspark_verify_b(
        _ptr(target_logits, "target_logits", torch.float32), _ptr(row_start, "row_start", torch.int64, B),
        _ptr(base_logits, "base_logits", torch.float32), _ptr(op_rows, "op_rows", torch.bfloat16, B * K * r),
        _ptr(Bf, "Bf", torch.bfloat16, r * V), r, _ptr(lse_q, "lse_q", torch.float64, B * K),
        _ptr(q_tok, "q_tok", torch.float32, B * K), _ptr(draft_tokens, "draft_tokens", torch.int32, B * K),
        _ptr(verify_len, "verify_len", torch.int32, B), _ptr(u_accept, "u_accept", torch.float32, B * K),
        _ptr(u_resample, "u_resample", torch.float32, B), B, K, V,
        _ptr(accepted, "accepted", torch.int32, B), _ptr(out_tokens, "out_tokens", torch.int32, B * (K + 1)),
        _ptr(n_out, "n_out", torch.int32, B), _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
        _stream(stream))
    _check("dspark_verify_b", st)


def dspark_calibrate(conf_logits, verify_len, accepted, temps, workspace, eta: float, t_min: float, t_max: float,
                     stream=None) -> None:
    """One online step of the sequential temperatures (temps updated in place)."""
    B, K = conf_logits.shape
    st = lib.dspark_calibrate(
        _ptr(conf_logits, "conf_logits", torch.float32), _ptr(verify_len, "verify_len", torch.int32, B),
        _ptr(accepted, "accepted", torch.int32, B), B, K, float(eta), float(t_min), float(t_max),
        _ptr(temps, "temps", torch.float32, K), _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
        _stream(stream))
    _check("dspark_calibrate", st)


def dspark_advance_anchor(out_tokens, n_out, anchor, workspace, stream=None) -> None:
    """anchor[b] = out_tokens[b, n_out[b]-1], for the next round."""
    B, K1 = out_tokens.shape
    st = lib.dspark_advance_anchor(
        _ptr(out_tokens, "out_tokens", torch.int32), _ptr(n_out, "n_out", torch.int32, B), B, K1 - 1,
        _ptr(anchor, "anchor", torch.int32, B), _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
        _stream(stream))
    _check("dspark_advance_anchor", st)


DSPARK_MAX_TOP_K, DSPARK_MAX_EMBED_R = 32, 8192
_DTYPES = {torch.float32: DSPARK_F32, torch.bfloat16: DSPARK_BF16}


def _dtype(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected float32 or bfloat16, got {t.dtype}")
    return code


def _rows(t: torch.Tensor, name: str) -> tuple[int, int, int, int]:
    """(pointer, rows, columns, row stride) of a [rows, columns] CUDA tensor
    whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor (the library computes on the GPU only)")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected two dimensions, got {t.dim()}")
    rows, cols = t.shape
    if t.is_contiguous():
        return t.data_ptr(), rows, cols, cols
    stride, step = t.stride()
    if cols > 1 and step != 1 or rows > 1 and stride < cols:
        raise ValueError(f"{name}: expected contiguous rows at least {cols} elements apart")
    return t.data_ptr(), rows, cols, max(stride, cols)


def _on(dev: int, t: torch.Tensor | None, name: str, dtype, numel: int) -> int | None:
    """_ptr for a tensor that has to be on device `dev`. The calls of a small
    batch are bound by the time spent here, so the good case comes first."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.numel() == numel \
            and t.is_contiguous():
        return t.data_ptr()
    _ptr(t, name, dtype, numel)
    raise ValueError(f"{name}: expected a tensor on cuda:{dev}, got {t.device}")


def _launch_stream(name: str, dev: int, stream) -> int | None:
    """The stream's handle; None where the tensors' device is not the current
    one (the call is then made with it current)."""
    if dev < 0:
        raise ValueError(f"{name}: expected CUDA tensors (the library computes on the GPU only)")
    if stream is not None and isinstance(stream, torch.cuda.Stream) and stream.device.index != dev:
        raise ValueError(f"{name}: tensors on cuda:{dev}, stream on {stream.device}")
    if dev != torch._C._cuda_getDevice():
        return None
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _call(fn, name: str, dev: int, stream, *args) -> None:
    s = _launch_stream(name, dev, stream)
    if s is not None:
        status = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream(stream))
    if status != 0:
        raise DSparkError(name, status)


def dspark_logprobs(logits, tokens, logprob, entropy, stats, top_tokens, top_logprobs, workspace, row_start=None,
                    stream=None) -> None:
    """Log probabilities of tokens [B,C] (-1: left out) on rows of logits
    [rows,V] (float32 or bfloat16, rows any stride apart): row row_start[b] + c,
    or b*C + c without row_start. entropy, stats and (both) alternatives may be
    None; top_k is their last dimension."""
    dt = _dtype(logits, "logits")
    ptr, n_rows, V, ld = _rows(logits, "logits")
    dev = logits.get_device()
    B, C = tokens.shape
    n, k = B * C, 0
    if (top_tokens is None) != (top_logprobs is None):
        raise ValueError("top_tokens and top_logprobs: give both or neither")
    if top_tokens is not None:
        if top_tokens.dim() != 3:
            raise ValueError("top_tokens: expected [B,C,top_k]")
        k = top_tokens.shape[2]
    f32, i32 = torch.float32, torch.int32
    size = workspace.numel()
    _call(lib.dspark_logprobs, "dspark_logprobs", dev, stream, ptr, dt, n_rows, ld,
          _on(dev, row_start, "row_start", torch.int64, B), _on(dev, tokens, "tokens", i32, n), B, C, V, k,
          _on(dev, logprob, "logprob", f32, n), _on(dev, entropy, "entropy", f32, n),
          _on(dev, stats, "stats", f32, 2 * n), _on(dev, top_tokens, "top_tokens", i32, n * k),
          _on(dev, top_logprobs, "top_logprobs", f32, n * k), _on(dev, workspace, "workspace", torch.uint8, size),
          size)


def dspark_logprobs_grad(logits, tokens, stats, entropy, g_logprob, g_entropy, dlogits, workspace,
                         stream=None) -> None:
    """dlogits [N,V] = the gradient of dspark_logprobs' logprob (times
    g_logprob [N]) and entropy (times g_entropy [N], or None) with respect to
    logits [N,V]; tokens [N] or any shape of N elements. dlogits may be logits."""
    dt = _dtype(logits, "logits")
    if dlogits.dtype is not logits.dtype:
        raise TypeError("dlogits: expected the type of logits")
    ptr, N, V, ld = _rows(logits, "logits")
    gptr, gN, gV, gld = _rows(dlogits, "dlogits")
    if gN != N or gV != V:
        raise ValueError(f"dlogits: expected [{N},{V}], got [{gN},{gV}]")
    if g_entropy is not None and entropy is None:
        raise ValueError("entropy: needed with g_entropy")
    dev, f32, size = logits.get_device(), torch.float32, workspace.numel()
    if dlogits.get_device() != dev:
        raise ValueError(f"dlogits: expected a tensor on cuda:{dev}, got {dlogits.device}")
    _call(lib.dspark_logprobs_grad, "dspark_logprobs_grad", dev, stream, ptr, dt, ld,
          _on(dev, tokens, "tokens", torch.int32, N), _on(dev, stats, "stats", f32, 2 * N),
          _on(dev, entropy, "entropy", f32, N), _on(dev, g_logprob, "g_logprob", f32, N),
          _on(dev, g_entropy, "g_entropy", f32, N), N, V, gptr, gld,
          _on(dev, workspace, "workspace", torch.uint8, size), size)


def _embed_ptrs(dev: int, table, tokens, rows, name: str, workspace, n: int, V: int, r: int):
    """Pointers of a table [V,r], tokens [n], rows [n,r] (called `name`) and
    the workspace, all on device `dev`; one look at each tensor's properties."""
    size = workspace.numel()
    if (table.is_contiguous() and rows.is_contiguous() and tokens.is_contiguous() and workspace.is_contiguous()
            and tokens.dtype is torch.int32 and workspace.dtype is torch.uint8 and rows.numel() == n * r
            and tokens.get_device() == rows.get_device() == workspace.get_device() == dev):
        return table.data_ptr(), tokens.data_ptr(), rows.data_ptr(), workspace.data_ptr(), size
    _dtype(rows, name)      # say what is wrong
    return (_on(dev, table, "table" if name == "out" else "dtable", table.dtype, V * r),
            _on(dev, tokens, "tokens", torch.int32, n), _on(dev, rows, name, rows.dtype, n * r),
            _on(dev, workspace, "workspace", torch.uint8, size), size)


def dspark_embed(table, tokens, scale: float, out, workspace, stream=None) -> None:
    """out [n,r] = scale * table[tokens] (zeros for a token of -1); table [V,r]
    and out each float32 or bfloat16."""
    V, r = table.shape
    n, dev = tokens.numel(), table.get_device()
    t, tok, o, ws, size = _embed_ptrs(dev, table, tokens, out, "out", workspace, n, V, r)
    _call(lib.dspark_embed, "dspark_embed", dev, stream, t, _dtype(table, "table"), tok, n, V, r, scale, o,
          _dtype(out, "out"), ws, size)


def dspark_embed_grad_workspace_bytes(n: int, V: int, r: int) -> int:
    size = lib.dspark_embed_grad_workspace_bytes(n, V, r)
    if size == 0:
        raise DSparkError("dspark_embed_grad_workspace_bytes", 1)
    return int(size)


def dspark_embed_grad(dout, tokens, scale: float, dtable, workspace, accumulate: bool = False, stream=None) -> None:
    """dtable [V,r] = (accumulate: +=) scale * the sum of dout's rows [n,r] over
    the items of each token; dout and dtable each float32 or bfloat16."""
    V, r = dtable.shape
    n, dev = tokens.numel(), dtable.get_device()
    d, tok, o, ws, size = _embed_ptrs(dev, dtable, tokens, dout, "dout", workspace, n, V, r)
    _call(lib.dspark_embed_grad, "dspark_embed_grad", dev, stream, o, _dtype(dout, "dout"), tok, n, V, r, scale,
          1 if accumulate else 0, d, _dtype(dtable, "dtable"), ws, size)


DSPARK_INJECT_NONE, DSPARK_INJECT_DRAFT_SLICE_SUMS, DSPARK_INJECT_VERIFY_BARRIER = 0, 1, 2
DSPARK_INJECT_RESIDUAL_SLICE_SUMS = 3


def dspark_set_wait_budget(workspace, microseconds: int, stream=None) -> None:
    _check("dspark_set_wait_budget", lib.dspark_set_wait_budget(_ptr(workspace, "workspace", torch.uint8),
                                                                int(microseconds), _stream(stream)))


def dspark_inject_stall(workspace, where: int, cta: int = 0, stream=None) -> None:
    _check("dspark_inject_stall", lib.dspark_inject_stall(_ptr(workspace, "workspace", torch.uint8), int(where),
                                                          int(cta), _stream(stream)))


def dspark_read_device_error(workspace, stream=None) -> tuple[int, int]:
    detail = ctypes.c_uint32(0)
    st = lib.dspark_read_device_error(_ptr(workspace, "workspace", torch.uint8), _stream(stream),
                                      ctypes.byref(detail))
    if st in (1, 3):
        raise DSparkError("dspark_read_device_error", st)
    return int(st), int(detail.value)


def dspark_status_string(status: int) -> str:
    return lib.dspark_status_string(status).decode()
