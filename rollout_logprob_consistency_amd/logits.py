"""Operators on rows of logits (include/liblp_logits.h) on AMD Instinct MI355X.

A thin binding like the rest of the package: it checks and marshals arguments,
and every arithmetic step runs in the library's kernels.

    sample(logits, u, temperature, top_k, top_p, min_p)  -> token, logprob, processed, kept
    top_logprobs(logits, k, temperature)                 -> ids, logits, logprobs [N, k]
    distill(logits, ids, teacher, ...)                   -> loss [T], differentiable
    distill_forward / distill_backward                   -> the two directions by hand
    distill_step(logits, ids, teacher, weight, ...)      -> loss and gradient in one call

Rows of logits are [N, columns] bfloat16, float16 or float32 with unit column
stride and any row stride; `v_true` is the true vocabulary (columns behind it
are padding). distill() alone is differentiable: the other calls' results carry
no derivative, also where the logits require gradients. Scratch memory is
allocated per call unless `workspace` is given (a uint8 tensor of the library's
*_workspace_bytes, 256-byte aligned); calls that may overlap, captured graphs
among them, must not share one. `bad_rows` (int32 [1]) is a counter that a call
adds its bad rows to; with check=True a call raises for its own rows only.
"""

from __future__ import annotations

import torch
from torch.autograd import forward_ad

from ._lib import DISTILL_LOGPROBS, DISTILL_MAX_K, LP_OK, TOP_MAX, LpError, lib

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # LP_F32, LP_BF16, LP_F16


def _rows(name: str, t: torch.Tensor, v_true: int | None):
    """Checks rows of logits; returns (rows, columns, v_true, row stride, dtype code)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"expected {name} [rows, columns]")
    n, columns = t.shape
    vt = columns if v_true is None else int(v_true)
    if not 1 <= vt <= columns:
        raise ValueError(f"v_true must lie in [1, {columns}]")
    ld = t.stride(0) if n > 1 else columns
    if t.stride(1) != 1 and columns > 1 or ld < columns:
        raise ValueError(f"{name} needs unit column stride and rows that do not overlap")
    return n, columns, vt, ld, code


def _like(name: str, t, shape: tuple, dtype: torch.dtype, device: torch.device) -> int:
    """Checks a contiguous tensor beside the logits; returns its address."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on the logits' device")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}")
    return t.data_ptr()


def _setting(name: str, v, n: int, dtype: torch.dtype, device: torch.device):
    """A per-row setting: (address or None, scalar)."""
    if isinstance(v, torch.Tensor):
        return _like(name, v, (n,), dtype, device), 0
    return None, v


def _call(fn, device: torch.device, args: tuple, name: str) -> None:
    """Enqueues on the device's current stream, with that device current (the
    default stream's handle names the current device's)."""
    if device.index == torch.cuda.current_device():
        st = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if st != LP_OK:
        raise LpError(st, name)


def _workspace(ws: torch.Tensor | None, need: int, device: torch.device) -> torch.Tensor:
    if ws is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    if ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be contiguous on the logits' device")
    return ws


def _bad_rows(bad: torch.Tensor | None, check: bool, device: torch.device):
    """What a call counts its bad rows in: with `check` a counter of its own,
    as the caller's may hold the rows of earlier calls."""
    if bad is not None:
        _like("bad_rows", bad, (1,), torch.int32, device)
    return torch.zeros(1, dtype=torch.int32, device=device) if check else bad


def _raise_bad(count: torch.Tensor, bad: torch.Tensor | None, what: str) -> None:
    """After a checked call: its count goes to the caller's counter, and raises."""
    if bad is not None:
        bad.add_(count)
    n = int(count.item())
    if n:
        raise ValueError(f"{n} row(s) {what}")


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
           v_true: int | None = None, *, workspace: torch.Tensor | None = None,
           bad_rows: torch.Tensor | None = None, check: bool = False):
    """One token per row from given uniform random numbers u [N] fp32 (lp_sample).

    temperature, top_p, min_p (fp32) and top_k (int32) are numbers or tensors
    [N], one setting per row; temperature 0 is the greedy draw, top_k <= 0,
    top_p >= 1 and min_p <= 0 keep everything. Returns (token int64, logprob
    fp32 under the full vocabulary, processed fp32 under the kept tokens,
    kept int32), each [N]. Ties go to the lower index. With check=True the
    call synchronises and raises ValueError if a row has no valid draw (a NaN
    or +inf logit, no finite one, a NaN setting, or a temperature that is
    neither 0 nor a positive normal number); else its token is -1. The scores
    are detached from the logits.
    """
    n, _, vt, ld, code = _rows("logits", logits, v_true)
    dev = logits.device
    pu = _like("u", u, (n,), torch.float32, dev)
    pt, temperature = _setting("temperature", temperature, n, torch.float32, dev)
    pk, top_k = _setting("top_k", top_k, n, torch.int32, dev)
    pp, top_p = _setting("top_p", top_p, n, torch.float32, dev)
    pm, min_p = _setting("min_p", min_p, n, torch.float32, dev)
    top_k = max(-1, min(int(top_k), 2 ** 31 - 1))
    token = torch.empty(n, dtype=torch.int64, device=dev)
    logprob = torch.empty(n, dtype=torch.float32, device=dev)
    processed = torch.empty(n, dtype=torch.float32, device=dev)
    kept = torch.empty(n, dtype=torch.int32, device=dev)
    L = lib()
    ws = _workspace(workspace, L.lp_sample_workspace_bytes(n, vt, code), dev)
    count = _bad_rows(bad_rows, check, dev)
    _call(L.lp_sample, dev,
          (logits.data_ptr(), ld, code, n, vt, pu, pt, float(temperature), pk, top_k, pp,
           float(top_p), pm, float(min_p), token.data_ptr(), logprob.data_ptr(),
           processed.data_ptr(), kept.data_ptr(), None if count is None else count.data_ptr(),
           ws.data_ptr(), ws.numel() * ws.element_size()), "lp_sample")
    if check:
        _raise_bad(count, bad_rows, "have no valid draw")
    return token, logprob, processed, kept


def top_logprobs(logits: torch.Tensor, k: int, temperature: float = 1.0,
                 v_true: int | None = None, *, lse: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, bad_rows: torch.Tensor | None = None,
                 check: bool = False):
    """The k largest logits of every row (lp_top_logprobs), largest first,
    ties by lower index: (ids int64, logits fp32, logprobs fp32 at
    `temperature`), each [N, k]. A row with fewer finite logits ends in id -1
    and -inf. lse [N] fp32 receives the row's log-sum-exp. With check=True the
    call synchronises and raises ValueError if a row has a NaN or +inf logit
    or no finite one; else its ids are -1 and its values NaN. The results are
    detached from the logits."""
    n, _, vt, ld, code = _rows("logits", logits, v_true)
    k = int(k)
    if not 1 <= k <= min(vt, TOP_MAX):
        raise ValueError(f"k must lie in [1, {min(vt, TOP_MAX)}]")
    dev = logits.device
    plse = None if lse is None else _like("lse", lse, (n,), torch.float32, dev)
    ids = torch.empty((n, k), dtype=torch.int64, device=dev)
    values = torch.empty((n, k), dtype=torch.float32, device=dev)
    logprobs = torch.empty((n, k), dtype=torch.float32, device=dev)
    L = lib()
    ws = _workspace(workspace, L.lp_top_logprobs_workspace_bytes(n, vt, code), dev)
    count = _bad_rows(bad_rows, check, dev)
    _call(L.lp_top_logprobs, dev,
          (logits.data_ptr(), ld, code, n, vt, k, float(temperature), ids.data_ptr(),
           values.data_ptr(), logprobs.data_ptr(), plse, None if count is None else count.data_ptr(),
           ws.data_ptr(), ws.numel() * ws.element_size()), "lp_top_logprobs")
    if check:
        _raise_bad(count, bad_rows, "have a NaN or infinite logit, or no finite one")
    return ids, values, logprobs


def _teacher(logits, ids, teacher, v_true):
    n, columns, vt, ld, code = _rows("logits", logits, v_true)
    dev = logits.device
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("expected ids [T, K]")
    K = ids.shape[1]
    if not 1 <= K <= DISTILL_MAX_K:
        raise ValueError(f"K must lie in [1, {DISTILL_MAX_K}]")
    pi = _like("ids", ids, (n, K), torch.int64, dev)
    pt = _like("teacher", teacher, (n, K), torch.float32, dev)
    return n, columns, vt, ld, code, K, pi, pt, dev


def _out_grad(logits, out, dev):
    """The gradient's buffer and its row stride."""
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        return out, out.shape[1]
    if not isinstance(out, torch.Tensor) or out.device != dev or out.dtype != logits.dtype or \
            out.shape != logits.shape:
        raise ValueError("out must have the logits' shape, dtype and device")
    if out.requires_grad:
        raise ValueError("out must not require gradients")
    _, _, _, ld, _ = _rows("out", out, None)
    if out.data_ptr() == logits.data_ptr():
        if out.shape[0] > 1 and out.stride(0) != logits.stride(0):
            raise ValueError("out on the logits' own buffer needs their row stride")
    elif out.numel():
        a, b = logits.data_ptr(), out.data_ptr()
        size = logits.element_size()
        extent = lambda t: ((t.shape[0] - 1) * t.stride(0) + t.shape[1]) * size  # noqa: E731
        if a < b + extent(out) and b < a + extent(logits):
            raise ValueError("out must be the logits' own buffer or apart from it")
    torch.autograd.graph.increment_version(out)
    return out, ld


def distill_forward(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor,
                    temperature: float = 1.0, renormalize: bool = True,
                    v_true: int | None = None, *, workspace: torch.Tensor | None = None,
                    bad_rows: torch.Tensor | None = None, check: bool = False):
    """Loss against a teacher's top logits, without autograd (lp_distill_forward).

    ids [T, K] int64 (-1: absent) and teacher [T, K] fp32: the teacher's
    logits, renormalised over the row's entries at `temperature`, or with
    renormalize=False its logprobs, taken as they are. Returns (loss fp32
    [T], row_state [T, 4] fp64 for distill_backward). With check=True the call
    synchronises and raises ValueError if an id lies outside the vocabulary.
    """
    n, _, vt, ld, code, K, pi, pt, dev = _teacher(logits, ids, teacher, v_true)
    loss = torch.empty(n, dtype=torch.float32, device=dev)
    state = torch.empty((n, 4), dtype=torch.float64, device=dev)
    L = lib()
    ws = _workspace(workspace, L.lp_distill_workspace_bytes(n, vt, code), dev)
    count = _bad_rows(bad_rows, check, dev)
    _call(L.lp_distill_forward, dev,
          (logits.data_ptr(), ld, code, n, vt, pi, pt, K, float(temperature),
           0 if renormalize else DISTILL_LOGPROBS, loss.data_ptr(), state.data_ptr(),
           None if count is None else count.data_ptr(), ws.data_ptr(),
           ws.numel() * ws.element_size()), "lp_distill_forward")
    if check:
        _raise_bad(count, bad_rows, f"have a teacher id outside [0, {vt})")
    return loss, state


def distill_backward(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor,
                     row_state: torch.Tensor, grad_loss: torch.Tensor, temperature: float = 1.0,
                     renormalize: bool = True, v_true: int | None = None, *,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of the logits [T, columns] (lp_distill_backward) for grad_loss
    [T] fp32, from distill_forward's row_state and the same inputs. `out` may
    be the logits themselves: they are then overwritten."""
    n, columns, vt, ld, code, K, pi, pt, dev = _teacher(logits, ids, teacher, v_true)
    ps = _like("row_state", row_state, (n, 4), torch.float64, dev)
    pg = _like("grad_loss", grad_loss, (n,), torch.float32, dev)
    out, ldg = _out_grad(logits, out, dev)
    _call(lib().lp_distill_backward, dev,
          (logits.data_ptr(), ld, code, n, vt, columns, pi, pt, K, float(temperature),
           0 if renormalize else DISTILL_LOGPROBS, ps, pg, out.data_ptr(), ldg),
          "lp_distill_backward")
    return out


def distill_step(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor,
                 weight: torch.Tensor, temperature: float = 1.0, renormalize: bool = True,
                 v_true: int | None = None, *, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, bad_rows: torch.Tensor | None = None,
                 check: bool = False):
    """Loss [T] and gradient of sum(weight * loss) with respect to the logits,
    in one call (lp_distill_step): for a training step whose row weights
    (mask / number of tokens) are known beforehand. The same bits as
    distill_forward and distill_backward. `out` may be the logits themselves."""
    n, columns, vt, ld, code, K, pi, pt, dev = _teacher(logits, ids, teacher, v_true)
    pw = _like("weight", weight, (n,), torch.float32, dev)
    out, ldg = _out_grad(logits, out, dev)
    loss = torch.empty(n, dtype=torch.float32, device=dev)
    L = lib()
    ws = _workspace(workspace, L.lp_distill_workspace_bytes(n, vt, code), dev)
    count = _bad_rows(bad_rows, check, dev)
    _call(L.lp_distill_step, dev,
          (logits.data_ptr(), ld, code, n, vt, columns, pi, pt, K, float(temperature),
           0 if renormalize else DISTILL_LOGPROBS, pw, loss.data_ptr(), out.data_ptr(), ldg,
           None if count is None else count.data_ptr(), ws.data_ptr(),
           ws.numel() * ws.element_size()), "lp_distill_step")
    if check:
        _raise_bad(count, bad_rows, f"have a teacher id outside [0, {vt})")
    return loss, out


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, temperature, renormalize, v_true):
        loss, state = distill_forward(logits, ids, teacher, temperature, renormalize, v_true)
        ctx.save_for_backward(logits, ids, teacher, state)
        ctx.how = (temperature, renormalize, v_true)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss):
        logits, ids, teacher, state = ctx.saved_tensors
        grad = distill_backward(logits, ids, teacher, state, grad_loss.contiguous(), *ctx.how)
        return grad, None, None, None, None, None


def distill(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor,
            temperature: float = 1.0, renormalize: bool = True,
            v_true: int | None = None) -> torch.Tensor:
    """Distillation loss [T] fp32 against a teacher's top logits, differentiable
    once in the logits (arguments as for distill_forward; rows without an
    entry have loss and gradient 0), in reverse mode: dual tensors of forward
    mode raise NotImplementedError. The teacher gets no gradient. To record
    a step into a HIP graph, record distill_forward and distill_backward, or
    distill_step: an autograd graph of the same leaves must not be alive
    while a backward pass is being captured."""
    if isinstance(teacher, torch.Tensor) and teacher.requires_grad:
        raise ValueError("teacher must not require gradients")
    for name, t in (("logits", logits), ("teacher", teacher)):
        # (A dual tensor need not require gradients, and would lose its tangent.)
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError(f"distill has no forward-mode derivative: {name} has a tangent")
    if logits.requires_grad and torch.is_grad_enabled():
        return _Distill.apply(logits, ids, teacher, temperature, renormalize, v_true)
    return distill_forward(logits, ids, teacher, temperature, renormalize, v_true)[0]
