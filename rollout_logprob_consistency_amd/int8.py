"""The LM head in 8-bit integers (include/liblp_int8.h) on AMD Instinct MI355X.

A thin binding like the rest of the package: it checks and marshals arguments,
and every arithmetic step runs in the library's kernels.

    quantize_int8(x)                                       -> codes [R, H], scale [R]
    logits_int8(x, x_scale, w, w_scale, dtype)             -> rows of logits [T, V]
    score_int8(x, x_scale, w, w_scale, ids, temperature)   -> logprob [T]

A matrix in 8 bits is int8 codes [rows, H] with unit column stride and one fp32
scale per row. The head's rows start at multiples of 16 bytes, as quantize_int8
lays them out, and its last one has room for whole groups of 16; hidden states may
lie anywhere. Outputs lie apart from the inputs and from each other. The results
carry no derivative. Scratch memory is allocated per call unless `workspace` is
given (a uint8 tensor of the library's *_workspace_bytes, 256-byte aligned); calls
that may overlap, captured graphs among them, must not share one. `bad_rows` (int32
[1]) is a counter that a call adds its bad rows to; with check=True a call raises
for its own rows only.
"""

from __future__ import annotations

import torch

from ._lib import INT8_MAX_HIDDEN, lib
from .logits import _DTYPES, _bad_rows, _call, _like, _raise_bad, _rows, _workspace

_BF16_LOGITS = 2  # LP_SCORE_BF16_LOGITS


def _codes(name: str, t: torch.Tensor):
    """Checks a matrix of codes; returns (rows, H, row stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != torch.int8:
        raise ValueError(f"{name} must be int8, got {t.dtype}")
    if t.dim() != 2 or t.shape[1] < 1:
        raise ValueError(f"expected {name} [rows, H]")
    rows, h = t.shape
    ld = t.stride(0) if rows > 1 else (h + 15) // 16 * 16
    if t.stride(1) != 1 and h > 1 or ld < h:
        raise ValueError(f"{name} needs unit column stride and rows that do not overlap")
    return rows, h, ld


def _aligned_codes(name: str, t: torch.Tensor):
    rows, h, ld = _codes(name, t)
    if ld % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name}'s rows must start at multiples of 16 bytes "
                         "(as quantize_int8 lays them out)")
    last = t.storage_offset() + (rows - 1) * ld + (h + 15) // 16 * 16
    if rows and t.untyped_storage().nbytes() < last:
        raise ValueError(f"{name} needs room for whole 16-byte groups in its last row")
    return rows, h, ld


def _extent(t: torch.Tensor, width: int | None = None) -> int:
    """Bytes from the first element's to the last one's end, of rows or of a
    contiguous vector; `width`: elements that a row takes."""
    if t.dim() == 2:
        return ((t.shape[0] - 1) * t.stride(0) + (width or t.shape[1])) * t.element_size()
    return t.numel() * t.element_size()


def _given(name: str, t, shape: tuple, device: torch.device) -> int:
    """Checks a given fp32 vector that a call writes; returns its address."""
    p = _like(name, t, shape, torch.float32, device)
    if t.requires_grad:
        raise ValueError(f"{name} must not require gradients")
    return p


def _apart(name: str, out: torch.Tensor, others: dict, width: int | None = None):
    """Refuses an output whose memory, from its first row to its last, reaches into
    what else the call reads or writes."""
    if not out.numel():
        return
    b = out.data_ptr()
    end = b + _extent(out, width)
    for other, t in others.items():
        if t.numel() and t.data_ptr() < end and b < t.data_ptr() + _extent(t):
            raise ValueError(f"{name} must lie apart from {other}")


def quantize_int8(x: torch.Tensor, *, out: torch.Tensor | None = None,
                  scale: torch.Tensor | None = None, bad_rows: torch.Tensor | None = None,
                  check: bool = False):
    """Rows in 8 bits (lp_quantize_int8): (codes int8 [R, H], scale fp32 [R]),
    scale = max |x| / 127 of the row (by fp32's reciprocal of 127) and codes the
    integers nearest to x / scale, ties to even.

    x [R, H] bf16, fp16 or fp32 with unit column stride and any row stride. The
    codes' rows start at multiples of 16 bytes; `out` (and `scale`) may be given
    in that layout, with room for whole 16-byte groups: what lies between H and
    the next multiple of 16 is set to zero. With check=True the call
    synchronises and raises ValueError if a row holds a NaN or an infinity (else
    its scale is NaN and its codes are 0).
    """
    r, h, _, ld, code = _rows("x", x, None)
    dev, h16 = x.device, (h + 15) // 16 * 16
    if out is None:
        out, ldq = torch.empty((r, h16), dtype=torch.int8, device=dev), h16
        if h != h16:
            out = out[:, :h]
    else:
        if not isinstance(out, torch.Tensor) or out.device != dev or tuple(out.shape) != (r, h):
            raise ValueError(f"out must be [{r}, {h}] on x's device")
        _, _, ldq = _aligned_codes("out", out)
        _apart("out", out, dict(x=x), h16)
        torch.autograd.graph.increment_version(out)
    if scale is None:
        scale = torch.empty(r, dtype=torch.float32, device=dev)
        ps = scale.data_ptr()
    else:
        ps = _given("scale", scale, (r,), dev)
        _apart("scale", scale, dict(x=x))
        _apart("out", out, dict(scale=scale), h16)
        torch.autograd.graph.increment_version(scale)
    count = _bad_rows(bad_rows, check, dev)
    _call(lib().lp_quantize_int8, dev,
          (x.data_ptr(), ld, code, r, h, out.data_ptr(), ldq, ps,
           None if count is None else count.data_ptr()), "lp_quantize_int8")
    if check:
        _raise_bad(count, bad_rows, "have a NaN or infinite element")
    return out, scale


def _operands(x, x_scale, w, w_scale):
    t, h, ldx = _codes("x", x)
    dev = x.device
    v, hw, ldw = _aligned_codes("w", w)
    if hw != h or w.device != dev:
        raise ValueError("x [T, H] and w [V, H] must have one H and lie on one device")
    if v < 1:
        raise ValueError("w must have a row")
    if h > INT8_MAX_HIDDEN:
        raise ValueError(f"H must be at most {INT8_MAX_HIDDEN}")
    px = _like("x_scale", x_scale, (t,), torch.float32, dev)
    pw = _like("w_scale", w_scale, (v,), torch.float32, dev)
    return t, h, v, dev, (x.data_ptr(), ldx, px, w.data_ptr(), ldw, pw)


def logits_int8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                dtype: torch.dtype = torch.bfloat16, *, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Rows of logits [T, V] from an 8-bit head (lp_logits_int8):
    x_scale[t] * w_scale[v] * sum_k x[t, k] w[v, k], the sum exact, in `dtype`
    (bfloat16, float16 or float32), for sample(), verify() and top_logprobs().

    x [T, H] and w [V, H] int8 codes with their scales (quantize_int8). `out`
    [T, V] may be rows of a wider buffer (a padded vocabulary's padding is left
    as it is); its dtype then is the logits'.
    """
    t, h, v, dev, ptrs = _operands(x, x_scale, w, w_scale)
    if out is None:
        code, ld = _DTYPES.get(dtype), v
        if code is None:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
        out = torch.empty((t, v), dtype=dtype, device=dev)
    else:
        if not isinstance(out, torch.Tensor) or out.device != dev or tuple(out.shape) != (t, v):
            raise ValueError(f"out must be [{t}, {v}] on x's device")
        if out.requires_grad:
            raise ValueError("out must not require gradients")
        _, _, _, ld, code = _rows("out", out, None)
        _apart("out", out, dict(x=x, x_scale=x_scale, w=w, w_scale=w_scale))
        torch.autograd.graph.increment_version(out)
    L = lib()
    ws = _workspace(workspace, L.lp_logits_int8_workspace_bytes(t, h), dev)
    _call(L.lp_logits_int8, dev,
          (*ptrs, t, h, v, out.data_ptr(), ld, code, ws.data_ptr(),
           ws.numel() * ws.element_size()), "lp_logits_int8")
    return out


def score_int8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
               ids: torch.Tensor, temperature: float = 1.0, v_true: int | None = None, *,
               bf16_logits: bool = False, out: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               bad_rows: torch.Tensor | None = None, check: bool = False) -> torch.Tensor:
    """Logprob [T] fp32 of the tokens ids [T] int64 under an 8-bit head
    (lp_score_int8): score() for the logits that logits_int8 gives in fp32, or
    with bf16_logits=True in bf16, without writing them. v_true: the head's rows
    from there on are padding. With check=True the call synchronises and raises
    ValueError if a target id lies outside [0, v_true); else its score is NaN."""
    t, h, v, dev, ptrs = _operands(x, x_scale, w, w_scale)
    vt = v if v_true is None else int(v_true)
    if not 1 <= vt <= v:
        raise ValueError(f"v_true must lie in [1, {v}]")
    pi = _like("ids", ids, (t,), torch.int64, dev)
    inputs = dict(x=x, x_scale=x_scale, w=w, w_scale=w_scale, ids=ids)
    if out is None:
        out = torch.empty(t, dtype=torch.float32, device=dev)
        po = out.data_ptr()
    else:
        po = _given("out", out, (t,), dev)
        _apart("out", out, inputs)
        torch.autograd.graph.increment_version(out)
    pl = None
    if lse is not None:
        pl = _given("lse", lse, (t,), dev)
        _apart("lse", lse, dict(inputs, out=out))
        torch.autograd.graph.increment_version(lse)
    L = lib()
    ws = _workspace(workspace, L.lp_score_int8_workspace_bytes(t, h, vt), dev)
    count = _bad_rows(bad_rows, check, dev)
    _call(L.lp_score_int8, dev,
          (*ptrs, pi, t, h, vt, float(temperature), _BF16_LOGITS if bf16_logits else 0, po, pl,
           None if count is None else count.data_ptr(), ws.data_ptr(),
           ws.numel() * ws.element_size()), "lp_score_int8")
    if check:
        _raise_bad(count, bad_rows, f"have a target id outside [0, {vt})")
    return out
