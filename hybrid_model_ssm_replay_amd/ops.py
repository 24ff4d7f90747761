"""The operators around the recurrence, on torch tensors.

Each function checks its tensors, allocates its outputs and workspace with torch
and forwards to the library on the current stream; the arithmetic is in the HIP
kernels.  See include/replayssm.h for the definitions.

* ``short_conv_prompt`` / ``short_conv_step``: the short causal convolution in
  front of the recurrence, for packed prompts and for one token or T drafts.
* ``scan_prompt``: the Mamba-2 recurrence over packed prompts, into a state that
  the decode step continues from.
* ``gated_norm``: the gated group norm behind the recurrence.
* ``accept_drafts``: how many drafts to commit, and the token after them.
"""
from __future__ import annotations

import torch

from . import binding as B

_DT = {torch.float32: B.DT_F32, torch.bfloat16: B.DT_BF16}


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _on_gpu(t, name, dtypes, shape=None, contiguous=True) -> torch.Tensor:
    """t, if it is a device tensor of one of dtypes and of shape (None: any extent)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a device tensor of {' or '.join(str(d) for d in dtypes)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and (t.dim() != len(shape) or any(w is not None and g != w for g, w in zip(t.shape, shape))):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple('*' if w is None else w for w in shape)}")
    return t


def _rows_apart(t, name) -> None:
    """The last axis is dense; the others may have any (non-negative) stride."""
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be dense along its last axis")


def _same_device(*tensors) -> None:
    devices = {t.device for t in tensors if t is not None}
    if len(devices) > 1:
        raise ValueError(f"tensors are on several devices: {sorted(map(str, devices))}")


def _ptr(t) -> int:
    return t.data_ptr() if t is not None else 0


def _prompt(tokens, seq_start, rows, resume, status) -> B.replay_prompt:
    _on_gpu(seq_start, "seq_start", (torch.int32,), (None,))
    n = seq_start.shape[0] - 1
    if n < 1:
        raise ValueError("seq_start needs one entry more than there are sequences")
    if rows is not None:
        _on_gpu(rows, "rows", (torch.int32,), (n,))
    if resume is not None:
        _on_gpu(resume, "resume", (torch.uint8, torch.bool), (n,))
    if status is not None:
        _on_gpu(status, "status", (torch.int32,))
    return B.replay_prompt(tokens, n, seq_start.data_ptr(), _ptr(rows), _ptr(resume), _ptr(status))


def _short_conv(x, weight, ring, pos, widths, bias, activation, status):
    _on_gpu(x, "x", tuple(_DT), contiguous=False)
    _rows_apart(x, "x")
    C = x.shape[-1]
    widths = tuple(int(w) for w in widths)
    if not 1 <= len(widths) <= 3 or sum(widths) != C or min(widths) < 0:
        raise ValueError(f"widths {widths} must be one to three extents that add up to {C} channels")
    _on_gpu(weight, "weight", (torch.float32,), (C, None))
    _on_gpu(ring, "ring", (x.dtype,), (None, None, C))
    if bias is not None:
        _on_gpu(bias, "bias", (torch.float32,), (C,))
    if pos is not None:
        _on_gpu(pos, "pos", (torch.int32,), (ring.shape[1],))
    if status is not None:
        _on_gpu(status, "status", (torch.int32,))
    if activation not in ("silu", None):
        raise ValueError(f"unknown activation {activation!r}")
    _same_device(x, weight, ring, bias, pos, status)
    w3 = widths + (0,) * (3 - len(widths))
    conv = B.replay_short_conv(C, weight.shape[1], ring.shape[0], ring.shape[1], _DT[x.dtype],
                               1 if activation == "silu" else 0, w3, 0, weight.data_ptr(), _ptr(bias),
                               ring.data_ptr(), _ptr(pos), _ptr(status))
    outs = [torch.empty(x.shape[:-1] + (w,), dtype=x.dtype, device=x.device) for w in widths]
    return conv, outs


def short_conv_step(x, weight, ring, pos, widths, *, bias=None, activation="silu", status=None):
    """The convolution for T tokens of every batch row: one decode token, or T drafts.

    x [batch, T, channels] float32 or bfloat16 (rows may be strided, e.g. a slice
    of the input projection); weight float32 [channels, taps]; ring [slots, batch,
    channels] in x's type, slots >= taps - 1 + T, updated in place; pos int32
    [batch], the position of the first token (``ReplayLayer.pointers()[0]``);
    widths: how the channels are split into outputs.  Returns one contiguous
    [batch, T, width] tensor for each width.  Rejected drafts need no restore:
    the next call at the smaller pos writes over them."""
    if isinstance(x, torch.Tensor) and x.dim() != 3:
        raise ValueError("x must be [batch, T, channels]")
    conv, outs = _short_conv(x, weight, ring, pos, widths, bias, activation, status)
    if pos is None or x.shape[0] != ring.shape[1]:
        raise ValueError(f"x has {x.shape[0]} rows, ring {ring.shape[1]}, and pos is needed")
    B.replay_short_conv_step(conv, x.data_ptr(), x.stride(0), x.stride(1), x.shape[1],
                             [_ptr(o) for o in outs] + [0] * (3 - len(outs)), _stream(x))
    return outs


def short_conv_prompt(x, weight, ring, seq_start, widths, *, bias=None, activation="silu", rows=None, pos=None,
                      resume=None, status=None):
    """The convolution over packed prompts.

    x [tokens, channels], sequence i in rows seq_start[i]:seq_start[i + 1]
    (int32, on the device); rows int32 [sequences]: their batch rows (None: 0, 1,
    ...), all different; resume uint8 or bool [sequences]: continue from the ring's
    history (None: no sequence does); pos as for a step (None: 0).  The ring's rows
    are left so that a step at pos continues the sequence.  Returns one contiguous
    [tokens, width] tensor for each width."""
    if isinstance(x, torch.Tensor) and x.dim() != 2:
        raise ValueError("x must be [tokens, channels]")
    conv, outs = _short_conv(x, weight, ring, pos, widths, bias, activation, status)
    prompt = _prompt(x.shape[0], seq_start, rows, resume, status)
    _same_device(x, seq_start, rows, resume)
    B.replay_short_conv_prompt(conv, prompt, x.data_ptr(), x.stride(0), [_ptr(o) for o in outs] + [0] * (3 - len(outs)),
                               _stream(x))
    return outs


def scan_prompt(x, Bm, Cm, dt, A, D, seq_start, state, *, initial=None, rows=None, resume=None, out_dtype=None,
                status=None):
    """The Mamba-2 recurrence over packed prompts: y for every token, and the state after the last.

    x [tokens, heads, head_dim], Bm and Cm [tokens, groups, state_dim], all float32
    or all bfloat16; dt float32 [tokens, heads] (positive); A, D float32 [heads];
    seq_start, rows as for ``short_conv_prompt``; state float32 [batch, heads,
    head_dim, state_dim]: the sequences' rows are written, the others kept.
    initial (same shape, may be ``state`` itself): where sequences start, all of
    them or those with resume nonzero; None: from zero.  out_dtype: float32
    (default) or, with bfloat16 inputs, bfloat16."""
    _on_gpu(x, "x", tuple(_DT), (None, None, None))
    tokens, H, P = x.shape
    _on_gpu(Bm, "Bm", (x.dtype,), (tokens, None, None))
    G, N = Bm.shape[1:]
    _on_gpu(Cm, "Cm", (x.dtype,), (tokens, G, N))
    _on_gpu(dt, "dt", (torch.float32,), (tokens, H))
    _on_gpu(A, "A", (torch.float32,), (H,))
    _on_gpu(D, "D", (torch.float32,), (H,))
    _on_gpu(state, "state", (torch.float32,), (None, H, P, N))
    if initial is not None:
        _on_gpu(initial, "initial", (torch.float32,), tuple(state.shape))
    elif resume is not None:
        raise ValueError("resume needs initial")
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    if out_dtype not in _DT:
        raise ValueError(f"out_dtype {out_dtype} is not float32 or bfloat16")
    prompt = _prompt(tokens, seq_start, rows, resume, status)
    _same_device(x, Bm, Cm, dt, A, D, state, initial, seq_start, rows, resume, status)
    cfg = B.make_config(B.KIND_MAMBA2, state.shape[0], H, G, P, N, 1,
                        flags=B.FLAG_BF16_RECORDS if x.dtype == torch.bfloat16 else 0)
    y = torch.empty((tokens, H, P), dtype=out_dtype, device=x.device)
    nbytes = B.replay_scan_workspace_bytes(cfg, tokens, prompt.sequences)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
    rec = B.make_record(x.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), dt.data_ptr())
    B.replay_scan_prompt(cfg, prompt, rec, A.data_ptr(), D.data_ptr(), _ptr(initial), state.data_ptr(), y.data_ptr(),
                         _DT[out_dtype], _ptr(ws), _stream(x))
    return y


def gated_norm(y, z, weight, group, *, eps=1e-5, norm_first=False, out_dtype=None):
    """RMS norm over groups of ``group`` channels with the gate silu(z), per token.

    y, z [tokens, channels] float32 or bfloat16, rows may be strided; weight
    float32 [channels], or [group] shared by the groups.  norm_first False: the
    norm of y silu(z); True: the norm of y, then the gate.  out_dtype: z's type
    if None."""
    _on_gpu(y, "y", tuple(_DT), (None, None), contiguous=False)
    _on_gpu(z, "z", tuple(_DT), tuple(y.shape), contiguous=False)
    _rows_apart(y, "y")
    _rows_apart(z, "z")
    tokens, C = y.shape
    _on_gpu(weight, "weight", (torch.float32,), (None,))
    out_dtype = z.dtype if out_dtype is None else out_dtype
    if out_dtype not in _DT:
        raise ValueError(f"out_dtype {out_dtype} is not float32 or bfloat16")
    if group < 1 or C % group or weight.shape[0] not in (C, group):
        raise ValueError(f"group {group} must divide {C} channels, and weight has {weight.shape[0]} of {C} or {group} values")
    _same_device(y, z, weight)
    out = torch.empty((tokens, C), dtype=out_dtype, device=y.device)
    args = B.replay_gated_norm_args(tokens, C, group, weight.shape[0], _DT[y.dtype], _DT[z.dtype], _DT[out_dtype],
                                    1 if norm_first else 0, eps, 0, y.stride(0), z.stride(0), C, y.data_ptr(),
                                    z.data_ptr(), weight.data_ptr(), out.data_ptr())
    B.replay_gated_norm(args, _stream(y))
    return out


def accept_drafts(tokens, target, uniforms, *, draft=None, lengths=None):
    """How many drafts of each sequence are kept, and the token that follows them.

    tokens int32 [batch, T]; target [batch, T + 1, vocab]: the target's
    probabilities after each prefix; draft [batch, T, vocab]: those the drafts
    were drawn from (None: the drafts were certain); both float32 or bfloat16,
    dense along vocab, the other strides free; uniforms float32 [batch, T + 1] in
    [0, 1): T acceptance numbers and the sampling number; lengths int32 [batch]:
    drafts of each sequence (None: T).  Returns (accepted, next), int32 [batch];
    accepted goes to ``ReplayLayer.commit``."""
    _on_gpu(tokens, "tokens", (torch.int32,), (None, None))
    batch, T = tokens.shape
    _on_gpu(target, "target", tuple(_DT), (batch, T + 1, None), contiguous=False)
    V = target.shape[-1]
    _rows_apart(target, "target")
    if draft is not None:
        _on_gpu(draft, "draft", tuple(_DT), (batch, T, V), contiguous=False)
        _rows_apart(draft, "draft")
    _on_gpu(uniforms, "uniforms", (torch.float32,), (batch, T + 1))
    if lengths is not None:
        _on_gpu(lengths, "lengths", (torch.int32,), (batch,))
    if batch < 1 or V < 1:
        raise ValueError("accept_drafts needs a sequence and a vocabulary")
    _same_device(tokens, target, uniforms, draft, lengths)
    accepted, following = torch.empty((2, batch), dtype=torch.int32, device=tokens.device)
    ws = torch.empty(B.replay_accept_workspace_bytes(batch, V), dtype=torch.uint8, device=tokens.device)
    ds = (draft.stride(0), draft.stride(1)) if draft is not None else (0, 0)
    args = B.replay_accept_args(batch, T, V, _DT[target.dtype], _DT[draft.dtype] if draft is not None else 0, 0,
                                target.stride(0), target.stride(1), *ds, tokens.data_ptr(), _ptr(lengths),
                                target.data_ptr(), _ptr(draft), uniforms.data_ptr(), accepted.data_ptr(),
                                following.data_ptr())
    B.replay_accept_drafts(args, ws.data_ptr(), _stream(tokens))
    return accepted, following
