"""The operators around the recurrence, on torch tensors.

Each function checks its tensors, allocates its outputs and workspace with torch
and forwards to the library on the current stream of its tensors' device, which
need not be the current one; the arithmetic is in the HIP kernels.  See
include/replayssm.h for the definitions.

* ``short_conv_prompt`` / ``short_conv_step``: the short causal convolution in
  front of the recurrence, for packed prompts and for one token or T drafts.
* ``scan_prompt``: the Mamba-2 recurrence over packed prompts, into a state that
  the decode step continues from.
* ``delta_prompt``: the same for the Gated DeltaNet recurrence.
* ``gated_norm``: the gated group norm behind the recurrence.
* ``residual_norm``: the norm of the residual stream, with the addition before it;
  outputs in 8 bits with scales if asked.
* ``token_logprobs``: log probabilities of given tokens, entropy, the largest words.
* ``accept_drafts``: how many drafts to commit, and the token after them.

The kernels of a decode step take a few microseconds, so what Python adds to a
call counts: the checks are plain comparisons, and only a tensor that fails one
is looked at again to say what is wrong with it.
"""
from __future__ import annotations

import struct

import torch

from . import binding as B

_E4M3 = torch.float8_e4m3fn
_DT = {torch.float32: B.DT_F32, torch.bfloat16: B.DT_BF16}
_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
# The library's structs as bytes, in the order of their fields (native alignment).
_PROMPT = struct.Struct("@2i4P").pack
_CONV = struct.Struct("@10i5P").pack
_NORM = struct.Struct("@8ifi3q4P").pack
_ACCEPT = struct.Struct("@6i4q7P").pack
_STREAM = struct.Struct("@6ifi4q6P").pack
_LOGPROBS = struct.Struct("@4i2q6P").pack
_CONFIG = struct.Struct("@10iQ2I").pack
_RECORD = struct.Struct("@5P").pack
_raw_stream = torch._C._cuda_getCurrentRawStream  # of a device index, as an integer
_device = torch._C._cuda_getDevice  # the index of the current device


def _refuse(t, name, dtypes, shape, dense=True):
    """Raise what keeps t from being a device tensor of one of dtypes and of shape (None: any extent)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a device tensor of {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != len(shape) or any(w is not None and g != w for g, w in zip(t.shape, shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple('*' if w is None else w for w in shape)}")
    raise ValueError(f"{name} must be contiguous" if dense else f"{name} must be dense along its last axis")


def launch(call, at, *args):
    """call(*args, stream) with device `at`, the tensors', current: kernels go to the
    current device, and the default stream's handle is the same on every one."""
    if _device() == at:
        call(*args, _raw_stream(at))
    else:
        with torch.cuda.device(at):
            call(*args, _raw_stream(at))


def _check(t, name, dtype, shape, at):
    """t is a contiguous tensor of dtype and shape on device `at`; its address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == at:
            return t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != at:
        raise ValueError(f"tensors are on several devices: {name} is on {t.device}")
    _refuse(t, name, (dtype,), shape)


def _vectors(t, name, dims):
    """The first tensor of a call: float32 or bfloat16, dims axes, dense along the last; its device index."""
    if (not isinstance(t, torch.Tensor) or t.dtype not in _DT or not t.is_cuda or t.dim() != dims
            or (t.stride(-1) != 1 and t.shape[-1] > 1)):
        _refuse(t, name, tuple(_DT), (None,) * dims, False)
    return t.get_device()


def _prompt(tokens, seq_start, rows, resume, status, at) -> tuple[bytes, int]:
    if not isinstance(seq_start, torch.Tensor) or seq_start.dim() != 1 or seq_start.shape[0] < 2:
        raise ValueError("seq_start must be int32 [sequences + 1], on the device")
    n = seq_start.shape[0] - 1
    start = _check(seq_start, "seq_start", _I32, (n + 1,), at)
    if resume is not None:
        resume = _check(resume, "resume", torch.bool if resume.dtype is torch.bool else torch.uint8, (n,), at)
    return _PROMPT(tokens, n, start, _check(rows, "rows", _I32, (n,), at) if rows is not None else 0, resume or 0,
                   _status(status, at)), n


def _status(status, at) -> int:
    return 0 if status is None else _check(status, "status", _I32, tuple(status.shape), at)


def _short_conv(x, weight, ring, pos, widths, bias, activation, status, dims):
    at = _vectors(x, "x", dims)
    shape = x.shape
    C = shape[-1]
    parts = len(widths)
    w0, w1, w2 = (*widths, 0, 0)[:3] if 0 < parts < 3 else widths if parts == 3 else (-1, 0, 0)
    if w0 < 0 or w1 < 0 or w2 < 0 or w0 + w1 + w2 != C:
        raise ValueError(f"widths {tuple(widths)} must be one to three extents that add up to {C} channels")
    if activation not in ("silu", None):
        raise ValueError(f"unknown activation {activation!r}")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be float32 [channels, taps], on the device")
    if not isinstance(ring, torch.Tensor) or ring.dim() != 3:
        raise ValueError("ring must be [slots, batch, channels], on the device")
    taps = weight.shape[1]
    slots, batch, _ = ring.shape
    dtype = x.dtype
    conv = _CONV(C, taps, slots, batch, _DT[dtype], 1 if activation else 0, w0, w1, w2, 0,
                 _check(weight, "weight", _F32, (C, taps), at),
                 0 if bias is None else _check(bias, "bias", _F32, (C,), at),
                 _check(ring, "ring", dtype, (slots, batch, C), at),
                 0 if pos is None else _check(pos, "pos", _I32, (batch,), at),
                 0 if status is None else _status(status, at))
    empty = x.new_empty
    if dims == 3:
        n, T, _ = shape
        outs = [empty(n, T, w) for w in widths]
    else:
        n = shape[0]
        outs = [empty(n, w) for w in widths]
    to = [o.data_ptr() for o in outs]
    return at, conv, batch, outs, to if parts == 3 else (to + [0, 0])[:3]


def short_conv_step(x, weight, ring, pos, widths, *, bias=None, activation="silu", status=None):
    """The convolution for T tokens of every batch row: one decode token, or T drafts.

    x [batch, T, channels] float32 or bfloat16 (rows may be strided, e.g. a slice
    of the input projection); weight float32 [channels, taps]; ring [slots, batch,
    channels] in x's type, slots >= taps - 1 + T, updated in place; pos int32
    [batch], the position of the first token (``ReplayLayer.pointers()[0]``);
    widths: how the channels are split into outputs.  Returns one contiguous
    [batch, T, width] tensor for each width.  Rejected drafts need no restore:
    the next call at the smaller pos writes over them."""
    at, conv, batch, outs, to = _short_conv(x, weight, ring, pos, widths, bias, activation, status, 3)
    if pos is None or x.shape[0] != batch:
        raise ValueError(f"x has {x.shape[0]} rows, ring {batch}, and pos is needed")
    launch(B.replay_short_conv_step, at, conv, x.data_ptr(), x.stride(0), x.stride(1), x.shape[1], to)
    return outs


def short_conv_prompt(x, weight, ring, seq_start, widths, *, bias=None, activation="silu", rows=None, pos=None,
                      resume=None, status=None):
    """The convolution over packed prompts.

    x [tokens, channels], sequence i in rows seq_start[i]:seq_start[i + 1]
    (int32, on the device); rows int32 [sequences]: their batch rows (None: 0, 1,
    ...), all different; resume uint8 or bool [sequences]: continue from the ring's
    history (None: no sequence does); pos as for a step (None: 0).  The ring's rows
    are left so that a step at pos continues the sequence.  Returns one contiguous
    [tokens, width] tensor for each width; rows outside every sequence are not written."""
    at, conv, _, outs, to = _short_conv(x, weight, ring, pos, widths, bias, activation, status, 2)
    prompt, _ = _prompt(x.shape[0], seq_start, rows, resume, status, at)
    launch(B.replay_short_conv_prompt, at, conv, prompt, x.data_ptr(), x.stride(0), to)
    return outs


def scan_prompt(x, Bm, Cm, dt, A, D, seq_start, state, *, initial=None, rows=None, resume=None, out_dtype=None,
                status=None):
    """The Mamba-2 recurrence over packed prompts: y for every token of a sequence (other rows
    are not written), and the state after the last.

    x [tokens, heads, head_dim], Bm and Cm [tokens, groups, state_dim], all float32
    or all bfloat16; dt float32 [tokens, heads] (positive); A, D float32 [heads];
    seq_start, rows as for ``short_conv_prompt``; state float32 [batch, heads,
    head_dim, state_dim]: the sequences' rows are written, the others kept.
    initial (same shape, may be ``state`` itself): where sequences start, all of
    them or those with resume nonzero; None: from zero.  out_dtype: float32
    (default) or, with bfloat16 inputs, bfloat16."""
    at, args, y, _ = scan_call(x, Bm, Cm, dt, A, D, seq_start, state, initial, rows, resume, out_dtype, status)
    launch(B.replay_scan_prompt, at, *args)
    return y


def scan_call(x, Bm, Cm, dt, A, D, seq_start, state, initial, rows, resume, out_dtype, status):
    """scan_prompt up to its launch, which then refuses nothing: (device index, arguments, y, workspace)."""
    at = _vectors(x, "x", 3)
    tokens, H, P = x.shape
    dtype = x.dtype
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != 3:
        raise ValueError("Bm must be [tokens, groups, state_dim], on the device")
    G, N = Bm.shape[1:]
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be float32 [batch, heads, head_dim, state_dim], on the device")
    batch = state.shape[0]
    out_dtype = _F32 if out_dtype is None else out_dtype
    if out_dtype not in _DT:
        raise ValueError(f"out_dtype {out_dtype} is not float32 or bfloat16")
    if out_dtype is _BF16 and dtype is _F32:
        raise ValueError("bfloat16 outputs are for bfloat16 inputs")
    if initial is None and resume is not None:
        raise ValueError("resume needs initial")
    xs, Bs, Cs = (_check(x, "x", dtype, (tokens, H, P), at), _check(Bm, "Bm", dtype, (tokens, G, N), at),
                  _check(Cm, "Cm", dtype, (tokens, G, N), at))
    rec = _RECORD(xs, Bs, Cs, _check(dt, "dt", _F32, (tokens, H), at), 0)
    to = _check(state, "state", _F32, (batch, H, P, N), at)
    start = 0 if initial is None else to if initial is state else _check(initial, "initial", _F32, (batch, H, P, N), at)
    if tokens > 1 << 30 or H * P >= 1 << 23 or G * N >= 1 << 23:
        raise ValueError(f"{tokens} tokens of {H} x {P} and {G} x {N} values: at most 2^30, below 2^23 and below 2^23")
    if (xs | Bs | Cs | to | start) & 15:
        raise ValueError("x, Bm, Cm, state and initial must start at multiples of 16 bytes")
    prompt, n = _prompt(tokens, seq_start, rows, resume, status, at)
    cfg = _CONFIG(B.KIND_MAMBA2, batch, H, G, P, N, 1, 0, 0, 0, 0, B.FLAG_BF16_RECORDS if dtype is _BF16 else 0, 0)
    nbytes = B.replay_scan_workspace_bytes(cfg, tokens, n)
    y = x.new_empty(tokens, H, P, dtype=out_dtype)
    ws = x.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    args = (cfg, prompt, rec, _check(A, "A", _F32, (H,), at), _check(D, "D", _F32, (H,), at), start, to, y.data_ptr(),
            _DT[out_dtype], ws.data_ptr() if nbytes else 0)
    return at, args, y, ws


def delta_prompt(q, k, v, alpha, beta, seq_start, state, *, initial=None, rows=None, resume=None, out_dtype=None,
                 status=None):
    """The Gated DeltaNet recurrence over packed prompts: o for every token of a sequence (other
    rows are not written), and the state after the last.

    q, k [tokens, heads, state_dim] and v [tokens, heads, head_dim], all float32 or all
    bfloat16; alpha in [0, 1] and beta float32 [tokens, heads]; state float32 [batch,
    heads, head_dim, state_dim]; everything else as for ``scan_prompt``."""
    at, args, y, _ = delta_call(q, k, v, alpha, beta, seq_start, state, initial, rows, resume, out_dtype, status)
    launch(B.replay_delta_prompt, at, *args)
    return y


def delta_call(q, k, v, alpha, beta, seq_start, state, initial, rows, resume, out_dtype, status):
    """delta_prompt up to its launch, which then refuses nothing: (device index, arguments, y, workspace)."""
    at = _vectors(q, "q", 3)
    tokens, H, N = q.shape
    dtype = q.dtype
    if not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("v must be [tokens, heads, head_dim], on the device")
    P = v.shape[2]
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be float32 [batch, heads, head_dim, state_dim], on the device")
    batch = state.shape[0]
    out_dtype = _F32 if out_dtype is None else out_dtype
    if out_dtype not in _DT:
        raise ValueError(f"out_dtype {out_dtype} is not float32 or bfloat16")
    if out_dtype is _BF16 and dtype is _F32:
        raise ValueError("bfloat16 outputs are for bfloat16 inputs")
    if initial is None and resume is not None:
        raise ValueError("resume needs initial")
    qs, ks, vs = (_check(q, "q", dtype, (tokens, H, N), at), _check(k, "k", dtype, (tokens, H, N), at),
                  _check(v, "v", dtype, (tokens, H, P), at))
    rec = _RECORD(qs, ks, vs, _check(alpha, "alpha", _F32, (tokens, H), at), _check(beta, "beta", _F32, (tokens, H), at))
    to = _check(state, "state", _F32, (batch, H, P, N), at)
    start = 0 if initial is None else to if initial is state else _check(initial, "initial", _F32, (batch, H, P, N), at)
    if tokens > 1 << 30 or H * P >= 1 << 23 or H * N >= 1 << 23:
        raise ValueError(f"{tokens} tokens of {H} x {P} and {H} x {N} values: at most 2^30, below 2^23 and below 2^23")
    if (qs | ks | vs | to | start) & 15:
        raise ValueError("q, k, v, state and initial must start at multiples of 16 bytes")
    prompt, n = _prompt(tokens, seq_start, rows, resume, status, at)
    cfg = _CONFIG(B.KIND_GDN, batch, H, H, P, N, 1, 0, 0, 0, 0, B.FLAG_BF16_RECORDS if dtype is _BF16 else 0, 0)
    nbytes = B.replay_delta_workspace_bytes(cfg, tokens, n, _DT[out_dtype])
    y = v.new_empty(tokens, H, P, dtype=out_dtype)
    ws = q.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    return at, (cfg, prompt, rec, start, to, y.data_ptr(), _DT[out_dtype], ws.data_ptr() if nbytes else 0), y, ws


def gated_norm(y, z, weight, group, *, eps=1e-5, norm_first=False, out_dtype=None):
    """RMS norm over groups of ``group`` channels with the gate silu(z), per token.

    y, z [tokens, channels] float32 or bfloat16, rows may be strided; weight
    float32 [channels], or [group] shared by the groups.  norm_first False: the
    norm of y silu(z); True: the norm of y, then the gate.  out_dtype: z's type
    if None."""
    at = _vectors(y, "y", 2)
    if _vectors(z, "z", 2) != at:
        raise ValueError("tensors are on several devices")
    tokens, C = y.shape
    if z.shape != y.shape:
        raise ValueError(f"z has shape {tuple(z.shape)}, expected {tuple(y.shape)}")
    out_dtype = z.dtype if out_dtype is None else out_dtype
    if out_dtype not in _DT:
        raise ValueError(f"out_dtype {out_dtype} is not float32 or bfloat16")
    wn = weight.shape[0] if isinstance(weight, torch.Tensor) and weight.dim() == 1 else -1
    if group < 1 or C % group or (wn != C and wn != group):
        raise ValueError(f"group {group} must divide {C} channels, and weight be [{C}] or [{group}]")
    out = z.new_empty(tokens, C) if out_dtype is z.dtype else z.new_empty(tokens, C, dtype=out_dtype)
    launch(B.replay_gated_norm, at,
           _NORM(tokens, C, group, wn, _DT[y.dtype], _DT[z.dtype], _DT[out_dtype], 1 if norm_first else 0, eps, 0, y.stride(0),
                 z.stride(0), C, y.data_ptr(), z.data_ptr(), _check(weight, "weight", _F32, (wn,), at), out.data_ptr()))
    return out


def residual_norm(x, residual, weight, *, eps=1e-5, out_dtype=None, scale_group=None):
    """The residual stream's addition and the RMS norm over its channels, per token.

    x, residual [tokens, channels] float32 or bfloat16, rows may be strided; residual
    None: nothing is added; weight float32 [channels], or None: 1.  The norm is that of
    x + residual in float32.  Returns (out, total): total is x + residual in a new tensor of
    residual's type, or x itself without one; out has out_dtype (x's type if None).  With out_dtype
    torch.float8_e4m3fn it returns (codes, scales, total): scale_group channels (a power
    of two from 16 to 512, or all of them: None) share a scale, float32 [tokens,
    channels / scale_group], and code times scale is the value."""
    at = _vectors(x, "x", 2)
    tokens, C = x.shape
    out_dtype = x.dtype if out_dtype is None else out_dtype
    codes = out_dtype is _E4M3
    if not codes and out_dtype not in _DT:
        raise ValueError(f"out_dtype {out_dtype} is not float32, bfloat16 or float8_e4m3fn")
    if not codes and scale_group is not None:
        raise ValueError("scale_group is for float8_e4m3fn outputs")
    group = 0 if not codes else C if scale_group is None else scale_group
    if C < 1 or codes and (group < 1 or C % group or (group != C and group not in (16, 32, 64, 128, 256, 512))):
        raise ValueError(f"scale_group {group} must be all of {C} channels, or a power of two from 16 to 512 that divides them")
    rs, rt, stride, to, total = 0, 0, 0, 0, x
    if residual is not None:
        if _vectors(residual, "residual", 2) != at:
            raise ValueError(f"tensors are on several devices: residual is on {residual.device}")
        if residual.shape != x.shape:
            raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {tuple(x.shape)}")
        total = residual.new_empty(tokens, C)
        rs, rt, stride, to = residual.data_ptr(), _DT[residual.dtype], residual.stride(0), total.data_ptr()
    out = x.new_empty(tokens, C) if out_dtype is x.dtype else x.new_empty(tokens, C, dtype=out_dtype)
    scales = x.new_empty(tokens, C // group, dtype=_F32) if codes else None
    launch(B.replay_residual_norm, at,
           _STREAM(tokens, C, group, _DT[x.dtype], rt, B.DT_E4M3 if codes else _DT[out_dtype], eps, 0, x.stride(0), stride, C, C,
                   x.data_ptr(), rs, 0 if weight is None else _check(weight, "weight", _F32, (C,), at), out.data_ptr(),
                   scales.data_ptr() if codes else 0, to))
    return (out, scales, total) if codes else (out, total)


def token_logprobs(logits, tokens, *, top=0):
    """What logits say of given tokens: softmax probabilities of each row, in natural logarithms.

    logits [rows, vocab] float32 or bfloat16, rows may be strided; tokens int32 [rows];
    top: 0 to 32 alternatives.  Returns (logprobs, entropy, top_logprobs, top_tokens): float32
    [rows], float32 [rows], float32 and int32 [rows, top], the largest words first and of
    equal ones the lower.  -inf and NaN have no weight: such a word, or a token outside the
    vocabulary, has -inf, and missing alternatives are -inf and -1."""
    at = _vectors(logits, "logits", 2)
    rows, V = logits.shape
    if V < 1 or not 0 <= top <= B.MAX_TOP:
        raise ValueError(f"token_logprobs needs a vocabulary, and top from 0 to {B.MAX_TOP}")
    words = _check(tokens, "tokens", _I32, (rows,), at)
    logprobs, entropy = logits.new_empty(rows, dtype=_F32), logits.new_empty(rows, dtype=_F32)
    best, which = logits.new_empty(rows, top, dtype=_F32), tokens.new_empty(rows, top)
    if rows:
        nbytes = B.replay_token_logprobs_workspace_bytes(rows, V, top)
        ws = logits.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
        launch(B.replay_token_logprobs, at,
               _LOGPROBS(rows, V, top, _DT[logits.dtype], logits.stride(0), 0, logits.data_ptr(), words, logprobs.data_ptr(),
                         entropy.data_ptr(), best.data_ptr(), which.data_ptr()), ws.data_ptr() if nbytes else 0)
    return logprobs, entropy, best, which


def accept_drafts(tokens, target, uniforms, *, draft=None, lengths=None):
    """How many drafts of each sequence are kept, and the token that follows them.

    tokens int32 [batch, T]; target [batch, T + 1, vocab]: the target's
    probabilities after each prefix; draft [batch, T, vocab]: those the drafts
    were drawn from (None: the drafts were certain); both float32 or bfloat16,
    dense along vocab, the other strides free; uniforms float32 [batch, T + 1] in
    [0, 1): T acceptance numbers and the sampling number; lengths int32 [batch]:
    drafts of each sequence (None: T).  Returns (accepted, next), int32 [batch];
    accepted goes to ``ReplayLayer.commit``."""
    at = _vectors(target, "target", 3)
    batch, T, V = target.shape
    T -= 1
    if batch < 1 or V < 1 or T < 0:
        raise ValueError("accept_drafts needs a sequence, a row of probabilities and a vocabulary")
    ds, q, qt = (0, 0), 0, 0
    if draft is not None:
        if _vectors(draft, "draft", 3) != at or draft.shape != (batch, T, V):
            _refuse(draft, "draft", tuple(_DT), (batch, T, V))
        ds, q, qt = draft.stride(), draft.data_ptr(), _DT[draft.dtype]
    ts = target.stride()
    drafts = _check(tokens, "tokens", _I32, (batch, T), at)
    accepted, following = tokens.new_empty(batch), tokens.new_empty(batch)
    ws = target.new_empty(B.replay_accept_workspace_bytes(batch, V), dtype=torch.uint8)
    args = _ACCEPT(batch, T, V, _DT[target.dtype], qt, 0, ts[0], ts[1], ds[0], ds[1],
                   drafts, 0 if lengths is None else _check(lengths, "lengths", _I32, (batch,), at), target.data_ptr(), q,
                   _check(uniforms, "uniforms", _F32, (batch, T + 1), at), accepted.data_ptr(), following.data_ptr())
    launch(B.replay_accept_drafts, at, args, ws.data_ptr())
    return accepted, following
