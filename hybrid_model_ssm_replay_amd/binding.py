"""ctypes mirror of include/replayssm.h.  Argument marshalling only.

Every function here takes plain integers (device addresses, sizes, a
hipStream_t handle) and calls the C function of the same name; a negative
return code raises ``ReplayError``.
"""
from __future__ import annotations

import ctypes
import os

KIND_MAMBA2, KIND_GDN = 0, 1
FMT_F32, FMT_F16_SR, FMT_F8E4M3, FMT_F4E2M1_B16, FMT_F4E2M1_CS = 0, 1, 2, 3, 4
STATUS_ACCEPT_CLAMPED, STATUS_BAD_POINTERS, STATUS_BAD_PROMPT = 0x1, 0x2, 0x4
DT_F32, DT_BF16, DT_E4M3 = 0, 1, 2
MAX_TOP = 32
FLAG_DECAY_SKIP = 0x1
FLAG_BF16_RECORDS = 0x2
FLAG_RECORDS_IN_RING = 0x4
OK, EINVAL, EHIP, ENOTSUP = 0, -1, -2, -3

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "libreplayssm.so")


class ReplayError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({_strerror(code)})")
        self.code = code


class replay_config(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("batch", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("state_dim", ctypes.c_int32),
                ("window", ctypes.c_int32), ("max_draft", ctypes.c_int32), ("ckpt_fmt", ctypes.c_int32),
                ("read_fmt", ctypes.c_int32), ("seed", ctypes.c_uint64), ("flags", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class replay_buffers(ctypes.Structure):
    _fields_ = [("ckpt", ctypes.c_void_p), ("read_copy", ctypes.c_void_p), ("ring", ctypes.c_void_p),
                ("pointers", ctypes.c_void_p), ("status", ctypes.c_void_p), ("A", ctypes.c_void_p),
                ("D", ctypes.c_void_p)]


class replay_record(ctypes.Structure):
    _fields_ = [("f0", ctypes.c_void_p), ("f1", ctypes.c_void_p), ("f2", ctypes.c_void_p),
                ("f3", ctypes.c_void_p), ("f4", ctypes.c_void_p)]


class replay_ring_view(ctypes.Structure):
    _fields_ = [("f", ctypes.c_void_p * 5), ("slots", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class replay_ctx(ctypes.Structure):
    _fields_ = [("cfg", replay_config), ("buf", replay_buffers), ("parity", ctypes.c_int32),
                ("t_pending", ctypes.c_int32), ("magic", ctypes.c_uint32), ("reserved", ctypes.c_int32)]


class replay_prompt(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("sequences", ctypes.c_int32), ("seq_start", ctypes.c_void_p),
                ("rows", ctypes.c_void_p), ("resume", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class replay_short_conv(ctypes.Structure):
    _fields_ = [("channels", ctypes.c_int32), ("taps", ctypes.c_int32), ("slots", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("dtype", ctypes.c_int32), ("silu", ctypes.c_int32),
                ("width", ctypes.c_int32 * 3), ("reserved", ctypes.c_int32), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("ring", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class replay_gated_norm_args(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("channels", ctypes.c_int32), ("group", ctypes.c_int32),
                ("weight_len", ctypes.c_int32), ("y_dtype", ctypes.c_int32), ("z_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("norm_first", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("y_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("y", ctypes.c_void_p), ("z", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class replay_accept_args(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("drafts", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("target_dtype", ctypes.c_int32), ("draft_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("target_seq_stride", ctypes.c_int64), ("target_row_stride", ctypes.c_int64),
                ("draft_seq_stride", ctypes.c_int64), ("draft_row_stride", ctypes.c_int64),
                ("tokens", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("target", ctypes.c_void_p),
                ("draft", ctypes.c_void_p), ("uniforms", ctypes.c_void_p), ("accepted", ctypes.c_void_p),
                ("next", ctypes.c_void_p)]


class replay_residual_norm_args(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("channels", ctypes.c_int32), ("group", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("residual_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32), ("x_stride", ctypes.c_int64),
                ("residual_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64), ("sum_stride", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("sum", ctypes.c_void_p)]


class replay_token_logprobs_args(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("vocab", ctypes.c_int32), ("top", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("stride", ctypes.c_int64), ("reserved", ctypes.c_int64), ("logits", ctypes.c_void_p),
                ("tokens", ctypes.c_void_p), ("logprobs", ctypes.c_void_p), ("entropy", ctypes.c_void_p),
                ("top_logprobs", ctypes.c_void_p), ("top_tokens", ctypes.c_void_p)]


class replay_scan_layout(ctypes.Structure):
    _fields_ = [("segment", ctypes.c_int32), ("adds", ctypes.c_int32), ("columns", ctypes.c_int32),
                ("workgroups", ctypes.c_int32)]


_lib = None

_P = ctypes.c_void_p
_SIG = {
    "replay_validate_config": (ctypes.c_int, [ctypes.POINTER(replay_config)]),
    "replay_ckpt_bytes": (ctypes.c_size_t, [ctypes.POINTER(replay_config)]),
    "replay_read_copy_bytes": (ctypes.c_size_t, [ctypes.POINTER(replay_config)]),
    "replay_ring_bytes": (ctypes.c_size_t, [ctypes.POINTER(replay_config)]),
    "replay_pointer_words": (ctypes.c_size_t, [ctypes.POINTER(replay_config)]),
    "replay_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "replay_abi_sizeof": (ctypes.c_size_t, [ctypes.c_int]),
    "replay_init": (ctypes.c_int, [ctypes.POINTER(replay_ctx), ctypes.POINTER(replay_config),
                                   ctypes.POINTER(replay_buffers), _P]),
    "replay_set_state": (ctypes.c_int, [ctypes.POINTER(replay_ctx), _P, _P]),
    "replay_renew_read_copy": (ctypes.c_int, [ctypes.POINTER(replay_ctx), _P, _P]),
    "replay_step": (ctypes.c_int, [ctypes.POINTER(replay_ctx), ctypes.POINTER(replay_record), _P, _P]),
    "replay_flush": (ctypes.c_int, [ctypes.POINTER(replay_ctx), _P, _P]),
    "replay_verify": (ctypes.c_int, [ctypes.POINTER(replay_ctx), ctypes.c_int32, ctypes.POINTER(replay_record),
                                     _P, _P]),
    "replay_commit": (ctypes.c_int, [ctypes.POINTER(replay_ctx), _P, _P]),
    "replay_current_pointers": (ctypes.c_int, [ctypes.POINTER(replay_ctx), ctypes.POINTER(ctypes.c_void_p),
                                               ctypes.POINTER(ctypes.c_void_p)]),
    "replay_ring_fields": (ctypes.c_int, [ctypes.POINTER(replay_ctx), ctypes.POINTER(replay_ring_view)]),
    "replay_record_slots": (ctypes.c_int, [ctypes.POINTER(replay_ctx), _P, _P]),
    "replay_conv_step": (ctypes.c_int, [ctypes.POINTER(replay_config), _P, _P, _P, ctypes.POINTER(replay_record),
                                        _P, _P]),
    "replay_snapshot_verify": (ctypes.c_int, [ctypes.POINTER(replay_config), _P, _P, ctypes.c_int32, _P, _P,
                                              ctypes.POINTER(replay_record), _P, _P]),
    "replay_snapshot_commit": (ctypes.c_int, [ctypes.POINTER(replay_config), _P, _P, ctypes.c_int32, _P]),
    # The operators around the recurrence take their structs by address: a ctypes
    # structure, or the same bytes packed (a third of the time to make).
    "replay_short_conv_step": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, _P, _P, _P, _P]),
    "replay_short_conv_prompt": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, _P, _P, _P, _P]),
    "replay_scan_workspace_bytes": (ctypes.c_size_t, [_P, ctypes.c_int32, ctypes.c_int32]),
    "replay_scan_plan": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(replay_scan_layout)]),
    "replay_scan_prompt": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _P]),
    "replay_delta_workspace_bytes": (ctypes.c_size_t, [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]),
    "replay_delta_prompt": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _P]),
    "replay_gated_norm": (ctypes.c_int, [_P, _P]),
    "replay_residual_norm": (ctypes.c_int, [_P, _P]),
    "replay_token_logprobs_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32] * 3),
    "replay_token_logprobs": (ctypes.c_int, [_P, _P, _P]),
    "replay_accept_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "replay_accept_drafts": (ctypes.c_int, [_P, _P, _P]),
    "replay_hbm_probe": (ctypes.c_int, [_P, _P, ctypes.c_size_t, ctypes.c_int, _P]),
}
EXPORTS = tuple(_SIG)


def load_library(path: str | None = None):
    """Load libreplayssm.so (once) and check that the struct sizes agree."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or lib_path()
    # The library must bind to the HIP runtime that PyTorch (which owns the
    # device memory and streams) has loaded; load torch first if it is present.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(p):
        raise ImportError(f"{p} is not built; run `python -m hybrid_model_ssm_replay_amd.build`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIG.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    for i, st in enumerate((replay_config, replay_buffers, replay_record, replay_ctx, replay_ring_view, replay_prompt,
                            replay_short_conv, replay_gated_norm_args, replay_accept_args, replay_scan_layout,
                            replay_residual_norm_args, replay_token_logprobs_args)):
        if lib.replay_abi_sizeof(i) != ctypes.sizeof(st):
            raise ImportError(f"ABI mismatch for {st.__name__}: C {lib.replay_abi_sizeof(i)} "
                              f"vs ctypes {ctypes.sizeof(st)}")
    _lib = lib
    return lib


def _strerror(code: int) -> str:
    try:
        return load_library().replay_strerror(code).decode()
    except Exception:
        return "?"


def _check(fn: str, rc: int) -> None:
    if rc != OK:
        raise ReplayError(fn, rc)


def make_config(kind, batch, heads, groups, head_dim, state_dim, window, max_draft=0,
                ckpt_fmt=FMT_F32, read_fmt=FMT_F32, seed=0, flags=0) -> replay_config:
    return replay_config(kind, batch, heads, groups, head_dim, state_dim, window, max_draft, ckpt_fmt,
                         read_fmt, seed, flags, 0)


def make_record(*fields) -> replay_record:
    vals = list(fields) + [0] * (5 - len(fields))
    return replay_record(*[ctypes.c_void_p(v or None) for v in vals])


# ---- one wrapper per C call -------------------------------------------------
def replay_validate_config(cfg: replay_config) -> int:
    return load_library().replay_validate_config(ctypes.byref(cfg))


def replay_ckpt_bytes(cfg) -> int:
    return load_library().replay_ckpt_bytes(ctypes.byref(cfg))


def replay_read_copy_bytes(cfg) -> int:
    return load_library().replay_read_copy_bytes(ctypes.byref(cfg))


def replay_ring_bytes(cfg) -> int:
    return load_library().replay_ring_bytes(ctypes.byref(cfg))


def replay_pointer_words(cfg) -> int:
    return load_library().replay_pointer_words(ctypes.byref(cfg))


def replay_init(ctx: replay_ctx, cfg: replay_config, buf: replay_buffers, stream: int) -> None:
    _check("replay_init", load_library().replay_init(ctypes.byref(ctx), ctypes.byref(cfg), ctypes.byref(buf),
                                                     stream or None))


def replay_set_state(ctx, state: int, stream: int) -> None:
    _check("replay_set_state", load_library().replay_set_state(ctypes.byref(ctx), state, stream or None))


def replay_renew_read_copy(ctx, mask: int | None, stream: int) -> None:
    _check("replay_renew_read_copy", load_library().replay_renew_read_copy(ctypes.byref(ctx), mask or None, stream or None))


def replay_step(ctx, rec: replay_record, y: int, stream: int) -> None:
    _check("replay_step", load_library().replay_step(ctypes.byref(ctx), ctypes.byref(rec), y, stream or None))


def replay_flush(ctx, seq_mask: int, stream: int) -> None:
    _check("replay_flush", load_library().replay_flush(ctypes.byref(ctx), seq_mask or None, stream or None))


def replay_verify(ctx, T: int, drafts: replay_record, y: int, stream: int) -> None:
    _check("replay_verify", load_library().replay_verify(ctypes.byref(ctx), T, ctypes.byref(drafts), y,
                                                         stream or None))


def replay_commit(ctx, accepted: int, stream: int) -> None:
    _check("replay_commit", load_library().replay_commit(ctypes.byref(ctx), accepted, stream or None))


def replay_current_pointers(ctx) -> tuple[int, int]:
    pos, ck = ctypes.c_void_p(), ctypes.c_void_p()
    _check("replay_current_pointers",
           load_library().replay_current_pointers(ctypes.byref(ctx), ctypes.byref(pos), ctypes.byref(ck)))
    return pos.value, ck.value


def replay_ring_fields(ctx) -> replay_ring_view:
    view = replay_ring_view()
    _check("replay_ring_fields", load_library().replay_ring_fields(ctypes.byref(ctx), ctypes.byref(view)))
    return view


def replay_record_slots(ctx, slots: int, stream: int) -> None:
    _check("replay_record_slots", load_library().replay_record_slots(ctypes.byref(ctx), slots, stream))


def replay_conv_step(cfg, state: int, A: int, D: int, rec: replay_record, y: int, stream: int) -> None:
    _check("replay_conv_step", load_library().replay_conv_step(ctypes.byref(cfg), state, A or None, D or None,
                                                               ctypes.byref(rec), y, stream or None))


def replay_snapshot_verify(cfg, slots: int, cur: int, T: int, A: int, D: int, drafts: replay_record, y: int,
                           stream: int) -> None:
    _check("replay_snapshot_verify",
           load_library().replay_snapshot_verify(ctypes.byref(cfg), slots, cur, T, A or None, D or None,
                                                 ctypes.byref(drafts), y, stream or None))


def replay_snapshot_commit(cfg, cur: int, accepted: int, T: int, stream: int) -> None:
    _check("replay_snapshot_commit",
           load_library().replay_snapshot_commit(ctypes.byref(cfg), cur, accepted, T, stream or None))


def replay_hbm_probe(src: int, dst: int, nbytes: int, mode: int, stream: int) -> None:
    _check("replay_hbm_probe", load_library().replay_hbm_probe(src, dst, nbytes, mode, stream or None))


def _by_address(st):
    return st if isinstance(st, bytes) else ctypes.byref(st)


def replay_short_conv_step(conv, x: int, seq_stride: int, row_stride: int, T: int, outs, stream: int) -> None:
    rc = (_lib or load_library()).replay_short_conv_step(_by_address(conv), x, seq_stride, row_stride, T, *outs, stream)
    if rc:
        _check("replay_short_conv_step", rc)


def replay_short_conv_prompt(conv, prompt, x: int, row_stride: int, outs, stream: int) -> None:
    rc = (_lib or load_library()).replay_short_conv_prompt(_by_address(conv), _by_address(prompt), x, row_stride, *outs,
                                                           stream)
    if rc:
        _check("replay_short_conv_prompt", rc)


def replay_scan_workspace_bytes(cfg, tokens: int, sequences: int) -> int:
    return (_lib or load_library()).replay_scan_workspace_bytes(_by_address(cfg), tokens, sequences)


def replay_scan_plan(cfg, tokens: int, sequences: int) -> replay_scan_layout:
    layout = replay_scan_layout()
    _check("replay_scan_plan", load_library().replay_scan_plan(_by_address(cfg), tokens, sequences, ctypes.byref(layout)))
    return layout


def replay_scan_prompt(cfg, prompt, rec, A: int, D: int, initial: int, state: int, y: int, y_dtype: int, workspace: int,
                       stream: int) -> None:
    rc = (_lib or load_library()).replay_scan_prompt(_by_address(cfg), _by_address(prompt), _by_address(rec), A, D,
                                                     initial, state, y, y_dtype, workspace, stream)
    if rc:
        _check("replay_scan_prompt", rc)


def replay_delta_workspace_bytes(cfg, tokens: int, sequences: int, y_dtype: int) -> int:
    return (_lib or load_library()).replay_delta_workspace_bytes(_by_address(cfg), tokens, sequences, y_dtype)


def replay_delta_prompt(cfg, prompt, rec, initial: int, state: int, y: int, y_dtype: int, workspace: int, stream: int) -> None:
    rc = (_lib or load_library()).replay_delta_prompt(_by_address(cfg), _by_address(prompt), _by_address(rec), initial, state,
                                                      y, y_dtype, workspace, stream)
    if rc:
        _check("replay_delta_prompt", rc)


def replay_gated_norm(args, stream: int) -> None:
    rc = (_lib or load_library()).replay_gated_norm(_by_address(args), stream)
    if rc:
        _check("replay_gated_norm", rc)


def replay_residual_norm(args, stream: int) -> None:
    rc = (_lib or load_library()).replay_residual_norm(_by_address(args), stream)
    if rc:
        _check("replay_residual_norm", rc)


def replay_token_logprobs_workspace_bytes(rows: int, vocab: int, top: int) -> int:
    return (_lib or load_library()).replay_token_logprobs_workspace_bytes(rows, vocab, top)


def replay_token_logprobs(args, workspace: int, stream: int) -> None:
    rc = (_lib or load_library()).replay_token_logprobs(_by_address(args), workspace, stream)
    if rc:
        _check("replay_token_logprobs", rc)


def replay_accept_workspace_bytes(batch: int, vocab: int) -> int:
    return (_lib or load_library()).replay_accept_workspace_bytes(batch, vocab)


def replay_accept_drafts(args, workspace: int, stream: int) -> None:
    rc = (_lib or load_library()).replay_accept_drafts(_by_address(args), workspace, stream)
    if rc:
        _check("replay_accept_drafts", rc)
