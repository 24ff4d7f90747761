"""What the operators around the recurrence refuse, before anything is enqueued (no GPU)."""
import pytest
import torch

P16 = 4096  # an address that is never followed: every call here is refused on the host


@pytest.fixture(scope="module")
def B():
    from hybrid_model_ssm_replay_amd import binding
    binding.load_library()
    return binding


def _refused(B, fn, code=None):
    with pytest.raises(B.ReplayError) as e:
        fn()
    assert e.value.code == (B.EINVAL if code is None else code)


def _conv(B, **kw):
    d = dict(channels=48, taps=4, slots=4, batch=2, dtype=B.DT_BF16, silu=1, width=(16, 16, 16), reserved=0, weight=P16,
             bias=0, ring=P16, pos=P16, status=0)
    d.update(kw)
    return B.replay_short_conv(*[d[n] for n, _ in B.replay_short_conv._fields_])


@pytest.mark.parametrize("bad", [
    dict(taps=1), dict(taps=5), dict(slots=2), dict(batch=0), dict(dtype=2), dict(silu=2), dict(width=(16, 16, 17)),
    dict(width=(-16, 48, 16)), dict(weight=0), dict(ring=0), dict(ring=P16 + 1), dict(weight=P16 + 4), dict(channels=0),
    dict(reserved=1)])
def test_short_conv_refuses(B, bad):
    c = _conv(B, **bad)
    p = B.replay_prompt(8, 1, P16, 0, 0, 0)
    _refused(B, lambda: B.replay_short_conv_step(c, P16, 48, 48, 1, [P16] * 3, 0))
    _refused(B, lambda: B.replay_short_conv_prompt(c, p, P16, 48, [P16] * 3, 0))


def test_short_conv_step_refuses_calls(B):
    c = _conv(B)
    _refused(B, lambda: B.replay_short_conv_step(c, 0, 48, 48, 1, [P16] * 3, 0))
    _refused(B, lambda: B.replay_short_conv_step(c, P16 + 1, 48, 48, 1, [P16] * 3, 0))
    _refused(B, lambda: B.replay_short_conv_step(c, P16, 48, 48, 2, [P16] * 3, 0))      # slots hold one token
    _refused(B, lambda: B.replay_short_conv_step(c, P16, 48, 48, 0, [P16] * 3, 0))
    _refused(B, lambda: B.replay_short_conv_step(c, P16, -48, 48, 1, [P16] * 3, 0))
    _refused(B, lambda: B.replay_short_conv_step(c, P16, 48, 48, 1, [P16, 0, P16], 0))
    _refused(B, lambda: B.replay_short_conv_step(_conv(B, pos=0), P16, 48, 48, 1, [P16] * 3, 0))


@pytest.mark.parametrize("prompt", [(-1, 1, P16), (8, 0, P16), (8, 3, P16), (8, 1, 0)])
def test_packed_prompts_refused(B, prompt):
    p = B.replay_prompt(*prompt, 0, 0, 0)
    _refused(B, lambda: B.replay_short_conv_prompt(_conv(B), p, P16, 48, [P16] * 3, 0))
    cfg = B.make_config(0, 2, 4, 2, 32, 64, 1)
    rec = B.make_record(P16, P16, P16, P16)
    _refused(B, lambda: B.replay_scan_prompt(cfg, p, rec, P16, P16, 0, P16, P16, B.DT_F32, P16, 0))


@pytest.mark.parametrize("cfg", [(1, 2, 4, 4, 64, 64, 1), (0, 0, 4, 2, 32, 64, 1), (0, 2, 4, 3, 32, 64, 1),
                                 (0, 2, 4, 2, 24, 64, 1), (0, 2, 4, 2, 144, 64, 1), (0, 2, 4, 2, 32, 48, 1)])
def test_scan_refuses_shapes(B, cfg):
    c = B.make_config(*cfg)
    assert B.replay_scan_workspace_bytes(c, 100, 1) == 0
    p = B.replay_prompt(8, 1, P16, 0, 0, 0)
    _refused(B, lambda: B.replay_scan_prompt(c, p, B.make_record(P16, P16, P16, P16), P16, P16, 0, P16, P16, B.DT_F32,
                                             P16, 0))


def test_scan_refuses_calls(B):
    c, p, rec = B.make_config(0, 2, 4, 2, 32, 64, 1), B.replay_prompt(8, 1, P16, 0, 0, 0), B.make_record(P16, P16, P16, P16)
    good = [c, p, rec, P16, P16, 0, P16, P16, B.DT_F32, P16, 0]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return lambda: B.replay_scan_prompt(*a)

    for i in (3, 4, 6, 7):
        _refused(B, with_(i, 0))
    for i in (5, 6, 7):
        _refused(B, with_(i, P16 + 4))
    _refused(B, with_(8, 2))
    _refused(B, with_(8, B.DT_BF16), B.ENOTSUP)  # bf16 outputs of float32 records
    for i in range(4):
        f = [P16] * 4
        f[i] = 0
        _refused(B, with_(2, B.make_record(*f)))


def test_gated_norm_refuses(B):
    good = dict(tokens=4, channels=64, group=16, weight_len=64, y_dtype=0, z_dtype=1, out_dtype=1, norm_first=0, eps=1e-5,
                reserved=0, y_stride=64, z_stride=64, out_stride=64, y=P16, z=P16, weight=P16, out=P16)
    for bad in (dict(tokens=-1), dict(group=0), dict(group=24), dict(weight_len=32), dict(y_dtype=3), dict(z_dtype=-1),
                dict(out_dtype=2), dict(norm_first=2), dict(eps=-1.0), dict(eps=float("nan")), dict(y=0), dict(z=0),
                dict(weight=0), dict(out=0), dict(y=P16 + 2), dict(z=P16 + 1), dict(y_stride=-1), dict(out_stride=63),
                dict(reserved=7)):
        a = B.replay_gated_norm_args(*[{**good, **bad}[n] for n, _ in B.replay_gated_norm_args._fields_])
        _refused(B, lambda: B.replay_gated_norm(a, 0))


def test_accept_refuses(B):
    good = dict(batch=2, drafts=3, vocab=100, target_dtype=0, draft_dtype=1, reserved=0, target_seq_stride=400,
                target_row_stride=100, draft_seq_stride=300, draft_row_stride=100, tokens=P16, lengths=0, target=P16,
                draft=P16, uniforms=P16, accepted=P16, next=P16)
    for bad in (dict(batch=0), dict(drafts=-1), dict(vocab=0), dict(target_dtype=5), dict(draft_dtype=5), dict(tokens=0),
                dict(target=0), dict(uniforms=0), dict(accepted=0), dict(next=0), dict(target=P16 + 2), dict(draft=P16 + 1),
                dict(target_row_stride=-1), dict(draft_seq_stride=-1), dict(reserved=1)):
        a = B.replay_accept_args(*[{**good, **bad}[n] for n, _ in B.replay_accept_args._fields_])
        _refused(B, lambda: B.replay_accept_drafts(a, P16, 0))
    a = B.replay_accept_args(*[good[n] for n, _ in B.replay_accept_args._fields_])
    _refused(B, lambda: B.replay_accept_drafts(a, 0, 0))
    _refused(B, lambda: B.replay_accept_drafts(a, P16 + 8, 0))
    assert B.replay_accept_workspace_bytes(0, 5) == 0 and B.replay_accept_workspace_bytes(2, 100) > 0


def test_python_wrappers_refuse_host_tensors(B):
    from hybrid_model_ssm_replay_amd import ops
    f, i = torch.zeros, torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.short_conv_step(f(2, 1, 8), f(8, 4), f(4, 2, 8), i, (8,))
    with pytest.raises(ValueError):
        ops.short_conv_prompt(f(5, 8), f(8, 4), f(4, 2, 8), i, (8,))
    with pytest.raises(ValueError):
        ops.scan_prompt(f(5, 2, 16), f(5, 1, 16), f(5, 1, 16), f(5, 2), f(2), f(2), i, f(2, 2, 16, 16))
    with pytest.raises(ValueError):
        ops.gated_norm(f(5, 8), f(5, 8), f(8), 4)
    with pytest.raises(ValueError):
        ops.accept_drafts(torch.zeros(1, 2, dtype=torch.int32), f(1, 3, 9), f(1, 3))


def test_extents_past_32_bit_indexes_are_refused(B):
    """2^30 tokens, sequences or words of a vocabulary is the most: offsets a little past it still fit."""
    most = 1 << 30
    for tokens, n in ((most + 1, 1), (5, most + 1)):
        p = B.replay_prompt(tokens, n, P16, 0, 0, 0)
        _refused(B, lambda: B.replay_short_conv_prompt(_conv(B, batch=n), p, P16, 48, [P16] * 3, 0))
        cfg = B.make_config(0, n, 1, 1, 16, 16, 1)
        _refused(B, lambda: B.replay_scan_prompt(cfg, p, B.make_record(P16, P16, P16, P16), P16, P16, 0, P16, P16, B.DT_F32, P16, 0))
        assert B.replay_scan_workspace_bytes(cfg, tokens, n) == 0
    assert B.replay_accept_workspace_bytes(1, most) > 0 and B.replay_accept_workspace_bytes(1, most + 1) == 0
    args = B.replay_accept_args(1, 1, most + 1, 0, 0, 0, 0, 0, 0, 0, P16, 0, P16, 0, P16, P16, P16)
    _refused(B, lambda: B.replay_accept_drafts(args, P16, 0))


def test_packed_structs_have_the_librarys_sizes(B):
    """The Python functions pass the structs as packed bytes: as long as the C ones, field by field as ctypes lays them out."""
    import ctypes
    import struct
    lib = B.load_library()
    codes = {ctypes.c_int32: "i", ctypes.c_uint32: "I", ctypes.c_int64: "q", ctypes.c_uint64: "Q", ctypes.c_float: "f",
             ctypes.c_void_p: "P", ctypes.POINTER(ctypes.c_float): "P", ctypes.c_int32 * 3: "3i"}
    from hybrid_model_ssm_replay_amd import ops
    for which, st, pack in ((5, B.replay_prompt, ops._PROMPT), (6, B.replay_short_conv, ops._CONV),
                            (7, B.replay_gated_norm_args, ops._NORM), (8, B.replay_accept_args, ops._ACCEPT),
                            (0, B.replay_config, ops._CONFIG), (2, B.replay_record, ops._RECORD)):
        fields = "@" + "".join(codes[t] for _, t in st._fields_)
        assert struct.Struct(fields).size == pack.__self__.size == lib.replay_abi_sizeof(which)
        n = len(struct.unpack(fields, bytes(struct.calcsize(fields))))
        assert pack(*range(n)) == struct.pack(fields, *range(n))
