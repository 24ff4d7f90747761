"""What the residual norm and the log probabilities refuse before anything is enqueued, and where they launch (no GPU)."""
import contextlib
import ctypes
import struct

import pytest
import torch

from _fake_device import Placed

P16 = 4096  # an address that is never followed: every call here is refused on the host


@pytest.fixture(scope="module")
def B():
    from hybrid_model_ssm_replay_amd import binding
    binding.load_library()
    return binding


def _refused(B, fn):
    with pytest.raises(B.ReplayError) as e:
        fn()
    assert e.value.code == B.EINVAL


def test_residual_norm_refuses(B):
    good = dict(tokens=4, channels=64, group=0, x_dtype=1, residual_dtype=0, out_dtype=1, eps=1e-5, reserved=0, x_stride=64,
                residual_stride=64, out_stride=64, sum_stride=64, x=P16, residual=P16, weight=P16, out=P16, scales=P16, sum=P16)
    codes = dict(out_dtype=2, group=16)
    for bad in (dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(channels=0), dict(channels=(1 << 30) + 1), dict(x_dtype=2), dict(x_dtype=-1),
                dict(residual_dtype=2), dict(out_dtype=3), dict(out_dtype=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(reserved=1),
                dict(group=16), dict(x=0), dict(out=0), dict(sum=0), dict(x=P16 + 1), dict(residual=P16 + 2), dict(weight=P16 + 2),
                dict(out=P16 + 1), dict(sum=P16 + 2), dict(x_stride=-1), dict(residual_stride=-1), dict(out_stride=63), dict(sum_stride=63),
                dict(codes, group=0), dict(codes, group=24), dict(codes, group=8), dict(codes, group=128), dict(codes, scales=0),
                dict(codes, scales=P16 + 2), dict(codes, channels=1000, out_stride=1000, sum_stride=1000, group=500),
                dict(codes, channels=2048, out_stride=2048, sum_stride=2048, group=1024)):
        a = B.replay_residual_norm_args(*[{**good, **bad}[n] for n, _ in B.replay_residual_norm_args._fields_])
        _refused(B, lambda: B.replay_residual_norm(a, 0))
    for bad in (dict(tokens=1 << 24, channels=4096, out_stride=4096, sum_stride=4096),      # workgroups of 256: below 2^24
                dict(tokens=1 << 24, channels=20000, out_stride=20000, sum_stride=20000)):
        a = B.replay_residual_norm_args(*[{**good, **bad}[n] for n, _ in B.replay_residual_norm_args._fields_])
        _refused(B, lambda: B.replay_residual_norm(a, 0))
    none = B.replay_residual_norm_args(*[{**good, "tokens": 0, "x": 0, "out": 0}[n] for n, _ in B.replay_residual_norm_args._fields_])
    B.replay_residual_norm(none, 0)  # nothing to do: nothing is launched


def test_token_logprobs_refuses(B):
    good = dict(rows=2, vocab=5000, top=3, dtype=0, stride=5000, reserved=0, logits=P16, tokens=P16, logprobs=P16, entropy=P16,
                top_logprobs=P16, top_tokens=P16)
    for bad in (dict(rows=-1), dict(rows=(1 << 30) + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(top=-1), dict(top=33), dict(dtype=2),
                dict(stride=-1), dict(reserved=1), dict(logits=0), dict(logits=P16 + 2), dict(tokens=0), dict(logprobs=0), dict(entropy=0),
                dict(top_logprobs=0), dict(top_tokens=0), dict(rows=1 << 24, vocab=10)):
        a = B.replay_token_logprobs_args(*[{**good, **bad}[n] for n, _ in B.replay_token_logprobs_args._fields_])
        _refused(B, lambda: B.replay_token_logprobs(a, P16, 0))
    a = B.replay_token_logprobs_args(*[good[n] for n, _ in B.replay_token_logprobs_args._fields_])
    _refused(B, lambda: B.replay_token_logprobs(a, 0, 0))       # two rows of 5000 are cut: a workspace
    _refused(B, lambda: B.replay_token_logprobs(a, P16 + 16, 0))
    for rows, vocab, top in ((0, 5, 1), (5, 0, 1), (5, 5, 33), (5, 5, -1), ((1 << 30) + 1, 5, 1), (1, (1 << 30) + 1, 1)):
        assert B.replay_token_logprobs_workspace_bytes(rows, vocab, top) == 0
    assert B.replay_token_logprobs_workspace_bytes(4096, 1 << 17, 32) == 0 < B.replay_token_logprobs_workspace_bytes(1, 1 << 30, 0)
    none = B.replay_token_logprobs_args(*[{**good, "rows": 0, "logits": 0}[n] for n, _ in B.replay_token_logprobs_args._fields_])
    B.replay_token_logprobs(none, 0, 0)


def _on(*shape, dtype=torch.float32, at=0):
    return Placed.of(torch.zeros(shape, dtype=dtype), at)


E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("x,residual,weight,more", [
    (torch.zeros(4, 64), None, None, {}), (_on(4, 64), torch.zeros(4, 64), None, {}), (_on(4, 64), None, torch.zeros(64), {}),
    (_on(4, 64, dtype=torch.float16), None, None, {}), (_on(64), None, None, {}), (_on(4, 8, 8), None, None, {}),
    (_on(64, 4).t(), None, None, {}), (_on(4, 64), _on(4, 32), None, {}), (_on(4, 64), _on(3, 64), None, {}), (_on(4, 0), None, None, {}),
    (_on(4, 64), _on(4, 64, dtype=E4M3), None, {}), (_on(4, 64), _on(4, 64, at=1), None, {}), (_on(4, 64), None, _on(32), {}),
    (_on(4, 64), None, _on(64, dtype=torch.bfloat16), {}), (_on(4, 64), None, _on(64, at=1), {}),
    (_on(4, 64), None, None, dict(out_dtype=torch.float16)), (_on(4, 64), None, None, dict(scale_group=16)),
    (_on(4, 64), None, None, dict(out_dtype=E4M3, scale_group=0)), (_on(4, 64), None, None, dict(out_dtype=E4M3, scale_group=8)),
    (_on(4, 64), None, None, dict(out_dtype=E4M3, scale_group=24)), (_on(4, 64), None, None, dict(out_dtype=E4M3, scale_group=128)),
    (_on(4, 96), None, None, dict(out_dtype=E4M3, scale_group=48)),
])
def test_residual_norm_checks_its_tensors(monkeypatch, B, x, residual, weight, more):
    from hybrid_model_ssm_replay_amd import ops
    monkeypatch.setattr(B, "replay_residual_norm", lambda *a: pytest.fail("enqueued"))
    with pytest.raises(ValueError):
        ops.residual_norm(x, residual, weight, **more)


I32 = torch.int32


@pytest.mark.parametrize("logits,tokens,top", [
    (torch.zeros(4, 9), _on(4, dtype=I32), 0), (_on(4, 9), torch.zeros(4, dtype=I32), 0), (_on(4, 9), _on(3, dtype=I32), 0),
    (_on(4, 9), _on(4, dtype=torch.int64), 0), (_on(4, 9), _on(4, dtype=I32, at=1), 0), (_on(9, 4).t(), _on(9, dtype=I32), 0),
    (_on(4, 9, dtype=torch.float16), _on(4, dtype=I32), 0), (_on(9), _on(1, dtype=I32), 0), (_on(4, 9), _on(4, dtype=I32), -1),
    (_on(4, 9), _on(4, dtype=I32), 33), (_on(4, 0), _on(4, dtype=I32), 0), (_on(4, 9), _on(8, dtype=I32)[::2], 0),
])
def test_token_logprobs_checks_its_tensors(monkeypatch, B, logits, tokens, top):
    from hybrid_model_ssm_replay_amd import ops
    monkeypatch.setattr(B, "replay_token_logprobs", lambda *a: pytest.fail("enqueued"))
    with pytest.raises(ValueError):
        ops.token_logprobs(logits, tokens, top=top)


def test_packed_structs_have_the_librarys_sizes(B):
    from hybrid_model_ssm_replay_amd import ops
    lib = B.load_library()
    codes = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_void_p: "P"}
    for which, st, pack in ((10, B.replay_residual_norm_args, ops._STREAM), (11, B.replay_token_logprobs_args, ops._LOGPROBS)):
        fields = "@" + "".join(codes[t] for _, t in st._fields_)
        assert struct.Struct(fields).size == pack.__self__.size == lib.replay_abi_sizeof(which) == ctypes.sizeof(st)
        n = len(st._fields_)
        assert pack(*range(n)) == struct.pack(fields, *range(n))


def _calls(ops):
    on = lambda *s, **k: _on(*s, at=1, **k)  # noqa: E731
    return {
        "replay_delta_prompt": lambda: ops.delta_prompt(on(5, 2, 16), on(5, 2, 16), on(5, 2, 16), on(5, 2), on(5, 2), on(2, dtype=I32),
                                                        on(2, 2, 16, 16)),
        "replay_residual_norm": lambda: ops.residual_norm(on(5, 8), on(5, 8), on(8)),
        "replay_token_logprobs": lambda: ops.token_logprobs(on(5, 8), on(5, dtype=I32), top=2),
    }


@pytest.mark.parametrize("name", ["replay_delta_prompt", "replay_residual_norm", "replay_token_logprobs"])
@pytest.mark.parametrize("current", [0, 1])
def test_a_call_runs_on_its_tensors_device(monkeypatch, B, name, current):
    from hybrid_model_ssm_replay_amd import ops
    now, seen = [current], []

    @contextlib.contextmanager
    def device(at):
        before, now[0] = now[0], at
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(ops, "_device", lambda: now[0])
    monkeypatch.setattr(ops, "_raw_stream", lambda at: 100 + at)
    monkeypatch.setattr(B, name, lambda *a: seen.append((now[0], a[-1])))
    _calls(ops)[name]()
    assert seen == [(1, 101)] and now == [current]
