"""The operators launch on the device of their tensors, whichever is current (no GPU)."""
import contextlib

import pytest
import torch

from _fake_device import Placed

OTHER = 1


def _calls(ops):
    def on(*shape, dtype=torch.float32):
        return Placed.of(torch.zeros(shape, dtype=dtype), OTHER)

    def i32(*shape):
        return on(*shape, dtype=torch.int32)

    return {
        "replay_short_conv_step": lambda: ops.short_conv_step(on(2, 1, 8), on(8, 4), on(4, 2, 8), i32(2), (8,)),
        "replay_short_conv_prompt": lambda: ops.short_conv_prompt(on(5, 8), on(8, 4), on(4, 2, 8), i32(2), (8,)),
        "replay_scan_prompt": lambda: ops.scan_prompt(on(5, 2, 16), on(5, 1, 16), on(5, 1, 16), on(5, 2), on(2), on(2),
                                                      i32(2), on(2, 2, 16, 16)),
        "replay_gated_norm": lambda: ops.gated_norm(on(5, 8), on(5, 8), on(8), 4),
        "replay_accept_drafts": lambda: ops.accept_drafts(i32(1, 2), on(1, 3, 9), on(1, 3)),
    }


@pytest.mark.parametrize("name", ["replay_short_conv_step", "replay_short_conv_prompt", "replay_scan_prompt",
                                  "replay_gated_norm", "replay_accept_drafts"])
@pytest.mark.parametrize("current", [0, OTHER])
def test_a_call_runs_on_its_tensors_device(monkeypatch, name, current):
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    now, seen = [current], []

    @contextlib.contextmanager
    def device(at):
        before, now[0] = now[0], at
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(ops, "_device", lambda: now[0], raising=False)
    monkeypatch.setattr(ops, "_raw_stream", lambda at: 100 + at)
    monkeypatch.setattr(B, name, lambda *a: seen.append((now[0], a[-1])))
    _calls(ops)[name]()
    assert seen == [(OTHER, 100 + OTHER)] and now == [current]
