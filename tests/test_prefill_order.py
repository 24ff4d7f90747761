"""A layer's prefill looks at every argument before it flushes: a call that raises leaves the drafts alone (no GPU)."""
import pytest
import torch

from _fake_device import Placed

TOKENS, BATCH, H, G, P, N = 5, 3, 4, 2, 32, 64


def _on(*shape, dtype=torch.float32):
    return Placed.of(torch.zeros(shape, dtype=dtype))


def _good(dtype=torch.float32):
    return dict(x=_on(TOKENS, H, P, dtype=dtype), B=_on(TOKENS, G, N, dtype=dtype), C=_on(TOKENS, G, N, dtype=dtype), dt=_on(TOKENS, H),
                seq_start=_on(BATCH + 1, dtype=torch.int32), rows=_on(BATCH, dtype=torch.int32), resume=_on(BATCH, dtype=torch.bool),
                out_dtype=None)


@pytest.fixture
def layer(monkeypatch):
    """A layer on host memory; its calls to the device are noted in ``done``."""
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer, _kind, _Shapes

    def make(flags=0):
        lay = object.__new__(ReplayLayer)
        lay.shapes = _Shapes(_kind("mamba2"), BATCH, H, G, P, N, flags)
        lay.cfg = B.make_config(_kind("mamba2"), BATCH, H, G, P, N, 4, 0, 0, 0, 0, flags)
        lay.ckpt, lay.read_copy, lay.status_word = _on(BATCH * H * P * N * 4, dtype=torch.uint8), None, _on(4, dtype=torch.int32)
        lay.A, lay.D = _on(H), _on(H)
        lay.done = []
        lay.flush = lambda mask: lay.done.append("flush")
        monkeypatch.setattr(B, "replay_scan_prompt", lambda *a: lay.done.append("scan"))
        return lay

    B.load_library()
    monkeypatch.setattr(ops, "_device", lambda: 0)
    monkeypatch.setattr(ops, "_raw_stream", lambda at: 0)
    return make


def _call(lay, **args):
    a = {**_good(lay.shapes.vec_dtype), **args}
    return lay.prefill({n: a.pop(n) for n in ("x", "B", "C", "dt")}, **a)


def test_a_good_call_flushes_and_scans(layer):
    lay = layer()
    _call(lay)
    assert lay.done == ["flush", "scan"]


def _off(shape):  # an address that is not a multiple of 16
    t = Placed.of(torch.zeros(1 + torch.Size(shape).numel())[1:].view(shape))
    assert t.data_ptr() % 16
    return t


@pytest.mark.parametrize("flags,bad", [
    (0, dict(x=_on(TOKENS, H, 2 * P))), (0, dict(x=_on(TOKENS, P, H).transpose(1, 2))), (0, dict(x=_off((TOKENS, H, P)))),
    (0, dict(B=_on(TOKENS, H, N), C=_on(TOKENS, H, N))),  # more groups than the layer has
    (0, dict(B=_on(TOKENS, G, N), C=_on(TOKENS, G, 2 * N))), (0, dict(B=_on(TOKENS + 1, G, N))), (0, dict(C=_off((TOKENS, G, N)))),
    (0, dict(B=_on(TOKENS, G, N, dtype=torch.bfloat16))), (0, dict(dt=_on(TOKENS, H, dtype=torch.bfloat16))),
    (0, dict(dt=_on(TOKENS, 1))), (0, dict(dt=_on(H, TOKENS).t())), (0, dict(dt=torch.zeros(TOKENS, H))),
    (0, dict(seq_start=_on(BATCH + 1, dtype=torch.int64))), (0, dict(rows=_on(2 * BATCH, dtype=torch.int32)[::2])),
    (0, dict(resume=_on(BATCH + 1, dtype=torch.bool))), (0, dict(resume=_on(BATCH))), (0, dict(out_dtype=torch.float16)),
    (0, dict(out_dtype=torch.bfloat16)),               # of float32 records
    (2, dict(C=_on(TOKENS, G, N))), (2, dict(out_dtype=torch.float64)),
])
def test_refused_before_anything_is_enqueued(layer, flags, bad):
    lay = layer(flags)
    with pytest.raises(ValueError):
        _call(lay, **bad)
    assert not lay.done


def test_a_record_without_a_field_is_refused_before_anything_is_enqueued(layer):
    lay, good = layer(), _good()
    with pytest.raises((ValueError, KeyError)):
        lay.prefill({n: good[n] for n in ("x", "B", "C")}, good["seq_start"])
    assert not lay.done
