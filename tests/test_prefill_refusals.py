"""What a layer's prefill refuses, before anything is enqueued (no GPU)."""
import pytest
import torch


def _layer(kind="mamba2", cf=0, rf=0, flags=0):
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer, _kind, _Shapes
    lay = object.__new__(ReplayLayer)
    lay.shapes = _Shapes(_kind(kind), 3, 4, 4, 128, 128, flags)
    lay.cfg = B.make_config(_kind(kind), 3, 4, 4, 128, 128, 4, 0, cf, rf, 0, flags)
    lay.flush = lambda mask: pytest.fail("enqueued")
    return lay


def _rec(dtype=torch.float32):
    return {"x": torch.zeros(5, 4, 128, dtype=dtype), "B": torch.zeros(5, 4, 128, dtype=dtype),
            "C": torch.zeros(5, 4, 128, dtype=dtype), "dt": torch.zeros(5, 4)}


START = torch.zeros(4, dtype=torch.int32)


@pytest.mark.parametrize("layer,rec,start,more,says", [
    (dict(kind="gdn"), _rec(), START, {}, "Mamba-2"),
    (dict(), _rec(), [0, 5], {}, "seq_start"),
    (dict(), _rec(), START[:1], {}, "seq_start"),
    (dict(), _rec(), torch.zeros(5, dtype=torch.int32), {}, "4 prompts for 3"),
    (dict(), _rec(torch.bfloat16), START, {}, "float32"),
    (dict(flags=2), _rec(), START, {}, "bfloat16"),
    (dict(), _rec(), START, dict(rows=START[:3]), "rows"),
    (dict(cf=1, rf=3), _rec(), START, dict(resume=torch.ones(3, dtype=torch.bool)), "below float32"),
    (dict(cf=2, rf=3), _rec(), START[:3], {}, "below float32"),
])
def test_prefill_refuses(layer, rec, start, more, says):
    with pytest.raises(ValueError, match=says):
        _layer(**layer).prefill(rec, start, **more)


def test_generate_refuses_arguments():
    from hybrid_model_ssm_replay_amd import generate
    for bad in (["--batch", "0"], ["--drafted", "8"], ["--prompt", "0"], ["--tokens", "0"]):
        with pytest.raises(SystemExit):
            generate.main(bad)
