"""What generate refuses before the model runs (no GPU)."""
import types

import pytest
import torch


def _model(batch=2, vocab=8, max_draft=8):
    state = types.SimpleNamespace(shapes=types.SimpleNamespace(batch=batch), cfg=types.SimpleNamespace(max_draft=max_draft))
    return types.SimpleNamespace(embed=torch.zeros(vocab, 4), mixers=[types.SimpleNamespace(state=state)],
                                 prefill=lambda *a: pytest.fail("the model ran"))


@pytest.mark.parametrize("prompts,drafted,says", [
    ([[1, 2], []], 4, "empty"),                  # would be sampled behind another sequence's token
    ([[1]], 4, "1 prompts for 2"), ([[1], [2], [3]], 4, "3 prompts for 2"),
    ([[1], [8]], 4, "0 to 7"), ([[1], [-1]], 4, "0 to 7"),
    ([[1], [2]], 8, "drafted"), ([[1], [2]], -1, "drafted"),
])
def test_generate_refuses(prompts, drafted, says):
    from hybrid_model_ssm_replay_amd.generate import generate
    with pytest.raises(ValueError, match=says):
        generate(_model(), prompts, 5, drafted)
