"""What scoring prompts refuses before the model runs (no GPU)."""
import types

import pytest
import torch


def _model(batch=2, vocab=8):
    state = types.SimpleNamespace(shapes=types.SimpleNamespace(batch=batch))
    return types.SimpleNamespace(embed=torch.zeros(vocab, 4), mixers=[types.SimpleNamespace(state=state)],
                                 logits=lambda *a: pytest.fail("the model ran"))


@pytest.mark.parametrize("prompts,says", [([[1, 2], []], "empty"), ([[1]], "1 prompts for 2"), ([[1], [8]], "0 to 7"), ([[1], [-1]], "0 to 7")])
def test_score_refuses(prompts, says):
    from hybrid_model_ssm_replay_amd.generate import score
    with pytest.raises(ValueError, match=says):
        score(_model(), prompts)


def test_commands_and_kinds_refused():
    from hybrid_model_ssm_replay_amd import generate
    for bad in (["--kind", "rnn"], ["--top", "-1"], ["--top", "33"]):
        with pytest.raises(SystemExit):
            generate.main(bad)
    with pytest.raises(ValueError, match="kind"):
        generate.Model(kind="rnn")


@pytest.mark.parametrize("top", [-1, 33])
def test_score_refuses_alternatives_before_the_model_runs(top):
    """A refused call leaves the model's sequences where they were."""
    from hybrid_model_ssm_replay_amd.generate import score
    with pytest.raises(ValueError, match="top is 0 to 32"):
        score(_model(), [[1, 2], [3]], top=top)
