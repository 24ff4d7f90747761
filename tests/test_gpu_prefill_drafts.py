"""Prompts of Gated DeltaNet layers whose drafts are still pending: discarded, as by a step."""
import pytest

from _gpu import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("flags", [0, 2])
@pytest.mark.parametrize("rf", ["FMT_F32", "FMT_F4E2M1_B16", "FMT_F4E2M1_CS"])
@pytest.mark.parametrize("rows,resume", [([1], None), ([3, 0], [1, 0]), (None, [0, 1, 1, 0]), (None, None)])
def test_prefill_discards_pending_drafts(flags, rf, rows, resume):
    """A layer that verified drafts without a commit, and one that never saw them, are the same behind a prompt."""
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer
    announce("gdn prefill over drafts", flags, rf, rows, resume)
    H, P, N, batch = 4, 64, 128, 4
    g = torch.Generator(device="cuda").manual_seed(8)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    vec = torch.bfloat16 if flags else torch.float32
    unit = lambda *s: torch.nn.functional.normalize(rand(*s), dim=-1).to(vec)  # noqa: E731
    rec = lambda *n: {"q": unit(*n, H, N), "k": unit(*n, H, N), "v": rand(*n, H, P).to(vec),  # noqa: E731
                      "alpha": torch.exp(-rand(*n, H).abs() * 0.1), "beta": torch.sigmoid(rand(*n, H))}
    with_drafts, without = (ReplayLayer("gdn", batch, H, P, N, 8, max_draft=3, read_fmt=getattr(B, rf), flags=flags) for _ in range(2))
    begin, steps, drafts = rand(batch, H, P, N), [rec(batch) for _ in range(3)], rec(batch, 3)
    n = batch if rows is None else len(rows)
    lens = [70, 1, 20, 130][:n]
    prompt, start = rec(sum(lens)), torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    at = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    known = None if resume is None else torch.tensor(resume, dtype=torch.bool, device="cuda")
    after = [rec(batch) for _ in range(9)]  # past a fold
    got = []
    for lay in (with_drafts, without):
        lay.set_state(begin)
        for r in steps:  # with the drafts six records: none of the windows of eight folds
            lay.step(r)
        if lay is with_drafts:
            lay.verify(drafts)
        got.append([lay.prefill(prompt, start, rows=at, resume=known), lay.pointers()[0].clone(), lay.checkpoint.clone()]
                   + [lay.step(r) for r in after] + [lay.checkpoint.clone()])
        assert lay.t_pending == 0 and lay.status == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
