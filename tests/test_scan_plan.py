"""The scan's plan of a call (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def B():
    from hybrid_model_ssm_replay_amd import binding
    binding.load_library()
    return binding


def test_a_plan_agrees_with_the_workspace(B):
    for H, G, P, N, tokens, n in ((128, 8, 64, 128, 8192, 1), (128, 8, 64, 128, 16384, 24), (64, 4, 64, 128, 2048, 5), (2, 1, 64, 128, 321, 1),
                                  (2, 1, 64, 128, 320, 1), (12, 4, 80, 32, 900, 30)):
        cfg = B.make_config(0, n, H, G, P, N, 1)
        p, ws = B.replay_scan_plan(cfg, tokens, n), B.replay_scan_workspace_bytes(cfg, tokens, n)
        assert (p.segment > 0) == (ws > 0) and p.columns in (16, 32) and p.workgroups >= n * G
        if ws:
            items = tokens // p.segment + n
            assert ws == (items * H * 4 + 255) // 256 * 256 + items * H * P * N * 4


def test_a_plan_is_refused_as_its_call_is(B):
    cfg = B.make_config(0, 2, 4, 2, 32, 64, 1)
    for c, tokens, n in ((cfg, -1, 1), (cfg, 8, 0), (cfg, 8, 3), (B.make_config(0, 2, 4, 2, 24, 64, 1), 8, 1)):
        with pytest.raises(B.ReplayError):
            B.replay_scan_plan(c, tokens, n)
