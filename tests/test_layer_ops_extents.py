"""Extents that the kernels' 32-bit indexes do not hold are refused on the host (no GPU)."""
import pytest

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


@pytest.mark.parametrize("heads,groups,P,N", [(1 << 16, 1, 128, 16), (1 << 19, 1 << 19, 16, 16), (1 << 16, 1 << 16, 16, 128),
                                              (1 << 20, 4, 64, 128)])
def test_scan_rows_past_32_bits_are_refused(B, heads, groups, P, N):
    """64 rows of heads * head_dim, or of groups * state_dim, float32 values are addressed by 32 bits: both below 2^23."""
    cfg = B.make_config(0, 1, heads, groups, P, N, 1)
    assert B.replay_scan_workspace_bytes(cfg, 1000, 1) == 0
    p = B.replay_prompt(8, 1, P16, 0, 0, 0)
    _refused(B, lambda: B.replay_scan_prompt(cfg, p, B.make_record(P16, P16, P16, P16), P16, P16, 0, P16, P16, B.DT_F32, P16, 0))


def test_convolutions_of_more_channels_or_rows_than_2_to_30_are_refused(B):
    for channels, batch in (((1 << 31) - 1, 1), ((1 << 30) + 1, 1), (8, (1 << 31) - 1), (8, (1 << 30) + 1)):
        c = B.replay_short_conv(channels, 4, 4, batch, B.DT_BF16, 1, (channels, 0, 0), 0, P16, 0, P16, P16, 0)
        _refused(B, lambda: B.replay_short_conv_step(c, P16, channels, channels, 1, [P16, 0, 0], 0))
        p = B.replay_prompt(8, 1, P16, 0, 0, 0)
        _refused(B, lambda: B.replay_short_conv_prompt(c, p, P16, channels, [P16, 0, 0], 0))


def _norm(B, tokens, channels, group):
    return B.replay_gated_norm_args(tokens, channels, group, group, 0, 0, 0, 0, 1e-5, 0, 0, 0, channels, P16, P16, P16, P16)


def test_norms_of_more_tokens_or_channels_than_2_to_30_are_refused(B):
    for tokens, channels, group in (((1 << 31) - 1, 1, 1), ((1 << 30) + 1, 8, 8), (1, (1 << 31) - 1, (1 << 31) - 1),
                                    (1, (1 << 30) + 128, 128)):
        _refused(B, lambda: B.replay_gated_norm(_norm(B, tokens, channels, group), 0))


def test_grids_past_2_to_32_work_items_are_refused(B):
    """A launch holds fewer than 2^32 work-items: workgroups of 256 below 2^24."""
    _refused(B, lambda: B.replay_gated_norm(_norm(B, 1 << 20, 1 << 13, 8), 0))                # 16 groups a workgroup: 2^26
    _refused(B, lambda: B.replay_gated_norm(_norm(B, 1 << 15, 1 << 21, 1 << 12), 0))          # one: 2^24
    c = B.replay_short_conv(1 << 20, 4, 8, 1 << 18, B.DT_BF16, 1, (1 << 20, 0, 0), 0, P16, 0, P16, P16, 0)
    _refused(B, lambda: B.replay_short_conv_step(c, P16, 0, 0, 1, [P16, 0, 0], 0))            # 2^18 rows in pairs, 512 each: 2^26
    p = B.replay_prompt(1 << 24, 1 << 18, P16, 0, 0, 0)
    _refused(B, lambda: B.replay_short_conv_prompt(c, p, P16, 0, [P16, 0, 0], 0))
    cfg = B.make_config(0, 1 << 20, 128, 8, 64, 128, 1)
    _refused(B, lambda: B.replay_scan_prompt(cfg, B.replay_prompt(1 << 20, 1 << 20, P16, 0, 0, 0), B.make_record(P16, P16, P16, P16),
                                             P16, P16, 0, P16, P16, B.DT_F32, 0, 0))          # 64 workgroups a sequence
    a = B.replay_accept_args(1 << 24, 1, 4, 0, 0, 0, 0, 0, 0, 0, P16, 0, P16, 0, P16, P16, P16)
    _refused(B, lambda: B.replay_accept_drafts(a, P16, 0))
