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
