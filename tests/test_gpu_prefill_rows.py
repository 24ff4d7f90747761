"""A prompt writes the stored copies of its own rows alone, in layers with a separate read copy too.

The float32 state is the scan's own, so everything is compared bit by bit."""
import numpy as np
import pytest

from _gpu import announce

pytestmark = pytest.mark.gpu
H, G, P, N, BATCH = 4, 2, 64, 128, 5


def _starts(lens):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _setup(bf16, seed=4):
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    vec = torch.bfloat16 if bf16 else torch.float32
    A, D = -torch.rand(H, device="cuda", generator=g) - 0.1, rand(H)
    rec = lambda *n: {"x": rand(*n, H, P).to(vec), "B": rand(*n, G, N).to(vec), "C": rand(*n, G, N).to(vec),  # noqa: E731
                      "dt": rand(*n, H).abs() * 0.1}
    make = lambda: ReplayLayer("mamba2", BATCH, H, P, N, 4, groups=G, ckpt_fmt=B.FMT_F32, read_fmt=B.FMT_F4E2M1_B16, A=A,  # noqa: E731
                               D=D, flags=B.FLAG_BF16_RECORDS if bf16 else 0)
    return make, rec, A, D


def _by_row(read_copy):
    """The read copy's codes and block scales, [batch, ...] each."""
    n = BATCH * H * P * N
    codes, at = read_copy[:n // 2], (n // 2 + 255) // 256 * 256
    return codes.view(BATCH, -1), read_copy[at:at + n // 16].view(BATCH, -1)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows,lens,resume", [([3], [70], None), ([4, 0], [5, 130], [1, 0]), ([2], [0], None), (None, [9, 40], [0, 1]),
                                              ([1, 3, 0, 2, 4], [3, 1, 2, 400, 20], None), (None, [3, 1, 2, 60, 20], [1, 1, 0, 1, 1])])
def test_a_prompt_writes_its_own_rows_of_both_copies(bf16, rows, lens, resume):
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("prefill rows", bf16, rows, lens, resume)
    make, rec, A, D = _setup(bf16)
    lay, ref = make(), make()
    begin = torch.randn(BATCH, H, P, N, device="cuda")
    steps = [rec(BATCH) for _ in range(6)]  # past a fold, then two records in every window
    for layer in (lay, ref):
        layer.set_state(begin)
        for r in steps:
            layer.step(r)
    mine = list(range(len(lens))) if rows is None else rows
    others = [b for b in range(BATCH) if b not in mine]
    prompt, at = rec(sum(lens)), None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    flags = None if resume is None else torch.tensor(resume, dtype=torch.bool, device="cuda")
    for part in _by_row(lay.read_copy):  # what nothing but an encoding of these rows would write over
        part[others] = 0x5A
    kept = [part.clone() for part in _by_row(lay.read_copy)] + [lay.checkpoint.clone()]
    y = lay.prefill(prompt, _starts(lens), rows=at, resume=flags)
    for part, was in zip([*_by_row(lay.read_copy), lay.checkpoint], kept):
        assert torch.equal(part[others], was[others])
    assert torch.equal(lay.pointers()[0], ref.pointers()[0])
    # The prompted rows: the scan over the flushed state, encoded by set_state.
    ref.flush()
    state = ref.checkpoint.clone()
    want = ops.scan_prompt(prompt["x"], prompt["B"], prompt["C"], prompt["dt"], A, D, _starts(lens), state,
                           initial=None if resume is None else state, rows=at, resume=flags)
    ref.set_state(state)
    assert torch.equal(y, want) and torch.equal(lay.checkpoint[mine], state[mine])
    for part, full in zip(_by_row(lay.read_copy), _by_row(ref.read_copy)):
        assert torch.equal(part[mine], full[mine])


def test_other_sequences_continue_with_the_same_bits():
    """Sequences in the middle of their windows, beside one that takes a prompt."""
    import torch
    announce("prefill beside running sequences")
    make, rec, _, _ = _setup(False)
    lay, alone = make(), make()
    begin = torch.randn(BATCH, H, P, N, device="cuda")
    steps, prompt = [rec(BATCH) for _ in range(12)], rec(30)
    lay.set_state(begin), alone.set_state(begin)
    for i, r in enumerate(steps):
        if i == 6:
            lay.prefill(prompt, _starts([30]), rows=torch.tensor([2], dtype=torch.int32, device="cuda"))
        y, want = lay.step(r), alone.step(r)
        same = [0, 1, 3, 4] if i >= 6 else range(BATCH)
        assert all(torch.equal(y[b], want[b]) for b in same)


def test_renewing_a_read_copy_refuses_other_formats():
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer
    announce("renew refusals")
    one = torch.ones(4, device="cuda")
    for cf, rf in ((B.FMT_F32, B.FMT_F32), (B.FMT_F16_SR, B.FMT_F4E2M1_B16), (B.FMT_F8E4M3, B.FMT_F8E4M3)):
        lay = ReplayLayer("mamba2", BATCH, H, P, N, 4, groups=G, ckpt_fmt=cf, read_fmt=rf, A=-one, D=one)
        with pytest.raises(B.ReplayError) as e:
            B.replay_renew_read_copy(lay.ctx, None, 0)
        assert e.value.code == B.ENOTSUP


@pytest.mark.parametrize("kind,rf", [("gdn", "FMT_F4E2M1_CS"), ("gdn", "FMT_F4E2M1_B16"), ("mamba2", "FMT_F4E2M1_B16")])
@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("rows", [[1, 4], None])
def test_renewing_a_read_copy_is_set_state_of_the_masked_rows(kind, rf, P, rows):
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer
    announce("renew read copy", kind, rf, P, rows)
    g = torch.Generator(device="cuda").manual_seed(P)
    params = dict(A=-torch.ones(H, device="cuda"), D=torch.ones(H, device="cuda"), groups=G) if kind == "mamba2" else {}
    make = lambda: ReplayLayer(kind, BATCH, H, P, N, 4, read_fmt=getattr(B, rf), **params)  # noqa: E731
    lay, ref = make(), make()
    state = torch.randn(BATCH, H, P, N, generator=g, device="cuda")
    n = BATCH * H * P * N
    scales = (n // 2 + 255) // 256 * 256
    cols = (scales + n // 16 + 255) // 256 * 256

    def parts(copy):
        got = [copy[:n // 2].view(BATCH, -1), copy[scales:scales + n // 16].view(BATCH, -1)]
        return got + ([copy[cols:cols + BATCH * H * N].view(BATCH, -1)] if rf == "FMT_F4E2M1_CS" else [])

    ref.set_state(state)
    lay.checkpoint.copy_(state)
    lay.read_copy.fill_(0x5A)
    mask = None
    if rows is not None:
        mask = torch.zeros(BATCH, dtype=torch.uint8, device="cuda")
        mask[rows] = 1
    B.replay_renew_read_copy(lay.ctx, None if mask is None else mask.data_ptr(), torch.cuda.current_stream().cuda_stream)
    mine = list(range(BATCH)) if rows is None else rows
    others = [b for b in range(BATCH) if b not in mine]
    for part, want in zip(parts(lay.read_copy), parts(ref.read_copy)):
        assert torch.equal(part[mine], want[mine]) and bool((part[others] == 0x5A).all())
    assert torch.equal(lay.checkpoint, state)
