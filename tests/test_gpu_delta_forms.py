"""Prompts of Gated DeltaNet layers: 32 rows of a head's state to a workgroup (float32 records), several passes, far tokens."""
import numpy as np
import pytest

from _delta import DeltaPrompts, check
from _gpu import announce

pytestmark = pytest.mark.gpu

# At least 512 workgroups of 16 rows, and rows in 32s: with fewer, or other head sizes, a workgroup has 16.
CASES = [
    # H, P, N, lengths, resumed
    (32, 128, 128, [20, 300, 1, 0, 64], [1, 0, 1, 1, 0]),
    (64, 64, 64, [65, 130], "all"),
    (64, 96, 32, [70, 1, 129], None),
    (128, 32, 16, [3, 66], [0, 1]),
    (32, 128, 128, [190, 63], None),
    (43, 32, 64, [64, 0, 128, 5, 31, 33, 17], "all"),
    (16, 128, 16, [40, 129, 2, 64], [1, 1, 0, 0]),
    (1, 64, 128, [7, 64, 65, 0, 1] * 26, [1, 0, 1, 1, 0] * 26),
]


@pytest.mark.parametrize("H,P,N,lens,resumed", CASES)
def test_delta_prompt_of_32_rows(H, P, N, lens, resumed):
    announce("delta_prompt float32", H, P, N, len(lens), lens[:8], resumed if resumed is None else resumed[:8])
    assert P % 32 == 0 and len(lens) * H * (P // 16) >= 512
    p = DeltaPrompts(H, P, N, lens, resumed, "f32", tail=200).surround()
    check(p, "f32", *p.run("f32"))


@pytest.mark.parametrize("what", ["same keys", "alpha 0", "tiny alpha", "beta 0", "beta 2", "zero keys"])
def test_delta_prompt_of_32_rows_extremes(what):
    announce("delta_prompt float32 extremes", what)
    p = DeltaPrompts(64, 64, 64, [150, 70], "all", "f32", seed=3)
    r = np.random.default_rng(5)
    if what == "same keys":
        p.k[:], p.beta[:], p.alpha[:] = p.k[:1], 1.0, 1.0
    elif what == "alpha 0":
        p.alpha[r.random(p.alpha.shape) < 0.1] = 0.0
    elif what == "tiny alpha":
        p.alpha[r.random(p.alpha.shape) < 0.3] = 1e-38
    elif what == "beta 0":
        p.beta[r.random(p.beta.shape) < 0.5] = 0.0
    elif what == "beta 2":
        p.beta[:] = 2.0
    else:
        p.k[r.random(p.tokens) < 0.5] = 0.0
        p.q[r.random(p.tokens) < 0.2] = 0.0
    p.surround()
    check(p, "f32", *p.run("f32"))


@pytest.mark.parametrize("H,P,lens", [(64, 128, (6016,)), (64, 128, (64, 2560, 320, 3100)), (32, 48, (11008, 70)), (32, 32, (64, 5500, 30, 6016))])
def test_several_passes_are_bit_equal_to_calls_of_whole_chunks(H, P, lens):
    """More chunks than one pass holds (40 of 64 heads, 81 of 32); calls of 1024 tokens are one pass each, of as many
    rows to a workgroup (32 with 64 heads of 128; 16 with the others, also for all their sequences)."""
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    announce("delta_prompt float32 passes", H, P, lens)
    N, tokens, n = 128, sum(lens), len(lens)
    c = B.make_config(1, n, H, H, P, N, 1)
    size = lambda t: B.replay_delta_workspace_bytes(c, t, n, B.DT_F32)  # noqa: E731
    assert size(1024) < size(tokens) == size(1 << 30)
    assert (P % 32 == 0 and H * (P // 16) >= 512) or P % 32 or n * H * (P // 16) < 512
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k = (torch.nn.functional.normalize(rand(tokens, H, N), dim=-1) for _ in range(2))
    v, alpha, beta = rand(tokens, H, P), torch.rand(tokens, H, generator=g, device="cuda"), torch.rand(
        tokens, H, generator=g, device="cuda")
    start = [0]
    for m in lens:
        start.append(start[-1] + m)
    init = rand(n, H, P, N)
    state = init.clone()
    y = ops.delta_prompt(q, k, v, alpha, beta, torch.tensor(start, dtype=torch.int32, device="cuda"), state, initial=state)
    want, parts = init.clone(), []
    for i in range(n):
        for a in range(start[i], start[i + 1], 1024):
            b = min(a + 1024, start[i + 1])
            parts.append(ops.delta_prompt(*[t[a:b] for t in (q, k, v, alpha, beta)],
                                          torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), want, initial=want,
                                          rows=torch.tensor([i], dtype=torch.int32, device="cuda")))
    assert torch.equal(y, torch.cat(parts)) and torch.equal(state, want)


@pytest.mark.parametrize("name,H,P,N", [("f32", 33, 48, 128), ("bf16", 8, 64, 128), ("bf16", 128, 64, 64)])
def test_tokens_whose_offsets_pass_32_bits(name, H, P, N):
    """Sequences behind 2^31 values of q and k: each one's results are those of a call of its own."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("delta_prompt far", name, H, P, N)
    far = (1 << 31) // (H * N) // 64 * 64 + 64
    lens, at = [70, 130], [3, far]
    tokens = far + lens[1] + 5
    dt = torch.float32 if name == "f32" else torch.bfloat16
    q, k = (torch.empty(tokens, H, N, dtype=dt, device="cuda") for _ in range(2))
    v, alpha, beta = torch.empty(tokens, H, P, dtype=dt, device="cuda"), *(torch.empty(tokens, H, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(5)
    for a, m in zip(at, lens):
        for t in (q, k):
            t[a:a + m] = torch.nn.functional.normalize(torch.randn(m, H, N, generator=g, device="cuda"), dim=-1).to(dt)
        v[a:a + m] = torch.randn(m, H, P, generator=g, device="cuda").to(dt)
        for t in (alpha, beta):
            t[a:a + m] = torch.rand(m, H, generator=g, device="cuda")
    for first, m in zip(at, lens):
        start = torch.tensor([first, first + m], dtype=torch.int32, device="cuda")
        state, alone = (torch.zeros(1, H, P, N, device="cuda") for _ in range(2))
        y = ops.delta_prompt(q, k, v, alpha, beta, start, state)
        short = [t[first:first + m].clone() for t in (q, k, v, alpha, beta)]
        want = ops.delta_prompt(*short, torch.tensor([0, m], dtype=torch.int32, device="cuda"), alone)
        off = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
        # Either form of the walk: 16 U each way (see TOGETHER).
        assert off(y[first:first + m], want) <= 32 * 2.0 ** -24 and off(state, alone) <= 32 * 2.0 ** -24
