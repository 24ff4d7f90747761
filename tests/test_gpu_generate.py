"""Prompts, steps and drafts together: a layer, and a model that samples from itself.

All float32.  The bar for two ways through a layer: the convolution's 13 u, the
scan's (N + 64 + 112 + 4 n / 64) u relative to the size of its terms, taken as up
to 32 times the outputs', the decode step's sums of N + L terms likewise, two
norms' (group + 24) u; with N = 64, n below 600 and u = 2^-24 these are 12600 u of
either way's outputs, and the projections (sums of 256 and fewer) add less: 2^-10
of the largest output is 16384 u."""
import numpy as np
import pytest

from _gpu import announce

pytestmark = pytest.mark.gpu
BAR = 2.0 ** -10


def _mixer(batch, seed=3, **kw):
    import torch
    from hybrid_model_ssm_replay_amd.generate import Mixer
    rng = torch.Generator(device="cuda")
    rng.manual_seed(seed)
    return Mixer(96, 4, 32, 2, 64, batch, dtype=torch.float32, rng=rng, **kw)


def _starts(lens):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _inputs(lens, seed=1):
    import torch
    rng = torch.Generator(device="cuda")
    rng.manual_seed(seed)
    return [torch.randn((n, 96), generator=rng, device="cuda") for n in lens]


def _same(got, want):
    assert float((got - want).abs().max()) <= BAR * float(want.abs().max())


@pytest.mark.parametrize("firsts", [(300, 1, 64), (5, 130, 0)])
def test_prompt_steps_and_drafts_are_the_whole_prompt(firsts):
    """A prompt, steps past a full window, drafts of which some are kept, a second prompt, a step."""
    import torch
    announce("mixer", firsts)
    kept_runs = [(2, 0, 5), (5, 1, 3)]
    more, steps = (40, 0, 3), 19
    lens = [f + steps + sum(k[i] for k in kept_runs) + m + 1 for i, (f, m) in enumerate(zip(firsts, more))]
    xs = _inputs(lens)
    whole = _mixer(3).prefill(torch.cat(xs), _starts(lens)).split(lens)
    mix = _mixer(3)
    at = list(firsts)
    y = mix.prefill(torch.cat([x[:f] for x, f in zip(xs, firsts)]), _starts(firsts)).split(firsts)
    for i in range(3):
        if firsts[i]:
            _same(y[i], whole[i][:firsts[i]])
    for _ in range(steps):
        y = mix.tokens(torch.stack([x[a:a + 1] for x, a in zip(xs, at)]), False)
        _same(y[:, 0], torch.stack([w[a] for w, a in zip(whole, at)]))
        at = [a + 1 for a in at]
    for kept in kept_runs:
        d = torch.stack([torch.cat([x[a:a + k], torch.full((5 - k, 96), 7.0, device="cuda")]) for x, a, k in zip(xs, at, kept)])
        y = mix.tokens(d, True)
        for i, k in enumerate(kept):
            if k:
                _same(y[i, :k], whole[i][at[i]:at[i] + k])
        mix.commit(torch.tensor(kept, dtype=torch.int32, device="cuda"))
        at = [a + k for a, k in zip(at, kept)]
    y = mix.prefill(torch.cat([x[a:a + m] for x, a, m in zip(xs, at, more)]), _starts(more),
                    resume=torch.ones(3, dtype=torch.bool, device="cuda")).split(more)
    for i, m in enumerate(more):
        if m:
            _same(y[i], whole[i][at[i]:at[i] + m])
    # the positions of the layer count decoded tokens, so the second prompt's history sits behind the same position
    at = [a + m for a, m in zip(at, more)]
    y = mix.tokens(torch.stack([x[a:a + 1] for x, a in zip(xs, at)]), False)
    _same(y[:, 0], torch.stack([w[-1] for w in whole]))
    assert mix.state.status == 0


def test_a_new_prompt_in_a_row_leaves_the_other_sequences_alone():
    import torch
    announce("prompt into a running batch")
    xs = _inputs((30, 30, 30, 83))
    runs = []
    for enters in (False, True):
        mix = _mixer(3)
        mix.prefill(torch.cat([x[:10] for x in xs[:3]]), _starts((10, 10, 10)))
        out = []
        for t in range(10, 30):
            if enters and t == 17:
                row = torch.tensor([1], dtype=torch.int32, device="cuda")
                mix.prefill(xs[3][:70], _starts((70,)), rows=row)
            out.append(mix.tokens(torch.stack([xs[0][t:t + 1], xs[3][53 + t:54 + t] if enters and t >= 17 else xs[1][t:t + 1],
                                               xs[2][t:t + 1]]), False)[:, 0])
        runs.append(torch.stack(out, 1))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][2], runs[1][2])
    whole = _mixer(1).prefill(xs[3], _starts((83,)))
    _same(runs[1][1][7:], whole[70:])


@pytest.mark.parametrize("cf,rf", [(0, 0), (0, 3), (1, 3), (2, 3)])
def test_prefill_stores_the_state_in_the_layers_formats(cf, rf):
    import torch
    from hybrid_model_ssm_replay_amd import ops
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer
    announce("prefill formats", cf, rf)
    r = torch.Generator(device="cuda")
    r.manual_seed(9)
    rand = lambda *s: torch.randn(s, generator=r, device="cuda")
    H, G, P, N, lens = 4, 2, 64, 128, (90, 0, 33)
    A, D = -torch.rand(H, device="cuda", generator=r) - 0.1, rand(H)
    rec = {"x": rand(123, H, P), "B": rand(123, G, N), "C": rand(123, G, N), "dt": rand(123, H).abs() * 0.1}
    make = lambda: ReplayLayer("mamba2", 3, H, P, N, 4, groups=G, ckpt_fmt=cf, read_fmt=rf, A=A, D=D)
    lay, plain = make(), make()
    step = {n: t[:3].contiguous() for n, t in rec.items()}
    lay.step(step)  # what the prompts replace
    y = lay.prefill(rec, _starts(lens))
    state = torch.full((3, H, P, N), float("nan"), device="cuda")
    want = ops.scan_prompt(rec["x"], rec["B"], rec["C"], rec["dt"], A, D, _starts(lens), state)
    plain.step(step)
    plain.flush()
    plain.set_state(state)
    assert torch.equal(y, want)
    for a, b in zip(lay.stored_copies(), plain.stored_copies()):
        assert (a is None and b is None) or torch.equal(a, b)
    assert torch.equal(lay.step(step), plain.step(step))
    if cf:
        with pytest.raises(ValueError):
            lay.prefill(rec, _starts(lens), resume=torch.ones(3, dtype=torch.bool, device="cuda"))
        with pytest.raises(ValueError):
            lay.prefill(rec, _starts(lens[:2]))


@pytest.mark.parametrize("drafted", [0, 3, 7])
def test_generate_agrees_with_its_own_prompt(drafted):
    """After sampling with drafts, the running model and a fresh one that reads everything as a
    prompt give the same distribution (two layers and a head of slope below 4: eight bars)."""
    import torch
    from hybrid_model_ssm_replay_amd.generate import Model, generate
    announce("generate", drafted)
    make = lambda: Model(vocab=96, width=64, batch=3, dtype=torch.float32, heads=4, head_dim=32, state_dim=32)
    model, fresh = make(), make()
    rng = torch.Generator(device="cuda")
    rng.manual_seed(drafted)
    prompts = [[(7 * i + 3 * j) % 96 for j in range(n)] for i, n in enumerate((70, 1, 20))]
    new, calls = generate(model, prompts, 30, drafted, rng)
    assert min(map(len, new)) >= 30 and 1 < calls <= 31
    last = torch.tensor([[n[-1]] for n in new], dtype=torch.int32, device="cuda")
    got = model.tokens(last, drafts=False)[:, 0]
    lens = [len(p) + len(n) for p, n in zip(prompts, new)]
    want = fresh.prefill(torch.tensor([t for p, n in zip(prompts, new) for t in p + n], device="cuda"), _starts(lens))
    want = want[_starts(lens)[1:].long() - 1]
    assert float((got - want).abs().max()) <= 8 * BAR * float(want.max())
    assert all(m.state.status == 0 for m in model.mixers)
