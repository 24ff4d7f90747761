"""A Gated DeltaNet layer and model through prompts, steps, drafts and scores, all float32.

The bar for two ways through a layer: the convolution's 13 u, the prompt's and the
decode steps' (2 N + 16 + 3 * 64 + 48) u relative to the size of their terms, taken as up
to 32 times the outputs', two norms' (group + 24) u; with N = 64 and u = 2^-24 these are
below 12600 u of either way's outputs, and the projections (sums of 256 and fewer) add
less: 2^-10 of the largest output is 16384 u."""
import numpy as np
import pytest

from _gpu import announce

pytestmark = pytest.mark.gpu
BAR = 2.0 ** -10


def _mixer(batch, seed=3, **kw):
    import torch
    from hybrid_model_ssm_replay_amd.generate import DeltaMixer
    rng = torch.Generator(device="cuda")
    rng.manual_seed(seed)
    return DeltaMixer(96, 4, 64, 64, batch, dtype=torch.float32, rng=rng, **kw)


def _starts(lens):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _same(got, want):
    assert float((got - want).abs().max()) <= BAR * float(want.abs().max())


@pytest.mark.parametrize("firsts", [(300, 1, 64), (5, 130, 0)])
def test_prompt_steps_and_drafts_are_the_whole_prompt(firsts):
    """A prompt, steps past a full window, drafts of which some are kept, a second prompt, a step."""
    import torch
    announce("delta mixer", firsts)
    kept_runs = [(2, 0, 5), (5, 1, 3)]
    more, steps = (40, 0, 3), 19
    lens = [f + steps + sum(k[i] for k in kept_runs) + m + 1 for i, (f, m) in enumerate(zip(firsts, more))]
    rng = torch.Generator(device="cuda")
    rng.manual_seed(1)
    xs = [torch.randn((n, 96), generator=rng, device="cuda") for n in lens]
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
    y = mix.tokens(torch.stack([w[-1:] for w in xs]), False)
    _same(y[:, 0], torch.stack([w[-1] for w in whole]))
    assert mix.state.status == 0


def _model(batch=3, **kw):
    import torch
    from hybrid_model_ssm_replay_amd.generate import Model
    return Model(vocab=96, width=64, batch=batch, kind="gdn", heads=4, head_dim=64, state_dim=32, **{"dtype": torch.float32, **kw})


@pytest.mark.parametrize("drafted", [0, 3, 7])
def test_generate_agrees_with_its_own_prompt(drafted):
    """After sampling with drafts, the running model and a fresh one that reads everything as a
    prompt give the same distribution (two layers and a head of slope below 4: eight bars)."""
    import torch
    from hybrid_model_ssm_replay_amd.generate import generate
    announce("generate gdn", drafted)
    model, fresh = _model(), _model()
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


@pytest.mark.parametrize("kind", ["gdn", "mamba2"])
def test_score_is_the_models_own_distribution(kind):
    """Log probabilities of a prompt's tokens from the same logits, by log_softmax in float64."""
    import torch
    from hybrid_model_ssm_replay_amd.generate import Model, score
    announce("score", kind)
    make = lambda: Model(vocab=300, width=64, batch=3, kind=kind)  # noqa: E731
    prompts = [[(7 * i + 3 * j) % 300 for j in range(n)] for i, n in enumerate((70, 1, 20))]
    got = score(make(), prompts, top=3)
    assert [len(g) for g in got] == [69, 0, 19]
    logits = make().logits(torch.tensor([t for p in prompts for t in p], device="cuda"), _starts([70, 1, 20])).double()
    logp = torch.log_softmax(logits, -1)
    entropy = -(logp.exp() * logp).sum(-1)
    for i, (p, at) in enumerate(zip(prompts, (0, 70, 71))):
        for j, (lp, e, best) in enumerate(got[i]):
            row = logp[at + j]
            assert abs(lp - float(row[p[j + 1]])) <= 1e-5 and abs(e - float(entropy[at + j])) <= 1e-5  # sums of 300: 2^-24 * 168
            first = torch.sort(logits[at + j], descending=True, stable=True).indices[:3].tolist()
            assert [w for w, _ in best] == first and all(abs(b - float(row[w])) <= 1e-5 for w, b in best)


def test_the_residual_stream_is_the_plain_one():
    """The model's own layers around elementary additions and norms (bf16 activations: both ways
    round each layer's output, sum and norm, six roundings of 2^-8 each, and the head's)."""
    import torch
    announce("gdn stream")
    a, b = _model(dtype=torch.bfloat16), _model(dtype=torch.bfloat16)
    tokens, start = torch.arange(90, device="cuda") % 96, _starts([40, 30, 20])
    got = a.logits(tokens, start).float()

    def norm(h, w):
        return (h.float() * torch.rsqrt((h.float() ** 2).mean(-1, keepdim=True) + 1e-5) * w).bfloat16()

    h = b.embed[tokens]
    for m, w in zip(b.mixers, b.norms):
        h = h + m.prefill(norm(h, w), start)
    want = (norm(h, b.norms[-1]) @ b.head).float()
    assert float((got - want).norm()) <= 8 * 2.0 ** -8 * float(want.norm())


def test_the_command_runs(capsys):
    announce("generate command")
    from hybrid_model_ssm_replay_amd import generate
    generate.main(["--kind", "gdn", "--batch", "2", "--prompt", "30", "--tokens", "5", "--top", "2"])
    out = capsys.readouterr().out
    assert "prompt 1:" in out and "sequence 1:" in out
