"""A small Mamba-2 model that serves prompts, decode steps and drafted tokens.

``Mixer`` is one layer as it is served: input projection, short convolution,
recurrence, gated norm, output projection, on the operators of ``ops`` and the
state of a ``layer.ReplayLayer``.  ``Model`` stacks mixers between an embedding
and a head (random weights), and ``generate`` samples from it with drafts of a
bigram table.  The projections are torch products; everything in between is the
library's.

    python -m hybrid_model_ssm_replay_amd.generate --batch 4 --prompt 200 --tokens 64
"""
from __future__ import annotations

import argparse
import time

import torch
import torch.nn.functional as F

from . import binding as B
from . import ops
from .layer import ReplayLayer


class Mixer:
    """One layer for a fixed number of sequences.

    Positions, and with them the convolution's ring and the recurrent state's
    window, are those of the ReplayLayer: ``commit`` moves them, so rejected
    drafts need no restore in either."""

    def __init__(self, width, heads, head_dim, groups, state_dim, batch, window=16, max_draft=8, taps=4,
                 dtype=torch.bfloat16, rng=None, device="cuda"):
        inner, bc = heads * head_dim, groups * state_dim
        self.heads, self.head_dim, self.groups, self.state_dim = heads, head_dim, groups, state_dim
        self.widths = (inner, bc, bc)
        channels = inner + 2 * bc

        def normal(*shape, scale=1.0):
            return torch.randn(shape, generator=rng, device=device) * scale

        self.w_in = normal(width, inner + channels + heads, scale=width ** -0.5).to(dtype)
        self.w_out = normal(inner, width, scale=inner ** -0.5).to(dtype)
        self.w_conv, self.b_conv = normal(channels, taps, scale=taps ** -0.5), normal(channels, scale=0.1)
        self.dt_bias = normal(heads, scale=0.5) - 3.0
        self.w_norm = 1.0 + normal(inner, scale=0.1)
        A = -torch.rand(heads, generator=rng, device=device) * 4.0 - 0.5
        self.state = ReplayLayer("mamba2", batch, heads, head_dim, state_dim, window, groups=groups,
                                 max_draft=max_draft, A=A, D=normal(heads), device=device,
                                 flags=B.FLAG_BF16_RECORDS if dtype == torch.bfloat16 else 0)
        self.ring = torch.zeros((taps - 1 + max(1, max_draft), batch, channels), dtype=dtype, device=device)

    def _split(self, h):
        """z, the convolution's input and dt of every token: slices of one projection."""
        z, xbc, dt = torch.split(h @ self.w_in, (self.widths[0], sum(self.widths), self.heads), dim=-1)
        return z, xbc, F.softplus(dt.float() + self.dt_bias)

    def _record(self, x, Bm, Cm, dt):
        lead = x.shape[:-1]
        return {"x": x.view(*lead, self.heads, self.head_dim), "B": Bm.view(*lead, self.groups, self.state_dim),
                "C": Cm.view(*lead, self.groups, self.state_dim), "dt": dt}

    def _out(self, y, z):
        """Gated norm and output projection of [tokens, ...]."""
        y = ops.gated_norm(y.flatten(1), z, self.w_norm, self.widths[0] // self.groups)
        return y @ self.w_out

    def prefill(self, h, seq_start, rows=None, resume=None):
        """h [tokens, width]: packed prompts, as for ``ops.scan_prompt``."""
        z, xbc, dt = self._split(h)
        parts = ops.short_conv_prompt(xbc, self.w_conv, self.ring, seq_start, self.widths, bias=self.b_conv, rows=rows,
                                      pos=self.state.pointers()[0], resume=resume, status=self.state.status_word)
        return self._out(self.state.prefill(self._record(*parts, dt), seq_start, rows, resume, out_dtype=h.dtype), z)

    def tokens(self, h, drafts):
        """h [batch, T, width]: one token of every sequence (drafts False, T = 1), or T
        drafts, of which ``commit`` keeps the first ones."""
        batch, T, _ = h.shape
        z, xbc, dt = self._split(h)
        parts = ops.short_conv_step(xbc, self.w_conv, self.ring, self.state.pointers()[0], self.widths,
                                    bias=self.b_conv, status=self.state.status_word)
        if drafts:
            y = self.state.verify(self._record(*parts, dt))
        else:
            y = self.state.step({n: t[:, 0] for n, t in self._record(*parts, dt).items()})
        return self._out(y.view(batch * T, *y.shape[-2:]), z.flatten(0, 1)).view(batch, T, -1)

    def commit(self, accepted):
        self.state.commit(accepted)


class Model:
    """Embedding, ``layers`` mixers on a residual stream, head."""

    def __init__(self, vocab=512, width=256, layers=2, batch=4, seed=0, dtype=torch.bfloat16, device="cuda", **mixer):
        rng = torch.Generator(device=device)
        rng.manual_seed(seed)
        shape = dict(heads=8, head_dim=64, groups=2, state_dim=64)
        shape.update(mixer)
        self.embed = torch.randn((vocab, width), generator=rng, device=device).to(dtype)
        self.head = (torch.randn((width, vocab), generator=rng, device=device) * 1.5 * width ** -0.5).to(dtype)
        self.mixers = [Mixer(width, batch=batch, dtype=dtype, rng=rng, device=device, **shape) for _ in range(layers)]
        self.drafts = torch.softmax(torch.randn((vocab, vocab), generator=rng, device=device), -1)  # row: token before

    def _probabilities(self, h):
        return torch.softmax((F.rms_norm(h, h.shape[-1:]) @ self.head).float(), -1)

    def prefill(self, tokens, seq_start, rows=None, resume=None):
        """Packed prompt tokens [tokens]: the distribution after each."""
        h = self.embed[tokens.long()]
        for m in self.mixers:
            h = h + m.prefill(F.rms_norm(h, h.shape[-1:]), seq_start, rows, resume)
        return self._probabilities(h)

    def tokens(self, tokens, drafts):
        """tokens [batch, T]: the distribution after each (see ``Mixer.tokens``)."""
        h = self.embed[tokens.long()]
        for m in self.mixers:
            h = h + m.tokens(F.rms_norm(h, h.shape[-1:]), drafts)
        return self._probabilities(h)

    def commit(self, accepted):
        for m in self.mixers:
            m.commit(accepted)


def generate(model, prompts, count, drafted=4, rng=None):
    """At least ``count`` new tokens behind each prompt (lists of at least one token
    number, one for every sequence of the model).  Returns the new tokens, a list for each prompt, and
    how many calls of the model made them.

    Each call runs the last token and ``drafted`` drafts; the drafts are drawn from the
    model's bigram table, and the kept tokens follow the model's own distribution."""
    device, vocab = model.embed.device, model.embed.shape[0]
    batch, state = len(prompts), model.mixers[0].state
    if batch != state.shapes.batch:
        raise ValueError(f"{batch} prompts for {state.shapes.batch} sequences")
    if not all(len(p) for p in prompts):
        raise ValueError("a prompt is empty")
    if not all(0 <= t < vocab for p in prompts for t in p):
        raise ValueError(f"token numbers are 0 to {vocab - 1}")
    if not 0 <= drafted < state.cfg.max_draft:
        raise ValueError(f"drafted is 0 to {state.cfg.max_draft - 1}: a call runs the last token too")
    start = torch.tensor([0] + [len(p) for p in prompts], device=device).cumsum(0).to(torch.int32)
    probs = model.prefill(torch.tensor([t for p in prompts for t in p], device=device), start)
    last = torch.multinomial(probs[start[1:].long() - 1], 1, generator=rng).to(torch.int32)  # [batch, 1]
    new = [[t] for t in last[:, 0].tolist()]
    calls = 1
    while min(len(n) for n in new) < count:
        chain, rows = [last], []
        for _ in range(drafted):
            rows.append(model.drafts[chain[-1][:, 0].long()])
            chain.append(torch.multinomial(rows[-1], 1, generator=rng).to(torch.int32))
        tokens = torch.cat(chain, 1)
        target = model.tokens(tokens, drafts=True)
        uniforms = torch.rand((batch, drafted + 1), generator=rng, device=device)
        accepted, following = ops.accept_drafts(tokens[:, 1:].contiguous(), target, uniforms,
                                                draft=torch.stack(rows, 1) if rows else None)
        model.commit(accepted + 1)  # the last token itself and the drafts that were kept
        for n, kept, row, after in zip(new, accepted.tolist(), tokens[:, 1:].tolist(), following.tolist()):
            n += row[:kept] + [after]
        last = following[:, None]
        calls += 1
    return new, calls


def main(argv=None) -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--prompt", type=int, default=200, help="tokens of the longest prompt")
    p.add_argument("--tokens", type=int, default=64, help="new tokens of each sequence")
    p.add_argument("--drafted", type=int, default=4, help="drafts of each call (0..7)")
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    if a.batch < 1 or a.prompt < 1 or a.tokens < 1 or not 0 <= a.drafted <= 7:
        p.error("batch, prompt and tokens are at least 1, drafted is 0 to 7")
    model = Model(batch=a.batch, seed=a.seed)
    rng = torch.Generator(device="cuda")
    rng.manual_seed(a.seed + 1)
    lengths = [max(1, a.prompt - 7 * i) for i in range(a.batch)]
    prompts = [torch.randint(model.embed.shape[0], (n,), generator=rng, device="cuda").tolist() for n in lengths]
    t0 = time.perf_counter()
    new, calls = generate(model, prompts, a.tokens, a.drafted, rng)
    print(f"{sum(map(len, new))} tokens of {a.batch} sequences in {calls} calls, {time.perf_counter() - t0:.2f} s")
    for i, n in enumerate(new):
        print(f"sequence {i}: prompt of {lengths[i]}, then {n[:16]}{' ...' if len(n) > 16 else ''}")


if __name__ == "__main__":
    main()
