"""A small model of Mamba-2 or Gated DeltaNet layers that serves prompts, decode steps and drafted tokens.

``Mixer`` is one Mamba-2 layer as it is served: input projection, short
convolution, recurrence, gated norm, output projection, on the operators of
``ops`` and the state of a ``layer.ReplayLayer``; ``DeltaMixer`` is a Gated
DeltaNet one.  ``Model`` stacks mixers between an embedding and a head (random
weights), ``generate`` samples from it with drafts of a bigram table, and
``score`` says how likely it finds the tokens of prompts.  The projections are
torch products; nearly everything in between is the library's.

    python -m hybrid_model_ssm_replay_amd.generate --batch 4 --prompt 200 --tokens 64
    python -m hybrid_model_ssm_replay_amd.generate --kind gdn --top 3
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


class DeltaMixer(Mixer):
    """The same for Gated DeltaNet: q, k and v through the convolution, q and k of length 1,
    gates alpha and beta of each head, a norm over each head before the gate."""

    def __init__(self, width, heads, head_dim, state_dim, batch, window=16, max_draft=8, taps=4, dtype=torch.bfloat16,
                 rng=None, device="cuda"):
        inner, keys = heads * head_dim, heads * state_dim
        self.heads, self.head_dim, self.state_dim = heads, head_dim, state_dim
        self.inner, self.widths = inner, (keys, keys, inner)
        channels = 2 * keys + inner

        def normal(*shape, scale=1.0):
            return torch.randn(shape, generator=rng, device=device) * scale

        self.w_in = normal(width, inner + channels + 2 * heads, scale=width ** -0.5).to(dtype)
        self.w_out = normal(inner, width, scale=inner ** -0.5).to(dtype)
        self.w_conv, self.b_conv = normal(channels, taps, scale=taps ** -0.5), normal(channels, scale=0.1)
        self.rate = -torch.exp(normal(heads) - 1.0)
        self.w_norm = 1.0 + normal(head_dim, scale=0.1)
        self.state = ReplayLayer("gdn", batch, heads, head_dim, state_dim, window, max_draft=max_draft, device=device,
                                 flags=B.FLAG_BF16_RECORDS if dtype == torch.bfloat16 else 0)
        self.ring = torch.zeros((taps - 1 + max(1, max_draft), batch, channels), dtype=dtype, device=device)

    def _split(self, h):
        z, qkv, a, b = torch.split(h @ self.w_in, (self.inner, sum(self.widths), self.heads, self.heads), dim=-1)
        return z, qkv, (torch.exp(self.rate * F.softplus(a.float())), torch.sigmoid(b.float()))

    def _record(self, q, k, v, gates):
        lead = q.shape[:-1]
        q, k = (F.normalize(t.view(*lead, self.heads, self.state_dim).float(), dim=-1).to(t.dtype) for t in (q, k))
        return {"q": q, "k": k, "v": v.view(*lead, self.heads, self.head_dim), "alpha": gates[0], "beta": gates[1]}

    def _out(self, y, z):
        return ops.gated_norm(y.flatten(1), z, self.w_norm, self.head_dim, norm_first=True) @ self.w_out


class Model:
    """Embedding, ``layers`` mixers (kind "mamba2" or "gdn") on a residual stream, head.  The
    norms of a GDN model have weights, and add to the stream what the layer before them made."""

    def __init__(self, vocab=512, width=256, layers=2, batch=4, seed=0, dtype=torch.bfloat16, device="cuda", kind="mamba2", **mixer):
        if kind not in ("mamba2", "gdn"):
            raise ValueError(f"unknown kind {kind!r}")
        rng = torch.Generator(device=device)
        rng.manual_seed(seed)
        shape = dict(heads=8, head_dim=64, state_dim=64, **({"groups": 2} if kind == "mamba2" else {}))
        shape.update(mixer)
        self.embed = torch.randn((vocab, width), generator=rng, device=device).to(dtype)
        self.head = (torch.randn((width, vocab), generator=rng, device=device) * 1.5 * width ** -0.5).to(dtype)
        mixers = {"mamba2": Mixer, "gdn": DeltaMixer}[kind]
        self.mixers = [mixers(width, batch=batch, dtype=dtype, rng=rng, device=device, **shape) for _ in range(layers)]
        self.drafts = torch.softmax(torch.randn((vocab, vocab), generator=rng, device=device), -1)  # row: token before
        self.norms = None if kind == "mamba2" else [1.0 + 0.1 * torch.randn(width, generator=rng, device=device)
                                                    for _ in range(layers + 1)]

    def _logits(self, tokens, run):
        """The layers, each as run(mixer, its input), and the head."""
        h = self.embed[tokens.long()]
        if self.norms is None:
            for m in self.mixers:
                h = h + run(m, F.rms_norm(h, h.shape[-1:]))
            return F.rms_norm(h, h.shape[-1:]) @ self.head
        lead = h.shape[:-1]
        n, stream = ops.residual_norm(h.flatten(0, -2), None, self.norms[0])
        for m, w in zip(self.mixers, self.norms[1:]):
            n, stream = ops.residual_norm(run(m, n.view(*lead, -1)).flatten(0, -2), stream, w)
        return n.view(*lead, -1) @ self.head

    def logits(self, tokens, seq_start, rows=None, resume=None):
        """Packed prompt tokens [tokens]: the logits after each."""
        return self._logits(tokens, lambda m, n: m.prefill(n, seq_start, rows, resume))

    def prefill(self, tokens, seq_start, rows=None, resume=None):
        """Packed prompt tokens [tokens]: the distribution after each."""
        return torch.softmax(self.logits(tokens, seq_start, rows, resume).float(), -1)

    def tokens(self, tokens, drafts):
        """tokens [batch, T]: the distribution after each (see ``Mixer.tokens``)."""
        return torch.softmax(self._logits(tokens, lambda m, n: m.tokens(n, drafts)).float(), -1)

    def commit(self, accepted):
        for m in self.mixers:
            m.commit(accepted)


def _packed(model, prompts):
    """The prompts' tokens one after the other, and where each starts."""
    device, vocab = model.embed.device, model.embed.shape[0]
    if len(prompts) != model.mixers[0].state.shapes.batch:
        raise ValueError(f"{len(prompts)} prompts for {model.mixers[0].state.shapes.batch} sequences")
    if not all(len(p) for p in prompts):
        raise ValueError("a prompt is empty")
    if not all(0 <= t < vocab for p in prompts for t in p):
        raise ValueError(f"token numbers are 0 to {vocab - 1}")
    start = torch.tensor([0] + [len(p) for p in prompts], device=device).cumsum(0).to(torch.int32)
    return torch.tensor([t for p in prompts for t in p], device=device), start


def score(model, prompts, top=0):
    """How likely the model finds each prompt's tokens, given those before them (the first is
    given): for each prompt a list of (log probability, entropy, [(word, its log probability),
    ...] of the ``top`` words, 0 to 32) for its second token, third token, ...  Prompts as for
    ``generate``.  The model's sequences start anew, and are left behind their prompts' last tokens."""
    tokens, start = _packed(model, prompts)
    if not 0 <= top <= B.MAX_TOP:
        raise ValueError(f"top is 0 to {B.MAX_TOP}")
    following = torch.cat([tokens[1:], tokens[:1]]).to(torch.int32)
    following[start[1:].long() - 1] = -1  # nothing follows a prompt's last token
    got = ops.token_logprobs(model.logits(tokens, start), following, top=top)
    rows = list(zip(*(t.tolist() for t in got)))
    at, out = 0, []
    for p in prompts:
        out.append([(lp, entropy, list(zip(words, best))) for lp, entropy, best, words in rows[at:at + len(p) - 1]])
        at += len(p)
    return out


def generate(model, prompts, count, drafted=4, rng=None):
    """At least ``count`` new tokens behind each prompt (lists of at least one token
    number, one for every sequence of the model).  Returns the new tokens, a list for each prompt, and
    how many calls of the model made them.

    Each call runs the last token and ``drafted`` drafts; the drafts are drawn from the
    model's bigram table, and the kept tokens follow the model's own distribution."""
    device, batch, most = model.embed.device, len(prompts), model.mixers[0].state.cfg.max_draft
    tokens, start = _packed(model, prompts)
    if not 0 <= drafted < most:
        raise ValueError(f"drafted is 0 to {most - 1}: a call runs the last token too")
    probs = model.prefill(tokens, start)
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
    p.add_argument("--kind", choices=("mamba2", "gdn"), default="mamba2", help="layers of the model")
    p.add_argument("--top", type=int, default=0, help="score the prompts too, with so many alternatives of the last token (0: no scores)")
    a = p.parse_args(argv)
    if not 0 <= a.top <= 32:
        p.error("top is 0 to 32")
    if a.batch < 1 or a.prompt < 1 or a.tokens < 1 or not 0 <= a.drafted <= 7:
        p.error("batch, prompt and tokens are at least 1, drafted is 0 to 7")
    model = Model(batch=a.batch, seed=a.seed, kind=a.kind)
    rng = torch.Generator(device="cuda")
    rng.manual_seed(a.seed + 1)
    lengths = [max(1, a.prompt - 7 * i) for i in range(a.batch)]
    prompts = [torch.randint(model.embed.shape[0], (n,), generator=rng, device="cuda").tolist() for n in lengths]
    if a.top:
        for i, tokens in enumerate(score(model, prompts, a.top)):
            if tokens:
                mean, last = sum(t[0] for t in tokens) / len(tokens), tokens[-1]
                print(f"prompt {i}: {mean:.3f} a token; instead of the last "
                      + ", ".join(f"{word} ({lp:.3f})" for word, lp in last[2]) + f" (entropy {last[1]:.3f})")
    t0 = time.perf_counter()
    new, calls = generate(model, prompts, a.tokens, a.drafted, rng)
    print(f"{sum(map(len, new))} tokens of {a.batch} sequences in {calls} calls, {time.perf_counter() - t0:.2f} s")
    for i, n in enumerate(new):
        print(f"sequence {i}: prompt of {lengths[i]}, then {n[:16]}{' ...' if len(n) > 16 else ''}")


if __name__ == "__main__":
    main()
