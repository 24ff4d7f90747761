"""Inputs, one call and the float64 definition of a Gated DeltaNet prompt (no arithmetic of the path here)."""
import numpy as np

from _scan import HALF, U, _dev, _dt, near, values
from oracle import layer_ops as L


def unit(a):
    return a / np.maximum(np.sqrt((a * a).sum(-1, keepdims=True)), 1e-30)


class DeltaPrompts:
    """Ragged prompts of one layer; NaN in the rows around them and in states that are not resumed.

    resumed: None (no initial state), "all", or a flag for each sequence."""

    def __init__(self, H, P, N, lens, resumed, name, seed=0, lead=5, tail=4, spare=2):
        r = np.random.default_rng(seed + H * 1000 + P + N)
        self.lens, self.name, self.resumed = lens, name, resumed
        n, self.batch = len(lens), len(lens) + spare
        self.lead, self.tail, self.tokens = lead, tail, lead + sum(lens) + tail
        self.start = lead + np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.rows = r.permutation(self.batch)[:n].astype(np.int32)
        self.known = [0] * n if resumed is None else [1] * n if resumed == "all" else list(resumed)
        self.q, self.k = (unit(r.normal(size=(self.tokens, H, N))).astype(np.float32) for _ in range(2))
        self.v = r.normal(size=(self.tokens, H, P)).astype(np.float32)
        rate = np.exp(r.uniform(np.log(0.01), np.log(4.0), H))
        self.alpha = np.exp(-rate * np.log1p(np.exp(r.normal(size=(self.tokens, H))))).astype(np.float32)
        self.beta = (1.0 / (1.0 + np.exp(-r.normal(size=(self.tokens, H))))).astype(np.float32)
        self.init = r.normal(size=(self.batch, H, P, N)).astype(np.float32)
        for i in range(n):
            if not self.known[i]:
                self.init[self.rows[i]] = np.nan
        self.shape = (H, P, N)

    def surround(self):
        """NaN in every row outside the sequences."""
        for a in (self.q, self.k, self.v, self.alpha, self.beta):
            a[:self.lead] = np.nan
            a[self.tokens - self.tail:] = np.nan
        return self

    def tensors(self):
        return [_dev(a, self.name) for a in (self.q, self.k, self.v)] + [_dev(self.alpha), _dev(self.beta)]

    def run(self, out):
        """y [tokens, H, P] and state [batch, H, P, N] as float64 arrays; unwritten states are 5."""
        import torch
        from hybrid_model_ssm_replay_amd import ops
        state = torch.full((self.batch,) + self.shape, 5.0, device="cuda")
        y = ops.delta_prompt(*self.tensors(), _dev(self.start), state, initial=None if self.resumed is None else _dev(self.init),
                             rows=_dev(self.rows), resume=_dev(np.array(self.known, np.uint8)) if isinstance(self.resumed, list) else None,
                             out_dtype=_dt(out))
        torch.cuda.synchronize()
        return values(y), values(state)

    def exact(self):
        """For each sequence: its index and rows, then o, S and size of the oracle."""
        import torch
        q, k, v = (torch.from_numpy(a).to(_dt(self.name)).double().numpy() for a in (self.q, self.k, self.v))
        for i, n in enumerate(self.lens):
            s = slice(self.start[i], self.start[i] + n)
            yield (i, s) + L.delta(q[s], k[s], v[s], self.alpha[s], self.beta[s], self.init[self.rows[i]] if self.known[i] else None)


def bar(N):
    """Roundings that a value can carry, each at most U of the size of what is summed: a product with
    the state (N terms), the substitution and its product (64 each), the output's (64), the weights'
    and pieces' own (48).  What earlier chunks left is not added: the rows of the state shrink."""
    return (N + 64 + 64 + 64 + 48) * U


# Roundings of random sign: fewer than 256 of a value, each uniform within a step of U, leave
# sqrt(256 / 3) U = 9.2 U in the 2-norm where the terms are no larger than their sum; 16 leaves
# room for terms that cancel.
TOGETHER = 16 * U


def check(p, out, y, state):
    H, P, N = p.shape
    errors = [[], []]
    for i, s, o, S, size in p.exact():
        # bf16 outputs: their own rounding, and before it 2^-16 of each term for S and for U.
        rough = 2 * 2.0 ** -16 if out == "bf16" else 0.0
        near(y[s], o, (bar(N) + rough) * size + HALF[out] * np.abs(o) + 1e-37)
        near(state[p.rows[i]], S, bar(N) * size[..., None] + 1e-37)
        if p.lens[i]:
            errors[0].append((y[s] - o, o))
        errors[1].append((state[p.rows[i]] - S, S))
    for kind, e in zip(("f32" if out == "f32" else None, "f32"), errors):
        off, all_ = (np.sqrt(sum((a[j] ** 2).sum() for a in e)) for j in (0, 1))
        assert kind is None or off <= TOGETHER * all_, f"{off / all_:.3e} of the result"
    for b in set(range(p.batch)) - set(p.rows.tolist()):
        assert (state[b] == 5).all()
