"""Inputs, one call and the float64 definition of a prompt scan (no arithmetic of the path here)."""
import numpy as np

from oracle import layer_ops as L

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _dev(a, name="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(_dt(name) if a.dtype.kind == "f" else None).cuda()


def values(t):
    return t.detach().double().cpu().numpy()


class Prompts:
    """Ragged prompts of one layer; NaN in the rows around them and in states that are not resumed.

    resumed: None (no initial state), "all", or a flag for each sequence."""

    def __init__(self, H, G, P, N, lens, resumed, name, seed=0, lead=5, tail=4, spare=2):
        r = np.random.default_rng(seed + H * 1000 + P + N)
        self.lens, self.name, self.resumed = lens, name, resumed
        n, self.batch = len(lens), len(lens) + spare
        self.tokens = lead + sum(lens) + tail
        self.start = lead + np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.rows = r.permutation(self.batch)[:n].astype(np.int32)
        self.known = [0] * n if resumed is None else [1] * n if resumed == "all" else list(resumed)

        def field(*shape):
            a = r.normal(size=(self.tokens,) + shape).astype(np.float32)
            a[:lead], a[self.tokens - tail:] = np.nan, np.nan
            return a

        self.x, self.B, self.C = (_dev(field(*s), name) for s in ((H, P), (G, N), (G, N)))
        self.dt = np.log1p(np.exp(field(H) - 2.0)).astype(np.float32)
        self.A, self.D = -np.exp(r.uniform(0, np.log(16), H)).astype(np.float32), r.normal(size=H).astype(np.float32)
        self.init = r.normal(size=(self.batch, H, P, N)).astype(np.float32)
        for i in range(n):
            if not self.known[i]:
                self.init[self.rows[i]] = np.nan
        self.shape = (H, P, N)

    def run(self, out):
        """y [tokens, H, P] and state [batch, H, P, N] as float64 arrays; unwritten states are 5."""
        import torch
        from hybrid_model_ssm_replay_amd import ops
        state = torch.full((self.batch,) + self.shape, 5.0, device="cuda")
        y = ops.scan_prompt(self.x, self.B, self.C, _dev(self.dt), _dev(self.A), _dev(self.D), _dev(self.start), state,
                            initial=None if self.resumed is None else _dev(self.init), rows=_dev(self.rows),
                            resume=_dev(np.array(self.known, np.uint8)) if isinstance(self.resumed, list) else None,
                            out_dtype=_dt(out))
        torch.cuda.synchronize()
        return values(y), values(state)

    def exact(self):
        """For each sequence: its rows, then y, S and the sizes of the terms of both (see the oracle)."""
        x, B, C = values(self.x), values(self.B), values(self.C)
        for i, n in enumerate(self.lens):
            s = slice(self.start[i], self.start[i] + n)
            yield (i, s) + L.scan(x[s], B[s], C[s], self.dt[s], self.A, self.D, self.init[self.rows[i]] if self.known[i] else None)


def near(got, want, bar):
    bad = ~(np.abs(got - want) <= bar)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} values off, the worst "
                           f"{np.max(np.abs(got - want) / np.maximum(bar, 1e-300)):.2f} times its bar, first at {np.argwhere(bad)[0]}")
