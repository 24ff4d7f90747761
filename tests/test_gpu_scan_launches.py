"""The prompt scan in every launch shape, each named by the library's own plan of the call.

Prompts are whole or cut, the segments of cut ones add up where they start or have
that done by a launch, and a wave holds 16 or 32 columns of x.  Every case asserts
which of these it is, so that a threshold that moves cannot take the cases off a kernel.

Bars, u = 2^-24, s the size of an output's terms (see the scan's bars beside the other
operators): f = (N + 64 + 112 + 4 (n / 64 + 1)) u s for float32 outputs and the state;
bf16 outputs: e (1 + 2^-8) + 2^-8 |y| with e = f + 2^-16 s (two pieces of weights and
state, each rounded to nearest).

And of the root mean squares, the state and float32 outputs within 2^-20: roundings of u
have either sign and add in quadrature, and 256 of them, more than the accumulations of
a value over its decay, are 16 u.  A piece less of any factor is 2^-16 of its terms.
"""
import numpy as np
import pytest

from _gpu import announce
from _scan import HALF, U, Prompts, near

pytestmark = pytest.mark.gpu
TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]


def _plan(H, G, P, N, tokens, n, batch, name):
    from hybrid_model_ssm_replay_amd import binding as B
    cfg = B.make_config(B.KIND_MAMBA2, batch, H, G, P, N, 1, flags=B.FLAG_BF16_RECORDS if name == "bf16" else 0)
    got = B.replay_scan_plan(cfg, tokens, n)
    return got.segment, bool(got.adds), got.columns, got.workgroups


def _rms(a):
    return float(np.sqrt(np.mean(np.concatenate([v.ravel() for v in a]) ** 2)))


def _check(p, N, out):
    y, state = p.run(out)
    off, val = {"y": [], "S": []}, {"y": [], "S": []}
    for i, s, want, S, size, Sa in p.exact():
        f = (N + 64 + 112 + 4 * (p.lens[i] / 64 + 1)) * U
        e = (f + (2.0 ** -16 if out == "bf16" else 0.0)) * size
        near(y[s], want, e * (1 + HALF[out]) + HALF[out] * np.abs(want) + 1e-37)
        near(state[p.rows[i]], S, f * Sa + U * np.abs(S) + 1e-37)
        for k, got, exact in (("y", y[s], want), ("S", state[p.rows[i]], S)):
            off[k].append(got - exact)
            val[k].append(exact)
    for k in ("S", "y") if out == "f32" else ("S",):
        assert _rms(off[k]) <= 2.0 ** -20 * _rms(val[k]), (k, _rms(off[k]) / _rms(val[k]))
    for b in set(range(p.batch)) - set(p.rows.tolist()):
        assert (state[b] == 5).all()


def _ragged(n, most, seed):
    return [int(v) for v in np.random.default_rng(seed).integers(0, most + 1, n)]


# Three heads a group: workgroups of two heads have one left over, and heads of 48, 80
# and 112 columns a last wave with one tile of its two.
SHAPES = [(16, 64), (32, 16), (48, 128), (64, 128), (80, 32), (112, 64), (128, 128)]


@pytest.mark.parametrize("name,out", TYPES)
@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("mode", ["whole", "adds", "launch"])
def test_waves_of_32_columns(mode, P, N, name, out):
    announce("scan launches", mode, P, N, name, out)
    G, H = 4, 12
    lens = {"whole": [65, 130] + _ragged(138, 4, P), "adds": [200, 192, 0, 193] + _ragged(66 if P < 48 else 26, 1, P),
            "launch": [300, 257, 0, 128, 129] + _ragged(65 if P < 48 else 25, 3, P)}[mode]
    known = [int(v) for v in np.random.default_rng(P + N).integers(0, 2, len(lens))]
    p = Prompts(H, G, P, N, lens, known, name)
    segment, adds, columns, groups = _plan(H, G, P, N, p.tokens, len(lens), p.batch, name)
    assert columns == 32 and groups > 256 and (segment > 0) == (mode != "whole") and (segment == 0 or adds == (mode == "adds"))
    assert mode == "whole" or max(lens) > segment
    _check(p, N, out)


@pytest.mark.parametrize("name,out", TYPES)
@pytest.mark.parametrize("P,N", SHAPES)
@pytest.mark.parametrize("lens", [[70, 3, 0, 129], [330, 2, 200], [500, 300, 40]])
def test_waves_of_16_columns(P, N, name, out, lens):
    announce("scan launches", P, N, name, out, lens)
    p = Prompts(6, 2, P, N, lens, "all", name)
    segment, adds, columns, groups = _plan(6, 2, P, N, p.tokens, len(lens), p.batch, name)
    assert columns == 16 and (segment > 0) == (sum(lens) > 300) and (segment == 0 or adds == (sum(lens) < 600))
    _check(p, N, out)


@pytest.mark.parametrize("tokens,segment,adds", [(320, 0, False), (321, 128, True), (512, 128, True), (513, 192, True),
                                                 (768, 192, True), (769, 128, False)])
@pytest.mark.parametrize("H,G,P,N,name,out", [(2, 1, 64, 128, "bf16", "bf16"), (4, 2, 48, 64, "bf16", "f32"), (2, 2, 128, 16, "f32", "f32")])
def test_around_the_lengths_at_which_prompts_are_cut(tokens, segment, adds, H, G, P, N, name, out):
    announce("scan cuts", tokens, H, G, P, N, name, out)
    for lens in ([tokens], [tokens - 130, 130]):
        p = Prompts(H, G, P, N, lens, "all", name, lead=0, tail=0)
        assert _plan(H, G, P, N, p.tokens, len(lens), p.batch, name)[:2] == (segment, adds)
        _check(p, N, out)


@pytest.mark.parametrize("lens", [(8192,), (5000, 2900, 100)])
def test_in_place_where_more_segments_add_up_than_the_card_holds(lens):
    """Segments that wait for a place read where their sequence starts after its last segment has written the state."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("scan in place, segments that add up", lens)
    H, G, P, N, n = 256, 8, 64, 128, sum(lens)
    segment, adds, columns, groups = _plan(H, G, P, N, n, len(lens), len(lens), "bf16")
    assert segment and adds and max(lens) > segment and groups > 512
    torch.manual_seed(3)
    rand = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, Bm, Cm, dt = rand(n, H, P), rand(n, G, N), rand(n, G, N), torch.rand(n, H, device="cuda") * 0.01
    A, D = -torch.rand(H, device="cuda"), torch.randn(H, device="cuda")
    seq = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    start = torch.randn(len(lens), H, P, N, device="cuda")
    apart, place = torch.empty_like(start), start.clone()
    y0 = ops.scan_prompt(x, Bm, Cm, dt, A, D, seq, apart, initial=start)
    y1 = ops.scan_prompt(x, Bm, Cm, dt, A, D, seq, place, initial=place)
    assert torch.equal(y0, y1) and torch.equal(apart, place)
