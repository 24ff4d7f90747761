"""Log probabilities, entropy and the largest words against their definition in float64."""
import numpy as np
import pytest

from _gpu import announce
from _scan import U, _dev, values
from oracle import layer_ops as L

pytestmark = pytest.mark.gpu
INF, LOWEST = np.inf, np.finfo(np.float32).min


def _check(x, tokens, top):
    import torch
    from hybrid_model_ssm_replay_amd import ops
    logits = x if isinstance(x, torch.Tensor) else _dev(np.asarray(x, np.float32))
    toks = torch.tensor(np.asarray(tokens), dtype=torch.int32, device="cuda")
    got = [values(t) for t in ops.token_logprobs(logits, toks, top=top)]
    want = L.token_logprobs(values(logits), tokens, top)
    rows, V = logits.shape
    # A sum of V weights in lanes of at most V / 256 + 64 additions; an exponent d has a rounding of its own and
    # of its product with log2 e, 2 |d| U of the weight, largest where e^d d is: below 1, and 2 U of the
    # exponential; the logarithm 2 U, the difference one.  Each sum relative to itself, so its logarithm absolutely.
    sums = (V / 256 + 64 + 8) * U
    live = np.isfinite(want[0])
    assert np.array_equal(live, np.isfinite(got[0])) and (got[0][~live] == -INF).all()
    bars = sums + 4 * U * np.abs(np.where(live, want[0], 0)) + 4 * U * np.log(V + 1)
    assert (np.abs(got[0][live] - want[0][live]) <= bars[live]).all(), np.abs(got[0][live] - want[0][live]).max()
    # entropy: log s - t / s, of t the same roundings on terms that add up to at most the entropy and log V
    assert (np.abs(got[1] - want[1]) <= 3 * sums * (1 + np.log(V + 1))).all(), np.abs(got[1] - want[1]).max()
    assert np.array_equal(got[3], want[3])
    live = np.isfinite(want[2])
    assert (got[2][~live] == -INF).all()
    assert (np.abs(got[2][live] - want[2][live]) <= (sums + 4 * U * np.abs(want[2][live]) + 4 * U * np.log(V + 1))).all()


@pytest.mark.parametrize("rows,V", [(1, 1), (2, 3), (1, 64), (5, 63), (3, 513), (1, 2048), (2, 2049), (1, 10000), (7, 5003), (1, 131072),
                                    (40, 50021), (300, 3000), (2100, 700)])
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
def test_token_logprobs(rows, V, name, top):
    announce("token_logprobs", rows, V, name, top)
    r = np.random.default_rng(rows + V + top)
    x = _dev((3.0 * r.normal(size=(rows, V))).astype(np.float32), name)
    _check(x, r.integers(0, V, rows), top)


@pytest.mark.parametrize("V", [9, 700, 2500, 30000])
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["rising", "falling", "equal", "steps", "one large", "masked", "all but one masked", "lowest", "large", "spread"])
def test_orders_ties_and_masks(V, name, kind):
    announce("token_logprobs", V, name, kind)
    r = np.random.default_rng(V)
    i = np.arange(V)
    x = {"rising": i * 0.01, "falling": -i * 0.01, "equal": 0 * i + 1.5, "steps": (i // 7) % 5 * 1.0, "one large": np.where(i == V // 2, 80.0, 0.0),
         "masked": np.where(r.random(V) < 0.7, -INF, r.normal(size=V)), "all but one masked": np.where(i == V - 1, 2.0, -INF),
         "lowest": np.where(r.random(V) < 0.5, LOWEST, r.normal(size=V)), "large": 1e30 * r.normal(size=V), "spread": 40.0 * r.normal(size=V)}[kind]
    rows = np.stack([x, np.roll(x, 3), x[::-1]]).astype(np.float32)
    _check(_dev(rows, name), [0, V - 1, V // 2], 20)


@pytest.mark.parametrize("V", [5, 700, 30000])
def test_rows_without_weight_nan_infinity_and_tokens_outside(V):
    import torch
    announce("token_logprobs specials", V)
    x = np.random.default_rng(1).normal(size=(9, V)).astype(np.float32)
    x[0] = -INF                               # nothing left
    x[1] = LOWEST                             # all at the lowest: even
    x[2, 1::2] = np.nan
    x[3, 2] = INF
    x[4, [1, 3]] = INF
    x[5] = np.nan
    x[6] = np.where(np.arange(V) == 0, LOWEST, -INF)
    _check(x, [0, 1, 1, 2, 3, 0, 0, -1, V], 4)
    for name in (torch.float32, torch.bfloat16):
        _check(torch.from_numpy(x).to(name).cuda(), [0, 1, 0, 1, 1, 0, 1, V + 5, -7], 3)


def test_strided_and_repeated_rows():
    import torch
    announce("token_logprobs strides")
    wide = torch.randn(6, 2 * 3001, device="cuda").bfloat16()
    _check(wide[:, 1:3002], np.arange(6) * 500, 3)
    _check(wide[::2, :2999], [0, 1, 2], 3)
    _check(torch.randn(1, 1000, device="cuda").expand(4, 1000), [1, 2, 3, 4], 3)


def test_more_rows_than_one_slice_each_and_none():
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("token_logprobs rows")
    out = ops.token_logprobs(torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), top=3)
    assert [tuple(t.shape) for t in out] == [(0,), (0,), (0, 3), (0, 3)]
    x = torch.randn(1500, 2100, device="cuda")  # more than 2048 workgroups of 2048 words: whole rows
    tok = torch.randint(0, 2100, (1500,), device="cuda", dtype=torch.int32)
    whole = ops.token_logprobs(x, tok, top=7)
    few = ops.token_logprobs(x[:5], tok[:5], top=7)  # cut in two
    assert torch.equal(whole[3][:5], few[3])
    for a, b in zip(whole[:3], few[:3]):
        assert float((a[:5] - b).abs().max()) <= 80 * U * 20


def test_replays_and_streams_give_the_same_bits():
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("token_logprobs graph")
    x, tok = torch.randn(3, 20000, device="cuda"), torch.tensor([5, 19999, 7], dtype=torch.int32, device="cuda")
    ops.token_logprobs(x, tok, top=20)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ops.token_logprobs(x, tok, top=20)
    side = torch.cuda.Stream()
    for _ in range(3):
        x.mul_(1.25)
        want = ops.token_logprobs(x, tok, top=20)
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = ops.token_logprobs(x, tok, top=20)
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, other):
            assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("V,stride,first", [(1, 3, 1), (2, 3, 1), (8, 9, 0), (7, 15, 2), (2047, 2049, 1), (2048, 2049, 0), (2048, 2051, 1),
                                            (4096, 4097, 1), (5003, 5003, 0), (50021, 50023, 1), (131072, 131073, 1)])
@pytest.mark.parametrize("around", [np.nan, INF, 1e30])
@pytest.mark.parametrize("rows", [3, 9])
def test_what_is_between_the_rows_counts_for_nothing(V, stride, first, around, rows):
    """Rows that start between two words, slices and their ends, the values around them large or no numbers."""
    import torch
    announce("token_logprobs between", V, stride, first, around, rows)
    r = np.random.default_rng(V + stride + rows)
    flat = torch.full((rows * stride + 9,), float(around), device="cuda", dtype=torch.bfloat16)
    x = torch.as_strided(flat, (rows, V), (stride, 1), first)
    x.copy_(_dev((3.0 * r.normal(size=(rows, V))).astype(np.float32), "bf16"))
    for top in (0, 5):
        _check(x, r.integers(0, V, rows), top)


@pytest.mark.parametrize("V", [7, 1000, 9001])
@pytest.mark.parametrize("first", [0, 1])
def test_rows_that_repeat_one_from_between_two_words(V, first):
    """Stride 0 from an even and an odd element of bf16, alone and as part of every row: nothing before them is theirs."""
    import torch
    announce("token_logprobs repeated", V, first)
    r = np.random.default_rng(V)
    flat = torch.full((V + 9,), float("nan"), device="cuda", dtype=torch.bfloat16)
    row = flat[first:first + V]
    row.copy_(_dev((3.0 * r.normal(size=V)).astype(np.float32), "bf16"))
    for top in (0, 5):
        _check(row.expand(4, V), [0, V - 1, V // 2, 3], top)
        _check(torch.as_strided(flat, (3, V - 2), (1, 1), first), [0, V - 3, 2], top)  # each row a value further on
