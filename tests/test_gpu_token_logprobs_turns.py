"""Log probabilities of calls with so many rows that a workgroup works on a row, or on a long slice, in several turns."""
import numpy as np
import pytest

from _gpu import announce
from _scan import U, _dev, values
from oracle import layer_ops as L

pytestmark = pytest.mark.gpu
INF, LOWEST = np.inf, np.finfo(np.float32).min
TURN = 4096  # words that a workgroup reads at a time


def _compare(x, tokens, top, some, want):
    """Rows `some` of a call's results beside `want`, the oracle's."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    V = x.shape[1]
    got = ops.token_logprobs(x, torch.tensor(np.asarray(tokens), dtype=torch.int32, device="cuda"), top=top)
    got = [values(t)[some] for t in got]
    # A lane adds V / 256 weights of a row at most and joins fewer than 64 others (the lanes, the waves and 16
    # slices a lane).  A turn in which the maximum grows scales the sum: a product, and an exponential whose
    # argument's roundings are those of the weight itself, counted with it: 2 |d| U of a weight e^d (|d| e^d is below
    # 1) and 2 U.  The logarithm 2 U, the difference one.
    sums = (V / 256 + 64 + 8 + 4 * (V / TURN + 1)) * U
    size = 4 * U * np.log(V + 1)
    live = np.isfinite(want[0])
    assert (got[0][~live] == -INF).all() and np.isfinite(got[0][live]).all()
    assert (np.abs(got[0][live] - want[0][live]) <= sums + 4 * U * np.abs(want[0][live]) + size).all()
    assert (np.abs(got[1] - want[1]) <= 3 * sums * (1 + np.log(V + 1))).all(), np.abs(got[1] - want[1]).max()
    assert np.array_equal(got[3], want[3])
    live = np.isfinite(want[2])
    assert (got[2][~live] == -INF).all()
    assert (np.abs(got[2][live] - want[2][live]) <= sums + 4 * U * np.abs(want[2][live]) + size).all()


# Whole rows of two to four turns, of an even and an odd vocabulary; slices of 16384 and of 4096 words that are joined.
SHAPES = [(1030, 9001), (1100, 12289), (1026, 8192), (256, 50021), (100, 30000)]


@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("top", [0, 5, 32])
def test_rows_of_several_turns(rows, V, name, top):
    announce("token_logprobs turns", rows, V, name, top)
    r = np.random.default_rng(rows + V + top)
    x = _dev((3.0 * r.normal(size=(rows, V))).astype(np.float32), name)
    tokens = r.integers(0, V, rows)
    some = np.unique(np.concatenate([[0, 1, 2, rows - 2, rows - 1], r.integers(0, rows, 60)]))
    _compare(x, tokens, top, some, L.token_logprobs(values(x[some.tolist()]), tokens[some], top))


def _patterns(V):
    """Orders, ties, masks and values that are no numbers, a row each."""
    r, i = np.random.default_rng(V), np.arange(V)
    rows = [i * 0.01, -i * 0.01, 0 * i + 1.5, (i // 7) % 5 * 1.0, (i // 1000) * 1.0, np.where(i == V // 2, 80.0, 0.0),
            np.where(i == V - 1, 2.0, -INF), np.where(r.random(V) < 0.7, -INF, r.normal(size=V)),
            np.where(r.random(V) < 0.5, LOWEST, r.normal(size=V)), 1e30 * r.normal(size=V), 40.0 * r.normal(size=V), r.normal(size=V),
            np.full(V, -INF), np.full(V, np.nan), np.full(V, LOWEST), np.where(i % 2 == 1, np.nan, r.normal(size=V)),
            np.where(i < V - 3, -INF, 1.0), np.where((i == 2) | (i == V - 2), INF, r.normal(size=V)), np.where(i > V // 2, i * 0.01, -INF)]
    return np.stack(rows).astype(np.float32)


@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("top", [0, 5, 32])
def test_orders_ties_masks_and_no_numbers_over_several_turns(rows, V, name, top):
    import torch
    announce("token_logprobs turns, patterns", rows, V, name, top)
    base = _dev(_patterns(V), name)
    n, r = len(base), np.random.default_rng(top)
    which = r.permutation(np.arange(rows) % n)  # each pattern in many places, and so at both parities of an odd vocabulary
    tokens = r.integers(0, V, n)[which]
    tokens[:3] = -1, V, V + 70000
    some = np.unique(np.concatenate([[0, 1, 2, rows - 1], [np.nonzero(which == p)[0][k] for p in range(n) for k in (0, 1, -1)]]))
    x = base[torch.from_numpy(which).cuda()]
    _compare(x, tokens, top, some, L.token_logprobs(values(x[some.tolist()]), tokens[some], top))


def test_rows_whose_offsets_pass_32_bits():
    """The last rows start behind 2^32 bytes, then 2^32 values."""
    import torch
    announce("token_logprobs far rows")
    V, r = 5001, np.random.default_rng(0)
    for stride in ((1 << 30) + 1, (1 << 31) + 3):
        flat = torch.empty(2 * stride + V, device="cuda", dtype=torch.bfloat16)
        x = torch.as_strided(flat, (3, V), (stride, 1), 0)
        x.copy_(_dev((3.0 * r.normal(size=(3, V))).astype(np.float32), "bf16"))
        tokens = r.integers(0, V, 3)
        _compare(x, tokens, 5, np.arange(3), L.token_logprobs(values(x), tokens, 5))
        del flat, x
