"""Short convolution, prompt scan, gated norm and draft acceptance against their float64 definitions.

Bars, with u = 2^-24 (half a float32 step) and r = the half step of the output
type (bf16: 2^-8; float32: u), all relative to the value or to the size of the
terms that a sum adds:

* convolution: K + 1 roundings of a sum whose terms have size s, carried through
  silu (slope at most 1.1); silu itself: exponential, sum, reciprocal, product
  (8 u) and the argument's rounding inside the exponential (2 |v| u).
* scan: an output adds N + Q products of size s in float32 blocks (Q = 64 tokens
  of a stretch); every weight is a product of at most four exponentials with
  arguments of at most 24 where the weight is above 2^-24 of its term, each
  rounded (4 (24 + 4) u), and a state passes n / 64 stretches.  So
  (N + 64 + 112 + 4 n / 64) u s.  With bf16 outputs the two factors that enter
  the matrix products besides the inputs may be bf16 themselves: 2^-8 s each.
* norm: the sum of squares has relative error (group + 4) u and enters under a
  root (half of it), then silu twice (2 (8 + 2 |z|) u) and four products.
* acceptance: whole numbers, equal.
"""
import numpy as np
import pytest

from _gpu import announce, host
from oracle import layer_ops as L

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _dev(a, name="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(_dt(name) if a.dtype.kind == "f" else None).cuda()


def _values(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _near(got, want, bar):
    got, bad = np.asarray(got, np.float64), ~(np.abs(got - want) <= bar)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} values off, the worst {np.max(np.abs(got - want) / np.maximum(bar, 1e-300)):.2f} "
                           f"times its bar, first at {np.argwhere(bad)[0]}")


# ---- short convolution ---------------------------------------------------------------
def _conv_bar(v, size, y, K, act, name):
    return (1.1 * (K + 1) * size + (8 + 2 * np.abs(v)) * np.abs(y) * act) * U + HALF[name] * np.abs(y) + 1e-37


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("K,widths,batch,T,act,bias,wide", [
    (4, (64, 16, 16), 3, 1, True, True, True),
    (4, (64, 16, 16), 5, 8, True, False, False),
    (2, (7, 1, 5), 2, 3, False, True, False),
    (3, (513,), 1, 1, True, True, True),
    (4, (4096, 2048), 2, 2, True, True, True),
    (4, (0, 24, 8), 4, 16, False, False, True),
])
def test_short_conv_step(name, K, widths, batch, T, act, bias, wide):
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("short_conv_step", name, K, widths, batch, T, act, bias, wide)
    r = np.random.default_rng(K * 1000 + batch)
    C, slots = sum(widths), K - 1 + T + (3 if wide else 0)
    proj = _dev(r.normal(size=(batch, T, C + (24 if wide else 3))).astype(np.float32), name)
    off = 16 if wide else 2
    x = proj[..., off:off + C]
    w, b = r.normal(size=(C, K)).astype(np.float32), r.normal(size=C).astype(np.float32)
    ring0 = _dev(r.normal(size=(slots, batch, C)).astype(np.float32), name)
    pos = r.integers(0, 1 << 30, batch).astype(np.int32)
    pos[0] = 0  # a sequence at its first token: history slots below position 0 wrap
    ring = ring0.clone()
    outs = ops.short_conv_step(x, _dev(w), ring, _dev(pos), widths, bias=_dev(b) if bias else None,
                               activation="silu" if act else None)
    torch.cuda.synchronize()
    xs, old, new = _values(x), _values(ring0), _values(ring)
    want_ring = old.copy()
    assert [tuple(o.shape) for o in outs] == [(batch, T, k) for k in widths]
    got = np.concatenate([_values(o) for o in outs], -1)
    for i in range(batch):
        hist = np.stack([old[(int(pos[i]) - k) % slots, i] for k in range(K - 1, 0, -1)])
        y, v, size, _ = L.short_conv(xs[i], w, b if bias else None, hist, act)
        _near(got[i], y, _conv_bar(v, size, y, K, act, name))
        for t in range(T):
            want_ring[(int(pos[i]) + t) % slots, i] = xs[i, t]
    np.testing.assert_array_equal(new, want_ring)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("K,widths,lens,resumed,wide", [
    (4, (64, 16, 16), [1], [0], True),
    (4, (64, 16, 16), [2, 0, 1, 3, 31, 32, 33], [1, 1, 0, 0, 1, 0, 1], True),
    (4, (2056, 8), [0, 100, 0, 5], None, True),
    (3, (5, 2), [40, 1, 1, 64], [1, 1, 0, 1], False),
    (2, (129,), [0, 0], [1, 0], False),
    (4, (16, 16, 16), [1, 1, 1, 1, 1, 1, 1, 1], [1, 0, 1, 0, 1, 0, 1, 0], True),
])
def test_short_conv_prompt(name, K, widths, lens, resumed, wide):
    """Ragged prompts, some empty or shorter than the taps; rows of NaN around the
    packed ones and stale NaN in rings that are not resumed must not be seen."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("short_conv_prompt", name, K, widths, lens, resumed, wide)
    r = np.random.default_rng(len(lens) * 100 + K)
    C, n, batch, slots, lead, tail = sum(widths), len(lens), len(lens) + 2, K + 4, 3, 2
    tokens = lead + sum(lens) + tail
    xs = r.normal(size=(tokens, C)).astype(np.float32)
    xs[:lead], xs[tokens - tail:] = np.nan, np.nan
    buf = _dev(np.concatenate([xs, np.full((tokens, 8 if wide else 1), np.nan, np.float32)], 1), name)
    x = buf[:, :C]
    start = lead + np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = r.permutation(batch)[:n].astype(np.int32)
    pos = r.integers(0, 1000, batch).astype(np.int32)
    w, b = r.normal(size=(C, K)).astype(np.float32), r.normal(size=C).astype(np.float32)
    ring0 = r.normal(size=(slots, batch, C)).astype(np.float32)
    for i in range(n):
        if resumed is None or not resumed[i]:
            ring0[:, rows[i]] = np.nan
    ring0 = _dev(ring0, name)
    ring = ring0.clone()
    res = None if resumed is None else _dev(np.array(resumed, np.uint8))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = ops.short_conv_prompt(x, _dev(w), ring, _dev(start), widths, bias=_dev(b), rows=_dev(rows), pos=_dev(pos),
                                 resume=res, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    got, xv, old, new = np.concatenate([_values(o) for o in outs], -1), _values(x), _values(ring0), _values(ring)
    want = old.copy()
    for i in range(n):
        at = [(int(pos[rows[i]]) - k) % slots for k in range(K - 1, 0, -1)]
        hist = old[at, rows[i]] if resumed is not None and resumed[i] else None
        y, v, size, last = L.short_conv(xv[start[i]:start[i + 1]], w, b, hist)
        _near(got[start[i]:start[i + 1]], y, _conv_bar(v, size, y, K, True, name))
        want[at, rows[i]] = last
    np.testing.assert_array_equal(new, want)


def test_short_conv_prompt_then_steps_is_one_prompt():
    """A prompt, then drafts of which a part is kept, then a step: the outputs of the whole sequence at once."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("short_conv prompt, drafts, step")
    r = np.random.default_rng(5)
    C, K, n = 32, 4, 20
    x, w = _dev(r.normal(size=(n, C)).astype(np.float32)), _dev(r.normal(size=(C, K)).astype(np.float32))
    one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ring = torch.zeros(K - 1 + 6, 1, C, device="cuda")
    whole, = ops.short_conv_prompt(x, w, ring.clone(), one, (C,))
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    first, = ops.short_conv_prompt(x[:7], w, ring, torch.tensor([0, 7], dtype=torch.int32, device="cuda"), (C,), pos=pos)
    assert torch.equal(first, whole[:7])
    at = 7
    for kept in (2, 0, 6, 1):
        drafts = torch.cat([x[at:at + kept], torch.full((6 - kept, C), 9.0, device="cuda")])[None]
        y, = ops.short_conv_step(drafts, w, ring, pos, (C,))
        assert torch.equal(y[0, :kept], whole[at:at + kept])
        pos += kept
        at += kept
    y, = ops.short_conv_step(x[None, at:at + 1].contiguous(), w, ring, pos, (C,))
    assert torch.equal(y[0, 0], whole[at])


def test_bad_rows_and_positions_are_skipped_and_flagged():
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    announce("bad rows")
    C, K = 16, 4
    x, w = torch.ones(6, C, device="cuda"), torch.ones(C, K, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ring, status = torch.zeros(8, 2, C, device="cuda"), i32([0])
    ops.short_conv_prompt(x, w, ring, i32([0, 3, 6]), (C,), rows=i32([1, 2]), status=status)
    assert int(status) == B.STATUS_BAD_PROMPT
    assert torch.equal(ring[:, 0], torch.zeros(8, C, device="cuda")) and int((ring[:, 1] != 0).sum()) == 3 * C
    status.zero_()
    before = ring.clone()
    ops.short_conv_step(torch.ones(2, 1, C, device="cuda"), w, ring, i32([0, -1]), (C,), status=status)
    assert int(status) == B.STATUS_BAD_POINTERS and torch.equal(ring[:, 1], before[:, 1])
    state = torch.full((2, 2, 16, 16), 7.0, device="cuda")
    status.zero_()
    ops.scan_prompt(torch.ones(6, 2, 16, device="cuda"), torch.ones(6, 1, 16, device="cuda"), torch.ones(6, 1, 16, device="cuda"),
                    torch.ones(6, 2, device="cuda"), -torch.ones(2, device="cuda"), torch.ones(2, device="cuda"), i32([0, 3, 6]),
                    state, rows=i32([-1, 0]), status=status)
    assert int(status) == B.STATUS_BAD_PROMPT
    assert bool((state[1] == 7).all()) and not bool((state[0] == 7).any())
    # Offsets outside the packed rows are clamped, never followed.
    y, = ops.short_conv_prompt(x, w, ring, i32([0, 100]), (C,))
    assert torch.isfinite(y).all()


# ---- prompt scan ------------------------------------------------------------------------
def _scan_bars(size, n, N, name, out):
    rough = 2 * 2.0 ** -8 if out == "bf16" else 0.0
    return (N + 64 + 112 + 4 * (n / 64 + 1)) * U + rough


SCANS = [
    # H, G, P, N, lengths, resumed (None: no initial; "all": every one), in, out
    (4, 2, 64, 128, [1], None, "bf16", "f32"),
    (4, 1, 64, 128, [64, 65, 63], "all", "bf16", "bf16"),
    (4, 4, 64, 128, [0, 3, 130, 0, 200, 17], [1, 1, 0, 0, 1, 1], "bf16", "f32"),
    (2, 1, 16, 16, [5, 70], [0, 1], "f32", "f32"),
    (6, 2, 48, 32, [33, 100], "all", "f32", "f32"),
    (3, 1, 80, 64, [129], None, "bf16", "bf16"),
    (7, 7, 128, 128, [31, 97], "all", "bf16", "f32"),
    (2, 2, 128, 64, [190], [1], "f32", "f32"),
    (5, 1, 112, 16, [65], None, "bf16", "f32"),
    (2, 1, 32, 128, [700], [1], "bf16", "bf16"),
    (2, 1, 64, 128, [1500, 20], [1, 0], "f32", "f32"),
    (8, 2, 64, 64, [2100], None, "bf16", "f32"),
]


@pytest.mark.parametrize("H,G,P,N,lens,resumed,name,out", SCANS)
def test_scan_prompt(H, G, P, N, lens, resumed, name, out):
    """Against the recurrence token by token; NaN in the rows between and around the
    sequences and in states that are not resumed must not be seen."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("scan_prompt", H, G, P, N, lens, resumed, name, out)
    r = np.random.default_rng(H * 1000 + P + N)
    n, batch, lead, tail = len(lens), len(lens) + 2, 5, 4
    tokens = lead + sum(lens) + tail

    def field(*shape):
        a = r.normal(size=(tokens,) + shape).astype(np.float32)
        a[:lead], a[tokens - tail:] = np.nan, np.nan
        return a

    x, Bm, Cm = _dev(field(H, P), name), _dev(field(G, N), name), _dev(field(G, N), name)
    dt = np.log1p(np.exp(field(H) - 2.0)).astype(np.float32)
    A, D = -np.exp(r.uniform(0, np.log(16), H)).astype(np.float32), r.normal(size=H).astype(np.float32)
    start = lead + np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = r.permutation(batch)[:n].astype(np.int32)
    known = [0] * n if resumed is None else [1] * n if resumed == "all" else resumed
    init = r.normal(size=(batch, H, P, N)).astype(np.float32)
    for i in range(n):
        if not known[i]:
            init[rows[i]] = np.nan
    state = torch.full((batch, H, P, N), 5.0, device="cuda")
    y = ops.scan_prompt(x, Bm, Cm, _dev(dt), _dev(A), _dev(D), _dev(start), state,
                        initial=None if resumed is None else _dev(init), rows=_dev(rows),
                        resume=_dev(np.array(known, np.uint8)) if isinstance(resumed, list) else None, out_dtype=_dt(out))
    torch.cuda.synchronize()
    yv, sv = _values(y), _values(state)
    xv, Bv, Cv = _values(x), _values(Bm), _values(Cm)
    for i in range(n):
        s = slice(start[i], start[i + 1])
        want, S, size, Sa = L.scan(xv[s], Bv[s], Cv[s], dt[s], A, D, init[rows[i]] if known[i] else None)
        k = _scan_bars(size, lens[i], N, name, out)
        _near(yv[s], want, k * size + HALF[out] * np.abs(want) + 1e-37)
        _near(sv[rows[i]], S, _scan_bars(Sa, lens[i], N, name, "f32") * Sa + 1e-37)
    for b in set(range(batch)) - set(rows.tolist()):
        assert bool((state[b] == 5).all())


@pytest.mark.parametrize("H,G,P,N,lens,resumed,name,out", [
    # A token around each length at which a prompt is cut, and pieces of exactly that length.
    (2, 1, 64, 128, [256], "all", "bf16", "bf16"),
    (2, 1, 64, 128, [257], [1], "bf16", "f32"),
    (2, 1, 64, 128, [320], [1], "bf16", "f32"),
    (2, 1, 64, 128, [321], [1], "bf16", "bf16"),
    (2, 1, 64, 128, [384], "all", "bf16", "bf16"),
    (2, 1, 64, 128, [385], None, "f32", "f32"),
    (4, 2, 48, 64, [512], [1], "bf16", "bf16"),        # four segments add up their starts
    (4, 2, 48, 64, [513], [1], "bf16", "bf16"),        # five: the states are combined apart
    (4, 2, 48, 64, [768], [1], "bf16", "bf16"),
    (4, 2, 48, 64, [769], [1], "bf16", "bf16"),
    (4, 2, 64, 128, [1000, 3, 400, 0, 128, 129], [1, 0, 0, 1, 1, 0], "bf16", "bf16"),
    (2, 2, 128, 16, [600, 130, 256], [0, 1, 1], "f32", "f32"),
    (64, 8, 64, 128, [640, 130], "all", "bf16", "f32"),
])
def test_scan_prompt_around_its_cuts(H, G, P, N, lens, resumed, name, out):
    test_scan_prompt(H, G, P, N, lens, resumed, name, out)


def test_scan_prompt_long_steps_and_fast_decay():
    """Heads whose decay over one token underflows, and heads that hardly decay."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("scan_prompt decay extremes")
    r = np.random.default_rng(9)
    H, G, P, N, n = 4, 2, 64, 128, 200
    x, Bm, Cm = (_dev(r.normal(size=s).astype(np.float32), "bf16") for s in ((n, H, P), (n, G, N), (n, G, N)))
    dt = np.abs(r.normal(size=(n, H))).astype(np.float32) * np.array([40.0, 1e-4, 0.0, 1.0], np.float32)
    A, D = -np.array([16.0, 1.0, 4.0, 90.0], np.float32), np.zeros(H, np.float32)
    init = r.normal(size=(1, H, P, N)).astype(np.float32)
    state = torch.empty(1, H, P, N, device="cuda")
    seq = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    y = ops.scan_prompt(x, Bm, Cm, _dev(dt), _dev(A), _dev(D), seq, state, initial=_dev(init))
    want, S, size, Sa = L.scan(_values(x), _values(Bm), _values(Cm), dt, A, D, init[0])
    _near(_values(y), want, _scan_bars(size, n, N, "bf16", "f32") * size + 1e-37)
    _near(_values(state[0]), S, _scan_bars(Sa, n, N, "bf16", "f32") * Sa + 1e-37)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("cuts", [[100, 300], [64, 64], [1, 500]])
def test_scan_prompt_in_place_continues(name, cuts):
    """A prompt in two calls, the second from the state in place, against the definition."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("scan_prompt in place", name, cuts)
    r = np.random.default_rng(11)
    H, G, P, N, n = 4, 2, 64, 128, sum(cuts)
    x, Bm, Cm = (_dev(r.normal(size=s).astype(np.float32), name) for s in ((n, H, P), (n, G, N), (n, G, N)))
    dt = np.log1p(np.exp(r.normal(size=(n, H)) - 2)).astype(np.float32)
    A, D = -np.exp(r.uniform(0, 2.7, H)).astype(np.float32), r.normal(size=H).astype(np.float32)
    state = torch.full((1, H, P, N), float("nan"), device="cuda")
    got = []
    for a, b in ((0, cuts[0]), (cuts[0], n)):
        seq = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        got.append(ops.scan_prompt(x[a:b], Bm[a:b], Cm[a:b], _dev(dt[a:b]), _dev(A), _dev(D), seq, state,
                                   initial=state if a else None))
    want, S, size, Sa = L.scan(_values(x), _values(Bm), _values(Cm), dt, A, D)
    _near(_values(torch.cat(got)), want, _scan_bars(size, n, N, name, "f32") * size + 1e-37)
    _near(_values(state[0]), S, _scan_bars(Sa, n, N, name, "f32") * Sa + 1e-37)


@pytest.mark.parametrize("G,lens", [(8, (1400, 100, 1500)), (1, (900, 1100, 30, 970)), (8, (8000,)), (8, (700, 90)),
                                    (8, (6000, 100, 2500, 3000))])
def test_scan_prompt_in_place_is_bit_equal_where_segments_outnumber_the_card(G, lens):
    """Segments that read where their sequence starts must not meet the state that its last one leaves."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("scan_prompt in place, wide", G, lens)
    torch.manual_seed(3)
    H, P, N, n = 128, 64, 128, sum(lens)
    rand = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, Bm, Cm, dt = rand(n, H, P), rand(n, G, N), rand(n, G, N), torch.rand(n, H, device="cuda") * 0.01
    A, D = -torch.rand(H, device="cuda"), torch.randn(H, device="cuda")
    seq = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    start = torch.randn(len(lens), H, P, N, device="cuda")
    apart, place = torch.empty_like(start), start.clone()
    y0 = ops.scan_prompt(x, Bm, Cm, dt, A, D, seq, apart, initial=start)
    y1 = ops.scan_prompt(x, Bm, Cm, dt, A, D, seq, place, initial=place)
    assert torch.equal(y0, y1) and torch.equal(apart, place)


def test_scan_prompt_bad_values_stay_in_their_sequence():
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("scan_prompt NaN and inf")
    H, G, P, N = 2, 1, 64, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    n = 150
    x, Bm, Cm = mk(n, H, P), mk(n, G, N), mk(n, G, N)
    dt = torch.full((n, H), 0.1, device="cuda")
    seq = torch.tensor([0, 50, 100, 150], dtype=torch.int32, device="cuda")
    A, D = -torch.ones(H, device="cuda"), torch.ones(H, device="cuda")
    s0, s1 = torch.zeros(3, H, P, N, device="cuda"), torch.zeros(3, H, P, N, device="cuda")
    y0 = ops.scan_prompt(x, Bm, Cm, dt, A, D, seq, s0)
    x[60, 0], Bm[70] = float("inf"), float("nan")
    y1 = ops.scan_prompt(x, Bm, Cm, dt, A, D, seq, s1)
    for a, b in ((0, 50), (100, 150)):
        assert torch.equal(y0[a:b], y1[a:b])
    assert torch.equal(s0[0], s1[0]) and torch.equal(s0[2], s1[2]) and not torch.isfinite(s1[1]).all()


def test_scan_prompt_runs_are_equal_and_a_long_prompt_split_gives_the_same_bits_twice():
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("scan_prompt determinism")
    g = torch.Generator(device="cuda").manual_seed(4)
    H, G, P, N, n = 8, 2, 64, 128, 3000
    x, Bm, Cm = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((n, H, P), (n, G, N), (n, G, N)))
    dt, A, D = torch.rand(n, H, generator=g, device="cuda"), -torch.rand(H, generator=g, device="cuda"), torch.ones(H, device="cuda")
    seq = torch.tensor([0, 900, 3000], dtype=torch.int32, device="cuda")
    runs = []
    for _ in range(2):
        st = torch.empty(2, H, P, N, device="cuda")
        runs.append((ops.scan_prompt(x, Bm, Cm, dt, A, D, seq, st), st))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


# ---- gated norm --------------------------------------------------------------------------
@pytest.mark.parametrize("ty,tz,to", [("f32", "bf16", "bf16"), ("bf16", "bf16", "bf16"), ("f32", "f32", "f32"),
                                      ("bf16", "f32", "f32")])
@pytest.mark.parametrize("T,C,group,shared,first,pad", [
    (1, 8, 8, False, False, 0), (3, 4096, 128, True, True, 8), (5, 2048, 1024, False, False, 16), (2, 21, 7, False, True, 1),
    (4, 99, 33, True, False, 2), (2, 8192, 8192, False, False, 0), (1, 1, 1, False, False, 0), (7, 520, 40, True, True, 8),
    (2, 4800, 2400, False, True, 0), (3, 20000, 20000, False, False, 0)])
def test_gated_norm(ty, tz, to, T, C, group, shared, first, pad):
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("gated_norm", ty, tz, to, T, C, group, shared, first, pad)
    r = np.random.default_rng(C + group)
    y = _dev(r.normal(size=(T, C + pad)).astype(np.float32), ty)[:, :C]
    z = _dev(3 * r.normal(size=(T, C + 2 * pad)).astype(np.float32), tz)[:, pad:pad + C]
    w = r.normal(size=group if shared else C).astype(np.float32)
    out = ops.gated_norm(y, z, _dev(w), group, eps=1e-5, norm_first=first, out_dtype=_dt(to))
    torch.cuda.synchronize()
    want = L.gated_norm(_values(y), _values(z), w, group, 1e-5, first)
    _near(_values(out), want, (((group + 4) / 2 + 2 * (8 + 2 * np.abs(_values(z)).max()) + 6) * U + HALF[to]) * np.abs(want) + 1e-37)


def test_gated_norm_of_zeros_and_of_rows_that_repeat():
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("gated_norm zeros")
    y, z, w = torch.zeros(2, 64, device="cuda"), torch.randn(2, 64, device="cuda"), torch.ones(64, device="cuda")
    assert not ops.gated_norm(y, z, w, 16).any()
    one = torch.randn(1, 64, device="cuda")
    out = ops.gated_norm(one.expand(5, 64), z[:1].expand(5, 64), w, 16)
    assert torch.equal(out, out[:1].expand(5, 64)) and ops.gated_norm(y[:0], z[:0], w, 16).shape == (0, 64)


# ---- draft acceptance ---------------------------------------------------------------------
@pytest.mark.parametrize("name,qname", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", None), ("bf16", None)])
@pytest.mark.parametrize("batch,T,V,pad", [(1, 4, 1000, 0), (5, 1, 7, 1), (9, 8, 5003, 5), (3, 3, 65536, 0), (2, 0, 300, 0),
                                           (4, 2, 1, 0), (17, 16, 64, 8)])
def test_accept_drafts(name, qname, batch, T, V, pad):
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("accept_drafts", name, qname, batch, T, V, pad)
    r = np.random.default_rng(V + T)
    base = r.normal(size=(batch, 1, V))

    def probs(rows):
        e = np.exp(base + 0.3 * r.normal(size=(batch, rows, V)))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)

    target = _dev(np.concatenate([probs(T + 1), np.full((batch, T + 1, pad), np.nan, np.float32)], -1), name)[..., :V]
    draft = _dev(probs(max(T, 1))[:, :T], qname) if qname else None
    tokens = r.integers(0, V, (batch, T)).astype(np.int32)
    lengths = r.integers(0, T + 1, batch).astype(np.int32)
    lengths[0] = T
    u = r.uniform(size=(batch, T + 1)).astype(np.float32)
    u[:, :T] *= 0.9
    u[0, T] = 0.0
    acc, nxt = ops.accept_drafts(_dev(tokens), target, _dev(u), draft=draft, lengths=_dev(lengths))
    torch.cuda.synchronize()
    tv, qv = _values(target), _values(draft) if qname else None
    for b in range(batch):
        want = L.accept(tokens[b], tv[b], u[b], None if qv is None else qv[b], lengths[b])
        assert (int(acc[b]), int(nxt[b])) == want, (b, want)


def test_accept_drafts_edges():
    """No weight anywhere, NaN and negative entries, a residual without weight, u at the ends, bad tokens."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("accept_drafts edges")
    V, nan = 700, float("nan")
    p, q = np.zeros((8, 2, V), np.float32), np.zeros((8, 1, V), np.float32)
    tok, u = np.zeros((8, 1), np.int32), np.full((8, 2), 0.5, np.float32)
    p[1, 0, [3, 650]], q[1, 0, [3, 650]] = 0.5, 0.5             # p = q: refused only by u = 1, then p itself
    tok[1], u[1] = 3, [1.0, 0.9]
    p[2, 0, :], p[2, 0, 5], p[2, 0, 6] = nan, 0.25, -3.0          # only one entry has weight
    tok[2] = 9
    p[3, :, 10], p[3, :, 699], tok[3], u[3] = 0.5, 0.5, -1, [0.0, 0.999]
    p[4, :, 0], p[4, :, 699], tok[4], u[4] = 0.5, 0.5, V, [0.0, 1.0]
    p[5, 0, 8], q[5, 0, 8], p[5, 1, 100], tok[5], u[5] = 1.0, 1.0, 1.0, 8, [0.999, 0.0]
    p[6, 0, :4], q[6, 0, 0], tok[6] = 0.25, 1.0, 0
    p[7, 0, 1], q[7, 0, :], tok[7] = 1.0, nan, 1
    acc, nxt = ops.accept_drafts(_dev(tok), _dev(p), _dev(u), draft=_dev(q))
    got = list(zip(host(acc).tolist(), host(nxt).tolist()))
    want = [L.accept(tok[b], p[b], u[b], q[b]) for b in range(8)]
    assert got == want
    assert want[0] == (0, -1) and want[1] == (0, 650) and want[2] == (0, 5) and want[5] == (1, 100)


# ---- streams and graphs ---------------------------------------------------------------------
def test_operators_in_a_captured_graph_on_another_stream():
    """One layer's operators captured on a side stream; every replay equals the eager run."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("layer operators in a graph")
    H, G, P, N, K, n, V = 4, 2, 64, 128, 4, 300, 1003
    g = torch.Generator(device="cuda").manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    widths = (H * P, G * N, G * N)
    C = sum(widths)
    xin, z, w, seq = mk(n, C).bfloat16(), mk(n, H * P).bfloat16(), mk(C, K), torch.tensor([0, 120, n], dtype=torch.int32, device="cuda")
    dt, A, D, nw = torch.rand(n, H, generator=g, device="cuda"), -torch.ones(H, device="cuda"), mk(H), mk(H * P)
    p, q = torch.softmax(mk(2, 4, V), -1), torch.softmax(mk(2, 3, V), -1)
    tok, u = torch.randint(0, V, (2, 3), generator=g, device="cuda", dtype=torch.int32), torch.rand(2, 4, generator=g, device="cuda")
    ring, state = torch.zeros(8, 2, C, device="cuda").bfloat16(), torch.zeros(2, H, P, N, device="cuda")

    def layer():
        x, b, c = ops.short_conv_prompt(xin, w, ring, seq, widths)
        y = ops.scan_prompt(x.view(n, H, P), b.view(n, G, N), c.view(n, G, N), dt, A, D, seq, state, out_dtype=torch.bfloat16)
        o = ops.gated_norm(y.view(n, H * P), z, nw, H * P // G)
        return [o, *ops.accept_drafts(tok, p, u, draft=q)]

    want = [t.clone() for t in layer()]
    want_state = state.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = layer()
    for _ in range(4):
        state.zero_()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.relu(torch.randn(1000, device="cuda")).sum().item()  # the program's own work between replays
        assert eager > 0 and all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(state, want_state)
