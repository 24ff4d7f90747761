"""Prompts of Gated DeltaNet layers against the recurrence token by token, in float64."""
import numpy as np
import pytest

from _delta import DeltaPrompts, check
from _gpu import announce
from _scan import values

pytestmark = pytest.mark.gpu

CASES = [
    # H, P, N, lengths, resumed (None: no initial; "all": every one), in, out
    (1, 16, 16, [1], None, "bf16", "f32"),
    (4, 128, 128, [37], "all", "bf16", "bf16"),
    (4, 64, 128, [64, 65, 63], "all", "bf16", "bf16"),
    (3, 128, 128, [0, 3, 130, 0, 200, 17], [1, 1, 0, 0, 1, 1], "bf16", "f32"),
    (2, 16, 16, [5, 70], [0, 1], "f32", "f32"),
    (6, 48, 32, [33, 100], "all", "f32", "f32"),
    (3, 80, 64, [129], None, "bf16", "bf16"),
    (7, 128, 128, [31, 97], "all", "bf16", "f32"),
    (2, 128, 64, [190], [1], "f32", "f32"),
    (5, 112, 16, [65], None, "bf16", "f32"),
    (2, 32, 128, [700], [1], "bf16", "bf16"),
    (2, 128, 128, [500, 20], [1, 0], "f32", "f32"),
    (8, 64, 64, [1100], None, "bf16", "f32"),
    (9, 32, 128, [64] * 9, [1, 0] * 4 + [1], "bf16", "bf16"),
    (33, 16, 32, [128, 1, 2, 3], "all", "f32", "f32"),
]


@pytest.mark.parametrize("H,P,N,lens,resumed,name,out", CASES)
def test_delta_prompt(H, P, N, lens, resumed, name, out):
    announce("delta_prompt", H, P, N, lens, resumed, name, out)
    p = DeltaPrompts(H, P, N, lens, resumed, name).surround()
    check(p, out, *p.run(out))


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["same keys", "few keys", "alpha 0", "alpha 1", "tiny alpha", "beta 0", "beta 2", "zero keys"])
def test_delta_prompt_extremes(name, what):
    """Keys that are alike (the powers of T grow, its inverse does not), gates at the ends of their ranges."""
    announce("delta_prompt extremes", name, what)
    p = DeltaPrompts(4, 32, 64, [150, 70], "all", name, seed=3)
    r = np.random.default_rng(5)
    if what == "same keys":
        p.k[:], p.beta[:], p.alpha[:] = p.k[:1], 1.0, 1.0
    elif what == "few keys":
        p.k[:] = p.k[r.integers(0, 3, p.tokens)]
    elif what == "alpha 0":
        p.alpha[r.random(p.alpha.shape) < 0.1] = 0.0
    elif what == "alpha 1":
        p.alpha[:] = 1.0
    elif what == "tiny alpha":
        p.alpha[r.random(p.alpha.shape) < 0.3] = 1e-38
    elif what == "beta 0":
        p.beta[r.random(p.beta.shape) < 0.5] = 0.0
    elif what == "beta 2":
        p.beta[:] = 2.0
    else:
        p.k[r.random(p.tokens) < 0.5] = 0.0
        p.q[r.random(p.tokens) < 0.2] = 0.0
    if name == "bf16" and what in ("same keys", "beta 2"):  # bf16 keys are longer than 1 by up to 2^-8: shrink them
        p.k *= np.float32(1 - 2.0 ** -7)
    p.surround()
    check(p, "f32", *p.run("f32"))


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("cuts", [[100, 300], [64, 64], [1, 300]])
def test_delta_prompt_in_place_continues(name, cuts):
    """A prompt in two calls, the second from the state in place, against the definition."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("delta_prompt in place", name, cuts)
    p = DeltaPrompts(4, 64, 128, [sum(cuts)], None, name, lead=0, tail=0, spare=0)
    t = p.tensors()
    state = torch.full((1,) + p.shape, float("nan"), device="cuda")
    got = []
    for a, b in ((0, cuts[0]), (cuts[0], sum(cuts))):
        seq = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        got.append(ops.delta_prompt(*[x[a:b] for x in t], seq, state, initial=state if a else None))
    check(p, "f32", values(torch.cat(got)), values(state))


@pytest.mark.parametrize("lens", [(12032,), (64, 11000, 320, 9000, 30), (11008, 11008)])
def test_delta_prompt_in_several_passes_is_bit_equal_to_calls_of_whole_chunks(lens):
    """More chunks than one pass holds; a call of each 64 k tokens has the same chunks, one pass each."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("delta_prompt passes", lens)
    H, N, P, tokens = 32, 128, 32, sum(lens)
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k = (torch.nn.functional.normalize(rand(tokens, H, N), dim=-1).bfloat16() for _ in range(2))
    v, alpha, beta = rand(tokens, H, P).bfloat16(), torch.rand(tokens, H, generator=g, device="cuda"), torch.rand(
        tokens, H, generator=g, device="cuda")
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    init = rand(len(lens), H, P, N)
    state = init.clone()
    y = ops.delta_prompt(q, k, v, alpha, beta, torch.tensor(start, dtype=torch.int32, device="cuda"), state, initial=state)
    want, parts = init.clone(), []
    for i, n in enumerate(lens):
        for a in range(start[i], start[i + 1], 4096):
            b = min(a + 4096, start[i + 1])
            parts.append(ops.delta_prompt(*[t[a:b] for t in (q, k, v, alpha, beta)],
                                          torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), want, initial=want,
                                          rows=torch.tensor([i], dtype=torch.int32, device="cuda")))
    assert torch.equal(y, torch.cat(parts)) and torch.equal(state, want)


def test_bad_rows_are_skipped_and_flagged_and_offsets_clamped():
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    announce("delta_prompt bad rows")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    one = torch.ones(6, 2, 16, device="cuda")
    gate = torch.full((6, 2), 0.5, device="cuda")
    state, status = torch.full((2, 2, 16, 16), 7.0, device="cuda"), i32([0])
    ops.delta_prompt(one, one, one, gate, gate, i32([0, 3, 6]), state, rows=i32([-1, 0]), status=status)
    assert int(status) == B.STATUS_BAD_PROMPT
    assert bool((state[1] == 7).all()) and not bool((state[0] == 7).any())
    for start in ([0, 100], [-5, 6], [4, 2], [0, 5, 2], [6, 0, 6]):  # clamped, never followed outside; decreasing: empty
        n = len(start) - 1
        ops.delta_prompt(one, one, one, gate, gate, i32(start), state[:n].contiguous() if n < 3 else state)
    torch.cuda.synchronize()


def test_a_nan_stays_in_its_sequence_and_head():
    announce("delta_prompt NaN")
    p = DeltaPrompts(3, 32, 64, [90, 80, 70], "all", "bf16", lead=0, tail=0, spare=0)
    clean, states = p.run("f32")
    p.v[100, 1, 3] = np.nan                          # the second sequence, head 1
    y, state = p.run("f32")
    hit = np.zeros(p.tokens, bool)
    hit[90:170] = True
    assert np.array_equal(y[~hit], clean[~hit]) and np.array_equal(y[:, [0, 2]], clean[:, [0, 2]])
    assert np.isnan(y[100, 1, 3]) and np.isnan(y[169, 1, 3])
    assert np.array_equal(state[p.rows[[0, 2]]], states[p.rows[[0, 2]]])


@pytest.mark.parametrize("steps", [1, 5])
def test_steps_continue_a_prompt(steps):
    """replay_step from the state that a prompt leaves is the recurrence's next tokens."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer
    announce("steps after a delta prompt", steps)
    n = 70
    p = DeltaPrompts(4, 64, 64, [n + steps], None, "f32", lead=0, tail=0, spare=0)
    t = p.tensors()
    lay = ReplayLayer("gdn", 1, 4, 64, 64, 4)
    got = [ops.delta_prompt(*[x[:n] for x in t], torch.tensor([0, n], dtype=torch.int32, device="cuda"), lay.checkpoint)]
    for i in range(n, n + steps):
        got.append(lay.step(dict(zip(("q", "k", "v", "alpha", "beta"), (x[i:i + 1] for x in t)))))
    lay.flush()
    check(p, "f32", values(torch.cat(got)), values(lay.checkpoint))



@pytest.mark.parametrize("flags", [0, 2])
@pytest.mark.parametrize("rows,lens,resume", [([3], [70], None), ([4, 0], [5, 130], [1, 0]), ([2], [0], None), (None, [9, 40], [0, 1]),
                                              (None, [3, 1, 2, 60, 20], [1, 1, 0, 1, 1])])
@pytest.mark.parametrize("rf", ["FMT_F32", "FMT_F4E2M1_B16", "FMT_F4E2M1_CS"])
def test_prefill_of_a_layer_with_records_in_its_windows(flags, rows, lens, resume, rf):
    """Prompted rows: the prompt over the flushed state, in both copies; the others keep their bits."""
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer
    announce("gdn prefill", flags, rows, lens, resume, rf)
    H, P, N, batch = 4, 64, 128, 5
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    vec = torch.bfloat16 if flags else torch.float32
    unit = lambda *s: torch.nn.functional.normalize(rand(*s), dim=-1).to(vec)  # noqa: E731
    rec = lambda *n: {"q": unit(*n, H, N), "k": unit(*n, H, N), "v": rand(*n, H, P).to(vec),  # noqa: E731
                      "alpha": torch.exp(-rand(*n, H).abs() * 0.1), "beta": torch.sigmoid(rand(*n, H))}
    lay, ref = (ReplayLayer("gdn", batch, H, P, N, 4, max_draft=2, read_fmt=getattr(B, rf), flags=flags) for _ in range(2))
    begin = rand(batch, H, P, N)
    steps = [rec(batch) for _ in range(6)]  # past a fold, then two records in every window
    for layer in (lay, ref):
        layer.set_state(begin)
        for r in steps:
            layer.step(r)
    mine = list(range(len(lens))) if rows is None else rows
    others = [b for b in range(batch) if b not in mine]
    start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    prompt, at = rec(sum(lens)), None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    known = None if resume is None else torch.tensor(resume, dtype=torch.bool, device="cuda")
    before = lay.checkpoint.clone()
    y = lay.prefill(prompt, start, rows=at, resume=known)
    assert torch.equal(lay.checkpoint[others], before[others]) and torch.equal(lay.pointers()[0], ref.pointers()[0])
    running = {n: t.clone() for n, t in rec(batch).items()}
    after = lay.step(running)
    unprompted = ref.step(running)
    assert torch.equal(after[others], unprompted[others])
    ref2 = ReplayLayer("gdn", batch, H, P, N, 4, max_draft=2, read_fmt=getattr(B, rf), flags=flags)
    ref2.set_state(begin)
    for r in steps:
        ref2.step(r)
    ref2.flush()
    state = ref2.checkpoint.clone()
    want = ops.delta_prompt(*(prompt[n] for n in ("q", "k", "v", "alpha", "beta")), start, state,
                            initial=None if resume is None else state, rows=at, resume=known)
    ref2.set_state(state)
    assert torch.equal(y, want) and torch.equal(lay.checkpoint[mine], state[mine])
    assert torch.equal(after[mine], ref2.step(running)[mine])


@pytest.mark.parametrize("cf,rf", [("FMT_F16_SR", "FMT_F4E2M1_B16"), ("FMT_F8E4M3", "FMT_F8E4M3")])
def test_prefill_into_formats_below_float32(cf, rf):
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer
    announce("gdn prefill low", cf, rf)
    p = DeltaPrompts(4, 64, 128, [30, 70], None, "f32", lead=0, tail=0, spare=0)
    t = p.tensors()
    rec = dict(zip(("q", "k", "v", "alpha", "beta"), t))
    start = torch.tensor([0, 30, 100], dtype=torch.int32, device="cuda")
    lay, ref = (ReplayLayer("gdn", 2, 4, 64, 128, 4, ckpt_fmt=getattr(B, cf), read_fmt=getattr(B, rf)) for _ in range(2))
    y = lay.prefill(rec, start)
    state = torch.empty(2, 4, 64, 128, device="cuda")
    want = ops.delta_prompt(*t, start, state)
    ref.set_state(state)
    assert torch.equal(y, want)
    for a, b in zip(lay.stored_copies(), ref.stored_copies()):
        assert (a is None and b is None) or torch.equal(a, b)


def test_other_stream_and_captured_calls():
    """On another stream than the current one's default, and replayed from a graph between eager calls."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("delta_prompt streams and graphs")
    p = DeltaPrompts(4, 64, 64, [150, 90], "all", "bf16", lead=0, tail=0, spare=0)
    t, start, rows = p.tensors(), torch.tensor([0, 150, 240], dtype=torch.int32, device="cuda"), torch.tensor(
        p.rows, dtype=torch.int32, device="cuda")
    init = torch.from_numpy(p.init).cuda()
    state = torch.empty_like(init)
    call = lambda s: ops.delta_prompt(*t, start, s, initial=init, rows=rows, out_dtype=torch.bfloat16)  # noqa: E731
    want = call(state).clone()
    kept = state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        state.zero_()
        y = call(state)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(state, kept)
    graphs, outs, states = [], [], []
    for _ in range(2):  # two graphs, replayed in turn
        s = torch.empty_like(init)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(s))
        graphs.append(graph), states.append(s)
    for turn in range(3):
        t[2].mul_(-1.0)  # eager work between the replays: other inputs
        eager_state = torch.empty_like(init)
        eager = call(eager_state)
        for graph, y, s in zip(graphs, outs, states):
            y.zero_(), s.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, eager) and torch.equal(s, eager_state), turn


def spread(n, tokens, seed):
    """n lengths that differ widely and add up to about `tokens`."""
    r = np.random.default_rng(seed).exponential(1.0, n) ** 2
    return [int(x) for x in r * tokens / r.sum()]


MANY = [
    # sequences x heads that fill the card, as above
    (128, 64, 64, [130], None, "bf16"),
    (64, 128, 128, [1, 200], [1, 0], "f32"),
    (64, 96, 128, [65, 64], "all", "bf16"),
    (43, 80, 64, [70, 0, 3], [0, 1, 1], "f32"),
    (32, 128, 128, [20, 300, 1, 900, 64, 250, 0, 100], [1, 0, 1, 1, 0, 1, 1, 0], "f32"),
    (32, 112, 64, [900, 64, 300, 1, 250, 20, 0, 100], "all", "bf16"),
    (64, 64, 128, [100, 500, 0, 450, 65], None, "bf16"),
    (3, 32, 64, [17, 0, 1, 64, 65, 2] * 32, "all", "f32"),
    (1, 32, 64, spread(300, 60000, 1), "all", "bf16"),
    (2, 16, 64, spread(800, 3000, 2), "all", "f32"),
]


@pytest.mark.parametrize("H,P,N,lens,resumed,out", MANY)
def test_delta_prompt_of_many_heads_and_sequences(H, P, N, lens, resumed, out):
    announce("delta_prompt many", H, P, N, len(lens), lens[:8], resumed, out)
    p = DeltaPrompts(H, P, N, lens, resumed, "bf16", tail=200).surround()
    check(p, out, *p.run(out))


@pytest.mark.parametrize("H,P,N,lens,name", [(4, 64, 128, [65, 30], "bf16"), (3, 32, 32, [1, 64], "f32"), (70, 64, 64, [65, 30], "bf16")])
def test_rows_behind_the_last_sequence_are_not_read_nor_written(H, P, N, lens, name):
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    announce("delta_prompt rows behind", H, P, N, lens, name)
    p = DeltaPrompts(H, P, N, lens, "all", name, tail=200).surround()
    check(p, "f32", *p.run("f32"))
    # The outputs of those rows stay what they are.
    t, state, start = p.tensors(), torch.zeros((p.batch,) + p.shape, device="cuda"), torch.from_numpy(p.start).cuda()
    at, args, y, ws = ops.delta_call(*t, start, state, None, None, None, None, None)
    y.fill_(7.0)
    ops.launch(B.replay_delta_prompt, at, *args)
    torch.cuda.synchronize()
    assert bool((y[:p.lead] == 7).all()) and bool((y[p.tokens - p.tail:] == 7).all())
    assert bool(torch.isfinite(y).all()) and not bool((y[p.lead:p.tokens - p.tail] == 7).all())


@pytest.mark.parametrize("what", ["same keys", "alpha 0", "tiny alpha", "beta 2", "zero keys"])
def test_delta_prompt_of_many_heads_extremes(what):
    announce("delta_prompt many extremes", what)
    p = DeltaPrompts(64, 64, 64, [150, 70], "all", "bf16", seed=3)
    r = np.random.default_rng(5)
    if what == "same keys":
        p.k[:], p.beta[:], p.alpha[:] = p.k[:1], 1.0, 1.0
    elif what == "alpha 0":
        p.alpha[r.random(p.alpha.shape) < 0.1] = 0.0
    elif what == "tiny alpha":
        p.alpha[r.random(p.alpha.shape) < 0.3] = 1e-38
    elif what == "beta 2":
        p.beta[:] = 2.0
    else:
        p.k[r.random(p.tokens) < 0.5] = 0.0
        p.q[r.random(p.tokens) < 0.2] = 0.0
    if what in ("same keys", "beta 2"):  # bf16 keys are longer than 1 by up to 2^-8: shrink them
        p.k *= np.float32(1 - 2.0 ** -7)
    p.surround()
    check(p, "f32", *p.run("f32"))


@pytest.mark.parametrize("H,lens", [(64, [1, 200]), (32, [20, 300, 1, 900, 64, 250, 0, 100])])
def test_many_heads_on_another_stream_in_place_and_captured(H, lens):
    """Two streams at once, and replays of a graph, give what one call gives."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("delta_prompt many captured", H, lens)
    p = DeltaPrompts(H, 128, 128, lens, "all", "bf16")
    t, start, rows = p.tensors(), torch.from_numpy(p.start).cuda(), torch.from_numpy(p.rows).cuda()
    init = torch.from_numpy(p.init).nan_to_num(0.0).cuda()
    want_s = init.clone()
    want = ops.delta_prompt(*t, start, want_s, initial=want_s, rows=rows)
    torch.cuda.synchronize()
    states, got, streams = [init.clone(), init.clone()], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, st in zip(streams, states):
        with torch.cuda.stream(s):
            got.append(ops.delta_prompt(*t, start, st, initial=st, rows=rows))
    torch.cuda.synchronize()
    inside = slice(p.lead, p.tokens - p.tail)
    for y, st in zip(got, states):
        assert torch.equal(y[inside], want[inside]) and torch.equal(st, want_s)
    state, graph = init.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.delta_prompt(*t, start, state, initial=state, rows=rows)
    for _ in range(3):
        state.copy_(init)
        y.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y[inside], want[inside]) and torch.equal(state, want_s)


def test_bad_rows_and_offsets_of_many_heads():
    """Rows outside the batch, offsets past the tokens, falling ones (empty): nothing else is touched."""
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    announce("delta_prompt many, bad rows")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    tokens, H, P, N = 6400, 64, 80, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k = (torch.nn.functional.normalize(torch.randn(tokens, H, N, generator=g, device="cuda"), dim=-1).bfloat16() for _ in range(2))
    v = torch.randn(tokens, H, P, generator=g, device="cuda").bfloat16()
    alpha, beta = (torch.rand(tokens, H, generator=g, device="cuda") for _ in range(2))
    state, status = torch.full((4, H, P, N), 7.0, device="cuda"), i32([0])
    ops.delta_prompt(q, k, v, alpha, beta, i32([0, 3000, 3001, 6400]), state, rows=i32([-1, 2, 9]), status=status)
    assert int(status) == B.STATUS_BAD_PROMPT
    assert bool((state[[0, 1, 3]] == 7).all()) and not bool((state[2] == 7).any())
    one = torch.empty(1, H, P, N, device="cuda")
    ops.delta_prompt(q, k, v, alpha, beta, i32([0, tokens]), one)
    for start in ([0, tokens] * 4 + [0], [-5, tokens + 9, 70], [tokens, 0, tokens], [9, 9, 9, 9]):
        n = len(start) - 1
        state = torch.full((n, H, P, N), 7.0, device="cuda")
        ops.delta_prompt(q, k, v, alpha, beta, i32(start), state)
        at = np.clip(start, 0, tokens)
        for i in range(n):
            if at[i + 1] <= at[i]:
                assert bool((state[i] == 0).all())
            elif at[i + 1] - at[i] == tokens:
                assert bool(((state[i] - one[0]).abs() <= 1e-5 * one[0].abs() + 1e-6).all())


def test_more_heads_than_one_launch_walks():
    """A token a sequence from a state of zeros: o = beta v (k . q), S = beta v k^T.  In passes, by the form with a workspace."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("delta_prompt most heads")
    H, P, N, n = 32, 32, 64, ((1 << 32) - 1) // 768 // 32 + 1
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k = (torch.nn.functional.normalize(torch.randn(n, H, N, generator=g, device="cuda"), dim=-1).bfloat16() for _ in range(2))
    v = torch.randn(n, H, P, generator=g, device="cuda").bfloat16()
    alpha, beta = (torch.rand(n, H, generator=g, device="cuda") for _ in range(2))
    state = torch.full((n, H, P, N), float("nan"), device="cuda")
    y = ops.delta_prompt(q, k, v, alpha, beta, torch.arange(n + 1, dtype=torch.int32, device="cuda"), state)
    # Products of three factors and pieces that hold 24 bits: the state within 4 U, o within its sum's N more of |k| . |q|.
    for at in range(0, n, 8192):
        kd, qd, vd = (t[at:at + 8192].double() for t in (k, q, v))
        u = beta[at:at + 8192].double()[..., None] * vd
        want = u[..., :, None] * kd[..., None, :]
        assert bool(((state[at:at + 8192] - want).abs() <= 4 * 2.0 ** -24 * want.abs() + 1e-37).all())
        dot, size = (kd * qd).sum(-1, keepdim=True), (kd * qd).abs().sum(-1, keepdim=True)
        assert bool(((y[at:at + 8192] - u * dot).abs() <= (N + 8) * 2.0 ** -24 * u.abs() * size + 1e-37).all())
