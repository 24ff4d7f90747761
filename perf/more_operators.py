"""Timing cases of the operators of a served stack of layers.

The gated delta rule over packed prompts, the norm of the residual stream (its
addition, and outputs in bf16 or in 8 bits with scales) and the log
probabilities of given tokens.  With ``own`` false ``run`` computes them from
elementary torch operations in float32 (float64 for sums of log decays); with
``own`` true it calls the library.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2}
EPS = 1e-5
CHUNK = 64
E4M3_MAX, LEAST_SCALE = 448.0, 2.0 ** -126


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # One prompt of 8192 tokens alone, a layer with 32 heads of 128 and states of 128: the recurrence is one
        # long chain for each head.
        dict(name="delta_one_8k", op="delta", dtype="bf16", out="bf16", tokens=8192, sequences=1, heads=32, head_dim=128,
             state_dim=128, resume=False),
        # A prefill batch: 16384 tokens of 24 requests of uneven length, each continuing an earlier part.
        dict(name="delta_ragged_16k", op="delta", dtype="bf16", out="f32", tokens=16384, sequences=24, heads=32,
             head_dim=128, state_dim=128, resume=True),
        # Float32 records (the library's default), 2048 tokens of five requests.
        dict(name="delta_f32_2k", op="delta", dtype="f32", out="f32", tokens=2048, sequences=5, heads=32, head_dim=128,
             state_dim=128, resume=True),
        # The last few tokens of a prompt: latency counts.
        dict(name="delta_short", op="delta", dtype="bf16", out="bf16", tokens=37, sequences=1, heads=32, head_dim=128,
             state_dim=128, resume=True),
        # Between two layers of a decode step of 256 sequences.
        dict(name="norm_step_b256", op="norm", dtype="bf16", stream="bf16", out="bf16", tokens=256, channels=4096, group=0),
        # The same over a prompt, a wider stream.
        dict(name="norm_prompt_8k", op="norm", dtype="bf16", stream="bf16", out="bf16", tokens=8192, channels=8192, group=0),
        # 8-bit inputs for the next projection, a scale for every 128 channels, over a prompt's part.
        dict(name="norm_e4m3_2k", op="norm", dtype="bf16", stream="bf16", out="e4m3", tokens=2048, channels=4096, group=128),
        # A float32 stream of an odd width, a scale for every token.
        dict(name="norm_e4m3_odd", op="norm", dtype="bf16", stream="f32", out="e4m3", tokens=1001, channels=5003, group=5003),
        # One sequence's next token with twenty alternatives, float32 logits of a large vocabulary: latency counts.
        dict(name="logprobs_one", op="logprobs", dtype="f32", rows=1, vocab=131072, top=20, masked=False),
        # 128 sequences, nine positions each (a token and eight drafts), an odd vocabulary, a part of it masked.
        dict(name="logprobs_b1152", op="logprobs", dtype="bf16", rows=1152, vocab=50021, top=5, masked=True),
        # A prompt's own tokens: 4096 positions of a large vocabulary, no alternatives.
        dict(name="logprobs_prompt_4k", op="logprobs", dtype="bf16", rows=4096, vocab=131072, top=0, masked=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "norm", "logprobs"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "delta":
        heads, head_dim, state_dim = _log_int(rng, 1, 64), rng.choice([16, 32, 48, 64, 96, 128, 128]), rng.choice([16, 32, 64, 128, 128])
        most = 8192 * 32 * 128 * 128 // (1 if dtype == "bf16" else 4)
        tokens = _log_int(rng, 1, min(8192, most // (heads * head_dim * state_dim)))
        return dict(op=op, dtype=dtype, out="f32" if dtype == "f32" else rng.choice(["f32", "bf16"]), tokens=tokens,
                    sequences=_log_int(rng, 1, 24), heads=heads, head_dim=head_dim, state_dim=state_dim, resume=rng.random() < 0.5)
    if op == "norm":
        out = rng.choice(["f32", "bf16", "e4m3", "e4m3"])
        group = rng.choice([0, 32, 64, 128, 256]) if out == "e4m3" else 0
        channels = group * _log_int(rng, 1, 8192 // group) if group else _log_int(rng, 64, 8192)
        return dict(op=op, dtype=dtype, stream=rng.choice(["f32", "bf16"]), out=out, tokens=_log_int(rng, 1, 4096),
                    channels=channels, group=(group or channels) if out == "e4m3" else 0)
    return dict(op=op, dtype=dtype, rows=_log_int(rng, 1, 2048), vocab=_log_int(rng, 1000, 131072),
                top=rng.choice([0, 1, 5, 20, rng.randint(1, 32)]), masked=rng.random() < 0.4)


def _lengths(tokens, sequences):
    """Uneven lengths that add up to tokens, the same for every seed; zeros occur where tokens are few."""
    r = random.Random(1000003 * tokens + sequences)
    cuts = sorted(r.randint(0, tokens) for _ in range(sequences - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [tokens])]


# ---- inputs -----------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case)
    if op == "delta":
        T, n, H, P, N = (case[k] for k in ("tokens", "sequences", "heads", "head_dim", "state_dim"))
        s["lengths"] = _lengths(T, n)
        start = [0]
        for length in s["lengths"]:
            start.append(start[-1] + length)
        s["seq_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        batch = n + 3  # the decode batch has more rows than this call's requests
        s["rows"] = torch.tensor(random.Random(seed).sample(range(batch), n), dtype=torch.int32, device="cuda")
        s["resumed"] = (rand(n) < 0.75).to(torch.uint8) if case["resume"] else None
        q, k = randn(T, H, N), randn(T, H, N)
        s["q"] = (q / q.square().sum(-1, keepdim=True).sqrt()).to(dt)
        s["k"] = (k / k.square().sum(-1, keepdim=True).sqrt()).to(dt)
        s["v"] = randn(T, H, P, dtype=dt)
        rate = torch.exp(math.log(0.01) + rand(H) * math.log(400.0))  # heads from long to short memory
        s["alpha"] = torch.exp(-rate * torch.nn.functional.softplus(randn(T, H)))
        s["beta"] = torch.sigmoid(randn(T, H))
        s["initial"] = randn(batch, H, P, N) if case["resume"] else None
        s["state"] = torch.zeros(batch, H, P, N, device="cuda")
    elif op == "norm":
        T, C = case["tokens"], case["channels"]
        s["x"] = randn(T, C, dtype=dt)                                     # a layer's output
        s["residual"] = 2.0 * randn(T, C, dtype=torch.float32)
        s["residual"] = s["residual"].to(DTYPES[case["stream"]])
        s["weight"] = 1.0 + 0.2 * randn(C)
    else:
        R, V = case["rows"], case["vocab"]
        logits = randn(R, V, dtype=dt)
        logits *= 3.0
        s["tokens"] = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
        if case["masked"]:  # words that a grammar forbids, the same for every position
            logits[:, rand(V) < 0.3] = -math.inf
        s["logits"] = logits
    return s


# ---- one pass ---------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"delta": _delta, "norm": _norm, "logprobs": _logprobs}[s["op"]](s)


def _run_own(s):
    from hybrid_model_ssm_replay_amd import ops
    if s["op"] == "delta":
        y = ops.delta_prompt(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["seq_start"], s["state"], initial=s["initial"],
                             rows=s["rows"], resume=s["resumed"], out_dtype=DTYPES[s["out"]])
        return [y, s["state"]]
    if s["op"] == "norm":
        if s["out"] != "e4m3":
            return list(ops.residual_norm(s["x"], s["residual"], s["weight"], eps=EPS, out_dtype=DTYPES[s["out"]]))
        codes, scales, total = ops.residual_norm(s["x"], s["residual"], s["weight"], eps=EPS, out_dtype=torch.float8_e4m3fn,
                                                 scale_group=s["group"])
        return [_stands_for(codes, scales, s["group"]), scales, total]
    return list(ops.token_logprobs(s["logits"], s["tokens"], top=s["top"]))


def _stands_for(codes, scales, group):
    """8-bit codes times their scales, in bf16."""
    T, C = codes.shape
    out = torch.empty(T, C // group, group, dtype=torch.bfloat16, device=codes.device)
    torch.mul(codes.to(torch.bfloat16).view(T, C // group, group), scales[..., None], out=out)
    return out.view(T, C)


def _inverse(T):
    """(I + T)^-1 for strictly lower triangular T [..., 64, 64]: diagonal blocks of 1, 2, 4, ... 32 joined in pairs."""
    A = torch.eye(CHUNK, device=T.device).expand_as(T).contiguous()
    for size in (1, 2, 4, 8, 16, 32):
        n = CHUNK // (2 * size)
        pairs = A.unflatten(-1, (n, 2, size)).unflatten(-4, (n, 2, size))           # pair, half, row, pair, half, column
        below = T.unflatten(-1, (n, 2, size)).unflatten(-4, (n, 2, size))
        d = torch.arange(n, device=T.device)
        upper, lower = pairs[..., d, 0, :, d, 0, :], pairs[..., d, 1, :, d, 1, :]   # pair first, then the batch
        A.unflatten(-1, (n, 2, size)).unflatten(-4, (n, 2, size))[..., d, 1, :, d, 0, :] = -torch.matmul(
            torch.matmul(lower, below[..., d, 1, :, d, 0, :].contiguous()), upper.contiguous())
    return A


def _delta(s):
    q, k, v, alpha, beta = s["q"], s["k"], s["v"], s["alpha"], s["beta"]
    tokens, H, N = q.shape
    P, Q, dev = v.shape[-1], CHUNK, q.device
    start, rows = s["seq_start"].long(), s["rows"].long()
    n = rows.numel()
    base = start[:-1] // Q + torch.arange(n, device=dev)                            # first chunk of each sequence
    c = torch.arange(tokens // Q + n, device=dev)
    seq = torch.searchsorted(base, c, right=True) - 1
    t = start[seq][:, None] + (c - base[seq])[:, None] * Q + torch.arange(Q, device=dev)
    there = t < start[seq + 1][:, None]
    t = t.clamp(max=tokens - 1)

    def chunked(a, empty):  # chunk, head, token, ...
        a = torch.where(there.reshape(*there.shape, *[1] * (a.dim() - 1)), a[t].float(), empty)
        return a.transpose(1, 2).contiguous()

    qc, kc, vc, bc = chunked(q, 0.0), chunked(k, 0.0), chunked(v, 0.0), chunked(beta, 0.0)
    g = torch.cumsum(torch.log(chunked(alpha, 1.0).double()), -1)
    low = torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
    L = torch.exp(torch.where(low, g[..., :, None] - g[..., None, :], -math.inf)).float()
    kt = kc.transpose(-1, -2).contiguous()
    A = _inverse(torch.matmul(kc, kt) * (L * bc[..., :, None]).tril(-1)) * bc[..., None, :]
    M = torch.matmul(qc, kt) * L
    eg, left = torch.exp(g).float()[..., None], torch.exp(g[..., -1:] - g).float()
    Av, Ak = torch.matmul(A, vc), torch.matmul(A, kc * eg)
    kl = (kc * left[..., None]).transpose(-1, -2).contiguous()                      # chunk, head, N, token
    whole = eg[..., -1:, :]
    S = torch.zeros(n, H, N, P, device=dev)                                         # the state, transposed
    if s["initial"] is not None:
        first = s["initial"][rows].transpose(-1, -2)
        S = first.contiguous() if s["resumed"] is None else torch.where(s["resumed"].bool()[:, None, None, None], first, 0.0)
    o = torch.empty(c.numel(), H, Q, P, device=dev)
    for i in range((max(s["lengths"]) + Q - 1) // Q):                               # the state goes from chunk to chunk
        live = [j for j, length in enumerate(s["lengths"]) if length > i * Q]
        j = torch.tensor(live, device=dev) if len(live) < n else slice(None)
        at, cur = base[j] + i, S[j]
        u = Av[at] - torch.matmul(Ak[at], cur)
        o[at] = torch.matmul(qc[at] * eg[at], cur) + torch.matmul(M[at], u)
        S[j] = cur * whole[at] + torch.matmul(kl[at], u)
    out = torch.empty(tokens, H, P, dtype=DTYPES[s["out"]], device=dev)
    out[t[there]] = o.transpose(1, 2)[there].to(out.dtype)
    s["state"][rows] = S.transpose(-1, -2)
    return [out, s["state"]]


def _norm(s):
    x, G = s["x"].float(), s["group"]
    T, C = x.shape
    h = x + s["residual"].float()
    out = h * torch.rsqrt((h * h).sum(-1, keepdim=True) / C + EPS) * s["weight"]
    total = h.to(s["residual"].dtype)
    if s["out"] != "e4m3":
        return [out.to(DTYPES[s["out"]]), total]
    out = out.view(T, C // G, G)
    scales = (out.abs().amax(-1) / E4M3_MAX).clamp(min=LEAST_SCALE)
    codes = (out / scales[..., None]).to(torch.float8_e4m3fn).view(T, C)
    return [_stands_for(codes, scales, G), scales, total]


def _logprobs(s):
    x, top = s["logits"].float(), s["top"]
    d = x - x.amax(-1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(-1)
    log = torch.log(total)
    logprob = torch.gather(d, 1, s["tokens"].long()[:, None])[:, 0] - log
    entropy = log - torch.where(e > 0, e * d, 0.0).sum(-1) / total
    if not top:
        return [logprob, entropy, logprob.new_empty(len(logprob), 0), s["tokens"].new_empty(len(logprob), 0)]
    values, words, left = [], [], x.clone()
    for _ in range(top):
        at = (left == left.amax(-1, keepdim=True)).int().argmax(-1, keepdim=True)   # ties: the lowest index
        values.append(torch.gather(d, 1, at)[:, 0] - log)
        words.append(at[:, 0].to(torch.int32))
        left.scatter_(1, at, -math.inf)
    return [logprob, entropy, torch.stack(values, 1), torch.stack(words, 1)]


# ---- what a pass cannot do without -----------------------------------------
def work(case):
    op, e = case["op"], ESIZE[case["dtype"]]
    if op == "delta":
        T, n, H, P, N = (case[k] for k in ("tokens", "sequences", "heads", "head_dim", "state_dim"))
        states = n * H * P * N * 4 * (2 if case["resume"] else 1)
        return {"bytes": T * H * ((2 * N + P) * e + P * ESIZE[case["out"]] + 8) + states, "flops": T * H * P * N * 6}
    if op == "norm":
        n, C = case["tokens"] * case["channels"], case["channels"]
        out = n * ESIZE[case["out"]] if case["out"] != "e4m3" else n + 4 * n // case["group"]
        return {"bytes": n * (e + 2 * ESIZE[case["stream"]]) + out + 4 * C, "flops": n * 6}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * e + case["rows"] * (12 + 8 * case["top"]), "flops": n * 5}


# ---- the definitions in 64 bits ---------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "norm": _exact_norm, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_delta(s):
    """The recurrence itself, token after token; sequences advance together, longest first."""
    lens, start, rows = s["lengths"], s["seq_start"].tolist(), s["rows"].tolist()
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    S = torch.zeros(len(lens), s["heads"], s["head_dim"], s["state_dim"], dtype=torch.float64, device="cuda")
    for i, o in enumerate(order):
        if s["initial"] is not None and (s["resumed"] is None or bool(s["resumed"][o])):
            S[i] = s["initial"][rows[o]].double()
    y = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    begin = torch.tensor([start[o] for o in order], device="cuda")
    for t in range(max(lens)):
        live = sum(1 for v in lens if v > t)
        at = begin[:live] + t
        k, v, q = s["k"][at].double(), s["v"][at].double(), s["q"][at].double()
        cur = S[:live]
        cur.mul_(s["alpha"][at].double()[..., None, None])
        u = s["beta"][at].double()[..., None] * (v - torch.matmul(cur, k[..., None])[..., 0])
        cur.addcmul_(u[..., :, None], k[..., None, :])
        y[at] = torch.matmul(cur, q[..., None])[..., 0]
    state = s["state"].double()
    state[torch.tensor([rows[o] for o in order], device="cuda")] = S
    return [y, state]


def _exact_norm(s):
    h = s["x"].double() + s["residual"].double()
    out = h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
    if s["out"] != "e4m3":
        return [out, h]
    out = out.unflatten(1, (-1, s["group"]))
    scales = (out.abs().amax(-1) / E4M3_MAX).clamp(min=LEAST_SCALE)
    r = (out / scales[..., None]).abs()
    step = torch.exp2(torch.floor(torch.log2(r.clamp(min=2.0 ** -6))) - 3.0)         # of e4m3 at r: 3 bits, from 2^-6 on
    code = (torch.round(r / step) * step).clamp(max=E4M3_MAX) * torch.sign(out)
    return [(code * scales[..., None]).flatten(1), scales, h]


def _exact_logprobs(s):
    top, parts = s["top"], []
    for x, tok in zip(s["logits"].split(256), s["tokens"].long().split(256)):
        logp = torch.log_softmax(x.double(), -1)
        got = [logp.gather(1, tok[:, None])[:, 0], torch.special.entr(logp.exp()).sum(-1)]
        first = torch.sort(x.double(), dim=-1, descending=True, stable=True).indices[:, :top]
        parts.append(got + [logp.gather(1, first), first.to(torch.int32)])
    return [torch.cat(p) for p in zip(*parts)]
