"""What prompts of Gated DeltaNet layers refuse, before anything is enqueued (no GPU)."""
import pytest
import torch

from _fake_device import Placed

P16 = 4096  # an address that is never followed: every call here is refused on the host
TOKENS, BATCH, H, P, N = 5, 3, 4, 32, 64


@pytest.fixture(scope="module")
def B():
    from hybrid_model_ssm_replay_amd import binding
    binding.load_library()
    return binding


def _refused(B, fn, code=None):
    with pytest.raises(B.ReplayError) as e:
        fn()
    assert e.value.code == (B.EINVAL if code is None else code)


def _record(B, n=5):
    return B.make_record(*[P16] * n)


@pytest.mark.parametrize("cfg", [(0, 2, 4, 4, 64, 64, 1), (1, 0, 4, 4, 64, 64, 1), (1, 2, 4, 2, 64, 64, 1), (1, 2, 0, 0, 64, 64, 1),
                                 (1, 2, 4, 4, 24, 64, 1), (1, 2, 4, 4, 144, 64, 1), (1, 2, 4, 4, 64, 48, 1),
                                 (1, 1, 1 << 16, 1 << 16, 128, 16, 1), (1, 1, 1 << 16, 1 << 16, 16, 128, 1)])
def test_shapes(B, cfg):
    c = B.make_config(*cfg)
    assert B.replay_delta_workspace_bytes(c, 100, 1, B.DT_F32) == 0
    p = B.replay_prompt(8, 1, P16, 0, 0, 0)
    _refused(B, lambda: B.replay_delta_prompt(c, p, _record(B), 0, P16, P16, B.DT_F32, P16, 0))


def test_calls(B):
    c, p = B.make_config(1, 2, 4, 4, 32, 64, 1), B.replay_prompt(8, 1, P16, 0, 0, 0)
    good = [c, p, _record(B), 0, P16, P16, B.DT_F32, P16, 0]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return lambda: B.replay_delta_prompt(*a)

    for i in (4, 5, 7):
        _refused(B, with_(i, 0))
    for i in (3, 4, 5, 7):
        _refused(B, with_(i, P16 + 4))
    _refused(B, with_(6, 2))
    _refused(B, with_(6, B.DT_BF16), B.ENOTSUP)  # bf16 outputs of float32 records
    for i in range(5):
        f = [P16] * 5
        f[i] = 0
        _refused(B, with_(2, B.make_record(*f)))
    for i in range(3):
        f = [P16] * 5
        f[i] = P16 + 8
        _refused(B, with_(2, B.make_record(*f)))
    for bad in ((-1, 1, P16), (8, 0, P16), (8, 3, P16), (8, 1, 0), ((1 << 30) + 1, 1, P16)):
        _refused(B, with_(1, B.replay_prompt(*bad, 0, 0, 0)))


def test_workspace(B):
    """None without tokens, for a chunk or so a sequence and for many heads; bounded however many
    tokens there are; none for what is refused."""
    c, low = B.make_config(1, 200, 32, 32, 128, 128, 1, flags=B.FLAG_BF16_RECORDS), B.make_config(1, 2, 32, 32, 128, 128, 1)
    assert B.replay_delta_workspace_bytes(c, 0, 3, B.DT_F32) == 0
    sizes = [B.replay_delta_workspace_bytes(c, n, 3, B.DT_BF16) for n in (1, 1000, 100000, 1 << 30)]
    assert 0 == sizes[0] < sizes[1] < sizes[2] == sizes[3] <= 256 << 20
    assert B.replay_delta_workspace_bytes(c, 1 << 30, 4, B.DT_BF16) == 0 == B.replay_delta_workspace_bytes(c, 192, 3, B.DT_F32)
    assert 0 < B.replay_delta_workspace_bytes(c, 193, 3, B.DT_F32) and 0 < B.replay_delta_workspace_bytes(low, 1, 1, B.DT_F32)
    assert B.replay_delta_workspace_bytes(low, 100, 1, B.DT_BF16) == 0 < B.replay_delta_workspace_bytes(low, 100, 1, B.DT_F32)
    assert B.replay_delta_workspace_bytes(c, 100, 201, B.DT_F32) == 0 and B.replay_delta_workspace_bytes(c, -1, 1, B.DT_F32) == 0


def test_workspace_of_wide_layers(B):
    """Eight chunks of all heads at least, and otherwise 256 MB at most, however many tokens there are."""
    seen = set()
    for heads in (32, 300, 326, 327, 400, 4000):
        for flags, P, N in ((0, 128, 128), (0, 64, 64), (0, 16, 16), (B.FLAG_BF16_RECORDS, 128, 128)):
            c = B.make_config(1, 1, heads, heads, P, N, 1, flags=flags)
            if flags and heads > 100:
                continue  # these walk
            size = [B.replay_delta_workspace_bytes(c, n, 1, B.DT_F32) for n in (7 * 64, 1 << 20, 1 << 30)]
            assert 0 < size[0] <= size[1] == size[2] and size[0] % (8 * heads) == 0
            assert size[2] == size[0] if size[0] > 256 << 20 else size[2] <= 256 << 20
            if (flags, N) == (0, 128):
                seen.add(size[0] > 256 << 20)
                assert (size[0] > 256 << 20) == (heads > 326)
    assert seen == {False, True}


def test_workspace_of_more_heads_than_one_launch_walks(B):
    """Workgroups of 768 threads, one for a head and 16 more: below 2^32 work-items.  Others go in passes, with a workspace."""
    most = ((1 << 32) - 1) // 768 - 16
    for sequences, some in (((1 << 22) // 32, 0), (most // 32, 0), (most // 32 + 1, 1), (1 << 18, 1)):
        for P, N in ((32, 64), (128, 128)):
            c = B.make_config(1, 1 << 18, 32, 32, P, N, 1, flags=B.FLAG_BF16_RECORDS)
            size = B.replay_delta_workspace_bytes(c, sequences, sequences, B.DT_F32)
            assert (0 < size <= 256 << 20) if some else size == 0, (sequences, P)


def _on(*shape, dtype=torch.float32):
    return Placed.of(torch.zeros(shape, dtype=dtype))


def _good(dtype=torch.float32):
    return dict(q=_on(TOKENS, H, N, dtype=dtype), k=_on(TOKENS, H, N, dtype=dtype), v=_on(TOKENS, H, P, dtype=dtype),
                alpha=_on(TOKENS, H), beta=_on(TOKENS, H), seq_start=_on(BATCH + 1, dtype=torch.int32),
                rows=_on(BATCH, dtype=torch.int32), resume=_on(BATCH, dtype=torch.bool), out_dtype=None)


def _off(shape):  # an address that is not a multiple of 16
    t = Placed.of(torch.zeros(1 + torch.Size(shape).numel())[1:].view(shape))
    assert t.data_ptr() % 16
    return t


BAD = [
    dict(q=_on(TOKENS, H, 2 * N)), dict(q=_on(TOKENS, N, H).transpose(1, 2)), dict(q=_off((TOKENS, H, N))), dict(k=_off((TOKENS, H, N))),
    dict(k=_on(TOKENS, H, 2 * N)), dict(k=_on(TOKENS + 1, H, N)), dict(k=_on(TOKENS, H, N, dtype=torch.bfloat16)),
    dict(v=_on(TOKENS, H, 2 * P)), dict(v=_on(TOKENS, H + 1, P)), dict(v=_on(TOKENS, H * P)), dict(v=_off((TOKENS, H, P))),
    dict(alpha=_on(TOKENS, H, dtype=torch.bfloat16)), dict(alpha=_on(TOKENS, 1)), dict(alpha=_on(H, TOKENS).t()),
    dict(beta=torch.zeros(TOKENS, H)), dict(beta=_on(TOKENS - 1, H)), dict(seq_start=_on(BATCH + 1, dtype=torch.int64)),
    dict(rows=_on(2 * BATCH, dtype=torch.int32)[::2]), dict(resume=_on(BATCH + 1, dtype=torch.bool)), dict(resume=_on(BATCH)),
    dict(out_dtype=torch.float16), dict(out_dtype=torch.bfloat16),
]


@pytest.mark.parametrize("bad", BAD)
def test_python_function(monkeypatch, B, bad):
    from hybrid_model_ssm_replay_amd import ops
    monkeypatch.setattr(B, "replay_delta_prompt", lambda *a: pytest.fail("enqueued"))
    a = {**_good(), **bad}
    state = _on(BATCH, H, P, N)
    with pytest.raises(ValueError):
        ops.delta_prompt(*[a.pop(n) for n in ("q", "k", "v", "alpha", "beta", "seq_start")], state, initial=state, **a)


@pytest.fixture
def layer(monkeypatch, B):
    """A layer on host memory; its calls to the device are noted in ``done``."""
    from hybrid_model_ssm_replay_amd import ops
    from hybrid_model_ssm_replay_amd.layer import ReplayLayer, _kind, _Shapes
    lay = object.__new__(ReplayLayer)
    lay.shapes = _Shapes(_kind("gdn"), BATCH, H, H, P, N, 0)
    lay.cfg = B.make_config(_kind("gdn"), BATCH, H, H, P, N, 4)
    lay.ckpt, lay.read_copy, lay.status_word = _on(BATCH * H * P * N * 4, dtype=torch.uint8), None, _on(4, dtype=torch.int32)
    lay.A = lay.D = None
    lay.done = []
    lay.flush = lambda mask: lay.done.append("flush")
    monkeypatch.setattr(B, "replay_delta_prompt", lambda *a: lay.done.append("delta"))
    monkeypatch.setattr(ops, "_device", lambda: 0)
    monkeypatch.setattr(ops, "_raw_stream", lambda at: 0)
    return lay


def _prefill(lay, **args):
    a = {**_good(), **args}
    return lay.prefill({n: a.pop(n) for n in ("q", "k", "v", "alpha", "beta")}, **a)


def test_a_good_prefill_flushes_and_runs(layer):
    y = _prefill(layer)
    assert layer.done == ["flush", "delta"] and tuple(y.shape) == (TOKENS, H, P)


@pytest.mark.parametrize("bad", BAD)
def test_prefill_refuses_before_anything_is_enqueued(layer, bad):
    with pytest.raises(ValueError):
        _prefill(layer, **bad)
    assert not layer.done


def test_prefill_refuses_a_record_without_a_field(layer):
    a = _good()
    for gone in ("q", "k", "v", "alpha", "beta"):
        with pytest.raises(ValueError, match="q, k, v, alpha and beta"):
            layer.prefill({n: a[n] for n in ("q", "k", "v", "alpha", "beta") if n != gone}, a["seq_start"])
    assert not layer.done
