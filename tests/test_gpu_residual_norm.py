"""The residual stream's norm against its definition in float64."""
import numpy as np
import pytest

from _gpu import announce
from _scan import HALF, U, _dev, _dt, near, values
from oracle import layer_ops as L

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 7), (5, 64), (2, 511), (9, 512), (4, 513), (7, 2047), (3, 2048), (5, 2049), (6, 4096), (2, 5003), (3, 8192),
          (2, 8193), (3, 16384), (1, 20011), (257, 128)]


def _inputs(T, C, x, stream, seed=0, pad=0):
    r = np.random.default_rng(seed + 100 * T + C)
    rows = [_dev((s * r.normal(size=(T, C + pad))).astype(np.float32), n)[:, :C] for s, n in ((1.0, x), (2.0, stream))]
    return rows[0], rows[1], _dev((1.0 + 0.2 * r.normal(size=C)).astype(np.float32))


def _bar(C):
    """Roundings of a value: the sum's half (the addition of h), C / 2 of the squares in a tree of at most
    C / 256 + 40 additions, the root 2, three products; relative to the value."""
    return (C / 256 + 40 + 8) * U


@pytest.mark.parametrize("T,C", SHAPES)
@pytest.mark.parametrize("x,stream,out", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "f32", "bf16"), ("f32", "bf16", "f32")])
@pytest.mark.parametrize("with_residual,with_weight,pad", [(True, True, 0), (False, True, 3), (True, False, 5)])
def test_residual_norm(T, C, x, stream, out, with_residual, with_weight, pad):
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm", T, C, x, stream, out, with_residual, with_weight, pad)
    a, res, w = _inputs(T, C, x, stream, pad=pad)
    res, w = res if with_residual else None, w if with_weight else None
    before = [t.clone() for t in (a, res) if t is not None]
    got, total = ops.residual_norm(a, res, w, eps=1e-5, out_dtype=_dt(out))
    assert all(torch.equal(t, b) for t, b in zip((a, res), before))
    want, h = L.residual_norm(values(a), None if res is None else values(res), None if w is None else values(w), 1e-5)
    assert got.dtype == _dt(out) and got.is_contiguous()
    near(values(got), want, _bar(C) * np.abs(want) + U * np.abs(want / np.where(h == 0, 1, h)) * np.abs(h) + HALF[out] * np.abs(want) + 1e-37)
    if res is None:
        assert total is a
    else:
        assert total.dtype == res.dtype
        near(values(total), h, (HALF[stream] + U) * np.abs(h))


def _codes(got, scales, group):
    T, C = got.shape
    return values(got.float()).reshape(T, C // group, group), values(scales)[..., None]


@pytest.mark.parametrize("T,C,group", [(3, 16, 16), (5, 128, 32), (2, 512, 512), (4, 1024, 256), (3, 4096, 128), (1, 8192, 64),
                                       (2, 16384, 128), (2, 12800, 512), (3, 7, 7), (2, 511, 511), (5, 2048, 2048), (2, 5003, 5003),
                                       (3, 20011, 20011), (33, 96, 32), (2, 8192, 16)])
@pytest.mark.parametrize("x,stream", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_codes_and_scales(T, C, group, x, stream):
    """Scales to float32 rounding; a code is a value that the quotient, known to float32 rounding, may round to."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm e4m3", T, C, group, x, stream)
    a, res, w = _inputs(T, C, x, stream, seed=1)
    got, scales, total = ops.residual_norm(a, res, w, out_dtype=torch.float8_e4m3fn, scale_group=None if group == C else group)
    assert got.dtype == torch.float8_e4m3fn and scales.shape == (T, C // group)
    want, h = L.residual_norm(values(a), values(res), values(w), 1e-5)
    near(values(total), h, (HALF[stream] + U) * np.abs(h))
    want = want.reshape(T, C // group, group)
    code, scale = _codes(got, scales, group)
    exact = np.maximum(np.abs(want).max(-1, keepdims=True) / 448.0, 2.0 ** -126)
    near(scale, exact, (_bar(C) + 2 * U) * exact)
    off = 2 * _bar(C) + 4 * U
    low, high = (L.e4m3(np.abs(want) / exact * f) for f in (1 - off, 1 + off))
    assert ((np.abs(code) >= low) & (np.abs(code) <= high) & ((code == 0) | (np.sign(code) == np.sign(want)))).all()
    assert (np.abs(code).max(-1) == 448).all()


def test_codes_of_zeros_tiny_rows_and_nan():
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm e4m3 specials")
    C = 256
    x = torch.zeros(4, C, device="cuda")
    x[1] = 1e-30
    x[2, 5], x[3] = float("nan"), 3.0
    w = torch.ones(C, device="cuda")
    w[64:128] = 0.0
    codes, scales, _ = ops.residual_norm(x, None, w, out_dtype=torch.float8_e4m3fn, scale_group=64, eps=1e-5)
    v = values(codes.float())
    assert (v[0] == 0).all() and (scales[0] == 2.0 ** -126).all()          # nothing in the row
    assert (v[1, :64] == 448).all() and (v[1, 64:128] == 0).all()
    assert np.isnan(v[2]).all()                                             # a NaN is in every value's root
    assert (v[3, 64:128] == 0).all() and scales[3, 1] == 2.0 ** -126 and (v[3, 128:] == 448).all()
    out, _ = ops.residual_norm(x, None, w, eps=0.0)
    assert np.isnan(values(out)[0]).all()                                   # 0 / 0 without eps


def test_a_nan_or_infinity_stays_in_its_row():
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm NaN")
    for C in (100, 3000, 9000):
        a, res, w = _inputs(5, C, "f32", "f32")
        clean, total = ops.residual_norm(a, res, w)
        a[2, C // 2], a[4, 0] = float("nan"), float("inf")
        got, after = ops.residual_norm(a, res, w)
        assert torch.equal(got[[0, 1, 3]], clean[[0, 1, 3]]) and torch.equal(after[[0, 1, 3]], total[[0, 1, 3]])
        assert bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[4, 0])) and bool((got[4, 1:] == 0).all())


@pytest.mark.parametrize("C", [300, 4000, 10000])
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_the_sum_may_take_the_place_of_an_input(C, name):
    """Through the C call: sum at residual's, then at x's address."""
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm in place", C, name)
    a, res, w = (t.contiguous() for t in _inputs(6, C, name, name))
    want, total = ops.residual_norm(a, res, w)
    dt = B.DT_BF16 if name == "bf16" else B.DT_F32
    for place in (0, 1):
        x, r = a.clone(), res.clone()
        out = torch.empty_like(want)
        args = B.replay_residual_norm_args(6, C, 0, dt, dt, dt, 1e-5, 0, C, C, C, C, x.data_ptr(), r.data_ptr(), w.data_ptr(),
                                           out.data_ptr(), 0, (r, x)[place].data_ptr())
        B.replay_residual_norm(args, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal((r, x)[place], total)


def test_no_tokens_repeated_rows_and_nothing_past_the_outputs():
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm edges")
    out, total = ops.residual_norm(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, device="cuda"), None)
    assert out.shape == total.shape == (0, 64)
    one = torch.randn(1, 700, device="cuda")
    got, total = ops.residual_norm(one.expand(5, 700), one.expand(5, 700), None)
    assert torch.equal(got, got[:1].expand(5, 700)) and torch.equal(total, (2 * one).expand(5, 700))
    for C in (77, 700, 9001):
        x = torch.randn(3, C, device="cuda").bfloat16()
        room = torch.full((3, C + 9), 7.0, device="cuda").bfloat16()
        rest = room.clone()
        args = B.replay_residual_norm_args(3, C, 0, 1, 1, 1, 1e-5, 0, C, C, C + 9, C + 9, x.data_ptr(), x.data_ptr(), 0,
                                           room.data_ptr(), 0, rest.data_ptr())
        B.replay_residual_norm(args, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert bool((room[:, C:] == 7).all()) and bool((rest[:, C:] == 7).all()) and bool((rest[:, :C] == 2 * x).all())


def test_replayed_from_a_graph():
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm graph")
    a, res, w = _inputs(6, 4096, "bf16", "bf16")
    graph = torch.cuda.CUDAGraph()
    ops.residual_norm(a, res, w)
    with torch.cuda.graph(graph):
        got = ops.residual_norm(a, res, w, out_dtype=torch.float8_e4m3fn, scale_group=128)
    for _ in range(3):
        a.mul_(1.5)
        want = ops.residual_norm(a, res, w, out_dtype=torch.float8_e4m3fn, scale_group=128)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g.view(torch.uint8), e.view(torch.uint8)) for g, e in zip(got, want))


@pytest.mark.parametrize("T,C,pad", [(5, 600, 0), (5, 1000, 3), (9, 1024, 0), (600, 600, 0), (600, 2049, 0), (600, 4096, 0), (513, 5003, 0),
                                     (600, 8192, 8), (520, 10000, 0), (514, 16384, 0), (2049, 4096, 0), (2100, 2056, 8), (2060, 8192, 0),
                                     (2050, 8200, 0), (2055, 4099, 0), (2055, 4096, 1), (20001, 1016, 0)])
@pytest.mark.parametrize("out", ["bf16", "e4m3"])
def test_rows_by_other_numbers_of_threads(T, C, pad, out):
    """From a wave to 1024 threads a row, which the numbers of rows and channels decide."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm threads", T, C, pad, out)
    a, res, w = _inputs(T, C, "bf16", "bf16", seed=2, pad=pad)
    want, h = L.residual_norm(values(a), values(res), values(w), 1e-5)
    if out == "bf16":
        got, total = ops.residual_norm(a, res, w)
        near(values(got), want, (_bar(C) + U + HALF["bf16"]) * np.abs(want) + 1e-37)
    else:
        group = 128 if C % 128 == 0 else C
        got, scales, total = ops.residual_norm(a, res, w, out_dtype=torch.float8_e4m3fn, scale_group=group)
        want = want.reshape(T, C // group, group)
        code, scale = _codes(got, scales, group)
        exact = np.maximum(np.abs(want).max(-1, keepdims=True) / 448.0, 2.0 ** -126)
        near(scale, exact, (_bar(C) + 2 * U) * exact)
        off = 2 * _bar(C) + 4 * U
        low, high = (L.e4m3(np.abs(want) / exact * f) for f in (1 - off, 1 + off))
        assert ((np.abs(code) >= low) & (np.abs(code) <= high) & ((code == 0) | (np.sign(code) == np.sign(want)))).all()
    near(values(total), h, (HALF["bf16"] + U) * np.abs(h))


@pytest.mark.parametrize("T,C,out", [((1 << 22) + 5, 4104, "e4m3"), ((1 << 23) + 3, 2056, "bf16")])
def test_as_many_rows_as_a_launch_of_256_threads_each_holds(T, C, out):
    """More rows than a launch of 512 or 1024 threads each: below 2^32 work-items."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm rows", T, C, out)
    a, _, w = _inputs(1, C, "bf16", "bf16")
    x = a.expand(T, C)
    want, _ = L.residual_norm(values(a), None, values(w), 1e-5)
    if out == "bf16":
        got, _ = ops.residual_norm(x, None, w)
        near(values(got[:1]), want, (_bar(C) + U + HALF["bf16"]) * np.abs(want) + 1e-37)
    else:
        got, scales, _ = ops.residual_norm(x, None, w, out_dtype=torch.float8_e4m3fn)
        assert bool((scales == scales[0]).all())
        near(values(scales[0]), np.abs(want).max(-1) / 448.0, (_bar(C) + 2 * U) * np.abs(want).max(-1) / 448.0)
        got = got.view(torch.uint8)
    for at in range(0, T, 1 << 20):
        assert bool((got[at:at + (1 << 20)] == got[:1]).all())
