"""The residual stream's norm of rows above 16384 channels, which are read twice, against its definition in float64."""
import numpy as np
import pytest

from _gpu import announce
from _scan import HALF, U, _dev, _dt, near, values
from oracle import layer_ops as L

pytestmark = pytest.mark.gpu


def _inputs(T, C, x, stream, seed=0, pad=0):
    r = np.random.default_rng(seed + 100 * T + C)
    rows = [_dev((s * r.normal(size=(T, C + pad))).astype(np.float32), n)[:, :C] for s, n in ((1.0, x), (2.0, stream))]
    return rows[0], rows[1], _dev((1.0 + 0.2 * r.normal(size=C)).astype(np.float32))


def _bar(C):
    """Roundings of a value: the sum's half (the addition of h), a lane's C / 256 squares and the tree over lanes and
    waves, the root 2, three products; relative to the value."""
    return (C / 256 + 40 + 8) * U


@pytest.mark.parametrize("T,C,pad", [(3, 16385, 0), (2, 17001, 3), (1, 18432, 0), (300, 16392, 8), (2, 40003, 0)])
@pytest.mark.parametrize("x,stream,out", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "f32", "bf16"), ("f32", "bf16", "f32")])
@pytest.mark.parametrize("with_residual,with_weight", [(True, True), (False, True), (True, False)])
def test_rows_read_twice(T, C, pad, x, stream, out, with_residual, with_weight):
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm long", T, C, pad, x, stream, out, with_residual, with_weight)
    a, res, w = _inputs(T, C, x, stream, pad=pad)
    res, w = res if with_residual else None, w if with_weight else None
    got, total = ops.residual_norm(a, res, w, out_dtype=_dt(out))
    want, h = L.residual_norm(values(a), None if res is None else values(res), None if w is None else values(w), 1e-5)
    near(values(got), want, (_bar(C) + U + HALF[out]) * np.abs(want) + 1e-37)
    if res is None:
        assert total is a
    else:
        near(values(total), h, (HALF[stream] + U) * np.abs(h))


@pytest.mark.parametrize("T,C,group", [(2, 16896, 512), (3, 20480, 16), (2, 24576, 128), (5, 16416, 32), (2, 18496, 64), (2, 17152, 256),
                                       (3, 20011, 20011), (2, 20480, 20480)])
@pytest.mark.parametrize("x,stream", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_codes_and_scales(T, C, group, x, stream):
    """Scales to float32 rounding; a code is a value that the quotient, known to float32 rounding, may round to."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm long e4m3", T, C, group, x, stream)
    a, res, w = _inputs(T, C, x, stream, seed=1)
    got, scales, total = ops.residual_norm(a, res, w, out_dtype=torch.float8_e4m3fn, scale_group=group)
    want, h = L.residual_norm(values(a), values(res), values(w), 1e-5)
    near(values(total), h, (HALF[stream] + U) * np.abs(h))
    want = want.reshape(T, C // group, group)
    code, scale = values(got.float()).reshape(want.shape), values(scales)[..., None]
    exact = np.maximum(np.abs(want).max(-1, keepdims=True) / 448.0, 2.0 ** -126)
    near(scale, exact, (_bar(C) + 2 * U) * exact)
    off = 2 * _bar(C) + 4 * U
    low, high = (L.e4m3(np.abs(want) / exact * f) for f in (1 - off, 1 + off))
    assert ((np.abs(code) >= low) & (np.abs(code) <= high) & ((code == 0) | (np.sign(code) == np.sign(want)))).all()
    assert (np.abs(code).max(-1) == 448).all()


@pytest.mark.parametrize("C", [16385, 20000])
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
def test_the_sum_may_take_the_place_of_an_input(C, name, out):
    """Through the C call: sum at residual's, then at x's address."""
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm long in place", C, name, out)
    a, res, w = (t.contiguous() for t in _inputs(6, C, name, name))
    group, codes = (32 if C % 32 == 0 else C) if out == "e4m3" else 0, out == "e4m3"
    want, *scales, total = ops.residual_norm(a, res, w, out_dtype=torch.float8_e4m3fn if codes else _dt(out), scale_group=group or None)
    dt = {"f32": B.DT_F32, "bf16": B.DT_BF16, "e4m3": B.DT_E4M3}
    for place in (0, 1):
        x, r = a.clone(), res.clone()
        got, scale = torch.empty_like(want), torch.empty_like(scales[0]) if codes else None
        args = B.replay_residual_norm_args(6, C, group, dt[name], dt[name], dt[out], 1e-5, 0, C, C, C, C, x.data_ptr(), r.data_ptr(),
                                           w.data_ptr(), got.data_ptr(), scale.data_ptr() if codes else 0, (r, x)[place].data_ptr())
        B.replay_residual_norm(args, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        same = (lambda g, e: torch.equal(g.view(torch.uint8), e.view(torch.uint8)))  # noqa: E731
        assert same(got, want) and same((r, x)[place], total) and (not codes or torch.equal(scale, scales[0]))


def test_a_nan_or_infinity_stays_in_its_row():
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm long NaN")
    for C, group in ((20000, None), (16896, 512)):
        a, res, w = _inputs(5, C, "f32", "f32")
        clean, total = ops.residual_norm(a, res, w)
        codes, scales, _ = ops.residual_norm(a, res, w, out_dtype=torch.float8_e4m3fn, scale_group=group)
        a[2, C // 2], a[4, 0] = float("nan"), float("inf")
        got, after = ops.residual_norm(a, res, w)
        fine = [0, 1, 3]
        assert torch.equal(got[fine], clean[fine]) and torch.equal(after[fine], total[fine])
        assert bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[4, 0])) and bool((got[4, 1:] == 0).all())
        codes2, scales2, _ = ops.residual_norm(a, res, w, out_dtype=torch.float8_e4m3fn, scale_group=group)
        assert torch.equal(codes2.view(torch.uint8)[fine], codes.view(torch.uint8)[fine]) and torch.equal(scales2[fine], scales[fine])
        assert bool(torch.isnan(codes2[2].float()).all()) and bool(torch.isnan(codes2[4, 0].float())) and bool((codes2[4, 1:].float() == 0).all())


@pytest.mark.parametrize("C", [17001, 16392])
def test_repeated_rows_and_nothing_past_the_outputs(C):
    import torch
    from hybrid_model_ssm_replay_amd import binding as B
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm long edges", C)
    one = torch.randn(1, C, device="cuda")
    got, total = ops.residual_norm(one.expand(5, C), one.expand(5, C), None)
    assert torch.equal(got, got[:1].expand(5, C)) and torch.equal(total, (2 * one).expand(5, C))
    x = torch.randn(3, C, device="cuda").bfloat16()
    for out in (B.DT_BF16, B.DT_F32, B.DT_E4M3):
        room = torch.full((3, C + 9), 7.0, device="cuda", dtype=(torch.float32, torch.bfloat16, torch.float8_e4m3fn)[out])
        rest, scales = torch.full((3, C + 9), 7.0, device="cuda").bfloat16(), torch.full((4,), 7.0, device="cuda")
        args = B.replay_residual_norm_args(3, C, C if out == B.DT_E4M3 else 0, 1, 1, out, 1e-5, 0, C, C, C + 9, C + 9, x.data_ptr(),
                                           x.data_ptr(), 0, room.data_ptr(), scales.data_ptr(), rest.data_ptr())
        B.replay_residual_norm(args, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert bool((room[:, C:].float() == 7).all()) and bool((rest[:, C:] == 7).all()) and bool((rest[:, :C] == 2 * x).all())
        assert float(scales[3]) == 7 and bool((scales[:3] == 7).all()) == (out != B.DT_E4M3)


@pytest.mark.parametrize("C", [20000, 4096])
def test_rows_whose_offsets_pass_32_bits(C):
    """Rows that start behind 2^32 bytes, then 2^32 values."""
    import torch
    from hybrid_model_ssm_replay_amd import ops
    announce("residual_norm far rows", C)
    a, res, w = _inputs(3, C, "bf16", "bf16")
    want, total = ops.residual_norm(a, res, w)
    for stride in ((1 << 30) + 1, (1 << 31) + 8):
        flat = torch.empty(2 * stride + C, device="cuda", dtype=torch.bfloat16)
        x = torch.as_strided(flat, (3, C), (stride, 1), 0)
        x.copy_(a)
        got, after = ops.residual_norm(x, res, w)
        assert torch.equal(got, want) and torch.equal(after, total)
        x.copy_(res)
        got, after = ops.residual_norm(a, x, w)
        assert torch.equal(got, want) and torch.equal(after, total)
        del flat, x
