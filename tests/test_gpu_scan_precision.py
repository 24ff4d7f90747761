"""bf16 outputs of the prompt scan are off by their own rounding, in every launch shape.

The weights and the state enter the output products as two bf16 pieces, each
rounded to nearest: within 2^-16 of each term (half steps of 2^-8 of 2^-8).  So with
s the size of an output's terms and f = (N + 64 + 112 + 4 (n / 64 + 1)) 2^-24 the
float32 part (N + 64 products of a block; four exponentials of arguments up to 24,
each rounded; n / 64 stretches), the sum before the output's rounding is within
e = (f + 2^-16) s, and the output within e (1 + 2^-8) + 2^-8 |y|.

Over many outputs the rounding of the sums to bf16 has a relative size of about
2^-9.2; e, even if every term's rounding pointed the same way and s were ten times
|y|, 2^-12.7: together 1.004 times the rounding alone.  The bar is 1.01.
"""
import numpy as np
import pytest

from _gpu import announce
from _scan import HALF, U, Prompts, near

pytestmark = pytest.mark.gpu


def _rms(a):
    return float(np.sqrt(np.mean(np.concatenate([v.ravel() for v in a]) ** 2)))


@pytest.mark.parametrize("H,G,P,N,lens,resumed", [
    (32, 8, 64, 128, [5], "all"),                                 # the last tokens of one prompt
    (128, 8, 64, 128, [1 + i % 5 for i in range(24)], "all"),     # of 24
    (128, 8, 64, 128, [1 + i % 5 for i in range(24)], None),
    (128, 8, 64, 128, [64, 33, 1, 0, 20, 9, 70, 5], "all"),
    (128, 8, 64, 64, [130, 90, 115], "all"),                      # cut
    (256, 8, 16, 16, [300, 170], "all"),
    (64, 8, 128, 32, [100, 60, 3, 2, 1, 7, 30, 9, 20, 11], "all"),
    (2, 1, 32, 128, [700], "all"),
])
def test_bf16_outputs_are_off_by_their_own_rounding(H, G, P, N, lens, resumed):
    import torch
    announce("scan precision", H, G, P, N, lens, resumed)
    p = Prompts(H, G, P, N, lens, resumed, "bf16")
    y, _ = p.run("bf16")
    off, own = [], []
    for i, s, want, S, size, Sa in p.exact():
        e = ((N + 64 + 112 + 4 * (lens[i] / 64 + 1)) * U + 2.0 ** -16) * size
        near(y[s], want, e * (1 + HALF["bf16"]) + HALF["bf16"] * np.abs(want) + 1e-37)
        off.append(y[s] - want)
        own.append(torch.from_numpy(want).to(torch.bfloat16).double().numpy() - want)
    assert _rms(off) <= 1.01 * _rms(own), (_rms(off), _rms(own))
