"""The activations relative to their own size, down to where they leave the normal numbers.

Every sum here is one BF16 value times 1, so exact.  Bars, relative to |act(v)|, in units of
2^-23 (one unit in the last place of FP32 at most):
  gelu = v Φ(v), for v < 0 v · t P(t) e^(-v²/2), t = 1 / (1 + 0.305|v|): the exponent is off by
    three roundings of 2^-24 of v²/2, 0.75 v² units; beside them the quotient by 2.5, of which at
    most 2.62 times as much reaches t P(t); P by 4.8 in its evaluation and 0.8 in its fit; the
    exponential by 2, three products by 1.5: 16 + 0.75 v²; for v >= 0, where it is
    v (1 - ...), no more;
  silu = v / (1 + e^-v): the exponential is off by 2 + 1.18|v| units, the sum and the quotient
    by 3: 5 + 1.18|v|;
  gelu_tanh = v / (1 + e^-z), z = 1.596 (v + 0.0447 v³): z is off by seven roundings of 2^-24,
    3.5|z| units of the exponential, beside the same as silu's: 5 + 4.7|z|.
Beside them the result's own rounding, 2^-8 for BF16 and 2^-24 for FP32.  Results below 2^-118
(silu, gelu_tanh) or 2^-126 (gelu) may be zero."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sab():
    from sliding_window_anchor_b200 import build
    build.build()
    import sliding_window_anchor_b200 as m
    return m


def want(v, act):
    """act(v) in float64 without cancellation, its relative bar, and what may be zero."""
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v * math.sqrt(0.5)), (16 + 0.75 * v * v) * 2.0 ** -23, 2.0 ** -126
    z = v if act == "silu" else math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)
    units = 5 + (1.18 if act == "silu" else 4.7) * z.abs()
    return v * torch.sigmoid(z), units * 2.0 ** -23, 2.0 ** -118


# one token, tiles of tokens, tokens as columns
@pytest.mark.parametrize("T,F,K", [(1, 641, 8), (40, 641, 8), (300, 641, 64), (300, 12288, 2560)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("fp32", [False, True])
def test_tails(sab, T, F, K, act, fp32):
    bf = torch.bfloat16
    x = torch.zeros(T, K, dtype=bf, device="cuda")
    x[:, 0] = 1
    w, one = (torch.zeros(F, K, dtype=bf, device="cuda") for _ in range(2))
    w[:, 0] = torch.linspace(-16, 16, F, device="cuda").to(bf)
    one[:, 0] = 1
    v = w[:, 0].double().expand(T, F)
    y, rel, floor = want(v, act)
    bar = y.abs() * (rel + (2.0 ** -24 if fp32 else 2.0 ** -8)) + floor
    for got in (sab.linear_fused(x, w, act=act, fp32_out=fp32),
                sab.gated_linear(x, w, one, act=act, fp32_out=fp32)):
        off = (got.double() - y).abs()
        worst = int((off / bar).argmax())
        assert bool((off <= bar).all()), (float(v.reshape(-1)[worst]),
                                          float(got.reshape(-1)[worst]),
                                          float(y.reshape(-1)[worst]))
    assert sab.last_call_error() == 0
