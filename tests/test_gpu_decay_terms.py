"""The state that prompts leave, to the last of the three BF16 terms that its values enter as.

Only one token in 113 has a k, so that a state's element is a sum of few decayed products, and
what one of them loses shows.  Per product, relative to its size, with exponents of less than 8
in all (decays of less than 2^-8):
  three terms of a value of 24 bits lose nothing; its decay is one FP32 exponential of 2^-22 at
  most, of an exponent rounded to 2^-22 (times ln 2), and one product's rounding: 2^-21.1;
  every chunk behind it multiplies by one more such exponential (2^-21.1), the join likewise;
  a sum of so few FP32 values on the tensor cores, in three accumulators, and their two adds: 2^-21
  at most in each chunk that has such a token, and in each that follows.
Together |Δ| <= n · 2^-19.9 · A for n chunks of 128 tokens that the values pass through one after
another: at most all of the prompt's, or what one segment has where it is cut, plus one for each
segment.  A second term less would lose up to 2^-16 of a value: `two` below is what that gives,
and must not pass."""
import math

import pytest
import torch

from tests.test_gpu_decay import Case

CHUNK = 128


def terms(x, n):
    """x (float64) as the sum of n BF16 values, each the rounding of what the others leave."""
    s = torch.zeros_like(x)
    for _ in range(n):
        s = s + (x - s).to(torch.bfloat16).double()
    return s


def exact(S, ids, cu, k, v, g, n=None):
    """The state and the sum of its terms' sizes in float64; n: with each chunk's decayed values
    cut to that many BF16 terms."""
    S = S.double().clone()
    A = S.abs()
    rep = v.shape[1] // k.shape[1]
    for b, row in enumerate(ids):
        for t0 in range(cu[b], cu[b + 1], CHUNK):
            t1 = min(cu[b + 1], t0 + CHUNK)
            G = g[t0:t1].double().cumsum(0)
            w = torch.exp(G[-1] - G)
            vt = v[t0:t1].double() * w[..., None]
            if n:
                vt = terms(vt.float().double(), n)
            kk = k[t0:t1].double().repeat_interleave(rep, 1)
            end = torch.exp(G[-1])[:, None, None]
            S[row] = S[row] * end + torch.einsum("thk,thv->hkv", kk, vt)
            A[row] = A[row] * end + torch.einsum("thk,thv->hkv", kk.abs(), vt.abs())
    return S, A


def sparse(c, seed):
    """All k but every 113th zero."""
    keep = torch.arange(c.T, device=c.k.device) % 113 == seed % 113
    c.k.mul_(keep[:, None, None])


@pytest.mark.gpu
@pytest.mark.parametrize("HK,HV,DK,DV", [(2, 4, 64, 64), (2, 2, 128, 128), (1, 3, 128, 64)])
@pytest.mark.parametrize("lengths,chunks", [([128], 1), ([100], 1), ([256], 2), ([150, 129], 2),
                                            ([700, 90], 6), ([1500], 12)])
def test_states_hold_all_three_terms(HK, HV, DK, DV, lengths, chunks):
    from sliding_window_anchor_b200 import build
    build.build()
    import sliding_window_anchor_b200 as sab
    # -10^-2.6 a token at most: 1500 tokens decay by 2^-5.5
    c = Case(lengths, HK, HV, DK, DV, rate=(-4, -2.6), decay="head")
    sparse(c, 57)
    c.state.zero_()
    S = c.state.clone()
    sab.decay_prefill(S, c.ids, c.cu, c.q, c.k, c.v, c.g)
    assert sab.last_call_error() == 0
    g = c.g.expand(c.T, HV)
    want, A = exact(c.state, c.ids.tolist(), c.cu.tolist(), c.k, c.v, g)
    bar = chunks * 2.0 ** -19.9 * A + 1e-30
    off = (S.double() - want).abs()
    print("worst of the bar", float((off / bar).max()))
    assert bool((off <= bar).all()), float((off / bar).max())


def test_two_terms_would_not_pass():
    """The bar on the CPU: three terms keep far inside it, two break it."""
    gen = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen)
    for T, chunks in ((128, 1), (256, 2), (700, 6)):
        k, v = n(T, 1, 64).to(torch.bfloat16), n(T, 2, 64).to(torch.bfloat16)
        k.mul_((torch.arange(T) % 113 == 57)[:, None, None])
        g = -torch.logspace(-4, -2.6, 2).expand(T, 2)
        S = torch.zeros(1, 2, 64, 64)
        want, A = exact(S, [0], [0, T], k, v, g)
        bar = chunks * 2.0 ** -19.9 * A + 1e-30
        three, two = (exact(S, [0], [0, T], k, v, g, n)[0] for n in (3, 2))
        assert bool(((three - want).abs() <= bar / 8).all())
        assert not bool(((two - want).abs() <= bar).all())
