"""A NaN log-decay of one token, wherever it stands among the four tokens of a lane, the 32
of a block, the chunk or the segment: its head is NaN from that token on, and nothing in
front of it, of another head or of another sequence depends on it."""
import math

import pytest
import torch

from tests.test_gpu_decay import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sab():
    from sliding_window_anchor_b200 import build
    build.build()
    import sliding_window_anchor_b200 as m
    return m


def check(sab, c, at, head):
    n = c.lengths[0]
    S, N = c.state.clone(), c.state.clone()
    clean = sab.decay_prefill(S, c.ids, c.cu, c.q, c.k, c.v, c.g)
    c.g[at, head] = math.nan
    o = sab.decay_prefill(N, c.ids, c.cu, c.q, c.k, c.v, c.g)
    assert sab.last_call_error() == 0
    rest = [h for h in range(c.HV) if h != head]
    assert torch.equal(o[:, rest], clean[:, rest])
    early = [t for t in range(at) if not torch.equal(o[t, head], clean[t, head])]
    assert early == [], (at, early)
    assert torch.equal(o[n:], clean[n:])
    assert bool(o[at:n, head].isnan().all())
    a, b = c.ids.tolist()
    assert bool(N[a, head].isnan().all()) and torch.equal(N[b], S[b])
    assert torch.equal(N[a, rest], S[a, rest])


# by the tokens of few (12), a chunk and parts of one
@pytest.mark.parametrize("n,at", [(12, t) for t in (1, 6, 11)] + [
    (200, t) for t in (1, 2, 3, 31, 33, 34, 35, 63, 65, 97, 101, 102, 103, 127, 129, 130, 131,
                       198, 199)])
@pytest.mark.parametrize("DK,DV", [(64, 64), (128, 128)])
def test_nan_decay_reaches_no_earlier_token(sab, n, at, DK, DV):
    check(sab, Case([n, 150], 2, 4, DK, DV), at, 2)


@pytest.mark.parametrize("at", [2, 1281, 4098, 4227, 8998, 8999])
def test_nan_decay_within_a_cut_prompt(sab, at):
    check(sab, Case([9000, 40], 1, 2, 64, 64, rate=(-5, -4)), at, 1)
