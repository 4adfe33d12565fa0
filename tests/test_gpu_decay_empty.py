"""A state row listed twice is told to the caller whatever the sequences' lengths, empty ones
among them, and whichever launch takes the call's lengths."""
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


@pytest.mark.parametrize("lengths,same", [
    ([4, 0], (0, 1)), ([0, 0, 5], (0, 1)), ([300, 0], (0, 1)), ([0, 300], (0, 1)),
    ([1000, 0, 0], (1, 2)), ([0, 2000, 0, 700, 0], (0, 4)), ([6000, 0, 300], (0, 1)),
    ([200] * 40 + [0], (35, 40)), ([0] * 40 + [9000], (3, 39))])
def test_empty_sequences_with_a_row_twice(sab, lengths, same):
    c = Case(lengths, 2, 2, 64, 64, rows=len(lengths) + 1)
    S = c.state.clone()
    sab.decay_prefill(S, c.ids, c.cu, c.q, c.k, c.v, c.g)
    assert sab.last_call_error() == 0
    ids, first, again = c.ids.clone(), *same
    ids[again] = ids[first]
    S = c.state.clone()
    sab.decay_prefill(S, ids, c.cu, c.q, c.k, c.v, c.g)
    assert sab.last_call_error() == -1 and sab.last_call_error() == 0
    rows = [int(c.ids[b]) for b in range(c.B) if lengths[b] == 0 and b != first and b != again]
    assert torch.equal(S[rows], c.state[rows])


def test_no_token_asks_nothing(sab):
    """A call without tokens launches nothing and looks at nothing on the device."""
    c = Case([0, 0], 2, 2, 64, 64)
    n = sab.launch_count()
    sab.decay_prefill(c.state, [0, 0], [0, 0, 0], c.q, c.k, c.v, c.g)
    assert sab.launch_count() == n and sab.last_call_error() == 0
