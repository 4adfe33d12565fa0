"""The binding of the fused products and the decayed attention on the host: arguments by name,
workspaces by device (CPU only)."""
import contextlib
import inspect
from types import SimpleNamespace

import pytest
import torch

import sliding_window_anchor_b200 as sab

BF = torch.bfloat16
X, W = torch.zeros(4, 64, dtype=BF), torch.zeros(24, 64, dtype=BF)
QK, V = torch.zeros(2, 2, 64, dtype=BF), torch.zeros(2, 4, 64, dtype=BF)
DECAY = dict(state=torch.zeros(2, 4, 64, 64), seq_ids=[0, 1], q=QK, k=QK, v=V,
             log_decay=torch.zeros(2, 4))
CALLS = [("linear_fused", dict(x=X, w=W)), ("gated_linear", dict(x=X, w_gate=W, w_up=W)),
         ("decay_decode", DECAY), ("decay_prefill", dict(DECAY, cu_tokens=[0, 1, 2]))]


@pytest.mark.parametrize("name,args", CALLS)
def test_every_argument_can_be_named(name, args):
    """The call looks at its tensors (which are on no GPU here), whatever way they came."""
    call = getattr(sab, name)
    first = next(iter(args))
    with pytest.raises(ValueError, match=f"{first} must be a CUDA tensor"):
        call(**args)
    with pytest.raises(ValueError, match=f"{first} must be a CUDA tensor"):
        call(args[first], **{n: v for n, v in args.items() if n != first})
    other = SimpleNamespace(device=torch.device("cuda:7"))
    with pytest.raises(ValueError, match="the stream is on cuda:7, the tensors on cpu"):
        call(**args, stream=other)
    with pytest.raises(TypeError, match=f"'{first}'"):
        call(stream=other, **{n: v for n, v in args.items() if n != first})


@pytest.mark.parametrize("name,args", CALLS)
def test_signatures(name, args):
    shown = inspect.signature(getattr(sab, name)).parameters
    assert next(iter(shown)) == next(iter(args)) and set(args) <= set(shown)
    assert shown["stream"].default is None


def test_workspace_size_is_that_of_the_tensors_device(monkeypatch):
    """Devices of different SM counts need workspaces of different sizes for the same call."""
    at = {"current": 0}

    @contextlib.contextmanager
    def device(index):
        was, at["current"] = at["current"], index
        yield
        at["current"] = was

    sizes = {0: 4096, 1: 8192}
    fake = SimpleNamespace(
        er_decay_prefill_workspace_bytes=lambda sh, B, T: sizes[at["current"]] + B + T)
    monkeypatch.setattr(sab, "lib", lambda: fake)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at["current"])
    a = (16, 32, 128, 128, 2, 77773)
    try:
        for current in (0, 1, 0):
            at["current"] = current
            assert sab.decay_prefill_workspace_bytes(*a) == sizes[current] + 77775
            for index in (1, 0):
                assert sab.decay_prefill_workspace_bytes(*a, device=f"cuda:{index}") == \
                    sizes[index] + 77775
                assert sab._prefill_bytes(index, a[:4], *a[4:]) == sizes[index] + 77775
            assert at["current"] == current
    finally:
        sab._prefill_bytes.cache_clear()


def test_workspace_size_without_a_device():
    if torch.cuda.is_available():
        pytest.skip("there is a device")
    assert sab.decay_prefill_workspace_bytes(2, 4, 64, 128, 4, 100) > 0
    assert sab.decay_prefill_workspace_bytes(2, 4, 64, 100, 4, 100) == 0
