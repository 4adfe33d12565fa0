"""Refusals of the fused products and of the decayed attention, before anything is
enqueued (CPU only: argument checks of the C entry points and of the binding)."""
import ctypes

import pytest
import torch

OK, W, Y, S, V = (n << 40 for n in range(1, 6))  # aligned addresses that nothing reads
ODD = (1 << 40) + 2   # aligned to two bytes only
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    from sliding_window_anchor_b200 import build, _lib
    build.build()
    return _lib.lib()


@pytest.fixture()
def unlaunched(L):
    before = L.er_launch_count()
    yield L
    assert L.er_launch_count() == before


LINEAR = dict(x=OK, ldx=64, T=4, w=W, F=24, K=64, bias=None, act=0, residual=None, ldr=24, y=Y,
              y_fp32=0, ldy=24, dev_error=None, stream=None)
GATED = dict(x=OK, ldx=64, T=4, w_gate=W, w_up=W, F=24, K=64, act=1, y=Y, y_fp32=0, ldy=24,
             dev_error=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(F=0), dict(F=-8), dict(K=0), dict(K=60, ldx=64), dict(K=-8), dict(ldx=56),
    dict(ldx=68), dict(ldy=23), dict(act=4), dict(act=-1), dict(y_fp32=2), dict(x=None),
    dict(w=None), dict(y=None), dict(x=ODD), dict(w=ODD), dict(y=ODD, y_fp32=1), dict(y=OK + 1),
    dict(residual=OK, ldr=23), dict(residual=OK + 1), dict(residual=ODD, y_fp32=1),
    dict(bias=OK + 1), dict(y=OK), dict(y=W), dict(bias=Y), dict(residual=Y, ldr=32)])
def test_linear_fused_refuses(unlaunched, change):
    assert unlaunched.er_linear_fused(*{**LINEAR, **change}.values()) == -1


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(F=0), dict(K=12), dict(ldx=60), dict(ldy=20), dict(act=9), dict(y_fp32=-1),
    dict(x=None), dict(w_gate=None), dict(w_up=None), dict(y=None), dict(x=ODD), dict(w_gate=ODD),
    dict(w_up=ODD), dict(y=OK + 1), dict(y=ODD, y_fp32=1), dict(y=OK), dict(y=W), dict(w_up=Y)])
def test_gated_linear_refuses(unlaunched, change):
    assert unlaunched.er_gated_linear(*{**GATED, **change}.values()) == -1


def test_no_tokens_launch_nothing(unlaunched):
    assert unlaunched.er_linear_fused(*{**LINEAR, "T": 0, "x": None, "y": None}.values()) == 0
    assert unlaunched.er_gated_linear(*{**GATED, "T": 0, "x": None, "y": None}.values()) == 0


def shape(*dims):
    from sliding_window_anchor_b200._lib import CDecayShape
    return ctypes.byref(CDecayShape(*dims))


def decay_args(prefill, **change):
    a = dict(state=S, s_max=8, seq_ids=OK, cu=OK, B=4, T=100, sh=(2, 4, 64, 128), q=OK, ldq=128,
             k=OK, ldk=128, v=V, ldv=512, g=OK, ldg=4, scale=1.0, o=Y, ldo=512, ws=OK,
             ws_bytes=BIG, dev_error=None, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    a["sh"] = None if a["sh"] is None else shape(*a["sh"])
    if not prefill:
        for n in ("cu", "T", "ws", "ws_bytes"):
            del a[n]
    return list(a.values())


BAD_DECAY = [dict(s_max=0), dict(B=-1), dict(B=65536, s_max=70000), dict(sh=None),
             dict(sh=(0, 4, 64, 64)), dict(sh=(3, 4, 64, 64)), dict(sh=(4, 2, 64, 64)),
             dict(sh=(2, 4, 96, 64)), dict(sh=(2, 4, 64, 32)), dict(sh=(2, 4, 64, 256)),
             dict(sh=(1, 4097, 64, 64)), dict(ldq=120), dict(ldq=132), dict(ldk=64),
             dict(ldv=504), dict(ldv=516), dict(ldo=8), dict(ldo=514), dict(ldg=3), dict(ldg=-4),
             dict(state=None), dict(seq_ids=None), dict(q=None), dict(k=None), dict(v=None),
             dict(g=None), dict(o=None), dict(state=ODD), dict(q=ODD), dict(k=ODD), dict(v=ODD),
             dict(o=ODD), dict(g=ODD), dict(seq_ids=ODD), dict(o=OK), dict(o=V), dict(o=S)]


@pytest.mark.parametrize("change", BAD_DECAY)
def test_decay_calls_refuse(unlaunched, change):
    assert unlaunched.er_decay_decode(*decay_args(False, **change)) == -1
    assert unlaunched.er_decay_prefill(*decay_args(True, **change)) == -1


def test_decay_capacity_and_workspace(unlaunched):
    L = unlaunched
    assert L.er_decay_decode(*decay_args(False, B=9)) == -2
    assert L.er_decay_prefill(*decay_args(True, B=9)) == -2
    assert L.er_decay_prefill(*decay_args(True, T=-1)) == -1
    assert L.er_decay_prefill(*decay_args(True, cu=None)) == -1
    assert L.er_decay_prefill(*decay_args(True, cu=ODD)) == -1
    assert L.er_decay_prefill(*decay_args(True, ws=None)) == -1
    assert L.er_decay_prefill(*decay_args(True, ws=OK + 16)) == -1
    need = L.er_decay_prefill_workspace_bytes(shape(2, 4, 64, 128), 4, 100)
    assert need > 0
    assert L.er_decay_prefill(*decay_args(True, ws_bytes=need - 1)) == -2
    assert L.er_decay_prefill_workspace_bytes(None, 4, 100) == 0
    assert L.er_decay_prefill_workspace_bytes(shape(2, 4, 64, 100), 4, 100) == 0
    assert L.er_decay_prefill_workspace_bytes(shape(2, 4, 64, 128), 0, 100) == 0
    assert L.er_decay_prefill_workspace_bytes(shape(2, 4, 64, 128), 4, -1) == 0
    # nothing to do: nothing is launched, and pointers are not looked at
    assert L.er_decay_decode(*decay_args(False, B=0, state=None, q=None)) == 0
    assert L.er_decay_prefill(*decay_args(True, B=0, state=None, q=None)) == 0
    assert L.er_decay_prefill(*decay_args(True, T=0, q=None, ws=None)) == 0


def test_binding_refuses_on_the_host(unlaunched):
    import sliding_window_anchor_b200 as sab
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(24, 64, dtype=bf)
    with pytest.raises(ValueError):
        sab.linear_fused(x, w)  # not on a GPU
    with pytest.raises(ValueError):
        sab.gated_linear(x, w, w)
    S = torch.zeros(2, 4, 64, 64)
    q, v = torch.zeros(2, 2, 64, dtype=bf), torch.zeros(2, 4, 64, dtype=bf)
    with pytest.raises(ValueError):
        sab.decay_decode(S, [0, 1], q, q, v, torch.zeros(2, 4))
    with pytest.raises(ValueError):
        sab.decay_prefill(S, [0, 1], [0, 1, 2], q, q, v, torch.zeros(2, 4))


@pytest.mark.parametrize("make,err", [
    (lambda: torch.zeros(4, 64), TypeError),
    (lambda: torch.zeros(4, 65, dtype=torch.bfloat16), ValueError),
    (lambda: torch.zeros(3, 64, dtype=torch.bfloat16), ValueError),
    (lambda: torch.zeros(64, 4, dtype=torch.bfloat16).T, ValueError),
    (lambda: torch.zeros(1, 64, dtype=torch.bfloat16).expand(4, 64), ValueError),
    (lambda: torch.zeros(4, 64, dtype=torch.bfloat16, device="meta"), ValueError)])
def test_row_arguments(make, err):
    from sliding_window_anchor_b200 import _arg
    with pytest.raises(err):
        _arg(make(), torch.device("cpu"), torch.bfloat16, (4, 64), "x")


def test_row_arguments_accept_strided_rows():
    from sliding_window_anchor_b200 import _arg
    rows = torch.zeros(4, 200, dtype=torch.bfloat16)
    cpu, bf = torch.device("cpu"), torch.bfloat16
    p, ld = _arg(rows[:, 40:168].unflatten(1, (2, 64)), cpu, bf, (4, 2, 64), "q")
    assert (p, ld) == (rows.data_ptr() + 80, 200)
    # one row alone: its stride says nothing
    assert _arg(rows[:1, 40:168], cpu, bf, (1, 128), "x")[1] == 128
    with pytest.raises(ValueError):
        from sliding_window_anchor_b200 import _act
        _act("tanh")
