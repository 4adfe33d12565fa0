"""The fused operators as a hybrid model runs them around an SWA∥RMA layer: a recurrent
block (projection with bias, decayed attention, output projection onto the residual
stream), a gated feed-forward block, then the SWA∥RMA layer's own call, for prompts and
for single tokens.

Every stage is compared with its formula in float64 on the stage's actual input, by the
bars of the operators' own tests.
"""
import pytest
import torch

from tests.test_gpu_decay import Case
from tests.test_gpu_fused_linear import close, gated64, linear64, normal

pytestmark = pytest.mark.gpu

HID, HK, HV, D, FF = 2560, 4, 8, 128, 1736


@pytest.fixture(scope="module")
def sab():
    from sliding_window_anchor_b200 import build
    build.build()
    import sliding_window_anchor_b200 as m
    return m


class Block:
    """One recurrent block and one feed-forward block, random weights."""

    QKV = 2 * HK * D + HV * D

    def __init__(self):
        w = lambda seed, f, k: normal(seed, f, k, scale=k ** -0.5)
        self.w_qkv, self.b_qkv = w(1, self.QKV, HID), normal(2, self.QKV, scale=0.1)
        self.w_g, self.b_g = w(3, HV, HID), normal(4, HV, scale=0.5)
        self.w_o = w(5, HID, HV * D)
        self.w_gate, self.w_up, self.w_down = w(6, FF, HID), w(7, FF, HID), w(8, HID, FF)

    def run(self, sab, x, state, ids, cu=None, check=False):
        """x BF16 [T, HID] → the residual stream behind both blocks."""
        qkv = sab.linear_fused(x, self.w_qkv, bias=self.b_qkv)
        u = sab.linear_fused(x, self.w_g, bias=self.b_g, fp32_out=True)
        g = -torch.nn.functional.softplus(u) * 0.05
        q = qkv[:, :HK * D].unflatten(1, (HK, D))
        k = torch.nn.functional.normalize(qkv[:, HK * D:2 * HK * D].unflatten(1, (HK, D)).float(),
                                          dim=2).to(torch.bfloat16)
        v = qkv[:, 2 * HK * D:].unflatten(1, (HV, D))
        before = state.clone() if check else None
        if cu is None:
            o = sab.decay_decode(state, ids, q, k, v, g)
        else:
            o = sab.decay_prefill(state, ids, cu, q, k, v, g)
        o = o.flatten(1)
        y = sab.linear_fused(o, self.w_o, residual=x)
        h = sab.gated_linear(y, self.w_gate, self.w_up)
        z = sab.linear_fused(h, self.w_down, residual=y)
        if check:
            close(qkv, linear64(x, self.w_qkv, self.b_qkv, "none", None, False))
            close(u, linear64(x, self.w_g, self.b_g, "none", None, True))
            c = Case.__new__(Case)
            c.B, c.HK, c.HV, c.DK, c.DV, c.T = ids.numel(), HK, HV, D, D, x.shape[0]
            c.begin = list(range(x.shape[0] + 1)) if cu is None else cu.tolist()
            c.lengths = [c.begin[b + 1] - c.begin[b] for b in range(c.B)]
            c.ids, c.q, c.k, c.v, c.g, c.state = ids, q, k, v, g, before
            c.check(o.unflatten(1, (HV, D)), state, decode=cu is None)
            close(y, linear64(o, self.w_o, None, "none", x, False))
            close(h, gated64(y, self.w_gate, self.w_up, "silu", False))
            close(z, linear64(h, self.w_down, None, "none", y, False))
        return z


def test_prompts_and_tokens_through_the_blocks(sab):
    """Three prompts of odd lengths, then tokens, into an SWA∥RMA layer."""
    from synth import workloads as wl
    block, lengths = Block(), [70, 1, 201]
    ids = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 70, 71, 272], dtype=torch.int32, device="cuda")
    state = torch.zeros(3, HV, D, D, device="cuda")
    w = sab.LayerWeights.from_dict(wl.make_weights(5, 0, device="cuda"))
    layer = sab.State(3, 1)
    sab.state_init(layer, range(3))
    x = normal(11, 272, HID)
    z = block.run(sab, x, state, ids, cu, check=True)
    for b, row in enumerate(ids.tolist()):
        rows = z[int(cu[b]):int(cu[b + 1])].contiguous()
        out = sab.swa_rma_prefill_chunk(layer, w, 0, row, rows)
        sab.advance(layer, [row], lengths[b])
        assert bool(out.isfinite().all())
    for step in range(4):
        x = normal(20 + step, 3, HID)
        z = block.run(sab, x, state, ids, check=True)
        out = sab.swa_rma_decode(layer, w, 0, ids, z)
        sab.advance(layer, ids)
        assert bool(out.isfinite().all())
    assert sab.last_device_error(layer) == 0 and sab.last_call_error() == 0
    assert [int(layer.meta[r, 0]) for r in ids.tolist()] == [74, 5, 205]


def test_a_captured_step_equals_the_eager_ones(sab):
    """A decode step of both blocks and the layer, captured once and replayed."""
    from synth import workloads as wl
    block = Block()
    ids = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    w = sab.LayerWeights.from_dict(wl.make_weights(5, 0, device="cuda"))
    state, layer = torch.zeros(2, HV, D, D, device="cuda"), sab.State(2, 1)
    state2, layer2 = torch.zeros_like(state), sab.State(2, 1)
    sab.state_init(layer, [0, 1])
    sab.state_init(layer2, [0, 1])
    x, out = normal(30, 2, HID), torch.empty(2, HID, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(sab.decode_workspace_bytes(2), dtype=torch.uint8, device="cuda")

    def step(s, l, to):
        z = block.run(sab, x, s, ids)
        sab.swa_rma_decode(l, w, 0, ids, z, out=to, ws=ws)
        sab.advance(l, ids)

    spare, warm = torch.zeros_like(state), sab.State(2, 1)
    sab.state_init(warm, [0, 1])
    step(spare, warm, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(state, layer, out)
    want = torch.empty_like(out)
    for seed in range(31, 35):
        x.copy_(normal(seed, 2, HID))
        graph.replay()
        torch.cuda.synchronize()
        step(state2, layer2, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(state, state2)
    assert torch.equal(layer.meta, layer2.meta)
