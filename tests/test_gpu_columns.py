"""Products whose tokens are the columns of one tile a pair (k_columns): a few hundred tokens
by so many features that tiles of 256 tokens would need a second round, and gated products of
up to 64 tokens over many features.  Compared with float64 by the bars of the fused products'
own tests; what ran is read from the launches' names."""
import pytest
import torch

from tests.test_gpu_fused_linear import close, gated64, linear64, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sab():
    from sliding_window_anchor_b200 import build
    build.build()
    import sliding_window_anchor_b200 as m
    return m


def takes_columns(call):
    """Whether k_columns is among the kernels that a call launches (True as well where the
    profiler reports none of the call's launches)."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    names = [e.name for e in prof.events() if "k_" in e.name]
    return not names or any("k_columns" in n for n in names)


# two accumulators of 160, 224 and 256 tokens; from 385 tokens of N = 448 and 512 on the sums
# go out in two passes; odd F and K
LINEAR = [(257, 9985, 1032), (260, 18000, 2000), (300, 12288, 2560), (300, 18944, 520),
          (385, 18944, 2568), (400, 11003, 4104), (511, 10241, 5000), (512, 12288, 8192)]
# one accumulator of 32 and 64 tokens, and two
GATED = [(9, 5000, 1000), (33, 9000, 2560), (64, 9472, 520), (257, 4737, 1032),
         (300, 9000, 2560), (385, 6911, 2568), (500, 9400, 8192)]


@pytest.mark.parametrize("T,F,K", LINEAR)
def test_linear(sab, T, F, K):
    x, w = normal(T, T, K), normal(F, F, K, scale=K ** -0.5)
    b, r = normal(3, F), normal(4, T, F)
    assert takes_columns(lambda: sab.linear_fused(x, w))
    close(sab.linear_fused(x, w), linear64(x, w, None, "none", None, False))
    close(sab.linear_fused(x, w, bias=b, act="silu", residual=r),
          linear64(x, w, b, "silu", r, False))
    close(sab.linear_fused(x, w, bias=b, act="gelu", residual=r.float(), fp32_out=True),
          linear64(x, w, b, "gelu", r, True))
    close(sab.linear_fused(x, w, act="gelu_tanh", fp32_out=True),
          linear64(x, w, None, "gelu_tanh", None, True))
    assert sab.last_call_error() == 0


@pytest.mark.parametrize("T,F,K", GATED)
def test_gated(sab, T, F, K):
    x = normal(T, T, K)
    wg, wu = normal(F, F, K, scale=K ** -0.5), normal(F + 1, F, K, scale=K ** -0.5)
    assert takes_columns(lambda: sab.gated_linear(x, wg, wu))
    for act in ("none", "silu", "gelu", "gelu_tanh"):
        close(sab.gated_linear(x, wg, wu, act=act), gated64(x, wg, wu, act, False))
        close(sab.gated_linear(x, wg, wu, act=act, fp32_out=True), gated64(x, wg, wu, act, True))
    assert sab.last_call_error() == 0


@pytest.mark.parametrize("T,F,K", [(300, 9985, 1032), (400, 11003, 4104)])
def test_strides_repeats_and_replay(sab, T, F, K):
    """Rows of y and of the residual that are no whole 16-byte units, the residual in place,
    what lies between the rows; the same bits again, and from a captured call."""
    x, w, b = normal(1, T, K + 8)[:, :K], normal(2, F, K, scale=K ** -0.5), normal(3, F + 1)[1:]
    for fp32 in (False, True):
        dt = torch.float32 if fp32 else torch.bfloat16
        r = normal(4, T, F, dtype=dt)
        whole = torch.full((T + 1, F + 3), 7.0, dtype=dt, device="cuda")
        y = whole[:T, 1:1 + F]
        y.copy_(r)
        got = sab.linear_fused(x, w, bias=b, residual=y, fp32_out=fp32, out=y)
        close(got, linear64(x, w, b, "none", r, fp32))
        assert bool((whole[:, 0] == 7).all()) and bool((whole[:, 1 + F:] == 7).all())
        assert bool((whole[T] == 7).all())
        want = got.clone()
        dense = sab.linear_fused(x, w, bias=b, residual=r, fp32_out=fp32)
        assert torch.equal(dense, want)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            again = sab.linear_fused(x, w, bias=b, residual=r, fp32_out=fp32)
        for _ in range(3):
            again.zero_()
            graph.replay()
            assert torch.equal(again, want)
    assert sab.last_call_error() == 0


@pytest.mark.parametrize("T,F,K", [(300, 12288, 2560), (512, 10241, 5000)])
def test_non_finite_values_stay_in_their_rows(sab, T, F, K):
    x, w = normal(1, T, K), normal(2, F, K, scale=K ** -0.5)
    clean = sab.linear_fused(x, w)
    for bad in (float("inf"), float("nan")):
        y, wn = x.clone(), w.clone()
        y[T // 2, 5] = bad
        got = sab.linear_fused(y, w)
        others = [t for t in range(T) if t != T // 2]
        assert torch.equal(got[others], clean[others])
        assert not bool(got[T // 2].isfinite().any())
        wn[7, 3] = bad
        got = sab.linear_fused(x, wn)
        keep = [f for f in range(F) if f != 7]
        assert torch.equal(got[:, keep], clean[:, keep]) and not bool(got[:, 7].isfinite().any())
