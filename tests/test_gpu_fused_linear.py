"""GPU parity of the fused products (er_linear_fused, er_gated_linear) with their formulas
in float64.

Bars, per element, from the arithmetic:
  sums: FP32 accumulation of K exact BF16 products, |Δ| <= 2^-17·Σ|x·w| (as for er_linear)
    plus one FP32 rounding of the bias add;
  activation: SiLU and the GELUs have a slope of at most 1.13, and an FP32 evaluation
    of a few roundings, 2^-20 of |v| + |act(v)|;
  gate product: the product rule over both sums;
  residual and output: one FP32 rounding each (2^-24), and for BF16 out one rounding of
    half a step, 2^-8 of the value.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

ACTS = ("none", "silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def sab():
    from sliding_window_anchor_b200 import build
    build.build()
    import sliding_window_anchor_b200 as m
    return m


def normal(seed, *shape, scale=1.0, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def act64(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * 0.5 * torch.erfc(-v * 0.5 ** 0.5)
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3)))
    return v


def sums64(x, w):
    x, w = x.double(), w.double()
    return x @ w.T, x.abs() @ w.abs().T * 2.0 ** -17


def out_bar(y, fp32):
    return y.abs() * (2.0 ** -23 if fp32 else 2.0 ** -8) + 1e-30


def linear64(x, w, bias, act, residual, fp32):
    v, bar = sums64(x, w)
    if bias is not None:
        v = v + bias.double()
        bar = bar + v.abs() * 2.0 ** -24
    a = act64(v, act)
    bar = 1.13 * bar + (a.abs() + v.abs()) * 2.0 ** -20 * (act != "none")
    y = a if residual is None else a + residual.double()
    return y, bar + out_bar(y, fp32)


def gated64(x, wg, wu, act, fp32):
    g, bg = sums64(x, wg)
    u, bu = sums64(x, wu)
    a = act64(g, act)
    ba = 1.13 * bg + (a.abs() + g.abs()) * 2.0 ** -20 * (act != "none")
    y = a * u
    return y, ba * u.abs() + a.abs() * bu + ba * bu + out_bar(y, fp32)


def close(got, want):
    y, bar = want
    off = (got.double() - y).abs()
    assert bool((off <= bar).all()), float((off / bar).max())


# one token, the tile edges, odd counts; features and depths that fill no tile; the
# layer's projections
SIZES = [(1, 2560, 4096), (1, 1, 8), (2, 3, 16), (5, 63, 72), (8, 4099, 2568), (9, 130, 264),
         (16, 2560, 2560), (17, 96, 1000), (31, 1025, 136), (32, 256, 64), (33, 2560, 4096),
         (64, 777, 520), (100, 2561, 96), (127, 128, 2560), (128, 2560, 4096), (129, 511, 192),
         (200, 3000, 328), (255, 257, 1032), (256, 256, 256), (300, 1100, 2560), (385, 520, 72),
         (512, 2560, 4096), (700, 1411, 200), (1025, 2560, 640), (2050, 333, 136),
         # wide products of a few hundred tokens (tokens as columns), odd ones among them
         (260, 19000, 136), (300, 9000, 264), (301, 18945, 72), (512, 18944, 200),
         (513, 9601, 136), (700, 19001, 72), (100, 9473, 520), (9, 18945, 264), (33, 9500, 72)]


@pytest.mark.parametrize("T,F,K", SIZES)
def test_linear_sizes(sab, T, F, K):
    x, w = normal(T, T, K), normal(F, F, K, scale=K ** -0.5)
    b, r = normal(3, F), normal(4, T, F)
    close(sab.linear_fused(x, w), linear64(x, w, None, "none", None, False))
    close(sab.linear_fused(x, w, bias=b, act="silu", residual=r),
          linear64(x, w, b, "silu", r, False))
    close(sab.linear_fused(x, w, bias=b, act="gelu", residual=r.float(), fp32_out=True),
          linear64(x, w, b, "gelu", r, True))
    assert sab.last_call_error() == 0


@pytest.mark.parametrize("T,F,K", SIZES)
def test_gated_sizes(sab, T, F, K):
    x = normal(T, T, K)
    wg, wu = normal(F, F, K, scale=K ** -0.5), normal(F + 1, F, K, scale=K ** -0.5)
    close(sab.gated_linear(x, wg, wu), gated64(x, wg, wu, "silu", False))
    close(sab.gated_linear(x, wg, wu, act="gelu_tanh", fp32_out=True),
          gated64(x, wg, wu, "gelu_tanh", True))
    assert sab.last_call_error() == 0


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(sab, T, act):
    """Sums from -40 to 40: the activations' tails and their middle."""
    K, F = 64, 801
    x = torch.zeros(T, K, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = 1
    x[:, 1] = 2.0 ** -7 * torch.arange(T, device="cuda") / T
    w = torch.zeros(F, K, device="cuda", dtype=torch.bfloat16)
    w[:, 0] = torch.linspace(-40, 40, F, device="cuda").to(torch.bfloat16)
    w[:, 1] = 1
    u = normal(9, F, K)
    for fp32 in (False, True):
        close(sab.linear_fused(x, w, act=act, fp32_out=fp32),
              linear64(x, w, None, act, None, fp32))
        close(sab.gated_linear(x, w, u, act=act, fp32_out=fp32), gated64(x, w, u, act, fp32))


@pytest.mark.parametrize("T", [1, 7, 20, 100, 300, 600])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("ldy", [520, 521, 527])
def test_row_strides_and_what_lies_between(sab, T, fp32, ldy):
    """x, y and the residual with strides of their own; what lies behind y's columns and
    rows stays as it was; odd strides and bases leave no row 16-byte aligned."""
    F, K = 517, 264
    dt = torch.float32 if fp32 else torch.bfloat16
    x = normal(1, T, K + 24)[:, 8:8 + K]
    w, wu, b = normal(2, F, K, scale=K ** -0.5), normal(5, F, K, scale=K ** -0.5), normal(3, F)
    r = normal(4, T, F + 5, dtype=dt)[:, 3:3 + F]
    for shift in (0, 1):
        for gated in (False, True):
            flat = torch.full((shift + (T + 2) * ldy,), 7.0, dtype=dt, device="cuda")
            whole = flat[shift:].view(T + 2, ldy)
            out = whole[:T, :F]
            if gated:
                got = sab.gated_linear(x, w, wu, fp32_out=fp32, out=out)
                close(got, gated64(x, w, wu, "silu", fp32))
            else:
                got = sab.linear_fused(x, w, bias=b, residual=r, fp32_out=fp32, out=out)
                close(got, linear64(x, w, b, "none", r, fp32))
            assert got is out
            assert bool((whole[:, F:] == 7).all()) and bool((whole[T:] == 7).all())
            assert bool((flat[:shift] == 7).all())


@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("F", [256, 1001])
def test_bias_from_an_odd_element(sab, T, F):
    """Bias and weights that start inside a larger tensor (the bias off 16 bytes)."""
    K = 136
    x, w = normal(1, T, K), normal(2, F + 3, K, scale=K ** -0.5)[3:]
    b = normal(3, F + 5)[5:]
    for fp32 in (False, True):
        close(sab.linear_fused(x, w, bias=b, fp32_out=fp32),
              linear64(x, w, b, "none", None, fp32))
    g = normal(4, 2 * F, K, scale=K ** -0.5)  # the halves of one stacked weight
    close(sab.gated_linear(x, g[:F], g[F:]), gated64(x, g[:F], g[F:], "silu", False))


@pytest.mark.parametrize("T", [1, 24, 90, 520])
def test_residual_in_place_and_repeats(sab, T):
    """The residual may be the output; the same inputs give the same bits."""
    F, K = 2560, 1024
    x, w, r = normal(1, T, K), normal(2, F, K, scale=K ** -0.5), normal(3, T, F)
    want = sab.linear_fused(x, w, residual=r)
    y = r.clone()
    sab.linear_fused(x, w, residual=y, out=y)
    assert torch.equal(y, want)
    close(y, linear64(x, w, None, "none", r, False))
    for _ in range(3):
        assert torch.equal(sab.linear_fused(x, w, residual=r), want)


@pytest.mark.parametrize("T", [1, 3, 40, 300])
def test_infinities_and_nans_stay_in_their_rows(sab, T):
    F, K = 300, 128
    x, w = normal(1, T, K), normal(2, F, K, scale=K ** -0.5)
    clean = sab.linear_fused(x, w)
    gated = sab.gated_linear(x, w, w)
    for bad in (float("inf"), float("nan")):
        y, g = x.clone(), x.clone()
        y[T // 2, 5] = g[T // 2, 5] = bad
        got, got_g = sab.linear_fused(y, w), sab.gated_linear(g, w, w)
        others = [t for t in range(T) if t != T // 2]
        assert torch.equal(got[others], clean[others])
        assert torch.equal(got_g[others], gated[others])
        assert not bool(torch.isfinite(got[T // 2]).any())
    # a feature row of NaN weights touches its own column alone
    wn = w.clone()
    wn[7] = float("nan")
    got = sab.linear_fused(x, wn)
    keep = [f for f in range(F) if f != 7]
    assert torch.equal(got[:, keep], clean[:, keep]) and bool(got[:, 7].isnan().all())


@pytest.mark.parametrize("T", [1, 12, 100, 400])
def test_captured_calls_and_streams(sab, T):
    """A captured call replays on new values; calls on two streams at once give what each
    gives alone."""
    F, K = 1000, 512
    x, w, wu = normal(1, T, K), normal(2, F, K, scale=K ** -0.5), normal(5, F, K, scale=K ** -0.5)
    y, z = torch.empty(T, F, dtype=torch.bfloat16, device="cuda"), None
    sab.linear_fused(x, w, out=y)
    sab.gated_linear(x, w, wu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sab.linear_fused(x, w, act="silu", out=y)
        z = sab.gated_linear(x, w, wu)
    for seed in (6, 7):
        x.copy_(normal(seed, T, K))
        graph.replay()
        torch.cuda.synchronize()
        close(y, linear64(x, w, None, "silu", None, False))
        close(z, gated64(x, w, wu, "silu", False))
    want, want_z = y.clone(), z.clone()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append((sab.linear_fused(x, w, act="silu", stream=one), want))
        got.append((sab.gated_linear(x, w, wu, stream=two), want_z))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)


def test_offsets_past_32_bits(sab):
    """Rows of x and y more than 2^31 elements apart."""
    ld = 1 << 30
    x = torch.empty(3 * ld, dtype=torch.bfloat16, device="cuda")
    rows = x.view(3, ld)[:, :64]
    rows.copy_(normal(1, 3, 64))
    w = normal(2, 40, 64, scale=0.1)
    out = torch.empty(3 * ld, dtype=torch.bfloat16, device="cuda").view(3, ld)[:, :40]
    sab.linear_fused(rows, w, out=out)
    close(out, linear64(rows, w, None, "none", None, False))
    T, ld = 200, 12 << 20
    del x, rows, out
    x = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)[:, :64]
    x.copy_(normal(1, T, 64))
    y = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)[:, :40]
    sab.linear_fused(x, w, out=y)
    close(y, linear64(x, w, None, "none", None, False))
    sab.gated_linear(x, w, w, out=y)
    close(y, gated64(x, w, w, "silu", False))


def test_refusals_on_the_gpu(sab):
    x, w = normal(1, 4, 64), normal(2, 24, 64)
    with pytest.raises(TypeError):
        sab.linear_fused(x.float(), w)
    with pytest.raises(TypeError):
        sab.linear_fused(x, w, residual=normal(1, 4, 24, dtype=torch.float32))
    with pytest.raises(ValueError):
        sab.linear_fused(x, w.cpu())
    with pytest.raises(ValueError):
        sab.linear_fused(x, w, bias=normal(1, 23))
    with pytest.raises(ValueError):
        sab.gated_linear(x, w, normal(2, 25, 64))
    with pytest.raises(sab.ERError):  # K is no multiple of 8
        sab.linear_fused(x[:, :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(sab.ERError):  # rows of x start off 16 bytes
        sab.linear_fused(normal(1, 4, 72)[:, 1:65], w)
    assert sab.linear_fused(x[:0], w).shape == (0, 24)
    assert sab.gated_linear(x[:0], w, w).shape == (0, 24)
