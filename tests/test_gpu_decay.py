"""GPU parity of the linear attention with a decay for each head (er_decay_decode,
er_decay_prefill) with the recurrence in float64, token by token.

Bars, per element.  Beside the state S runs A = e^g A + |k| |v|ᵀ (from |S_0|), the sum of
the terms' sizes, and beside o runs m = |scale| · Aᵀ |q|:
  state: every term enters as BF16 parts (of two, 2^-16 is lost at most; the kernel takes
    three), decayed by a few FP32 exponentials and summed in FP32: |Δ| <= 2^-15·A;
  o: each term meets one BF16 rounding on its way (of the masked q·k product, or of the
    state it is read from), 2^-8 of it, and the sum is rounded once:
    |Δ| <= (2^-8 + 2^-14)·m + 2^-8·|o|.
Decodes keep FP32 throughout: |Δ| <= 2^-18·A, and 2^-16·m + 2^-8·|o|.
"""
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


class Case:
    """Inputs of sequences of the given lengths; q, k and v are slices of packed rows."""

    def __init__(self, lengths, HK, HV, DK, DV, seed=0, rows=None, lead=0, tail=0, decay="token",
                 rate=(-3.5, -0.15)):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed + 1000 * len(lengths) + sum(lengths))
        n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        B = len(lengths)
        self.B, self.HK, self.HV, self.DK, self.DV = B, HK, HV, DK, DV
        ends = torch.tensor([0] + list(lengths)).cumsum(0) + lead
        self.T = int(ends[-1]) + tail
        self.lengths, self.begin = list(lengths), ends.tolist()
        self.cu = ends.to(torch.int32).cuda()
        x = n(self.T, 2 * HK * DK + HV * DV).to(torch.bfloat16)
        x[:, HK * DK:2 * HK * DK].mul_(DK ** -0.5)
        self.x = x
        self.q = x[:, :HK * DK].unflatten(1, (HK, DK))
        self.k = x[:, HK * DK:2 * HK * DK].unflatten(1, (HK, DK))
        self.v = x[:, 2 * HK * DK:].unflatten(1, (HV, DV))
        r = torch.logspace(*rate, HV, device="cuda")
        self.g = -r if decay == "head" else -r * n(self.T, HV).abs()
        rows = rows or B
        self.ids = torch.randperm(rows, generator=gen, device="cuda")[:B].to(torch.int32)
        self.state = n(rows, HV, DK, DV)

    def want(self, scale=None):
        """(o, its bar's m, state, its bar's A), float64; rows of no sequence are NaN in o."""
        scale = self.DK ** -0.5 if scale is None else scale
        head = torch.arange(self.HV, device="cuda") // (self.HV // self.HK)
        S, A = self.state.double(), self.state.double().abs()
        o = torch.full((self.T, self.HV, self.DV), math.nan, dtype=torch.float64, device="cuda")
        m = o.clone()
        g = self.g.double().expand(self.T, self.HV)
        for t in range(max(self.lengths, default=0)):
            on = [b for b in range(self.B) if self.lengths[b] > t]
            at = torch.tensor([self.begin[b] + t for b in on], device="cuda")
            ids = self.ids[on].long()
            a = g[at].exp()[..., None, None]
            q, k, v = (y[at].double() for y in (self.q, self.k, self.v))
            q, k = q[:, head, :, None], k[:, head, :, None]
            v = v[:, :, None, :]
            new, mag = S[ids] * a + k * v, A[ids] * a + (k * v).abs()
            S[ids], A[ids] = new, mag
            o[at], m[at] = scale * (q * new).sum(2), abs(scale) * (q.abs() * mag).sum(2)
        return o, m, S, A

    def check(self, o, state, decode=False, scale=None):
        want, m, S, A = self.want(scale)
        off = (state.double() - S).abs()
        bar = A * (2.0 ** -18 if decode else 2.0 ** -15) + 1e-30
        assert bool((off <= bar).all()), float((off / bar).max())
        there = ~want.isnan()
        off = (o.double() - want).abs()[there]
        bar = (m * (2.0 ** -16 if decode else 2.0 ** -8 + 2.0 ** -14) + want.abs() * 2.0 ** -8)
        bar = bar[there] + 1e-30
        assert bool((off <= bar).all()), float((off / bar).max())
        return there


HEADS = [(1, 1, 64, 64), (2, 4, 64, 128), (3, 3, 128, 64), (4, 16, 128, 128), (16, 32, 128, 128)]


@pytest.mark.parametrize("HK,HV,DK,DV", HEADS)
@pytest.mark.parametrize("B", [1, 2, 7, 33])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_decode(sab, B, HK, HV, DK, DV, decay):
    c = Case([1] * B, HK, HV, DK, DV, rows=B + 3, decay=decay)
    S = c.state.clone()
    o = sab.decay_decode(S, c.ids, c.q, c.k, c.v, c.g)
    assert sab.last_call_error() == 0
    c.check(o, S, decode=True)
    others = [r for r in range(B + 3) if r not in c.ids.tolist()]
    assert torch.equal(S[others], c.state[others])
    # the same inputs, the same bits; another scale
    again = c.state.clone()
    assert torch.equal(sab.decay_decode(again, c.ids, c.q, c.k, c.v, c.g), o)
    assert torch.equal(again, S)
    S = c.state.clone()
    c.check(sab.decay_decode(S, c.ids, c.q, c.k, c.v, c.g, scale=-3.0), S, True, -3.0)


@pytest.mark.parametrize("HK,HV,DK,DV", HEADS)
@pytest.mark.parametrize("lengths", [
    [1], [2], [63], [64], [65], [127], [128], [129], [200], [256], [513], [1000],
    [1, 1, 1], [5, 0, 70, 0], [0, 130], [300, 1, 64, 129, 17, 0, 255, 128]])
def test_prefill(sab, lengths, HK, HV, DK, DV):
    decay = "head" if len(lengths) % 2 == 0 else "token"
    c = Case(lengths, HK, HV, DK, DV, rows=len(lengths) + 2, lead=3, tail=70, decay=decay)
    S = c.state.clone()
    out = torch.full((c.T, HV, DV), 7.0, dtype=torch.bfloat16, device="cuda")
    sab.decay_prefill(S, c.ids, c.cu, c.q, c.k, c.v, c.g, out=out)
    assert sab.last_call_error() == 0
    there = c.check(out, S)
    # rows of no sequence, states of no sequence, states of empty sequences
    assert bool((out[~there] == 7).all())
    empty = [int(c.ids[b]) for b in range(c.B) if lengths[b] == 0]
    others = [r for r in range(c.B + 2) if r not in c.ids.tolist()] + empty
    assert torch.equal(S[others], c.state[others])
    again, out2 = c.state.clone(), torch.full_like(out, 7.0)
    sab.decay_prefill(again, c.ids, c.cu, c.q, c.k, c.v, c.g, out=out2)
    assert torch.equal(again, S) and torch.equal(out, out2)


@pytest.mark.parametrize("HK,HV,DK,DV", HEADS)
@pytest.mark.parametrize("lengths", [
    [3], [16], [17], [4] * 3, [16] * 40, [2, 0, 7, 16, 1, 5, 0, 13], [1] * 300, [0] * 40 + [9],
    [1] * 50 + [700], [17, 16, 15] * 12, [30] * 9, [600] + [3] * 70])
def test_short_sequences(sab, lengths, HK, HV, DK, DV):
    """Sequences of few tokens, alone and among longer ones.  Where all have 16 at most, each
    step costs an exponential (2^-22) and a rounding (2^-24) of A: together 2^-17 at most."""
    decay = "head" if len(lengths) % 3 == 0 else "token"
    c = Case(lengths, HK, HV, DK, DV, rows=len(lengths) + 2, decay=decay)
    S = c.state.clone()
    o = sab.decay_prefill(S, c.ids, c.cu, c.q, c.k, c.v, c.g)
    assert sab.last_call_error() == 0
    c.check(o, S)
    if max(lengths) <= 16:
        _, _, want, A = c.want()
        assert bool(((S.double() - want).abs() <= 2.0 ** -17 * A + 1e-30).all())
    unused = [r for r in range(c.B + 2) if r not in c.ids.tolist()]
    unused += [int(c.ids[b]) for b in range(c.B) if lengths[b] == 0]
    assert torch.equal(S[unused], c.state[unused])
    again = c.state.clone()
    assert torch.equal(sab.decay_prefill(again, c.ids, c.cu, c.q, c.k, c.v, c.g), o)
    assert torch.equal(again, S)


@pytest.mark.parametrize("lengths", [[3, 4, 5, 2], [3, 200, 5, 20]])
def test_short_sequences_with_bad_rows(sab, lengths):
    c = Case(lengths, 2, 4, 64, 64, rows=6)
    for at, bad in ((2, -1), (2, 6), (2, int(c.ids[0])), (3, int(c.ids[1]))):
        ids = c.ids.clone()
        ids[at] = bad
        S, out = c.state.clone(), torch.full((c.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        sab.decay_prefill(S, ids, c.cu, c.q, c.k, c.v, c.g, out=out)
        assert sab.last_call_error() == -1 and sab.last_call_error() == 0
        d = Case(lengths, 2, 4, 64, 64, rows=6)
        d.lengths[at] = 0
        there = d.check(out, S)
        assert bool((out[~there] == 7).all())
        assert int((~there).all(2).all(1).sum()) == lengths[at]


@pytest.mark.parametrize("HK,HV,DK,DV,n", [(1, 1, 128, 128, 9000), (1, 2, 64, 64, 20011),
                                           (2, 2, 64, 128, 4097), (1, 1, 128, 64, 6300)])
def test_long_prompts(sab, HK, HV, DK, DV, n):
    """Lengths that are split over many blocks, beside a short one."""
    c = Case([n, 40], HK, HV, DK, DV, rate=(-4.5, -1))
    S = c.state.clone()
    c.check(sab.decay_prefill(S, c.ids, c.cu, c.q, c.k, c.v, c.g), S)
    assert sab.last_call_error() == 0


@pytest.mark.parametrize("cuts", [[1], [64], [100, 101, 356], [128, 256]])
def test_prefill_in_pieces_equals_prefill_and_decode(sab, cuts):
    """Prompts cut anywhere, single tokens by the decode call among them."""
    c = Case([400], 2, 4, 128, 128)
    whole = c.state.clone()
    o = sab.decay_prefill(whole, c.ids, c.cu, c.q, c.k, c.v, c.g)
    c.check(o, whole)
    S, parts = c.state.clone(), []
    for a, b in zip([0] + cuts, cuts + [400]):
        at = slice(a, b)
        if b - a == 1:
            parts.append(sab.decay_decode(S, c.ids, c.q[at], c.k[at], c.v[at], c.g[at]))
        else:
            parts.append(sab.decay_prefill(S, c.ids, [0, b - a], c.q[at], c.k[at], c.v[at],
                                           c.g[at]))
    c.check(torch.cat(parts), S)


@pytest.mark.parametrize("n", [1, 70, 300, 3000])
def test_decays_at_their_ends(sab, n):
    """No decay at all; a decay that forgets everything (-inf, -2000, -150) at some tokens,
    the first and the last of a sequence and of a block among them; strong decays beside
    weak ones; growth."""
    c = Case([n, n], 1, 3, 64, 64, rate=(-5, -3))
    c.g[:, 0] = 0
    cut = [t for t in (0, 5, 63, 64, 127, 128, 191, n - 1) if t < n]
    for j, b in enumerate((-math.inf, -2000.0, -150.0)):
        c.g[cut[j % len(cut)::2], 1] = b
    c.g[n + torch.tensor(cut, device="cuda"), 1] = -math.inf
    c.g[:, 2] = torch.where(torch.arange(2 * n, device="cuda") % 7 == 3, -30.0, 1e-3)
    if n > 1000:
        c.g[:, 2] = -0.5
    S = c.state.clone()
    o = sab.decay_prefill(S, c.ids, c.cu, c.q, c.k, c.v, c.g)
    assert bool(o.isfinite().all()) and bool(S.isfinite().all())
    c.check(o, S)
    if n == 1:
        S = c.state.clone()
        c.check(sab.decay_decode(S, c.ids, c.q, c.k, c.v, c.g), S, True)


def test_nan_stays_in_its_head_and_behind_its_token(sab):
    c = Case([200, 150], 2, 4, 64, 64)
    S = c.state.clone()
    clean = sab.decay_prefill(S, c.ids, c.cu, c.q, c.k, c.v, c.g)
    c.g[100, 2] = math.nan  # sequence 0, head 2, its 101st token
    N = c.state.clone()
    o = sab.decay_prefill(N, c.ids, c.cu, c.q, c.k, c.v, c.g)
    heads = [0, 1, 3]
    assert torch.equal(o[:, heads], clean[:, heads])
    assert torch.equal(o[:100, 2], clean[:100, 2]) and torch.equal(o[200:], clean[200:])
    assert bool(o[100:200, 2].isnan().all())
    a, b = c.ids.tolist()
    assert bool(N[a, 2].isnan().all()) and torch.equal(N[b], S[b])
    assert torch.equal(N[a, heads], S[a, heads])


@pytest.mark.parametrize("n,at", [(1, 0), (150, 0), (150, 63), (150, 149), (300, 130), (2000, 700)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_non_finite_values_reach_no_earlier_token(sab, n, at, bad):
    """An infinite or NaN v: its column of its head from its token on, and of the state; k:
    its head from its token on; q: its own token's heads.  Nothing in front, beside, or of
    another sequence."""
    c = Case([n, 90], 2, 4, 128, 64, rate=(-5, -3))
    S = c.state.clone()
    clean = sab.decay_prefill(S, c.ids, c.cu, c.q, c.k, c.v, c.g)
    a, b = c.ids.tolist()

    def spoiled(part, where):
        keep = part[at][where].clone()
        part[at][where] = bad
        N = c.state.clone()
        o = sab.decay_prefill(N, c.ids, c.cu, c.q, c.k, c.v, c.g)
        part[at][where] = keep
        assert torch.equal(o[:at], clean[:at]) and torch.equal(o[n:], clean[n:])
        assert torch.equal(N[b], S[b])
        return o, N

    o, N = spoiled(c.v, (1, 37))
    rest = torch.ones(4, 64, dtype=torch.bool, device="cuda")
    rest[1, 37] = False
    assert torch.equal(o[:, rest], clean[:, rest])
    assert not bool(o[at:n, 1, 37].isfinite().any())
    assert torch.equal(N[a].transpose(1, 2)[rest], S[a].transpose(1, 2)[rest])
    assert not bool(N[a, 1, :, 37].isfinite().any())

    o, N = spoiled(c.k, (0, 5))  # heads 0 and 1
    assert torch.equal(o[:, 2:], clean[:, 2:]) and torch.equal(N[a, 2:], S[a, 2:])
    assert not bool(o[at, :2].isfinite().any())
    assert not bool(N[a, :2, 5].isfinite().any())

    o, N = spoiled(c.q, (1, 0))  # heads 2 and 3
    assert torch.equal(N, S) and torch.equal(o[:, :2], clean[:, :2])
    assert torch.equal(o[at + 1:], clean[at + 1:])
    assert not bool(o[at, 2:].isfinite().any())


def test_bad_rows_are_skipped_and_told(sab):
    """State rows out of range or listed twice, rows of tokens out of range."""
    c = Case([60, 70, 80, 90], 2, 2, 64, 64, rows=6)
    ids = c.ids.clone()
    for bad in (-1, 6, 1 << 30, int(ids[0])):
        ids[2] = bad
        S, out = c.state.clone(), torch.full((c.T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        sab.decay_prefill(S, ids, c.cu, c.q, c.k, c.v, c.g, out=out)
        assert sab.last_call_error() == -1 and sab.last_call_error() == 0
        d = Case([60, 70, 80, 90], 2, 2, 64, 64, rows=6)
        d.lengths[2] = 0
        there = d.check(out, S)
        assert bool((out[~there] == 7).all()) and int((~there).all(2).all(1).sum()) == 80
        S = c.state.clone()
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        first = c.q[:4], c.k[:4], c.v[:4], c.g[:4]
        out = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        sab.decay_decode(S, ids, *first, out=out, dev_error=word)
        assert int(word) == -1 and sab.last_call_error() == 0
        good, want = c.state.clone(), out.clone()
        keep = [0, 1, 3]
        o = sab.decay_decode(good, c.ids[keep], *(y[keep] for y in first))
        want[keep] = o
        want[2] = 7
        assert torch.equal(S, good) and torch.equal(out, want)
    for cu in ([0, 60, 130, 120, 300], [-1, 60, 130, 210, 300], [0, 60, 130, 210, 301],
               [0, 60, 1 << 30, 210, 300]):
        S, out = c.state.clone(), torch.full((c.T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        sab.decay_prefill(S, c.ids, cu, c.q, c.k, c.v, c.g, out=out)
        assert sab.last_call_error() == -1
        for b in range(4):
            fine = 0 <= cu[b] <= cu[b + 1] <= c.T
            row = int(c.ids[b])
            assert fine or torch.equal(S[row], c.state[row])


@pytest.mark.parametrize("lengths", [[1] * 5, [300, 20], [3000, 7]])
def test_captured_calls_and_streams(sab, lengths):
    c = Case(lengths, 2, 4, 128, 128)
    decode = max(lengths) == 1
    S = c.state.clone()
    ws = torch.empty(sab.decay_prefill_workspace_bytes(2, 4, 128, 128, c.B, c.T),
                     dtype=torch.uint8, device="cuda")

    def call(state, **kw):
        if decode:
            return sab.decay_decode(state, c.ids, c.q, c.k, c.v, c.g, **kw)
        return sab.decay_prefill(state, c.ids, c.cu, c.q, c.k, c.v, c.g, **kw)

    call(c.state.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call(S) if decode else call(S, ws=ws)
    for seed in (3, 4):
        d = Case(lengths, 2, 4, 128, 128, seed=seed)
        c.x.copy_(d.x), c.g.copy_(d.g), S.copy_(d.state)
        c.state = d.state
        graph.replay()
        torch.cuda.synchronize()
        c.check(o, S, decode)
    # two streams at once, each with states of its own
    want_s, want = c.state.clone(), None
    want = call(want_s)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    states = [c.state.clone() for _ in range(20)]
    torch.cuda.synchronize()
    got = [call(s, stream=streams[i % 2]) for i, s in enumerate(states)]
    torch.cuda.synchronize()
    assert all(torch.equal(s, want_s) for s in states)
    assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("lengths,heads", [([16000], (8, 16, 128, 128)),
                                           ([900, 33, 2000], (4, 8, 64, 64))])
def test_many_calls_in_a_row(sab, lengths, heads):
    """Calls behind one another, enough of them for a warp that runs ahead of another to
    show: every one gives the same bits, and no wait gives up."""
    c = Case(lengths, *heads)
    want_s = c.state.clone()
    want = sab.decay_prefill(want_s, c.ids, c.cu, c.q, c.k, c.v, c.g)
    states = [c.state.clone() for _ in range(4)]
    for _ in range(40):
        for s in states:
            s.copy_(c.state)
        outs = [sab.decay_prefill(s, c.ids, c.cu, c.q, c.k, c.v, c.g) for s in states]
        assert all(torch.equal(s, want_s) for s in states)
        assert all(torch.equal(o, want) for o in outs)
    assert sab.last_call_error() == 0
    c.check(want, want_s)


def test_offsets_past_32_bits(sab):
    """State rows, and token rows, more than 2^31 elements from the first."""
    rows = 2 ** 31 // (32 * 128 * 128) + 3
    c = Case([1, 1, 1], 16, 32, 128, 128)
    S = torch.empty(rows, 32, 128, 128, device="cuda")
    ids = torch.tensor([rows - 1, 0, rows - 2], dtype=torch.int32, device="cuda")
    S[ids.long()] = c.state[c.ids.long()]
    o = sab.decay_decode(S, ids, c.q, c.k, c.v, c.g)
    small = c.state.clone()
    small[c.ids.long()] = S[ids.long()]
    c.check(o, small, decode=True)
    d = Case([150, 33], 16, 32, 128, 128)
    S[ids[:2].long()] = d.state[d.ids.long()]
    o = sab.decay_prefill(S, ids[:2], d.cu, d.q, d.k, d.v, d.g)
    small = d.state.clone()
    small[d.ids.long()] = S[ids[:2].long()]
    d.check(o, small)
    del S
    # rows of v and o far apart
    e = Case([130, 70], 1, 1, 64, 64)
    far = torch.empty(200 * (12 << 20), dtype=torch.bfloat16, device="cuda").view(200, 12 << 20)
    v, out = far[:, :64].unflatten(1, (1, 64)), far[:, 64:128].unflatten(1, (1, 64))
    v.copy_(e.v)
    S = e.state.clone()
    e.check(sab.decay_prefill(S, e.ids, e.cu, e.q, e.k, v, e.g, out=out), S)


def test_refusals_on_the_gpu(sab):
    c = Case([4, 4], 2, 4, 64, 64)
    a = (c.q, c.k, c.v, c.g)
    with pytest.raises(ValueError):
        sab.decay_prefill(c.state, c.ids, [0, 8], *a)
    with pytest.raises(TypeError):
        sab.decay_prefill(c.state.half(), c.ids, c.cu, *a)
    with pytest.raises(TypeError):
        sab.decay_prefill(c.state, c.ids, c.cu, c.q.float(), c.k, c.v, c.g)
    with pytest.raises(ValueError):
        sab.decay_prefill(c.state.transpose(2, 3), c.ids, c.cu, *a)
    with pytest.raises(ValueError):
        sab.decay_prefill(c.state, c.ids, c.cu, c.q, c.k, c.v[:, :3], c.g)
    with pytest.raises(ValueError):
        sab.decay_decode(c.state, c.ids, *a)  # eight rows for two sequences
    with pytest.raises(sab.ERError):
        sab.decay_decode(c.state, [0, 1, 0], *(x[:3] for x in a))
    with pytest.raises(sab.ERError):
        S = torch.zeros(2, 4, 32, 64, device="cuda")
        qk = c.q[:2, :, :32].contiguous()
        sab.decay_decode(S, [0, 1], qk, qk, c.v[:2], c.g[:2])
    with pytest.raises(ValueError):
        sab.decay_decode(c.state, torch.zeros(2, dtype=torch.int32), *(x[:2] for x in a),
                         dev_error=torch.zeros(1, dtype=torch.int32))
    n = sab.launch_count()
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    assert sab.decay_decode(c.state, empty, *(x[:0] for x in a)).shape == (0, 4, 64)
    assert sab.launch_count() == n
