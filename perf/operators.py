"""Measured cases of the fused linear product, the gated feed-forward product and the
decayed linear attention: their inputs, their plain forms and their exact values.

With `own` false, run() computes an operator from elementary torch operations in FP32
(FP64 for sums of log-decays); with `own` true it makes the library's calls.
"""
import math

import torch

own = False

#: Tokens per block of the plain form of the attention over prompts.
BLOCK = 64


def listed():
    """The listed cases: each operator from its smallest call to its largest."""
    return [
        # a single decoded token through the shared output projection (2560 x 4096), added
        # to the residual stream
        {"name": "linear one token", "op": "linear", "T": 1, "F": 2560, "K": 4096, "bias": False,
         "act": "none", "residual": True, "fp32": False},
        # a small ragged batch through an odd-sized head with bias, FP32 out
        {"name": "linear 37 odd", "op": "linear", "T": 37, "F": 4099, "K": 2568, "bias": True,
         "act": "silu", "residual": False, "fp32": True},
        # the 512-sequence decode batch through the output projection
        {"name": "linear batch 512", "op": "linear", "T": 512, "F": 2560, "K": 4096,
         "bias": False, "act": "none", "residual": True, "fp32": False},
        # a long prompt through a feed-forward projection with bias and activation
        {"name": "linear prompt 8192", "op": "linear", "T": 8192, "F": 10240, "K": 2560,
         "bias": True, "act": "gelu_tanh", "residual": False, "fp32": False},
        # the feed-forward block of a single decoded token
        {"name": "gated one token", "op": "gated", "T": 1, "F": 6912, "K": 2560, "act": "silu",
         "fp32": False},
        # a ragged decode batch, features that fill no tile
        {"name": "gated 300 ragged", "op": "gated", "T": 300, "F": 9000, "K": 2560,
         "act": "gelu", "fp32": False},
        # a long prompt through the feed-forward block
        {"name": "gated prompt 4096", "op": "gated", "T": 4096, "F": 10240, "K": 2560,
         "act": "silu", "fp32": False},
        # a single sequence's next token through one recurrent layer
        {"name": "decay decode 1", "op": "decode", "B": 1, "HK": 16, "HV": 32, "DK": 128,
         "DV": 128, "fixed": False},
        # the 512-sequence decode batch through one recurrent layer
        {"name": "decay decode 512", "op": "decode", "B": 512, "HK": 16, "HV": 32, "DK": 128,
         "DV": 128, "fixed": False},
        # one 256-token prefill chunk of one sequence that already has a state
        {"name": "decay chunk 256", "op": "prompt", "B": 1, "longest": 256, "ragged": False,
         "HK": 16, "HV": 32, "DK": 128, "DV": 128, "fixed": False},
        # nine prompts of odd lengths, narrow heads with a fixed decay for each head
        {"name": "decay 9 ragged prompts", "op": "prompt", "B": 9, "longest": 2043,
         "ragged": True, "HK": 8, "HV": 8, "DK": 64, "DV": 64, "fixed": True},
        # one long prompt
        {"name": "decay prompt 32768", "op": "prompt", "B": 1, "longest": 32768,
         "ragged": False, "HK": 16, "HV": 32, "DK": 128, "DV": 128, "fixed": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    op = rng.choice(["linear", "linear", "gated", "decode", "prompt", "prompt"])
    if op in ("linear", "gated"):
        most = 8192 * 10240 * 2560 if op == "linear" else 4096 * 10240 * 2560
        while True:
            T, F, K = _log(rng, 1, 8192), _log(rng, 40, 12288), 8 * _log(rng, 8, 1024)
            if rng.random() < 0.5:
                F = 64 * max(1, F // 64)
            if T * F * K <= most:
                break
        case = {"op": op, "T": T, "F": F, "K": K, "act": rng.choice(["silu", "gelu", "gelu_tanh"]),
                "fp32": rng.random() < 0.3}
        if op == "linear":
            if rng.random() < 0.4:
                case["act"] = "none"
            case["bias"], case["residual"] = rng.random() < 0.5, rng.random() < 0.5
        return case
    HK = rng.choice([1, 2, 4, 8, 16])
    HV = HK * rng.choice([r for r in (1, 2, 4) if HK * r <= 32])
    case = {"op": op, "HK": HK, "HV": HV, "DK": rng.choice([64, 128]), "DV": rng.choice([64, 128]),
            "fixed": rng.random() < 0.3}
    if op == "decode":
        case["B"] = _log(rng, 1, 512)
    else:
        case["B"] = _log(rng, 1, 16)
        case["longest"] = _log(rng, 1, 32768 // case["B"])
        case["ragged"] = case["B"] > 1 and rng.random() < 0.7
    return case


def _lengths(case):
    """The prompts' lengths, without randomness: the longest first, the others spread
    unevenly below it, one of them a single token."""
    B, n = case["B"], case["longest"]
    if not case["ragged"]:
        return [n] * B
    return [n] + [1 + (n - 1) * ((37 * b) % 101) // 101 for b in range(1, B - 1)] + [1]


def prepare(case, seed):
    """What the caller has before the call, on the GPU, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        x = torch.empty(*shape, dtype=dtype, device="cuda").normal_(generator=gen)
        return x.mul_(scale) if scale != 1.0 else x

    s = dict(case)
    if case["op"] in ("linear", "gated"):
        T, F, K = case["T"], case["F"], case["K"]
        y = torch.float32 if case["fp32"] else torch.bfloat16
        s["x"] = normal(T, K)
        s["out"] = torch.empty(T, F, dtype=y, device="cuda")
        if case["op"] == "gated":
            s["w_gate"], s["w_up"] = (normal(F, K, scale=K ** -0.5) for _ in range(2))
        else:
            s["w"] = normal(F, K, scale=K ** -0.5)
            s["b"] = normal(F, scale=0.1) if case["bias"] else None
            s["r"] = normal(T, F, dtype=y) if case["residual"] else None
        return s
    B, HK, HV, DK, DV = (case[n] for n in ("B", "HK", "HV", "DK", "DV"))
    if case["op"] == "prompt":
        lengths = _lengths(case)
        ends = torch.tensor([0] + lengths).cumsum(0)
        T, s["longest"] = int(ends[-1]), max(lengths)
        s["cu"] = ends.to(torch.int32).cuda()
    else:
        T = B
    # q, k and v are slices of one projection's rows; k has unit length about
    rows = normal(T, 2 * HK * DK + HV * DV)
    rows[:, HK * DK:2 * HK * DK].mul_(DK ** -0.5)
    s["q"] = rows[:, :HK * DK].unflatten(1, (HK, DK))
    s["k"] = rows[:, HK * DK:2 * HK * DK].unflatten(1, (HK, DK))
    s["v"] = rows[:, 2 * HK * DK:].unflatten(1, (HV, DV))
    # decays of e^-0.7 to e^-0.0002 a token, spread over the heads; the state that tokens
    # before these have left, in rows of its own order
    rate = torch.logspace(-3.5, -0.15, HV, device="cuda")
    if case["fixed"]:
        s["log_decay"] = -rate
    else:
        s["log_decay"] = -rate * torch.nn.functional.softplus(normal(T, HV, dtype=torch.float32))
    s["ids"] = torch.randperm(B, generator=gen, device="cuda").to(torch.int32)
    s["state"] = normal(B, HV, DK, DV, dtype=torch.float32)
    s["out"] = torch.empty(T, HV, DV, dtype=torch.bfloat16, device="cuda")
    return s


def _act(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _linear(s):
    v = s["x"].float() @ s["w"].float().T
    if s["b"] is not None:
        v = v + s["b"].float()
    v = _act(v, s["act"])
    if s["r"] is not None:
        v = v + s["r"].float()
    return v.to(s["out"].dtype)


def _gated(s):
    x = s["x"].float()
    v = _act(x @ s["w_gate"].float().T, s["act"]) * (x @ s["w_up"].float().T)
    return v.to(s["out"].dtype)


def _decode(s):
    HV, DK = s["HV"], s["DK"]
    rep, ids = HV // s["HK"], s["ids"].long()
    q, k = (s[n].float().repeat_interleave(rep, 1) for n in ("q", "k"))
    new = s["state"][ids] * torch.exp(s["log_decay"]).expand(s["B"], HV)[..., None, None]
    new = new + k[..., None] * s["v"].float()[..., None, :]
    s["state"][ids] = new
    o = (q[..., None, :] @ new)[..., 0, :] * DK ** -0.5
    return {"o": o.to(torch.bfloat16), "state": s["state"]}


def _prompt(s):
    """Blocks of BLOCK tokens: within a block the masked products of all its tokens, from
    block to block one product of the blocks' states with their decays."""
    B, HV, DK, DV = (s[n] for n in ("B", "HV", "DK", "DV"))
    rep, ids, cu = HV // s["HK"], s["ids"].long(), s["cu"].long()
    T, C = s["q"].shape[0], BLOCK
    N = -(-s["longest"] // C)
    # the packed rows on a padded grid of [B, N * C]; the rows behind a sequence are zero
    # with no decay
    at = cu[:-1, None] + torch.arange(N * C, device=cu.device)
    there = at < cu[1:, None]
    at = torch.where(there, at, 0)

    def grid(x):
        x = torch.where(there[..., None, None], x[at].float(), 0.0)
        return x.view(B, N, C, x.shape[2], x.shape[3]).permute(0, 3, 1, 2, 4)

    q, k = (grid(s[n]).repeat_interleave(rep, 1) for n in ("q", "k"))
    v = grid(s["v"])
    g = s["log_decay"].double().expand(T, HV)[at]
    g = torch.where(there[..., None], g, 0.0).permute(0, 2, 1)
    G = g.cumsum(2)
    end = G.view(B, HV, N, C)[..., -1]
    begin = torch.cat([torch.zeros_like(end[..., :1]), end[..., :-1]], 2)
    G = G.view(B, HV, N, C)
    lower = torch.ones(C, C, dtype=torch.bool, device=cu.device).tril()
    D = torch.where(lower, torch.exp(torch.where(lower, G[..., :, None] - G[..., None, :], 0.0)), 0.0)
    o = (q @ k.transpose(-1, -2) * D.float()) @ v
    # what each block leaves behind, and what each block finds
    left = (k * torch.exp(end[..., None] - G).float()[..., None]).transpose(-1, -2) @ v
    since = torch.cat([begin, end[..., -1:]], 2)
    before = torch.ones(N + 1, N, dtype=torch.bool, device=cu.device).tril(-1)
    W = torch.where(before, torch.exp(torch.where(before, since[..., :, None] - end[..., None, :], 0.0)), 0.0)
    found = (W.float() @ left.reshape(B, HV, N, DK * DV)).view(B, HV, N + 1, DK, DV)
    found = found + torch.exp(since).float()[..., None, None] * s["state"][ids][:, :, None]
    o = o + torch.exp(G - begin[..., None]).float()[..., None] * (q @ found[:, :, :N])
    s["state"][ids] = found[:, :, N]
    o = (o * DK ** -0.5).permute(0, 2, 3, 1, 4).reshape(B, N * C, HV, DV)
    return {"o": o[there].to(torch.bfloat16), "state": s["state"]}


def run(state):
    """One pass through a case's operator."""
    s = state
    if own:
        import sliding_window_anchor_b200 as sab
        if s["op"] == "linear":
            return sab.linear_fused(s["x"], s["w"], bias=s["b"], act=s["act"], residual=s["r"],
                                    fp32_out=s["fp32"], out=s["out"])
        if s["op"] == "gated":
            return sab.gated_linear(s["x"], s["w_gate"], s["w_up"], act=s["act"],
                                    fp32_out=s["fp32"], out=s["out"])
        if s["op"] == "decode":
            o = sab.decay_decode(s["state"], s["ids"], s["q"], s["k"], s["v"], s["log_decay"],
                                 out=s["out"])
        else:
            o = sab.decay_prefill(s["state"], s["ids"], s["cu"], s["q"], s["k"], s["v"],
                                  s["log_decay"], out=s["out"])
        return {"o": o, "state": s["state"]}
    return {"linear": _linear, "gated": _gated, "decode": _decode, "prompt": _prompt}[s["op"]](s)


def work(case):
    """Bytes and operations that one pass cannot do without."""
    if case["op"] in ("linear", "gated"):
        T, F, K = case["T"], case["F"], case["K"]
        y, n = (4 if case["fp32"] else 2), (2 if case["op"] == "gated" else 1)
        extra = (2 * F if case.get("bias") else 0) + (y * T * F if case.get("residual") else 0)
        return {"bytes": 2 * T * K + 2 * n * F * K + y * T * F + extra, "flops": 2 * n * T * F * K}
    B, HK, HV, DK, DV = (case[n] for n in ("B", "HK", "HV", "DK", "DV"))
    T = B if case["op"] == "decode" else sum(_lengths(case))
    rows = T * (2 * (2 * HK * DK + HV * DV) + 2 * HV * DV)
    decays = 4 * HV * (1 if case["fixed"] else T)
    # per token and head: the decayed state, the outer product, the read with q
    return {"bytes": rows + decays + 8 * B * HV * DK * DV, "flops": 5 * T * HV * DK * DV}


def exact(case, seed):
    """What run() returns, in FP64 from the definitions, token by token."""
    s = prepare(case, seed)
    if case["op"] in ("linear", "gated"):
        x = s["x"].to(torch.float64)
        phi = {"none": lambda a: a,
               "silu": lambda a: a * torch.sigmoid(a),
               "gelu": lambda a: a * 0.5 * torch.erfc(-a / 2 ** 0.5),
               "gelu_tanh": lambda a: a * torch.sigmoid(
                   (8 / math.pi) ** 0.5 * (a + 0.044715 * a ** 3))}[case["act"]]
        if case["op"] == "gated":
            gate = torch.einsum("tk,fk->tf", x, s["w_gate"].to(torch.float64))
            up = torch.einsum("tk,fk->tf", x, s["w_up"].to(torch.float64))
            return phi(gate) * up
        a = torch.einsum("tk,fk->tf", x, s["w"].to(torch.float64))
        if s["b"] is not None:
            a += s["b"].to(torch.float64)[None]
        a = phi(a)
        return a if s["r"] is None else a + s["r"].to(torch.float64)
    B, HK, HV, DK, DV = (case[n] for n in ("B", "HK", "HV", "DK", "DV"))
    cu = s["cu"].tolist() if case["op"] == "prompt" else list(range(B + 1))
    ids = s["ids"].tolist()
    head = torch.arange(HV, device="cuda") // (HV // HK)
    S = torch.stack([s["state"][i] for i in ids]).to(torch.float64)
    decay = torch.exp(s["log_decay"].to(torch.float64))
    if case["fixed"]:
        decay = decay[None].repeat(cu[-1], 1)
    o = torch.empty(cu[-1], HV, DV, dtype=torch.float64, device="cuda")
    lengths = [cu[b + 1] - cu[b] for b in range(B)]
    # the sequences by length, so that those still running are the first ones
    order = sorted(range(B), key=lambda b: -lengths[b])
    S = S[order]
    for t in range(max(lengths)):
        live = [b for b in order if lengths[b] > t]
        n, at = len(live), [cu[b] + t for b in live]
        at = slice(at[0], at[0] + 1) if n == 1 else torch.tensor(at, device="cuda")
        q, k = (s[m][at].to(torch.float64)[:, head] for m in ("q", "k"))
        S[:n] *= decay[at][..., None, None]
        S[:n] += torch.einsum("bhk,bhv->bhkv", k, s["v"][at].to(torch.float64))
        o[at] = torch.einsum("bhk,bhkv->bhv", q, S[:n]) / DK ** 0.5
    new = s["state"].to(torch.float64)
    for j, b in enumerate(order):
        new[ids[b]] = S[j]
    return {"o": o, "state": new}
