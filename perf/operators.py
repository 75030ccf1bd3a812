"""The layer operators for serving and training around the scan: cases, plain forms and the library's calls.

Four operators, each with its directions:

  conv      the short depthwise causal convolution over packed ragged sequences, with a carried
            state (``ssd_conv``), and its gradients (``ssd_conv_bwd``)
  scan      the selective scan over packed ragged prompts, float32 states in slots (``ssd_scan_ragged``)
  step      one token of a Mamba-2 layer per row: convolution, SiLU, softplus and recurrence, both
            states updated in place (``mamba2_step``)
  ffn       the gated feed-forward block (``ffn_block``), and its gradients (``ffn_block_bwd``)
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a serving engine's prompt batch through the 1.3B layer's convolution (conv_dim 64 x 64 + 2 x 128),
        # every sequence continued from its slot
        {"name": "conv prompts", "op": "conv", "io": "bf16", "nseq": 8, "tokens": 16384, "channels": 4352, "width": 4,
         "direction": 1, "carry": True, "silu": True},
        # short ragged right-to-left blocks in float32: the smallest calls, where latency counts
        {"name": "conv short blocks f32", "op": "conv", "io": "f32", "nseq": 5, "tokens": 143, "channels": 320, "width": 3,
         "direction": -1, "carry": False, "silu": True},
        # the training step's gradient of the same convolution
        {"name": "conv gradients", "op": "conv_bwd", "io": "bf16", "nseq": 3, "tokens": 16001, "channels": 4352, "width": 4,
         "direction": 1, "silu": True},
        # a prompt batch through the 1.3B layer's scan, raw dt, states carried in slots
        {"name": "scan prompts", "op": "scan", "io": "bf16", "nseq": 8, "tokens": 16384, "heads": 64, "headdim": 64,
         "dstate": 128, "groups": 1, "direction": 1, "carry": True, "raw_dt": True},
        # one long prompt: few sequences, so the work has to be split over its length
        {"name": "scan one long prompt", "op": "scan", "io": "bf16", "nseq": 1, "tokens": 32741, "heads": 64, "headdim": 64,
         "dstate": 128, "groups": 1, "direction": 1, "carry": False, "raw_dt": False},
        # a small float32 model's right-to-left blocks, grouped B and C
        {"name": "scan blocks f32", "op": "scan", "io": "f32", "nseq": 7, "tokens": 533, "heads": 8, "headdim": 32,
         "dstate": 64, "groups": 2, "direction": -1, "carry": True, "raw_dt": False},
        # decoding, one sequence: latency
        {"name": "step one row", "op": "step", "io": "bf16", "rows": 1, "slots": 4, "heads": 64, "headdim": 64, "dstate": 128,
         "groups": 1, "width": 4},
        # decoding, a full batch: the float32 states stream through
        {"name": "step 96 rows", "op": "step", "io": "bf16", "rows": 96, "slots": 112, "heads": 64, "headdim": 64,
         "dstate": 128, "groups": 1, "width": 4},
        # decoding through the feed-forward block: the weights stream through
        {"name": "ffn three tokens", "op": "ffn", "tokens": 3, "d_model": 2048, "d_ff": 8192, "act": "silu"},
        # a training batch's forward pass
        {"name": "ffn batch", "op": "ffn", "tokens": 8177, "d_model": 2048, "d_ff": 8192, "act": "silu"},
        # the same batch's gradients
        {"name": "ffn gradients", "op": "ffn_bwd", "tokens": 8177, "d_model": 2048, "d_ff": 8192, "act": "silu"},
        # odd sizes, the other activation
        {"name": "ffn gradients odd", "op": "ffn_bwd", "tokens": 333, "d_model": 488, "d_ff": 1160, "act": "gelu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "scan", "scan", "step", "ffn", "ffn_bwd"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv", "conv_bwd"):
        tokens, channels = _log(rng, 8, 16000), 8 * _log(rng, 5, 540)
        c = {"op": op, "io": io, "nseq": min(tokens, rng.randint(1, 24)), "tokens": tokens, "channels": channels,
             "width": rng.randint(2, 4), "direction": rng.choice([1, -1]), "silu": rng.random() < 0.8}
        return dict(c, carry=rng.random() < 0.5) if op == "conv" else c
    if op == "scan":
        big = rng.random() < 0.6            # the tensor-core head shape, or the small ones
        heads, groups = 8 * rng.randint(1, 8), rng.choice([1, 1, 2])
        tokens = _log(rng, 8, 16000 if big else 3000)
        return {"op": op, "io": "bf16" if big else io, "nseq": min(tokens, rng.randint(1, 12)), "tokens": tokens,
                "heads": heads if big else heads // 2, "headdim": 64 if big else rng.choice([16, 32, 64]),
                "dstate": 128 if big else rng.choice([16, 32, 64]), "groups": groups,
                "direction": rng.choice([1, 1, -1]), "carry": rng.random() < 0.6, "raw_dt": rng.random() < 0.5}
    if op == "step":
        rows = _log(rng, 1, 90)
        return {"op": op, "io": io, "rows": rows, "slots": rows + rng.randint(0, 9), "heads": 8 * rng.randint(1, 8),
                "headdim": rng.choice([32, 64]), "dstate": rng.choice([64, 128]), "groups": rng.choice([1, 1, 2]),
                "width": rng.randint(2, 4)}
    return {"op": op, "tokens": _log(rng, 1, 6000), "d_model": 8 * _log(rng, 16, 250), "d_ff": 8 * _log(rng, 30, 1000),
            "act": rng.choice(["silu", "silu", "gelu"])}


def _lengths(nseq, tokens):
    """Uneven lengths of `nseq` sequences that fill `tokens`: weights 1, 2, 3, ... with every third one short."""
    if nseq == 1:
        return [tokens]
    w = [(i + 1) if i % 3 else 0.02 for i in range(nseq)]
    left = tokens - nseq
    lens = [1 + int(left * x / sum(w)) for x in w]
    lens[-1] += tokens - sum(lens)
    return lens


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    op, s = case["op"], dict(case)
    if op.startswith("ffn"):
        T, D, F = case["tokens"], case["d_model"], case["d_ff"]
        bf = torch.bfloat16
        s["u"] = randn(T, D).to(bf)
        s["W_in"] = (randn(2 * F, D) / D ** 0.5).to(bf)     # gate rows, then up rows
        s["W_out"] = (randn(D, F) / F ** 0.5).to(bf)
        if op == "ffn_bwd":
            s["gu"] = s["u"] @ s["W_in"].t()                # the projections that the forward pass saved
            s["gy"] = randn(T, D).to(bf)
        return s
    io = _DT[case["io"]]
    if op == "step":
        R, H, P, N, G, K = (case[k] for k in ("rows", "heads", "headdim", "dstate", "groups", "width"))
        C = H * P + 2 * G * N
        s["xBC"], s["dt"] = randn(R, C).to(io), randn(R, H).to(io)
        s["conv_w"], s["conv_b"] = rand(C, K) - 0.5, 0.1 * randn(C)
        s["dt_bias"], s["A"], s["D"] = _dt_bias(rand(H)), -torch.exp(rand(H) * math.log(16.0)), rand(H)
        s["conv_state"] = randn(case["slots"], K - 1, C).to(io)
        s["ssm_state"] = 0.3 * randn(case["slots"], H, P, N)
        s["slot_idx"] = torch.randperm(case["slots"], generator=g, device=DEV)[:R].to(torch.int32)
        return s
    nseq, T = case["nseq"], case["tokens"]
    lens = _lengths(nseq, T)
    s["max_len"] = max(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if case.get("carry"):
        s["slot_idx"] = torch.randperm(nseq + 3, generator=g, device=DEV)[:nseq].to(torch.int32)
    if op in ("conv", "conv_bwd"):
        C, K = case["channels"], case["width"]
        s["x"] = randn(T, C).to(io)
        s["w"], s["bias"] = rand(C, K) - 0.5, 0.1 * randn(C)
        if op == "conv_bwd":
            s["gy"] = randn(T, C).to(io)
        elif case["carry"]:
            s["pool"] = randn(nseq + 3, K - 1, C).to(io)
        return s
    H, P, N, G = (case[k] for k in ("heads", "headdim", "dstate", "groups"))
    # x, B and C are the column blocks of one packed convolution output, as a layer has them
    packed = randn(T, H * P + 2 * G * N)
    packed[:, H * P:] /= N ** 0.5
    s["packed"] = packed.to(io)
    raw = randn(T, H)
    s["dt"] = (raw if case["raw_dt"] else torch.nn.functional.softplus(raw - 4)).to(io)
    s["dt_bias"] = _dt_bias(rand(H)) if case["raw_dt"] else None
    s["A"], s["D"] = -torch.exp(rand(H) * math.log(16.0)), rand(H)
    if case["carry"]:
        s["pool"] = 0.3 * randn(nseq + 3, H, P, N)
    return s


def _dt_bias(u):
    """The inverse softplus of a time step drawn log-uniformly from [1e-3, 1e-1]."""
    dt = torch.exp(u * math.log(100.0) + math.log(1e-3))
    return dt + torch.log(-torch.expm1(-dt))


def _views(s):
    """x, B, C of a scan case: views of the packed convolution output."""
    H, P, N, G = (s[k] for k in ("heads", "headdim", "dstate", "groups"))
    T, di = s["tokens"], H * P
    p = s["packed"]
    return (p[:, :di].unflatten(1, (H, P)), p[:, di:di + G * N].unflatten(1, (G, N)), p[:, di + G * N:].unflatten(1, (G, N)))


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    import bidirectional_mamba_ssd_bidir_b200 as ssd
    op = s["op"]
    if op == "ffn":
        return ssd.ffn_block(s["u"], s["W_in"], s["W_out"], activation=s["act"])
    if op == "ffn_bwd":
        return ssd.ffn_block_bwd(s["u"], s["W_in"], s["W_out"], s["gu"], s["gy"], activation=s["act"])
    if op == "step":
        y = ssd.mamba2_step(s["xBC"], s["dt"], s["conv_w"], s["conv_b"], s["dt_bias"], s["A"], s["D"], s["conv_state"],
                            s["ssm_state"], slots=s["slot_idx"], ngroups=s["groups"])
        return {"y": y, "conv_state": s["conv_state"], "ssm_state": s["ssm_state"]}
    if op == "conv_bwd":
        return ssd.ssd_conv_bwd(s["x"], s["w"], s["bias"], s["gy"], cu_seqlens=s["cu"], direction=s["direction"], silu=s["silu"])
    carry = dict(state_in=s["pool"], state_out=s["pool"], slots_in=s["slot_idx"], slots_out=s["slot_idx"]) if s["carry"] else {}
    if op == "conv":
        y = ssd.ssd_conv(s["x"], s["w"], s["bias"], cu_seqlens=s["cu"], direction=s["direction"], silu=s["silu"], **carry)
        return {"y": y, "state": s["pool"]} if s["carry"] else {"y": y}
    x, B, C = _views(s)
    if not s["carry"]:
        H, P, N = (s[k] for k in ("heads", "headdim", "dstate"))
        carry = dict(state_out=torch.empty(s["nseq"], H, P, N, device=DEV))
    y = ssd.ssd_scan_ragged(x, s["dt"], s["A"], B, C, s["D"], cu_seqlens=s["cu"], dt_bias=s["dt_bias"],
                            direction=s["direction"], **carry)
    return {"y": y, "state": carry["state_out"]}


# ---------------------------------------------------------------- the plain forms

def run(state):
    if own:
        return _run_own(state)
    return {"conv": _conv, "conv_bwd": _conv_bwd, "scan": _scan, "step": _step, "ffn": _ffn, "ffn_bwd": _ffn_bwd}[state["op"]](state)


def _silu(v):
    return v * torch.sigmoid(v)


def _d_silu(v):
    p = torch.sigmoid(v)
    return p * (1 + v * (1 - p))


def _gelu(v):
    return 0.5 * v * (1 + torch.erf(v * 0.7071067811865476))


def _d_gelu(v):
    return 0.5 * (1 + torch.erf(v * 0.7071067811865476)) + v * torch.exp(-0.5 * v * v) * 0.3989422804014327


_ACT = {"silu": (_silu, _d_silu), "gelu": (_gelu, _d_gelu)}


def _place(s):
    """Of each packed token: its sequence, and its place in scan order (0 first)."""
    cu = s["cu"].long()
    t = torch.arange(s["tokens"], device=DEV)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return cu, t, seq, (t - cu[seq] if s["direction"] > 0 else cu[seq + 1] - 1 - t)


def _back(s, x, steps, place):
    """The rows of x `steps` tokens back in scan order; zero, or the carried state's row, before the first."""
    cu, t, seq, k = place
    src = t - s["direction"] * steps
    inside = k >= steps
    v = x[torch.where(inside, src, t)]
    if s.get("carry"):
        # the state's rows, oldest first: row (width - 1) + (k - steps) for a negative k - steps
        row = (s["width"] - 1 + k - steps).clamp(0, s["width"] - 2)
        return torch.where(inside[:, None], v, s["pool"][s["slot_idx"].long()[seq], row].float())
    return torch.where(inside[:, None], v, 0.0)


def _conv_sum(s, x, place):
    K = s["width"]
    return s["bias"] + sum(s["w"][:, K - 1 - j] * _back(s, x, j, place) for j in range(K))


def _conv(s):
    x, place = s["x"].float(), _place(s)
    acc = _conv_sum(s, x, place)
    y = (_silu(acc) if s["silu"] else acc).to(s["x"].dtype)
    if not s["carry"]:
        return {"y": y}
    # the new state: the last width - 1 tokens of the old state followed by the sequence
    cu, K, slots = place[0], s["width"], s["slot_idx"].long()
    n = cu[1:] - cu[:-1]
    at = n[:, None] - (K - 1) + torch.arange(K - 1, device=DEV)            # place in scan order, oldest first
    tok = (cu[:-1, None] + at if s["direction"] > 0 else cu[1:, None] - 1 - at).clamp(0, s["tokens"] - 1)
    old = s["pool"][slots].gather(1, (at + K - 1).clamp(0, K - 2)[:, :, None].expand(-1, -1, s["channels"]))
    s["pool"][slots] = torch.where((at >= 0)[:, :, None], s["x"][tok], old)
    return {"y": y, "state": s["pool"]}


def _conv_bwd(s):
    x, place, K = s["x"].float(), _place(s), s["width"]
    gs = s["gy"].float()
    if s["silu"]:
        gs = gs * _d_silu(_conv_sum(s, x, place))
    cu, t, seq, k = place
    n = (cu[1:] - cu[:-1])[seq]
    fwd = lambda j: torch.where((k + j < n)[:, None], gs[(t + s["direction"] * j).clamp(0, s["tokens"] - 1)], 0.0)  # noqa: E731
    gx = sum(s["w"][:, K - 1 - j] * fwd(j) for j in range(K))
    gw = torch.stack([(gs * _back(s, x, K - 1 - j, place)).sum(0, dtype=torch.float64) for j in range(K)], 1)
    return {"x": gx.to(s["x"].dtype), "w": gw.float(), "bias": gs.sum(0, dtype=torch.float64).float()}


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _scan(s):
    H, P, N, G, Q = s["heads"], s["headdim"], s["dstate"], s["groups"], 64
    x, B, C = (v.float() for v in _views(s))
    cu, t, seq, k = _place(s)
    nc = -(-s["max_len"] // Q)
    S = s["nseq"]
    at = seq * (nc * Q) + k                                 # each token's place in a padded batch
    pad = lambda v: torch.zeros(S * nc * Q, *v.shape[1:], device=DEV).index_copy(0, at, v).unflatten(0, (S, nc, Q))  # noqa: E731
    dt = s["dt"].float()
    if s["dt_bias"] is not None:
        dt = _softplus(dt + s["dt_bias"])
    xp, dtp, Bp, Cp = pad(x), pad(dt), pad(B), pad(C)
    a = (dtp * s["A"]).double().permute(0, 3, 1, 2)         # [S, H, nc, Q]
    cs = a.cumsum(-1)
    mask = torch.ones(Q, Q, dtype=torch.bool, device=DEV).tril()
    L = torch.exp((cs[..., :, None] - cs[..., None, :]).float().masked_fill(~mask, -math.inf))
    scores = torch.einsum("scign,scjgn->sgcij", Cp, Bp).repeat_interleave(H // G, 1)
    xd = xp * dtp[..., None]
    y = torch.einsum("shcij,scjhp->scihp", scores * L, xd)
    # the state that each chunk adds, and those that enter it from the chunks before and the carried one
    tail = torch.exp((cs[..., -1:] - cs).float()).permute(0, 2, 3, 1)
    Bh = Bp.repeat_interleave(H // G, 3)
    local = torch.einsum("scjhn,scjhp->shcpn", Bh, xd * tail[..., None])
    first = s["pool"][s["slot_idx"].long()] if s["carry"] else torch.zeros(S, H, P, N, device=DEV)
    every = torch.cat([first[:, :, None], local], 2)        # [S, H, nc + 1, P, N]
    total = torch.cat([torch.zeros(S, H, 1, dtype=torch.float64, device=DEV), cs[..., -1]], 2).cumsum(-1)
    low = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=DEV).tril()
    between = torch.exp((total[..., :, None] - total[..., None, :]).float().masked_fill(~low, -math.inf))
    enter = torch.matmul(between, every.flatten(3)).unflatten(3, (P, N))
    decay = torch.exp(cs.float()).permute(0, 2, 3, 1)
    Ch = Cp.repeat_interleave(H // G, 3)
    y = y + torch.einsum("scihn,shcpn->scihp", Ch, enter[:, :, :-1]) * decay[..., None]
    y = y.flatten(0, 2)[at] + s["D"][:, None] * x
    last = enter[:, :, -1]
    if s["carry"]:
        s["pool"][s["slot_idx"].long()] = last
        last = s["pool"]
    return {"y": y.to(s["packed"].dtype), "state": last}


def _step(s):
    H, P, N, G, K = (s[k] for k in ("heads", "headdim", "dstate", "groups", "width"))
    slots, di = s["slot_idx"].long(), H * P
    win = torch.cat([s["conv_state"][slots], s["xBC"][:, None]], 1)         # [rows, K, C], oldest first
    s["conv_state"][slots] = win[:, 1:]
    v = _silu((win.float() * s["conv_w"].t()).sum(1) + s["conv_b"])
    x = v[:, :di].unflatten(1, (H, P))
    B = v[:, di:di + G * N].unflatten(1, (G, N)).repeat_interleave(H // G, 1)
    C = v[:, di + G * N:].unflatten(1, (G, N)).repeat_interleave(H // G, 1)
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    S = s["ssm_state"][slots] * torch.exp(dt * s["A"])[:, :, None, None] + (x * dt[..., None])[..., None] * B[:, :, None]
    s["ssm_state"][slots] = S
    y = (S * C[:, :, None]).sum(-1) + s["D"][:, None] * x
    return {"y": y.to(s["xBC"].dtype), "conv_state": s["conv_state"], "ssm_state": s["ssm_state"]}


def _ffn(s):
    gu = s["u"].float() @ s["W_in"].float().t()
    g, up = gu.chunk(2, 1)
    return ((_ACT[s["act"]][0](g) * up) @ s["W_out"].float().t()).to(torch.bfloat16)


def _ffn_bwd(s):
    act, d_act = _ACT[s["act"]]
    g, up = s["gu"].float().chunk(2, 1)
    gy, u = s["gy"].float(), s["u"].float()
    gh = gy @ s["W_out"].float()
    ggu = torch.cat([gh * up * d_act(g), gh * act(g)], 1)
    out = {"u": ggu @ s["W_in"].float(), "W_in": ggu.t() @ u, "W_out": gy.t() @ (act(g) * up)}
    return {k: v.to(torch.bfloat16) for k, v in out.items()}


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op.startswith("ffn"):
        T, D, F = case["tokens"], case["d_model"], case["d_ff"]
        if op == "ffn":
            return {"bytes": 2 * (2 * T * D + 3 * D * F), "flops": 6 * T * D * F}
        return {"bytes": 2 * (3 * T * D + 2 * T * F + 6 * D * F), "flops": 12 * T * D * F}
    es = 2 if case["io"] == "bf16" else 4
    if op in ("conv", "conv_bwd"):
        T, C, K, S = case["tokens"], case["channels"], case["width"], case["nseq"]
        state = 2 * S * (K - 1) * C * es if case.get("carry") else 0
        if op == "conv":
            return {"bytes": 2 * T * C * es + state + 4 * C * (K + 1) + 4 * S, "flops": 2 * T * C * (K + 2)}
        return {"bytes": 3 * T * C * es + 8 * C * (K + 1) + 4 * S, "flops": 2 * T * C * (3 * K + 4)}
    H, P, N, G = (case[k] for k in ("heads", "headdim", "dstate", "groups"))
    if op == "step":
        R, K, C = case["rows"], case["width"], H * P + 2 * G * N
        return {"bytes": R * (8 * H * P * N + es * (C + H + H * P + 2 * (K - 1) * C)) + 4 * C * (K + 1),
                "flops": R * (5 * H * P * N + 2 * K * C)}
    T, S = case["tokens"], case["nseq"]
    return {"bytes": es * T * (2 * H * P + 2 * G * N + H) + 4 * S * H * P * N * (2 if case["carry"] else 1),
            "flops": 5 * T * H * P * N}


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "conv_bwd": _exact_conv_bwd, "scan": _exact_scan, "step": _exact_step,
            "ffn": _exact_ffn, "ffn_bwd": _exact_ffn_bwd}[case["op"]](s)


def _pieces(s):
    cu = s["cu"].tolist()
    return list(zip(cu[:-1], cu[1:]))


def _exact_conv_one(s, x, w, b, history):
    """One sequence's convolution, x [n, C] in scan order after `history` [K - 1, C]."""
    ext = torch.cat([history, x], 0)
    acc = torch.nn.functional.conv1d(ext.t()[None], w[:, None], b, groups=w.shape[0])[0].t()
    return (torch.nn.functional.silu(acc) if s["silu"] else acc), ext[-(s["width"] - 1):]


def _exact_conv(s):
    w, b, K = s["w"].double(), s["bias"].double(), s["width"]
    pool = s["pool"].double() if s["carry"] else None
    ys = []
    for i, (lo, hi) in enumerate(_pieces(s)):
        x = s["x"][lo:hi].double()
        x = x if s["direction"] > 0 else x.flip(0)
        slot = int(s["slot_idx"][i]) if s["carry"] else 0
        hist = pool[slot] if s["carry"] else torch.zeros(K - 1, s["channels"], dtype=torch.float64, device=DEV)
        y, last = _exact_conv_one(s, x, w, b, hist)
        if s["carry"]:
            pool[slot] = last
        ys.append(y if s["direction"] > 0 else y.flip(0))
    y = torch.cat(ys, 0)
    return {"y": y, "state": pool} if s["carry"] else {"y": y}


def _exact_conv_bwd(s):
    w, b = s["w"].double().requires_grad_(True), s["bias"].double().requires_grad_(True)
    zero = torch.zeros(s["width"] - 1, s["channels"], dtype=torch.float64, device=DEV)
    gx = []
    for lo, hi in _pieces(s):
        x = s["x"][lo:hi].double().requires_grad_(True)
        y, _ = _exact_conv_one(s, x if s["direction"] > 0 else x.flip(0), w, b, zero)
        gy = s["gy"][lo:hi].double()
        y.backward(gy if s["direction"] > 0 else gy.flip(0))
        gx.append(x.grad)
    return {"x": torch.cat(gx, 0), "w": w.grad, "bias": b.grad}


def _exact_scan(s):
    H, P, N, G = (s[k] for k in ("heads", "headdim", "dstate", "groups"))
    x, B, C = (v.double() for v in _views(s))
    dt = s["dt"].double()
    if s["dt_bias"] is not None:
        dt = torch.nn.functional.softplus(dt + s["dt_bias"].double(), threshold=1e9)
    A, D = s["A"].double(), s["D"].double()
    if s["carry"]:
        pool = s["pool"].double()
        S = pool[s["slot_idx"].long()]
    else:
        S = torch.zeros(s["nseq"], H, P, N, dtype=torch.float64, device=DEV)
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    y = torch.zeros(s["tokens"], H, P, dtype=torch.float64, device=DEV)
    order = torch.argsort(n, descending=True)               # the sequences still running come first
    lens = n[order].tolist()
    S = S[order].unflatten(1, (G, H // G))
    start = cu[:-1][order] if s["direction"] > 0 else cu[1:][order] - 1
    live = len(lens)
    for i in range(s["max_len"]):
        while lens[live - 1] <= i:
            live -= 1
        tok = start[:live] + s["direction"] * i
        d = dt[tok].unflatten(1, (G, H // G))
        S[:live] = S[:live] * torch.exp(d * A.unflatten(0, (G, H // G)))[..., None, None] + \
            (x[tok].unflatten(1, (G, H // G)) * d[..., None])[..., None] * B[tok][:, :, None, None]
        y[tok] = torch.matmul(S[:live], C[tok][:, :, None, :, None]).squeeze(-1).flatten(1, 2)
    y += D[:, None] * x
    S = torch.empty_like(S).index_copy_(0, order, S).flatten(1, 2)
    if s["carry"]:
        pool[s["slot_idx"].long()] = S
        S = pool
    return {"y": y, "state": S}


def _exact_step(s):
    H, P, N, G, K = (s[k] for k in ("heads", "headdim", "dstate", "groups", "width"))
    conv, ssm = s["conv_state"].double(), s["ssm_state"].double()
    slots = s["slot_idx"].long()
    ext = torch.cat([conv[slots], s["xBC"].double()[:, None]], 1).transpose(1, 2)       # [rows, C, K]
    v = torch.nn.functional.silu(torch.einsum("rck,ck->rc", ext, s["conv_w"].double()) + s["conv_b"].double())
    conv[slots] = ext[:, :, 1:].transpose(1, 2)
    x, B, C = v.split([H * P, G * N, G * N], 1)
    x, B, C = x.reshape(-1, G, H // G, P), B.reshape(-1, G, N), C.reshape(-1, G, N)
    dt = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=1e9).unflatten(1, (G, H // G))
    S = ssm[slots].unflatten(1, (G, H // G))
    S = torch.exp(dt * s["A"].double().unflatten(0, (G, H // G)))[..., None, None] * S + \
        torch.einsum("rgh,rghp,rgn->rghpn", dt, x, B)
    ssm[slots] = S.flatten(1, 2)
    y = torch.einsum("rghpn,rgn->rghp", S, C) + s["D"].double().unflatten(0, (G, H // G))[..., None] * x
    return {"y": y.flatten(1, 2), "conv_state": conv, "ssm_state": ssm}


def _exact_ffn_h(act, gu):
    F = gu.shape[1] // 2
    return getattr(torch.nn.functional, act)(gu[:, :F]) * gu[:, F:]


def _exact_ffn(s):
    return torch.mm(_exact_ffn_h(s["act"], torch.mm(s["u"].double(), s["W_in"].double().t())), s["W_out"].double().t())


def _exact_ffn_bwd(s):
    # the saved projections are an input: gradients of gu by differentiation, the rest by the chain rule
    gu = s["gu"].double().requires_grad_(True)
    h = _exact_ffn_h(s["act"], gu)
    gy = s["gy"].double()
    ggu, = torch.autograd.grad(h, gu, torch.mm(gy, s["W_out"].double()))
    return {"u": torch.mm(ggu, s["W_in"].double()), "W_in": torch.mm(ggu.t(), s["u"].double()),
            "W_out": torch.mm(gy.t(), h.detach())}
