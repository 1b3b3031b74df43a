"""Workloads of the operators that stand between a hybrid model's matrix products and its recurrent and
attention layers: the short causal convolution (short_conv) and the selective state space scan behind it, for
prompts (ssm_prefill_chunked) and for single tokens (ssm_decode_step); the rotation of queries and keys by
their positions with the append to the paged cache (attn_cache_append); and the root-mean-square norm with the
residual's addition (add_rms_norm), in 16 bits or in 8 with scales.

Each operator has a plain form in elementary torch operations (32-bit arithmetic, one rounding at the end) and
the library's own call; `own` picks which of the two run() makes.  Both take what prepare() gives.  listed()
names fixed workloads, draw() makes others of the same ranges, work() counts the bytes and operations a pass
cannot do without, and exact() evaluates the definition in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}
_F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _conv(name, seqs, longest, splits, taps, dtype):
    """seqs sequences, the longest of `longest` tokens (0: a step of one token each); the channels go to outputs of
    the widths `splits` ("2048+2048+4096")."""
    return {"name": name, "op": "conv", "seqs": seqs, "longest": longest, "splits": splits, "taps": taps, "dtype": dtype}


def _ssm(name, op, seqs, longest, heads, dim, groups, state, gated):
    return {"name": name, "op": op, "seqs": seqs, "longest": longest, "heads": heads, "dim": dim, "groups": groups,
            "state": state, "dtype": "bf16", "gated": gated}


def _append(name, seqs, longest, hq, hkv, dim, turned, pairs, page, dtype, cache):
    """`turned` of the `dim` features are rotated; pairs: "halves" (i, i + turned / 2) or "neighbours" (2 i, 2 i + 1)."""
    return {"name": name, "op": "append", "seqs": seqs, "longest": longest, "hq": hq, "hkv": hkv, "dim": dim, "turned": turned,
            "pairs": pairs, "page": page, "dtype": dtype, "cache": cache}


def _norm(name, tokens, width, dtype, held, group, added):
    """held: "same" (16 bits) or "e4m3" with a scale per `group` features (0: per token)."""
    return {"name": name, "op": "norm", "tokens": tokens, "width": width, "dtype": dtype, "held": held, "group": group, "added": added}


def listed():
    return [
        # one token of each of a batch of users, the state space layer's x, B and C
        _conv("conv step 64 seqs", 64, 0, "4096+128+128", 4, "bf16"),
        # packed prompts on their way into a delta-rule layer: q, k and v of 16 key and 32 value heads
        _conv("conv prompts 4 seqs", 4, 8192, "2048+2048+4096", 4, "bf16"),
        # one user generating: latency only
        _ssm("scan step 1 seq", "step", 1, 1, 64, 64, 1, 128, True),
        # a batch of users generating one token each
        _ssm("scan step 64 seqs", "step", 64, 1, 64, 64, 1, 128, True),
        # a window of a few tokens of each of a batch, on top of what their states hold
        _ssm("scan windows 32 seqs", "scan", 32, 8, 64, 64, 1, 128, False),
        # one long prompt alone, wide heads
        _ssm("scan prompt 1 seq", "scan", 1, 16384, 32, 128, 2, 64, False),
        # packed prompts of different lengths, gated
        _ssm("scan prompts 4 seqs", "scan", 4, 8192, 64, 64, 8, 128, True),
        # one token of each of a batch of sequences, 8-bit cache
        _append("append 64 tokens e4m3", 64, 1, 32, 8, 128, 128, "halves", 64, "bf16", "e4m3"),
        # packed prompts, 8-bit cache
        _append("append prompts 4 seqs e4m3", 4, 8192, 32, 8, 128, 128, "halves", 64, "bf16", "e4m3"),
        # packed prompts with heads of which a quarter is rotated, 16-bit cache
        _append("append prompts 9 seqs f16", 9, 4095, 16, 4, 256, 64, "neighbours", 16, "f16", "same"),
        # between two layers of a decode step
        _norm("norm 64 tokens", 64, 4096, "bf16", "same", 0, True),
        # between two layers of a prompt, ahead of a matrix product in 8 bits
        _norm("norm 16k tokens e4m3", 16383, 5120, "bf16", "e4m3", 128, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("conv", "step", "scan", "scan", "append", "norm"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if kind == "norm":
        width = 8 * _log_int(rng, 8, 2048)
        held = rng.choice(("same", "e4m3"))
        group = rng.choice((0, 64, 128)) if held == "e4m3" and width % 128 == 0 else 0
        return {"op": "norm", "tokens": _log_int(rng, 1, max(1, min(65536, 16383 * 5120 // width))), "width": width, "dtype": dtype,
                "held": held, "group": group, "added": rng.random() < 0.8}
    if kind == "append":
        seqs, dim = _log_int(rng, 1, 128), rng.choice((64, 128, 128, 256))
        hkv = rng.choice((1, 2, 4, 8, 16))
        hq = hkv * rng.choice((1, 2, 3, 4, 6, 8))
        turned = rng.choice((dim, dim, dim // 2, dim // 4))
        longest = 1 if rng.random() < 0.3 else _log_int(rng, 1, max(1, min(8192, 20000 * 48 * 128 // (seqs * (hq + 2 * hkv) * dim))))
        return {"op": "append", "seqs": seqs, "longest": longest, "hq": hq, "hkv": hkv, "dim": dim, "turned": turned,
                "pairs": rng.choice(("halves", "neighbours")), "page": rng.choice((16, 32, 48, 64, 128)), "dtype": dtype,
                "cache": rng.choice(("same", "e4m3"))}
    seqs = _log_int(rng, 1, 64)
    if kind == "conv":
        splits = [8 * _log_int(rng, 4, 512) for _ in range(rng.randint(1, 3))]
        longest = 0 if rng.random() < 0.3 else _log_int(rng, 1, max(1, min(8192, 20000 * 8192 // (seqs * sum(splits)))))
        return {"op": "conv", "seqs": seqs, "longest": longest, "splits": "+".join(map(str, splits)), "taps": rng.choice((2, 3, 4, 4)),
                "dtype": dtype}
    dim, state, groups = rng.choice((64, 64, 128)), rng.choice((64, 128, 128)), rng.choice((1, 1, 2, 4, 8))
    heads = groups * rng.randint(1, max(1, 80 // groups * 64 // dim))
    longest = 1
    if kind == "scan":
        longest = _log_int(rng, 1, max(1, min(16384, 23000 * 64 * 64 // (seqs * heads * dim))))
    elif seqs * heads * dim * state > 64 * 64 * 64 * 128:
        seqs = max(1, 64 * 64 * 64 * 128 // (heads * dim * state))
    return {"op": kind, "seqs": seqs, "longest": longest, "heads": heads, "dim": dim, "groups": groups, "state": state,
            "dtype": "bf16", "gated": rng.random() < 0.5}


def _lens(seqs, longest):
    """Ragged lengths: the first sequence has the longest, the others spread over 1/8 .. 1 of it."""
    return [max(1, int(longest * (1.0 if n == 0 else 0.125 + 0.875 * ((n * 0.6180339887498949) % 1.0)))) for n in range(seqs)]


def _widths(case):
    return [int(w) for w in case["splits"].split("+")]


def work(case):
    """Bytes: every input read once, every output written once.  Operations: two per product and sum."""
    two = 2
    if case["op"] == "norm":
        n = case["tokens"] * case["width"]
        held = two if case["held"] == "same" else 1 + 4 / (case["group"] or case["width"])
        return {"bytes": n * (two * (3 if case["added"] else 1) + held) + 4 * case["width"], "flops": 5 * n}
    tokens = sum(_lens(case["seqs"], case["longest"]))
    if case["op"] == "conv":
        width, taps = sum(_widths(case)), case["taps"]
        return {"bytes": 2 * two * tokens * width + 8 * case["seqs"] * width * (taps - 1) + 4 * width * (taps + 1),
                "flops": tokens * width * (2 * taps + 4)}
    if case["op"] == "append":
        held = two if case["cache"] == "same" else 1 + 4 / case["dim"]
        rows = case["hq"] * two * 2 + 2 * case["hkv"] * (two + held)
        return {"bytes": tokens * (rows * case["dim"] + 4 * case["turned"] + 16), "flops": 3 * tokens * (case["hq"] + case["hkv"]) * case["turned"]}
    inner = case["heads"] * case["dim"]
    bytes_ = tokens * two * (inner * (3 if case["gated"] else 2) + 2 * case["groups"] * case["state"] + case["heads"])
    return {"bytes": bytes_ + 8 * case["seqs"] * inner * case["state"], "flops": 4 * tokens * inner * case["state"]}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).cuda()


def _pool_slots(g, seqs):
    """A slot of its own for each sequence, in a pool with three to spare."""
    return torch.randperm(seqs + 3, generator=g, device="cuda")[:seqs]


def _rotation(turned, positions):
    """cos and sin of position * 10000^(-2 i / turned), side by side: what a program lays out once."""
    i = torch.arange(turned // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2.0 * i / turned)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    g = _gen(seed)
    s = {"op": case["op"], "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    dt = _DT[case["dtype"]]
    if case["op"] == "norm":
        tokens, width = case["tokens"], case["width"]
        # a few channels of the residual stream are larger than the others, as in trained models
        s["x"] = _randn(g, tokens, width).to(dt)
        s["residual"] = (2.0 * _randn(g, tokens, width) * torch.exp(0.5 * _randn(g, width))).to(dt) if case["added"] else None
        s["weight"] = 1.0 + 0.2 * _randn(g, width)
        s["eps"], s["f8"], s["group"] = 1e-6, case["held"] == "e4m3", case["group"]
        return s
    seqs = case["seqs"]
    lens = _lens(seqs, case["longest"])
    tokens = sum(lens)
    s["lens"], s["cu"] = lens, _cu(lens)
    if case["op"] == "append":
        hq, hkv, dim, page = case["hq"], case["hkv"], case["dim"], case["page"]
        # the fused projection's rows: queries, keys and values side by side; keys with a few larger channels
        size = torch.cat([torch.ones(hq, dim, device="cuda"), torch.exp(0.7 * _randn(g, hkv, dim)), torch.ones(hkv, dim, device="cuda")])
        rows = (_randn(g, tokens, hq + 2 * hkv, dim) * size).to(dt)
        s["q"], s["k"], s["v"] = rows.split([hq, hkv, hkv], 1)
        before = torch.randint(0, 4096, (seqs,), generator=g, device="cuda")  # tokens that the sequences already have
        n = torch.repeat_interleave(torch.arange(seqs, device="cuda"), torch.tensor(lens, device="cuda"))
        s["positions"] = before[n] + torch.arange(tokens, device="cuda") - s["cu"][n]
        s["rotation"], s["neighbours"] = _rotation(case["turned"], 4096 + case["longest"]), case["pairs"] == "neighbours"
        pages_of = [-(-k // page) + 1 for k in lens]  # the page that is already begun, and the new ones
        first = torch.tensor([0] + pages_of[:-1]).cumsum(0).cuda()
        perm = torch.randperm(sum(pages_of) + 3, generator=g, device="cuda")
        at = before[n] % page + torch.arange(tokens, device="cuda") - s["cu"][n]
        s["slots"] = perm[first[n] + at // page] * page + at % page
        f8 = case["cache"] == "e4m3"
        for name in ("k", "v"):
            c = torch.zeros((perm.numel(), hkv, page, dim), dtype=torch.uint8 if f8 else dt, device="cuda")
            s[name + "_cache"] = c.view(_F8) if f8 else c
            s[name + "_scale"] = torch.ones((perm.numel(), hkv, page), device="cuda") if f8 else None
        return s
    s["slots"], s["longest"] = _pool_slots(g, seqs), max(lens)
    if case["op"] == "conv":
        widths, taps = _widths(case), case["taps"]
        width = sum(widths)
        # the projection's rows: the convolution's channels, with a gate of the first part's width behind them
        s["x"] = _randn(g, tokens, width + widths[0]).to(dt)[:, :width]
        s["weight"], s["bias"] = _randn(g, width, taps) * taps ** -0.5, 0.1 * _randn(g, width)
        # what earlier tokens left: values of the rows' type
        s["hist"] = _randn(g, seqs + 3, width, taps - 1).to(dt).float()
        s["splits"], s["step"] = widths, case["longest"] == 0
        return s
    heads, dim, groups, state = case["heads"], case["dim"], case["groups"], case["state"]
    # what the convolution's activation leaves, and the projection's row that holds the gate and dt
    act = torch.nn.functional.silu
    s["x"], s["B"], s["C"] = (act(1.5 * _randn(g, tokens, *d)).to(dt) for d in ((heads, dim), (groups, state), (groups, state)))
    inner = heads * dim
    rows = _randn(g, tokens, inner + -(-heads // 8) * 8).to(dt)
    s["z"] = rows[:, :inner].unflatten(1, (heads, dim)) if case["gated"] else None
    s["dt"] = rows[:, inner:inner + heads]
    # steps of 0.001 .. 0.1 for a projection of zero, decays of 1 .. 16, as such layers start
    base = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(heads, generator=g, device="cuda"))
    s["dt_bias"] = base + torch.log(-torch.expm1(-base))
    s["A_log"] = torch.log(1.0 + 15.0 * torch.rand(heads, generator=g, device="cuda"))
    s["D"] = 1.0 + 0.1 * _randn(g, heads)
    s["state"] = 0.2 * _randn(g, seqs + 3, heads, dim, state)
    s["workspace"] = None
    if own and case["op"] == "scan":
        import gated_deltanet_delta_gb300 as gdn
        s["workspace"] = torch.empty(gdn.ssm_prefill_workspace_size(seqs, tokens, heads, dim, state), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def _norm_plain(s):
    r = s["x"].float()
    if s["residual"] is not None:
        s["residual"].copy_((r + s["residual"].float()).to(s["x"].dtype))
        r = s["residual"].float()
    y = r * (r.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * s["weight"]
    out = {} if s["residual"] is None else {"residual": s["residual"]}
    if not s["f8"]:
        return dict(out, y=y.to(s["x"].dtype))
    tokens, width = y.shape
    y = y.reshape(tokens, -1, s["group"] or width)
    amax = y.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, 1.0)
    return dict(out, y=(y / scale[..., None]).reshape(tokens, width).to(_F8), scale=scale)


def _conv_plain(s):
    x, taps = s["x"], s["weight"].shape[1]
    total = x.shape[0]
    cu = s["cu"]
    t = torch.arange(total, device="cuda")
    n = torch.bucketize(t, cu[1:], right=True)
    hist = s["hist"][s["slots"]]  # [N, C, taps - 1], oldest first
    back = torch.arange(taps - 1, -1, -1, device="cuda")  # tap j sees the token `back` before
    at = (t - cu[n])[:, None] - back  # position in the sequence; before its first token the history
    old = hist.transpose(1, 2)[n[:, None], (at + taps - 1).clamp(max=taps - 2)]
    seen = torch.where((at >= 0)[..., None], x[(t[:, None] - back).clamp(min=0)].float(), old)  # [T, taps, C]
    y = (seen * s["weight"].T).sum(1) + s["bias"]
    y = y * torch.sigmoid(y)
    # the last taps - 1 tokens of each sequence
    last = (cu[1:] - cu[:-1])[:, None] - back[:-1]
    new = torch.where((last >= 0)[:, :, None], x[(cu[:-1, None] + last).clamp(min=0)].float(),
                      hist.transpose(1, 2).gather(1, (last + taps - 1).clamp(max=taps - 2)[:, :, None].expand(-1, -1, x.shape[1])))
    s["hist"][s["slots"]] = new.transpose(1, 2)
    return {"y": [p.contiguous() for p in y.to(x.dtype).split(s["splits"], 1)], "hist": s["hist"]}


def _gates(s):
    """dt = softplus(raw + bias) and the logarithm of the decay, [T, H]."""
    raw = s["dt"].float() + s["dt_bias"]
    dt = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs()))
    return dt, -torch.exp(s["A_log"]) * dt


def _gated(y, s):
    y = y + s["D"][:, None] * s["x"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return y.to(s["x"].dtype)


def _step_plain(s):
    heads = s["x"].shape[1]
    dt, a = _gates(s)
    rep = heads // s["B"].shape[1]
    B, C = (s[w].float().repeat_interleave(rep, 1) for w in ("B", "C"))
    new = s["state"][s["slots"]] * a.exp()[:, :, None, None] + (dt[..., None] * s["x"].float())[..., None] * B[:, :, None]
    s["state"][s["slots"]] = new
    return {"y": _gated((new * C[:, :, None]).sum(-1), s), "state": s["state"]}


def _scan_plain(s):
    """Chunks of 64: within a chunk the products of all pairs, between chunks the products of the decays."""
    Q = 64
    x, cu = s["x"], s["cu"]
    total, heads, dim = x.shape
    n, groups, state = len(s["lens"]), s["B"].shape[1], s["B"].shape[2]
    chunks = -(-max(s["lens"]) // Q)
    i = torch.arange(chunks * Q, device="cuda")
    row = (cu[:-1, None] + i).clamp(max=total - 1)  # sequences padded to [n, chunks * Q]
    there = i < (cu[1:] - cu[:-1])[:, None]
    dt, a = (torch.where(there[..., None], v[row], 0.0).reshape(n, chunks, Q, heads).permute(0, 1, 3, 2) for v in _gates(s))
    fold = lambda v: torch.where(there[..., None, None], v[row], 0.0).float().reshape(n, chunks, Q, *v.shape[1:]).transpose(2, 3)  # noqa: E731
    xs, B, C = fold(x), fold(s["B"]), fold(s["C"])  # [n, chunks, heads or groups, Q, ...]
    G = (C @ B.transpose(3, 4)).repeat_interleave(heads // groups, 2)
    B, C = (v.repeat_interleave(heads // groups, 2) for v in (B, C))
    cum = a.double().cumsum(-1)  # [n, chunks, heads, Q]
    sees = i[:Q, None] >= i[:Q]
    decay = torch.where(sees, cum[..., :, None] - cum[..., None, :], -math.inf).exp().float()
    y = (G * decay * dt[..., None, :]) @ xs
    # each chunk's own contribution to the state behind it, then what stands ahead of each chunk
    own_part = (xs * (dt * (cum[..., -1:] - cum).exp().float())[..., None]).transpose(3, 4) @ B  # [n, chunks, heads, dim, state]
    start = s["state"][s["slots"]]
    parts = torch.cat([start[:, None], own_part], 1).transpose(1, 2).reshape(n, heads, chunks + 1, dim * state)
    gone = torch.nn.functional.pad(cum[..., -1].transpose(1, 2).cumsum(-1), (1, 0))  # [n, heads, chunks + 1]
    c = torch.arange(chunks + 1, device="cuda")
    weight = torch.where(c[:, None] >= c, gone[..., :, None] - gone[..., None, :], -math.inf).exp().float()
    ahead = (weight @ parts).reshape(n, heads, chunks + 1, dim, state)
    s["state"][s["slots"]] = ahead[:, :, -1]
    y = y + cum.exp().float()[..., None] * (C @ ahead[:, :, :-1].transpose(1, 2).transpose(3, 4))
    t = torch.arange(total, device="cuda")
    at = torch.bucketize(t, cu[1:], right=True)
    y = y.transpose(2, 3).reshape(n, chunks * Q, heads, dim)[at, t - cu[at]]
    return {"y": _gated(y, s), "state": s["state"]}


def _quantise(x):
    """e4m3 values of x [T, H, D] and their scale per (token, head): the least power of two with which the
    largest magnitude stays within 448 (1 where all are zero)."""
    amax = x.float().abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-100)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    return (x.float() / scale[..., None]).to(_F8), scale


def _turn(x, cos, sin, neighbours):
    half = cos.shape[-1]
    f, rest = x[..., :2 * half].float(), x[..., 2 * half:]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (f[..., 0::2], f[..., 1::2]) if neighbours else (f[..., :half], f[..., half:])
    u, v = a * cos - b * sin, b * cos + a * sin
    f = torch.stack([u, v], -1).flatten(-2) if neighbours else torch.cat([u, v], -1)
    return torch.cat([f.to(x.dtype), rest], -1)


def _append_plain(s):
    page = s["k_cache"].shape[2]
    at, off = s["slots"] // page, s["slots"] % page
    cos, sin = s["rotation"][s["positions"]].chunk(2, 1)
    q, k = (_turn(s[w], cos, sin, s["neighbours"]) for w in ("q", "k"))
    if s["k_scale"] is None:
        s["k_cache"][at, :, off] = k
        s["v_cache"][at, :, off] = s["v"]
        return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
    k, ks = _quantise(k)
    v, vs = _quantise(s["v"])
    s["k_cache"].view(torch.uint8)[at, :, off] = k.view(torch.uint8)
    s["v_cache"].view(torch.uint8)[at, :, off] = v.view(torch.uint8)
    s["k_scale"][at, :, off] = ks
    s["v_scale"][at, :, off] = vs
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def run(s):
    if own:
        import gated_deltanet_delta_gb300 as gdn
        if s["op"] == "norm":
            y = gdn.add_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=s["eps"], e4m3=s["f8"], group=s["group"])
            out = {} if s["residual"] is None else {"residual": s["residual"]}
            return dict(out, y=y[0], scale=y[1]) if s["f8"] else dict(out, y=y)
        if s["op"] == "conv":
            y = gdn.short_conv(s["x"], s["weight"], s["hist"], s["slots"], None if s["step"] else s["cu"], bias=s["bias"],
                               splits=s["splits"], dev_status=s["status"])
            return {"y": list(y), "hist": s["hist"]}
        if s["op"] == "step":
            y = gdn.ssm_decode_step(s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], s["state"], s["slots"], D=s["D"],
                                    z=s["z"], dev_status=s["status"])
            return {"y": y, "state": s["state"]}
        if s["op"] == "scan":
            y = gdn.ssm_prefill_chunked(s["x"], s["dt"], s["B"], s["C"], s["A_log"], s["dt_bias"], s["state"], s["slots"], s["cu"],
                                        s["longest"], D=s["D"], z=s["z"], workspace=s["workspace"], dev_status=s["status"])
            return {"y": y, "state": s["state"]}
        q = gdn.attn_cache_append(s["q"], s["k"], s["v"], s["rotation"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                                  k_scale=s["k_scale"], v_scale=s["v_scale"], neighbours=s["neighbours"], dev_status=s["status"])
        held = {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
        return held if s["k_scale"] is None else dict(held, k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"norm": _norm_plain, "conv": _conv_plain, "step": _step_plain, "scan": _scan_plain, "append": _append_plain}[s["op"]](s)


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _e4m3_grid(x):
    """x rounded to the nearest e4m3 value (ties to even), |x| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_norm(s):
    r, got = s["x"].double(), {}
    if s["residual"] is not None:
        r = (r + s["residual"].double()).to(s["x"].dtype).double()  # the stream is kept in 16 bits
        got["residual"] = r
    y = s["weight"].double() * r / torch.sqrt((r * r).mean(1, keepdim=True) + s["eps"])
    if not s["f8"]:
        return dict(got, y=y)
    width = s["group"] or y.shape[1]
    scale = torch.stack([p.abs().amax(1) for p in y.split(width, 1)], 1) / 448.0
    scale[scale == 0] = 1.0
    return dict(got, y=_e4m3_grid(y / scale.repeat_interleave(width, 1)), scale=scale)


def _exact_conv(s):
    w, b, ends = s["weight"].double(), s["bias"].double(), s["cu"].tolist()
    taps, hist, out = w.shape[1], s["hist"].double(), []
    for n, slot in enumerate(s["slots"].tolist()):
        line = torch.cat([hist[slot], s["x"][ends[n]:ends[n + 1]].double().T], 1)  # [C, taps - 1 + length]
        y = b[:, None] + sum(w[:, j:j + 1] * line[:, j:line.shape[1] - taps + 1 + j] for j in range(taps))
        out.append((y / (1.0 + torch.exp(-y))).T)
        hist[slot] = line[:, -(taps - 1):]
    return {"y": list(torch.cat(out).split(s["splits"], 1)), "hist": hist}


def _exact_scan(s):
    """Token by token, all sequences side by side."""
    x = s["x"].double()
    total, heads, dim = x.shape
    lens, cu = s["lens"], s["cu"].tolist()
    rep = heads // s["B"].shape[1]
    B, C = s["B"].double(), s["C"].double()
    raw = s["dt"].double() + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    keep = torch.exp(-torch.exp(s["A_log"].double()) * dt)
    add = dt[..., None] * x
    h = s["state"].double()[s["slots"]]
    y = torch.empty_like(x)
    order = sorted(range(len(lens)), key=lambda n: -lens[n])  # the longest first: those still running are a prefix
    first = torch.tensor([cu[n] for n in order], device="cuda")
    h = h[torch.tensor(order, device="cuda")].unflatten(1, (-1, rep))  # [n, G, rep, dim, state]
    running = len(order)
    for t in range(max(lens)):
        while lens[order[running - 1]] <= t:
            running -= 1
        at = first[:running] + t
        now = h[:running]
        now.mul_(keep[at].unflatten(1, (-1, rep))[..., None, None])
        now.add_(add[at].unflatten(1, (-1, rep))[..., None] * B[at][:, :, None, None])
        y[at] = (now @ C[at][:, :, None, :, None]).squeeze(-1).flatten(1, 2)
    y = y + s["D"].double()[:, None] * x
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z / (1.0 + torch.exp(-z))
    end = s["state"].double()
    end[s["slots"][torch.tensor(order, device="cuda")]] = h.flatten(1, 2)
    return {"y": y, "state": end}


def _exact_append(s):
    size, dim = s["k_cache"].shape[2:]
    at, off = s["slots"] // size, s["slots"] % size
    angle = s["rotation"].double()[s["positions"]]
    half = angle.shape[1] // 2
    turn = torch.complex(angle[:, None, :half], angle[:, None, half:])
    first = torch.arange(half, device="cuda") * (2 if s["neighbours"] else 1)
    second = first + (1 if s["neighbours"] else half)
    got, rows = {}, {"v": s["v"].double()}
    for name in ("q", "k"):
        x = s[name].double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        rows[name] = x
    got["q"] = rows["q"]
    for name in ("k", "v"):
        x, f8 = rows[name], s[name + "_scale"] is not None
        cache = s[name + "_cache"].float().double()
        if f8:
            x = x.to(s["q"].dtype).double()  # the 8-bit cache quantises the rows that a 16-bit one would hold
            amax = x.abs().amax(-1)
            scale = torch.exp2(torch.round(torch.log2(amax.clamp(min=1e-30) / 448.0)) - 1)  # at most the one wanted
            for _ in range(3):
                scale = torch.where(amax > 448.0 * scale, 2.0 * scale, scale)
            scale = torch.where(amax > 0, scale.clamp(min=2.0 ** -100), 1.0)
            held = s[name + "_scale"].double()
            held[at, :, off] = scale
            got[name + "_scale"] = held
            x = _e4m3_grid(x / scale[..., None])
        cache[at, :, off] = x
        got[name] = cache
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "step": _exact_scan, "scan": _exact_scan, "append": _exact_append}[case["op"]](s)
