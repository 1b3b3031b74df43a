"""Workloads of the serving operators that surround the recurrent layers: attention of a chunk of new
tokens over a paged cache (attn_paged), writing a cache with quantisation and reading it back
(attn_cache_write, attn_cache_read), and the verification of drafted tokens (draft_verify).

Each operator has a plain form in elementary torch operations (32-bit arithmetic, one rounding at the
end) and the library's own call; `own` picks which of the two run() makes.  Both take what prepare()
gives.  listed() names fixed workloads, draw() makes others of the same ranges, work() counts the
bytes and operations a pass cannot do without, and exact() evaluates the definition in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}
_F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _attn(name, seqs, new, kv, hq, hkv, dim, page, dtype, cache):
    """seqs sequences; the longest has `kv` cached keys of which its last `new` tokens are queries."""
    return {"name": name, "op": "attn", "seqs": seqs, "new": new, "kv": kv, "hq": hq, "hkv": hkv, "dim": dim,
            "page": page, "dtype": dtype, "cache": cache}


def _cache(name, op, seqs, kv, hkv, dim, page, dtype, cache):
    return {"name": name, "op": op, "seqs": seqs, "kv": kv, "hkv": hkv, "dim": dim, "page": page, "dtype": dtype,
            "cache": cache}


def listed():
    return [
        # one user generating, a short context: one token, latency only
        _attn("attn 1 token 1 seq", 1, 1, 1001, 32, 8, 128, 16, "bf16", "same"),
        # a batch of users generating one token each, ragged contexts, unquantised cache
        _attn("attn 1 token 64 seqs", 64, 1, 8192, 32, 8, 128, 64, "bf16", "same"),
        # the same service with the cache held in 8 bits, so that longer contexts fit
        _attn("attn 1 token 64 seqs e4m3", 64, 1, 16384, 32, 4, 128, 64, "bf16", "e4m3"),
        # a decode window of 8 tokens per sequence (drafted tokens being verified), 256-wide heads
        _attn("attn window 32 seqs e4m3", 32, 8, 15360, 16, 2, 256, 64, "bf16", "e4m3"),
        # chunks of long prompts on top of what is cached already
        _attn("attn chunk 2 seqs", 2, 4096, 15360, 32, 8, 128, 64, "bf16", "same"),
        # whole prompts of different lengths in one call, 64-wide heads, fp16
        _attn("attn prompts 9 seqs f16", 9, 4096, 4096, 16, 4, 64, 32, "f16", "same"),
        # one token of each of a batch of sequences enters the cache
        _cache("cache write 64 tokens", "write", 64, 1, 8, 128, 64, "bf16", "e4m3"),
        # packed prompts enter the cache in one call
        _cache("cache write prompts", "write", 4, 8192, 16, 128, 64, "bf16", "e4m3"),
        # cached prompts are handed to another kernel or machine as dense rows
        _cache("cache read prompts", "read", 4, 8192, 16, 128, 64, "bf16", "e4m3"),
        # one user, four drafted tokens, a small vocabulary
        {"name": "verify 4 drafts 1 seq", "op": "verify", "seqs": 1, "drafts": 4, "vocab": 32000, "noise": 0.5},
        # a batch with a window of 8: seven drafted tokens and the one after them
        {"name": "verify 7 drafts 64 seqs", "op": "verify", "seqs": 64, "drafts": 7, "vocab": 131072, "noise": 0.5},
        # a large batch, an odd vocabulary, a draft that is often wrong
        {"name": "verify 3 drafts 255 seqs", "op": "verify", "seqs": 255, "drafts": 3, "vocab": 100003, "noise": 1.5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("attn", "attn", "attn", "write", "read", "verify"))
    if kind == "verify":
        return {"op": "verify", "seqs": _log_int(rng, 1, 255), "drafts": rng.randint(1, 8), "vocab": _log_int(rng, 1000, 131072),
                "noise": round(rng.uniform(0.2, 2.0), 2)}
    dim, dtype, cache = rng.choice((64, 128, 128, 256)), rng.choice(("bf16", "bf16", "f16")), rng.choice(("same", "e4m3"))
    page = rng.choice((16, 32, 48, 64, 128, 256))
    hkv = rng.choice((1, 2, 4, 8))
    if kind != "attn":
        seqs = _log_int(rng, 1, 128)
        kv = _log_int(rng, 1, max(2, min(8192, 15360 * 16 * 128 // (seqs * hkv * dim))))
        return {"op": kind, "seqs": seqs, "kv": kv, "hkv": hkv, "dim": dim, "page": page, "dtype": dtype, "cache": cache}
    group = rng.choice((1, 2, 3, 4, 6, 8, 16))
    form = rng.choice(("token", "window", "chunk"))
    if form == "chunk":  # queries x keys x heads x dim at most the listed chunk's
        seqs = rng.randint(1, 6)
        new = _log_int(rng, 9, 4096)
        most = 2 * 4096 * 15360 * 32 * 128 // (seqs * new * hkv * group * dim)
        kv = _log_int(rng, new, max(new, min(15360, most // 2)))
    else:  # bytes of the cache at most the listed batch's
        seqs = _log_int(rng, 1, 128)
        new = 1 if form == "token" else rng.randint(2, 8)
        kv = _log_int(rng, max(new, 16), max(32, min(16384, 64 * 8192 * 8 * 128 // (2 * seqs * hkv * dim))))
    return {"op": "attn", "seqs": seqs, "new": new, "kv": kv, "hq": hkv * group, "hkv": hkv, "dim": dim, "page": page,
            "dtype": dtype, "cache": cache}


def _lens(seqs, longest):
    """Ragged lengths: the first sequence has the longest, the others spread over 1/8 .. 1 of it."""
    return [max(1, int(longest * (1.0 if n == 0 else 0.125 + 0.875 * ((n * 0.6180339887498949) % 1.0)))) for n in range(seqs)]


def _attn_lens(case):
    kv = _lens(case["seqs"], case["kv"])
    new = [min(a, b) for a, b in zip(kv, _lens(case["seqs"], case["new"]) if case["new"] > 8 else [case["new"]] * case["seqs"])]
    return new, kv


def work(case):
    """Bytes: every input read once, every output written once.  Operations: two per product and sum of
    the matrix products over the keys that each query may see."""
    if case["op"] == "verify":
        # the accepted draft's probability pairs are a few bytes; a row of the target, and after a
        # rejection one of the draft, has to be read (about half of the sequences see a rejection)
        n, t, v = case["seqs"], case["drafts"], case["vocab"]
        return {"bytes": n * v * 4 * 1.5 + n * t * 20, "flops": n * v * 3}
    row = case["hkv"] * case["dim"]
    two = 2
    held = (1 + 4 / case["dim"]) if case["cache"] == "e4m3" else two  # bytes per cached value, its share of a scale included
    if case["op"] == "attn":
        new, kv = _attn_lens(case)
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(new, kv))
        out = sum(new) * case["hq"] * (case["dim"] * two * 2 + 4)
        return {"bytes": out + 2 * sum(kv) * row * held, "flops": 4 * pairs * case["hq"] * case["dim"]}
    tokens = sum(_lens(case["seqs"], case["kv"]))
    return {"bytes": 2 * tokens * row * (two + held), "flops": 2 * tokens * row * 2}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _page_table(g, pages_of, total):
    """Distinct pages in shuffled order; entries past a sequence's own pages are -1."""
    perm = torch.randperm(total, generator=g, device="cuda")
    table = torch.full((len(pages_of), max(max(pages_of), 1)), -1, dtype=torch.int64)
    at = torch.arange(table.shape[1])[None, :] < torch.tensor(pages_of)[:, None]
    table = table.cuda()
    table[at.cuda()] = perm[: sum(pages_of)]
    return table


def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).cuda()


def _slots(table, lens, page):
    """Flat cache slot (page * page_size + offset) of every packed token, and its sequence and position."""
    n = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
    pos = torch.arange(sum(lens), device="cuda") - _cu(lens)[:-1][n]
    return table[n, pos // page] * page + pos % page, n, pos


def _filled_cache(g, case, table, lens, total):
    """A cache that holds `lens` tokens; what no token was written to is left as memory is found: NaN.
    Keys have a few channels of larger size, and values a mean, as trained layers' have."""
    hkv, dim, page = case["hkv"], case["dim"], case["page"]
    slots, _, _ = _slots(table, lens, page)
    size = torch.exp(0.7 * _randn(g, hkv, dim))
    out = []
    for shift in (0.0, 0.3):
        rows = (_randn(g, slots.numel(), hkv, dim) * size + shift).to(_DT[case["dtype"]])
        if case["cache"] == "e4m3":
            rows, sc = _quantise(rows)
            rows = rows.view(torch.uint8)
            cache = torch.full((total, hkv, page, dim), 0x7F, dtype=torch.uint8, device="cuda")
            scale = torch.full((total, hkv, page), float("nan"), device="cuda")
            scale[slots // page, :, slots % page] = sc
        else:
            cache = torch.full((total, hkv, page, dim), float("nan"), dtype=_DT[case["dtype"]], device="cuda")
            scale = None
        cache[slots // page, :, slots % page] = rows
        out += [cache.view(_F8) if case["cache"] == "e4m3" else cache, scale]
    return out


def prepare(case, seed):
    g = _gen(seed)
    s = {"op": case["op"]}
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "verify":
        n, t, v = case["seqs"], case["drafts"], case["vocab"]
        logits = _randn(g, n, t + 1, v).mul_(2.5)
        s["target"] = torch.softmax(logits, -1)
        # the draft model's logits: the target's with noise
        s["draft"] = torch.softmax(logits[:, :t] + case["noise"] * _randn(g, n, t, v), -1)
        s["tokens"] = torch.multinomial(s["draft"].reshape(n * t, v), 1, generator=g).reshape(n, t)
        s["u"] = torch.rand((n, t), generator=g, device="cuda")
        s["u_sample"] = torch.rand((n,), generator=g, device="cuda")
        return s
    page, dt = case["page"], _DT[case["dtype"]]
    lens = _attn_lens(case)[1] if case["op"] == "attn" else _lens(case["seqs"], case["kv"])
    pages_of = [-(-k // page) for k in lens]
    total = sum(pages_of) + 3
    s["table"] = _page_table(g, pages_of, total)
    if case["op"] == "write":
        # keys and values as the fused projection leaves them: slices of one wider row per token
        hkv, dim = case["hkv"], case["dim"]
        rows = torch.cat([_randn(g, sum(lens), hkv, dim) * torch.exp(0.7 * _randn(g, hkv, dim)),
                          _randn(g, sum(lens), hkv, dim) + 0.3], 1).to(dt)
        s["k"], s["v"] = rows[:, :hkv], rows[:, hkv:]
        s["slots"] = _slots(s["table"], lens, page)[0]
        f8 = case["cache"] == "e4m3"
        for name in ("k", "v"):
            c = torch.zeros((total, hkv, page, dim), dtype=torch.uint8 if f8 else dt, device="cuda")
            s[name + "_cache"] = c.view(_F8) if f8 else c
            s[name + "_scale"] = torch.ones((total, hkv, page), device="cuda") if f8 else None
        return s
    s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"] = _filled_cache(g, case, s["table"], lens, total)
    if case["op"] == "read":
        s["cu"], s["total"], s["dtype"] = _cu(lens), sum(lens), dt
        return s
    new, kv = _attn_lens(case)
    s["q"] = (_randn(g, sum(new), case["hq"], case["dim"]) * 1.5).to(dt)
    s["cu"], s["kv_lens"] = _cu(new), torch.tensor(kv, dtype=torch.int64, device="cuda")
    s["max_new"], s["max_kv"] = max(new), max(kv)
    s["scale"] = case["dim"] ** -0.5
    s["lse"] = torch.empty((sum(new), case["hq"]), device="cuda")
    s["workspace"] = None
    if own:
        import gated_deltanet_delta_gb300 as gdn
        s["workspace"] = torch.empty(gdn.attn_paged_workspace_size(case["dim"]), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def _quantise(x):
    """e4m3 values of x [T, H, D] and their scale per (token, head): the least power of two with which
    the largest magnitude stays within 448 (1 where all are zero)."""
    amax = x.float().abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-100)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    return (x.float() / scale[..., None]).to(_F8), scale


def _write_plain(s):
    page = s["k_cache"].shape[2]
    at, off = s["slots"] // page, s["slots"] % page
    if s["k_scale"] is None:
        s["k_cache"][at, :, off] = s["k"]
        s["v_cache"][at, :, off] = s["v"]
        return {"k": s["k_cache"], "v": s["v_cache"]}
    k, ks = _quantise(s["k"])
    v, vs = _quantise(s["v"])
    s["k_cache"].view(torch.uint8)[at, :, off] = k.view(torch.uint8)
    s["v_cache"].view(torch.uint8)[at, :, off] = v.view(torch.uint8)
    s["k_scale"][at, :, off] = ks
    s["v_scale"][at, :, off] = vs
    return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _rows(cache, scale, page, off):
    """Cached rows at (page, off), widened and scaled: [..., H, D]."""
    if scale is None:
        return cache[page, :, off].float()
    return cache.view(torch.uint8)[page, :, off].view(_F8).float() * scale[page, :, off][..., None]


def _read_plain(s):
    size = s["k_cache"].shape[2]
    t = torch.arange(s["total"], device="cuda")
    n = torch.bucketize(t, s["cu"], right=True) - 1
    pos = t - s["cu"][n]
    page, off = s["table"][n, pos // size], pos % size
    return {"k": _rows(s["k_cache"], s["k_scale"], page, off).to(s["dtype"]),
            "v": _rows(s["v_cache"], s["v_scale"], page, off).to(s["dtype"])}


def _attn_plain(s):
    q, size = s["q"], s["k_cache"].shape[2]
    total, hq, dim = q.shape
    hkv = s["k_cache"].shape[1]
    n = s["kv_lens"].shape[0]
    cu, kv = s["cu"], s["kv_lens"]
    new = cu[1:] - cu[:-1]
    i = torch.arange(s["max_new"], device="cuda")
    j = torch.arange(s["max_kv"], device="cuda")
    # queries padded to [n, hkv, group, max_new, dim]
    row = (cu[:-1, None] + i).clamp(max=total - 1)
    qp = q[row].float().reshape(n, s["max_new"], hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4)
    # keys and values padded to [n, hkv, max_kv, dim]; what is past a sequence's end is unwritten memory
    page = s["table"][:, j // size].clamp(min=0)
    there = (j < kv[:, None])[:, None, :, None]
    k = torch.where(there, _rows(s["k_cache"], s["k_scale"], page, (j % size).expand(n, -1)).transpose(1, 2), 0.0)
    v = torch.where(there, _rows(s["v_cache"], s["v_scale"], page, (j % size).expand(n, -1)).transpose(1, 2), 0.0)
    sc = qp.reshape(n, hkv, -1, dim) @ k.transpose(2, 3)
    sc = sc.reshape(n, hkv, hq // hkv, s["max_new"], s["max_kv"]).mul_(s["scale"])
    # query i stands at position kv - new + i and sees the keys up to its own
    hidden = j > (kv - new)[:, None, None] + i[:, None]
    sc.masked_fill_(hidden[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    z = p.sum(-1, keepdim=True)
    o = (p.reshape(n, hkv, -1, s["max_kv"]) @ v).reshape(n, hkv, hq // hkv, s["max_new"], dim)
    o = torch.where(z > 0, o / z, 0.0)
    lse = (m + z.log()).squeeze(-1)
    t = torch.arange(total, device="cuda")
    at = torch.bucketize(t, cu, right=True) - 1
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(n, s["max_new"], hq, dim)[at, t - cu[at]].to(q.dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(n, s["max_new"], hq)[at, t - cu[at]]}


def _verify_plain(s):
    p, q, x = s["target"], s["draft"], s["tokens"]
    n, t, _ = q.shape
    px = p[:, :t].gather(2, x[..., None]).squeeze(-1)
    qx = q.gather(2, x[..., None]).squeeze(-1)
    count = (s["u"] * qx < px).long().cumprod(1).sum(1)
    at = torch.arange(n, device="cuda")
    pr = p[at, count]
    qr = torch.where((count < t)[:, None], q[at, count.clamp(max=t - 1)], 0.0)
    # probabilities in whole units of 2^-36: exact, and their sums do not depend on the order
    pw, qw = ((x.clamp(0.0, 1.0) * 2.0 ** 36).long() for x in (pr, qr))
    w = (pw - qw).clamp(min=0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, pw)
    mark = (w.sum(1) * (s["u_sample"] * 2.0 ** 24).long()) >> 24
    token = (w.cumsum(1) <= mark[:, None]).sum(1)
    i = torch.arange(t + 1, device="cuda")
    padded = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(i < count[:, None], padded, torch.where(i == count[:, None], token[:, None], -1))
    return {"accepted": count, "tokens": tokens}


def run(s):
    if own:
        import gated_deltanet_delta_gb300 as gdn
        if s["op"] == "attn":
            out = gdn.attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu"], s["max_new"],
                                 scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"], lse=s["lse"],
                                 workspace=s["workspace"], dev_status=s["status"])
            return {"out": out, "lse": s["lse"]}
        if s["op"] == "write":
            gdn.attn_cache_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"], dev_status=s["status"])
            held = {"k": s["k_cache"], "v": s["v_cache"]}
            return held if s["k_scale"] is None else dict(held, k_scale=s["k_scale"], v_scale=s["v_scale"])
        if s["op"] == "read":
            k, v = gdn.attn_cache_read(s["k_cache"], s["v_cache"], s["table"], s["cu"], s["total"], dtype=s["dtype"],
                                       k_scale=s["k_scale"], v_scale=s["v_scale"], dev_status=s["status"])
            return {"k": k, "v": v}
        accepted, tokens = gdn.draft_verify(s["target"], s["draft"], s["tokens"], s["u"], s["u_sample"], dev_status=s["status"])
        return {"accepted": accepted, "tokens": tokens}
    return {"attn": _attn_plain, "write": _write_plain, "read": _read_plain, "verify": _verify_plain}[s["op"]](s)


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _wide(cache, scale):
    c = cache.view(torch.uint8).view(_F8).double() if scale is not None else cache.double()
    return c if scale is None else c * scale.double()[..., None]


def _one_sequence(s, which, n, length):
    """Sequence n's cached rows in 64 bits: [H, length, D]."""
    cache, scale = s[which + "_cache"], s[which + "_scale"]
    pages = s["table"][n, : -(-length // cache.shape[2])]
    rows = _wide(cache[pages], None if scale is None else scale[pages])
    return rows.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :length]


def _exact_attn(s):
    cu, kv = s["cu"].tolist(), s["kv_lens"].tolist()
    total, hq, dim = s["q"].shape
    out = torch.zeros((total, hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((total, hq), -math.inf, dtype=torch.float64, device="cuda")
    for n, length in enumerate(kv):
        first, last = cu[n], cu[n + 1]
        k, v = _one_sequence(s, "k", n, length), _one_sequence(s, "v", n, length)
        sees = torch.arange(length, device="cuda")[None] <= torch.arange(first, last, device="cuda")[:, None] + (length - last)
        for h in range(hq):
            g = h // (hq // k.shape[0])
            score = torch.mm(s["q"][first:last, h].double(), k[g].T) * s["scale"]
            score = torch.where(sees, score, -math.inf)
            z = torch.logsumexp(score, 1)
            lse[first:last, h] = z
            out[first:last, h] = torch.nan_to_num(torch.exp(score - z[:, None])) @ v[g]
    return {"out": out, "lse": lse}


def _e4m3_grid(x):
    """x rounded to the nearest e4m3 value (ties to even), |x| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_write(s):
    size, got = s["k_cache"].shape[2], {}
    at, off = s["slots"] // size, s["slots"] % size
    for name in ("k", "v"):
        x = s[name].double()
        cache = _wide(s[name + "_cache"], None if s[name + "_scale"] is None else torch.ones_like(s[name + "_scale"]))
        if s[name + "_scale"] is not None:
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


def _exact_verify(s):
    p, q = s["target"], s["draft"]
    n, t, vocab = q.shape
    accepted, tokens = [], []
    for a in range(n):
        x, u = s["tokens"][a].tolist(), s["u"][a].double().tolist()
        pick = torch.arange(t, device="cuda"), s["tokens"][a]
        px, qx = p[a][pick].double().tolist(), q[a][pick].double().tolist()
        r = next((i for i in range(t) if not u[i] * qx[i] < px[i]), t)
        whole = torch.floor(p[a, r].double() * 2.0 ** 36)
        units = (whole - torch.floor(q[a, r].double() * 2.0 ** 36)).clamp(min=0).long() if r < t else whole.long()
        if int(units.sum()) == 0:
            units = whole.long()
        mark = int(units.sum()) * int(float(s["u_sample"][a]) * 2 ** 24) // 2 ** 24
        token = int(torch.searchsorted(units.cumsum(0), torch.tensor(mark, device="cuda"), right=True))
        accepted.append(r)
        tokens.append(x[:r] + [token] + [-1] * (t - r))
    return {"accepted": torch.tensor(accepted), "tokens": torch.tensor(tokens)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s)
    if case["op"] == "write":
        return _exact_write(s)
    if case["op"] == "verify":
        return _exact_verify(s)
    lens = (s["cu"][1:] - s["cu"][:-1]).tolist()
    return {w: torch.cat([_one_sequence(s, w, n, length).transpose(0, 1) for n, length in enumerate(lens)]) for w in ("k", "v")}
