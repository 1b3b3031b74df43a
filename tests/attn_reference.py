"""Plain 64-bit forms of paged attention, cache quantisation and draft verification (numpy and torch on
the CPU), written from the definitions in include/gdn.h, for the tests of those operations."""
import numpy as np
import torch


def e4m3_round(x):
    """float64 -> the nearest e4m3 value, ties to even, by the format's step (|x| <= 448)."""
    a = np.abs(x)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.sign(x) * np.round(a / step) * step


def quantise(x):
    """x [.., D] -> (values float64 [.., D], scale float64 [..]) of an e4m3 cache."""
    x = np.asarray(x, np.float64)
    finite = np.isfinite(x)
    amax = np.where(finite, np.abs(x), 0.0).max(-1)
    scale = np.ones_like(amax)
    for idx in np.ndindex(*amax.shape):
        if amax[idx] > 0:
            s = 2.0 ** -100
            while amax[idx] > 448.0 * s:
                s *= 2.0
            scale[idx] = s
    return np.where(finite, e4m3_round(np.where(finite, x, 0.0) / scale[..., None]), np.nan), scale


def gather(cache, scale, table, length):
    """Cached rows of one sequence: [H, length, D] float64."""
    page_size = cache.shape[2]
    rows = []
    for t in range(length):
        page, off = int(table[t // page_size]), t % page_size
        r = cache[page, :, off].double()
        rows.append(r if scale is None else r * scale[page, :, off].double()[:, None])
    return torch.stack(rows, 1) if rows else torch.zeros((cache.shape[1], 0, cache.shape[3]), dtype=torch.float64)


def attention(q, k_cache, v_cache, k_scale, v_scale, table, kv_lens, cu, scale):
    """(out, lse, weighted |v|, largest sum |q k| scale, most keys, largest |v|), all float64, on the CPU.
    The last four are what error bounds are made of."""
    T, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    wabs = torch.zeros((T, Hq, D), dtype=torch.float64)
    lse = torch.full((T, Hq), -np.inf, dtype=torch.float64)
    size, keys, vmax = 0.0, 0, 0.0
    for n, L in enumerate(kv_lens):
        m = cu[n + 1] - cu[n]
        k = gather(k_cache, k_scale, table[n], L)
        v = gather(v_cache, v_scale, table[n], L)
        keys = max(keys, L)
        if L:
            vmax = max(vmax, float(v.abs().max()))
        for i in range(m):
            vis = L - m + i + 1
            if vis <= 0:
                continue
            for h in range(Hq):
                g = h // (Hq // Hkv)
                x = q[cu[n] + i, h].double()
                s = (k[g, :vis] @ x) * scale
                size = max(size, float((k[g, :vis].abs() @ x.abs()).max()) * abs(scale))
                z = torch.logsumexp(s, 0)
                w = torch.exp(s - z)
                lse[cu[n] + i, h] = z
                out[cu[n] + i, h] = w @ v[g, :vis]
                wabs[cu[n] + i, h] = w @ v[g, :vis].abs()
    return out, lse, wabs, size, keys, vmax


def verify(target, draft, drafts, u, us, num_drafts=None):
    """(accepted, tokens) by exact integer arithmetic; target, draft float32 arrays."""
    N, T = drafts.shape
    V = target.shape[2]
    accepted, tokens = [], []

    def whole(row):  # floor(clamp(p, 0, 1) 2^36), exact in float64; NaN counts as 0
        r = np.where(np.isnan(row), 0.0, row.astype(np.float64))
        return [int(x) for x in np.floor(np.clip(r, 0.0, 1.0) * 2.0 ** 36)]
    for n in range(N):
        nd = T if num_drafts is None else min(max(int(num_drafts[n]), 0), T)
        r = nd
        for t in range(nd):
            x = int(drafts[n, t])
            if not (0 <= x < V and np.float32(u[n, t]) * np.float32(draft[n, t, x]) < target[n, t, x]):
                r = t
                break
        P = whole(target[n, r])
        w = P
        if r < nd:
            w = [max(a - b, 0) for a, b in zip(P, whole(draft[n, r]))]
            if sum(w) == 0:
                w = P
        token = 0
        if sum(w) > 0:
            mark = sum(w) * int(np.float64(us[n]) * 2 ** 24) // 2 ** 24
            acc = 0
            for i, x in enumerate(w):
                acc += x
                if acc > mark:
                    token = i
                    break
        accepted.append(r)
        tokens.append([int(drafts[n, t]) for t in range(r)] + [token] + [-1] * (T - r))
    return np.array(accepted), np.array(tokens).reshape(N, T + 1)
