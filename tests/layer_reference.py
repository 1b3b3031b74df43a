"""The short convolution, the state space scan, the rotation and the norm from their definitions, in 64 bits and token by
token, with what the derived tolerances of the tests need: the same sums over magnitudes."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half a step of the subnormal numbers


def ragged(lens):
    return torch.tensor([0] + list(lens)).cumsum(0)


def conv(x, w, bias, hist, slots, lens, silu):
    """x [T, C], hist [pool, C, taps - 1] (64 bits): outputs, sums of magnitudes ahead of the activation, new history."""
    taps, hist = w.shape[1], hist.clone()
    y, mag, at = torch.zeros_like(x), torch.zeros_like(x), 0
    b = torch.zeros(x.shape[1], dtype=x.dtype) if bias is None else bias
    for slot, n in zip(slots, lens):
        line = torch.cat([hist[slot].T, x[at:at + n]])  # [taps - 1 + n, C]
        for t in range(n):
            seen = line[t:t + taps]
            s = b + (w.T * seen).sum(0)
            y[at + t] = s * torch.sigmoid(s) if silu else s
            mag[at + t] = b.abs() + (w.T * seen).abs().sum(0)
        hist[slot] = line[line.shape[0] - (taps - 1):].T
        at += n
    return y, mag, hist


def scan(x, dt, B, C, z, A_log, D, dt_bias, state, slots, lens):
    """All in 64 bits.  Returns y, the state pool, and the same with every product's magnitude: what roundings inside
    the sums are relative to (the D term apart)."""
    state, mags = state.clone(), state.abs()
    rep = x.shape[1] // B.shape[1]
    B, C = B.repeat_interleave(rep, 1), C.repeat_interleave(rep, 1)
    step = torch.nn.functional.softplus(dt + dt_bias, threshold=1e9)
    keep = torch.exp(-torch.exp(A_log) * step)
    y, ymag, at = torch.zeros_like(x), torch.zeros_like(x), 0
    for slot, n in zip(slots, lens):
        s, m = state[slot], mags[slot]
        for t in range(at, at + n):
            add = (step[t][:, None] * x[t])[:, :, None] * B[t][:, None]
            s = keep[t][:, None, None] * s + add
            m = keep[t][:, None, None] * m + add.abs()
            y[t] = (s * C[t][:, None]).sum(-1) + D[:, None] * x[t]
            ymag[t] = (m * C[t][:, None].abs()).sum(-1)
        state[slot], mags[slot] = s, m
        at += n
    if z is not None:
        gate = z * torch.sigmoid(z)
        y, ymag = y * gate, ymag * gate.abs()
    return y, state, ymag, mags


def turn(x, table, neighbours):
    """x [T, H, D] rotated by the rows [T, R] of the table, in fp32 with every product and sum rounded, as documented."""
    half = table.shape[1] // 2
    cos, sin = table[:, None, :half], table[:, None, half:]
    i = torch.arange(half) * (2 if neighbours else 1)
    j = i + (1 if neighbours else half)
    out = x.clone()
    a, b = x[..., i].float(), x[..., j].float()
    out[..., i] = (a * cos - b * sin).to(x.dtype)
    out[..., j] = (b * cos + a * sin).to(x.dtype)
    return out
