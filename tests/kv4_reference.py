"""Plain 64-bit statements of the 4-bit cache's operators, for the tests: numpy and
torch on the host, nothing of the library."""
import math

import numpy as np
import torch

BLOCK = 16


def quantize_rows(x):
    """x float16 [..., D] -> codes uint8, step float16 bits, zero point: the cache's grid in IEEE float32."""
    f = x.astype(np.float32)
    lo = np.minimum(f.min(-1), np.float32(0))
    hi = np.maximum(f.max(-1), np.float32(0))
    r = np.maximum(hi - lo, np.float32(1e-5))
    step = (r / np.float32(15)).astype(np.float16)
    s = step.astype(np.float32)
    z = np.clip(np.rint(-lo / s), 0, 15).astype(np.float32)
    inv = np.float32(1) / s
    q = np.clip(np.rint(f * inv[..., None]) + z[..., None], 0, 15).astype(np.uint8)
    return q, step, z.astype(np.uint16)


def store(cache, k, v, slots, page):
    """Writes tokens into a host copy of the cache, uint8 [pages, heads, bytes]."""
    T, H, D = k.shape
    bb = 16 * D + 128
    blocks = cache.reshape(cache.shape[0], H, page // BLOCK, bb)
    for i, x in enumerate((k, v)):
        q, step, z = quantize_rows(x)
        packed = q[..., 0::2] | (q[..., 1::2] << 4)
        meta = np.stack([step.view(np.uint16), z], -1).view(np.uint8).reshape(T, H, 4)
        for t in range(T):
            if slots[t] < 0:
                continue
            p, off = divmod(int(slots[t]), page)
            b, row = divmod(off, BLOCK)
            at = i * 8 * D + row * (D // 2)
            blocks[p, :, b, at: at + D // 2] = packed[t]
            at = 16 * D + 64 * i + 4 * row
            blocks[p, :, b, at: at + 4] = meta[t]


def values(cache, slots, page, D):
    """float64 (k, v) [T, H, D] of the slots; and the steps [T, H]."""
    H = cache.shape[1]
    blocks = cache.reshape(cache.shape[0], H, page // BLOCK, 16 * D + 128)
    out = []
    slots = np.asarray(slots)
    p, off = slots // page, slots % page
    b, row = off // BLOCK, off % BLOCK
    for i in range(2):
        codes = blocks[..., i * 8 * D: (i + 1) * 8 * D].reshape(*blocks.shape[:3], BLOCK, D // 2)[p, :, b, row]
        meta = np.ascontiguousarray(
            blocks[..., 16 * D + 64 * i: 16 * D + 64 * (i + 1)].reshape(*blocks.shape[:3], BLOCK, 4)[p, :, b, row])
        w = meta.view(np.uint16).reshape(len(slots), H, 2)
        step = np.ascontiguousarray(w[..., 0]).view(np.float16).astype(np.float64)
        q = np.stack([codes & 15, codes >> 4], -1).reshape(len(slots), H, D).astype(np.float64)
        out.append((q - w[..., 1:].astype(np.float64)) * step[..., None])
        out.append(step)
    k, ks, v, vs = out
    return k, v, ks, vs


def attention(q, cache, table, lens, cu, page, scale, window=0):
    """float64 attention of q [T, Hq, D] (float16 tensor): (out, bound), the second the largest error that the
    kernel's roundings allow, element by element.

    The bound: the output's rounding and that of each weight times step to float16, half a step each (2^-11); the sum
    over tokens in float32 (one addition per block of 16 tokens, 2^-23 of what the codes add up to); the logits (8
    products of 16 channels and a few float operations: 2^-19 of the terms' sum), twice, for numerator and denominator."""
    T, Hq, D = q.shape
    Hk = cache.shape[1]
    g = Hq // Hk
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    bound = torch.zeros(T, Hq, D, dtype=torch.float64)
    qd = q.double().cpu()
    for b in range(len(lens)):
        n, a, e = int(lens[b]), int(cu[b]), int(cu[b + 1])
        m = e - a
        if m == 0 or n == 0:
            continue
        pos = np.arange(n)
        slots = np.asarray(table[b])[pos // page].astype(np.int64) * page + pos % page
        k, v, ks, vs = (torch.from_numpy(x) for x in values(cache, slots, page, D))
        at = torch.arange(n - m, n)[:, None]
        j = torch.arange(n)[None]
        seen = (j <= at) & (at >= 0)
        if window:
            seen &= j > at - window
        some = seen.any(1)
        for h in range(Hk):
            qh = qd[a:e, h * g: (h + 1) * g].transpose(0, 1)                  # [g, m, D]
            s = qh @ k[:, h].T * scale
            s = s.masked_fill(~seen, -math.inf)
            top = s.amax(-1, keepdim=True).nan_to_num(neginf=0.0)
            w = torch.exp(s - top)
            w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
            o = w @ v[:, h]
            av = w @ v[:, h].abs()
            a15 = (w * (15 * vs[:, h])).sum(-1, keepdim=True)
            eps_s = 2.0 ** -19 * abs(scale) * 15 * ks[:, h].max() * qh.abs().sum(-1, keepdim=True)
            bd = 2.0 ** -11 * (o.abs() + av) * 1.01 + (n / 16 + 32) * 2.0 ** -23 * a15 + 2 * eps_s * av + 2.0 ** -24
            o[:, ~some] = 0
            out[a:e, h * g: (h + 1) * g] = o.transpose(0, 1)
            bound[a:e, h * g: (h + 1) * g] = bd.transpose(0, 1)
    return out, bound


def reserve(new, lens, table, free, count, page, total):
    """(slots, positions, cu, lens, count, table) after the step, plain Python."""
    table = table.copy()
    slots, positions, cu = [], [], [0]
    for b, n in enumerate(new):
        for i in range(n):
            pos = int(lens[b]) + i
            col = pos // page
            if pos % page == 0:
                count -= 1
                table[b, col] = free[count]
            slots.append(int(table[b, col]) * page + pos % page)
            positions.append(pos)
        cu.append(len(slots))
    pad = total - len(slots)
    return (np.array(slots + [-1] * pad), np.array(positions + [-1] * pad), np.array(cu),
            np.asarray(lens) + np.asarray(new), count, table)
