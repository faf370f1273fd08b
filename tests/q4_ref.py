"""64-bit reference of the 4-bit KV cache: the record format, quantisation and the
operators over it, in plain torch float64 on the CPU, from the definitions in
include/gqa_attn.h. Shares no code with the library."""
import math

import torch

F8 = torch.float64


def record_bytes(D):
    return -(-36 * (D // 32) // 16) * 16


def round_bf16(x):
    """x >= 0 (float64) rounded once to bf16, ties to even, the subnormal grid below 2^-126."""
    m, e = torch.frexp(x)
    unit = torch.ldexp(torch.ones_like(x), (e - 8).clamp(min=-133))
    return torch.where(x > 0, torch.round(x / unit) * unit, 0.0)


def quantise(x):
    """x [..., D] -> codes [..., m, 32], scales [..., m] (float64; NaN for a group with an
    inf or NaN, its codes 0)."""
    g = x.to(F8).unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(g).all(-1)
    g = torch.where(bad[..., None], 0.0, g)
    s = round_bf16(g.abs().amax(-1) / 7)
    c = torch.where(s[..., None] > 0, torch.round(g / torch.where(s > 0, s, 1.0)[..., None]), 0.0)
    return c.clamp(-7, 7), torch.where(bad, math.nan, s)


def stands_for(x):
    c, s = quantise(x)
    return (c * s[..., None]).flatten(-2)


def pack(k, v):
    """uint8 records [..., record_bytes] of k, v [..., D], byte by byte from the layout."""
    D = k.shape[-1]
    m = D // 32
    rec = torch.zeros(*k.shape[:-1], record_bytes(D), dtype=torch.int64)
    for part, x in enumerate((k, v)):
        c, s = quantise(x)
        u = (c + 8).to(torch.int64).flatten(-2)
        for d in range(D):
            g, e = divmod(d, 32)
            if part == 0:
                bit = 32 * ((e // 8) * m + g) + 4 * (e % 8)
            else:
                bit = 128 * m + 16 * ((e // 4) * m + g) + 4 * (e % 4)
            rec[..., bit // 8] |= u[..., d] << bit % 8
        bits = s.to(torch.float32).to(torch.bfloat16).view(torch.int16).to(torch.int64) & 0xffff
        for g in range(m):
            at = (32 + 2 * part) * m + 2 * g
            rec[..., at], rec[..., at + 1] = bits[..., g] & 255, bits[..., g] >> 8
    return rec.to(torch.uint8)


def unpack(rec, D):
    """float64 (k, v) [..., D] that records stand for."""
    rec, m, out = rec.cpu().to(torch.int64), D // 32, []
    for part in range(2):
        x = torch.empty(*rec.shape[:-1], D, dtype=F8)
        for d in range(D):
            g, e = divmod(d, 32)
            if part == 0:
                bit = 32 * ((e // 8) * m + g) + 4 * (e % 8)
            else:
                bit = 128 * m + 16 * ((e // 4) * m + g) + 4 * (e % 4)
            at = (32 + 2 * part) * m + 2 * g
            s = (rec[..., at] | rec[..., at + 1] << 8) << 16
            s = torch.where(s >= 1 << 31, s - (1 << 32), s).to(torch.int32).view(torch.float32)
            x[..., d] = ((rec[..., bit // 8] >> bit % 8 & 15) - 8).to(F8) * s.to(F8)
        out.append(x)
    return out


def rotate(x, pos, table, norm_w=None, eps=1e-6):
    """RMSNorm (norm_w) and RoPE of x [B, h, L, D], row b's token l at pos[b] + l, angles
    from the fp32 table [positions, R / 2, 2]; eps as the library gets it (fp32)."""
    x = x.to(F8)
    if norm_w is not None:
        e = float(torch.tensor(eps, dtype=torch.float32))
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + e) * norm_w.to(F8)
    if table is None:
        return x
    h = table.shape[1]
    p = torch.as_tensor(pos).view(-1, 1) + torch.arange(x.shape[2])
    cs = table.to(F8)[p][:, None]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat([a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1],
                      x[..., 2 * h:]], -1)


def decode(q, k, v, live, softcap=0.0, scale=0.0):
    """q [B, H, 1, D] over the first live[b] of k, v [B, Hkv, n, D]: (out, weights [B, Hkv, n],
    largest |score|)."""
    B, H, _, D = q.shape
    Hkv, n = k.shape[1:3]
    out, w, top = torch.zeros(B, H, 1, D, dtype=F8), torch.zeros(B, Hkv, n, dtype=F8), 0.0
    for b in range(B):
        L = int(live[b])
        s = q[b, :, 0].to(F8).view(Hkv, H // Hkv, D) @ k[b, :, :L].to(F8).transpose(-1, -2)
        s = s * (scale if scale > 0 else D ** -0.5)
        if softcap > 0:
            s = softcap * torch.tanh(s / softcap)
        p = torch.softmax(s, -1)
        out[b] = (p @ v[b, :, :L].to(F8)).reshape(H, 1, D)
        w[b, :, :L] = p.sum(1)
        top = max(top, float(s.abs().max()))
    return out, w, top


def evict(weights, n, budget, recent):
    """Kept slots, in order, of one head's n live slots."""
    if n <= budget:
        return list(range(n))
    old = n - recent
    w = [math.inf if math.isnan(x) else x for x in weights[:old].tolist()]
    nan_first = [not math.isnan(x) for x in weights[:old].tolist()]
    best = sorted(range(old), key=lambda i: (-w[i], nan_first[i], i))[:budget - recent]
    return sorted(best) + list(range(old, n))
