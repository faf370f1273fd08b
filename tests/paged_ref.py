"""The 16-bit paged operators from their formulas in 64 bits, and how far a result may be from them.

A rounding to a 16-bit type is off by at most half a step, H(t) = eps / 2 of the value (bf16 2^-8,
fp16 2^-11; below fp16's normal numbers 2^-25). In what follows u = 2^-24.
"""
import torch

import gqa_causal_attention_gb300 as g

U = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def rotate(x, pos, table, norm_w, eps):
    """RMSNorm (norm_w given) and RoPE of x [n, heads, D] at positions pos [n] (table [P, R/2, 2]),
    float64; and the magnitude sum of each value's two products."""
    x = x.double()
    if norm_w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * norm_w.double()
    if table is None:
        return x, x.abs()
    cs = table.double()[pos.long()][:, None]
    c, s, r = cs[..., 0], cs[..., 1], table.shape[1]
    a, b, rest = x[..., :r], x[..., r:2 * r], x[..., 2 * r:]
    y = torch.cat([a * c - b * s, b * c + a * s, rest], -1)
    mag = torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs(), rest.abs()], -1)
    return y, mag


def rotate_tol(y, mag, t):
    """One rounding of y, and fp32's in the two products, their sum, the norm's factor (a sum of D
    squares in a tree, its root within 2 ulp) and the weights: at most 20 of u each."""
    return half_step(t) * y.abs() * (1 + 2.0 ** -8) + 20 * U * mag + 2.0 ** -25


def attend(q, k, v, seen, softcap=0.0, scale=None):
    """q [Lq, H, D] over k, v [n, Hkv, D] (float64), seen [Lq, n]: out, sum w |v| / sum w, and a bound of
    what fp32 scores leave uncertain of the weights (relative)."""
    Lq, H, D = q.shape
    Hkv = k.shape[1]
    scale = D ** -0.5 if not scale or scale <= 0 else scale
    q = q.double().view(Lq, Hkv, H // Hkv, D).permute(1, 2, 0, 3)
    k, v = k.double().permute(1, 0, 2)[:, None], v.double().permute(1, 0, 2)[:, None]
    s = scale * (q @ k.transpose(-1, -2))
    # (D + 4) roundings of a sum of magnitudes; the rest (scale, log2 e, reference, 2^x) a few u of the score
    mag = scale * (q.abs() @ k.abs().transpose(-1, -2))
    if softcap > 0:
        s = softcap * torch.tanh(s / softcap)
    unsure = (D + 4) * U * mag + 8 * U * (s.abs() + softcap) + 8 * U
    unsure = torch.where(seen, unsure, 0.0).amax(-1, keepdim=True)
    s = torch.where(seen, s, float("-inf"))
    m = s.amax(-1, keepdim=True)
    w = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    v = torch.where(seen.any(0)[:, None], v, 0.0)
    back = lambda x: x.permute(2, 0, 1, 3).reshape(Lq, H, -1)   # noqa: E731
    return back(w @ v), back(w @ v.abs()), back(unsure)


def attend_tol(out, vabs, unsure, t, weights_rounded):
    """The output's rounding; weights off by `unsure` (above and below the line: twice); and, where the
    weights are rounded to t for the second product (tensor cores), half a step of each. (Split in
    two parts of t they are off by its square; fp16's smallest step, 2^-24 of a weight of 1, adds
    up to 2^-12 for the longest sums tested; sums of fp32: n u, below 2^-12 too.)"""
    w = half_step(t) if weights_rounded else half_step(t) ** 2 + 2.0 ** -14
    return half_step(t) * out.abs() * (1 + 2.0 ** -6) + (w * (1 + 2.0 ** -6) + 2 * unsure + 2.0 ** -16) * vabs + 2.0 ** -24


def check(got, want, tol, what=""):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() / tol
    assert over.max().item() <= 1.0, f"{what}: {over.max().item():.2f} of what is allowed"


# ---------------------------------------------------------------- inputs

def dev():
    return torch.device("cuda:0")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


def status():
    return torch.zeros(1, dtype=torch.int32, device=dev())


def gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


def normal(gn, shape, t=torch.float32):
    return torch.randn(shape, generator=gn, device=dev()).to(t)


def rows(gn, T, heads, D, t, layout="slice"):
    """[T, heads, D]: a slice of wider rows, head-major, or contiguous."""
    if layout == "slice":
        return normal(gn, (T, heads + 3, D + 8), t)[:, 1:heads + 1, :D] if D % 8 == 0 else None
    if layout == "heads":
        return normal(gn, (heads, T, D), t).transpose(0, 1)
    return normal(gn, (T, heads, D), t)


class Cache:
    """Pools whose pages are handed out in a random order; what is not in use holds NaNs."""

    def __init__(self, gn, pages, Hkv, page, D, t, fused=False):
        self.page, self.D, self.Hkv, self.t = page, D, Hkv, t
        if fused:                                # k and v of a page side by side: a page stride
            both = torch.full((pages, 2, Hkv, page, D), float("nan"), dtype=t, device=dev())
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k = torch.full((pages, Hkv, page, D), float("nan"), dtype=t, device=dev())
            self.v = torch.full_like(self.k, float("nan"))
        self.free = torch.randperm(pages, generator=gn, device=dev()).tolist()

    def table(self, lens, extra=1, unused=-1):
        need = [-(-n // self.page) for n in lens]
        t = torch.full((len(lens), max(need) + extra), unused, dtype=torch.int32)
        for b, n in enumerate(need):
            t[b, :n] = torch.tensor([self.free.pop() for _ in range(n)], dtype=torch.int32)
        return t.to(dev())

    def fill(self, gn, table, lens, scale=1.0):
        """Random keys and values for the rows of a table; returns them, [n, Hkv, D] each."""
        out = []
        for row, n in zip(table.tolist(), lens):
            k = normal(gn, (n, self.Hkv, self.D)) * scale
            k, v = k.to(self.t), normal(gn, (n, self.Hkv, self.D), self.t)
            self.put(row, 0, k, v)
            out.append((k, v))
        return out

    def put(self, row, first, k, v):
        for i in range(0, k.shape[0]):
            p = first + i
            self.k[row[p // self.page], :, p % self.page] = k[i]
            self.v[row[p // self.page], :, p % self.page] = v[i]

    def read(self, pool, row, n):
        pages = pool[torch.tensor(row[:-(-n // self.page)], device=dev()).long()]
        return pages.transpose(1, 2).flatten(0, 1)[:n]


def rope(D, R, positions, theta=1e4):
    rp = g.RopeParams.make(theta=theta, rope_dim=R, max_positions=positions)
    table = g.rope_table(rp, D, dev())
    return rp, table, table.view(positions, (R or D) // 2, 2)
