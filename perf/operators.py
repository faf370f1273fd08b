"""The 4-bit KV cache operators: what is measured, on which inputs, in plain torch and by the library.

A cache record holds one position of one kv head: D / 32 groups of 32 key values and as many of
32 value values, each group as 4-bit codes c in [-7, 7] (stored as c + 8) with one bf16 scale s,
standing for c * s. D = 32 m. Byte layout of a record:
  16 m bytes  key codes: 32-bit word w = a * m + g (a < 4, g < m) holds dims 32 g + 8 a + i,
              i = 0..7, at bits 4 i
  16 m bytes  value codes: 16-bit unit u = n * m + g (n < 8, g < m) holds dims 32 g + 4 n + j,
              j = 0..3, at bits 4 j
  2 m bytes   key scales (bf16), 2 m bytes value scales (bf16), padding to a multiple of 16
A group's scale is its largest magnitude / 7 rounded to bf16, its codes the values / scale
rounded to nearest, ties to even.

Operators: kv_cache_append_q4 and kv_cache_read_q4 (timed together as the round trip a chunk's
keys and values make), gqa_attn_decode_q4 (with or without the per-slot attention weights),
gqa_attn_decode_step_q4, kv_cache_evict_q4.
"""
import math

import torch

own = False          # set by the caller: False: the plain forms, True: the library's calls

EPS = 1e-6
LOG = math.log


# ---------------------------------------------------------------- cases

def listed():
    return [
        # serving: the new token of 64 rows enters the cache (RoPE, quantise) and is read back
        dict(name="append 64 x 1 token", op="append", B=64, Hkv=8, D=128, L=1, cap=8193, start=8000,
             window=0, R=128, norm=False, k_out=False, theta=5e5),
        # prompt: four 2048-token prompts enter the cache, rotated keys kept for the prefill,
        # the stored values read back for the next chunk's prefill
        dict(name="append 4 x 2048 tokens", op="append", B=4, Hkv=8, D=128, L=2048, cap=2048,
             start=0, window=0, R=128, norm=False, k_out=True, theta=5e5),
        # a chunk that wraps a sliding-window ring, wide heads with k RMSNorm
        dict(name="append ring 4096, D 256", op="append", B=1, Hkv=8, D=256, L=4001, cap=4096,
             start=12001, window=4096, R=256, norm=True, k_out=False, theta=1e4),
        # one short conversation, one token: latency
        dict(name="decode 1 x 500", op="decode", B=1, H=32, Hkv=8, D=128, lo=500, hi=500, cap=1024,
             window=0, softcap=0.0, weights=False),
        # batched serving, ragged lengths
        dict(name="decode 64 x 512..8192", op="decode", B=64, H=32, Hkv=8, D=128, lo=512, hi=8192,
             cap=8193, window=0, softcap=0.0, weights=False),
        # one very long context, 8 query heads per kv head
        dict(name="decode 1 x 131072, G 8", op="decode", B=1, H=64, Hkv=8, D=128, lo=131072,
             hi=131072, cap=131072, window=0, softcap=0.0, weights=False),
        # the same attention also accumulating each slot's attention weight for the eviction
        dict(name="decode+weights 8 x 4000", op="decode", B=8, H=64, Hkv=8, D=128, lo=3001, hi=4000,
             cap=4097, window=0, softcap=0.0, weights=True),
        # whole decode steps: raw q, k, v in; batched serving
        dict(name="step 64 x 512..8192", op="step", B=64, H=32, Hkv=8, D=128, lo=512, hi=8192,
             cap=8193, window=0, softcap=0.0, weights=False, R=128, norm=False, theta=5e5),
        # eight rows at 1024..2047 positions, partial rotary
        dict(name="step 8 x 1024..2047, R 64", op="step", B=8, H=64, Hkv=8, D=128, lo=1024, hi=2047,
             cap=2048, window=0, softcap=0.0, weights=False, R=64, norm=False, theta=1e6),
        # sliding-window ring, wide heads, softcap, q/k RMSNorm, one row
        dict(name="step ring 4096, D 256", op="step", B=1, H=16, Hkv=8, D=256, lo=16000, hi=16000,
             cap=4096, window=4096, softcap=50.0, weights=False, R=256, norm=True, theta=1e4),
        # one row trimmed by a few slots
        dict(name="evict 1 x 1100 to 1024", op="evict", B=1, Hkv=8, D=128, lo=1100, hi=1100,
             cap=1200, budget=1024, recent=256, cap_out=1200),
        # a batch trimmed to half
        dict(name="evict 16 x 8192 to 4096", op="evict", B=16, Hkv=8, D=128, lo=6001, hi=8192,
             cap=8192, budget=4096, recent=512, cap_out=4224),
    ]


def _span(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(LOG(lo), LOG(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "step", "evict"])
    D = rng.choice([32, 64, 96, 128, 128, 160, 192, 256])
    B = _span(rng, 1, 64)
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 4, 7, 8, 8, 12, 16])
    if op == "append":
        # values entering: at most those of the listed prompt case
        L = _span(rng, 1, max(1, min(8192, 4 * 8 * 2048 * 128 // (B * Hkv * D))))
        ring = rng.random() < 0.3
        cap = _span(rng, L, 2 * L + 64)
        start = rng.randint(0, 5000) if ring else rng.randint(0, cap - L)
        return dict(op=op, B=B, Hkv=Hkv, D=D, L=L, cap=cap, start=start, window=cap if ring else 0,
                    R=rng.choice([D, D, D // 2]), norm=rng.random() < 0.4,
                    k_out=rng.random() < 0.5, theta=rng.choice([1e4, 5e5]))
    if op == "evict":
        most = max(64, min(65536, 16 * 8 * 7096 * 128 // (B * Hkv * D)))
        hi = _span(rng, 64, most)
        budget = rng.randint(max(1, hi // 8), hi)
        return dict(op=op, B=B, Hkv=Hkv, D=D, lo=max(1, hi // 2), hi=hi, cap=hi + rng.randint(0, 9),
                    budget=budget, recent=rng.randint(0, budget),
                    cap_out=budget + rng.randint(0, 70))
    # cached slots: at most those of the listed batched case, and query heads' work as there
    most = max(16, min(131072, 64 * 8 * 4300 * 128 // (B * Hkv * D * max(1, G // 4))))
    hi = _span(rng, 1, most)
    lo = max(1, rng.randint(hi // 4, hi))
    ring = rng.random() < 0.2 and hi > 8
    c = dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, D=D, lo=lo, hi=hi, cap=hi + rng.randint(1, 40),
             window=0, softcap=rng.choice([0.0, 0.0, 30.0]), weights=not ring and rng.random() < 0.3)
    if ring:
        c["cap"] = c["window"] = max(1, rng.randint(hi // 2, hi))
    if op == "step":
        c.update(R=rng.choice([D, D, D // 2]), norm=rng.random() < 0.4,
                 theta=rng.choice([1e4, 5e5]))
    return c


# ---------------------------------------------------------------- the record format

def _record_bytes(D):
    return (36 * (D // 32) + 15) // 16 * 16


def _bf16(x):
    """x (float64) rounded once to bf16's eight significant bits (45 of 53 dropped), ties to even."""
    b = x.view(torch.int64)
    return ((b + (1 << 44) - 1 + (b >> 45 & 1)) >> 45 << 45).view(torch.float64)


def _quantise(x):
    """x [..., D] to (codes [..., D / 32, 32], scales [..., D / 32, 1]), float64."""
    g = x.double().unflatten(-1, (-1, 32))
    s = _bf16(g.abs().amax(-1, keepdim=True) / g.new_full((1,), 7.0))   # by a tensor: divided,
    # not multiplied by 1 / 7 rounded, which moves ties of the scale's last bit
    c = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, 1.0)), 0.0)
    return c.clamp(-7, 7), s


def _pack(k, v):
    """Records [..., record bytes] (uint8) of k and v [..., D]."""
    m = k.shape[-1] // 32
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    kn = (kc + 8).to(torch.uint8).unflatten(-1, (4, 8)).transpose(-2, -3).reshape(*k.shape[:-1], -1, 2)
    vn = (vc + 8).to(torch.uint8).unflatten(-1, (8, 4)).transpose(-2, -3).reshape(*k.shape[:-1], -1, 2)
    sc = [s.squeeze(-1).float().to(torch.bfloat16).contiguous().view(torch.uint8) for s in (ks, vs)]
    pad = torch.zeros(*k.shape[:-1], _record_bytes(32 * m) - 36 * m, dtype=torch.uint8, device=k.device)
    return torch.cat([kn[..., 0] | kn[..., 1] << 4, vn[..., 0] | vn[..., 1] << 4, *sc, pad], -1)


def _unpack(rec, D):
    """(k, v) [..., D] fp32 that records stand for."""
    m = D // 32
    def codes(b, a):
        n = torch.stack([b & 15, b >> 4], -1).flatten(-2).unflatten(-1, (a, m, 32 // a))
        return n.transpose(-2, -3).reshape(*b.shape[:-1], m, 32).float() - 8
    def scales(b):
        return b.contiguous().view(torch.bfloat16).float().unsqueeze(-1)
    k = codes(rec[..., :16 * m], 4) * scales(rec[..., 32 * m:34 * m])
    v = codes(rec[..., 16 * m:32 * m], 8) * scales(rec[..., 34 * m:36 * m])
    return k.flatten(-2), v.flatten(-2)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _keys(gen, *shape):
    """Keys or values: normal, a few channels of each head larger, as trained layers have them."""
    x = torch.randn(*shape, generator=gen, device="cuda")
    ch = torch.randn(shape[1], 1, shape[-1], generator=gen, device="cuda")
    return x * torch.exp(0.4 * ch) + 0.3 * ch


def _cache(gen, B, Hkv, cap, D):
    """A filled cache [B, Hkv, cap, record bytes], quantised a few thousand slots at a time."""
    rec = torch.empty(B, Hkv, cap, _record_bytes(D), dtype=torch.uint8, device="cuda")
    rows = max(1, (1 << 27) // (B * Hkv * D))
    for i in range(0, cap, rows):
        n = min(rows, cap - i)
        rec[:, :, i:i + n] = _pack(_keys(gen, B, Hkv, n, D), _keys(gen, B, Hkv, n, D))
    return rec


def _table(n, R, theta):
    """cos/sin table [n, R / 2, 2]: angles in 64 bits, rounded once."""
    f = theta ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def prepare(case, seed):
    c, gen = case, _gen(seed)
    B, Hkv, D, dev = c["B"], c["Hkv"], c["D"], "cuda"
    s = {"case": dict(c), "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    if c["op"] == "append":
        s["k"], s["v"] = _keys(gen, B, Hkv, c["L"], D), _keys(gen, B, Hkv, c["L"], D)
        s["cache"] = torch.zeros(B, Hkv, c["cap"], _record_bytes(D), dtype=torch.uint8, device=dev)
        s["start"] = c["start"] - torch.randint(0, min(c["start"], 97) + 1, (B,), generator=gen,
                                                device=dev).to(torch.int32)
        s["k_read"], s["v_read"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        s["k_rot"] = torch.empty_like(s["k"]) if c["k_out"] else None
        s["table"] = _table(c["start"] + c["L"], c["R"], c["theta"])
        s["k_norm"] = 1 + 0.1 * torch.randn(D, generator=gen, device=dev) if c["norm"] else None
        return s
    s["cache"] = _cache(gen, B, Hkv, c["cap"], D)
    s["len"] = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=gen, device=dev).to(torch.int32)
    if c["op"] == "evict":
        # accumulated attention: a few slots hold most of it, some hold none (ties)
        w = torch.rand(B, Hkv, c["cap"], generator=gen, device=dev) ** 8
        s["w"] = torch.where(torch.rand(w.shape, generator=gen, device=dev) < 0.1, 0.0, w)
        s["cache_out"] = torch.zeros(B, Hkv, c["cap_out"], _record_bytes(D), dtype=torch.uint8,
                                     device=dev)
        s["w_out"] = torch.empty(B, Hkv, c["cap_out"], device=dev)
        s["index"] = torch.empty(B, Hkv, c["budget"], dtype=torch.int32, device=dev)
        s["len_out"] = torch.empty(B, dtype=torch.int32, device=dev)
        return s
    s["q"] = torch.randn(B, c["H"], 1, D, generator=gen, device=dev)
    s["out"] = torch.empty_like(s["q"])
    s["w"] = torch.zeros(B, Hkv, c["cap"], device=dev) if c["weights"] else None
    if c["op"] == "step":
        s["k"], s["v"] = _keys(gen, B, Hkv, 1, D), _keys(gen, B, Hkv, 1, D)
        s["k_read"], s["v_read"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        s["table"] = _table(c["hi"] + 1, c["R"], c["theta"])
        for n in ("q_norm", "k_norm"):
            s[n] = 1 + 0.1 * torch.randn(D, generator=gen, device=dev) if c["norm"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _rotate(x, pos, table, norm_w):
    """RMSNorm (norm_w given) and RoPE of x [B, h, L, D] at positions pos [B, L], in 64 bits."""
    x = x.double()
    if norm_w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * norm_w.double()
    cs = table.double()[pos.long()][:, None]
    h = table.shape[1]
    a, b, rest = x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
    return torch.cat([a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1], rest], -1)


def _stands_for(x):
    c, s = _quantise(x)
    return (c * s).flatten(-2).float()


def _attend(c, q, k, v, live, weights):
    """q [B, H, 1, D] over k, v [B, Hkv, n, D], of which the first live[b] count."""
    B, Hkv, n, D = k.shape
    s = q.view(B, Hkv, -1, D) @ k.transpose(-1, -2) * D ** -0.5
    if c["softcap"] > 0:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    seen = torch.arange(n, device=q.device) < live.view(B, 1, 1, 1)
    s = torch.where(seen, s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    if weights is not None:
        weights[:, :, :n] += p.sum(2)
    return (p @ torch.where(seen.view(B, 1, n, 1), v, 0.0)).view(B, -1, 1, D)


def _plain_append(s):
    c = s["case"]
    pos = s["start"].view(-1, 1) + torch.arange(c["L"], device="cuda")
    k = _rotate(s["k"], pos, s["table"], s["k_norm"])
    out = [_stands_for(k), _stands_for(s["v"])]
    return out + [k.float()] if c["k_out"] else out


def _plain_decode(s):
    c = s["case"]
    live = s["len"].clamp(max=c["cap"])
    k, v = _unpack(s["cache"], c["D"])
    out = _attend(c, s["q"], k, v, live, s["w"])
    return [out] if s["w"] is None else [out, s["w"]]


def _plain_step(s):
    c = s["case"]
    pos = s["len"].view(-1, 1)
    q = _rotate(s["q"], pos, s["table"], s["q_norm"]).float()
    kn = _stands_for(_rotate(s["k"], pos, s["table"], s["k_norm"]))
    vn = _stands_for(s["v"])
    k, v = _unpack(s["cache"], c["D"])
    slot = (pos % c["cap"]).long().view(-1, 1, 1, 1).expand(-1, c["Hkv"], 1, c["D"])
    k.scatter_(2, slot, kn)
    v.scatter_(2, slot, vn)
    out = [_attend(c, q, k, v, (s["len"] + 1).clamp(max=c["cap"]), s["w"]), kn, vn]
    return out if s["w"] is None else out + [s["w"]]


def _plain_evict(s):
    c = s["case"]
    n = s["len"].view(-1, 1, 1)
    slot = torch.arange(c["cap"], device="cuda")
    key = torch.where(slot >= n - c["recent"], math.inf, s["w"])
    key = torch.where(slot >= n, -math.inf, key)
    first = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :c["budget"]]
    kept = n.clamp(max=c["budget"])
    rank = torch.arange(c["budget"], device="cuda")
    pad = c["cap_out"] - c["budget"]
    index = torch.where(rank[:first.shape[-1]] < kept, first, c["cap"]).sort(-1).values
    index = torch.nn.functional.pad(index, (0, c["budget"] - index.shape[-1]), value=c["cap"])
    there = index < c["cap"]
    at = torch.where(there, index, 0)
    w = torch.where(there, s["w"].gather(-1, at), 0.0)
    rec = s["cache"].view(torch.int32)
    rec = rec.gather(2, at.unsqueeze(-1).expand(-1, -1, -1, rec.shape[-1]))
    rec = torch.where(there.unsqueeze(-1), rec, 0)
    pads = torch.nn.functional.pad
    return [pads(rec, (0, 0, 0, pad)), pads(w, (0, pad)), torch.where(there, index, -1).int(),
            kept.flatten().int()]


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import gqa_causal_attention_gb300 as g
    c = s["case"]
    if "kept" not in s:      # what a program makes once per layer: parameters and workspace
        s["kept"] = kept = {}
        if "table" in s:
            kept["rp"] = g.RopeParams.make(theta=c["theta"], rope_dim=c["R"],
                                           max_positions=s["table"].shape[0])
        if c["op"] in ("decode", "step"):
            top = c["hi"] + 1 if c["op"] == "step" else c["hi"]
            size = (g.gqa_attn_decode_step_q4_workspace_size if c["op"] == "step"
                    else g.gqa_attn_decode_q4_workspace_size)
            n = size(c["B"], c["H"], c["Hkv"], c["D"], top, c["window"], c["weights"])
            kept["ws"] = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    kept = s["kept"]
    if c["op"] == "append":
        g.kv_cache_append_q4(s["k"], s["v"], s["cache"], s["start"], c["start"], kept["rp"],
                             s["table"], s["k_norm"], EPS, k_out=s["k_rot"], window=c["window"],
                             status=s["status"])
        g.kv_cache_read_q4(s["cache"], s["k_read"], s["v_read"], s["start"], c["start"],
                           window=c["window"], status=s["status"])
        out = [s["k_read"], s["v_read"]]
        return out + [s["k_rot"]] if c["k_out"] else out
    if c["op"] == "decode":
        g.gqa_attn_decode_q4(s["q"], s["cache"], s["len"], c["hi"], s["out"], weights=s["w"],
                             window=c["window"], softcap=c["softcap"], workspace=kept["ws"],
                             status=s["status"])
        return [s["out"]] if s["w"] is None else [s["out"], s["w"]]
    if c["op"] == "step":
        g.gqa_attn_decode_step_q4(s["q"], s["k"], s["v"], s["out"], s["cache"], s["len"], c["hi"],
                                  kept["rp"], s["table"], s["q_norm"], s["k_norm"], EPS,
                                  weights=s["w"], window=c["window"], softcap=c["softcap"],
                                  workspace=kept["ws"], status=s["status"])
        g.kv_cache_read_q4(s["cache"], s["k_read"], s["v_read"], s["len"], c["hi"],
                           window=c["window"], status=s["status"])
        out = [s["out"], s["k_read"], s["v_read"]]
        return out if s["w"] is None else out + [s["w"]]
    g.kv_cache_evict_q4(s["cache"], s["w"], s["len"], c["hi"], c["budget"], c["recent"],
                        s["cache_out"], s["w_out"], s["index"], s["len_out"], status=s["status"])
    return [s["cache_out"].view(torch.int32), s["w_out"], s["index"], s["len_out"]]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "decode": _plain_decode, "step": _plain_step,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work

def work(case):
    c = case
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    rec = 36 * (D // 32)                       # codes and scales of one position of one kv head
    if c["op"] == "append":
        n = B * Hkv * c["L"]
        stored = B * Hkv * min(c["L"], c["cap"])
        b = n * D * 8 + stored * rec           # k, v in; records out
        b += stored * rec + stored * D * 8     # records in; k, v out
        b += n * D * 4 if c["k_out"] else 0
        b += c["L"] * c["R"] * 4               # one row's angles at least
        return {"bytes": b, "flops": n * D * 8}
    if c["op"] == "evict":
        mean = (c["lo"] + c["hi"]) / 2
        kept = B * Hkv * min(mean, c["budget"])
        return {"bytes": B * Hkv * mean * 4 + kept * (2 * rec + 8) + B * Hkv * c["cap_out"] * 4,
                "flops": B * Hkv * mean}
    live = min((c["lo"] + c["hi"]) / 2 + (c["op"] == "step"), c["cap"])
    b = B * Hkv * live * rec + 2 * B * c["H"] * D * 4
    b += B * Hkv * live * 8 if c["weights"] else 0
    if c["op"] == "step":
        b += B * Hkv * (D * 16 + 2 * rec) + B * c["R"] * 4
    return {"bytes": b, "flops": 4 * B * c["H"] * D * live}


# ---------------------------------------------------------------- exact values

def _places(D):
    """(byte, shift) of each dim's key code and value code in a record."""
    m, d = D // 32, torch.arange(D, device="cuda")
    g, e = d // 32, d % 32
    kb = 4 * ((e // 8) * m + g) + (e % 8) // 2
    vb = 16 * m + 2 * ((e // 4) * m + g) + (e % 4) // 2
    return (kb, 4 * (e % 2)), (vb, 4 * (e % 2))


def _values(rec, D):
    """k, v [..., D] in float64 of records, dim by dim."""
    m, d, got = D // 32, torch.arange(D, device="cuda"), []
    for (byte, shift), at in zip(_places(D), (32 * m, 34 * m)):
        code = (rec[..., byte].int() >> shift.int() & 15) - 8
        lo = rec[..., at + 2 * (d // 32)].int()
        hi = rec[..., at + 2 * (d // 32) + 1].int()
        got.append(code.double() * (lo << 16 | hi << 24).view(torch.float32).double())
    return got


def _exact_rotate(x, p, table, w):
    """One row x [h, D] at position p."""
    x = x.double()
    if w is not None:
        x = x * w.double() * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    h = table.shape[1]
    c, s = table[p, :, 0].double(), table[p, :, 1].double()
    y = x.clone()
    y[:, :h] = x[:, :h] * c - x[:, h:2 * h] * s
    y[:, h:2 * h] = x[:, h:2 * h] * c + x[:, :h] * s
    return y


def _exact_codes(x):
    """What 4 bits make of x [..., D] (float64): borders compared by products, no division."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    top = g.abs().amax(-1)
    # bf16 neighbours of top / 7: the one nearer, an even last bit at a tie
    _, e = torch.frexp(top / 7)
    ulp = (e - 8 + 127 << 23).view(torch.float32).double()          # 2^(e - 8)
    low = torch.floor(top / 7 / ulp)
    off = top - 7 * low * ulp
    up = (2 * off > 7 * ulp) | ((2 * off == 7 * ulp) & (low % 2 == 1))
    s = ((low + up.double()) * ulp)[..., None]
    a = g.abs()
    c = torch.zeros_like(a)
    for i in range(7):                   # past the border i + 1/2; at it only to an even code
        c += (a > (i + 0.5) * s) | ((a == (i + 0.5) * s) & (i % 2 == 1))
    return (torch.sign(g) * c * s).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    c, B, Hkv, D = case, case["B"], case["Hkv"], case["D"]
    if c["op"] == "append":
        k, v = torch.empty_like(s["k"], dtype=torch.float64), s["v"].double()
        for b in range(B):
            p0 = int(s["start"][b])
            p = torch.arange(p0, p0 + c["L"], device="cuda")
            for h in range(Hkv):
                x = s["k"][b, h].double()
                if c["norm"]:
                    x = x * s["k_norm"].double() * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
                r = c["R"] // 2
                cs, sn = s["table"][p, :, 0].double(), s["table"][p, :, 1].double()
                k[b, h] = x
                k[b, h, :, :r] = x[:, :r] * cs - x[:, r:2 * r] * sn
                k[b, h, :, r:2 * r] = x[:, r:2 * r] * cs + x[:, :r] * sn
        out = [_exact_codes(k), _exact_codes(v)]
        return out + [k] if c["k_out"] else out
    if c["op"] == "evict":
        ws, lens = s["w"].cpu().tolist(), s["len"].tolist()
        if B * Hkv * c["hi"] > 2_000_000:
            return None
        w = torch.zeros(B, Hkv, c["cap_out"], dtype=torch.float64)
        for b in range(B):
            n = lens[b]
            old = max(0, n - c["recent"])
            for h in range(Hkv):
                row = ws[b][h]
                best = sorted(range(old), key=lambda i: (-row[i], i))[:max(0, c["budget"] - (n - old))]
                keep = sorted(best) + list(range(old, n)) if n > c["budget"] else list(range(n))
                w[b, h, :len(keep)] = torch.tensor([row[i] for i in keep], dtype=torch.float64)
        return [None, w, None, None]
    outs, ws = [], []
    kn, vn = [], []
    for b in range(B):
        q = s["q"][b, :, 0].double()
        n = int(s["len"][b])
        live = min(n + (c["op"] == "step"), c["cap"])
        k, v = _values(s["cache"][b, :, :live], D)
        if c["op"] == "step":
            q = _exact_rotate(q, n, s["table"], s["q_norm"])
            kn.append(_exact_codes(_exact_rotate(s["k"][b, :, 0], n, s["table"], s["k_norm"])))
            vn.append(_exact_codes(s["v"][b, :, 0].double()))
            k[:, n % c["cap"]], v[:, n % c["cap"]] = kn[-1], vn[-1]
        G = c["H"] // Hkv
        z = torch.einsum("hgd,hnd->hgn", q.view(Hkv, G, D), k) / math.sqrt(D)
        if c["softcap"] > 0:
            z = torch.tanh(z / c["softcap"]) * c["softcap"]
        p = torch.softmax(z, -1)
        outs.append(torch.einsum("hgn,hnd->hgd", p, v).reshape(c["H"], 1, D))
        if s["w"] is not None:
            row = torch.zeros(Hkv, c["cap"], dtype=torch.float64, device="cuda")
            row[:, :live] = p.sum(1)
            ws.append(row)
    got = [torch.stack(outs)]
    if c["op"] == "step":
        got += [torch.stack(kn)[:, :, None], torch.stack(vn)[:, :, None]]
    return got + [torch.stack(ws)] if ws else got
