"""Serving in 16 bits from a paged KV cache: what is measured, on which inputs, in plain torch and
by the library.

A paged cache is two pools k_cache, v_cache [pages, Hkv, page, D] (bf16 or fp16). Row b's position
p lies in slot p % page of the pool's page block_table[b, p // page]. Queries, keys and values come
token-major, [T, heads, D], as slices of one fused projection.

Operators: kv_cache_append_paged (RMSNorm and RoPE of the queries and keys of packed sequences,
keys and values to their pages), gqa_attn_decode_paged (one query per row over its pages),
gqa_attn_decode_shared (the same for rows that all begin with one long prefix, whose pages are
read once for all), gqa_attn_prefill_packed (causal attention of whole prompts, packed).
"""
import math
import random

import torch

own = False          # set by the caller: False: the plain forms, True: the library's calls

EPS = 1e-6
LOG = math.log
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
# lo, hi: the sequences' lengths (append: new tokens; decode: cached positions; shared: positions
# after the prefix), spread over that range by the case's "mix". empty: every such row is empty.

def listed():
    return [
        # serving: the new token of each of 64 conversations enters the cache, its query rotated
        dict(name="append 64 x 1", op="append", type="bf16", B=64, H=32, Hkv=8, D=128, page=16,
             lo=1, hi=1, start=8000, R=128, norm=False, theta=5e5, mix=1, empty=0, pad=0),
        # prompts: five of different lengths, some after a cached beginning, q/k RMSNorm
        dict(name="append 5 prompts", op="append", type="fp16", B=5, H=32, Hkv=8, D=128, page=64,
             lo=301, hi=4000, start=1000, R=128, norm=True, theta=1e6, mix=2, empty=0, pad=37),
        # one short conversation, one token: latency
        dict(name="decode 1 x 500", op="decode", type="bf16", B=1, H=32, Hkv=8, D=128, page=16,
             lo=500, hi=500, window=0, softcap=0.0, mix=3, empty=0),
        # batched serving, ragged lengths, small pages
        dict(name="decode 64 x 512..8192", op="decode", type="bf16", B=64, H=32, Hkv=8, D=128,
             page=16, lo=512, hi=8192, window=0, softcap=0.0, mix=4, empty=0),
        # few very long contexts, 8 query heads per kv head
        dict(name="decode 8 x 32768, G 8", op="decode", type="fp16", B=8, H=64, Hkv=8, D=128,
             page=64, lo=32768, hi=32768, window=0, softcap=0.0, mix=5, empty=0),
        # a small model with a sliding window and softcap; rows without a request in the batch
        dict(name="decode window 1000, D 64", op="decode", type="fp16", B=23, H=14, Hkv=2, D=64,
             page=32, lo=1, hi=5000, window=1000, softcap=30.0, mix=6, empty=5),
        # a long system prompt shared by 64 conversations
        dict(name="shared 8192 + 64 x 1..500", op="shared", type="bf16", B=64, H=32, Hkv=8, D=128,
             page=16, prefix=8192, lo=1, hi=500, softcap=0.0, mix=7, empty=0),
        # five samples of one prompt that ends inside a page, some not yet begun
        dict(name="shared 2001 + 5 x 0..40", op="shared", type="fp16", B=5, H=28, Hkv=4, D=64,
             page=32, prefix=2001, lo=0, hi=40, softcap=0.0, mix=8, empty=2),
        # one short prompt: latency
        dict(name="prefill 1 x 77", op="prefill", type="fp16", B=1, H=32, Hkv=8, D=128, lo=77,
             hi=77, window=0, softcap=0.0, mix=9, empty=0, pad=0),
        # mixed prompts of a batch, padded to a round number of rows
        dict(name="prefill 16 x 1..2048", op="prefill", type="bf16", B=16, H=32, Hkv=8, D=128,
             lo=1, hi=2048, window=0, softcap=0.0, mix=10, empty=1, pad=100),
        # a sliding window and softcap, narrow heads
        dict(name="prefill 9 x 100..1800, window 512", op="prefill", type="fp16", B=9, H=16,
             Hkv=4, D=64, lo=100, hi=1800, window=512, softcap=50.0, mix=11, empty=0, pad=3),
        # one long document
        dict(name="prefill 1 x 8192", op="prefill", type="bf16", B=1, H=32, Hkv=8, D=128, lo=8192,
             hi=8192, window=0, softcap=0.0, mix=12, empty=0, pad=0),
    ]


def _span(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm (0 and 1 alike)."""
    hi = max(lo, hi)
    return max(lo, min(hi, int(round(math.exp(rng.uniform(LOG(max(lo, 1)), LOG(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "shared", "prefill", "prefill"])
    D = rng.choice([32, 64, 64, 80, 96, 128, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 4, 6, 7, 8, 8, 16])
    H = Hkv * G
    page = rng.choice([16, 16, 32, 64, 128, 256])
    B = _span(rng, 1, 64)
    c = dict(op=op, type=rng.choice(["bf16", "fp16"]), B=B, H=H, Hkv=Hkv, D=D,
             mix=rng.randint(0, 10 ** 6), empty=rng.choice([0, 0, 0, 3]))
    if op == "append":
        # values entering: at most those of the listed prompts
        most = max(1, 5 * 2150 * 48 * 128 // (B * (H + 2 * Hkv) * D))
        hi = 1 if rng.random() < 0.3 else _span(rng, 1, min(8192, most))
        c.update(page=page, lo=rng.randint(1, hi), hi=hi, start=_span(rng, 1, 9000),
                 R=rng.choice([D, D, D // 2]), norm=rng.random() < 0.4,
                 theta=rng.choice([1e4, 5e5]), pad=rng.choice([0, 0, 19]))
        return c
    c["softcap"] = rng.choice([0.0, 0.0, 30.0])
    if op == "prefill":
        # scores of the padded plain form: at most those of the listed long document
        hi = _span(rng, 1, min(16384, int(math.sqrt(32 * 8192 ** 2 / (B * H)))))
        c.update(lo=rng.randint(1, hi), hi=hi, pad=rng.choice([0, 0, 41]),
                 window=rng.choice([0, 0, 0, _span(rng, 1, hi)]))
        return c
    # cached positions: at most those of the listed batched case
    most = max(16, 64 * 8 * 4300 * 128 // (B * Hkv * D * max(1, G // 4)))
    if op == "shared":
        pre = _span(rng, 1, 8192)
        hi = _span(rng, 1, max(16, min(8192, most // 4)))
        c.update(page=page, prefix=pre, lo=rng.randint(0, hi), hi=hi)
        return c
    hi = _span(rng, 1, min(65536, most))
    c.update(page=page, lo=rng.randint(1, hi), hi=hi,
             window=rng.choice([0, 0, 0, _span(rng, 1, hi)]))
    return c


def _lens(c):
    rng = random.Random(c["mix"])
    n = [rng.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    return [0 if c["empty"] and b % (c["empty"] + 1) == c["empty"] else n[b] for b in range(c["B"])]


def _starts(c):
    rng = random.Random(c["mix"] + 77)
    return [rng.randint(c["start"] // 2, c["start"]) for _ in range(c["B"])]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 6271 + 29)


def _fused(gen, T, c):
    """q, k, v [T, heads, D]: slices of one fused projection's output. A few channels of each head
    are larger, as trained layers have them."""
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    x = torch.randn(T, H + 2 * Hkv, D, generator=gen, device="cuda")
    ch = torch.randn(H + 2 * Hkv, D, generator=gen, device="cuda")
    x = (x * torch.exp(0.4 * ch) + 0.3 * ch).to(TYPES[c["type"]])
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]


def _pools(gen, pages, c):
    shape = (pages, c["Hkv"], c["page"], c["D"])
    ch = torch.randn(2, c["Hkv"], 1, c["D"], generator=gen, device="cuda")
    return [(torch.randn(shape, generator=gen, device="cuda") * torch.exp(0.4 * ch[i])
             + 0.3 * ch[i]).to(TYPES[c["type"]]) for i in range(2)]


def _tables(gen, needs, c, spare=3):
    """Block tables (a list of int32 [B, most], unused entries -1) for lists of position counts, the
    pages of all of them in one random order, and the pool's size."""
    counts = [[-(-n // c["page"]) for n in need] for need in needs]
    total = sum(map(sum, counts)) + spare
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    out, at = [], 0
    for need in counts:
        t = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
        mask = (torch.arange(t.shape[1], device="cuda")
                < torch.tensor(need, device="cuda").view(-1, 1))
        t[mask] = order[at:at + sum(need)]
        at += sum(need)
        out.append(t)
    return out, total


def _table(n, R, theta):
    """cos/sin table [n, R / 2, 2]: angles in 64 bits, rounded once."""
    f = theta ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, gen, lens = case, _gen(seed), _lens(case)
    B, H, D, t = c["B"], c["H"], c["D"], TYPES[c["type"]]
    s = {"case": dict(c), "status": torch.zeros(1, dtype=torch.int32, device="cuda"),
         "lens": _i32(lens)}
    if c["op"] in ("append", "prefill"):
        cu = [sum(lens[:b]) for b in range(B + 1)]
        s["cu"], T = _i32(cu), cu[B] + c["pad"]
        s["q"], s["k"], s["v"] = _fused(gen, max(1, T), c)
        if c["op"] == "prefill":
            s["max_len"] = max(lens)
            s["out"] = torch.zeros(s["q"].shape, dtype=t, device="cuda")
            return s
        start = _starts(c)
        s["start"] = _i32(start)
        s["max_pos"] = max(a + n for a, n in zip(start, lens))
        (s["block_table"],), pages = _tables(gen, [[a + n for a, n in zip(start, lens)]], c)
        s["k_cache"], s["v_cache"] = _pools(gen, pages, c)
        s["q_out"] = torch.zeros(s["q"].shape, dtype=t, device="cuda")
        # a prompt's rotated keys are wanted for its prefill, a single token's are not
        s["k_out"] = None if c["hi"] == 1 else torch.zeros(s["k"].shape, dtype=t, device="cuda")
        s["table"] = _table(s["max_pos"] + 1, c["R"], c["theta"])
        for n in ("q_norm", "k_norm"):
            s[n] = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda") if c["norm"] else None
        return s
    s["max_len"] = max(1, max(lens))
    if c["op"] == "shared":
        (pre, s["block_table"]), pages = _tables(gen, [[c["prefix"]], lens], c)
        s["prefix_table"] = pre[0].contiguous()
    else:
        (s["block_table"],), pages = _tables(gen, [lens], c)
    s["k_cache"], s["v_cache"] = _pools(gen, pages, c)
    s["q"] = _fused(gen, B, c)[0]
    s["out"] = torch.zeros(B, H, D, dtype=t, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms (fp32)

def _packed_rows(s, n):
    """Rows of the packed tensors for [B, n] (sequence, token) places, and which of them exist."""
    i = torch.arange(n, device="cuda")
    there = i < s["lens"].view(-1, 1)
    rows = torch.where(there, s["cu"][:-1].view(-1, 1).long() + i, 0)
    return rows, there


def _rotate(x, pos, table, norm_w):
    """RMSNorm (norm_w given) and RoPE of x [n, heads, D] at positions pos [n]."""
    x = x.float()
    if norm_w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * norm_w
    cs = table[pos.long()][:, None]
    h = table.shape[1]
    a, b, rest = x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
    return torch.cat([a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1], rest], -1)


def _attend(c, q, k, v, seen):
    """q [B, Lq, H, D] over k, v [B, n, Hkv, D]; seen [B, Lq, n]. Rows that see nothing: zeros."""
    B, Lq, H, D = q.shape
    q = q.float().view(B, Lq, c["Hkv"], -1, D).permute(0, 2, 3, 1, 4)      # [B, Hkv, G, Lq, D]
    k, v = (x.float().permute(0, 2, 1, 3).unsqueeze(2) for x in (k, v))    # [B, Hkv, 1, n, D]
    s = q @ k.transpose(-1, -2) * D ** -0.5
    if c["softcap"] > 0:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    s = torch.where(seen[:, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    v = torch.where(seen.any(1)[:, None, None, :, None], v, 0.0)
    return (p @ v).permute(0, 3, 1, 2, 4).reshape(B, Lq, H, D)


def _gather(pool, table, n):
    """The first n positions [B, n, Hkv, D] of the rows of a block table."""
    page = pool.shape[2]
    x = pool[table[:, :-(-n // page)].clamp(min=0).long()]                 # [B, m, Hkv, page, D]
    return x.transpose(2, 3).flatten(1, 2)[:, :n]


def _plain_append(s):
    rows, there = _packed_rows(s, max(1, s["case"]["hi"]))
    rows = rows[there]
    pos = (s["start"].view(-1, 1) + torch.arange(there.shape[1], device="cuda"))[there].long()
    b = there.nonzero()[:, 0]
    page = s["case"]["page"]
    where = s["block_table"][b, pos // page].long()
    q = _rotate(s["q"][rows], pos, s["table"], s["q_norm"]).to(s["q"].dtype)
    k = _rotate(s["k"][rows], pos, s["table"], s["k_norm"]).to(s["k"].dtype)
    s["q_out"][rows] = q
    if s["k_out"] is not None:
        s["k_out"][rows] = k
    s["k_cache"][where, :, pos % page] = k
    s["v_cache"][where, :, pos % page] = s["v"][rows]


def _plain_decode(s):
    c, n = s["case"], s["max_len"]
    j = torch.arange(n, device="cuda")
    last = s["lens"].view(-1, 1)
    seen = j < last
    if c["window"]:
        seen = seen & (j >= last - c["window"])
    s["out"][:] = _attend(c, s["q"][:, None], _gather(s["k_cache"], s["block_table"], n),
                          _gather(s["v_cache"], s["block_table"], n), seen[:, None])[:, 0]


def _plain_shared(s):
    c, n, B = s["case"], s["max_len"], s["case"]["B"]
    seen = torch.arange(n, device="cuda") < s["lens"].view(-1, 1)
    seen = torch.cat([torch.ones(B, c["prefix"], dtype=torch.bool, device="cuda"), seen], 1)
    k, v = (torch.cat([_gather(x, s["prefix_table"][None], c["prefix"]).expand(B, -1, -1, -1),
                       _gather(x, s["block_table"], n)], 1) for x in (s["k_cache"], s["v_cache"]))
    s["out"][:] = _attend(c, s["q"][:, None], k, v, seen[:, None])[:, 0]


def _plain_prefill(s):
    c, n = s["case"], max(1, s["max_len"])
    rows, there = _packed_rows(s, n)
    i = torch.arange(n, device="cuda")
    band = i <= i.view(-1, 1)
    if c["window"]:
        band = band & (i > i.view(-1, 1) - c["window"])
    o = _attend(c, s["q"][rows], s["k"][rows], s["v"][rows], band & there[:, None])
    s["out"][rows[there]] = o[there].to(s["out"].dtype)


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import gqa_causal_attention_gb300 as g
    c = s["case"]
    if "kept" not in s:      # what a program makes once per layer: parameters and workspace
        s["kept"] = kept = {}
        sizes = (c["B"], c["H"], c["Hkv"], c["D"])
        n = 0
        if c["op"] == "append":
            kept["rp"] = g.RopeParams.make(theta=c["theta"], rope_dim=c["R"],
                                           max_positions=s["table"].shape[0])
        elif c["op"] == "decode":
            n = g.gqa_attn_decode_paged_workspace_size(*sizes, s["max_len"], c["window"])
        elif c["op"] == "shared":
            n = g.gqa_attn_decode_shared_workspace_size(*sizes, c["prefix"], s["max_len"])
        kept["ws"] = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    kept = s["kept"]
    if c["op"] == "append":
        g.kv_cache_append_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"],
                                s["start"], max(0, s["max_pos"] - 1), kept["rp"], s["table"],
                                s["k_norm"],
                                EPS, cu_seqlens=s["cu"], q=s["q"], q_out=s["q_out"],
                                q_norm_w=s["q_norm"], k_out=s["k_out"], status=s["status"])
    elif c["op"] == "decode":
        g.gqa_attn_decode_paged(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"],
                                s["max_len"], s["out"], window=c["window"], softcap=c["softcap"],
                                workspace=kept["ws"], status=s["status"])
    elif c["op"] == "shared":
        g.gqa_attn_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"],
                                 c["prefix"], s["block_table"], s["lens"], s["max_len"], s["out"],
                                 softcap=c["softcap"], workspace=kept["ws"], status=s["status"])
    else:
        g.gqa_attn_prefill_packed(s["q"], s["k"], s["v"], s["cu"], s["max_len"], s["out"],
                                  window=c["window"], softcap=c["softcap"], status=s["status"])


def run(state):
    op = state["case"]["op"]
    if own:
        _own(state)
    else:
        {"append": _plain_append, "decode": _plain_decode, "shared": _plain_shared,
         "prefill": _plain_prefill}[op](state)
    if op != "append":
        return [state["out"]]
    got = [state["q_out"], state["k_cache"], state["v_cache"]]
    return got if state["k_out"] is None else got + [state["k_out"]]


# ---------------------------------------------------------------- work

def work(case):
    c, lens = case, _lens(case)
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    T = sum(lens)
    if c["op"] == "append":
        # q, k, v read; q, k, v (and the keys once more, where wanted) written; cos and sin
        heads = 2 * H + 4 * Hkv + (Hkv if c["hi"] > 1 else 0)
        return {"bytes": T * (2 * heads * D + 4 * c["R"]), "flops": T * (H + Hkv) * D * 6}
    if c["op"] == "prefill":
        w = c["window"] or 1 << 60
        pairs = sum(n * (n + 1) // 2 if n <= w else w * (w + 1) // 2 + (n - w) * w for n in lens)
        return {"bytes": 2 * T * D * (2 * H + 2 * Hkv), "flops": 4 * H * D * pairs}
    rows = 2 * 2 * c["B"] * H * D
    if c["op"] == "shared":
        return {"bytes": rows + 4 * Hkv * D * (c["prefix"] + T),
                "flops": 4 * H * D * (c["B"] * c["prefix"] + T)}
    seen = sum(min(n, c["window"] or n) for n in lens)
    return {"bytes": rows + 4 * Hkv * D * seen, "flops": 4 * H * D * seen}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_row(c, q, k, v):
    """One query [H, D] over [Hkv, n, D], all float64."""
    if k.shape[1] == 0:
        return torch.zeros_like(q)
    z = torch.einsum("hgd,hnd->hgn", q.view(c["Hkv"], -1, c["D"]), k) / math.sqrt(c["D"])
    if c["softcap"] > 0:
        z = torch.tanh(z / c["softcap"]) * c["softcap"]
    return torch.einsum("hgn,hnd->hgd", torch.softmax(z, -1), v).reshape(q.shape)


def _positions(pool, pages, lo, hi):
    """Positions [lo, hi) of a row whose page numbers are given: [Hkv, hi - lo, D], float64."""
    size = pool.shape[2]
    a, b = lo // size, -(-hi // size)
    if hi <= lo:
        return pool.new_zeros(pool.shape[1], 0, pool.shape[3]).double()
    x = torch.cat([pool[int(p)] for p in pages[a:b].tolist()], 1)
    return x[:, lo - a * size:hi - a * size].double()


def _exact_rotate(x, p, table, w):
    """x [heads, D] at position p."""
    x = x.double()
    if w is not None:
        x = x * w.double() * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    r = table.shape[1]
    cs, sn = table[p, :, 0].double(), table[p, :, 1].double()
    y = x.clone()
    y[:, :r] = x[:, :r] * cs - x[:, r:2 * r] * sn
    y[:, r:2 * r] = x[:, r:2 * r] * cs + x[:, :r] * sn
    return y


def exact(case, seed):
    c, lens = case, _lens(case)
    s = prepare(case, seed)
    if c["op"] == "append":
        if sum(lens) > 12000:
            return None
        q, k = s["q_out"].double(), s["k_out"]
        k = None if k is None else k.double()
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        tables, t = s["block_table"].tolist(), 0
        for b, (first, n) in enumerate(zip(_starts(c), lens)):
            for p in range(first, first + n):
                q[t] = _exact_rotate(s["q"][t], p, s["table"], s["q_norm"])
                key = _exact_rotate(s["k"][t], p, s["table"], s["k_norm"])
                at = tables[b][p // c["page"]]
                kc[at, :, p % c["page"]] = key
                vc[at, :, p % c["page"]] = s["v"][t].double()
                if k is not None:
                    k[t] = key
                t += 1
        return [q, kc, vc] if k is None else [q, kc, vc, k]
    out = s["out"].double()
    if c["op"] == "prefill":
        for b, n in enumerate(lens):
            t0 = sum(lens[:b])
            i = torch.arange(n, device="cuda")
            hidden = i > i.view(-1, 1)
            if c["window"]:
                hidden = hidden | (i < i.view(-1, 1) - (c["window"] - 1))
            for h in range(c["H"] if n else 0):
                j = h // (c["H"] // c["Hkv"])
                q, k, v = (x[t0:t0 + n, m].double() for x, m in ((s["q"], h), (s["k"], j),
                                                                 (s["v"], j)))
                z = q @ k.T / math.sqrt(c["D"])
                if c["softcap"] > 0:
                    z = torch.tanh(z / c["softcap"]) * c["softcap"]
                out[t0:t0 + n, h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v
        return [out]
    for b, n in enumerate(lens):
        lo = max(0, n - c["window"]) if c.get("window") else 0
        k, v = (_positions(s[x], s["block_table"][b], lo, n) for x in ("k_cache", "v_cache"))
        if c["op"] == "shared":
            k, v = (torch.cat([_positions(s[x], s["prefix_table"], 0, c["prefix"]), y], 1)
                    for x, y in (("k_cache", k), ("v_cache", v)))
        out[b] = _exact_row(c, s["q"][b].double(), k, v)
    return [out]
