"""16-bit paged serving on the GPU against its formulas in 64 bits (paged_ref.py)."""
import pytest
import torch

import gqa_causal_attention_gb300 as g
from paged_ref import (Cache, attend, attend_tol, check, dev, gen, i32, normal, rope, rotate,
                       rotate_tol, rows, status)

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def causal(n, window=0):
    i = torch.arange(n, device=dev())
    seen = i <= i[:, None]
    return seen & (i > i[:, None] - window) if window else seen


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("t,H,Hkv,D,R,page,norm,layout,inplace,lens,starts", [
    (BF, 8, 2, 128, 128, 16, False, "slice", False, [1, 1, 1], [0, 17, 300]),
    (FP, 32, 8, 128, 64, 64, True, "slice", False, [5, 0, 70, 1], [0, 9, 3, 64]),
    (BF, 3, 3, 64, 64, 32, True, "heads", True, [33, 31], [31, 1]),
    (FP, 14, 2, 80, 40, 16, True, "whole", True, [0, 19, 0, 0, 4], [5, 0, 2, 2, 60]),
    (BF, 5, 1, 96, 96, 128, False, "heads", False, [130], [127]),
    (FP, 2, 1, 16, 16, 16, True, "slice", True, [40, 2], [0, 0]),
    (BF, 4, 4, 40, 12, 1024, False, "whole", False, [3, 3], [1022, 5]),
    (FP, 64, 8, 128, 128, 16, True, "slice", False, [900, 300], [11, 0]),   # many warps: groups
    (BF, 7, 1, 128, 128, 16, False, "whole", False, [600] * 9, list(range(9))),
])
def test_append(t, H, Hkv, D, R, page, norm, layout, inplace, lens, starts):
    gn = gen(H * D + page)
    B, pad = len(lens), 3
    cu = [sum(lens[:b]) for b in range(B + 1)]
    T = cu[-1] + pad
    q, k, v = (rows(gn, T, h, D, t, layout) for h in (H, Hkv, Hkv))
    total = [s + n for s, n in zip(starts, lens)]
    c = Cache(gn, sum(-(-n // page) for n in total) + 3, Hkv, page, D, t, fused=D == 64)
    table = c.table(total)
    rp, tab, tab3 = rope(D, R, max(total) + 1)
    qn, kn = (1 + 0.2 * normal(gn, (D,)), 1 + 0.2 * normal(gn, (D,))) if norm else (None, None)
    raw_q, raw_k, raw_v = q.clone(), k.clone(), v.clone()
    q_out = q if inplace else torch.full_like(q, 7.0)
    k_out = k if inplace else torch.full_like(k, 7.0)
    st = status()
    g.kv_cache_append_paged(k, v, c.k, c.v, table, i32(starts), max(total) - 1, rp, tab, kn, 1e-5,
                            cu_seqlens=i32(cu), q=q, q_out=q_out, q_norm_w=qn, k_out=k_out,
                            status=st)
    assert st.item() == 0
    used = 0
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pos = torch.arange(starts[b], starts[b] + n, device=dev())
        at = slice(cu[b], cu[b + 1])
        yq, mq = rotate(raw_q[at], pos, tab3, qn, 1e-5)
        yk, mk = rotate(raw_k[at], pos, tab3, kn, 1e-5)
        check(q_out[at], yq, rotate_tol(yq, mq, t), "q")
        check(k_out[at], yk, rotate_tol(yk, mk, t), "k")
        row = table[b].tolist()
        assert torch.equal(c.read(c.k, row, total[b])[starts[b]:], k_out[at])
        assert torch.equal(c.read(c.v, row, total[b])[starts[b]:], raw_v[at])
        used += n * Hkv * D
    # nothing else of the pools was written, nor the rows behind the last sequence
    assert int(torch.isfinite(c.k).sum()) == used and int(torch.isfinite(c.v).sum()) == used
    tail = slice(cu[-1], None)
    want = raw_q if inplace else torch.full_like(raw_q, 7.0)
    assert torch.equal(q_out[tail], want[tail])


def test_append_one_token_each_without_rope_or_queries():
    gn, t = gen(5), BF
    B, Hkv, D, page = 70, 2, 64, 16
    k, v = rows(gn, B, Hkv, D, t), rows(gn, B, Hkv, D, t)
    start = [(7 * b) % 40 for b in range(B)]
    c = Cache(gn, 3 * B, Hkv, page, D, t)
    table = c.table([s + 1 for s in start])
    g.kv_cache_append_paged(k, v, c.k, c.v, table, i32(start), 39)
    for b in range(B):
        assert torch.equal(c.read(c.k, table[b].tolist(), start[b] + 1)[-1], k[b])
        assert torch.equal(c.read(c.v, table[b].tolist(), start[b] + 1)[-1], v[b])
    assert int(torch.isfinite(c.k).sum()) == B * Hkv * D


def test_append_skips_what_breaks_a_rule():
    gn, t = gen(6), FP
    H, Hkv, D, page = 4, 2, 32, 16
    lens = [2, 2, 2, 2]
    cu = [0, 2, 4, 6, 8]
    k, v, q = rows(gn, 8, Hkv, D, t), rows(gn, 8, Hkv, D, t), rows(gn, 8, H, D, t)

    def run(starts, table, cu, max_pos=31):
        c = Cache(gn, 12, Hkv, page, D, t)
        st, q_out = status(), torch.full_like(q, 7.0)
        g.kv_cache_append_paged(k, v, c.k, c.v, table, i32(starts), max_pos, cu_seqlens=i32(cu),
                                q=q, q_out=q_out, status=st)
        done = [bool((q_out[i] != 7.0).any()) for i in range(8)]
        return st.item(), done, int(torch.isfinite(c.k).sum()) // (Hkv * D)

    table = torch.arange(8, dtype=torch.int32, device=dev()).view(4, 2)
    assert run([0, 5, 15, 30], table, cu) == (0, [True] * 8, 8)
    s, done, n = run([0, -1, 31, 0], table, cu)          # before 0; past max_pos with its second token
    assert s == g.DEV_POSITION and done == [True, True] + [False] * 4 + [True, True] and n == 4
    bad = table.clone()
    bad[1, 0], bad[2, 1] = 12, -5                        # of 12 pages; needed by row 2's second token
    s, done, n = run([0, 0, 15, 0], bad, cu)
    assert s == g.DEV_PAGE and done == [True, True, False, False, True, False, True, True] and n == 5
    s, done, n = run([0, 0, 0, 0], table, [0, 2, 4, 9, 9])   # past the rows
    assert s == g.DEV_LENGTH and done[:4] == [True] * 4 and not any(done[4:])


# ---------------------------------------------------------------- decode

def decode(t, H, Hkv, D, page, lens, window=0, softcap=0.0, scale=0.0, kscale=1.0, seed=1, fused=False,
           layout="slice", max_len=None, keys=None):
    gn = gen(seed)
    c = Cache(gn, sum(-(-n // page) for n in lens) + 2, Hkv, page, D, t, fused)
    table = c.table(lens, unused=-77)
    kv = c.fill(gn, table, lens, kscale)
    if keys:
        for b in range(len(lens)):
            kv[b] = (keys(kv[b][0]), kv[b][1])
            c.put(table[b].tolist(), 0, *kv[b])
    if window:                                   # pages before the window may be anything, too
        for b, n in enumerate(lens):
            table[b, :max(0, n - window) // page] = 10 ** 6
    q = rows(gn, len(lens), H, D, t, layout)
    out = torch.full((len(lens), H, D), 7.0, dtype=t, device=dev())
    st = status()
    call = lambda o: g.gqa_attn_decode_paged(q, c.k, c.v, table, i32(lens), max_len or max(lens), o,  # noqa: E731
                                             window=window, softcap=softcap, scale=scale, status=st)
    call(out)
    again = torch.empty_like(out)
    call(again)
    assert st.item() == 0 and torch.equal(out, again)
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.equal(out[b], torch.zeros_like(out[b]))
            continue
        i = torch.arange(n, device=dev())
        seen = (i >= n - window)[None] if window else torch.ones(1, n, dtype=torch.bool, device=dev())
        o, vabs, unsure = attend(q[b][None], *kv[b], seen, softcap, scale)
        check(out[b], o[0], attend_tol(o, vabs, unsure, t, False)[0], f"row {b} of length {n}")


@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("H,Hkv,D,page,lens,window,softcap", [
    (8, 2, 128, 16, [1], 0, 0.0),
    (32, 8, 128, 16, [500], 0, 0.0),                         # one wide block a unit
    (4, 4, 64, 32, [1, 15, 16, 17, 31, 33, 0], 0, 0.0),
    (14, 2, 64, 32, [1000, 0, 3, 777, 1], 100, 30.0),
    (16, 1, 128, 64, [129, 64, 0], 64, 0.0),                 # two groups of 8 heads
    (9, 1, 96, 128, [300, 5], 0, 50.0),                      # nine heads: groups of 8 and 1
    (5, 5, 16, 16, [40, 1, 2], 7, 0.0),
    (20, 2, 80, 256, [257, 600], 0, 0.0),
    (32, 8, 128, 16, [2000, 37, 0, 5000], 0, 0.0),           # shared out over blocks
    (8, 8, 128, 64, [3000] * 3 + [1], 2500, 30.0),
    (16, 4, 64, 1024, [1500 + 97 * b for b in range(40)], 0, 0.0),
    (2, 1, 40, 16, [0, 0, 4100, 0], 0, 0.0),
    (8, 1, 128, 16, [100] * 300, 0, 0.0),
])
def test_decode(t, H, Hkv, D, page, lens, window, softcap):
    decode(t, H, Hkv, D, page, lens, window, softcap, seed=sum(lens) + D, fused=Hkv == 4,
           layout=("slice", "heads", "whole")[len(lens) % 3], max_len=max(lens) + len(lens) % 2)


@pytest.mark.parametrize("H,Hkv,D,page,lens,window", [
    (32, 8, 128, 16, [b % 30 for b in range(90)] + [5000, 4001, 0, 2], 0),   # shares of many starts
    (16, 4, 64, 32, [9000] + [b % 19 for b in range(200)], 0),
    (8, 1, 128, 64, [1] * 500 + [2500], 0),                  # more starts than tiles
    (6, 2, 96, 16, [0, 0, 2300] + [700, 16] * 30, 2200),
    (32, 8, 128, 16, [31 * b for b in range(64)], 0),        # a block a unit: more units than places
])
def test_decode_short_rows_beside_long_ones(H, Hkv, D, page, lens, window):
    decode(BF, H, Hkv, D, page, lens, window, seed=len(lens))


@pytest.mark.parametrize("t", [BF, FP])
def test_decode_where_the_reference_moves(t):
    """Keys that grow along the row: every tile holds a new maximum, by far more than 2^8."""
    ramp = lambda k: (k.float() * torch.linspace(0.1, 20, k.shape[0], device=dev())[:, None, None]).to(k.dtype)  # noqa: E731
    decode(t, 8, 2, 64, 16, [700, 3000], keys=ramp)
    decode(t, 8, 2, 128, 16, [90], scale=2.0, keys=ramp)


def test_decode_bad_lengths_and_pages():
    gn, t = gen(3), BF
    for lens_max in (64, 3000):                  # one block a unit; shared out
        c = Cache(gn, 400, 2, 16, 64, t)
        table = c.table([lens_max, lens_max])
        c.fill(gn, table, [lens_max, lens_max])
        q = rows(gn, 4, 4, 64, t)
        four = torch.cat([table, table])
        out, st = torch.full((4, 4, 64), 7.0, dtype=t, device=dev()), status()
        g.gqa_attn_decode_paged(q, c.k, c.v, four, i32([5, -1, lens_max + 1, 9]), lens_max, out,
                                status=st)
        assert st.item() == g.DEV_LENGTH
        assert torch.equal(out[1:3], torch.full_like(out[1:3], 7.0)) and (out[[0, 3]] != 7.0).any()
        want, st2 = torch.empty(2, 4, 64, dtype=t, device=dev()), status()
        g.gqa_attn_decode_paged(q[::3].contiguous(), c.k, c.v, table, i32([5, 9]), lens_max, want,
                                status=st2)
        assert torch.equal(out[[0, 3]], want) and st2.item() == 0
        four[0, 0] = 400                         # past the pool: reported, the other rows stand
        g.gqa_attn_decode_paged(q, c.k, c.v, four, i32([5, 0, 0, 9]), lens_max, out, status=st2)
        assert st2.item() == g.DEV_PAGE and torch.equal(out[3], want[1])


# ---------------------------------------------------------------- shared prefix

def shared(t, H, Hkv, D, page, prefix, lens, softcap=0.0, kscale=1.0, seed=1, keys=None):
    gn = gen(seed)
    B = len(lens)
    c = Cache(gn, -(-prefix // page) + sum(-(-n // page) for n in lens) + 2, Hkv, page, D, t)
    ptab = c.table([prefix])[0].contiguous()
    (pk, pv), = c.fill(gn, ptab[None], [prefix], kscale)
    if keys:
        pk = keys(pk)
        c.put(ptab.tolist(), 0, pk, pv)
    table = c.table(lens)
    kv = c.fill(gn, table, lens, kscale)
    q = rows(gn, B, H, D, t)
    out, again, st = torch.empty(B, H, D, dtype=t, device=dev()), torch.empty(B, H, D, dtype=t, device=dev()), status()
    for o in (out, again):
        g.gqa_attn_decode_shared(q, c.k, c.v, ptab, prefix, table, i32(lens), max(lens), o,
                                 softcap=softcap, status=st)
    assert st.item() == 0 and torch.equal(out, again)
    for b, n in enumerate(lens):
        k, v = torch.cat([pk, kv[b][0]]), torch.cat([pv, kv[b][1]])
        seen = torch.ones(1, prefix + n, dtype=torch.bool, device=dev())
        o, vabs, unsure = attend(q[b][None], k, v, seen, softcap)
        check(out[b], o[0], attend_tol(o, vabs, unsure, t, True)[0], f"row {b}")


@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("H,Hkv,D,page,prefix,lens,softcap", [
    (8, 2, 128, 16, 1, [0], 0.0),                            # read with the rows' own
    (28, 4, 64, 32, 2001, [0, 40, 7], 0.0),
    (16, 1, 80, 64, 130, [3, 0, 1000], 30.0),
    (16, 8, 128, 16, 4000, [1, 0, 77, 300, 5, 9, 33, 64, 2, 3], 0.0),   # tensor cores: one tile
    (64, 8, 128, 64, 3001, [b % 5 for b in range(16)], 30.0),
    (8, 8, 64, 128, 9000, [10 * b for b in range(40)], 0.0),
    (32, 8, 128, 16, 2111, [b * b % 700 for b in range(60)], 0.0),      # two tiles
    (20, 4, 96, 256, 4500, [2000, 0, 1] * 14, 0.0),          # five heads a kv head: 25 rows a tile
    (128, 1, 64, 32, 40000, [0, 5, 9, 100] * 5, 0.0),        # one row a tile
    (7, 7, 32, 16, 640, [600] * 400, 0.0),
])
def test_shared(t, H, Hkv, D, page, prefix, lens, softcap):
    shared(t, H, Hkv, D, page, prefix, lens, softcap, seed=prefix)


@pytest.mark.parametrize("H,Hkv,D,page,prefix,lens", [
    (32, 8, 128, 16, 3500, [b % 20 for b in range(44)] + [3001]),        # shares of many starts
    (12, 4, 64, 64, 9001, [0] * 50 + [4200] + [1, 17] * 20),
    (32, 8, 128, 32, 2500, [0] * 60),                        # nothing but the prefix
])
def test_shared_short_rows_beside_long_ones(H, Hkv, D, page, prefix, lens):
    shared(BF, H, Hkv, D, page, prefix, lens, seed=prefix)


@pytest.mark.parametrize("t", [BF, FP])
def test_shared_where_the_reference_moves(t):
    ramp = lambda k: (k.float() * torch.linspace(0.1, 12, k.shape[0], device=dev())[:, None, None]).to(k.dtype)  # noqa: E731
    shared(t, 16, 4, 128, 16, 6000, [3] * 20, keys=ramp)


def test_shared_bad_page_and_length():
    gn, t, B = gen(4), BF, 20
    c = Cache(gn, 600, 8, 16, 128, t)
    ptab = c.table([4000])[0].contiguous()
    c.fill(gn, ptab[None], [4000])
    table = c.table([3] * B)
    c.fill(gn, table, [3] * B)
    q, st = rows(gn, B, 16, 128, t), status()
    out = torch.full((B, 16, 128), 7.0, dtype=t, device=dev())
    lens = [3] * B
    lens[4] = 4
    g.gqa_attn_decode_shared(q, c.k, c.v, ptab, 4000, table, i32(lens), 3, out, status=st)
    assert st.item() == g.DEV_LENGTH and torch.equal(out[4], torch.full_like(out[4], 7.0))
    assert (out[5] != 7.0).any()
    ptab[17], st2 = 600, status()
    g.gqa_attn_decode_shared(q, c.k, c.v, ptab, 4000, table, i32([3] * B), 3, out, status=st2)
    assert st2.item() == g.DEV_PAGE


# ---------------------------------------------------------------- packed prompts

def prefill(t, H, Hkv, D, lens, window=0, softcap=0.0, scale=0.0, seed=1, layout="slice", pad=2, keys=None,
            some_rows=None):
    gn = gen(seed)
    B = len(lens)
    cu = [sum(lens[:b]) + 1 for b in range(B + 1)]           # row 0 belongs to no sequence
    T = cu[-1] + pad
    q, k, v = (rows(gn, T, h, D, t, layout) for h in (H, Hkv, Hkv))
    if keys:
        k.copy_(keys(k))
    for x in (q, k, v):                                      # rows of no sequence
        x[0] = float("nan")
        x[cu[-1]:] = float("inf")
    out = torch.full((T, H, D), 7.0, dtype=t, device=dev())
    st = status()
    g.gqa_attn_prefill_packed(q, k, v, i32(cu), max(lens), out, window=window, softcap=softcap,
                              scale=scale, status=st)
    assert st.item() == 0
    assert torch.equal(out[0], torch.full_like(out[0], 7.0))
    assert torch.equal(out[cu[-1]:], torch.full_like(out[cu[-1]:], 7.0))
    again = torch.empty_like(out)
    g.gqa_attn_prefill_packed(q, k, v, i32(cu), max(lens), again, window=window, softcap=softcap,
                              scale=scale, status=st)
    assert torch.equal(out[1:cu[-1]], again[1:cu[-1]])
    for b, n in enumerate(lens):
        if n == 0:
            continue
        at = slice(cu[b], cu[b + 1])
        pick = slice(None) if n <= 2600 else torch.arange(0, n, 97, device=dev())
        o, vabs, unsure = attend(q[at][pick], k[at], v[at], causal(n, window)[pick], softcap, scale)
        check(out[at][pick], o, attend_tol(o, vabs, unsure, t, True), f"sequence {b} of {n}")


@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("H,Hkv,D,lens,window,softcap", [
    (8, 2, 128, [1], 0, 0.0),
    (4, 4, 64, [1, 0, 2, 127, 128, 129], 0, 0.0),            # MHA: 128 tokens a tile
    (32, 8, 128, [77, 300, 0, 0, 5], 0, 0.0),
    (14, 2, 64, [63, 64, 65, 400], 50, 30.0),                # seven heads: 18 tokens a tile
    (5, 1, 80, [260, 1], 0, 0.0),
    (24, 8, 96, [500, 31], 128, 0.0),
    (64, 1, 32, [200, 3, 9], 0, 50.0),                       # two tokens a tile
    (128, 1, 16, [70, 1], 1, 0.0),                           # one token a tile; its own key only
    (6, 3, 40, [129] * 12, 129, 0.0),
    (8, 8, 128, [2100, 900], 0, 0.0),
    (8, 1, 128, [2300, 1111], 700, 0.0),
    (16, 4, 64, [5000], 0, 0.0),                             # several rounds of units
    (32, 8, 128, [4100], 1000, 30.0),
    (4, 2, 64, [(37 * b) % 190 for b in range(150)], 0, 0.0),   # more sequences than lanes
])
def test_prefill(t, H, Hkv, D, lens, window, softcap):
    prefill(t, H, Hkv, D, lens, window, softcap, seed=sum(lens),
            layout=("slice", "heads", "whole")[len(lens) % 3])


@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("lens,window", [([900], 0), ([700, 300], 200)])
def test_prefill_where_the_reference_moves(t, lens, window):
    ramp = lambda k: (k.float() * torch.linspace(0.1, 20, k.shape[0], device=dev())[:, None, None]).to(k.dtype)  # noqa: E731
    prefill(t, 8, 2, 128, lens, window, keys=ramp)
    prefill(t, 4, 4, 64, lens, window, scale=1.5, keys=ramp)


def test_prefill_bad_sequences():
    gn, t = gen(8), BF
    q, k, v = (rows(gn, 300, h, 64, t) for h in (4, 2, 2))

    def run(cu, max_len):
        out, st = torch.full((300, 4, 64), 7.0, dtype=t, device=dev()), status()
        g.gqa_attn_prefill_packed(q, k, v, i32(cu), max_len, out, status=st)
        return out, st.item()

    good, st = run([0, 100, 150, 300], 150)
    assert st == 0 and not (good == 7.0).all(-1).any()
    out, st = run([0, 100, 150, 300], 149)       # the last is longer than it may be
    assert st == g.DEV_LENGTH and torch.equal(out[:150], good[:150]) and (out[150:] == 7.0).all()
    out, st = run([0, 100, 150, 301], 300)       # past the rows
    assert st == g.DEV_LENGTH and torch.equal(out[:150], good[:150]) and (out[150:] == 7.0).all()
    out, st = run([0, 100, 90, 300], 300)        # backwards
    assert st == g.DEV_LENGTH and torch.equal(out[:100], good[:100]) and not (out[150:] == 7.0).all()
    out, st = run([0, 100], 0)
    assert st == g.DEV_LENGTH and (out == 7.0).all()


# ---------------------------------------------------------------- corners

def test_caps_of_next_to_nothing_and_scores_past_the_cap():
    prefill(BF, 4, 2, 64, [200], softcap=1e-30)
    prefill(FP, 4, 2, 64, [200, 150], softcap=2.0, scale=3.0)
    decode(FP, 4, 2, 64, 16, [200, 1500], softcap=1e-30)
    decode(BF, 4, 2, 64, 16, [200, 1500], softcap=2.0, scale=3.0)


def test_one_row_of_a_wider_tensor():
    """Axes of one element: their strides are not read."""
    gn, t, H, D = gen(23), BF, 4, 64
    wide = normal(gn, (9, H, 5, D), t)
    q = wide[4:5, :, 2]                          # [1, H, D], heads 5 D apart
    k, v = (normal(gn, (1, 1, D), t).expand(1, 1, D) for _ in range(2))
    out = torch.empty(1, H, D, dtype=t, device=dev())
    g.gqa_attn_prefill_packed(q, k, v, i32([0, 1]), 1, out)
    assert torch.equal(out, v.expand(1, H, D).contiguous())
    c = Cache(gn, 3, 1, 16, D, t)
    table = c.table([1])
    g.kv_cache_append_paged(k, v, c.k, c.v, table, i32([0]), 0, q=q, q_out=out)
    assert torch.equal(out, q.contiguous())
    g.gqa_attn_decode_paged(q, c.k, c.v, table, i32([1]), 1, out)
    assert torch.equal(out, v.expand(1, H, D).contiguous())


def test_values_that_are_not_finite_stay_with_the_rows_that_see_them():
    """A NaN in one row's cache or query, or in one sequence, leaves every other row as it was."""
    gn, t = gen(29), FP
    lens = [100, 3000, 2000]
    c = Cache(gn, 400, 2, 16, 64, t)
    table = c.table(lens)
    c.fill(gn, table, lens)
    q = rows(gn, 3, 8, 64, t)
    want, got = (torch.empty(3, 8, 64, dtype=t, device=dev()) for _ in range(2))
    call = lambda o: g.gqa_attn_decode_paged(q, c.k, c.v, table, i32(lens), max(lens), o)  # noqa: E731
    call(want)
    c.v[table[1, 7], 0, 3, 5] = float("inf")
    q[2, 6, 1] = float("nan")
    call(got)
    assert not torch.isfinite(got[1, :4, 5]).any() and torch.isnan(got[2, 6]).all()
    got[1, :4, 5], got[2, 6] = want[1, :4, 5], want[2, 6]
    assert torch.equal(got, want)
    q, k, v = rows(gn, 400, 8, 64, t), rows(gn, 400, 2, 64, t), rows(gn, 400, 2, 64, t)
    want, got = (torch.empty(400, 8, 64, dtype=t, device=dev()) for _ in range(2))
    cu = i32([0, 130, 260, 400])
    g.gqa_attn_prefill_packed(q, k, v, cu, 140, want)
    k[135], v[140, 1, 2], q[300, 3, 3] = float("nan"), float("inf"), float("nan")
    g.gqa_attn_prefill_packed(q, k, v, cu, 140, got)
    assert torch.equal(got[:130], want[:130]) and torch.isnan(got[135:260]).all()
    assert torch.isnan(got[300, 3]).all()
    got[300, 3] = want[300, 3]
    assert torch.equal(got[260:], want[260:])
