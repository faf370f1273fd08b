"""16-bit paged serving at its edges, against 64 bits: caps far above the scores, weights far below a row's
largest, rows that see mostly their own positions behind a shared prefix, many short prompts.

The bounds here are closer than paged_ref.py's: a score's error counts by the score, not by the cap, and an
fp16 weight's by its own size and 2^-37 of its row's largest.
"""
import pytest
import torch

import gqa_causal_attention_gb300 as g
from paged_ref import Cache, U, attend, attend_tol, check, dev, gen, half_step, i32, normal, rows, status

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def close_tol(q, k, v, seen, softcap, scale, t, parts=False):
    """Exact output of q [Lq, H, D] over k, v [n, Hkv, D], and how far a result may be from it.

    Scores: D + 4 roundings of the product's magnitudes (tanh only shrinks them). Cap: below 0.4 tanh's
    series, cut off at 9.3e-7 = 16 u of the value, and 6 roundings; above it 2^x (4 u), a reciprocal (2 u),
    and 1 - 2 / (e + 1), which is 0.38 at least: 14 u. Then a subtraction and 2^x: 2 u of the score, 8 u.
    Weights: two 16-bit parts leave half a step squared (half a step where P is one part: `parts`), in fp16
    half of its smallest step too, 2^-25 with the row's largest at 2^12 at least (2^7: `parts`). Sums: n u."""
    n, D = k.shape[0], q.shape[-1]
    out, vabs, _ = attend(q, k, v, seen, softcap, scale)
    scale = D ** -0.5 if not scale else scale
    G = q.shape[1] // k.shape[1]
    qq = q.double().permute(1, 0, 2)                          # [H, Lq, D]
    kk = k.double().permute(1, 2, 0).repeat_interleave(G, 0)  # [H, D, n]
    s, mag = scale * (qq @ kk), scale * (qq.abs() @ kk.abs())
    if softcap > 0:
        s = softcap * torch.tanh(s / softcap)
    unsure = torch.where(seen, (D + 4) * U * mag + 26 * U * s.abs() + 8 * U, 0.0).amax(-1).T[..., None]
    w = half_step(t) if parts else half_step(t) ** 2
    least = n * 2.0 ** (-32 if parts else -37) * v.double().abs().max() if t == FP else 0.0
    tol = (half_step(t) * (1 + 2.0 ** -6) * out.abs() + (w * (1 + 2.0 ** -6) + 2 * unsure + n * U) * vabs
           + least + (2.0 ** -24 if t == FP else 0.0))
    return out, tol


def all_seen(n):
    return torch.ones(1, n, dtype=torch.bool, device=dev())


# ---------------------------------------------------------------- softcap

@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("cap", [30.0, 1e3, 1e4, 1e6, 1e8, 1e38])
def test_decode_with_caps_far_above_the_scores(t, cap):
    """A cap that no score comes near changes next to nothing, whatever its size."""
    for D, lens, n_max in ((64, [40, 1, 150], 150), (128, [300, 17], 5000)):
        gn = gen(int(cap) % 1000 + D)
        c = Cache(gn, 60, 2, 16, D, t)
        table = c.table(lens, extra=400)
        kv = c.fill(gn, table, lens, 2.0)
        q = rows(gn, len(lens), 8, D, t)
        out, st = torch.empty(len(lens), 8, D, dtype=t, device=dev()), status()
        g.gqa_attn_decode_paged(q, c.k, c.v, table, i32(lens), n_max, out, softcap=cap, status=st)
        assert st.item() == 0
        for b, n in enumerate(lens):
            want, tol = close_tol(q[b][None], *kv[b], all_seen(n), cap, 0.0, t)
            check(out[b], want[0], tol[0], f"cap {cap:g}, row {b} of {n}")


@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("cap", [1e4, 1e8])
def test_shared_with_caps_far_above_the_scores(t, cap):
    """The prefix's part and a row's own are capped alike: by the tensor cores (many rows) and by the decode."""
    H, Hkv, D, page, lens = 16, 8, 128, 16, [40, 0, 13, 5] * 5
    for prefix, B, parts in ((3000, 20, True), (90, 3, False)):
        gn = gen(prefix)
        c = Cache(gn, -(-prefix // page) + 100, Hkv, page, D, t)
        ptab = c.table([prefix])[0].contiguous()
        (pk, pv), = c.fill(gn, ptab[None], [prefix], 2.0)
        table = c.table(lens[:B])
        kv = c.fill(gn, table, lens[:B], 2.0)
        q = rows(gn, B, H, D, t)
        out, st = torch.empty(B, H, D, dtype=t, device=dev()), status()
        g.gqa_attn_decode_shared(q, c.k, c.v, ptab, prefix, table, i32(lens[:B]), 40, out, softcap=cap,
                                 status=st)
        assert st.item() == 0
        for b in range(B):
            k, v = torch.cat([pk, kv[b][0]]), torch.cat([pv, kv[b][1]])
            want, tol = close_tol(q[b][None], k, v, all_seen(k.shape[0]), cap, 0.0, t, parts)
            check(out[b], want[0], tol[0], f"cap {cap:g}, prefix {prefix}, row {b}")


# ---------------------------------------------------------------- prompts with scores past the cap

@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("cap", [1e4, 1e6])
def test_prefill_where_scores_past_the_cap_stand_beside_small_ones(t, cap):
    """Every 16th query is large enough for its scores to pass the cap; the others' stay exact."""
    gn, n, H, Hkv, D = gen(int(cap)), 200, 4, 2, 64
    q, k, v = rows(gn, n, H, D, t), rows(gn, n, Hkv, D, t), rows(gn, n, Hkv, D, t)
    q[::16] *= 1e4 if t == FP else cap
    out, st = torch.empty(n, H, D, dtype=t, device=dev()), status()
    scale = 0.25 if t == BF else 0.25 * cap / 1e4
    k /= max(1.0, 8 * scale)
    g.gqa_attn_prefill_packed(q, k, v, i32([0, n]), n, out, softcap=cap, scale=scale, status=st)
    assert st.item() == 0
    i = torch.arange(n, device=dev())
    want, tol = close_tol(q, k, v, i <= i[:, None], cap, scale, t, True)
    small = i % 16 != 0
    check(out[small], want[small], tol[small], f"cap {cap:g}")


# ---------------------------------------------------------------- the smallest caps

@pytest.mark.parametrize("cap", [1e-38, 1e-39, 1e-45])
def test_caps_below_the_smallest_normal_number(cap):
    """2 scale / cap leaves fp32: a score of 0 is still 0 after the cap, and the weights are equal."""
    t, n, H, Hkv, D = BF, 40, 4, 2, 64
    gn = gen(7)
    q = torch.zeros(n, H, D, dtype=t, device=dev())
    k, v = rows(gn, n, Hkv, D, t), rows(gn, n, Hkv, D, t)
    c = Cache(gn, 8, Hkv, 16, D, t)
    table = c.table([n])
    c.put(table[0].tolist(), 0, k, v)
    one, out, st = torch.empty(1, H, D, dtype=t, device=dev()), torch.empty(n, H, D, dtype=t, device=dev()), status()
    g.gqa_attn_decode_paged(q[:1], c.k, c.v, table, i32([n]), n, one, softcap=cap, scale=1.0, status=st)
    g.gqa_attn_prefill_packed(q, k, v, i32([0, n]), n, out, softcap=cap, scale=1.0, status=st)
    assert st.item() == 0
    i = torch.arange(n, device=dev())
    want, tol = close_tol(q, k, v, i <= i[:, None], 0.0, 1.0, t, True)
    check(out, want, tol)
    check(one, want[-1:], tol[-1:])


# ---------------------------------------------------------------- small weights

@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("D,lens,prefix", [(64, [2000], 0), (128, [500, 7000], 0), (64, [30, 100], 300)])
def test_small_weights_beside_a_key_whose_value_is_zero(t, D, lens, prefix):
    """One key in 16 has nearly all of the weight and a value of zero: what is left of the output are keys
    of 2^-24 .. 2^-27 of its weight."""
    gn, H, Hkv, page = gen(D + prefix), 8, 2, 16
    c = Cache(gn, sum(-(-n // page) for n in lens) + -(-prefix // page) + 4, Hkv, page, D, t)

    def make(n):
        k, v = torch.zeros(n, Hkv, D, device=dev()), 1000 + 100 * normal(gn, (n, Hkv, D))
        first = torch.arange(n, device=dev()) % 16 == 3
        k[..., 0] = torch.where(first, 0.0, -24 * 0.6931 - torch.rand(n, generator=gn, device=dev()) * 2)[:, None]
        v[first] = 0
        return k.to(t), v.to(t)

    q = torch.zeros(len(lens), H, D, dtype=t, device=dev())
    q[..., 0] = 1
    table = c.table(lens)
    kv = [make(n) for n in lens]
    for b in range(len(lens)):
        c.put(table[b].tolist(), 0, *kv[b])
    out, st = torch.empty_like(q), status()
    if prefix:
        ptab = c.table([prefix])[0].contiguous()
        pre = make(prefix)
        c.put(ptab.tolist(), 0, *pre)
        kv = [(torch.cat([pre[0], k]), torch.cat([pre[1], v])) for k, v in kv]
        g.gqa_attn_decode_shared(q, c.k, c.v, ptab, prefix, table, i32(lens), max(lens), out, scale=1.0, status=st)
    else:
        g.gqa_attn_decode_paged(q, c.k, c.v, table, i32(lens), max(lens), out, scale=1.0, status=st)
    assert st.item() == 0
    for b in range(len(lens)):
        want, tol = close_tol(q[b][None], *kv[b], all_seen(kv[b][0].shape[0]), 0.0, 1.0, t)
        check(out[b], want[0], tol[0], f"row {b}")


# ---------------------------------------------------------------- shared prefixes

@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("H,Hkv,D,page,prefix,lens", [
    (28, 4, 64, 32, 2001, [0, 40, 7, 1]),                     # read with each row's own: P in two parts
    (16, 8, 128, 16, 1500, [3, 0, 1, 200]),
    (32, 8, 128, 16, 2560, [b % 6 for b in range(24)]),       # tensor cores: P in one
    (8, 8, 64, 128, 9000, [b % 3 for b in range(40)]),
])
def test_a_rows_own_positions_weigh_beside_a_long_prefix(t, H, Hkv, D, page, prefix, lens):
    """Own keys lie along their row's query, so that one of them outweighs the whole prefix; lost, or
    counted twice, it would change the output by its own size. By the shared call and, with the
    prefix's pages in every row's table, by the plain one."""
    gn, B = gen(prefix + D), len(lens)
    per = -(-prefix // page)
    c = Cache(gn, per + sum(-(-n // page) for n in lens) + 2, Hkv, page, D, t)
    ptab = c.table([prefix], extra=0)[0].contiguous()
    (pk, pv), = c.fill(gn, ptab[None], [prefix])
    q, own = rows(gn, B, H, D, t), c.table(lens)
    kv = []
    for b, n in enumerate(lens):
        k, v = normal(gn, (n, Hkv, D)), normal(gn, (n, Hkv, D), t)
        lead = q[b].float().view(Hkv, -1, D)[:, 0]            # the kv head's first query: |q|^2 / sqrt(D) ~ sqrt(D)
        k = (lead * (1.3 if D <= 64 else 1.0) + 0.3 * k).to(t)
        c.put(own[b].tolist(), 0, k, v)
        kv.append((torch.cat([pk, k]), torch.cat([pv, v])))
    st = status()
    a, p = (torch.empty(B, H, D, dtype=t, device=dev()) for _ in range(2))
    g.gqa_attn_decode_shared(q, c.k, c.v, ptab, prefix, own, i32(lens), max(lens), a, status=st)
    # own positions begin at a page of their own: the plain call needs the prefix to end with one
    whole = prefix % page == 0
    if whole:
        table = torch.cat([ptab.expand(B, -1), own], 1).contiguous()
        g.gqa_attn_decode_paged(q, c.k, c.v, table, i32([prefix + n for n in lens]), prefix + max(lens), p, status=st)
    assert st.item() == 0
    parts = 4 * B * prefix * Hkv * D > 64 << 20
    for b, n in enumerate(lens):
        args = (q[b][None], *kv[b], all_seen(prefix + n), 0.0, 0.0, t)
        want, tol = close_tol(*args, parts)
        check(a[b], want[0], tol[0], f"row {b}")
        if n:                                                 # what the test is for: losing one shows
            less, _, _ = attend(q[b][None], kv[b][0][:-1], kv[b][1][:-1], all_seen(prefix + n - 1))
            assert ((less - want).abs() / tol).max() > 4
        if whole:
            want, tol = close_tol(*args)
            check(p[b], want[0], tol[0], f"row {b}, its own table")


# ---------------------------------------------------------------- many prompts

def prompts(gn, lens, H, Hkv, D, t):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return i32(cu), cu, [rows(gn, cu[-1] + 1, h, D, t, "whole") for h in (H, Hkv, Hkv)]


@pytest.mark.parametrize("t,H,Hkv,D,lens", [
    (BF, 4, 2, 64, [(7 * b) % 23 for b in range(3000)]),
    (FP, 4, 1, 128, [(11 * b) % 9 for b in range(1500)] + [1300] + [0] * 40 + [3] * 60 + [700]),
    (FP, 8, 8, 32, [0] * 1100 + [400, 0, 1] + [0] * 1000),
    (BF, 8, 1, 64, [500] + [3] * 63),                         # the last number that is sorted,
    (BF, 8, 1, 64, [3] * 63 + [500, 2]),                      # and the first that is not
])
def test_thousands_of_prompts(t, H, Hkv, D, lens):
    gn = gen(len(lens))
    ct, cu, (q, k, v) = prompts(gn, lens, H, Hkv, D, t)
    out, st = torch.full_like(q, 7.0), status()
    g.gqa_attn_prefill_packed(q, k, v, ct, max(lens), out, status=st)
    assert st.item() == 0 and (out[cu[-1]:] == 7.0).all()
    assert not (out[:cu[-1]] == 7.0).all(-1).any()
    alone = torch.empty_like(out)
    for b in [b for b, n in enumerate(lens) if n >= 400] + list(range(0, len(lens), 97)):
        n, at = lens[b], slice(cu[b], cu[b + 1])
        if n == 0:
            continue
        i = torch.arange(n, device=dev())
        o, vabs, unsure = attend(q[at], k[at], v[at], i <= i[:, None])
        check(out[at], o, attend_tol(o, vabs, unsure, t, True), f"sequence {b} of {n}")
    # and every one of them as in calls of 60 prompts each
    for b0 in range(0, len(lens), 60):
        part = ct[b0:b0 + 61].contiguous()
        g.gqa_attn_prefill_packed(q, k, v, part, max(lens), alone, status=st)
    assert st.item() == 0 and torch.equal(alone[:cu[-1]], out[:cu[-1]])


def test_thousands_of_prompts_with_bad_ones_among_them():
    gn, lens = gen(2), [(5 * b) % 12 for b in range(2000)]
    ct, cu, (q, k, v) = prompts(gn, lens, 4, 2, 64, BF)
    want, out, st = torch.full_like(q, 7.0), torch.full_like(q, 7.0), status()
    g.gqa_attn_prefill_packed(q, k, v, ct, 11, want)
    g.gqa_attn_prefill_packed(q, k, v, ct, 10, out, status=st)   # the longest are skipped, and said
    assert st.item() == g.DEV_LENGTH
    long = torch.zeros(q.shape[0], dtype=torch.bool)
    for b, n in enumerate(lens):
        long[cu[b]:cu[b + 1]] = n > 10
    long = long.to(dev())
    assert (out[long] == 7.0).all() and torch.equal(out[~long], want[~long])


def test_the_time_of_many_prompts_grows_as_their_number():
    """16384 prompts of 4 tokens against 2048 of them: 8 times the work."""
    gn, took = gen(3), []
    for B in (2048, 16384):
        ct, cu, (q, k, v) = prompts(gn, [4] * B, 8, 8, 64, BF)
        out = torch.empty_like(q)
        call = lambda: g.gqa_attn_prefill_packed(q, k, v, ct, 4, out)  # noqa: E731, B023
        for _ in range(3):
            call()
        best = 1e9
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        took.append(best)
    assert took[1] < 16 * took[0], took


# ---------------------------------------------------------------- bounds that decrease

@pytest.mark.parametrize("R", [None, 0, 20])                  # without RoPE; whole head dims; partner dims one by one
def test_append_with_bounds_that_decrease(R):
    """cu_seqlens that goes back: no token is placed before its sequence's start, in another row's page or
    by another row's entry; what breaks the rule is reported."""
    gn, t, H, Hkv, D, page = gen(41), BF, 4, 2, 32, 16
    starts = [9, 9, 9, 9]
    for cu in ([0, 10, 12, 3, 4], [12, 10, 0, 11, 12], [5, 5, 2, 9, 1]):
        c = Cache(gn, 12, Hkv, page, D, t)
        table = torch.arange(8, dtype=torch.int32, device=dev()).view(4, 2)
        q, k, v = rows(gn, 12, H, D, t), rows(gn, 12, Hkv, D, t), rows(gn, 12, Hkv, D, t)
        rp, tab = (None, None) if R is None else (
            lambda p: (p, g.rope_table(p, D, dev())))(g.RopeParams.make(rope_dim=R, max_positions=64))
        q_out, k_out, st = torch.full_like(q, 7.0), torch.full_like(k, 7.0), status()
        g.kv_cache_append_paged(k, v, c.k, c.v, table, i32(starts), 31, rp, tab, cu_seqlens=i32(cu),
                                q=q, q_out=q_out, k_out=k_out, status=st)
        assert st.item() == g.DEV_LENGTH
        may = torch.zeros(12, page, dtype=torch.bool)         # slots of sequences whose own bounds hold
        here = torch.zeros(12, dtype=torch.bool)              # and their rows
        for b in range(4):
            if 0 <= cu[b] <= cu[b + 1] <= 12:
                here[cu[b]:cu[b + 1]] = True
                for i in range(cu[b + 1] - cu[b]):
                    p = starts[b] + i
                    may[2 * b + p // page, p % page] = True
        for pool in (c.k, c.v):
            assert not (torch.isfinite(pool).any(-1).any(1).cpu() & ~may).any()
        for x in (q_out, k_out):
            assert not ((x != 7.0).any(-1).any(1).cpu() & ~here).any()


def test_append_reports_bad_bounds_that_no_row_meets():
    gn, t, Hkv, D, page = gen(43), FP, 2, 64, 16
    k, v = rows(gn, 5, Hkv, D, t), rows(gn, 5, Hkv, D, t)
    for cu in ([0, 5, 3], [0, 5, 9], [0, 5] + [5] * 40 + [-1], [0, 5] + [6] * 70):
        B = len(cu) - 1
        c, st = Cache(gn, 4, Hkv, page, D, t), status()
        table = torch.zeros(B, 1, dtype=torch.int32, device=dev())
        g.kv_cache_append_paged(k, v, c.k, c.v, table, i32([0] * B), 15, cu_seqlens=i32(cu), status=st)
        assert st.item() == g.DEV_LENGTH, cu
        assert torch.equal(c.k[0, :, :5].transpose(0, 1), k) and int(torch.isfinite(c.k).sum()) == k.numel()
    st = status()
    g.kv_cache_append_paged(k, v, c.k, c.v, table, i32([0] * B), 15, cu_seqlens=i32([0, 5] + [5] * (B - 1)), status=st)
    assert st.item() == 0
