"""The 4-bit KV cache (kv_cache_append_q4, kv_cache_read_q4, gqa_attn_decode_q4,
gqa_attn_decode_step_q4, kv_cache_evict_q4) against the 64-bit reference in q4_ref.

Codes, scales, slots and kept sets are compared for equality: the library decides every
rounding as in exact arithmetic, the reference in fp64, whose own error (1e-16) meets a
border about once in 1e14 values.

Attention, to first order, with S the largest |score| in log2 units: a score is a sum of
D products whose operands hold 22 bits (2^-23 each) in fp32 sums (D / 16 truncating steps
of 2^-23 of the largest partial sum and one rounding per group), so it is off by at most
about 12 * 2^-23 of the sum of its terms' magnitudes, which for these inputs is under 8 S
+ 8; times ln 2 that is p's relative error, to which 2^ adds 2^-22. The output, a weighted mean of values, is
off by at most twice that times the largest value: with S = 20, 2 * 12 * 168 * 0.7 * 2^-23
= 3.4e-4 in the worst case and, the roundings being independent, some hundredth of that;
the bound used is the root of the count of terms instead of the count, 2e-6 (1 + S) max|v|.
"""
import math

import pytest
import torch

import gqa_causal_attention_gb300 as g
import q4_ref as ref
from gqa_causal_attention_gb300 import synthetic as syn

from gpu_util import dev

pytestmark = pytest.mark.gpu

F32 = torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


def status():
    return torch.zeros(1, dtype=torch.int32, device=dev())


def value(st):
    torch.cuda.synchronize()
    return int(st.item())


def table_of(n, R, D, theta=1e4):
    rp = g.RopeParams.make(theta=theta, rope_dim=R, max_positions=n)
    t = g.rope_table(rp, D, dev())
    return rp, t, t.cpu().view(n, R // 2, 2)


def filled(seed, B, Hkv, cap, D, scale=None):
    """Random records: (device cache, k, v float64 that they stand for)."""
    k, v = syn.normal(seed, "k", (B, Hkv, cap, D)), syn.normal(seed, "v", (B, Hkv, cap, D))
    if scale is not None:
        k, v = k * scale[0], v * scale[1]
    cache = torch.zeros(B, Hkv, cap, ref.record_bytes(D), dtype=torch.uint8, device=dev())
    st = status()
    g.kv_cache_append_q4(k.to(dev()), v.to(dev()), cache, i32([0] * B), 0, status=st)
    assert value(st) == 0
    return cache, ref.stands_for(k), ref.stands_for(v)


def close(got, want, tol):
    got = got.cpu().to(torch.float64)
    assert got.shape == want.shape
    err = (got - want).abs().max()
    assert torch.isfinite(got).all() and err <= tol, f"{float(err):.3e} > {tol:.3e}"


# ---------------------------------------------------------------- append and read

APPEND = [
    # B, Hkv, L, D, R, start, pos, cap, window, norm, k_out
    (2, 2, 5, 32, 32, (0, 3), None, 9, 0, False, None),
    (1, 3, 70, 64, 36, (4,), None, 80, 0, True, "new"),        # partners not quad-aligned
    (2, 1, 33, 96, 96, (7, 0), (100, 3), 41, 0, True, "in place"),
    (3, 2, 1, 128, 64, (0, 5, 199), None, 200, 0, False, None),
    (2, 2, 130, 128, 128, (1, 0), None, 131, 0, True, "new"),
    (1, 2, 50, 128, 128, (777,), None, 24, 24, False, "new"),  # a chunk longer than its ring
    (2, 1, 20, 160, 160, (30, 31), None, 27, 27, True, None),
    (1, 2, 9, 192, 2, (0,), (4000,), 9, 0, False, None),
    (1, 1, 17, 224, 224, (0,), None, 17, 0, True, "in place"),
    (2, 2, 40, 256, 256, (5, 60), None, 64, 64, True, "new"),
]


@pytest.mark.parametrize("B,Hkv,L,D,R,start,pos,cap,window,norm,k_out", APPEND)
def test_append_writes_the_exact_codes(B, Hkv, L, D, R, start, pos, cap, window, norm, k_out):
    seed = 5 + D
    k, v = syn.normal(seed, "k", (B, Hkv, L, D)), syn.normal(seed, "v", (B, Hkv, L, D))
    kn = syn.norm_weight(seed, "kn", D) if norm else None
    rp, table, tab = table_of(4096, R, D)
    before = torch.randint(0, 256, (B, Hkv, cap, ref.record_bytes(D)), dtype=torch.uint8)
    cache, st = before.to(dev()), status()
    kd, vd = k.to(dev()), v.to(dev())
    ko = {"new": torch.full_like(kd, math.nan), "in place": kd, None: None}[k_out]
    g.kv_cache_append_q4(kd, vd, cache, i32(start), max(start), rp, table,
                         None if kn is None else kn.to(dev()), 1e-6, k_out=ko,
                         pos=None if pos is None else i32(pos), max_pos=max(pos or (0,)),
                         window=window, status=st)
    assert value(st) == 0
    y = ref.rotate(k, pos or start, tab, kn)
    want = before.clone()
    rec = ref.pack(y, v)
    for b in range(B):
        for l in range(max(0, L - window) if window else 0, L):
            p = start[b] + l
            want[b, :, p % window if window else p] = rec[b, :, l]
    assert torch.equal(cache.cpu(), want)
    if ko is not None:       # sixteen roundings of 2^-24 of the two terms' magnitudes
        big = float(y.abs().max()) * 1.5
        close(ko, y, big * 2 ** -20)
    if k_out != "in place":
        assert torch.equal(kd.cpu(), k)
    assert torch.equal(vd.cpu(), v)

    n = min(L, window) if window else L
    first = [s + L - n for s in start]
    kr, vr = (torch.full((B, Hkv, n, D), math.nan, device=dev()) for _ in range(2))
    g.kv_cache_read_q4(cache, kr, vr, i32(first), max(first), window=window, status=st)
    assert value(st) == 0
    assert torch.equal(kr.cpu().double(), ref.stands_for(y)[:, :, L - n:])
    assert torch.equal(vr.cpu().double(), ref.stands_for(v)[:, :, L - n:])


def border_rows(D):
    """Rows whose values and group maxima sit on rounding borders, and odd magnitudes."""
    gen = torch.Generator().manual_seed(D)
    rows = []
    for e in (-140, -130, -126, -30, 0, 7, 120):
        n = torch.randint(128, 256, (D // 32,), generator=gen)
        s = n.double() * 2.0 ** (e - 7)                      # bf16 scales
        c = torch.randint(-7, 8, (D // 32, 32), generator=gen).double()
        half = torch.randint(0, 2, (D // 32, 32), generator=gen) * 0.5 * (c.abs() < 7)
        x = (c + half) * s[:, None]
        x[:, 0] = 7 * s
        rows.append(x.flatten())
        x = c * s[:, None]                                   # maxima half way between scales
        x[:, 0] = 7 * (n.double() + 0.5) * 2.0 ** (e - 7)
        rows.append(x.flatten())
    rows += [torch.zeros(D), torch.full((D,), 1.4e-45), torch.full((D,), -3.4e38)]
    return torch.stack([r.float() for r in rows])


@pytest.mark.parametrize("D", [32, 128, 256])
def test_append_on_borders_and_at_extremes(D):
    x = border_rows(D)
    n = x.shape[0]
    k, v = x.view(1, 1, n, D), x.flip(0).view(1, 1, n, D).contiguous()
    cache = torch.zeros(1, 1, n, ref.record_bytes(D), dtype=torch.uint8, device=dev())
    g.kv_cache_append_q4(k.to(dev()), v.to(dev()), cache, i32([0]), 0)
    assert torch.equal(cache.cpu(), ref.pack(k, v))


@pytest.mark.parametrize("kind", ["bf16", "spread", "decimals"])
@pytest.mark.parametrize("D,R,norm", [(64, 64, False), (96, 20, True), (128, 128, True), (256, 256, True)])
def test_append_of_many_rows(D, R, norm, kind):
    """Enough rows that hundreds of groups have a value or a scale next to a rounding border;
    values of 8 bits, of widely spread magnitude per dim, and of few decimals."""
    B, Hkv, L = 2, 2, 4000
    k, v = syn.normal(D, "k", (B, Hkv, L, D)), syn.normal(D, "v", (B, Hkv, L, D))
    if kind == "bf16":
        k, v = k.bfloat16().float(), v.bfloat16().float()
    elif kind == "spread":
        m = torch.exp2(torch.arange(D) * 5 % 23 - 11.0)
        k, v = k * m, v * m
    else:
        k, v = (k * 10).round() / 10, (v * 10).round() / 10
    kn = syn.norm_weight(D, "kn", D) if norm else None
    rp, table, tab = table_of(4100, R, D)
    cache, st = torch.zeros(B, Hkv, L, ref.record_bytes(D), dtype=torch.uint8, device=dev()), status()
    kd, vd = k.to(dev()), v.to(dev())
    g.kv_cache_append_q4(kd, vd, cache, i32([0, 0]), 0, rp, table,
                         None if kn is None else kn.to(dev()), 1e-6, pos=i32([0, 100]),
                         max_pos=100, status=st)
    g.kv_cache_read_q4(cache, kd, vd, i32([0, 0]), 0, status=st)
    assert value(st) == 0
    assert torch.equal(kd.cpu().double(), ref.stands_for(ref.rotate(k, [0, 100], tab, kn)))
    assert torch.equal(vd.cpu().double(), ref.stands_for(v))


def test_append_cancelling_rotation():
    """A whole group of rotated values that all but cancel: fp32 alone could not tell them."""
    D, L = 64, 40
    rp, table, tab = table_of(64, D, D)
    x = syn.normal(3, "x", (1, 1, L, D))
    cs = tab[torch.arange(L)].view(1, 1, L, D // 2, 2)
    x[..., :32] = x[..., 32:] * (cs[..., 1] / cs[..., 0])    # a cos - b sin = 0 up to rounding
    x = torch.where(torch.isfinite(x), x, 0.0).contiguous()
    cache = torch.zeros(1, 1, L, ref.record_bytes(D), dtype=torch.uint8, device=dev())
    v = torch.zeros_like(x)
    g.kv_cache_append_q4(x.to(dev()), v.to(dev()), cache, i32([0]), 0, rp, table)
    # the reference's fp64 has 2^-53 of the terms; the group's largest value is near 2^-24 of
    # them, so its own decisions hold to 2^-29
    got, want = ref.unpack(cache, D)[0], ref.stands_for(ref.rotate(x, [0], tab))
    assert torch.equal(got, want)


def test_groups_with_inf_or_nan_read_back_as_nan():
    B, Hkv, L, D = 1, 2, 6, 96
    k, v = syn.normal(1, "k", (B, Hkv, L, D)), syn.normal(1, "v", (B, Hkv, L, D))
    k[0, 0, 1, 40] = math.nan
    v[0, 1, 2, 95] = math.inf
    v[0, 1, 5, 0] = -math.inf
    cache = torch.zeros(B, Hkv, L, ref.record_bytes(D), dtype=torch.uint8, device=dev())
    kr, vr = (torch.zeros(B, Hkv, L, D, device=dev()) for _ in range(2))
    g.kv_cache_append_q4(k.to(dev()), v.to(dev()), cache, i32([0]), 0)
    g.kv_cache_read_q4(cache, kr, vr, i32([0]), 0)
    for got, x in ((kr, k), (vr, v)):
        want = ref.stands_for(x)
        assert torch.equal(got.cpu().double().nan_to_num(9.0), want.nan_to_num(9.0))
        assert int(want.isnan().sum()) in (32, 64)


@pytest.mark.parametrize("start,pos,bit", [((0, -1), None, g.DEV_POSITION),
                                           ((0, 7), None, g.DEV_CAPACITY),
                                           ((0, 1), (5, 62), g.DEV_POSITION)])
def test_append_and_read_skip_bad_rows(start, pos, bit):
    B, Hkv, L, D, cap = 2, 2, 3, 64, 8
    rp, table, _ = table_of(64, D, D)
    k, v = syn.normal(1, "k", (B, Hkv, L, D)).to(dev()), syn.normal(1, "v", (B, Hkv, L, D)).to(dev())
    cache, st = torch.full((B, Hkv, cap, ref.record_bytes(D)), 7, dtype=torch.uint8, device=dev()), status()
    ko = torch.full_like(k, 5.0)
    g.kv_cache_append_q4(k, v, cache, i32(start), 0, rp, table, k_out=ko,
                         pos=None if pos is None else i32(pos), status=st)
    assert value(st) == bit
    assert bool((cache[1] == 7).all()) and bool((ko[1] == 5.0).all())
    assert not bool((cache[0, :, :3] == 7).all())
    if pos is None:
        st.zero_()
        kr = torch.full_like(k, 5.0)
        vr = torch.full_like(k, 5.0)
        g.kv_cache_read_q4(cache, kr, vr, i32(start), 0, status=st)
        assert value(st) == bit
        assert bool((kr[1] == 5.0).all()) and bool((vr[1] == 5.0).all())
        assert torch.equal(kr[0].cpu().double(), ref.unpack(cache[0, :, :3], D)[0])


# ---------------------------------------------------------------- decode

DECODE = [
    # B, H, Hkv, D, lengths, cap, window, softcap, scale
    (1, 1, 1, 32, (1,), 1, 0, 0.0, 0.0),
    (3, 8, 8, 64, (1, 31, 33), 40, 0, 0.0, 0.0),               # one query head per kv head
    (2, 6, 2, 96, (32, 500), 501, 0, 30.0, 0.0),
    (4, 32, 8, 128, (1, 64, 700, 129), 700, 0, 0.0, 0.0),
    (1, 64, 8, 128, (4096,), 4100, 0, 0.0, 0.0),
    (2, 14, 2, 128, (65, 1000), 1000, 0, 0.0, 0.25),           # seven heads per kv head
    (2, 24, 2, 160, (90, 257), 300, 0, 0.0, 0.0),              # twelve: two groups of heads
    (1, 16, 1, 192, (900,), 1200, 0, 50.0, 0.0),
    (1, 4, 2, 224, (1300,), 1300, 0, 0.0, 0.0),
    (2, 16, 8, 256, (5000, 17), 300, 300, 50.0, 0.0),          # ring
    (1, 8, 1, 128, (20000,), 20001, 0, 0.0, 0.0),
]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("B,H,Hkv,D,lens,cap,window,softcap,scale", DECODE)
def test_decode_matches_the_reference(B, H, Hkv, D, lens, cap, window, softcap, scale, weights):
    if weights and window:
        pytest.skip("weights are not kept for rings")
    cache, k, v = filled(H + D, B, Hkv, cap, D)
    live = [min(n, window) if window else n for n in lens]
    for b in range(B):                       # slots behind the live ones: NaN scales, odd codes
        cache[b, :, live[b]:] = 255
    q = syn.normal(D, "q", (B, H, 1, D))
    out, st = torch.full((B, H, 1, D), math.nan, device=dev()), status()
    w0 = torch.rand(B, Hkv, cap)
    w = w0.to(dev()) if weights else None
    qd, cl = q.to(dev()), i32(lens)
    keep = cache.clone()
    g.gqa_attn_decode_q4(qd, cache, cl, max(lens), out, weights=w, window=window,
                         softcap=softcap, scale=scale, status=st)
    assert value(st) == 0
    want, ww, S = ref.decode(q, k, v, live, softcap, scale)
    tol = 2e-6 * (1 + S / math.log(2))
    close(out, want, tol * float(v.abs().max()))
    assert torch.equal(cache, keep) and torch.equal(qd.cpu(), q)
    if weights:
        close(w, w0.double() + ww, tol * (H // Hkv) + tol + 2 ** -23)
        for b in range(B):
            assert torch.equal(w[b, :, live[b]:].cpu(), w0[b, :, live[b]:])
    again = torch.empty_like(out)
    w2 = w0.to(dev()) if weights else None
    g.gqa_attn_decode_q4(qd, cache, cl, max(lens), again, weights=w2, window=window,
                         softcap=softcap, scale=scale)
    assert torch.equal(out, again) and (w is None or torch.equal(w, w2))


@pytest.mark.parametrize("kmag,vmag,qmag", [(1e-3, 1e-25, 1e3), (1e-30, 1e30, 1e25),
                                            (1e20, 1.0, 1e-20), (1.0, 1e36, 0.0)])
def test_decode_magnitudes(kmag, vmag, qmag):
    B, H, Hkv, D, n = 1, 4, 1, 64, 333
    cache, k, v = filled(3, B, Hkv, n, D, (kmag, vmag))
    q = syn.normal(4, "q", (B, H, 1, D)) * qmag
    out = torch.empty(B, H, 1, D, device=dev())
    g.gqa_attn_decode_q4(q.to(dev()), cache, i32([n]), n, out)
    want, _, S = ref.decode(q, k, v, [n])
    close(out, want, 2e-6 * (1 + S / math.log(2)) * float(v.abs().max()))


def test_decode_values_of_mixed_magnitude():
    """Value groups and positions 2^16 apart: each group's error stays relative to its own
    largest value. The reference exponent is shared, so the smallest keep 22 bits as long as
    they are within 2^16 of the largest."""
    B, H, Hkv, D, n = 1, 8, 1, 128, 700
    vmul = torch.ones(1, 1, n, D)
    vmul[..., 32:64] = 2.0 ** -8
    vmul[..., 64:96] = 2.0 ** 8
    vmul[:, :, ::3] *= 2.0 ** -8
    cache, k, v = filled(5, B, Hkv, n, D, (1.0, vmul))
    q = syn.normal(4, "q", (B, H, 1, D))
    out = torch.empty(B, H, 1, D, device=dev())
    g.gqa_attn_decode_q4(q.to(dev()), cache, i32([n]), n, out)
    want, _, S = ref.decode(q, k, v, [n])
    for gr in range(4):
        part = slice(32 * gr, 32 * gr + 32)
        close(out[..., part], want[..., part],
              2e-6 * (1 + S / math.log(2)) * float(v[..., part].abs().max()))


def test_decode_nan_stays_where_it_is():
    B, H, Hkv, D, n = 2, 8, 2, 128, 300
    k, v = syn.normal(1, "k", (B, Hkv, n, D)), syn.normal(1, "v", (B, Hkv, n, D))
    v[0, 0, 200, 70] = math.nan              # one value group of kv head 0
    k[1, 1, 10, 3] = math.nan                # a key: all of kv head 1 of row 1
    cache = torch.zeros(B, Hkv, n, ref.record_bytes(D), dtype=torch.uint8, device=dev())
    g.kv_cache_append_q4(k.to(dev()), v.to(dev()), cache, i32([0, 0]), 0)
    q = syn.normal(2, "q", (B, H, 1, D))
    q[0, 7, 0, 0] = math.nan                 # one query head
    out = torch.empty(B, H, 1, D, device=dev())
    g.gqa_attn_decode_q4(q.to(dev()), cache, i32([n, n]), n, out)
    bad = torch.zeros(B, H, 1, D, dtype=torch.bool)
    bad[0, :4, :, 64:96] = True
    bad[1, 4:] = True
    bad[0, 7] = True
    assert torch.equal(out.isnan().cpu(), bad)
    want, _, S = ref.decode(q.nan_to_num(0.0), ref.stands_for(k).nan_to_num(0.0),
                            ref.stands_for(v).nan_to_num(0.0), [n, n])
    err = (out.cpu().double() - want).abs()[~bad].max()
    assert err <= 2e-6 * (1 + S / math.log(2)) * float(v.nan_to_num(0.0).abs().max())


@pytest.mark.parametrize("B,H,n", [(1, 2, 20000), (40, 4, 4000), (1, 2, 300)])
def test_decode_nan_of_a_whole_split_is_not_lost(B, H, n):
    """Half the keys of one kv head NaN, so whole splits (and whole warps' shares) have no score
    at all; in the other kv head a NaN value whose softmax weight is 2^-200 or so: fp32 holds it
    as 0, and 0 times NaN is NaN all the same. Row 1 (if there is one) holds no NaN."""
    Hkv, D = 2, 64
    k, v = syn.normal(1, "k", (1, Hkv, n, D)), syn.normal(1, "v", (1, Hkv, n, D))
    q = syn.normal(2, "q", (1, H, 1, D))
    k[0, 1, -1] = 60 * q[0, -1, 0]           # the key that outweighs every other by far
    k, v = k.repeat(B, 1, 1, 1), v.repeat(B, 1, 1, 1)
    k[0, 0, n // 2:, 0] = math.nan
    v[0, 1, 3, 40] = math.nan
    cache = torch.zeros(B, Hkv, n, ref.record_bytes(D), dtype=torch.uint8, device=dev())
    g.kv_cache_append_q4(k.to(dev()), v.to(dev()), cache, i32([0] * B), 0)
    q = q.repeat(B, 1, 1, 1).to(dev())
    out, w, st = torch.empty_like(q), torch.zeros(B, Hkv, n, device=dev()), status()
    bad = torch.zeros(B, H, 1, D, dtype=torch.bool)
    bad[0, :H // 2] = True
    bad[0, H // 2:, :, 32:] = True
    for weights in (None, w):
        g.gqa_attn_decode_q4(q, cache, i32([n] * B), n, out, weights=weights, status=st)
        assert value(st) == 0
        assert torch.equal(out.isnan().cpu(), bad)
    assert bool(w[0, 0].isnan().all()) and not bool(w[0, 1].isnan().any() or w[1:].isnan().any())


def test_decode_skips_bad_rows_and_leaves_their_output():
    B, H, Hkv, D, cap = 4, 4, 2, 64, 600
    cache, k, v = filled(9, B, Hkv, cap, D)
    q = syn.normal(2, "q", (B, H, 1, D))
    out, st = torch.full((B, H, 1, D), 3.0, device=dev()), status()
    w = torch.full((B, Hkv, cap), 2.0, device=dev())
    g.gqa_attn_decode_q4(q.to(dev()), cache, i32([0, 600, 601, -5]), 600, out, weights=w, status=st)
    assert value(st) == g.DEV_LENGTH
    want, _, S = ref.decode(q, k, v, [1, 600, 1, 1])
    close(out[1], want[1], 2e-6 * (1 + S / math.log(2)) * float(v.abs().max()))
    for b in (0, 2, 3):
        assert bool((out[b] == 3.0).all()) and bool((w[b] == 2.0).all())


def test_decode_far_into_a_large_cache():
    """Records past 2^32 bytes from the cache's start."""
    B, Hkv, H, D, cap = 64, 8, 8, 128, 65536
    cache = torch.full((B, Hkv, cap, 144), 255, dtype=torch.uint8, device=dev())
    small, k, v = filled(2, 1, Hkv, 50, D)
    cache[B - 1, :, :50] = small[0]
    q = syn.normal(2, "q", (B, H, 1, D))
    out, st = torch.full((B, H, 1, D), 3.0, device=dev()), status()
    g.gqa_attn_decode_q4(q.to(dev()), cache, i32([0] * (B - 1) + [50]), cap, out, status=st)
    assert value(st) == g.DEV_LENGTH
    want, _, S = ref.decode(q[B - 1:], k, v, [50])
    close(out[B - 1:], want, 2e-6 * (1 + S / math.log(2)) * float(v.abs().max()))
    kr, vr = torch.empty(B, Hkv, 2, D, device=dev()), torch.empty(B, Hkv, 2, D, device=dev())
    g.kv_cache_read_q4(cache, kr, vr, i32([0] * B), 0)
    assert torch.equal(kr[B - 1].cpu().double(), k[0, :, :2])
    # an append and an eviction there
    x = syn.normal(7, "x", (B, Hkv, 1, D))
    g.kv_cache_append_q4(x.to(dev()), x.to(dev()), cache, i32([cap - 1] * B), cap - 1)
    assert torch.equal(ref.unpack(cache[B - 1, Hkv - 1, cap - 1], D)[0],
                       ref.stands_for(x[B - 1, Hkv - 1, 0]))


# ---------------------------------------------------------------- step

STEP = [
    # B, H, Hkv, D, R, start, pos, cap, window, softcap, norm, weights
    (3, 32, 8, 128, 128, (0, 31, 700), None, 701, 0, 0.0, False, True),
    (2, 64, 8, 128, 64, (32, 1023), None, 1024, 0, 0.0, True, False),
    (2, 4, 2, 256, 256, (10, 700), None, 64, 64, 50.0, True, False),   # ring, one row wrapped
    (2, 6, 2, 96, 36, (63, 64), (900, 64), 65, 0, 30.0, True, True),   # positions past the slots
    (1, 2, 2, 32, 32, (0,), None, 1, 0, 0.0, False, False),
]


@pytest.mark.parametrize("B,H,Hkv,D,R,start,pos,cap,window,softcap,norm,weights", STEP)
def test_step_matches_the_reference(B, H, Hkv, D, R, start, pos, cap, window, softcap, norm,
                                    weights):
    cache, kc, vc = filled(D, B, Hkv, cap, D)
    q = syn.normal(8, "q", (B, H, 1, D))
    k, v = syn.normal(8, "k", (B, Hkv, 1, D)), syn.normal(8, "v", (B, Hkv, 1, D))
    qn, kn = (syn.norm_weight(8, n, D) if norm else None for n in ("qn", "kn"))
    rp, table, tab = table_of(1024, R, D)
    before = cache.cpu().clone()
    out, st = torch.full((B, H, 1, D), math.nan, device=dev()), status()
    w = torch.zeros(B, Hkv, cap, device=dev()) if weights else None
    cu = lambda t: None if t is None else t.to(dev())  # noqa: E731
    qd, kd, vd = cu(q), cu(k), cu(v)
    g.gqa_attn_decode_step_q4(qd, kd, vd, out, cache, i32(start), max(start), rp, table, cu(qn),
                              cu(kn), 1e-6, pos=None if pos is None else i32(pos),
                              max_pos=max(pos or (0,)), weights=w, window=window,
                              softcap=softcap, status=st)
    assert value(st) == 0
    y = ref.rotate(k, pos or start, tab, kn)
    rec = ref.pack(y, v)
    for b in range(B):
        slot = start[b] % window if window else start[b]
        before[b, :, slot] = rec[b, :, 0]
        kc[b, :, slot], vc[b, :, slot] = ref.stands_for(y)[b, :, 0], ref.stands_for(v)[b, :, 0]
    assert torch.equal(cache.cpu(), before)
    live = [min(s + 1, window) if window else s + 1 for s in start]
    want, ww, S = ref.decode(ref.rotate(q, pos or start, tab, qn), kc, vc, live, softcap)
    tol = 2e-6 * (1 + S / math.log(2))
    close(out, want, tol * float(vc.abs().max()))
    if weights:
        close(w, ww, tol * (H // Hkv) + tol)
    assert torch.equal(qd.cpu(), q) and torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


@pytest.mark.parametrize("D", [32, 128, 256])
def test_step_of_many_heads_attends_to_the_final_codes(D):
    """16 and 20 query heads a kv head: several blocks append the token and read it back. The
    new keys and values sit on rounding borders, where first guesses at the codes are wrong;
    the step must give what a decode over the finished cache gives, bit for bit. (Position 0
    rotates by nothing.)"""
    x = border_rows(D)
    x = x[x.abs().amax(-1) < 2.0 ** 100]                     # scores stay finite
    n, Hkv = x.shape[0], 4
    for G, lens in ((16, (5, 700)), (20, (63, 2049))):
        B, cap = 8 * len(lens), max(lens) + 1
        start = [lens[b % len(lens)] for b in range(B)]
        cache, _, _ = filled(D + G, B, Hkv, cap, D)
        q = syn.normal(G, "q", (B, Hkv * G, 1, D)).to(dev())
        rp, table, _ = table_of(16, D, D)
        out, again, st = torch.empty_like(q), torch.empty_like(q), status()
        for r in range(8):
            at = (torch.arange(B * Hkv) + 5 * r) % n
            k = x[at].view(B, Hkv, 1, D).contiguous()
            v = x[(at + 3) % n].view(B, Hkv, 1, D).contiguous()
            g.gqa_attn_decode_step_q4(q, k.to(dev()), v.to(dev()), out, cache, i32(start),
                                      max(start), rp, table, pos=i32([0] * B), status=st)
            g.gqa_attn_decode_q4(q, cache, i32([s + 1 for s in start]), max(start) + 1, again,
                                 status=st)
            assert value(st) == 0
            assert torch.equal(out, again)
            rec = ref.pack(k, v)
            for b in range(B):
                assert torch.equal(cache[b, :, start[b]].cpu(), rec[b, :, 0])


def test_step_skips_bad_rows():
    B, H, Hkv, D, cap = 4, 4, 2, 64, 40
    cache, kc, vc = filled(2, B, Hkv, cap, D)
    rp, table, tab = table_of(64, D, D)
    q, k, v = (syn.normal(3, n, (B, h, 1, D)) for n, h in (("q", H), ("k", Hkv), ("v", Hkv)))
    before, out, st = cache.cpu().clone(), torch.full((B, H, 1, D), 3.0, device=dev()), status()
    g.gqa_attn_decode_step_q4(q.to(dev()), k.to(dev()), v.to(dev()), out, cache,
                              i32([-1, 40, 7, 8]), 39, rp, table, pos=i32([0, 0, 64, 5]),
                              max_pos=63, status=st)
    assert value(st) == g.DEV_POSITION | g.DEV_CAPACITY | g.DEV_LENGTH
    assert torch.equal(cache[:3].cpu(), before[:3]) and bool((out[:3] == 3.0).all())
    y = ref.rotate(k[3:], [5], tab)
    kc[3, :, 8], vc[3, :, 8] = ref.stands_for(y)[0, :, 0], ref.stands_for(v)[3, :, 0]
    want, _, S = ref.decode(ref.rotate(q[3:], [5], tab), kc[3:], vc[3:], [9])
    close(out[3:], want, 2e-6 * (1 + S / math.log(2)) * float(vc.abs().max()))


# ---------------------------------------------------------------- eviction

EVICT = [
    # B, Hkv, D, lengths, cap, budget, recent, cap_out
    (3, 2, 64, (10, 4, 0), 12, 4, 2, 5),
    (1, 3, 128, (1000,), 1001, 1000, 10, 1000),      # nothing to evict
    (2, 2, 128, (1001, 999), 1001, 1000, 10, 1003),  # one slot
    (2, 1, 32, (5000, 4097), 5003, 777, 0, 778),     # no recent slots
    (1, 2, 96, (300,), 300, 100, 100, 100),          # recent slots only
    (1, 1, 256, (9000,), 9001, 8190, 4000, 8200),
    (1, 1, 32, (50000,), 50000, 20001, 3, 20001),    # more keys than shared memory holds
    (2, 2, 160, (64, 65), 70, 1, 0, 1),
    # many heads: selected and moved by two kernels
    (21, 2, 32, tuple(90 + 17 * i for i in range(21)), 430, 100, 20, 101),
    (13, 3, 64, tuple(5000 - 230 * i for i in range(13)), 5003, 2500, 300, 2500),
]


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("B,Hkv,D,lens,cap,budget,recent,cap_out", EVICT)
def test_evict_keeps_the_heaviest(B, Hkv, D, lens, cap, budget, recent, cap_out, kind):
    gen = torch.Generator().manual_seed(cap + budget)
    w = torch.rand(B, Hkv, cap, generator=gen) ** 6
    if kind == "ties":
        w = (w * 3).round() / 3
    elif kind == "odd":                      # negatives, zeros of both signs, infinities, NaN
        w = torch.where(torch.rand(w.shape, generator=gen) < 0.3, -w, w)
        for x, share in ((0.0, 0.1), (-0.0, 0.1), (math.inf, 0.01), (-math.inf, 0.01), (math.nan, 0.01)):
            w = torch.where(torch.rand(w.shape, generator=gen) < share, torch.tensor(x), w)
    rec = torch.randint(0, 256, (B, Hkv, cap, ref.record_bytes(D)), generator=gen, dtype=torch.uint8)
    before = torch.randint(0, 256, (B, Hkv, cap_out, ref.record_bytes(D)), generator=gen,
                           dtype=torch.uint8)
    out, st = before.to(dev()), status()
    w_out = torch.full((B, Hkv, cap_out), math.nan, device=dev())
    index = torch.full((B, Hkv, budget), -7, dtype=torch.int32, device=dev())
    n_out = torch.full((B,), -7, dtype=torch.int32, device=dev())
    g.kv_cache_evict_q4(rec.to(dev()), w.to(dev()), i32(lens), max(lens), budget, recent, out,
                        w_out, index, n_out, status=st)
    assert value(st) == 0
    assert n_out.tolist() == [min(n, budget) for n in lens]
    for b in range(B):
        for h in range(Hkv):
            keep = ref.evict(w[b, h], lens[b], budget, recent)
            assert index[b, h].tolist() == keep + [-1] * (budget - len(keep))
            before[b, h, :len(keep)] = rec[b, h, keep]
            want = torch.cat([w[b, h, keep], torch.zeros(cap_out - len(keep))])
            assert torch.equal(w_out[b, h].cpu().nan_to_num(77.0), want.nan_to_num(77.0))
    assert torch.equal(out.cpu(), before)


def test_evict_skips_bad_rows():
    B, Hkv, D, cap = 3, 2, 64, 20
    cache, _, _ = filled(1, B, Hkv, cap, D)
    out = torch.full((B, Hkv, 8, 80), 9, dtype=torch.uint8, device=dev())
    w_out = torch.full((B, Hkv, 8), 9.0, device=dev())
    index = torch.full((B, Hkv, 8), 9, dtype=torch.int32, device=dev())
    n_out, st = i32([9, 9, 9]), status()
    g.kv_cache_evict_q4(cache, torch.rand(B, Hkv, cap, device=dev()), i32([21, 12, -1]), 20, 8, 2,
                        out, w_out, index, n_out, status=st)
    assert value(st) == g.DEV_LENGTH
    assert n_out.tolist() == [9, 8, 9]
    for b in (0, 2):
        assert bool((out[b] == 9).all()) and bool((w_out[b] == 9.0).all()) and bool((index[b] == 9).all())


def test_evict_of_many_heads_skips_bad_rows():
    """As above where the selection and the move are two kernels."""
    B, Hkv, D, cap = 12, 4, 32, 50
    cache, _, _ = filled(1, B, Hkv, cap, D)
    out = torch.full((B, Hkv, 8, 48), 9, dtype=torch.uint8, device=dev())
    w, w_out = torch.rand(B, Hkv, cap, device=dev()), torch.full((B, Hkv, 8), 9.0, device=dev())
    index = torch.full((B, Hkv, 8), 9, dtype=torch.int32, device=dev())
    lens = [51, 50, -1, 0, 7, 8, 9, 2 ** 31 - 1, 20, 30, 40, -2 ** 31]
    n_out, st = i32([9] * B), status()
    g.kv_cache_evict_q4(cache, w, i32(lens), 50, 8, 2, out, w_out, index, n_out, status=st)
    assert value(st) == g.DEV_LENGTH
    for b, n in enumerate(lens):
        if not 0 <= n <= 50:
            assert int(n_out[b]) == 9 and bool((out[b] == 9).all())
            assert bool((w_out[b] == 9.0).all()) and bool((index[b] == 9).all())
            continue
        assert int(n_out[b]) == min(n, 8)
        for h in range(Hkv):
            keep = ref.evict(w[b, h].cpu(), n, 8, 2)
            assert index[b, h].tolist() == keep + [-1] * (8 - len(keep))
            assert torch.equal(out[b, h, :len(keep)], cache[b, h, keep])
            assert bool((out[b, h, len(keep):] == 9).all()) and bool((w_out[b, h, len(keep):] == 0).all())


# ---------------------------------------------------------------- together

def test_captured_chunk_replays():
    """Append, read back and decode captured once, replayed on new contents and positions."""
    B, H, Hkv, D, L, cap = 2, 12, 2, 96, 37, 300
    rp, table, tab = table_of(512, D, D)
    k, v = (torch.randn(B, Hkv, L, D, device=dev()) for _ in range(2))
    q, ko, kr, vr = torch.randn(B, H, 1, D, device=dev()), *(torch.empty_like(k) for _ in range(3))
    cache = torch.zeros(B, Hkv, cap, ref.record_bytes(D), dtype=torch.uint8, device=dev())
    start, lens, st, out = i32([0, 0]), i32([L, L]), status(), torch.empty_like(q)
    ws = torch.empty(g.gqa_attn_decode_q4_workspace_size(B, H, Hkv, D, cap), dtype=torch.uint8,
                     device=dev())

    def chunk():
        g.kv_cache_append_q4(k, v, cache, start, cap - L, rp, table, k_out=ko, status=st)
        g.kv_cache_read_q4(cache, kr, vr, start, cap - L, status=st)
        g.gqa_attn_decode_q4(q, cache, lens, cap, out, workspace=ws, status=st)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        chunk()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        chunk()
    kc, vc = (torch.zeros(B, Hkv, cap, D, dtype=torch.float64) for _ in range(2))
    for i in range(4):
        at = [i * L, i * L]
        x = [syn.normal(30 + i, m, t.shape) for m, t in (("k", k), ("v", v), ("q", q))]
        for t, y in zip((k, v, q, start, lens), x + [i32(at), i32([a + L for a in at])]):
            t.copy_(y)
        graph.replay()
        assert value(st) == 0
        y = ref.rotate(x[0], at, tab)
        kc[:, :, i * L:(i + 1) * L], vc[:, :, i * L:(i + 1) * L] = ref.stands_for(y), ref.stands_for(x[1])
        assert torch.equal(kr.cpu().double(), ref.stands_for(y))
        assert torch.equal(vr.cpu().double(), ref.stands_for(x[1]))
        want, _, S = ref.decode(x[2], kc, vc, [a + L for a in at])
        close(out, want, 2e-6 * (1 + S / math.log(2)) * float(vc.abs().max()))


def test_serving_run_with_eviction():
    """A prompt enters a 4-bit cache and is attended; a second prompt chunk continues it (read
    back, gqa_attn_prefill_cached); tokens are decoded with weights; the cache is trimmed; more
    tokens follow at their true positions. Every stage against the 64-bit reference."""
    B, H, Hkv, D, R = 2, 8, 2, 128, 128
    L0, L1, T, cap = 60, 21, 9, 128
    rp, table, tab = table_of(512, R, D, 5e5)
    kn = syn.norm_weight(1, "kn", D)
    qn = syn.norm_weight(1, "qn", D)
    knd, qnd = kn.to(dev()), qn.to(dev())
    n = L0 + L1 + 2 * T
    q, k, v = (syn.normal(6, x, (B, h, n, D)) for x, h in (("q", H), ("k", Hkv), ("v", Hkv)))
    cut = lambda t, a, b: t[:, :, a:b].contiguous().to(dev())  # noqa: E731
    cache = torch.zeros(B, Hkv, cap, 144, dtype=torch.uint8, device=dev())
    st = status()
    y = ref.rotate(k, [0] * B, tab, kn)
    ks, vs = ref.stands_for(y), ref.stands_for(v)
    qr = ref.rotate(q, [0] * B, tab, qn)

    # the first chunk
    k_rot = torch.empty(B, Hkv, L0, D, device=dev())
    g.kv_cache_append_q4(cut(k, 0, L0), cut(v, 0, L0), cache, i32([0, 0]), 0, rp, table, knd,
                         k_out=k_rot, status=st)
    # the second: attends the stored prefix and its own keys
    k1 = torch.empty(B, Hkv, L1, D, device=dev())
    kf, vf = torch.empty(B, Hkv, L0, D, device=dev()), torch.empty(B, Hkv, L0, D, device=dev())
    g.kv_cache_read_q4(cache, kf, vf, i32([0, 0]), 0, status=st)
    g.kv_cache_append_q4(cut(k, L0, L0 + L1), cut(v, L0, L0 + L1), cache, i32([L0, L0]), L0, rp,
                         table, knd, k_out=k1, status=st)
    o1 = torch.empty(B, H, L1, D, device=dev())
    g.gqa_attn_prefill_cached(cut(q, L0, L0 + L1), k1, cut(v, L0, L0 + L1), kf, vf, o1,
                              i32([L0, L0]), L0, rp, table, qnd, status=st)
    assert value(st) == 0
    for l in (0, L1 // 2, L1 - 1):
        kk = torch.cat([ks[:, :, :L0], y[:, :, L0:]], 2)
        vv = torch.cat([vs[:, :, :L0], v[:, :, L0:].double()], 2)
        want, _, _ = ref.decode(qr[:, :, L0 + l:L0 + l + 1], kk, vv, [L0 + l + 1] * B)
        close(o1[:, :, l:l + 1], want, 5e-3)             # TF32 operands, as the prefill's own tests

    # single tokens, accumulating weights
    w = torch.zeros(B, Hkv, cap, device=dev())
    wr = torch.zeros(B, Hkv, cap, dtype=torch.float64)
    out = torch.empty(B, H, 1, D, device=dev())
    m = L0 + L1
    for t in range(m, m + T):
        g.gqa_attn_decode_step_q4(cut(q, t, t + 1), cut(k, t, t + 1), cut(v, t, t + 1), out, cache,
                                  i32([t] * B), t, rp, table, qnd, knd, weights=w, status=st)
        want, ww, S = ref.decode(qr[:, :, t:t + 1], ks, vs, [t + 1] * B)
        close(out, want, 2e-6 * (1 + S / math.log(2)) * float(v.abs().max()))
        wr[:, :, :t + 1] += ww[:, :, :t + 1]
    m += T
    close(w, wr, 2e-5 * (1 + S / math.log(2)) * (H // Hkv))

    # trim to 40 slots, the last 8 always kept
    budget, recent = 40, 8
    c2 = torch.full((B, Hkv, 64, 144), 255, dtype=torch.uint8, device=dev())
    w2, index = torch.empty(B, Hkv, 64, device=dev()), torch.empty(B, Hkv, budget, dtype=torch.int32, device=dev())
    n2 = torch.empty(B, dtype=torch.int32, device=dev())
    g.kv_cache_evict_q4(cache, w, i32([m] * B), m, budget, recent, c2, w2, index, n2, status=st)
    assert value(st) == 0 and n2.tolist() == [budget] * B
    for b in range(B):
        for h in range(Hkv):
            assert index[b, h].tolist() == ref.evict(w[b, h].cpu(), m, budget, recent)
    at = index.cpu().long()[..., None].expand(-1, -1, -1, D)
    k2, v2 = ks.gather(2, at), vs.gather(2, at)

    # and on: slots count from the trimmed length, positions from the true one
    for i in range(T):
        t = m + i
        g.gqa_attn_decode_step_q4(cut(q, t, t + 1), cut(k, t, t + 1), cut(v, t, t + 1), out, c2,
                                  n2, budget + i, rp, table, qnd, knd, pos=i32([t] * B), max_pos=t,
                                  weights=w2, status=st)
        n2 += 1
        k2, v2 = torch.cat([k2, ks[:, :, t:t + 1]], 2), torch.cat([v2, vs[:, :, t:t + 1]], 2)
        want, _, S = ref.decode(qr[:, :, t:t + 1], k2, v2, [budget + i + 1] * B)
        close(out, want, 2e-6 * (1 + S / math.log(2)) * float(v.abs().max()))
    assert value(st) == 0
    assert bool((w2[:, :, budget + T:] == 0).all())


def test_captured_steps_replay():
    """A step and an eviction captured once and replayed on new contents, on a side stream."""
    B, H, Hkv, D, cap, n = 2, 16, 2, 128, 3000, 2500
    cache, kc, vc = filled(11, B, Hkv, cap, D)
    rp, table, tab = table_of(4096, D, D)
    q, k, v = (torch.empty(B, h, 1, D, device=dev()) for h in (H, Hkv, Hkv))
    out, st, start = torch.empty(B, H, 1, D, device=dev()), status(), i32([n, n - 700])
    w = torch.zeros(B, Hkv, cap, device=dev())
    ws = torch.empty(g.gqa_attn_decode_step_q4_workspace_size(B, H, Hkv, D, cap - 1, 0, True),
                     dtype=torch.uint8, device=dev())
    c2 = torch.zeros(B, Hkv, 1100, 144, dtype=torch.uint8, device=dev())
    w2, idx = torch.zeros(B, Hkv, 1100, device=dev()), torch.zeros(B, Hkv, 1024, dtype=torch.int32, device=dev())
    n2 = i32([0, 0])
    s = torch.cuda.Stream()

    def both():
        g.gqa_attn_decode_step_q4(q, k, v, out, cache, start, cap - 1, rp, table, weights=w,
                                  workspace=ws, status=st)
        g.kv_cache_evict_q4(cache, w, start, cap, 1024, 64, c2, w2, idx, n2, status=st)

    for t in (q, k, v):
        t.normal_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        both()
    torch.cuda.synchronize()
    w.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    for i in range(3):
        x = [syn.normal(20 + i, m, t.shape) for m, t in (("q", q), ("k", k), ("v", v))]
        for t, y in zip((q, k, v), x):
            t.copy_(y)
        w.zero_()
        graph.replay()
        assert value(st) == 0
        at = start.tolist()
        y, z = ref.stands_for(ref.rotate(x[1], at, tab)), ref.stands_for(x[2])
        for b in range(B):
            kc[b, :, at[b]], vc[b, :, at[b]] = y[b, :, 0], z[b, :, 0]
        want, ww, S = ref.decode(ref.rotate(x[0], at, tab), kc, vc, [a + 1 for a in at])
        tol = 2e-6 * (1 + S / math.log(2))
        close(out, want, tol * float(vc.abs().max()))
        close(w, ww, tol * 8 + tol)
        for b in range(B):
            assert idx[b, 1].tolist() == ref.evict(w[b, 1].cpu(), at[b], 1024, 64)
        start += 1


def test_two_streams_with_their_own_workspaces():
    B, H, Hkv, D, n = 2, 8, 2, 128, 20000
    cache, k, v = filled(12, B, Hkv, n, D)
    q = [syn.normal(i, "q", (B, H, 1, D)).to(dev()) for i in range(2)]
    one = [torch.empty(B, H, 1, D, device=dev()) for _ in range(2)]
    two = [torch.empty(B, H, 1, D, device=dev()) for _ in range(2)]
    cl = i32([n, n - 1])
    for i in range(2):
        g.gqa_attn_decode_q4(q[i], cache, cl, n, one[i])
    size = g.gqa_attn_decode_q4_workspace_size(B, H, Hkv, D, n)
    ws = [torch.empty(size, dtype=torch.uint8, device=dev()) for _ in range(2)]
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            g.gqa_attn_decode_q4(q[i], cache, cl, n, two[i], workspace=ws[i], stream=st[i])
    torch.cuda.synchronize()
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_finite_check_covers_the_q4_calls():
    B, H, Hkv, D, cap, n = 1, 4, 2, 64, 32, 20
    k, v = syn.normal(1, "k", (B, Hkv, n, D)).to(dev()), syn.normal(1, "v", (B, Hkv, n, D)).to(dev())
    cache = torch.zeros(B, Hkv, cap, 80, dtype=torch.uint8, device=dev())
    cache[:, :, n:] = 255                    # dead slots may hold anything
    q = syn.normal(1, "q", (B, H, 1, D)).to(dev())
    out, st, zero = torch.full((B, H, 1, D), 3.0, device=dev()), status(), i32([0])
    prev = g.attn_set_check_finite(1)
    try:
        g.kv_cache_append_q4(k, v, cache, zero, 0, status=st)
        g.gqa_attn_decode_q4(q, cache, i32([n]), n, out, status=st)
        kr, vr = torch.empty_like(k), torch.empty_like(v)
        g.kv_cache_read_q4(cache, kr, vr, zero, 0, status=st)
        assert value(st) == 0 and not bool((out == 3.0).any())
        bad, kept = k.clone(), cache.clone()
        bad[0, 1, 7, 5] = math.inf
        g.kv_cache_append_q4(bad, v, cache, zero, 0, status=st)
        assert value(st) == g.DEV_NONFINITE and torch.equal(cache, kept)
        st.zero_()
        g.attn_set_check_finite(0)
        g.kv_cache_append_q4(bad, v, cache, zero, 0)         # now the record holds a NaN group
        g.attn_set_check_finite(1)
        out.fill_(3.0)
        g.gqa_attn_decode_q4(q, cache, i32([7]), n, out, status=st)      # not among the live slots
        assert value(st) == 0
        out.fill_(3.0)
        g.gqa_attn_decode_q4(q, cache, i32([8]), n, out, status=st)
        assert value(st) == g.DEV_NONFINITE and bool((out == 3.0).all())
        st.zero_()
        g.kv_cache_read_q4(cache, kr[:, :, :5].contiguous(), vr[:, :, :5].contiguous(), i32([8]), 8, status=st)
        assert value(st) == 0
        g.kv_cache_read_q4(cache, kr[:, :, :5].contiguous(), vr[:, :, :5].contiguous(), i32([3]), 8, status=st)
        assert value(st) == g.DEV_NONFINITE
        with pytest.raises(g.AttnError):
            g.gqa_attn_decode_q4(q, cache, i32([8]), n, out)
    finally:
        g.attn_set_check_finite(prev)


# ---------------------------------------------------------------- calls and shapes

@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    """A step with weights (or in a ring), then a decode over the same cache, at drawn shapes."""
    gen = torch.Generator().manual_seed(seed)
    pick = lambda *xs: xs[int(torch.randint(len(xs), (1,), generator=gen))]  # noqa: E731
    D, G, Hkv, B = pick(32, 64, 96, 128, 160, 192, 224, 256), pick(1, 2, 3, 4, 5, 8, 9, 16), pick(1, 2, 3), pick(1, 2, 5)
    H, R = G * Hkv, pick(D, D // 2, 2, D - 2)
    cap = pick(1, 33, 130, 513, 2049)
    ring = seed % 3 == 0
    window, norm, softcap = cap if ring else 0, seed % 2 == 0, pick(0.0, 20.0)
    cache, kc, vc = filled(seed, B, Hkv, cap, D)
    hi = 3000 if ring else cap
    start = torch.randint(0, hi, (B,), generator=gen).tolist()
    pos = torch.randint(0, 4000, (B,), generator=gen).tolist()
    rp, table, tab = table_of(4000, R, D)
    q, k, v = (syn.normal(seed + 100, n, (B, h, 1, D)) for n, h in (("q", H), ("k", Hkv), ("v", Hkv)))
    qn, kn = (syn.norm_weight(seed, n, D) if norm else None for n in ("qn", "kn"))
    cu = lambda t: None if t is None else t.to(dev())  # noqa: E731
    live = [min(s + 1, cap) for s in start]
    for b in range(B):
        cache[b, :, live[b]:] = 255
    out, st = torch.full((B, H, 1, D), math.nan, device=dev()), status()
    w = None if ring else torch.zeros(B, Hkv, cap, device=dev())
    g.gqa_attn_decode_step_q4(cu(q), cu(k), cu(v), out, cache, i32(start), max(start), rp, table,
                              cu(qn), cu(kn), pos=i32(pos), max_pos=max(pos), weights=w,
                              window=window, softcap=softcap, status=st)
    y, qr = ref.rotate(k, pos, tab, kn), ref.rotate(q, pos, tab, qn)
    for b in range(B):
        slot = start[b] % cap
        kc[b, :, slot], vc[b, :, slot] = ref.stands_for(y)[b, :, 0], ref.stands_for(v)[b, :, 0]
    want, ww, S = ref.decode(qr, kc, vc, live, softcap)
    tol = 2e-6 * (1 + S / math.log(2))
    assert value(st) == 0
    close(out, want, tol * float(vc.abs().max()))
    if w is not None:
        close(w, ww, tol * G + tol)
    got = torch.empty_like(out)
    g.gqa_attn_decode_q4(qr.float().to(dev()), cache, i32([s + 1 for s in start]), max(start) + 1, got,
                         window=window, softcap=softcap, status=st)
    assert value(st) == 0
    close(got, want, tol * float(vc.abs().max()))


def test_workspace_of_a_longer_length_serves_a_shorter_one():
    B, H, Hkv, D, cap = 3, 16, 2, 64, 4000
    cache, k, v = filled(4, B, Hkv, cap, D)
    q = syn.normal(4, "q", (B, H, 1, D))
    ws = torch.empty(g.gqa_attn_decode_q4_workspace_size(B, H, Hkv, D, cap, 0, True), dtype=torch.uint8, device=dev())
    for n in (1, 32, 513, 700, 2048, 4000):
        out, st = torch.empty(B, H, 1, D, device=dev()), status()
        w = torch.zeros(B, Hkv, cap, device=dev())
        ws.fill_(255)
        g.gqa_attn_decode_q4(q.to(dev()), cache, i32([n, max(1, n // 2), 1]), n, out, weights=w, workspace=ws, status=st)
        assert value(st) == 0
        want, ww, S = ref.decode(q, k, v, [n, max(1, n // 2), 1])
        close(out, want, 2e-6 * (1 + S / math.log(2)) * float(v.abs().max()))
        close(w, ww, 2e-6 * (1 + S / math.log(2)) * 9)


def test_binding_refuses_what_does_not_fit():
    B, H, Hkv, D, cap = 2, 4, 2, 64, 16
    d = dev()
    cache = torch.zeros(B, Hkv, cap, 80, dtype=torch.uint8, device=d)
    q, out = torch.zeros(B, H, 1, D, device=d), torch.zeros(B, H, 1, D, device=d)
    k = torch.zeros(B, Hkv, 1, D, device=d)
    cl, w = i32([1, 1]), torch.zeros(B, Hkv, cap, device=d)
    rp, table, _ = table_of(32, D, D)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=d)
    dec = lambda **x: g.gqa_attn_decode_q4(**{**dict(q=q, cache=cache, cache_len=cl, max_cache_len=4, out=out, workspace=ws), **x})  # noqa: E731
    app = lambda **x: g.kv_cache_append_q4(**{**dict(k=k, v=k, cache=cache, start=cl, max_start=1), **x})  # noqa: E731
    dec(), app()
    for bad in (dict(q=q.half()), dict(cache=cache.view(torch.int8)), dict(cache_len=cl.long()), dict(status=torch.zeros(1, device=d)),
                dict(q=None), dict(max_cache_len="4")):
        with pytest.raises(TypeError):
            dec(**bad)
    for bad in (dict(q=q.cpu()), dict(q=q[:, :2]), dict(out=out[..., :32]), dict(cache=cache[:1]), dict(cache=cache[..., :72]),
                dict(cache_len=i32([1])), dict(weights=w[:, :, :8]), dict(workspace=ws.cpu()), dict(workspace=ws[::2]),
                dict(q=torch.zeros(B, H, 2, D, device=d), out=torch.zeros(B, H, 2, D, device=d)),
                dict(status=torch.zeros(0, dtype=torch.int32, device=d))):
        with pytest.raises(ValueError):
            dec(**bad)
    for bad in (dict(v=k[:, :1]), dict(k_out=torch.zeros(B, Hkv, 2, D, device=d)), dict(pos=i32([1])),
                dict(params=rp, table=table[:10]), dict(params=rp, table=table, k_norm_w=torch.ones(32, device=d)),
                dict(k=k.transpose(0, 1))):
        with pytest.raises(ValueError):
            app(**bad)
    with pytest.raises(g.AttnError):
        dec(workspace=ws[:0], max_cache_len=17)
    with pytest.raises(g.AttnError):
        app(max_start=16)
    with pytest.raises(TypeError):
        app(params=b"no", table=table)


def test_empty_batches_are_no_ops():
    d, e = dev(), lambda *s: torch.zeros(*s, device=dev())  # noqa: E731
    cache = torch.zeros(0, 2, 8, 80, dtype=torch.uint8, device=d)
    none = torch.zeros(0, dtype=torch.int32, device=d)
    g.kv_cache_append_q4(e(0, 2, 3, 64), e(0, 2, 3, 64), cache, none, 0)
    g.kv_cache_read_q4(cache, e(0, 2, 3, 64), e(0, 2, 3, 64), none, 0)
    g.gqa_attn_decode_q4(e(0, 4, 1, 64), cache, none, 1, e(0, 4, 1, 64), workspace=e(4))
    g.kv_cache_evict_q4(cache, e(0, 2, 8), none, 8, 4, 1, cache.clone(), e(0, 2, 8),
                        torch.zeros(0, 2, 4, dtype=torch.int32, device=d), none.clone())
    full = torch.full((1, 2, 8, 80), 7, dtype=torch.uint8, device=d)
    g.kv_cache_append_q4(e(1, 2, 0, 64), e(1, 2, 0, 64), full, i32([8]), 8)
    torch.cuda.synchronize()
    assert bool((full == 7).all())


def test_calls_on_a_stream_of_their_own():
    """Every call takes a stream; without a workspace, one is kept alive until it has passed."""
    B, H, Hkv, D, cap, n = 2, 8, 2, 128, 3000, 2900
    cache, k, v = filled(21, B, Hkv, cap, D)
    q = syn.normal(1, "q", (B, H, 1, D)).to(dev())
    want = torch.empty_like(q)
    g.gqa_attn_decode_q4(q, cache, i32([n, n]), n, want)
    cl = i32([n, n])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [torch.zeros_like(q) for _ in range(20)]
    torch.cuda.synchronize()
    for o in outs:
        g.gqa_attn_decode_q4(q, cache, cl, n, o, stream=s)
        torch.empty(1 << 22, dtype=torch.uint8, device=dev()).fill_(255)   # would reuse a freed workspace
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
