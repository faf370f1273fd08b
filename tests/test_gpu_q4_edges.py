"""The 4-bit KV cache at the ends of its ranges: values of any magnitude, weights held to their
own size. Reference: q4_ref, in 64 bits.

Outputs here are held to their own weighted sums, A = sum p |v|, at scores of S <= 1/2 (log2
units): a score is off by at most 12 * 2^-23 of its terms' magnitudes (as in test_gpu_q4),
which are under 1/2, so p by 12 * 2^-23 / 2 * ln 2 + 2^-22 (the exponential) = 7.4e-7, numerator
and denominator each; p times a scale is split into 22 bits, 2^-23; sums of at most 10 tiles a
warp, 16 warps and 10 splits, each step 2^-24 of A, 2.2e-6. Together 3.9e-6 A; 4e-6 A is the
bound."""
import math

import pytest
import torch

import gqa_causal_attention_gb300 as g
import q4_ref as ref
from gqa_causal_attention_gb300 import synthetic as syn

from gpu_util import dev
from test_gpu_q4 import filled, i32, status, table_of, value

pytestmark = pytest.mark.gpu


def quiet(seed, B, H, Hkv, D, n, vmul):
    """A cache whose scores stay within 1/2, its values (normal) times vmul: (q, cache, k, v)."""
    cache, k, v = filled(seed, B, Hkv, n, D, (0.03, vmul))
    q = syn.normal(seed + 1, "q", (B, H, 1, D)).clamp(-2, 2)
    return q, cache, k, v


def held(q, cache, k, v, lens):
    """Decode with and without weights against the reference, each within 4e-6 of its own size."""
    B, H, _, D = q.shape
    Hkv, n = k.shape[1:3]
    want, ww, S = ref.decode(q, k, v, lens)
    size, _, _ = ref.decode(q, k, v.abs(), lens)
    assert S <= 0.5 / math.log2(math.e)
    for weights in (None, torch.zeros(B, Hkv, n, device=dev())):
        out, st = torch.full((B, H, 1, D), math.nan, device=dev()), status()
        g.gqa_attn_decode_q4(q.to(dev()), cache, i32(lens), n, out, weights=weights, status=st)
        assert value(st) == 0
        # fp32's own last bit, below 2^-126
        err = ((out.cpu().double() - want).abs() - 2.0 ** -149) / size.clamp(min=1e-300)
        assert bool(out.isfinite().all()) and float(err.max()) <= 4e-6, float(err.max())
        if weights is not None:
            err = (weights.cpu().double() - ww).abs() - 4e-6 * ww      # 0 behind the live slots
            assert float(err.max()) <= 0, float(err.max())


@pytest.mark.parametrize("D,G,n", [(64, 4, 333), (128, 8, 300), (256, 2, 200)])
@pytest.mark.parametrize("vmag", [1e-37, 1e-35, 1e-30, 1e-27, 1e-25, 1.0, 1e20, 1e30, 1e36, 4e37])
def test_decode_keeps_fp32_accuracy_of_values_of_any_magnitude(vmag, D, G, n):
    held(*quiet(D, 1, 2 * G, 2, D, n, vmag), [n])


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("early,late", [(0.0, 1e25), (1e25, 0.0), (1e-30, 1e25), (1e-35, 1e35), (1e35, 1e-35)])
@pytest.mark.parametrize("n", [300, 3000])
def test_decode_of_values_that_change_magnitude(n, early, late, one_sign):
    """Slots of one magnitude, then of another, up to 2^232 apart: those of the smaller values
    keep their share of the softmax. With one sign the values' sum is past fp32's largest number."""
    vmul = torch.full((1, 1, n, 1), early)
    vmul[:, :, n // 2:] = late
    if one_sign:
        vmul = vmul * torch.where(syn.normal(n, "v", (2, 2, n, 64)) < 0, -1.0, 1.0)
    q, cache, k, v = quiet(n, 2, 8, 2, 64, n, vmul)
    held(q, cache, k, v, [n, n - 1])


def sorted_keep(w, n, budget, recent):
    """The kept slots of one head's n live ones, in order (no NaN among the weights)."""
    old = n - recent
    first = torch.sort(w[:old], descending=True, stable=True).indices[:budget - recent]
    return torch.cat([first.sort().values, torch.arange(old, n, device=w.device)])


@pytest.mark.parametrize("B,cap,n,budget,recent", [
    (64, 65536, 65000, 300, 10),             # 512 heads: two kernels, keys reread from memory
    (1, 4200000, 4199999, 4100000, 1000),    # 8 heads, several blocks each if the shares fit
    (1, 4200000, 4100001, 70000, 0),
])
def test_evict_far_into_large_caches(B, cap, n, budget, recent):
    """Records past 2^32 bytes from the start of the cache, and of the output where it is as large."""
    Hkv, D, cap_out = 8, 128, cap
    d = dev()
    cache = torch.full((B, Hkv, cap, 144), 255, dtype=torch.uint8, device=d)
    cache[B - 1].random_(0, 256)
    w = torch.rand(B, Hkv, cap, device=d).mul_(1 << 12).floor_()      # ties throughout
    out = torch.full((B, Hkv, cap_out, 144), 9, dtype=torch.uint8, device=d)
    w_out = torch.full((B, Hkv, cap_out), math.nan, device=d)
    index = torch.empty(B, Hkv, budget, dtype=torch.int32, device=d)
    n_out, st = i32([-7] * B), status()
    g.kv_cache_evict_q4(cache, w, i32([0] * (B - 1) + [n]), cap, budget, recent, out, w_out, index,
                        n_out, status=st)
    assert value(st) == 0 and n_out.tolist() == [0] * (B - 1) + [budget]
    assert bool((index[:-1] == -1).all()) and bool((w_out[:-1] == 0).all())
    for h in (0, 3, Hkv - 1):
        keep = sorted_keep(w[B - 1, h], n, budget, recent)
        assert torch.equal(index[B - 1, h].long(), keep)
        assert torch.equal(w_out[B - 1, h, :budget], w[B - 1, h, keep])
        assert torch.equal(out[B - 1, h, :budget], cache[B - 1, h, keep])
        assert bool((w_out[B - 1, h, budget:] == 0).all()) and bool((out[B - 1, h, budget:] == 9).all())


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("B,H,Hkv,D,lens,softcap", [
    (1, 8, 1, 128, (20000,), 0.0), (2, 32, 8, 128, (700, 129), 0.0), (1, 32, 2, 64, (5000,), 30.0),
    (3, 4, 4, 96, (1, 33, 500), 0.0), (1, 10, 1, 256, (3001,), 0.0),
])
def test_weights_are_held_to_their_own_size(B, H, Hkv, D, lens, softcap, step):
    """Eviction ranks slots by these, so each is held to the outputs' bound (test_gpu_q4) times
    itself, however small; and every kv head's new weights sum to its query heads. (That sum
    differs by the exponentials' 2^-22, taken once for the sums and once for the weights, their
    arguments' rounding, 2^-20 ln 2 below 2^5, and the sums' own: under 3e-6 of it.)"""
    n, G = max(lens), H // Hkv
    cache, k, v = filled(H + D, B, Hkv, n, D)
    q = syn.normal(D, "q", (B, H, 1, D))
    out, st = torch.empty(B, H, 1, D, device=dev()), status()
    w = torch.zeros(B, Hkv, n, device=dev())
    if step:                                 # the last slot enters again, at position 0
        rp, table, _ = table_of(16, D, D)
        at = [x - 1 for x in lens]
        new = [syn.normal(7, name, (B, Hkv, 1, D)) for name in ("k", "v")]
        g.gqa_attn_decode_step_q4(q.to(dev()), new[0].to(dev()), new[1].to(dev()), out, cache,
                                  i32(at), n - 1, rp, table, pos=i32([0] * B), weights=w,
                                  softcap=softcap, status=st)
        for b in range(B):
            k[b, :, at[b]], v[b, :, at[b]] = (ref.stands_for(x)[b, :, 0] for x in new)
    else:
        g.gqa_attn_decode_q4(q.to(dev()), cache, i32(lens), n, out, weights=w, softcap=softcap,
                             status=st)
    assert value(st) == 0
    _, ww, S = ref.decode(q, k, v, lens, softcap)
    got = w.cpu().double()
    err = (got - ww).abs() - 2e-6 * (1 + S / math.log(2)) * ww
    assert float(err.max()) <= 2.0 ** -126
    assert float((got.sum(-1) / G - 1).abs().max()) <= 1e-5


@pytest.mark.parametrize("kmag,qmag", [(2e31, 5e-33), (1e20, 1e-21), (1e-10, 1e9), (1e-36, 1e35)])
def test_decode_keeps_fp32_accuracy_of_keys_of_any_magnitude(kmag, qmag):
    """Keys up to 1e32 in magnitude, queries to match (scores within 1/2)."""
    B, H, Hkv, D, n = 1, 8, 2, 64, 333
    cache, k, v = filled(8, B, Hkv, n, D, (kmag, 1.0))
    q = syn.normal(9, "q", (B, H, 1, D)).clamp(-2, 2) * (0.3 * qmag)
    assert float(k.abs().max()) <= 1e32
    held(q, cache, k, v, [n])
