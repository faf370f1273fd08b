"""The 16-bit paged calls on the host: what is refused before anything is enqueued, and the
workspaces (stand-in pointers, so only where no CUDA device is visible)."""
import ctypes

import pytest
import torch

import gqa_causal_attention_gb300 as g

no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="stand-in pointers are only used without a device")
P = 0x10000                                       # 16-byte aligned, never read
B, H, HKV, D, PAGE, PAGES, WIDTH = 3, 8, 2, 64, 16, 40, 8


def rows(p=P, token=None, head=None, heads=H, d=D):
    return g.Rows(p, heads * d if token is None else token, d if head is None else head)


def cache(k=P, v=P, stride=None, pages=PAGES, page=PAGE, d=D):
    return g.PagedKv(k, v, HKV * page * d if stride is None else stride, pages, page)


def ref(x):
    return None if x is None else ctypes.byref(x)


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def append(type=2, q=rows(), q_out=rows(), k=rows(heads=HKV), k_out=None, v=rows(heads=HKV), T=7,
           b=B, h=H, hkv=HKV, d=D, cu=P, start=P, max_pos=100, rp="default", table=P, qn=None,
           kn=None, eps=1e-6, kv=cache(), bt=P, width=WIDTH):
    rp = g.RopeParams.make(max_positions=128) if rp == "default" else rp
    return g.load().kv_cache_append_paged(
        type, ref(q), ref(q_out), ref(k), ref(k_out), ref(v), T, b, h, hkv, d, vp(cu), vp(start),
        max_pos, ref(rp), vp(table), vp(qn), vp(kn), eps, ref(kv), vp(bt), width, None, None)


def decode(type=1, q=rows(), kv=cache(), bt=P, width=WIDTH, lens=P, max_len=100, out=rows(), b=B, h=H,
           hkv=HKV, d=D, window=0, softcap=0.0, scale=0.0, ws=P, wbytes=1 << 30):
    return g.load().gqa_attn_decode_paged(type, ref(q), ref(kv), vp(bt), width, vp(lens), max_len,
                                          ref(out), b, h, hkv, d, window, softcap, scale, vp(ws),
                                          wbytes, None, None)


def shared(type=1, q=rows(), kv=cache(), pt=P, pwidth=WIDTH, prefix=100, bt=P, width=WIDTH, lens=P,
           max_len=100, out=rows(), b=B, h=H, hkv=HKV, d=D, softcap=0.0, scale=0.0, ws=P,
           wbytes=1 << 30):
    return g.load().gqa_attn_decode_shared(type, ref(q), ref(kv), vp(pt), pwidth, prefix, vp(bt),
                                           width, vp(lens), max_len, ref(out), b, h, hkv, d, softcap,
                                           scale, vp(ws), wbytes, None, None)


def prefill(type=2, q=rows(), k=rows(heads=HKV), v=rows(heads=HKV), cu=P, max_len=50, out=rows(), T=99,
            b=B, h=H, hkv=HKV, d=D, window=0, softcap=0.0, scale=0.0):
    return g.load().gqa_attn_prefill_packed(type, ref(q), ref(k), ref(v), vp(cu), max_len, ref(out), T,
                                            b, h, hkv, d, window, softcap, scale, None, None)


NULL, SHAPE, POSITION, CAPACITY, WORKSPACE, ALIGN, PARAM = range(-1, -8, -1)
nan, inf = float("nan"), float("inf")

ROWS = [                                          # what every call says of a tensor's rows
    (dict(p=None), NULL), (dict(p=P + 8), ALIGN), (dict(token=H * D + 4), ALIGN),
    (dict(head=D + 4), ALIGN), (dict(token=D - 8), SHAPE), (dict(head=D - 8), SHAPE),
    (dict(token=0), SHAPE), (dict(head=1 << 39), SHAPE),
]
CACHES = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=P + 2), ALIGN), (dict(v=P + 2), ALIGN),
    (dict(stride=HKV * PAGE * D - 8), SHAPE), (dict(stride=HKV * PAGE * D + 4), ALIGN),
    (dict(pages=0), SHAPE), (dict(page=8), SHAPE), (dict(page=24), SHAPE), (dict(page=2048), SHAPE),
]
SIZES = [
    (dict(type=0), SHAPE), (dict(type=3), SHAPE), (dict(d=12), SHAPE), (dict(d=136), SHAPE),
    (dict(d=8), SHAPE), (dict(h=7), SHAPE), (dict(hkv=0), SHAPE), (dict(h=0), SHAPE),
    (dict(h=258, hkv=2), SHAPE), (dict(b=-1), SHAPE),
]


@no_device
@pytest.mark.parametrize("call,tensors", [(append, ("q", "q_out", "k", "v")), (decode, ("q", "out")),
                                          (shared, ("q", "out")), (prefill, ("q", "k", "v", "out"))])
def test_sizes_rows_and_caches_are_checked(call, tensors):
    for kw, code in SIZES:
        assert call(**kw) == code, kw
    for name in tensors:
        heads = HKV if name in ("k", "v") else H
        for kw, code in ROWS:
            if kw.get("token") == H * D + 4:
                kw = dict(token=heads * D + 4)
            assert call(**{name: rows(heads=heads, **kw)}) == code, (name, kw)
    for name in tensors:                          # rows that overlap: an input may, an output may not
        over = rows(token=D, head=D)
        if name in ("q_out", "out"):
            assert call(**{name: over}) == PARAM
    if call is not prefill:
        for kw, code in CACHES:
            assert call(kv=cache(**kw)) == code, kw
        assert call(kv=None) == NULL and call(bt=None) == NULL and call(width=0) == SHAPE


@no_device
def test_append_refusals():
    assert append(k=None) == NULL and append(v=None) == NULL and append(start=None) == NULL
    assert append(q=None) == NULL and append(q_out=None) == NULL
    assert append(k_out=rows(P + 4, heads=HKV)) == ALIGN
    assert append(T=-1) == SHAPE and append(cu=None) == SHAPE          # one token each: T == B
    assert append(T=1 << 28) == SHAPE
    assert append(max_pos=-1) == POSITION and append(max_pos=128) == POSITION
    assert append(rp=None, table=None, max_pos=128) == CAPACITY        # 8 pages of 16
    assert append(table=None) == NULL and append(rp=None) == PARAM
    assert append(rp=None, table=None, kn=P) == PARAM
    assert append(rp=g.RopeParams.make(rope_dim=D + 2)) == PARAM
    assert append(rp=g.RopeParams.make(theta=0.0)) == PARAM
    assert append(eps=-1.0) == PARAM and append(eps=nan) == PARAM
    assert append(table=P + 4) == ALIGN and append(kn=P + 4) == ALIGN and append(qn=P + 4) == ALIGN
    assert append(q=None, q_out=None, qn=P) == PARAM
    assert append(T=0) == 0 and append(b=0) == 0                       # nothing to do


@no_device
@pytest.mark.parametrize("call", [decode, shared])
def test_decode_refusals(call):
    assert call(lens=None) == NULL and call(max_len=-1) == SHAPE
    assert call(max_len=WIDTH * PAGE + 1) == CAPACITY
    assert call(softcap=inf) == PARAM and call(scale=nan) == PARAM
    assert call(b=1 << 22) == SHAPE
    assert call(b=0) == 0


@no_device
def test_workspaces_are_checked_and_do_not_shrink():
    size = g.gqa_attn_decode_paged_workspace_size
    wide = dict(width=1 << 20, max_len=5000)
    need = size(B, H, HKV, D, 5000)
    assert need > 0
    assert decode(ws=None, **wide) == WORKSPACE and decode(wbytes=need - 1, **wide) == WORKSPACE
    assert decode(ws=P + 8, **wide) == ALIGN
    assert decode(window=-1) == SHAPE
    for b, h, hkv in ((1, 32, 8), (64, 32, 8), (3, 128, 1), (9000, 8, 8)):
        for window in (0, 5, 900, 5000):
            sizes = [size(b, h, hkv, 128, n, window) for n in range(0, 9000, 7)]
            sizes += [size(b, h, hkv, 128, n, window) for n in (1 << 20, 1 << 30)]
            assert sizes == sorted(sizes)
    size = g.gqa_attn_decode_shared_workspace_size
    for b, prefix in ((2, 50), (5, 2001), (64, 8192), (500, 100000)):
        sizes = [size(b, 32, 8, 128, prefix, n) for n in range(0, 3000, 13)]
        assert sizes == sorted(sizes)
    assert size(64, 32, 8, 128, 0, 5) == 0 and size(64, 31, 8, 128, 9, 5) == 0
    need = size(64, H, HKV, D, 20000, 100)
    big = dict(b=64, prefix=20000, pwidth=1 << 20)
    assert shared(ws=None, **big) == WORKSPACE and shared(wbytes=need - 1, **big) == WORKSPACE
    assert shared(ws=P + 8, **big) == ALIGN


@no_device
def test_workspaces_of_larger_batches_serve_smaller_ones():
    size = g.gqa_attn_decode_paged_workspace_size
    for h, hkv, d, n in ((32, 8, 128, 2000), (32, 8, 128, 1000), (16, 4, 64, 4000), (8, 1, 40, 300)):
        sizes = [size(b, h, hkv, d, n) for b in (1, 2, 5, 19, 20, 56, 57, 58, 100, 200, 8192, 8193, 20000)]
        assert sizes == sorted(sizes)


@no_device
def test_shared_refusals():
    assert shared(pt=None) == NULL
    assert shared(prefix=0) == SHAPE and shared(prefix=-3) == SHAPE and shared(pwidth=0) == SHAPE
    assert shared(prefix=WIDTH * PAGE + 1) == CAPACITY


@no_device
def test_prefill_refusals():
    assert prefill(cu=None) == NULL and prefill(T=-1) == SHAPE and prefill(max_len=-1) == SHAPE
    assert prefill(window=-1) == SHAPE and prefill(softcap=nan) == PARAM and prefill(scale=inf) == PARAM
    assert prefill(T=1 << 30) == SHAPE
    assert prefill(T=0) == 0 and prefill(b=0) == 0


def test_binding_refuses_tensors_that_do_not_fit():
    x = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 8, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        g.gqa_attn_prefill_packed(x, x, x, i, 3, x)
    with pytest.raises(TypeError, match="float16 or torch.bfloat16"):
        g.gqa_attn_prefill_packed(x.float(), x, x, i, 3, x)
    with pytest.raises(TypeError, match="None"):
        g.gqa_attn_prefill_packed(None, x, x, i, 3, x)
    with pytest.raises(ValueError, match="CUDA"):
        g.gqa_attn_decode_paged(x, pool, pool, i[:, None], i, 16, x, workspace=x)
    with pytest.raises(ValueError, match="CUDA"):
        g.kv_cache_append_paged(x, x, pool, pool, i[:, None], i, 3)
    with pytest.raises(ValueError, match="CUDA"):
        g.gqa_attn_decode_shared(x, pool, pool, i, 5, i[:, None], i, 3, x, workspace=x)
