"""The 4-bit KV cache calls on the host: what they refuse before anything is launched, their
workspace sizes, and the reference's own record format. No GPU is touched."""
import ctypes
import math

import pytest
import torch

import gqa_causal_attention_gb300 as g
import q4_ref as ref

no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="stand-in pointers are only used without a device")
P, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)
OK, NULL, SHAPE, POSITION, CAPACITY, WORKSPACE, ALIGN, PARAM = 0, -1, -2, -3, -4, -5, -6, -7


def rp(**kw):
    return ctypes.byref(g.RopeParams.make(**{"max_positions": 100, **kw}))


def test_record_bytes():
    assert [g.kv_q4_record_bytes(d) for d in (32, 64, 96, 128, 160, 192, 224, 256)] == \
        [ref.record_bytes(d) for d in range(32, 257, 32)] == [48, 80, 112, 144, 192, 224, 256, 288]
    assert [g.kv_q4_record_bytes(d) for d in (0, -32, 16, 48, 130, 288)] == [0] * 6


@pytest.mark.parametrize("D", [32, 96, 128, 256])
def test_reference_records_round_trip(D):
    gen = torch.Generator().manual_seed(D)
    k, v = torch.randn(3, 5, D, generator=gen), torch.randn(3, 5, D, generator=gen)
    v[0, 0, :32] = 0
    k2, v2 = ref.unpack(ref.pack(k, v), D)
    assert torch.equal(k2, ref.stands_for(k)) and torch.equal(v2, ref.stands_for(v))
    # half a step of the group's scale, which bf16 holds to 2^-8
    step = k.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True).double() / 7 * (1 + 2 ** -8)
    assert ((k2 - k.double()).unflatten(-1, (-1, 32)).abs() <= step * 0.51).all()


def test_reference_scale_rounding():
    x = torch.tensor([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1.7 * 2.0 ** -130, 0.0, 2.0 ** -134,
                      3 * 2.0 ** -134], dtype=torch.float64)
    want = [1.0, 1.0, 1 + 4 * 2.0 ** -8, 14 * 2.0 ** -133, 0.0, 0.0, 2.0 ** -132]
    assert ref.round_bf16(x).tolist() == want


Q = ctypes.c_void_p(64 << 20)


def append(k=P, v=P, k_out=None, B=2, Hkv=2, L=3, D=64, start=P, max_start=0, pos=None, max_pos=0,
           params=None, table=None, norm=None, eps=1e-6, cache=P, cap=16, window=0):
    return g.load().kv_cache_append_q4(k, v, k_out, B, Hkv, L, D, start, max_start, pos, max_pos,
                                       params, table, norm, eps, cache, cap, window, None, None)


@no_device
@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(D=48)), (SHAPE, dict(D=288)), (SHAPE, dict(D=16)), (SHAPE, dict(L=-1)),
    (SHAPE, dict(Hkv=0)), (SHAPE, dict(cap=0)), (SHAPE, dict(window=-1)), (SHAPE, dict(window=8)),
    (SHAPE, dict(B=1 << 20)), (OK, dict(B=0)), (OK, dict(L=0)),
    (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(start=None)), (NULL, dict(cache=None)),
    (NULL, dict(params=rp())), (PARAM, dict(table=P)), (PARAM, dict(norm=P)),
    (PARAM, dict(params=rp(rope_dim=3), table=P)), (PARAM, dict(params=rp(), table=P, eps=math.nan)),
    (POSITION, dict(max_start=-1)), (POSITION, dict(params=rp(), table=P, max_start=98, cap=200)),
    (POSITION, dict(params=rp(), table=P, pos=P, max_pos=98)), (POSITION, dict(pos=P, max_pos=-1)),
    (POSITION, dict(max_start=0x7fffffff, window=16)),
    (CAPACITY, dict(max_start=14)), (CAPACITY, dict(L=17)),
    (ALIGN, dict(k=ODD)), (ALIGN, dict(v=ODD)), (ALIGN, dict(cache=ODD)), (ALIGN, dict(k_out=ODD)),
    (ALIGN, dict(params=rp(), table=ODD)), (ALIGN, dict(params=rp(), table=P, norm=ODD)),
    # k_out one row into k, v itself, or ending inside v
    (PARAM, dict(v=Q, k_out=ctypes.c_void_p((1 << 20) + 256))), (PARAM, dict(v=Q, k_out=Q)),
    (PARAM, dict(v=Q, k_out=ctypes.c_void_p((64 << 20) - 256))),
])
def test_append_refusals(want, kw):
    assert append(**kw) == want


@no_device
@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(D=40)), (SHAPE, dict(window=8)), (SHAPE, dict(window=16, L=17)), (SHAPE, dict(cap=0)),
    (OK, dict(B=0)), (OK, dict(L=0)), (NULL, dict(cache=None)), (NULL, dict(k=None)),
    (NULL, dict(v=None)), (NULL, dict(start=None)), (POSITION, dict(max_start=-1)),
    (CAPACITY, dict(max_start=14)), (ALIGN, dict(cache=ODD)), (ALIGN, dict(k=ODD)), (ALIGN, dict(v=ODD)),
])
def test_read_refusals(want, kw):
    a = {**dict(cache=P, cap=16, window=0, k=P, v=P, B=2, Hkv=2, L=3, D=64, start=P, max_start=0), **kw}
    assert g.load().kv_cache_read_q4(a["cache"], a["cap"], a["window"], a["k"], a["v"], a["B"],
                                     a["Hkv"], a["L"], a["D"], a["start"], a["max_start"], None,
                                     None) == want


@no_device
@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(D=100)), (SHAPE, dict(H=5)), (SHAPE, dict(Hkv=0)), (SHAPE, dict(window=64)),
    (SHAPE, dict(window=4000, w=P)), (SHAPE, dict(n=0)), (SHAPE, dict(B=1 << 19)),
    (PARAM, dict(softcap=math.inf)), (PARAM, dict(scale=math.nan)), (OK, dict(B=0)),
    (CAPACITY, dict(n=4001)), (NULL, dict(q=None)), (NULL, dict(cache=None)), (NULL, dict(cl=None)),
    (NULL, dict(out=None)), (ALIGN, dict(q=ODD)), (ALIGN, dict(cache=ODD)), (ALIGN, dict(out=ODD)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(wsb=100)), (ALIGN, dict(ws=ODD)),
    (WORKSPACE, dict(n=20, w=P, wsb=8)),
])
def test_decode_refusals(want, kw):
    a = {**dict(q=P, cache=P, cl=P, n=4000, out=P, w=None, B=1, H=8, Hkv=2, D=64, cap=4000, window=0,
                softcap=0.0, scale=0.0, ws=P, wsb=1 << 40), **kw}
    assert g.load().gqa_attn_decode_q4(a["q"], a["cache"], a["cl"], a["n"], a["out"], a["w"], a["B"],
                                       a["H"], a["Hkv"], a["D"], a["cap"], a["window"], a["softcap"],
                                       a["scale"], a["ws"], a["wsb"], None, None) == want


@no_device
@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(D=36)), (SHAPE, dict(H=5)), (SHAPE, dict(window=64)), (SHAPE, dict(window=99, w=P)),
    (NULL, dict(params=None)), (PARAM, dict(params=rp(theta=0.0))), (PARAM, dict(eps=-1.0)),
    (PARAM, dict(softcap=math.nan)), (OK, dict(B=0)), (NULL, dict(q=None)), (NULL, dict(k=None)),
    (NULL, dict(v=None)), (NULL, dict(out=None)), (NULL, dict(start=None)), (NULL, dict(table=None)),
    (NULL, dict(cache=None)), (POSITION, dict(max_start=-1)), (CAPACITY, dict(max_start=99)),
    (POSITION, dict(max_start=100, cap=200)), (POSITION, dict(pos=P, max_pos=100)),
    (ALIGN, dict(q=ODD)), (ALIGN, dict(table=ODD)), (ALIGN, dict(qn=ODD)), (ALIGN, dict(kn=ODD)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(wsb=64)), (ALIGN, dict(ws=ODD)),
])
def test_step_refusals(want, kw):
    a = {**dict(q=P, k=P, v=P, out=P, B=1, H=8, Hkv=2, D=64, start=P, max_start=98, pos=None,
                max_pos=0, params=rp(), table=P, qn=None, kn=None, eps=1e-6, cache=P, w=None, cap=99,
                window=0, softcap=0.0, ws=P, wsb=1 << 40), **kw}
    assert g.load().gqa_attn_decode_step_q4(
        a["q"], a["k"], a["v"], a["out"], a["B"], a["H"], a["Hkv"], a["D"], a["start"],
        a["max_start"], a["pos"], a["max_pos"], a["params"], a["table"], a["qn"], a["kn"], a["eps"],
        a["cache"], a["w"], a["cap"], a["window"], a["softcap"], 0.0, a["ws"], a["wsb"], None,
        None) == want


def at(mib, offset=0):
    return ctypes.c_void_p((mib << 20) + offset)


P2, P3, P4 = at(2), at(3), at(4)


@no_device
@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(D=8)), (SHAPE, dict(budget=0)), (SHAPE, dict(recent=-1)), (SHAPE, dict(recent=9)),
    (SHAPE, dict(n=-1)), (SHAPE, dict(n=(1 << 30) + 1, cap=1 << 30)), (SHAPE, dict(B=70000, Hkv=1)), (OK, dict(B=0)), (CAPACITY, dict(n=21)),
    (CAPACITY, dict(cap_out=7)), (NULL, dict(cache=None)), (NULL, dict(w=None)), (NULL, dict(cl=None)),
    (NULL, dict(out=None)), (NULL, dict(w_out=None)), (NULL, dict(index=None)),
    (NULL, dict(len_out=None)), (PARAM, dict(out=P)), (PARAM, dict(w_out=P2)), (PARAM, dict(len_out=P3)),
    # outputs that begin or end inside an input (3200 bytes of records, 160 of weights)
    (PARAM, dict(out=at(1, 3184))), (PARAM, dict(out=at(1, -16))), (PARAM, dict(w_out=at(2, 156))),
    (PARAM, dict(index=at(2, -4))), (PARAM, dict(len_out=at(1, 0))), (PARAM, dict(index=at(3, 0))),
    (ALIGN, dict(cache=ODD)), (ALIGN, dict(out=ODD)),
])
def test_evict_refusals(want, kw):
    a = {**dict(cache=P, w=P2, cl=P3, n=20, budget=8, recent=2, out=P4, w_out=P4, index=P4, len_out=P4,
                B=1, Hkv=2, D=64, cap=20, cap_out=8), **kw}
    assert g.load().kv_cache_evict_q4(a["cache"], a["w"], a["cl"], a["n"], a["budget"], a["recent"],
                                      a["out"], a["w_out"], a["index"], a["len_out"], a["B"], a["Hkv"],
                                      a["D"], a["cap"], a["cap_out"], None, None) == want


def test_workspace_sizes_never_shrink():
    for B, H, Hkv, D, w in ((1, 8, 8, 128, 0), (1, 64, 8, 128, 1), (64, 32, 8, 128, 0), (3, 12, 1, 96, 1)):
        for f in (g.gqa_attn_decode_q4_workspace_size, g.gqa_attn_decode_step_q4_workspace_size):
            last = 0
            for n in list(range(1, 600, 7)) + [2 ** i + d for i in range(10, 21) for d in (-1, 0, 1)]:
                size = f(B, H, Hkv, D, n, 0, bool(w))
                assert size >= last
                last = size
    assert g.gqa_attn_decode_q4_workspace_size(1, 8, 2, 64, 20) == 0
    for bad in ((0, 8, 8, 128, 10), (1, 8, 3, 128, 10), (1, 8, 8, 100, 10), (1, 8, 8, 128, 0)):
        assert g.gqa_attn_decode_q4_workspace_size(*bad) == 0
    assert g.gqa_attn_decode_step_q4_workspace_size(1, 8, 8, 128, -1) == 0
    # a ring's size is that of its slots
    assert g.gqa_attn_decode_q4_workspace_size(1, 8, 8, 128, 99999, 4096) == \
        g.gqa_attn_decode_q4_workspace_size(1, 8, 8, 128, 4096)


def test_binding_refuses_host_tensors():
    k = torch.zeros(1, 2, 3, 64)
    cache = torch.zeros(1, 2, 8, 80, dtype=torch.uint8)
    start = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        g.kv_cache_append_q4(k.half(), k, cache, start, 0)
    with pytest.raises(ValueError):
        g.kv_cache_append_q4(k, k, cache, start, 0)
