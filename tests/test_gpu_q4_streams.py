"""Calls on streams other than the current one, without a workspace of the caller's: the bits
of the same call alone, whatever the current stream has queued or does next with memory of the
workspace's size."""
import pytest
import torch

import gqa_causal_attention_gb300 as g
import q4_ref as ref
from gqa_causal_attention_gb300 import synthetic as syn

from gpu_util import dev
from test_gpu_q4 import filled, i32, status, table_of, value

pytestmark = pytest.mark.gpu


def cases(n, weights):
    """(make outputs, call(outputs, stream), workspace bytes) of a decode and of a step."""
    B, H, Hkv, D, cap = 2, 8, 2, 128, n + 1
    cache, _, _ = filled(21, B, Hkv, cap, D)
    rp, table, _ = table_of(16, D, D)
    q = syn.normal(1, "q", (B, H, 1, D)).to(dev())
    k, v = (syn.normal(1, x, (B, Hkv, 1, D)).to(dev()) for x in ("k", "v"))
    zero, start, length = i32([0, 0]), i32([n, n]), i32([n, n])

    def outputs():
        return torch.zeros_like(q), torch.zeros(B, Hkv, cap, device=dev()) if weights else None

    def decode(o, stream):
        g.gqa_attn_decode_q4(q, cache, length, n, o[0], weights=o[1], stream=stream)

    def step(o, stream):
        g.gqa_attn_decode_step_q4(q, k, v, o[0], cache, start, n, rp, table, pos=zero,
                                  weights=o[1], stream=stream)

    return [(outputs, decode, g.gqa_attn_decode_q4_workspace_size(B, H, Hkv, D, n, 0, weights)),
            (outputs, step, g.gqa_attn_decode_step_q4_workspace_size(B, H, Hkv, D, n, 0, weights))]


def same(a, b):
    return torch.equal(a[0], b[0]) and (a[1] is None or torch.equal(a[1], b[1]))


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("n", [700, 3000, 30000])            # below and above 1 MB of workspace
def test_writes_still_queued_to_freed_memory_do_not_reach_a_call(n, weights):
    for outputs, call, size in cases(n, weights):
        want, got = outputs(), [outputs() for _ in range(40)]
        call(want, None)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda._sleep(2_000_000)         # about a millisecond, in which the writes pile up
        t = torch.empty(max(16, size), dtype=torch.uint8, device=dev())
        for _ in range(300):
            t.fill_(255)
        del t                                # free on the host, its writes to come
        for o in got:
            call(o, s)
        torch.cuda.synchronize()
        assert all(same(o, want) for o in got)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("n", [700, 3000, 30000])
def test_memory_taken_after_a_call_is_not_its_workspace(n, weights):
    for outputs, call, size in cases(n, weights):
        want, got = outputs(), [outputs() for _ in range(5)]
        call(want, None)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)     # the calls below wait behind this
        for o in got:
            call(o, s)
        for _ in range(100):
            torch.empty(max(16, size), dtype=torch.uint8, device=dev()).fill_(255)
        torch.cuda.synchronize()
        assert all(same(o, want) for o in got)


def test_captured_branches_that_join():
    """Two decodes on two branches of a captured stream, each with its own workspace, and behind
    the join an append, a step and a read of both results' cache; replayed on new contents."""
    B, H, Hkv, D, cap, n = 2, 8, 2, 64, 2000, 1900
    cache, k, v = filled(4, B, Hkv, cap, D)
    rp, table, tab = table_of(16, D, D)
    q = torch.empty(2, B, H, 1, D, device=dev())
    x = torch.empty(2, B, Hkv, 1, D, device=dev())
    out = torch.empty(3, B, H, 1, D, device=dev())
    kr, vr = torch.empty(B, Hkv, 2, D, device=dev()), torch.empty(B, Hkv, 2, D, device=dev())
    st, zero, at, at1, length = status(), i32([0, 0]), i32([n, n]), i32([n + 1] * 2), i32([n, n - 7])
    ws = [torch.empty(g.gqa_attn_decode_step_q4_workspace_size(B, H, Hkv, D, cap - 1),
                      dtype=torch.uint8, device=dev()) for _ in range(2)]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        side.wait_stream(main)
        g.gqa_attn_decode_q4(q[0], cache, length, cap, out[0], workspace=ws[0], status=st, stream=main)
        g.gqa_attn_decode_q4(q[1], cache, length, cap, out[1], workspace=ws[1], status=st, stream=side)
        main.wait_stream(side)
        g.kv_cache_append_q4(x[0], x[1], cache, at, n, rp, table, pos=zero, status=st, stream=main)
        g.gqa_attn_decode_step_q4(q[0], x[1], x[0], out[2], cache, at1, n + 1, rp, table, pos=zero,
                                  workspace=ws[0], status=st, stream=main)
        g.kv_cache_read_q4(cache, kr, vr, at, n, status=st, stream=main)

    q.normal_(), x.normal_()
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        work()
    for i in range(3):
        qs = [syn.normal(30 + i, m, (B, H, 1, D)) for m in ("a", "b")]
        xs = [syn.normal(30 + i, m, (B, Hkv, 1, D)) for m in ("k", "v")]
        q.copy_(torch.stack(qs)), x.copy_(torch.stack(xs))
        graph.replay()
        assert value(st) == 0
        for j in range(2):
            want, _, S = ref.decode(qs[j], k, v, [n, n - 7])
            assert (out[j].cpu().double() - want).abs().max() <= 2e-6 * (1 + 1.45 * S) * v.abs().max()
        a, b = (ref.stands_for(t) for t in xs)
        assert torch.equal(kr.cpu().double(), torch.cat([a, b], 2))
        assert torch.equal(vr.cpu().double(), torch.cat([b, a], 2))
        k2, v2 = torch.cat([k[:, :, :n], a, b], 2), torch.cat([v[:, :, :n], b, a], 2)
        want, _, S = ref.decode(qs[0], k2, v2, [n + 2] * 2)
        assert (out[2].cpu().double() - want).abs().max() <= 2e-6 * (1 + 1.45 * S) * v2.abs().max()


def test_captured_calls_on_branches_take_workspaces_of_their_own():
    """Decodes without a workspace on two branches of a captured stream, several on each."""
    B, H, Hkv, D, n = 2, 8, 2, 64, 3000
    cache, k, v = filled(5, B, Hkv, n, D)
    q = torch.stack([syn.normal(i, "q", (B, H, 1, D)) for i in range(6)]).to(dev())
    want, out = torch.empty_like(q), torch.zeros_like(q)
    length = i32([n, n - 5])
    for i in range(6):
        g.gqa_attn_decode_q4(q[i], cache, length, n, want[i])
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        for i in range(6):
            g.gqa_attn_decode_q4(q[i], cache, length, n, out[i], stream=side if i % 2 else None)
        main.wait_stream(side)
    for _ in range(5):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
