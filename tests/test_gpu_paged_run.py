"""16-bit paged serving as a program uses it: prompts appended and attended, then tokens decoded, on
streams and in graphs, with the finite check, and in pools past 2^32 elements."""
import pytest
import torch

import gqa_causal_attention_gb300 as g
from paged_ref import (Cache, attend, attend_tol, check, dev, gen, half_step, i32, normal, rope, rotate,
                       rows, status)

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("t,H,Hkv,D,page,window,softcap", [
    (BF, 8, 2, 128, 16, 0, 0.0), (FP, 6, 2, 64, 32, 40, 30.0), (BF, 4, 4, 80, 16, 0, 0.0),
])
def test_prompts_then_tokens(t, H, Hkv, D, page, window, softcap):
    """Three prompts enter, packed; then four tokens each. Every output against the whole history in
    64 bits, from the raw inputs: the library's rounded keys and queries stand for themselves."""
    gn, B, steps = gen(31), 3, 4
    lens = [50, 1, 131]
    qkv = H + 2 * Hkv
    c = Cache(gn, 40, Hkv, page, D, t)
    table = c.table([n + steps for n in lens])
    rp, tab, tab3 = rope(D, D, 200, 5e5)
    qn, kn = 1 + 0.1 * normal(gn, (D,)), 1 + 0.1 * normal(gn, (D,))
    st = status()
    cu = [0, 50, 51, 182]
    x = normal(gn, (cu[-1], qkv, D), t)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    qr, kr, out = (torch.empty(cu[-1], h, D, dtype=t, device=dev()) for h in (H, Hkv, H))
    g.kv_cache_append_paged(k, v, c.k, c.v, table, i32([0] * B), max(lens) - 1, rp, tab, kn, 1e-6,
                            cu_seqlens=i32(cu), q=q, q_out=qr, q_norm_w=qn, k_out=kr, status=st)
    g.gqa_attn_prefill_packed(qr, kr, v, i32(cu), max(lens), out, window=window, softcap=softcap,
                              status=st)
    hist = []
    for b, n in enumerate(lens):
        at = slice(cu[b], cu[b + 1])
        yk, _ = rotate(k[at], torch.arange(n, device=dev()), tab3, kn, 1e-6)
        assert ((kr[at].double() - yk).abs() <= half_step(t) * yk.abs() * 1.01 + 1e-5).all()
        i = torch.arange(n, device=dev())
        seen = i <= i[:, None]
        if window:
            seen &= i > i[:, None] - window
        o, vabs, unsure = attend(qr[at], kr[at], v[at], seen, softcap)
        check(out[at], o, attend_tol(o, vabs, unsure, t, True), f"prompt {b}")
        hist.append((kr[at].clone(), v[at].clone()))
    for s in range(steps):
        x = normal(gn, (B, qkv, D), t)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        pos = [n + s for n in lens]
        qr, kr, out = (torch.empty(B, h, D, dtype=t, device=dev()) for h in (H, Hkv, H))
        g.kv_cache_append_paged(k, v, c.k, c.v, table, i32(pos), max(pos), rp, tab, kn, 1e-6, q=q,
                                q_out=qr, q_norm_w=qn, k_out=kr, status=st)
        g.gqa_attn_decode_paged(qr, c.k, c.v, table, i32([p + 1 for p in pos]), max(pos) + 1, out,
                                window=window, softcap=softcap, status=st)
        for b in range(B):
            hist[b] = tuple(torch.cat([a, n[b:b + 1]]) for a, n in zip(hist[b], (kr, v)))
            n = hist[b][0].shape[0]
            seen = torch.arange(n, device=dev())[None] >= (n - window if window else 0)
            o, vabs, unsure = attend(qr[b][None], *hist[b], seen, softcap)
            check(out[b], o[0], attend_tol(o, vabs, unsure, t, False)[0], f"step {s} row {b}")
    assert st.item() == 0


def test_samples_of_one_prompt_share_its_pages():
    """The prompt is appended once; its samples decode over it, by the shared call and, with its pages
    in every sample's own table, by the plain one."""
    gn, t, B, H, Hkv, D, page, P = gen(7), BF, 24, 32, 8, 128, 16, 2560
    c = Cache(gn, P // page + 2 * B, Hkv, page, D, t)
    ptab = c.table([P], extra=0)[0].contiguous()
    k, v = rows(gn, P, Hkv, D, t), rows(gn, P, Hkv, D, t)
    g.kv_cache_append_paged(k, v, c.k, c.v, ptab[None], i32([0]), P - 1, cu_seqlens=i32([0, P]))
    lens = [b % 20 for b in range(B)]
    own = c.table(lens, extra=0)
    c.fill(gn, own, lens)
    q, st = rows(gn, B, H, D, t), status()
    a, b2 = (torch.empty(B, H, D, dtype=t, device=dev()) for _ in range(2))
    g.gqa_attn_decode_shared(q, c.k, c.v, ptab, P, own, i32(lens), max(lens), a, status=st)
    whole = torch.cat([ptab.expand(B, -1), own], 1).contiguous()
    g.gqa_attn_decode_paged(q, c.k, c.v, whole, i32([P + n for n in lens]), P + max(lens), b2, status=st)
    assert st.item() == 0
    # each within its own bounds of the same value: two roundings, and the tensor cores' weights
    # (half a step of values that average to |out| / 30 at these lengths, times |v| ~ 0.8)
    assert ((a.double() - b2.double()).abs() <= 2 * half_step(t) * (b2.double().abs() + 0.8)).all()


# ---------------------------------------------------------------- streams and graphs

def small_case(seed=3, t=BF, B=4, n=3000, H=16, Hkv=4, D=64, page=16):
    gn = gen(seed)
    c = Cache(gn, B * (n // page + 1) + 8, Hkv, page, D, t)
    lens = [n - 7 * b for b in range(B)]
    table = c.table(lens)
    c.fill(gn, table, lens)
    ptab = c.free[:4]
    return c, table, lens, rows(gn, B, H, D, t), i32(lens), i32(ptab)


def calls(seed=3, prefix=True):
    """name -> call(out, stream, workspace or None) and workspace bytes, of the three attentions."""
    c, table, lens, q, lt, _ = small_case(seed)
    n, (B, H, D) = max(lens), q.shape
    ptab = table[0].contiguous()
    many = q.repeat(30, 1, 1).contiguous()
    mtab, ml = table.repeat(30, 1).contiguous(), i32([5] * (30 * B))
    gn = gen(seed + 1)
    cu = i32([0, 100, 100, 400])
    pq, pk, pv = (rows(gn, 400, h, D, BF) for h in (H, 4, 4))
    size = g.gqa_attn_decode_paged_workspace_size(B, H, 4, D, n)
    ssize = g.gqa_attn_decode_shared_workspace_size(30 * B, H, 4, D, lens[0], 5)
    assert size > 0 and ssize > 0
    return {
        "decode": ((B, H, D), size, lambda o, s, w: g.gqa_attn_decode_paged(
            q, c.k, c.v, table, lt, n, o, workspace=w, stream=s)),
        "shared": ((30 * B, H, D), ssize, lambda o, s, w: g.gqa_attn_decode_shared(
            many, c.k, c.v, ptab, lens[0], mtab, ml, 5, o, workspace=w, stream=s)),
        "prefill": ((400, H, D), 0, lambda o, s, w: g.gqa_attn_prefill_packed(
            pq, pk, pv, cu, 300, o, stream=s)),
    }


@pytest.mark.parametrize("name", ["decode", "shared", "prefill"])
def test_another_stream_gives_the_same_bits(name):
    shape, size, call = calls()[name]
    want, got = (torch.zeros(shape, dtype=BF, device=dev()) for _ in range(2))
    call(want, None, None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(2_000_000)                 # the current stream is busy and writes freed memory
    t = torch.empty(max(16, size), dtype=torch.uint8, device=dev())
    for _ in range(100):
        t.fill_(255)
    del t
    call(got, s, None)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", ["decode", "shared", "prefill"])
def test_captured_calls_that_share_a_workspace(name):
    a, b = calls(3)[name], calls(11)[name]
    ws = torch.full((max(16, a[1], b[1]),), 255, dtype=torch.uint8, device=dev())
    outs, wants, graphs = [], [], []
    for shape, _, call in (a, b):
        want = torch.zeros(shape, dtype=BF, device=dev())
        call(want, None, None)
        wants.append(want)
        out = torch.zeros(shape, dtype=BF, device=dev())
        outs.append(out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(out, None, ws)
            call(out, None, ws)
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        outs[i].fill_(3)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], wants[i])


def test_a_captured_step_follows_lengths_and_tables_written_later():
    """One graph of append and decode serves every step: positions, lengths and pages are device values."""
    gn, t, B, H, Hkv, D, page = gen(13), FP, 3, 8, 2, 64, 16
    c = Cache(gn, 30, Hkv, page, D, t)
    full = c.table([100] * B)
    table = torch.full_like(full, -1)
    rp, tab, _ = rope(D, 0, 128)
    x = torch.zeros(B, H + 2 * Hkv, D, dtype=t, device=dev())
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    qr, out = (torch.zeros(B, H, D, dtype=t, device=dev()) for _ in range(2))
    start, length, st = i32([0] * B), i32([1] * B), status()
    ws = torch.empty(max(16, g.gqa_attn_decode_paged_workspace_size(B, H, Hkv, D, 100)),
                     dtype=torch.uint8, device=dev())

    def step(o):
        g.kv_cache_append_paged(k, v, c.k, c.v, table, start, 99, rp, tab, q=q, q_out=qr, status=st)
        g.gqa_attn_decode_paged(qr, c.k, c.v, table, length, 100, o, workspace=ws, status=st)

    table.copy_(full)
    step(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    table.fill_(-1)
    for p in (0, 1, 15, 16, 17, 99):
        x.copy_(normal(gn, x.shape, t))
        table[:, :p // page + 1] = full[:, :p // page + 1]
        c.k[full.long()] = normal(gn, c.k[full.long()].shape, t)
        c.v[full.long()] = normal(gn, c.v[full.long()].shape, t)
        start.fill_(p)
        length.fill_(p + 1)
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step(out)
        torch.cuda.synchronize()
        assert torch.equal(got, out) and st.item() == 0 and torch.isfinite(out).all()


# ---------------------------------------------------------------- the rest

def test_pools_past_2_to_the_32_elements():
    """Pages far into pools of 2^32 elements and more, left uninitialised but for those in use."""
    t, Hkv, D, page, H = BF, 8, 128, 1024, 16
    pages = (1 << 32) // (Hkv * page * D) + 40
    k, v = (torch.empty(pages, Hkv, page, D, dtype=t, device=dev()) for _ in range(2))
    assert k.numel() > 1 << 32
    gn, n = gen(17), 4 * page - 100
    ids = [pages - 1, 2, pages - 7, 30]
    kn, vn, q = normal(gn, (n, Hkv, D), t), normal(gn, (n, Hkv, D), t), normal(gn, (1, H, D), t)
    out, st, table = torch.empty_like(q), status(), i32([ids])
    g.kv_cache_append_paged(kn, vn, k, v, table, i32([0]), n - 1, cu_seqlens=i32([0, n]), status=st)
    assert torch.equal(k[ids[2], :, 5].contiguous(), kn[2 * page + 5])
    g.gqa_attn_decode_paged(q, k, v, table, i32([n]), n, out, status=st)
    o, vabs, unsure = attend(q, kn, vn, torch.ones(1, n, dtype=torch.bool, device=dev()))
    check(out, o, attend_tol(o, vabs, unsure, t, False))
    B = 40                                       # enough rows for the tensor cores
    qs, outs = normal(gn, (B, H, D), t), torch.empty(B, H, D, dtype=t, device=dev())
    g.gqa_attn_decode_shared(qs, k, v, table[0], n, torch.zeros(B, 1, dtype=torch.int32, device=dev()),
                             i32([0] * B), 0, outs, status=st)
    o, vabs, unsure = attend(qs, kn, vn, torch.ones(B, n, dtype=torch.bool, device=dev()))
    check(outs, o, attend_tol(o, vabs, unsure, t, True))
    assert st.item() == 0


@pytest.fixture
def checked():
    before = g.attn_set_check_finite(1)
    yield
    g.attn_set_check_finite(before)


def test_the_finite_check_covers_what_is_read(checked):
    gn, t, B, H, Hkv, D, page = gen(19), FP, 3, 8, 2, 64, 16
    c = Cache(gn, 20, Hkv, page, D, t)
    lens = [40, 0, 17]
    table = c.table(lens)
    c.fill(gn, table, lens)                      # what is not in use holds NaNs
    q, out = rows(gn, B, H, D, t), torch.full((B, H, D), 7.0, dtype=t, device=dev())
    call = lambda st, **kw: g.gqa_attn_decode_paged(q, c.k, c.v, table, i32(lens), 40, out, status=st, **kw)  # noqa: E731
    st = status()
    call(st)
    assert st.item() == 0 and (out[0] != 7.0).any()
    with pytest.raises(g.AttnError):
        call(None)
    c.v[table[2, 1], 1, 0, 3] = float("inf")     # row 2's last position
    out.fill_(7.0)
    call(st)
    assert st.item() == g.DEV_NONFINITE and (out == 7.0).all()
    lens[2], st = 16, status()
    call(st)
    assert st.item() == 0 and (out[0] != 7.0).any()
    # packed prompts and an append: rows of no sequence may hold anything
    x = normal(gn, (30, H + 2 * Hkv, D), t)
    q2, k2, v2 = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    x[25:] = float("nan")
    o2, st = torch.full((30, H, D), 7.0, dtype=t, device=dev()), status()
    g.gqa_attn_prefill_packed(q2, k2, v2, i32([0, 9, 25]), 20, o2, status=st)
    assert st.item() == 0 and (o2[:25] != 7.0).any(-1).all()
    v2[3, 1, 5] = float("inf")
    o2.fill_(7.0)
    g.gqa_attn_prefill_packed(q2, k2, v2, i32([0, 9, 25]), 20, o2, status=st)
    assert st.item() == g.DEV_NONFINITE and (o2 == 7.0).all()
    st, kc = status(), c.k.clone()
    g.kv_cache_append_paged(k2, v2, c.k, c.v, table[:2].contiguous(), i32([0, 0]), 20,
                            cu_seqlens=i32([0, 9, 9]), status=st)
    assert st.item() == g.DEV_NONFINITE and torch.equal(kc.view(torch.int16), c.k.view(torch.int16))
    # a shared prefix
    st, lens = status(), [5, 0, 3]
    ptab = table[0].contiguous()
    g.gqa_attn_decode_shared(q, c.k, c.v, ptab, 40, table, i32([5, 0, 3]), 5, out, status=st)
    assert st.item() == 0
    c.k[ptab[1], 0, 2, 0] = float("nan")
    g.gqa_attn_decode_shared(q, c.k, c.v, ptab, 40, table, i32([5, 0, 3]), 5, out, status=st)
    assert st.item() == g.DEV_NONFINITE


def test_two_calls_at_once_on_two_streams():
    shape, size, call = calls(3)["decode"]
    shape2, size2, call2 = calls(11)["shared"]
    shape3, _, call3 = calls(5)["prefill"]
    todo = [(shape, size, call), (shape2, size2, call2), (shape3, 0, call3)]
    wants = []
    for s, _, f in todo:
        w = torch.zeros(s, dtype=BF, device=dev())
        f(w, None, None)
        wants.append(w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in todo]
    outs = [[torch.zeros(s, dtype=BF, device=dev()) for _ in range(10)] for s, _, _ in todo]
    torch.cuda.synchronize()
    for i in range(10):
        for (s, _, f), st, o in zip(todo, streams, outs):
            f(o[i], st, None)
    torch.cuda.synchronize()
    for o, w in zip(outs, wants):
        assert all(torch.equal(x, w) for x in o)
