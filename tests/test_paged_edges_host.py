"""16-bit paged serving at its edges, on the host (stand-in pointers, so only where no CUDA device is
visible)."""
import itertools

import gqa_causal_attention_gb300 as g
from test_paged_host import ALIGN, CAPACITY, D, H, HKV, P, SHAPE, WORKSPACE, append, decode, no_device, prefill, rows, shared


@no_device
def test_shared_workspaces_never_shrink():
    """A workspace of the largest batch, prefix and own length serves every smaller one: over the
    boundaries of pairs of tiles, of key blocks, and of prefixes read with the rows' own positions."""
    size = g.gqa_attn_decode_shared_workspace_size
    batches = sorted({*range(1, 140), 200, 255, 256, 257, 511, 513, 2000, 8192, 8193, 20000})
    prefixes = sorted({1, 16, 100, *range(120, 9000, 61), *(128 * i + j for i in range(1, 40, 3) for j in (0, 1)),
                       20000, 100000, 1 << 20})
    for h, hkv, d in ((32, 8, 128), (8, 1, 64), (7, 7, 32), (28, 4, 64), (128, 1, 16), (65, 1, 128), (200, 200, 64),
                      (20, 4, 96), (6, 2, 40)):
        for n in (0, 500, 5000):
            grid = [[size(b, h, hkv, d, p, n) for p in prefixes] for b in batches]
            assert all(x == sorted(x) for x in grid)
            assert all(list(x) == sorted(x) for x in zip(*grid))
        for b, p in ((64, 8192), (3, 2001), (33, 40000)):
            sizes = [size(b, h, hkv, d, p, n) for n in range(0, 20000, 37)]
            assert sizes == sorted(sizes)


@no_device
def test_the_shared_call_takes_a_larger_batchs_workspace():
    need = g.gqa_attn_decode_shared_workspace_size
    for b, prefix in itertools.product((1, 2, 5, 32, 33, 64, 65, 200), (50, 2001, 8192, 20000)):
        call = lambda **kw: shared(b=b, prefix=prefix, pwidth=1 << 20, ws=P + 8, **kw)  # noqa: E731, B023
        own = need(b, H, HKV, D, prefix, 100)
        if own == 0:                             # nothing is asked for, and the call would be enqueued
            continue
        assert call(wbytes=own - 1) == WORKSPACE and call(wbytes=own) == ALIGN
        for more, longer in ((b + 1, prefix), (b, prefix + 130), (300, 30000)):
            assert call(wbytes=need(more, H, HKV, D, longer, 100)) == ALIGN   # enough: the address is next


@no_device
def test_the_largest_sizes():
    """Rows, sequences and positions whose last tile would pass 2^31 are refused, and no workspace is
    named for them."""
    top, most = (1 << 31) - 1, (1 << 31) - 1025
    one = dict(q=rows(heads=1), k=rows(heads=1), v=rows(heads=1), out=rows(heads=1), h=1, hkv=1)
    assert prefill(T=top, b=1, **one) == SHAPE and prefill(T=most + 1, b=1, **one) == SHAPE
    assert prefill(T=5, b=most - 4, **one) == SHAPE
    assert prefill(T=most - 1, b=1, **{**one, "q": rows(P + 8, heads=1)}) == ALIGN   # as far as the rows
    assert append(b=most + 1) == SHAPE and append(b=most, max_pos=-1) != SHAPE
    assert decode(max_len=most + 1) == SHAPE and decode(max_len=most) == CAPACITY
    assert shared(prefix=most + 1) == SHAPE and shared(prefix=most) == CAPACITY
    paged, both = g.gqa_attn_decode_paged_workspace_size, g.gqa_attn_decode_shared_workspace_size
    assert paged(3, 8, 2, 64, most) > 0 and both(3, 8, 2, 64, most, most) > 0
    for n in (most + 1, top):
        assert paged(3, 8, 2, 64, n) == 0 and paged(3, 8, 2, 64, n, top) == 0
        assert both(3, 8, 2, 64, n, 5) == 0 and both(3, 8, 2, 64, 100, n) == 0
    assert paged((1 << 24) + 1, 1, 1, 64, 5000) == 0 and both((1 << 21) + 1, 8, 2, 64, 100, 5) == 0
    assert paged(1 << 21, 8, 2, 64, 5000, most) > 0
