"""16-bit paged serving at its edges."""
import pytest
import torch

import gqa_causal_attention_gb300 as g
from paged_ref import Cache, dev, gen, i32, rows, status

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


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
