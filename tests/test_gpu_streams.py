"""Calls without a workspace on a stream other than the current one, while writes are still
queued there to freed memory of the workspace's size: the bits of the same call alone."""
import pytest
import torch

import gqa_causal_attention_gb300 as g
from gqa_causal_attention_gb300 import synthetic as syn

from gpu_util import dev

pytestmark = pytest.mark.gpu

B, H, HKV, L, D, CAP = 2, 16, 4, 300, 128, 4096


def calls(name):
    """(workspace bytes, call(out, stream), output shape)."""
    q, k, v = (syn.normal(3, n, (B, h, L, D)).to(dev()) for n, h in (("q", H), ("k", HKV), ("v", HKV)))
    kc, vc = (syn.normal(4, n, (B, HKV, CAP, D)).to(dev()) for n in ("kc", "vc"))
    q1, k1, v1 = (t[:, :, :1].contiguous() for t in (q, k, v))
    rp = g.RopeParams.make(max_positions=CAP)
    table = g.rope_table(rp, D, dev())
    zero, last = (torch.full((B,), n, dtype=torch.int32, device=dev()) for n in (0, CAP - 1))
    return {
        "prefill": (g.gqa_attn_prefill_workspace_size(B, HKV, L, D),
                    lambda o, s: g.gqa_attn_prefill(q, k, v, o, stream=s), q.shape),
        "cached": (g.gqa_attn_prefill_cached_workspace_size(B, H, HKV, L, D, 0, 0, rp),
                   lambda o, s: g.gqa_attn_prefill_cached(q, k, v, kc, vc, o, zero, 0, rp, table,
                                                          stream=s), q.shape),
        "prefill step": (g.gqa_attn_prefill_step_workspace_size(B, H, HKV, L, D, 0, rp),
                         lambda o, s: g.gqa_attn_prefill_step(q, k, v, o, kc, vc, rp, table,
                                                              stream=s), q.shape),
        "decode step": (g.gqa_attn_decode_step_workspace_size(B, H, HKV, D, CAP - 1, 0),
                        lambda o, s: g.gqa_attn_decode_step(q1, k1, v1, o, last, CAP - 1, kc, vc, rp,
                                                            table, stream=s), q1.shape),
    }[name]


@pytest.mark.parametrize("name", ["prefill", "cached", "prefill step", "decode step"])
def test_writes_still_queued_to_freed_memory_do_not_reach_a_call(name):
    size, call, shape = calls(name)
    want = torch.empty(shape, device=dev())
    call(want, None)
    got = [torch.zeros_like(want) for _ in range(20)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(2_000_000)             # about a millisecond, in which the writes pile up
    t = torch.empty(max(4, size // 4), device=dev())
    for _ in range(300):
        t.fill_(7.0)
    del t
    for o in got:
        call(o, s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)


def test_a_table_made_on_a_stream_is_not_written_by_another():
    rp = g.RopeParams.make(max_positions=8192)
    want = g.rope_table(rp, D, dev())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(2_000_000)
    t = torch.empty_like(want)
    for _ in range(300):
        t.fill_(7.0)
    del t
    got = g.rope_table(rp, D, dev(), stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
