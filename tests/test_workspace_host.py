"""Calls that take their own scratch do so on the stream they run on (no GPU is touched): a
block of another stream's pool may still be written by a kernel queued there."""
import contextlib
import types

import pytest
import torch

import gqa_causal_attention_gb300 as g

B, H, HKV, L, D, CAP = 2, 8, 2, 200, 64, 256


class Taken(Exception):
    pass


@pytest.fixture
def pool(monkeypatch):
    """Torch's allocator stopped at the binding's first request, which is raised as
    Taken(stream, bytes); streams are names, and host tensors pass for device ones."""
    current = ["current"]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream or current[-1])
        yield
        current.pop()

    def empty(n, dtype=torch.float32, device=None):
        raise Taken(current[-1], int(n) * torch.tensor([], dtype=dtype).element_size())

    for name in ("_f32", "_i32"):
        monkeypatch.setattr(g, name, lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)


def calls():
    z = torch.zeros
    q, k, c = z(B, H, L, D), z(B, HKV, L, D), z(B, HKV, CAP, D)
    q1, k1 = z(B, H, 1, D), z(B, HKV, 1, D)
    vt = types.SimpleNamespace(is_cuda=True, dtype=torch.float32, is_contiguous=lambda: True,
                               numel=lambda: B * HKV * D * g.gqa_attn_vt_pitch(L))
    rp = g.RopeParams.make()
    dm = H * D
    w = {"input_layernorm.weight": z(dm), "post_attention_layernorm.weight": z(dm),
         "q_proj.weight": z(dm, dm), "k_proj.weight": z(HKV * D, dm), "v_proj.weight": z(HKV * D, dm),
         "o_proj.weight": z(dm, dm), "gate_proj.weight": z(96, dm), "up_proj.weight": z(96, dm),
         "down_proj.weight": z(dm, 96)}
    x = z(B, L, dm)
    return {
        "prefill": (g.gqa_attn_prefill_workspace_size(B, HKV, L, D),
                    lambda s: g.gqa_attn_prefill(q, k, k, q, stream=s)),
        "rope": (g.gqa_attn_prefill_rope_workspace_size(B, H, HKV, L, D, rp),
                 lambda s: g.gqa_attn_prefill_rope(q, k, k, q, None, 0, rp, None, stream=s)),
        "ragged": (g.gqa_attn_prefill_ragged_workspace_size(B, H, HKV, L, D, rp),
                   lambda s: g.gqa_attn_prefill_ragged(q, k, k, q, z(B), rp, None, stream=s)),
        "rope_vt": (g.gqa_attn_prefill_rope_vt_workspace_size(B, H, L, D, rp),
                    lambda s: g.gqa_attn_prefill_rope_vt(q, k, vt, q, None, 0, rp, None, stream=s)),
        "cached": (g.gqa_attn_prefill_cached_workspace_size(B, H, HKV, L, D, 9, 0, rp),
                   lambda s: g.gqa_attn_prefill_cached(q, k, k, c, c, q, None, 9, rp, None, stream=s)),
        "prefill step": (g.gqa_attn_prefill_step_workspace_size(B, H, HKV, L, D, 0, rp),
                         lambda s: g.gqa_attn_prefill_step(q, k, k, q, c, c, rp, None, stream=s)),
        "decode step": (g.gqa_attn_decode_step_workspace_size(B, H, HKV, D, 9, 0),
                        lambda s: g.gqa_attn_decode_step(q1, k1, k1, q1, z(B), 9, c, c, rp, None, stream=s)),
        "block": (g.gqa_block_forward_workspace_size(B, L, H, HKV, D, 96, rp),
                  lambda s: g.gqa_block_forward(x, x, w, H, HKV, rp, None, stream=s)),
        "table": (g.attn_rope_table_bytes(rp, D), lambda s: g.rope_table(rp, D, stream=s)),
        "from host": (g.gqa_attn_prefill_from_host_workspace_size(B, H, HKV, L, D, CAP, rp),
                      lambda s: g.gqa_attn_prefill_from_host(q, k, k, q, q, k, k, q, c, c, None, 0,
                                                             rp, None, stream=s)),
    }


NAMES = ["prefill", "rope", "ragged", "rope_vt", "cached", "prefill step", "decode step", "block",
         "table", "from host"]


@pytest.mark.parametrize("stream", [None, "other"])
@pytest.mark.parametrize("name", NAMES)
def test_scratch_is_taken_on_the_stream_that_uses_it(pool, name, stream):
    size, call = calls()[name]
    with pytest.raises(Taken) as e:
        call(stream)
    assert e.value.args == (stream or "current", max(16, size))
