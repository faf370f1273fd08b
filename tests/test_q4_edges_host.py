"""The 4-bit KV cache on the host, next to test_q4_host: where a call's workspace comes from,
and
how its kernels read and give up."""
import contextlib
import glob
import os
import re

import pytest
import torch

import gqa_causal_attention_gb300 as g
from gqa_causal_attention_gb300 import _build


class Taken(Exception):
    pass


@pytest.fixture
def pool(monkeypatch):
    """Torch's allocator stopped at the binding's first request, which is raised as
    Taken(stream, bytes); streams are names."""
    current = ["current"]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(n, dtype=torch.float32, device=None):
        raise Taken(current[-1], int(n) * torch.tensor([], dtype=dtype).element_size())

    t = {name: torch.zeros(shape) for name, shape in (
        ("q", (2, 16, 1, 64)), ("k", (2, 2, 1, 64)), ("cache", (2, 2, 3000, 80)))}
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    return t


@pytest.mark.parametrize("stream", [None, "other"])
@pytest.mark.parametrize("weights", [None, True])
def test_a_workspace_is_taken_on_the_stream_that_uses_it(pool, stream, weights):
    q, k, cache = pool["q"], pool["k"], pool["cache"]
    calls = [
        (lambda: g.gqa_attn_decode_q4(q, cache, None, 2999, q, weights=weights, stream=stream),
         g.gqa_attn_decode_q4_workspace_size(2, 16, 2, 64, 2999, 0, bool(weights))),
        (lambda: g.gqa_attn_decode_step_q4(q, k, k, q, cache, None, 2999, None, None,
                                           weights=weights, stream=stream),
         g.gqa_attn_decode_step_q4_workspace_size(2, 16, 2, 64, 2999, 0, bool(weights)))]
    for call, size in calls:
        with pytest.raises(Taken) as e:
            call()
        assert e.value.args == (stream or "current", size)


def test_kernels_that_start_early_read_by_plain_loads():
    """A kernel launched by launch_dependent is resident while the ones before it still write:
    the read-only path (__ldg, ld.global.nc) wants data that nothing writes in that time."""
    csrc = os.path.join(os.path.dirname(g.__file__), "csrc")
    seen = 0
    for path in glob.glob(os.path.join(csrc, "*q4*")):
        code = re.sub(r"//[^\n]*", "", open(path).read())
        seen += "dependent_wait()" in code
        assert not re.search(r"__ldg|\.nc\b|__restrict__", code), path
    assert seen >= 3


def test_a_block_that_gives_up_lets_its_copies_land():
    """Where a wait for bulk copies into shared memory runs out, the block drains them before it
    reports and ends. (A copy that never comes cannot be made on the host; read in the source.)"""
    csrc = os.path.join(os.path.dirname(g.__file__), "csrc")
    seen = 0
    for path in glob.glob(os.path.join(csrc, "*q4*")):
        code = open(path).read()
        for m in re.finditer(r"report\([^;]*ATTN_DEV_TIMEOUT\)", code):
            seen += 1
            assert "mbar_drain(" in code[max(0, m.start() - 300):m.start()], path
    assert seen == 2


def test_the_library_loads_where_the_extension_cannot_be_built(monkeypatch):
    """Calls that never touch the 4-bit cache need neither torch's headers nor a compiler."""
    def none(*a, **kw):
        raise RuntimeError("no compiler")

    g.load()
    monkeypatch.setattr(_build, "build_ext", none)
    monkeypatch.setattr(_build.subprocess, "run", none)
    monkeypatch.setattr(g, "_lib", None)
    monkeypatch.setattr(g, "_ext", None)
    assert g.load() is g.load()
    assert g.attn_version() and g.gqa_attn_decode_workspace_size(1, 8, 2, 64, 500) > 0
    with pytest.raises(RuntimeError, match="no compiler"):
        g.kv_cache_read_q4(None, None, None, None, 0)


def test_an_extension_of_another_torch_is_not_taken(monkeypatch):
    path = _build.build_ext()
    assert _build.ext_up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not _build.ext_up_to_date() and _build.ext_path() != path


@pytest.mark.parametrize("B,H,Hkv,D", [(1, 8, 8, 128), (1, 1, 1, 32), (1, 1 << 17, 1, 32), (3, 24, 2, 96)])
def test_workspace_sizes_up_to_the_longest_caches(B, H, Hkv, D):
    last = 0
    for n in [(1 << i) + d for i in range(20, 31) for d in (0, 1)] + [2 ** 31 - d for d in range(70, 0, -1)]:
        size = g.gqa_attn_decode_q4_workspace_size(B, H, Hkv, D, n, 0, True)
        assert 4 * B * H * n <= size and last <= size < 2 ** 52
        last = size
