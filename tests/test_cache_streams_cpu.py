"""What the tensor-level functions allocate for a call on another stream, without a GPU: every
allocation happens while that stream is current (so it is that stream's memory, which no other
stream's earlier work can still be using), and results are recorded for the caller's stream.
The library's entry points are replaced by ones that do nothing."""

import contextlib

import pytest
import torch

from paged_kv_cache_exact_b200 import api
from paged_kv_cache_exact_b200 import binding as B

MINE, OTHER = object(), 4096                       # the current stream; another one's address


class Stream:
    def __init__(self, address=None, device=None):
        self.address = address


@pytest.fixture
def seen(monkeypatch):
    """What happened: ("new", the stream's address that is current) and ("record", address or MINE)."""
    log, now = [], [None]

    @contextlib.contextmanager
    def stream(s):
        was, now[0] = now[0], s.address
        yield
        now[0] = was

    def counted(f):
        def g(*a, **kw):
            log.append(("new", now[0]))
            return f(*a, **kw)
        return g

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(MINE if now[0] is None else now[0]))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("record", s.address)), raising=False)
    monkeypatch.setattr(torch.Tensor, "new_empty", counted(torch.Tensor.new_empty))
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, counted(getattr(torch, name)))
    monkeypatch.setattr(api, "_on_device", lambda *t: contextlib.nullcontext())
    monkeypatch.setattr(api, "_stream_of", lambda stream, t: stream)
    for name in ("attn_prefill", "paged_attn", "paged_attn_q8", "paged_attn_weights", "paged_kv_evict"):
        monkeypatch.setattr(B, name, lambda *a: None)
    return log


S, H, H_kv, PS, L = 64, 8, 4, 16, 4000


def _pool(dtype=torch.int8):
    k = torch.zeros((8, PS, H_kv, 128), dtype=dtype)
    return k, k, torch.ones((8, 1, H_kv)), torch.ones((8, 1, H_kv))


def _lens():
    return torch.zeros((S, 250), dtype=torch.int32), torch.ones(S, dtype=torch.int32)


def _q(q_len=1):
    return torch.zeros((S, H, q_len, 128), dtype=torch.bfloat16)


def q8(**kw):
    k, v, ks, vs = _pool()
    return api.paged_q8(_q(), k, v, ks, vs, *_lens(), PS, True, 0.1, L, **kw)


def weights(**kw):
    k, v, ks, vs = _pool()
    return api.paged_weights(_q(), k, v, *_lens(), PS, True, 0.1, L, torch.zeros((S, H_kv, L)), k_scales=ks,
                             v_scales=vs, **kw)


def evict(**kw):
    k, v, ks, vs = _pool()
    return api.evict(k, v, torch.zeros((S, H_kv, L)), *_lens(), 50, 5, L, k_scales=ks, v_scales=vs, **kw)


def paged(**kw):
    k, v, _, _ = _pool(torch.bfloat16)
    return api.paged(_q(), k, v, *_lens(), PS, True, 0.1, L, **kw)


def prefill(**kw):
    return api.prefill(_q(), _q(), _q(), True, 0.1, **kw)


CALLS = [(q8, 2, 1), (weights, 2, 1), (evict, 3, 2), (paged, 2, 1), (prefill, 1, 1)]     # allocations, results


@pytest.mark.parametrize("call,allocations,results", CALLS, ids=lambda x: getattr(x, "__name__", None))
def test_another_streams_call_allocates_from_that_stream(seen, call, allocations, results):
    call(stream=OTHER)
    new = [s for what, s in seen if what == "new"]
    assert len(new) >= allocations and set(new) == {OTHER}
    assert [s for what, s in seen if what == "record"].count(MINE) == results


@pytest.mark.parametrize("call,allocations,results", CALLS, ids=lambda x: getattr(x, "__name__", None))
def test_the_current_streams_call_allocates_as_ever(seen, call, allocations, results):
    call()
    assert {x for x in seen} == {("new", None)} and len(seen) >= allocations


@pytest.mark.parametrize("call", [q8, weights], ids=["q8", "weights"])
def test_what_is_passed_is_recorded_for_the_other_stream(seen, call):
    out, ws = _q(), torch.zeros(1 << 20, dtype=torch.uint8)
    seen.clear()
    assert call(stream=OTHER, out=out, workspace=ws) is out
    assert sorted(seen) == [("record", OTHER)] * 2
