"""The 8-bit cache, attention weights and eviction without a GPU: what the C entry
points and the tensor-level functions refuse, workspace sizes, and the allocator's
compaction.  Nothing here launches."""

import ctypes
import random

import pytest
import torch

from paged_kv_cache_exact_b200 import api
from paged_kv_cache_exact_b200 import binding as B

FAKE = 1 << 20                      # an aligned address that is never dereferenced
f32 = ctypes.c_float
INV, UNSUP, WS = B.PKV_ERR_INVALID_ARG, B.PKV_ERR_UNSUPPORTED, B.PKV_ERR_WORKSPACE


def _call(name, fields, defaults, kw):
    a = dict(zip(fields, defaults))
    assert set(kw) <= set(a), kw
    a.update(kw)
    return B.raw_status(name, *[f32(v) if k == "scale" else ctypes.c_size_t(v) if k == "ws_bytes" else v
                                for k, v in a.items()])


APPEND = "k_new v_new cu start table maxp S num_new k v ks vs P ps bt H_kv d dtype cache stream".split()
APPEND_OK = [FAKE] * 5 + [4, 2, 3] + [FAKE] * 4 + [8, 32, 16, 4, 128, B.PKV_BF16, B.PKV_I8, None]


@pytest.mark.parametrize("kw,status", [
    (dict(num_new=-1), INV), (dict(S=0), INV), (dict(maxp=0), INV), (dict(P=0), INV), (dict(H_kv=0), INV),
    (dict(ps=8), INV), (dict(ps=48), INV), (dict(ps=512), INV),
    (dict(bt=8), INV), (dict(bt=24), INV), (dict(bt=64), INV),            # no power of two in [16, page_size]
    (dict(dtype=B.PKV_I8), INV), (dict(cache=B.PKV_BF16), INV), (dict(cache=4), INV),
    (dict(d=64), UNSUP), (dict(P=1 << 24, ps=256), UNSUP),
    (dict(k_new=FAKE + 8), INV), (dict(v=FAKE + 4), INV), (dict(ks=None), INV), (dict(vs=FAKE + 2), INV),
    (dict(cu=None), INV), (dict(start=FAKE + 1), INV), (dict(table=None), INV),
    (dict(num_new=0, k_new=None, v_new=None, cu=None, start=None, table=None, ks=None, vs=None), B.PKV_OK),
])
def test_append_q8_rejects_bad_arguments(kw, status):
    assert _call("paged_kv_append_q8", APPEND, APPEND_OK, kw) == status


COPY = "k v ks vs src dst n P ps bt H_kv d cache stream".split()
COPY_OK = [FAKE] * 6 + [2, 8, 32, 16, 4, 128, B.PKV_E4M3, None]


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INV), (dict(P=0), INV), (dict(ps=24), INV), (dict(bt=64), INV), (dict(cache=B.PKV_F32), INV),
    (dict(d=32), UNSUP), (dict(k=FAKE + 4), INV), (dict(ks=None), INV), (dict(src=FAKE + 1), INV),
    (dict(n=0, k=None, v=None, ks=None, vs=None, src=None, dst=None), B.PKV_OK),
])
def test_copy_pages_q8_rejects_bad_arguments(kw, status):
    assert _call("paged_kv_copy_pages_q8", COPY, COPY_OK, kw) == status


ATTN = "q k v ks vs table lens ps bt S q_len H H_kv d P maxp max_len causal scale cache out".split()
ATTN_OK = [FAKE] * 7 + [32, 16, 2, 1, 8, 4, 128, 8, 64, 2000, 1, 0.1, B.PKV_I8, FAKE]
Q8_TAIL = ["ws", "ws_bytes", "stream"], [FAKE, 1 << 30, None]
W_TAIL = ["weights", "stride", "ws", "ws_bytes", "stream"], [FAKE, 2000, FAKE, 1 << 30, None]
ATTN_BAD = [
    (dict(q=None), INV), (dict(k=FAKE + 8), INV), (dict(out=FAKE + 4), INV), (dict(table=FAKE + 2), INV),
    (dict(lens=None), INV), (dict(ks=None), INV), (dict(vs=FAKE + 2), INV),
    (dict(ps=8), INV), (dict(ps=48), INV), (dict(bt=8), INV), (dict(bt=64), INV), (dict(bt=0), INV),
    (dict(S=0), INV), (dict(q_len=0), INV), (dict(H=6), INV), (dict(H_kv=0), INV), (dict(P=0), INV),
    (dict(maxp=1), INV), (dict(max_len=0), INV), (dict(q_len=2001), INV), (dict(causal=2), INV),
    (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(cache=7), INV), (dict(d=64), UNSUP), (dict(S=70000), UNSUP), (dict(P=1 << 28), UNSUP),
    (dict(ws=None), WS), (dict(ws=FAKE + 16), WS), (dict(ws_bytes=64), WS),
]


@pytest.mark.parametrize("kw,status", ATTN_BAD + [(dict(cache=B.PKV_BF16), INV), (dict(cache=B.PKV_F32), INV)])
def test_attn_q8_rejects_bad_arguments(kw, status):
    assert _call("paged_attn_q8", ATTN + Q8_TAIL[0], ATTN_OK + Q8_TAIL[1], kw) == status


@pytest.mark.parametrize("kw,status", ATTN_BAD + [
    (dict(weights=None), INV), (dict(weights=FAKE + 2), INV), (dict(stride=1999), INV),
    (dict(cache=B.PKV_F32), UNSUP), (dict(H=4 * 257), UNSUP), (dict(q_len=2, ws=None), WS),
])
def test_attn_weights_rejects_bad_arguments(kw, status):
    assert _call("paged_attn_weights", ATTN + W_TAIL[0], ATTN_OK + W_TAIL[1], kw) == status


EVICT = ("k v ks vs w wo stride table dst lens new_lens kept budget recent S H_kv d P ps bt maxp max_len cache "
         "ws ws_bytes stream").split()
EVICT_OK = [FAKE] * 6 + [2000] + [FAKE, FAKE, FAKE, FAKE + 64, FAKE] + [100, 10, 2, 4, 128, 8, 32, 16, 64, 2000,
                                                                      B.PKV_E4M3, FAKE, 1 << 30, None]


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INV), (dict(v=FAKE + 8), INV), (dict(w=None), INV), (dict(wo=FAKE + 1), INV),
    (dict(table=None), INV), (dict(dst=FAKE + 2), INV), (dict(lens=None), INV), (dict(kept=None), INV),
    (dict(new_lens=FAKE), INV),                                             # the lengths themselves
    (dict(ks=None), INV), (dict(bt=64), INV), (dict(budget=0), INV), (dict(recent=-1), INV), (dict(recent=101), INV),
    (dict(S=0), INV), (dict(H_kv=0), INV), (dict(P=0), INV), (dict(ps=20), INV), (dict(maxp=3), INV),
    (dict(max_len=0), INV), (dict(stride=1999), INV), (dict(cache=9), INV),
    (dict(d=64), UNSUP), (dict(budget=(1 << 30) + 1), UNSUP), (dict(d=96, cache=B.PKV_BF16), UNSUP), (dict(S=70000), UNSUP), (dict(P=1 << 28), UNSUP),
    (dict(ws=None), WS), (dict(ws=FAKE + 8), WS), (dict(ws_bytes=100), WS),
])
def test_evict_rejects_bad_arguments(kw, status):
    assert _call("paged_kv_evict", EVICT, EVICT_OK, kw) == status


def test_workspace_sizes():
    # one split: no workspace for the output, scores and (max, sum) pairs for the weights
    assert B.paged_attn_q8_workspace_size(4, 1, 8, 2, 300, 16) == 0
    assert B.paged_attn_weights_workspace_size(4, 1, 8, 2, 300, 16) >= 4 * 8 * 300 * 4 + 4 * 8 * 8
    n = B.paged_attn_q8_workspace_size(64, 1, 64, 8, 8192, 16)
    assert n >= 64 * 64 * 2 * 130 * 4 and n == B.paged_attn_q8_workspace_size(64, 1, 64, 8, 8192, 16)
    assert B.paged_attn_weights_workspace_size(64, 1, 64, 8, 8192, 16) >= n + 64 * 64 * 8192 * 4
    # query rows: a log-sum a row, in whole tiles, for the weights alone
    assert B.paged_attn_q8_workspace_size(2, 300, 8, 2, 5000, 16) == 0
    assert B.paged_attn_weights_workspace_size(2, 300, 8, 2, 5000, 16) == 2 * 8 * 384 * 4
    for bad in [(0, 1, 8, 2, 300, 16), (4, 0, 8, 2, 300, 16), (4, 1, 8, 3, 300, 16), (4, 1, 8, 2, 0, 16),
                (4, 1, 8, 2, 300, 20)]:
        assert B.paged_attn_q8_workspace_size(*bad) == 0 and B.paged_attn_weights_workspace_size(*bad) == 0
    assert B.paged_kv_evict_workspace_size(3, 4, 100, 16, B.PKV_I8) >= 3 * 4 * (100 + 7) * 8
    assert B.paged_kv_evict_workspace_size(3, 4, 100, 16, B.PKV_BF16) == 0
    assert B.paged_kv_evict_workspace_size(3, 4, 100, 0, B.PKV_F32) == 0


def _tensors(**kw):
    t = dict(q=torch.zeros((2, 8, 1, 128), dtype=torch.bfloat16), k=torch.zeros((8, 32, 4, 128), dtype=torch.int8),
             ks=torch.zeros((8, 2, 4)), table=torch.zeros((2, 4), dtype=torch.int32),
             lens=torch.ones(2, dtype=torch.int32), w=torch.zeros((2, 4, 100)))
    t.update(v=t["k"].clone(), vs=t["ks"].clone())
    t.update(kw)
    return t


def _q8(**kw):
    t = _tensors(**kw)
    return api.paged_q8(t["q"], t["k"], t["v"], t["ks"], t["vs"], t["table"], t["lens"], 32, True, 0.1, 100)


def _weights(**kw):
    t = _tensors(**kw)
    return api.paged_weights(t["q"], t["k"], t["v"], t["table"], t["lens"], 32, True, 0.1, 100, t["w"],
                             k_scales=t["ks"], v_scales=t["vs"])


def _evict(**kw):
    t = _tensors(**kw)
    return api.evict(t["k"], t["v"], t["w"], t["table"], t["lens"], 16, 4, 100, dst_table=t.get("dst"),
                     k_scales=t["ks"], v_scales=t["vs"])


def _append(**kw):
    t = _tensors(**kw)
    new = t.get("new", torch.zeros((3, 4, 128)))
    return api.append_q8(new, new, t.get("cu", torch.zeros(3, dtype=torch.int32)), t["lens"], t["table"], t["k"],
                         t["v"], t["ks"], t["vs"])


BF = torch.zeros((8, 32, 4, 128), dtype=torch.bfloat16)


@pytest.mark.parametrize("f,kw", [
    (_q8, {}), (_weights, {}), (_evict, {}), (_append, {}),                # tensors of the CPU
    (_q8, dict(q=torch.zeros((2, 8, 1, 128)))), (_q8, dict(q=torch.zeros((2, 8, 128), dtype=torch.bfloat16))),
    (_q8, dict(k=torch.zeros((8, 16, 4, 128), dtype=torch.int8))),
    (_q8, dict(ks=None)), (_q8, dict(ks=torch.zeros((8, 3, 4)))), (_q8, dict(ks=torch.zeros((8, 2, 2)))),
    (_q8, dict(vs=torch.zeros((8, 2, 4), dtype=torch.float64))),
    (_q8, dict(table=torch.zeros((2, 4), dtype=torch.int64))), (_q8, dict(lens=torch.ones(3, dtype=torch.int32))),
    (_weights, dict(w=torch.zeros((2, 4, 99)))), (_weights, dict(w=torch.zeros((2, 8, 100)))),
    (_weights, dict(w=torch.zeros((2, 4, 100), dtype=torch.float64))),
    (_weights, dict(k=BF, v=BF)),                                         # scales for a bf16 cache
    (_evict, dict(dst=torch.zeros((2, 5), dtype=torch.int32))), (_evict, dict(w=torch.zeros((2, 4, 50)))),
    (_append, dict(new=torch.zeros((3, 2, 128)))), (_append, dict(cu=torch.zeros(2, dtype=torch.int32))),
])
def test_tensor_functions_raise_value_error(f, kw):
    with pytest.raises(ValueError):
        f(**kw)


@pytest.mark.parametrize("f,kw", [
    (_q8, dict(k=BF, v=BF, ks=None, vs=None)), (_append, dict(k=BF, v=BF, ks=None, vs=None)),
    (_evict, dict(k=BF.half(), v=BF.half(), ks=None, vs=None)),
    (_append, dict(new=torch.zeros((3, 4, 128), dtype=torch.float16))),
])
def test_tensor_functions_raise_type_error(f, kw):
    with pytest.raises((TypeError, ValueError)):
        f(**kw)


# ------------------------------------------------------------------ the allocator's compaction --


def _table(a, s):
    rows, lens = a.block_table([s])
    return [p for p in rows[0] if p >= 0], lens[0]


def test_compact_keeps_private_pages_and_gives_up_the_rest():
    a = B.PageAllocator(10, 16, 8)
    a.add_seq(1)
    a.reserve(1, 100)                                                    # 7 pages
    before, _ = _table(a, 1)
    a.compact([1], [33])
    after, n = _table(a, 1)
    assert n == 33 and after == before[:3] and a.num_free() == 7
    a.compact([1], [33])                                                 # as long as it is: nothing changes
    assert _table(a, 1) == (after, 33)
    a.compact([1], [0])
    assert _table(a, 1) == ([], 0) and a.num_free() == 10
    start, cow = a.reserve(1, 5)
    assert (start, cow) == (0, None)


def test_compact_replaces_shared_pages_of_all_holders():
    """A page that two sequences of the call hold is a source of both: neither keeps it, and no fresh page is one
    that the call's sequences held before."""
    a = B.PageAllocator(20, 16, 8)
    a.add_seq(1)
    a.reserve(1, 80)
    a.fork(1, 2)
    a.reserve(2, 30)
    old = {s: _table(a, s)[0] for s in (1, 2)}
    a.compact([1, 2], [40, 20])
    new = {s: _table(a, s)[0] for s in (1, 2)}
    held = set(old[1]) | set(old[2])
    for s in (1, 2):
        assert not set(new[s]) & held
    assert not set(new[1]) & set(new[2])
    assert a.num_free() == 20 - 5
    a.free_seq(1)
    a.free_seq(2)
    assert a.num_free() == 20


def test_compact_leaves_a_sharer_that_is_not_listed_alone():
    a = B.PageAllocator(12, 16, 8)
    a.add_seq(1)
    a.reserve(1, 64)
    a.fork(1, 2)
    kept = _table(a, 2)
    a.compact([1], [30])
    assert _table(a, 2) == kept and all(a.page_refs(p) == 1 for p in kept[0])


@pytest.mark.parametrize("ids,lens,status", [
    ([9], [1], INV), ([1, 1], [5, 5], INV), ([1], [-1], INV), ([1], [81], INV),
    ([1], [64], B.PKV_ERR_OUT_OF_PAGES), ([2, 1], [10, 81], INV),
])
def test_compact_refuses_and_changes_nothing(ids, lens, status):
    a = B.PageAllocator(7, 16, 8)
    a.add_seq(1)
    a.reserve(1, 80)
    a.fork(1, 2)
    before = (_table(a, 1), _table(a, 2), a.num_free())
    with pytest.raises(B.PkvError) as e:
        a.compact(ids, lens)
    assert e.value.status == status
    assert (_table(a, 1), _table(a, 2), a.num_free()) == before
    with pytest.raises(ValueError):
        a.compact([1], [])
    assert B.raw_status("pkv_alloc_compact", None, None, 0, None) == INV
    assert B.raw_status("pkv_alloc_compact", a._h, None, 1, None) == INV


def test_compact_random_against_a_model():
    """References stay exact over random forks, growth, compactions and frees."""
    r = random.Random(3)
    a = B.PageAllocator(60, 16, 12)
    live, nxt = [], 0
    for _ in range(400):
        op = r.random()
        if op < 0.2 or not live:
            a.add_seq(nxt)
            live.append(nxt)
            nxt += 1
        elif op < 0.35:
            a.fork(r.choice(live), nxt)
            live.append(nxt)
            nxt += 1
        elif op < 0.65:
            try:
                a.reserve(r.choice(live), r.randint(0, 40))
            except B.PkvError as e:
                assert e.status in (B.PKV_ERR_OUT_OF_PAGES, INV)
        elif op < 0.85:
            some = r.sample(live, r.randint(1, min(3, len(live))))
            old = [set(_table(a, s)[0]) for s in some]
            try:
                a.compact(some, [r.randint(0, _table(a, s)[1]) for s in some])
                for s, o in zip(some, old):
                    for p in _table(a, s)[0]:
                        assert a.page_refs(p) == 1
                        assert p in o or not any(p in x for x in old)
            except B.PkvError as e:
                assert e.status == B.PKV_ERR_OUT_OF_PAGES
        else:
            a.free_seq(live.pop(r.randrange(len(live))))
        refs = {}
        for s in live:
            for p in _table(a, s)[0]:
                refs[p] = refs.get(p, 0) + 1
        assert a.num_free() == 60 - len(refs)
        assert all(a.page_refs(p) == n for p, n in refs.items())
