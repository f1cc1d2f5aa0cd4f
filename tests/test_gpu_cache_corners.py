"""Corners of the 8-bit paged cache, attention weights and eviction on the GPU: other streams, values that
are not finite, scales of zero, wide tables, many evictions.  Tolerances are those of test_gpu_cache.py
where a check does not say its own."""

import math

import pytest
import torch

from _cache_ref import attend, evict, nearest
from paged_kv_cache_exact_b200 import api
from paged_kv_cache_exact_b200 import binding as B
from test_gpu_cache import BF16, D, DEV, E4M3, I8, Cache, _errors, clean, pool, raw  # noqa: F401

pytestmark = pytest.mark.gpu


def busy():
    """Some milliseconds of work on the current stream."""
    x = torch.zeros((4096, 4096), dtype=BF16, device=DEV)
    for _ in range(100):
        x = x @ x


@pytest.mark.parametrize("op", ["attend", "weights", "evict"])
def test_another_streams_results_do_not_share_freed_memory(op):
    """A call on another stream, which waits for its inputs alone, while work that the current stream still has to do
    writes blocks of the results' sizes that were freed a moment ago."""
    c = Cache(I8, [700, 40, 1300], 16, 2, 16, 16, seed=9)
    first = [x.clone() for x in (c.k, c.v, c.ks, c.vs, c.w)]

    def run(**kw):
        if op == "attend":
            return (c.run(False, **kw),)
        if op == "weights":
            return c.run(True, **kw), c.w
        return api.evict(c.k, c.v, c.w, c.table, c.len_t, 90, 8, 1300, k_scales=c.ks, v_scales=c.vs, **kw) + (c.w, c.k)

    want = [x.clone() for x in run()]
    for x, y in zip((c.k, c.v, c.ks, c.vs, c.w), first):
        x.copy_(y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    made = [x for x in want if x.shape not in (c.w.shape, c.k.shape)]
    n = B.paged_attn_weights_workspace_size(3, 1, 16, 2, 1300, 16)
    busy()
    freed = [torch.empty_like(x) for x in made] + [torch.empty(n, dtype=torch.uint8, device=DEV)]
    for x in freed:
        x.fill_(77)
    at = {x.data_ptr() for x in freed}
    del freed, x
    got = run(stream=s)
    torch.cuda.synchronize()
    assert not at & {x.data_ptr() for x in got[:len(made)]}
    assert all(torch.equal(raw(a), raw(b)) for a, b in zip(got, want))


def test_results_of_another_stream_outlive_their_name():
    """A result that is dropped while the current stream still has to read it is not handed to the other stream."""
    c = Cache(I8, [900, 31], 16, 2, 16, 16, seed=10)
    want = c.run(False)
    s = torch.cuda.Stream()
    busy()
    (want + 0).fill_(5)                    # what is used below is loaded: loading waits for the device
    with torch.cuda.stream(s):
        torch.empty_like(want)
    torch.cuda.synchronize()
    out = c.run(False, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    busy()
    copy = out + 0
    at = out.data_ptr()
    del out
    with torch.cuda.stream(s):
        other = torch.empty_like(want).fill_(5)
    assert other.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


@pytest.mark.parametrize("form", ["stream", "address", "default stream"])
def test_a_stream_by_name_or_address(form):
    c = Cache(E4M3, [900, 31], 16, 2, 16, 16, seed=11)
    before = c.w.clone()
    want, w = c.run(True), c.w.clone()
    c.w.copy_(before)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = c.run(True, stream={"stream": s, "address": s.cuda_stream, "default stream": 0}[form])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(c.w, w)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


@pytest.mark.parametrize("address", [False, True], ids=["stream", "address"])
def test_captured_with_a_stream_and_what_the_call_allocates(address):
    """Outputs and workspaces of a captured call come from the graph's memory; two replays on other work's heels."""
    c = Cache(I8, [700, 40, 1300], 16, 2, 16, 16, seed=12)
    before = c.w.clone()
    want, w = c.run(True), c.w.clone()
    c.w.copy_(before)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = c.run(True, stream=s.cuda_stream if address else s)
    for _ in range(2):
        c.w.copy_(before)
        junk = [torch.full((1 << k,), 3.0, device=DEV) for k in range(8, 22)]
        g.replay()
        del junk
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c.w, w)


# ------------------------------------------------------------------- values that are not finite --


def check_weights(c, before, size, want):
    """The weights that a call added, against float64 ones, by the bound of test_gpu_cache.py."""
    rel = math.expm1(2 * 128 * 2.0 ** -24 * size) + 2.0 ** -20
    for s, n in enumerate(c.lens):
        got = c.w[s, :, :n].double() - before[s, :, :n].double()
        rel_w = rel + 2.0 ** -23 * (1.4427 * size + math.log2(max(n, 2)))
        tol = rel_w * 1.01 * want[s] + 2.0 ** -24 * (c.w[s, :, :n].double().abs() + before[s, :, :n].double())
        assert ((got - want[s]).abs() <= tol).all(), f"weights of {s}"
        assert torch.equal(c.w[s, :, n:], before[s, :, n:])


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
@pytest.mark.parametrize("q_len,lens,key", [
    (1, [100, 70], 96),                 # one split
    (1, [5000, 70], 2048),              # several splits
    (1, [40, 33], 0),
    (12, [100, 70], 96),                # seen from row 8 on
    (100, [100, 300], 48),              # the prefill kernel
    (300, [700, 300], 448),             # the block of a later tile: 52 rows do not see it
])
def test_a_nan_value_scale_leaves_the_weights_alone(dtype, q_len, lens, key):
    """The rows that see the block become NaN and no others; softmax weights, which the values do not enter, stay what
    the keys make them."""
    c = Cache(dtype, lens, 4, 2, 16, 16, q_len=q_len, seed=24)
    _, want, _, size = attend(c.q, c.k, c.v, c.ks, c.vs, c.table, lens, True, c.scale)
    c.vs[int(c.table[0, key // 16]), 0, 1] = float("nan")
    before = c.w.clone()
    out = c.run(True)
    first = max(0, key - (lens[0] - q_len))                          # the first row that sees the block
    assert torch.isnan(out[0, 2:, first:]).all()
    assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[0, 2:, :first]).all() and torch.isfinite(out[1]).all()
    check_weights(c, before, size, want)
    again = c.run(False)
    assert torch.equal(torch.isnan(again), torch.isnan(out))


@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("H,H_kv", [(2, 2), (10, 2), (8, 2), (16, 2)])       # 1, 5, 4 and 8 heads a kv head
@pytest.mark.parametrize("q_len", [1, 12, 90])
def test_a_bad_page_gets_no_weight_from_rows_that_are_nan(dtype, q_len, H, H_kv):
    """Whichever kernel takes the rows: keys of a page outside the pool, and keys past a row's own, get nothing."""
    c = Cache(dtype, [200, 130], H, H_kv, 16, 16, q_len=q_len, seed=25)
    c.table[0, 3] = 1 << 20                                          # keys 48 .. 63
    page = int(c.table[0, 5])
    if dtype == BF16:
        c.k[page, 2, 1] = float("nan")
    else:
        c.ks[page, 0, 1] = float("nan")
    before = c.w.clone()
    out = c.run(True)
    assert clean() == B.PKV_DEVERR_BAD_PAGE
    G = H // H_kv
    assert torch.isnan(out[0, G:]).all() and torch.isfinite(out[0, :G]).all() and torch.isfinite(out[1]).all()
    assert torch.equal(c.w[0, :, 48:64], before[0, :, 48:64])
    live = torch.ones(200, dtype=torch.bool)
    live[48:64] = False
    assert torch.isnan(c.w[0, 1, :200][live.to(DEV)]).all() and torch.isfinite(c.w[0, 0, :200]).all()
    assert torch.equal(c.w[0, :, 200:], before[0, :, 200:])


@pytest.mark.parametrize("q_len", [129, 200, 300])
def test_prompt_weights_of_an_infinite_key(q_len):
    """A key that scores minus infinity in every row gets no weight: rows past q_len, which a tile pads with zeros,
    must not make it NaN (0 times infinity)."""
    c = Cache(BF16, [q_len + 70], 4, 2, 16, 16, q_len=q_len, seed=26)
    c.q[..., 5] = c.q[..., 5].abs() + 0.25
    n = q_len + 70
    _, want, _, size = attend(c.q, c.k, c.v, None, None, c.table, [n], True, c.scale)
    key = 40                                                         # seen by every row
    c.k[int(c.table[0, key // 16]), key % 16, 0, 5] = -float("inf")
    _, want, _, _ = attend(c.q, c.k, c.v, None, None, c.table, [n], True, c.scale)
    assert torch.isfinite(want[0]).all() and (want[0][0, key] == 0).all()
    before = c.w.clone()
    out = c.run(True)
    assert torch.isfinite(out).all()
    check_weights(c, before, size, want)
    assert torch.equal(c.w[0, 0, key], before[0, 0, key])


# ------------------------------------------------------------------------------- eviction --


@pytest.mark.parametrize("place", ["in place", "to fresh pages"])
@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
@pytest.mark.parametrize("zero", ["k", "v", "both"])
def test_evict_moves_blocks_of_scale_zero(dtype, place, zero):
    """Some blocks' scales are zero (their rows stand for zeros): K's scale says nothing about V's, and a destination
    block's old scale does not stay behind."""
    gen = torch.Generator().manual_seed(31)
    L, budget, ps, H_kv = 160, 64, 16, 2
    table = torch.randperm(10, generator=gen).to(torch.int32)[None]
    dst = table.clone()
    if place != "in place":
        dst[0, :4] = torch.arange(10, 14)
    k, ks = pool(dtype, 14, ps, 16, H_kv, gen)
    v, vs = pool(dtype, 14, ps, 16, H_kv, gen)
    for x, name in ((ks, "k"), (vs, "v")):
        if zero in (name, "both"):
            for b in (0, 2, 3, 4, 5, 6, 7):
                x[int(table[0, b])] = 0
    w = torch.rand((1, H_kv, L), generator=gen)
    g = [x.to(DEV) for x in (k, v, w, table, torch.tensor([L], dtype=torch.int32), dst, ks, vs)]
    kept, _ = api.evict(g[0], g[1], g[2], g[3], g[4], budget, 8, L, dst_table=g[5], k_scales=g[6], v_scales=g[7])
    ids = evict(w, [L], budget, 8)
    for h in range(H_kv):
        i = torch.tensor(ids[0][h])
        assert kept[0, h].tolist() == ids[0][h]
        of = (table[0].long()[i // ps], i % ps, torch.full_like(i, h))
        j = torch.arange(budget)
        to = (dst[0].long()[j // ps], j % ps, torch.full_like(j, h))
        for codes, scales, now, now_s in ((k, ks, g[0], g[6]), (v, vs, g[1], g[7])):
            old = scales[of[0], 0, h]
            new = old.view(-1, 16).amax(-1)
            assert torch.equal(now_s.cpu()[dst[0, :4].long(), 0, h], new)
            new = new.repeat_interleave(16).double()
            y = codes[of].double() if dtype == I8 else raw(codes)[of].view(dtype).double()
            exp = torch.where(new[:, None] > 0, nearest((y * old.double()[:, None]) / new.clamp(min=1e-300)[:, None],
                                                        dtype), 0) * new[:, None]
            got = raw(now).cpu()[to].view(dtype).double() * new[:, None]
            assert torch.equal(got, exp)


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
def test_many_evictions_follow_the_rule_and_its_bound(dtype):
    """A token appended and one evicted, 70 times, in place.  Every step's codes and scales are the rule's to the bit,
    and a kept row is never further from what was appended than what its moves may have cost: half a step each time
    that it was rounded anew."""
    gen = torch.Generator().manual_seed(32)
    H_kv, ps, budget, recent = 2, 16, 64, 9
    table = torch.tensor([[3, 1, 4, 0, 2]], dtype=torch.int32)
    k, ks = pool(dtype, 5, ps, 16, H_kv, gen)
    k, ks = k.to(DEV), ks.to(DEV)
    v, vs, table_d = k.clone(), ks.clone(), table.to(DEV)
    w = torch.rand((1, H_kv, 80), generator=gen).to(DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731

    def rows(n, h):
        t = torch.arange(n)
        codes = raw(k).cpu()[table[0].long()[t // ps], t % ps, h].view(dtype).double()
        return codes, ks.cpu()[table[0].long()[t // ps], 0, h].double()

    new = torch.randn((budget, H_kv, D), generator=gen).to(BF16).to(DEV)
    api.append_q8(new, new, i32(0, budget), i32(0), table_d, k, v, ks, vs)
    first, slack = {}, {}
    for h in range(H_kv):
        c, s = rows(budget, h)
        first[h], slack[h] = c * s[:, None], torch.zeros((budget, D), dtype=torch.float64)
    for step in range(70):
        old = {h: rows(budget, h) for h in range(H_kv)}
        new = (torch.randn((1, H_kv, D), generator=gen) * (0.5 + step % 4)).to(BF16).to(DEV)
        api.append_q8(new, new, i32(0, 1), i32(budget), table_d, k, v, ks, vs)
        held = {h: rows(budget + 1, h) for h in range(H_kv)}
        w[0, :, budget] = torch.rand(H_kv, generator=gen).to(DEV)
        want = evict(w.cpu(), [budget + 1], budget, recent)
        kept, _ = api.evict(k, v, w, table_d, i32(budget + 1), budget, recent, budget + 1, k_scales=ks, v_scales=vs)
        for h in range(H_kv):
            assert kept[0, h].tolist() == want[0][h]
            i = torch.tensor(want[0][h])
            c, s = held[h][0][i], held[h][1][i]
            assert torch.equal(held[h][0][:budget], old[h][0])       # the new row has a block of its own
            s_new = s.view(-1, 16).amax(-1).repeat_interleave(16)
            exp = nearest(c * s[:, None] / s_new[:, None], dtype)
            got, got_s = rows(budget, h)
            assert torch.equal(got_s, s_new) and torch.equal(got, exp)
            was = torch.cat([first[h], held[h][0][budget:] * held[h][1][budget:, None]])[i]
            lost = torch.cat([slack[h], torch.zeros((1, D), dtype=torch.float64)])[i]
            # half a step: s / 2 for int8; 2^-4 of the value or 2^-10 s for e4m3
            half = (0.5 * s_new[:, None]).expand(-1, D) if dtype == I8 else \
                torch.maximum(2.0 ** -4 * (c * s[:, None]).abs(), 2.0 ** -10 * s_new[:, None])
            lost = lost + torch.where((s_new > s)[:, None], half, 0)
            assert ((got * got_s[:, None] - was).abs() <= lost * (1 + 1e-9)).all()
            first[h], slack[h] = was, lost
    assert torch.equal(raw(k), raw(v)) and torch.equal(ks, vs)


# ------------------------------------------------------------------------------ other sizes --


@pytest.mark.parametrize("q_len", [1, 12, 300])
def test_a_table_whose_tokens_pass_31_bits(q_len):
    """2^23 pages of 256 tokens in a row of the table: its tokens are one more than an int holds."""
    c = Cache(I8, [700], 4, 2, 256, 32, q_len=q_len, seed=33)
    before = c.w.clone()
    want, w = c.run(True), c.w.clone()
    c.w = before.clone()
    wide = torch.full((1, 1 << 23), -1, dtype=torch.int32, device=DEV)
    wide[0, :c.table.shape[1]] = c.table[0]
    narrow, c.table = c.table, wide
    out = c.run(True)
    assert torch.equal(out, want) and torch.equal(c.w, w)
    c.check(out, before)
    pools = [[x.clone() for x in (c.k, c.v, c.w, c.ks, c.vs)] for _ in range(2)]
    got = [api.evict(k, v, w, t, c.len_t, 100, 9, 700, k_scales=ks, v_scales=vs)
           for (k, v, w, ks, vs), t in zip(pools, (narrow, wide))]
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert all(torch.equal(raw(a).nan_to_num(0), raw(b).nan_to_num(0)) for a, b in zip(*pools))


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("q_len,lens,H,H_kv,ps,bt", [
    (2, [700, 2, 3, 4100], 8, 8, 16, 16),
    (3, [3, 257, 1030], 15, 3, 32, 32),
    (16, [16, 17, 900], 32, 2, 256, 64),          # 256 rows a kv head
    (7, [300], 2, 1, 16, 16),
])
def test_few_rows_round_the_weights_to_eleven_bits(dtype, q_len, lens, H, H_kv, ps, bt, causal):
    """Up to 16 rows a head and 256 a kv head go through the single-token kernel, whose P has 11 bits or more:
    2^-11 of sum p |v|, where the prefill kernel's bf16 P is off by up to 2^-8."""
    c = Cache(dtype, lens, H, H_kv, ps, bt, q_len=q_len, seed=60 + q_len, q_mul=2.0)
    want, _, spread, size = attend(c.q, c.k, c.v, c.ks, c.vs, c.table, lens, causal, c.scale)
    rel = math.expm1(2 * 128 * 2.0 ** -24 * size) + 2.0 ** -20
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + rel) * 1.01 * spread + 1e-30
    for weights in (False, True)[dtype == BF16:]:
        err = (c.run(weights, causal=causal).double() - want).abs()
        assert (err <= tol).all(), f"{float((err / tol).max()):.2f} of the bound"


@pytest.mark.parametrize("cu", [[0, 100, 20, 120], [0, 120, 0, 120], [0, 60, 5, 300], [50, 40, 30, 20], [-7, 20, 10, 120]])
def test_append_with_row_numbers_that_fall_stays_in_its_pages(cu):
    """cu_new must not fall.  If it does, which rows are written is open, but nothing outside the tables' pages is,
    and what is written are new rows: one value to all of them shows as that value or as nothing."""
    gen = torch.Generator().manual_seed(34)
    k, ks = pool(I8, 40, 32, 16, 2, gen)
    v, vs = pool(I8, 40, 32, 16, 2, gen)
    g = [x.to(DEV) for x in (k, v, ks, vs)]
    table = torch.arange(4, 28, dtype=torch.int32).view(3, 8)
    new = torch.ones((120, 2, D), dtype=BF16, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for _ in range(20):
        api.append_q8(new, new, i32(cu), i32([0, 16, 32]), table.to(DEV), *g)
    torch.cuda.synchronize()
    for x, y in zip((k, v, ks, vs), g):
        y = y.cpu()
        assert torch.equal(y[:4], x[:4]) and torch.equal(y[28:], x[28:])
    for codes, scales, was in ((g[0].cpu(), g[2].cpu(), k), (g[1].cpu(), g[3].cpu(), v)):
        value = codes.double() * scales.double().repeat_interleave(16, 1)[..., None]
        wrote = (codes != was).any(-1)
        one = ((value - 1).abs() < 1e-6).all(-1)
        fresh = (scales.repeat_interleave(16, 1) <= 1 / 127 * 1.0001)        # blocks begun in the call
        assert (one | ~wrote | ~fresh).all()


@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
def test_pages_beyond_32_bits(dtype):
    """A pool of more than 2^32 bytes whose sequences lie at its end, against the same pages in a small one: append,
    attention of one, a few and many rows with weights, page copies and eviction, to the bit."""
    H, H_kv, ps, lens, budget = 16, 8, 64, [900, 300], 200
    far = (1 << 32) // (ps * H_kv * D * (2 if dtype == BF16 else 1)) + 5

    def run(base):
        c = Cache(dtype, lens, H, H_kv, ps, 32, seed=35)
        n = c.k.shape[0]
        if base:
            for name in ("k", "v", "ks", "vs"):
                x = getattr(c, name)
                if x is not None:
                    big = torch.empty((base + n, *x.shape[1:]), dtype=x.dtype, device=DEV)
                    raw(big)[base:] = raw(x)
                    setattr(c, name, big)
            c.table = torch.where(c.table >= 0, c.table + base, -1).to(torch.int32)
        out = []
        gen = torch.Generator().manual_seed(36)
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        new = torch.randn((7, H_kv, D), generator=gen).to(BF16).to(DEV)
        if dtype != BF16:
            api.append_q8(new, new, i32(0, 3, 7), i32(897, 296), c.table, c.k, c.v, c.ks, c.vs)
            api.copy_pages_q8(c.k, c.v, c.ks, c.vs, c.table[:1, 1].contiguous(), c.table[1:, 2].contiguous())
        for q_len in (1, 5, 200):
            c.q = torch.randn((2, H, q_len, D), generator=gen).to(BF16).to(DEV)
            out.append(c.run(True))
        kept, new_lens = api.evict(c.k, c.v, c.w, c.table, c.len_t, budget, 20, 900, k_scales=c.ks, v_scales=c.vs)
        out += [kept, new_lens, c.w] + [x[base:].view(torch.uint8) for x in (c.k, c.v)]           # dead slots hold NaN
        return out + [x[base:].nan_to_num(-1) for x in (c.ks, c.vs) if x is not None]

    small, large = run(0), run(far)
    assert all(torch.equal(a, b) for a, b in zip(small, large)) and torch.isfinite(small[2]).all()


@pytest.mark.parametrize("dtype", [BF16, I8], ids=["bf16", "i8"])
@pytest.mark.parametrize("q_len", [1, 6, 100])
def test_an_output_in_the_place_of_q(dtype, q_len):
    """A few rows may be written over their queries (several splits, several CTAs a kv head); a prompt with weights
    is refused, as its queries are read again."""
    c = Cache(dtype, [1500, 130], 24, 2, 16, 16, q_len=q_len, seed=37)
    before = c.w.clone()
    want, w = c.run(True), c.w.clone()
    c.w = before.clone()
    if q_len > 16:
        q = c.q.clone()
        with pytest.raises(B.PkvError) as e:
            c.run(True, out=c.q)
        assert e.value.status == B.PKV_ERR_INVALID_ARG and torch.equal(c.q, q) and torch.equal(c.w, before)
        return
    assert c.run(True, out=c.q) is c.q
    assert torch.equal(c.q, want) and torch.equal(c.w, w)
