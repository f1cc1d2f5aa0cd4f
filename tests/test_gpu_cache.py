"""The 8-bit paged cache, attention weights and eviction on the GPU, against plain float64 forms.

Tolerances.  Rounding to a type is off by at most half a step, relative 2^-8 for
bf16 and 2^-11 for f16.  An output element is sum_j p_j v_j: its own rounding
gives 2^-8 |o|; rounding each p to the type of the product gives at most 2^-8
(bf16, in the prefill kernel), 2^-11 (f16, few rows over an 8-bit cache) or 2^-15
(two bf16 parts, few rows over a bf16 cache; taken as 2^-11) of sum_j p_j |v_j|.  A score is a float32
sum of 128 products, off by at most 128 * 2^-24 of sum |q||k| * scale (and a few
2^-24 of itself for its scales); an error e of every score changes p by a factor
within exp(2 e), and 2^-20 covers the exponential, the sums and the division.  A
weight is 2^(x - L) with x and the row's log2-sum L in float32, both at most
1.4427 * (sum |q||k| * scale) + log2(keys): half a step of each is 2^-24 of that.
"""

import math
import random

import pytest
import torch

from _cache_ref import D, POISON, QMAX, append, attend, evict, nearest, values
from paged_kv_cache_exact_b200 import api
from paged_kv_cache_exact_b200 import binding as B

pytestmark = pytest.mark.gpu

I8, E4M3, BF16 = torch.int8, torch.float8_e4m3fn, torch.bfloat16
DEV = "cuda"


def raw(x):
    return x.view(torch.uint8) if x.dtype == E4M3 else x


def clean():
    torch.cuda.synchronize()
    st, bits = B.pkv_last_device_error()
    return bits


@pytest.fixture(autouse=True)
def _errors():
    clean()
    yield
    assert clean() == 0, "a device error was left over"


def tables(lens, ps, seed=0, spare=2):
    """Shuffled pages: (int32 [S, max + 1] table, pages in the pool)."""
    r = random.Random(seed)
    need = [-(-n // ps) for n in lens]
    ids = list(range(sum(need) + spare))
    r.shuffle(ids)
    t = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        t[s, :n] = torch.tensor(ids[:n], dtype=torch.int32)
        ids = ids[n:]
    return t, sum(need) + spare


def pool(dtype, pages, ps, bt, H_kv, gen):
    if dtype in (BF16, torch.float32):
        return torch.randn((pages, ps, H_kv, D), generator=gen).to(dtype), None
    x = torch.randn((pages, ps, H_kv, D), generator=gen) * (QMAX[dtype] / 3.7)
    c = x.round().clamp(-127, 127).to(I8) if dtype == I8 else x.clamp(-448, 448).to(E4M3)
    return c, (torch.randn((pages, ps // bt, H_kv), generator=gen) * 0.4).exp() * (3.7 / QMAX[dtype])


def poison(codes, scales, table, lens, ps):
    """NaN (or the largest code) wherever no token lives; scales of blocks without tokens NaN."""
    bad = POISON[codes.dtype]
    live = torch.zeros(codes.shape[:2], dtype=torch.bool)
    for s, n in enumerate(lens):
        for t in range(0, n, ps):
            live[int(table[s, t // ps]), :min(ps, n - t)] = True
    raw(codes)[~live] = raw(torch.tensor(bad).to(codes.dtype)[None])
    if scales is not None:
        blocks = live.view(live.shape[0], scales.shape[1], -1).any(-1)
        scales[~blocks] = float("nan")


class Cache:
    def __init__(self, dtype, lens, H, H_kv, ps, bt=16, q_len=1, seed=0, q_mul=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.dtype, self.lens, self.ps, self.bt = dtype, lens, ps, bt
        self.table, pages = tables(lens, ps, seed)
        self.k, self.ks = pool(dtype, pages, ps, bt, H_kv, gen)
        self.v, self.vs = pool(dtype, pages, ps, bt, H_kv, gen)
        poison(self.k, self.ks, self.table, lens, ps)
        poison(self.v, self.vs, self.table, lens, ps)
        self.q = (torch.randn((len(lens), H, q_len, D), generator=gen) * q_mul).to(BF16)
        self.w = torch.rand((len(lens), H_kv, max(lens) + 3), generator=gen)
        self.scale = D ** -0.5
        for name in ("table", "k", "ks", "v", "vs", "q", "w"):
            x = getattr(self, name)
            setattr(self, name, None if x is None else x.to(DEV))
        self.len_t = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def run(self, weights, causal=True, max_len=None, **kw):
        max_len = max(self.lens) if max_len is None else max_len
        if weights:
            return api.paged_weights(self.q, self.k, self.v, self.table, self.len_t, self.ps, causal, self.scale,
                                     max_len, self.w, k_scales=self.ks, v_scales=self.vs, **kw)
        return api.paged_q8(self.q, self.k, self.v, self.ks, self.vs, self.table, self.len_t, self.ps, causal,
                            self.scale, max_len, **kw)

    def check(self, out, before=None, causal=True, lens=None):
        lens = self.lens if lens is None else lens
        want, ww, spread, size = attend(self.q, self.k, self.v, self.ks, self.vs, self.table, lens, causal, self.scale)
        e = 128 * 2.0 ** -24 * size
        rel = math.expm1(2 * e) + 2.0 ** -20
        # which kernel takes several rows is the library's choice: the looser of the two bounds
        p_round = 2.0 ** -8 if self.q.shape[2] > 1 else 2.0 ** -11
        tol = 2.0 ** -8 * want.abs() + (p_round + rel) * 1.01 * spread + 1e-30
        err = (out.double() - want).abs()
        assert torch.isfinite(out).all()
        assert (err <= tol).all(), f"out: {float((err / tol).max()):.2f} of the bound"
        if before is None:
            return
        for s, n in enumerate(lens):
            got = self.w[s, :, :n].double() - before[s, :, :n].double()
            # the exponent's rounding, the sum's terms (within 2^-20), the accumulator's rounding
            rel_w = rel + 2.0 ** -23 * (1.4427 * size + math.log2(max(n, 2)))
            tol = rel_w * 1.01 * ww[s] + 2.0 ** -24 * (self.w[s, :, :n].double().abs() + before[s, :, :n].double())
            err = (got - ww[s]).abs()
            assert (err <= tol).all(), f"weights of {s}: {float((err / tol).max()):.2f} of the bound"
            assert torch.equal(self.w[s, :, n:], before[s, :, n:]), "weights past the sequence changed"


CASES = [
    # lens, H, H_kv, page, block
    ([1, 2, 15, 16, 17, 31, 33], 8, 8, 16, 16),
    ([64, 65, 127, 129, 300], 8, 2, 32, 16),
    ([1, 700, 2049], 32, 4, 64, 64),
    ([513, 1000], 5, 1, 256, 32),
    ([257, 90], 24, 2, 128, 128),       # 12 heads: two tiles
    ([130], 40, 2, 16, 16),             # 20 heads: more than one CTA a kv head
    ([9000, 77, 4097], 6, 2, 64, 16),   # 3 heads; many splits
]


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_decode_over_an_8_bit_cache(dtype, case):
    lens, H, H_kv, ps, bt = CASES[case]
    c = Cache(dtype, lens, H, H_kv, ps, bt, seed=case)
    c.check(c.run(False))
    c.check(c.run(False, max_len=(c.table.shape[1]) * ps))       # a loose bound: another split plan


@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_decode_accumulates_weights(dtype, case):
    lens, H, H_kv, ps, bt = CASES[case]
    c = Cache(dtype, lens, H, H_kv, ps, bt, seed=10 + case, q_mul=3.0)
    before = c.w.clone()
    first = c.run(True)
    c.check(first, before)
    again, before = c.w.clone(), c.w.clone()
    c.check(c.run(True), again)
    # the same call on the same inputs gives the same bits
    mid = c.w.clone()
    c.w = before.clone()
    c.run(True)
    assert torch.equal(c.w, mid)


@pytest.mark.parametrize("H,H_kv", [(8, 8), (16, 2), (9, 3)])
@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
def test_decode_of_a_ragged_batch(dtype, H, H_kv):
    """Enough sequences that splits grow long, some of them one token."""
    r = random.Random(H)
    c = Cache(dtype, [r.choice([1, r.randint(2, 600), r.randint(600, 4500)]) for _ in range(60)] + [4500], H, H_kv,
              32, 16, seed=H)
    before = c.w.clone()
    c.check(c.run(True), before)
    if dtype != BF16:
        c.check(c.run(False))


def test_weights_of_a_step_sum_to_the_query_heads():
    c = Cache(I8, [5, 1200], 16, 4, 32, 16)
    c.w.zero_()
    c.run(True)
    for s, n in enumerate(c.lens):
        total = c.w[s, :, :n].double().sum(-1)
        assert (total - 4).abs().max() < 4 * 2.0 ** -16


@pytest.mark.parametrize("climb", [0.5, 9.0, 60.0])
@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
def test_scores_that_climb(dtype, climb):
    """Each 16-token block scores `climb` (base-2 units) above the last: the reference maximum moves in every chunk
    or in few, and early keys vanish against late ones."""
    n = 16 * 40
    c = Cache(dtype, [n], 2, 1, 16, 16, seed=3)
    c.q.zero_()
    c.q[..., 0] = 4.0
    raw(c.k)[..., 0] = raw(torch.tensor(64.0).to(dtype)[None]).to(DEV)
    step = climb * math.log(2) / (4.0 * c.scale)
    for i in range(40):
        page = int(c.table[0, i])
        if dtype == BF16:
            c.k[page, :, :, 0] = (i - 20) * step
        else:
            c.ks[page] = max(i, 0.01) * step / 64
    before = c.w.clone()
    c.check(c.run(True), before)


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
@pytest.mark.parametrize("mul", [2.0 ** -60, 2.0 ** -20, 2.0 ** 20])
def test_extreme_scales(dtype, mul):
    """Scales and queries far from 1, with the same products: q * 2^20 against ks * 2^-20, and so on."""
    c = Cache(dtype, [100, 333], 8, 2, 16, 16, seed=4)
    c.ks.mul_(mul)
    c.vs.mul_(mul)
    c.q = (c.q.float() / mul).to(BF16)
    before = c.w.clone()
    c.check(c.run(True), before)


def test_vastly_different_value_scales():
    """A block whose values are 2^40 times smaller holds nearly all the weight: its result must not drown in
    rounding against the scales of blocks that hold next to none."""
    c = Cache(I8, [64], 4, 1, 16, 16, seed=5)
    pages = [int(x) for x in c.table[0, :4]]
    for i, p in enumerate(pages):
        c.vs[p] = 2.0 ** -40 if i == 1 else 1.0
    c.q.zero_()
    c.q[..., 0] = 8.0
    c.k[..., 0] = -100
    c.k[pages[1], :, :, 0] = 100
    c.ks.fill_(1.0)
    c.check(c.run(False))


@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
def test_nan_in_a_live_block_is_seen(dtype):
    c = Cache(dtype, [40, 50], 4, 2, 16, 16, seed=6)
    page = int(c.table[1, 1])
    if dtype == BF16:
        c.k[page, 3, 1] = float("nan")
    else:
        c.ks[page, 0, 1] = float("nan")
    out = c.run(True)
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1, :2]).all()
    assert torch.isnan(out[1, 2:]).all()
    assert torch.isfinite(c.w[0, :, :40]).all() and torch.isnan(c.w[1, 1, :50]).all()


@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_decode_leaves_out_bad_pages(dtype, bad):
    c = Cache(dtype, [200, 90, 30], 8, 2, 16, 16, seed=7)
    c.table[0, 3] = bad
    c.table[2, :2] = bad                        # nothing left of sequence 2
    before = c.w.clone()
    out = c.run(True)
    assert clean() == B.PKV_DEVERR_BAD_PAGE
    c.check(out, before)
    assert (out[2] == 0).all()
    assert torch.equal(c.w[0, :, 48:64], before[0, :, 48:64])
    assert torch.equal(c.w[2], before[2])


@pytest.mark.parametrize("length,as_if", [(0, 0), (-5, 0), (10 ** 6, 64)])
def test_decode_clamps_bad_lengths(length, as_if):
    c = Cache(I8, [64, 50], 8, 2, 16, 16, seed=8)
    c.len_t[0] = length
    before = c.w.clone()
    out = c.run(True)
    assert clean() == B.PKV_DEVERR_BAD_LEN
    c.check(out, before, lens=[as_if, 50])


def test_decode_on_another_stream_and_in_two_graphs():
    """Two captured calls with a workspace each, replayed on two streams at once, match the eager calls."""
    a, b = Cache(E4M3, [700, 40, 1300], 16, 2, 16, 16, seed=9), Cache(I8, [900, 1], 16, 2, 16, 16, seed=10)
    want = []
    for c in (a, b):
        before = c.w.clone()
        want.append((c.run(True), c.w.clone()))
        c.w.copy_(before)
        c.before = before
    graphs, outs = [], []
    for c in (a, b):
        n = B.paged_attn_weights_workspace_size(len(c.lens), 1, 16, 2, max(c.lens), 16)
        c.ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        c.out = torch.empty_like(c.q)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph, stream=s):
            c.run(True, out=c.out, workspace=c.ws)
        graphs.append((gph, s))
    torch.cuda.synchronize()
    for rep in range(3):
        for c in (a, b):
            c.w.copy_(c.before)
        torch.cuda.synchronize()
        for gph, s in graphs:
            with torch.cuda.stream(s):
                gph.replay()
        torch.cuda.synchronize()
        for c, (o, w) in zip((a, b), want):
            assert torch.equal(c.out, o) and torch.equal(c.w, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = a.run(False, stream=s)
    s.synchronize()
    assert torch.equal(o, want[0][0])


PROMPTS = [
    # q_len, lens, H, H_kv, page, block
    (2, [2, 3, 40], 2, 1, 16, 16),
    (5, [5, 129, 64], 4, 4, 32, 16),
    (128, [128, 256, 200], 4, 2, 64, 64),
    (129, [129, 1000], 6, 2, 16, 16),
    (257, [300, 257], 3, 1, 256, 64),
    (300, [2051], 8, 2, 128, 32),
    (700, [5000, 701], 2, 2, 256, 256),
]


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_many_query_rows(dtype, case, causal):
    q_len, lens, H, H_kv, ps, bt = PROMPTS[case]
    c = Cache(dtype, lens, H, H_kv, ps, bt, q_len=q_len, seed=20 + case, q_mul=2.0)
    if dtype != BF16:
        c.check(c.run(False, causal=causal), causal=causal)
    before = c.w.clone()
    out = c.run(True, causal=causal, max_len=max(lens) + 3)
    c.check(out, before, causal=causal)
    if dtype == BF16 and q_len >= 257:      # the same kernel as without weights, to the bit
        plain = api.paged(c.q, c.k, c.v, c.table, c.len_t, ps, causal, c.scale, max(lens))
        assert torch.equal(plain, out)
    w = c.w.clone()
    c.w = before.clone()
    c.run(True, causal=causal, max_len=max(lens) + 3)
    assert torch.equal(c.w, w)


FEW = [
    # a few query rows a head, as many as a verifying step has: q_len, lens, H, H_kv, page, block
    (2, [700, 2, 3, 4100], 8, 8, 16, 16),
    (3, [3, 257, 1030], 15, 3, 32, 32),
    (5, [5, 6, 2600, 64], 16, 2, 64, 16),
    (16, [16, 17, 900], 32, 2, 256, 64),          # 256 rows a kv head
    (17, [2500], 4, 4, 16, 16),
    (60, [6000], 8, 2, 128, 32),
    (61, [400, 61], 4, 1, 16, 16),
]


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("case", range(len(FEW)))
def test_few_query_rows(dtype, case, causal):
    q_len, lens, H, H_kv, ps, bt = FEW[case]
    c = Cache(dtype, lens, H, H_kv, ps, bt, q_len=q_len, seed=40 + case, q_mul=2.0)
    if dtype != BF16:
        c.check(c.run(False, causal=causal), causal=causal)
    before = c.w.clone()
    c.check(c.run(True, causal=causal, max_len=max(lens) + 3), before, causal=causal)


@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
def test_few_query_rows_more_than_keys(dtype):
    c = Cache(dtype, [4, 9, 200], 4, 2, 16, 16, q_len=9, seed=50)
    before = c.w.clone()
    out = c.run(True)
    assert clean() == B.PKV_DEVERR_BAD_LEN
    c.check(out, before)
    assert (out[0, :, :5] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("climb", [7.5, 40.0])
def test_many_query_rows_with_climbing_scores(dtype, climb):
    """Every 64-token block scores `climb` (base-2 units) above the last."""
    n = 64 * 12
    c = Cache(dtype, [n], 2, 1, 64, 64, q_len=200, seed=3)
    c.q.zero_()
    c.q[..., 0] = 4.0
    raw(c.k)[..., 0] = raw(torch.tensor(64.0).to(dtype)[None]).to(DEV)
    step = climb * math.log(2) / (4.0 * c.scale)
    for i in range(12):
        page = int(c.table[0, i])
        if dtype == BF16:
            c.k[page, :, :, 0] = (i - 6) * step
        else:
            c.ks[page] = max(i, 0.01) * step / 64
    before = c.w.clone()
    c.check(c.run(True), before)


@pytest.mark.parametrize("ps", [16, 128])
@pytest.mark.parametrize("dtype", [BF16, I8, E4M3], ids=["bf16", "i8", "e4m3"])
def test_many_query_rows_leave_out_bad_pages(dtype, ps):
    c = Cache(dtype, [700, 300], 4, 2, ps, 16, q_len=90, seed=21)
    c.table[0, 2] = -1
    c.table[1, 0] = 1 << 20
    before = c.w.clone()
    out = c.run(True)
    assert clean() == B.PKV_DEVERR_BAD_PAGE
    c.check(out, before)
    assert torch.equal(c.w[0, :, 2 * ps:3 * ps], before[0, :, 2 * ps:3 * ps])


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_nan_behind_the_causal_mask_of_a_few_rows(dtype, which):
    """The same for 12 rows of 100 keys: the block of keys 96 .. 99 is seen from row 8 on."""
    c = Cache(dtype, [100, 70], 4, 2, 16, 16, q_len=12, seed=24)
    getattr(c, which)[int(c.table[0, 6]), 0, 1] = float("nan")
    out = c.run(True)
    assert torch.isfinite(out[1]).all() and torch.isfinite(out[0, :2]).all()
    assert torch.isfinite(out[0, 2:, :8]).all() and torch.isnan(out[0, 2:, 8:]).all()
    assert torch.isfinite(c.w[1, :, :70]).all() and torch.isfinite(c.w[0, 0, :100]).all()
    assert torch.isnan(c.w[0, 1, :100]).all()


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_nan_behind_the_causal_mask_stays_there(dtype, which):
    """A block whose scale is NaN reaches the rows that see it and no others, within one tile."""
    c = Cache(dtype, [100], 2, 1, 16, 16, q_len=100, seed=22)
    getattr(c, which)[int(c.table[0, 3]), 0, 0] = float("nan")       # keys 48 .. 63
    out = c.run(False)
    assert torch.isfinite(out[0, :, :48]).all() and torch.isnan(out[0, :, 48:]).all()


def test_more_query_rows_than_keys_is_flagged():
    c = Cache(I8, [200, 50], 4, 2, 16, 16, q_len=60, seed=23)
    before = c.w.clone()
    out = c.run(True)
    assert clean() == B.PKV_DEVERR_BAD_LEN
    c.check(out, before)
    assert (out[1, :, :10] == 0).all()            # rows before the first key see nothing


# ---------------------------------------------------------------------- the write side --


def run_append(dtype, row_dtype, lens, new, H_kv, ps, bt, seed=0, spoil=None):
    gen = torch.Generator().manual_seed(seed)
    total = [a + b for a, b in zip(lens, new)]
    table, pages = tables(total, ps, seed)
    k, ks = pool(dtype, pages, ps, bt, H_kv, gen)
    v, vs = pool(dtype, pages, ps, bt, H_kv, gen)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    kn = (torch.randn((cu[-1], H_kv, D), generator=gen) * torch.logspace(-2, 1, H_kv)[:, None]).to(row_dtype)
    vn = torch.randn((cu[-1], H_kv, D), generator=gen).to(row_dtype)
    if spoil:
        spoil(locals())
    want = [append(kn, lens, cu, table, k, ks), append(vn, lens, cu, table, v, vs)]
    g = [x.to(DEV) for x in (kn, vn, torch.tensor(cu, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32),
                             table, k, v, ks, vs)]
    api.append_q8(*g)
    torch.cuda.synchronize()
    for (val, sc), codes, scales in ((want[0], g[5], g[7]), (want[1], g[6], g[8])):
        assert torch.equal(torch.isnan(scales.cpu()), torch.isnan(sc))
        assert torch.equal(scales.cpu().nan_to_num(0), sc.nan_to_num(0)), "scales"
        got = codes.cpu().double()
        assert torch.equal(got.nan_to_num(999), val.nan_to_num(999)), \
            f"{int((got != val).sum())} codes differ of {got.numel()}"


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
@pytest.mark.parametrize("row_dtype", [BF16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,new,H_kv,ps,bt", [
    ([0, 0, 0], [1, 16, 17], 2, 16, 16),
    ([5, 15, 16, 31, 0], [1, 1, 1, 1, 1], 8, 32, 16),
    ([3, 100, 7], [300, 0, 45], 3, 64, 32),           # a sequence without new rows
    ([250], [520], 1, 256, 256),
    ([10, 20], [6, 44], 4, 128, 64),
])
def test_append_is_exact(dtype, row_dtype, lens, new, H_kv, ps, bt):
    run_append(dtype, row_dtype, lens, new, H_kv, ps, bt, seed=len(lens) + H_kv)


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
def test_append_rounds_ties_to_even(dtype):
    """Rows on half steps of a scale that is a power of two: int8 k + 1/2, e4m3 midpoints."""
    def spoil(d):
        if dtype == I8:
            x = (torch.arange(D) - 64).float() + 0.5
            x[0] = 127.0
        else:
            pos = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).float()
            mid = (pos[1:] + pos[:-1]) / 2
            x = torch.cat([mid[:126], torch.tensor([448.0, -3.25])])
        d["kn"][:] = x.to(d["kn"].dtype)
        d["vn"][:] = (-x).to(d["vn"].dtype)
    run_append(dtype, torch.float32, [0], [20], 2, 32, 16, spoil=spoil)


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
def test_append_of_zeros_subnormals_and_the_largest(dtype):
    def spoil(d):
        d["kn"][0] = 0
        d["kn"][1] = 2.0 ** -133
        d["kn"][2] = 3.0e38
        d["kn"][3] = -0.0
        d["vn"][:16] = 0
        d["vn"][16:] = 1e-38
    run_append(dtype, BF16, [0, 9], [40, 3], 2, 16, 16, spoil=spoil)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
def test_append_of_what_is_not_finite(dtype, value):
    """The block and head that take it in get scale NaN, the others are as ever; a later row into the block leaves it
    NaN, and the block is whole again once its first token is written anew."""
    def spoil(d):
        d["kn"][4, 1, 17] = value
    run_append(dtype, BF16, [3, 0], [30, 20], 2, 32, 16, spoil=spoil)
    def nan_scale(d):
        d["ks"][:] = float("nan")
    run_append(dtype, BF16, [3, 16], [5, 5], 2, 32, 16, spoil=nan_scale)


def test_append_skips_bad_pages_and_positions():
    def spoil(d):
        d["table"][1, 1] = d["pages"]
    run_append(I8, BF16, [0, 10], [20, 20], 2, 16, 16, spoil=spoil)
    assert clean() == B.PKV_DEVERR_BAD_PAGE
    gen = torch.Generator().manual_seed(0)
    k, ks = pool(I8, 4, 16, 16, 2, gen)
    g = [x.to(DEV) for x in (k, k, ks, ks)]
    g = [x.clone() for x in g]
    new = torch.ones((3, 2, D), dtype=BF16, device=DEV)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    api.append_q8(new, new, i(0, 2, 3), i(31, -1), i(0, 1, 2, 3).view(2, 2), *g)   # past the table; before its start
    assert clean() == B.PKV_DEVERR_BAD_LEN
    k2 = k.clone()
    # sequence 0's first row is position 31 (page 1, slot 15); everything else is skipped
    val, sc = append(torch.ones((1, 2, D), dtype=BF16), [31], [0, 1], torch.tensor([[0, 1]]), k2, ks)
    assert torch.equal(g[0].cpu().double(), val) and torch.equal(g[2].cpu(), sc)


def test_appending_step_by_step_reads_back():
    """Rows appended one by one into reused pages stay within half a step of the block's final scale for each time
    that the scale grew, plus half a step of their own rounding."""
    gen = torch.Generator().manual_seed(1)
    H_kv, ps, n = 2, 16, 40
    rows = (torch.randn((n, H_kv, D), generator=gen) * torch.linspace(0.2, 3, n)[:, None, None]).to(BF16).to(DEV)
    k, ks = [x.to(DEV) for x in pool(I8, 4, ps, 16, H_kv, gen)]
    v, vs = k.clone(), ks.clone()
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    grew = torch.zeros((4, H_kv), device=DEV)
    for t in range(n):
        was = ks[:, 0].clone()
        api.append_q8(rows[t:t + 1], rows[t:t + 1], cu, torch.tensor([t], dtype=torch.int32, device=DEV), table,
                      k, v, ks, vs)
        page = int(table[0, t // ps])
        grew[page] = 0 if t % ps == 0 else grew[page] + (ks[page, 0] > was[page])
    for h in range(H_kv):
        got, _ = values(k, ks, table[0], n, h)
        s = ks[table[0].long()[torch.arange(n, device=DEV) // ps], 0, h].double()
        g = grew[table[0].long()[torch.arange(n, device=DEV) // ps], h].double()
        assert ((got - rows[:, h].double()).abs() <= (0.5 * (1 + g) * s)[:, None] * (1 + 1e-6)).all()


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
def test_copy_pages_copies_codes_and_scales(dtype):
    gen = torch.Generator().manual_seed(2)
    k, ks = pool(dtype, 9, 64, 32, 3, gen)
    v, vs = pool(dtype, 9, 64, 32, 3, gen)
    g = [x.to(DEV) for x in (k, v, ks, vs)]
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    api.copy_pages_q8(*g, i(1, 5, 9), i(0, 8, 2))                  # page 9 is outside the pool
    assert clean() == B.PKV_DEVERR_BAD_PAGE
    for x, y in zip((k, v, ks, vs), g):
        want = raw(x).clone()
        want[0], want[8] = want[1], want[5]
        assert torch.equal(raw(y).cpu(), want)


# -------------------------------------------------------------------------- eviction --


def run_evict(dtype, lens, budget, recent, H_kv, ps, bt=16, seed=0, out_of_place=False, weights=None, d=D):
    gen = torch.Generator().manual_seed(seed)
    S = len(lens)
    table, pages = tables(lens, ps, seed, spare=0)
    dst = table.clone()
    if out_of_place:
        for s, n in enumerate(lens):
            for i in range(-(-min(n, budget) // ps)):
                dst[s, i] = pages
                pages += 1
    k, ks = pool(dtype, pages, ps, bt, H_kv, gen)
    v, vs = pool(dtype, pages, ps, bt, H_kv, gen)
    if d != D:
        k, v = k[..., :d].contiguous(), v[..., :d].contiguous()
    stride = max(lens) + 5
    w = torch.rand((S, H_kv, stride), generator=gen) if weights is None else weights(S, H_kv, stride, gen)
    g = [x if x is None else x.to(DEV) for x in (k, v, w, table, torch.tensor(lens, dtype=torch.int32), dst, ks, vs)]
    kept, new = api.evict(g[0], g[1], g[2], g[3], g[4], budget, recent, max(max(lens), 1), dst_table=g[5],
                          k_scales=g[6], v_scales=g[7])
    torch.cuda.synchronize()
    want = evict(w, lens, budget, recent)
    kept, new = kept.cpu(), new.cpu()
    for s, L in enumerate(lens):
        m = min(L, budget)
        assert int(new[s]) == m
        for h in range(H_kv):
            ids = want[s][h]
            assert kept[s, h].tolist() == ids + [-1] * (budget - m), f"kept tokens of {s}, {h}"
            ids = torch.tensor(ids, dtype=torch.long)
            exp = torch.cat([w[s, h, ids], torch.zeros(L - m), w[s, h, L:]])
            assert torch.equal(g[2][s, h].cpu().nan_to_num(7), exp.nan_to_num(7)), "weights"
            for codes, scales, now, now_s in ((k, ks, g[0], g[6]), (v, vs, g[1], g[7])):
                j = torch.arange(m)
                at = (dst[s].long()[j // ps], j % ps, torch.full_like(j, h))
                of = (table[s].long()[ids // ps], ids % ps, torch.full_like(j, h))
                x = raw(codes)[of]
                if scales is None:
                    assert torch.equal(raw(now).cpu()[at], x)
                    continue
                old = scales[of[0], of[1] // bt, h]
                block_max = torch.stack([old[b:b + bt].max() for b in range(0, m, bt)]) if m else old
                new_s = block_max.repeat_interleave(bt)[:m]
                assert torch.equal(now_s.cpu()[at[0], at[1] // bt, h], new_s), "scales"
                y = nearest(x.view(dtype).double() * old.double()[:, None] / new_s.double()[:, None], dtype)
                assert torch.equal(raw(now).cpu()[at].view(dtype).double(), y), "codes"
    # a page that is nobody's destination is as it was
    mine = set()
    for s, L in enumerate(lens):
        mine |= set(dst[s, :-(-min(L, budget) // ps)].tolist())
    for p in set(range(pages)) - mine:
        assert torch.equal(raw(g[0])[p].cpu(), raw(k)[p]) and torch.equal(raw(g[1])[p].cpu(), raw(v)[p])


EVICT = [
    # lens, budget, recent, H_kv, page, block
    ([1, 5, 16, 17], 5, 2, 2, 16, 16),
    ([0, 3, 200], 64, 64, 1, 16, 16),            # an empty sequence; nothing but the recent ones
    ([300, 1000, 129], 100, 0, 3, 32, 32),       # no recent ones
    ([2500, 40, 1024], 1024, 10, 2, 64, 16),     # longer than one sweep of the selection; exactly the budget
    ([3000], 1100, 33, 2, 256, 128),             # more than one chunk of rows
    ([1025, 700], 1, 1, 1, 128, 64),
    # the selection's other sizes: more than 4096, 8192, 16384 tokens, and rows read in several segments
    ([5000, 4097], 700, 100, 1, 64, 32),
    ([9000, 12], 2000, 0, 1, 256, 256),
    ([20000], 9000, 8999, 1, 128, 16),
    ([70000, 33000], 33500, 500, 1, 256, 64),
    ([37 * (i % 5) + i for i in range(60)], 50, 7, 6, 16, 16),      # many pairs: narrow CTAs, wide slices
]


@pytest.mark.parametrize("place", ["in place", "to fresh pages"])
@pytest.mark.parametrize("dtype", [BF16, torch.float32, I8, E4M3], ids=["bf16", "f32", "i8", "e4m3"])
@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict(dtype, case, place):
    lens, budget, recent, H_kv, ps, bt = EVICT[case]
    run_evict(dtype, lens, budget, recent, H_kv, ps, bt, seed=case, out_of_place=place != "in place")


@pytest.mark.parametrize("kind", ["equal", "few values", "infinities and NaN", "negative", "signed zeros"])
def test_evict_orders_weights(kind):
    def weights(S, H, n, gen):
        x = torch.rand((S, H, n), generator=gen)
        if kind == "equal":
            return torch.full_like(x, 0.25)
        if kind == "few values":
            return (x * 4).floor() / 4
        if kind == "negative":
            return x - 0.5
        if kind == "signed zeros":
            return torch.where(x < 0.5, -0.0, 0.0)
        x[..., ::7] = float("nan")
        x[..., 3::11] = float("inf")
        x[..., 5::13] = -float("inf")
        return x
    run_evict(BF16, [500, 77, 1300], 130, 17, 2, 16, seed=5, weights=weights)


@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "f32"])
def test_evict_head_dim_64(dtype):
    run_evict(dtype, [100, 333], 90, 8, 3, 32, seed=6, d=64)


def test_evict_flags_bad_pages_and_lengths():
    gen = torch.Generator().manual_seed(0)
    k, _ = pool(BF16, 8, 16, 16, 1, gen)
    g = k.to(DEV)
    v = g.clone()
    table = torch.tensor([[0, 99, 2, 3], [4, 5, 6, 7]], dtype=torch.int32, device=DEV)
    w = torch.zeros((2, 1, 64), device=DEV)
    w[0, 0, 16:20] = 5                                            # tokens of the bad page are the heaviest
    lens = torch.tensor([64, 1000], dtype=torch.int32, device=DEV)
    kept, new = api.evict(g, v, w, table, lens, 16, 8, 64)
    assert clean() == B.PKV_DEVERR_BAD_PAGE | B.PKV_DEVERR_BAD_LEN
    assert new.tolist() == [16, 16]
    assert kept[0, 0].tolist() == [0, 1, 2, 3, 16, 17, 18, 19] + list(range(56, 64))
    assert kept[1, 0].tolist() == list(range(8)) + list(range(56, 64))
    got = g.cpu()
    assert torch.equal(got[0, :4], k[0, :4]) and torch.equal(got[0, 8:16], k[3, 8:16])
    assert torch.equal(got[0, 4:8], k[0, 4:8])                    # rows of the bad page are not moved
    assert torch.equal(got[4, :8], k[4, :8]) and torch.equal(got[4, 8:16], k[7, 8:16])


@pytest.mark.parametrize("dtype", [BF16, I8], ids=["bf16", "i8"])
def test_evict_captured_and_replayed_on_two_streams(dtype):
    """Two captured evictions over one pool (other pages, weights and workspaces), replayed at once, thrice."""
    gen = torch.Generator().manual_seed(9)
    table, pages = tables([900, 1300, 700, 2000], 32, 1)
    k, ks = pool(dtype, pages, 32, 16, 3, gen)
    v, vs = pool(dtype, pages, 32, 16, 3, gen)
    w = torch.rand((4, 3, 2000), generator=gen)
    first = [x if x is None else x.to(DEV) for x in (k, v, ks, vs, w)]
    live = [x if x is None else x.clone() for x in first]
    lens = torch.tensor([900, 1300, 700, 2000], dtype=torch.int32, device=DEV)
    table = table.to(DEV)

    def run(x, rows, ws=None):
        at = slice(*rows)
        return api.evict(x[0], x[1], x[4][at], table[at], lens[at], 300, 50, 2000, k_scales=x[2], v_scales=x[3],
                         workspace=ws)

    want = [x if x is None else x.clone() for x in first]
    kept = [run(want, r)[0] for r in ((0, 2), (2, 4))]
    n = B.paged_kv_evict_workspace_size(2, 3, 300, 16, B.PKV_I8)
    graphs, got, spaces = [], [], [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    for i, r in enumerate(((0, 2), (2, 4))):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got.append(run(live, r, spaces[i] if dtype == I8 else None)[0])
        graphs.append((g, s))
    for rep in range(3):
        for x, y in zip(live, first):
            if x is not None:
                x.copy_(y)
        torch.cuda.synchronize()
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, kept))
        assert all(torch.equal(raw(a), raw(b)) for a, b in zip(live, want) if a is not None)


# ------------------------------------------------------------------ used together --


@pytest.mark.parametrize("dtype", [I8, E4M3], ids=["i8", "e4m3"])
def test_serving_under_a_budget(dtype):
    """A prompt, decode steps that append, attend and accumulate, a fork, and an eviction of both sequences whenever
    one passes its budget, all through the allocator; at every step attention is checked against the values that the
    cache holds, and after the last eviction the kept rows against what was appended."""
    H, H_kv, ps, budget, recent = 8, 2, 16, 96, 32
    gen = torch.Generator().manual_seed(11)
    alloc = B.PageAllocator(64, ps, 24)
    k = torch.zeros((64, ps, H_kv, D), dtype=dtype, device=DEV) if dtype == I8 else \
        torch.zeros((64, ps, H_kv, D), device=DEV).to(dtype)
    v = k.clone()
    ks = torch.full((64, 1, H_kv), float("nan"), device=DEV)
    vs = ks.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    seqs, w = [7], torch.zeros((2, H_kv, 24 * ps), device=DEV)
    alloc.add_seq(7)

    def extend(new):
        starts, cows = [], []
        for s, n in zip(seqs, new):
            start, cow = alloc.reserve(s, n)
            starts.append(start)
            if cow:
                cows.append(cow)
        if cows:
            api.copy_pages_q8(k, v, ks, vs, i32([a for a, _ in cows]), i32([b for _, b in cows]))
        rows, lens = alloc.block_table(seqs)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        kn, vn = (torch.randn((cu[-1], H_kv, D), generator=gen).to(BF16).to(DEV) for _ in range(2))
        api.append_q8(kn, vn, i32(cu), i32(starts), i32(rows), k, v, ks, vs)
        return i32(rows), lens

    evictions = 0
    for step in range(60):
        if step == 20:
            alloc.fork(7, 8)
            seqs.append(8)
            w[1] = w[0]
        table, lens = extend([70] if step == 0 else [1 if step % 9 else 5] * len(seqs))
        S = len(seqs)
        q = torch.randn((S, H, 1, D), generator=gen).to(BF16).to(DEV)
        before = w[:S].clone()
        out = api.paged_weights(q, k, v, table, i32(lens), ps, True, D ** -0.5, max(lens), w[:S],
                                k_scales=ks, v_scales=vs)
        want, ww, spread, size = attend(q, k, v, ks, vs, table, lens, True, D ** -0.5)
        rel = math.expm1(2 * 128 * 2.0 ** -24 * size) + 2.0 ** -20
        assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 + rel) * 1.01 * spread).all()
        if max(lens) > budget:
            new = [min(n, budget) for n in lens]
            alloc.compact(seqs, new)
            rows, _ = alloc.block_table(seqs)
            old = [[values(x, sc, table[s], lens[s], h)[0] for h in range(H_kv)] for x, sc in ((k, ks), (v, vs))
                   for s in range(S)]
            kept, new_lens = api.evict(k, v, w[:S], table, i32(lens), budget, recent, max(lens),
                                       dst_table=i32(rows), k_scales=ks, v_scales=vs)
            assert new_lens.tolist() == new
            evictions += 1
            for n, (x, sc) in enumerate(((k, ks), (v, vs))):
                for s in range(S):
                    for h in range(H_kv):
                        got, _ = values(x, sc, i32(rows)[s], new[s], h)
                        exp = old[n * S + s][h][kept[s, h, :new[s]].long()]
                        # requantising moves a value by at most half a step of its new block:
                        # s / 2 for int8, 2^-4 of the value (or 2^-10 s) for e4m3
                        step_s = sc[i32(rows)[s].long()[torch.arange(new[s], device=DEV) // ps], 0, h].double()[:, None]
                        tol = 0.5 * step_s if dtype == I8 else torch.maximum(2.0 ** -4 * exp.abs(), 2.0 ** -10 * step_s)
                        assert ((got - exp).abs() <= tol * (1 + 1e-6)).all()
            w[:S, :, budget:] = 0
    assert evictions >= 2 and S == 2
    alloc.free_seq(7)
    alloc.free_seq(8)
    assert alloc.num_free() == 64
