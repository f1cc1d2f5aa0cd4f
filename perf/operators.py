"""Measured cases of the 8-bit paged cache and of eviction by accumulated attention weight.

Four operators, which a server with a bounded cache uses together:

* ``append``  writes new K/V rows into a cache held in 8 bits (int8 or e4m3 codes, one float32
  scale for each block of tokens and kv head), growing a block's scale where a new row needs it;
* ``attend``  is attention over that cache, for single tokens and for chunks of a prompt;
* ``weights`` is attention that also adds every key's softmax weight, summed over the query rows
  and the query heads of its kv head, to an accumulator;
* ``evict``   keeps, for each sequence and kv head, the most recent tokens and those of the
  largest accumulated weight, and compacts the cache.

The plain forms below are elementary torch operations in float32, or float64 where a value next
to a rounding border decides a code.
"""

import math
import random

import torch

own = False

D = 128
I8, E4M3, BF16 = "int8", "e4m3", "bf16"
QMAX = {I8: 127.0, E4M3: 448.0}
CODE = {I8: torch.int8, E4M3: torch.float8_e4m3fn, BF16: torch.bfloat16}
TINY = 2.0 ** -126          # the smallest scale


# ------------------------------------------------------------------------------------ cases --
def _lens(case):
    """The sequences' lengths: spread over [lo, hi], the longest one hi."""
    r = random.Random(case["lens_seed"])
    return [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"] - 1)]


def _new(case):
    """How many tokens each sequence appends."""
    r = random.Random(case["lens_seed"] + 1)
    return [case["new_hi"]] + [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"] - 1)]


def _case(op, cache, seqs, lo, hi, H, H_kv, page, block=0, name=None, **more):
    c = dict(op=op, cache=cache, seqs=seqs, lo=lo, hi=hi, H=H, H_kv=H_kv, page=page, block=block,
             lens_seed=more.pop("lens_seed", 1), **more)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of 64 running sequences: a row each, most into a block already begun
        _case("append", I8, 64, 20, 8000, 8, 8, 16, 16, "append a step, int8", new_lo=1, new_hi=1),
        # the prompts of a batch, ragged, into empty sequences and behind cached prefixes
        _case("append", E4M3, 12, 0, 700, 8, 8, 64, 32, "append prompts, e4m3", new_lo=300, new_hi=4100),
        # one user, a short context: latency
        _case("attend", I8, 1, 437, 437, 32, 8, 16, 16, "decode one short, int8", q_len=1),
        # a full batch of one query head per kv head
        _case("attend", I8, 64, 512, 8192, 32, 32, 16, 16, "decode a batch, int8", q_len=1),
        # long contexts, grouped heads, large pages with larger blocks
        _case("attend", E4M3, 16, 600, 32768, 64, 8, 256, 64, "decode long, e4m3", q_len=1),
        # a chunk of a long prompt against what is cached of it
        _case("attend", I8, 2, 4000, 9001, 32, 8, 64, 16, "prompt chunk, int8", q_len=1025),
        # decode steps under a budget: the weights choose what will be evicted
        _case("weights", BF16, 64, 512, 8192, 64, 8, 16, 0, "weights of a step, bf16", q_len=1),
        _case("weights", E4M3, 8, 2000, 30001, 32, 8, 64, 32, "weights of a step, e4m3", q_len=1),
        # the weights of a whole prompt, before its first eviction
        _case("weights", BF16, 1, 4096, 4096, 32, 8, 16, 0, "weights of a prompt, bf16", q_len=4096),
        # one short sequence: latency
        _case("evict", BF16, 1, 1000, 1000, 8, 8, 16, 0, "evict one short, bf16", budget=256, recent=64),
        # a batch brought back to its budget
        _case("evict", BF16, 32, 2500, 8192, 8, 8, 16, 0, "evict a batch, bf16", budget=2048, recent=512),
        _case("evict", I8, 8, 3000, 32768, 8, 8, 64, 32, "evict long, int8", budget=4111, recent=777),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weights", "weights", "evict"])
    page = rng.choice([16, 32, 64, 128, 256])
    block = rng.choice([b for b in (16, 32, 64, 128, 256) if b <= page])
    cache = rng.choice([I8, E4M3])
    seed = rng.randrange(1 << 20)
    H_kv = rng.choice([1, 2, 4, 8])
    if op == "append":
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 4000)
        new_hi = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(3, 24000 // seqs))
        return _case(op, cache, seqs, 0, hi, H_kv, H_kv, page, block, new_lo=1, new_hi=new_hi, lens_seed=seed)
    if op == "evict":
        cache = rng.choice([BF16, BF16, I8, E4M3])
        seqs = _log_int(rng, 1, 32)
        hi = _log_int(rng, 40, min(32768, 200000 // seqs))
        recent = _log_int(rng, 1, max(2, hi // 8))
        budget = recent + _log_int(rng, 1, max(2, hi // 3))
        return _case(op, cache, seqs, max(1, hi // 3), hi, H_kv, H_kv, page, 0 if cache == BF16 else block,
                     budget=budget, recent=recent, lens_seed=seed)
    H = H_kv * rng.choice([1, 2, 4, 5, 8])
    if op == "weights":
        cache = rng.choice([BF16, I8, E4M3])
    if rng.random() < 0.6:
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(32768, 250000 // seqs))
        return _case(op, cache, seqs, 1, hi, H, H_kv, page, 0 if cache == BF16 else block, q_len=1, lens_seed=seed)
    seqs = rng.choice([1, 1, 2, 3])
    q_len = _log_int(rng, 2, 2048)
    hi = q_len + _log_int(rng, 1, 6000)
    while seqs * H * q_len * hi > 5e8:
        q_len, hi = q_len - q_len // 3, hi - q_len // 3
    return _case(op, cache, seqs, q_len, hi, H, H_kv, page, 0 if cache == BF16 else block, q_len=q_len, lens_seed=seed)


def work(case):
    lens, kv = _lens(case), case["H_kv"]
    one = 2 if case["cache"] == BF16 else 1
    row = 2 * kv * D * one                                          # K and V of a token
    scales = 0 if case["cache"] == BF16 else 2 * kv * 4 / case["block"]   # per token
    if case["op"] == "append":
        n = sum(_new(case))
        return {"bytes": n * (2 * kv * D * 2 + row + scales), "flops": 4.0 * n * 2 * kv * D}
    if case["op"] == "evict":
        kept = sum(min(t, case["budget"]) for t in lens)
        # the weights read, the kept rows read and written, the kept weights and indices written
        return {"bytes": 4 * kv * sum(lens) + kept * (2 * row + 2 * scales + 8 * kv), "flops": float(kv * sum(lens))}
    q = case["q_len"]
    total = sum(lens)
    pairs = case["H"] * sum(q * t - q * (q - 1) // 2 for t in lens)
    b = total * (row + scales) + 2 * case["seqs"] * case["H"] * q * D * 2
    if case["op"] == "weights":
        b += 8 * kv * total
    return {"bytes": float(b), "flops": 4.0 * D * pairs}


# ----------------------------------------------------------------------------------- inputs --
def _tables(pages_each, first, gen, dev):
    """int32 [S, most pages], -1 padded: the pool's pages from `first` on, shuffled."""
    n = torch.tensor(pages_each, device=dev)
    end = torch.cumsum(n, 0)
    perm = torch.randperm(int(end[-1]), generator=gen, device=dev) + first
    k = torch.arange(int(n.max()), device=dev)
    at = (end - n)[:, None] + k
    table = torch.where(k < n[:, None], perm[at.clamp(max=perm.numel() - 1)], -1)
    return table.to(torch.int32).contiguous(), int(end[-1])


def _rows(shape, gen, dev):
    """bf16 K/V rows: normal, with some head dims far larger than the rest."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    big = torch.rand(shape[-1], generator=gen, device=dev) < 0.03
    return x * torch.where(big, 6.0, 1.0).to(torch.bfloat16)


def _pool(case, pages, gen, dev):
    """(pages, scales) of a filled cache."""
    shape = (pages, case["page"], case["H_kv"], D)
    if case["cache"] == BF16:
        return _rows(shape, gen, dev), None
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    codes = (x * (QMAX[case["cache"]] / 3.7)).float()
    codes = codes.round_().clamp_(-127, 127).to(torch.int8) if case["cache"] == I8 else \
        codes.clamp_(-448, 448).to(torch.float8_e4m3fn)
    s = torch.randn((pages, case["page"] // case["block"], case["H_kv"]), generator=gen, device=dev)
    return codes, (s * 0.3).exp() * (3.7 / QMAX[case["cache"]])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, page = _lens(case), case["page"]
    s = {"case": case, "scale": 1.0 / math.sqrt(D)}
    if case["op"] == "append":
        new = _new(case)
        s["table"], pages = _tables([-(-(a + b) // page) for a, b in zip(lens, new)], 0, gen, dev)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu_new"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["start"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["k_new"] = _rows((cu[-1], case["H_kv"], D), gen, dev)
        s["v_new"] = _rows((cu[-1], case["H_kv"], D), gen, dev)
        s["k"], s["ks"] = _pool(case, pages, gen, dev)
        s["v"], s["vs"] = _pool(case, pages, gen, dev)
        return s
    s["table"], pages = _tables([-(-t // page) for t in lens], 0, gen, dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["max_len"] = max(lens)
    s["src_pages"] = pages
    if case["op"] == "evict":
        kept = [-(-min(t, case["budget"]) // page) for t in lens]
        s["dst"], more = _tables(kept, pages, gen, dev)
        pad = s["table"].shape[1] - s["dst"].shape[1]
        s["dst"] = torch.nn.functional.pad(s["dst"], (0, pad), value=-1).contiguous()
        pages += more
    s["k"], s["ks"] = _pool(case, pages, gen, dev)
    s["v"], s["vs"] = _pool(case, pages, gen, dev)
    if case["op"] == "evict":
        # accumulated weights: most near zero, a few heavy; some exactly equal
        w = torch.rand((len(lens), case["H_kv"], max(lens)), generator=gen, device=dev)
        s["weights"] = ((w ** 8) * 512).round() / 64
        s["weights_out"] = torch.zeros_like(s["weights"])
        return s
    shape = (len(lens), case["H"], case["q_len"], D)
    s["q"] = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16) * 2
    if case["op"] == "weights":
        s["weights"] = torch.rand((len(lens), case["H_kv"], max(lens)), generator=gen, device=dev)
    return s


# ------------------------------------------------------------------------------ plain forms --
def _values(codes, scales, block):
    """What a pool [P, page, H_kv, d] holds, as float32."""
    if scales is None:
        return codes
    P, page, H_kv, d = codes.shape
    return (codes.view(P, page // block, block, H_kv, d).float() * scales[:, :, None, :, None]).view(P, page, H_kv, d)


def _raw(x):
    """Codes as a type that every indexing operation takes."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _gather(codes, scales, case, table, T):
    """float32 [S, H_kv, T, d]: each sequence's rows through its table (rows of no page: page 0)."""
    t = torch.arange(T, device=table.device)
    page = table.clamp(min=0).long()[:, t // case["page"]]
    off = t % case["page"]
    x = _raw(codes)[page, off].view(codes.dtype).float()                                   # [S, T, H_kv, d]
    if scales is not None:
        x = x * scales[page, off // case["block"]][..., None]
    return x.transpose(1, 2)


def _plain_attend(s):
    case, T, q = s["case"], s["max_len"], s["q"]
    S, H, q_len, _ = q.shape
    kv = case["H_kv"]
    k = _gather(s["k"], s["ks"], case, s["table"], T)
    qf = q.float().view(S, kv, H // kv * q_len, D)
    x = torch.matmul(qf, k.transpose(2, 3)).view(S, kv, H // kv, q_len, T) * s["scale"]
    del k
    last = torch.arange(q_len, device=q.device) + (s["lens"][:, None] - q_len)       # [S, q_len]
    seen = torch.arange(T, device=q.device) <= last[..., None]                       # [S, q_len, T]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    del x
    p = p / p.sum(-1, keepdim=True)
    v = _gather(s["v"], s["vs"], case, s["table"], T)
    out = torch.matmul(p.view(S, kv, H // kv * q_len, T), v).view(S, H, q_len, D).to(torch.bfloat16)
    if case["op"] == "attend":
        return out
    s["weights"].add_(p.sum((2, 3)))
    return out, s["weights"]


def _to_codes(y, cache):
    """Quotients in float64 -> the nearest codes, ties to even."""
    if cache == I8:
        return y.round().clamp(-127, 127).to(torch.int8)
    step = torch.exp2(torch.frexp(y.abs())[1].clamp(min=-5).double() - 4)    # 4 significand bits, from 2^-9 up
    return ((y / step).round() * step).clamp(-448, 448).float().to(torch.float8_e4m3fn)


def _plain_append_one(s, new, pages, scales):
    """Appends one of K and V in place."""
    case = s["case"]
    page, block, cache, H_kv = case["page"], case["block"], case["cache"], case["H_kv"]
    per = page // block
    dev = new.device
    cu, start = s["cu_new"].long(), s["start"].long()
    row = torch.arange(new.shape[0], device=dev)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = start[seq] + row - cu[seq]
    slot = s["table"].long()[seq, pos // page] * page + pos % page
    blk, off = slot // block, slot % block
    n_blk = pages.shape[0] * per
    amax = torch.zeros((n_blk, H_kv), device=dev)
    amax.scatter_reduce_(0, blk[:, None].expand(-1, H_kv), new.float().abs().amax(-1), "amax")
    first = torch.full((n_blk,), block, device=dev).scatter_reduce_(0, blk, off, "amin")   # block: not touched
    touched = first < block
    s_old = scales.view(n_blk, H_kv)
    kept = torch.where((first == 0)[:, None], torch.zeros_like(s_old), s_old)   # a block begun anew has no scale yet
    # (a tensor over a number may be a product with its inverse; a scale is the rounded quotient)
    s_new = torch.maximum(kept, (amax.double() / QMAX[cache]).float()).clamp(min=TINY)
    s_new = torch.where(touched[:, None], s_new, s_old)
    old = _raw(pages.view(n_blk, block, H_kv, D))
    grown = touched[:, None] & (first > 0)[:, None] & (s_new > s_old)           # [n_blk, H_kv]
    change = (torch.arange(block, device=dev) < first[:, None])[:, :, None] & grown[:, None]
    at = change.nonzero(as_tuple=True)                                          # (block, offset, head)
    y = old[at].view(pages.dtype).double() * (s_old[at[0], at[2]].double())[:, None] / (s_new[at[0], at[2]].double())[:, None]
    old[at] = _raw(_to_codes(y, cache))
    codes = _to_codes(new.double() / s_new[blk].double()[..., None], cache)
    _raw(pages.view(n_blk * block, H_kv, D))[slot] = _raw(codes)
    scales.copy_(s_new.view(scales.shape))


def _plain_evict(s):
    case, T = s["case"], s["max_len"]
    budget, recent, page, block = case["budget"], case["recent"], case["page"], case["block"]
    w, L = s["weights"][:, :, :T], s["lens"].long()
    S, kv, _ = w.shape
    dev = w.device
    t = torch.arange(T, device=dev)
    new = torch.minimum(L, torch.tensor(budget, device=dev))
    live = t < L[:, None]
    # the recent tokens rank first, then the heaviest, ties to the lowest index; dead ones last
    rank = torch.where((live & (t >= (L - recent)[:, None]))[:, None], math.inf, w)
    rank = torch.where(live[:, None], rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    j = torch.arange(order.shape[-1], device=dev)
    has = (j < new[:, None])[:, None].expand_as(order)
    kept = torch.sort(torch.where(has, order, T), dim=-1).values        # ascending, T where none
    src = kept.clamp(max=T - 1)
    s["weights_out"][:, :, :T].masked_fill_(live[:, None], 0.0)
    s["weights_out"][:, :, : order.shape[-1]].copy_(
        torch.where(has, w.gather(-1, src), s["weights_out"][:, :, : order.shape[-1]]))
    head = torch.arange(kv, device=dev)[None, :, None]
    spage = s["table"].long().gather(1, (src // page).flatten(1)).view_as(src)
    at_seq, at_head, at_j = has.nonzero(as_tuple=True)
    dpage = s["dst"].long()[at_seq, at_j // page]
    for pages, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        rows = _raw(pages)[spage, src % page, head][at_seq, at_head, at_j].view(pages.dtype)     # [n, d]
        if scales is not None:
            old = scales[spage, (src % page) // block, head][at_seq, at_head, at_j]
            grid = torch.zeros_like(scales)
            at = (dpage * (page // block) + at_j % page // block) * kv + at_head
            new_s = grid.view(-1).scatter_reduce_(0, at, old, "amax")[at]
            scales[dpage, at_j % page // block, at_head] = new_s
            rows = _to_codes(rows.double() * old.double()[:, None] / new_s.double()[:, None], case["cache"])
        _raw(pages)[dpage, at_j % page, at_head] = _raw(rows)
    pad = torch.full((S, kv, budget), -1, dtype=torch.int32, device=dev)
    pad[..., : order.shape[-1]] = torch.where(has, kept, -1).to(torch.int32)
    return pad, new.to(torch.int32)


# -------------------------------------------------------------------------------------- run --
def _held(s, first=0):
    """The pools' values from page `first` on."""
    block = s["case"]["block"]
    cut = lambda x: None if x is None else x[first:]  # noqa: E731
    return {"k": _values(cut(s["k"]), cut(s["ks"]), block), "v": _values(cut(s["v"]), cut(s["vs"]), block)}


def run(s):
    case = s["case"]
    if own:
        from paged_kv_cache_exact_b200 import api
        if case["op"] == "append":
            api.append_q8(s["k_new"], s["v_new"], s["cu_new"], s["start"], s["table"], s["k"], s["v"], s["ks"], s["vs"])
        elif case["op"] == "attend":
            return api.paged_q8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"], case["page"], True,
                                s["scale"], s["max_len"])
        elif case["op"] == "weights":
            out = api.paged_weights(s["q"], s["k"], s["v"], s["table"], s["lens"], case["page"], True, s["scale"],
                                    s["max_len"], s["weights"], k_scales=s["ks"], v_scales=s["vs"])
            return out, s["weights"]
        else:
            kept, lens = api.evict(s["k"], s["v"], s["weights"], s["table"], s["lens"], case["budget"], case["recent"],
                                   s["max_len"], dst_table=s["dst"], weights_out=s["weights_out"],
                                   k_scales=s["ks"], v_scales=s["vs"])
    elif case["op"] == "append":
        _plain_append_one(s, s["k_new"], s["k"], s["ks"])
        _plain_append_one(s, s["v_new"], s["v"], s["vs"])
    elif case["op"] == "evict":
        kept, lens = _plain_evict(s)
    else:
        return _plain_attend(s)
    if case["op"] == "append":
        return dict(_held(s), ks=s["ks"], vs=s["vs"])
    return dict(_held(s, s["src_pages"]), kept=kept, lens=lens, weights=s["weights_out"])


# ------------------------------------------------------------------------------------ exact --
def _nearest(y, cache):
    """Float64 quotients -> the values of the nearest codes, by looking them up among all codes."""
    if cache == I8:
        grid = torch.arange(-127, 128, dtype=torch.float64, device=y.device)
        odd = (torch.arange(-127, 128, device=y.device) % 2) != 0
    else:
        m = torch.arange(0, 127, device=y.device)                     # 0 .. 448, the code 127 is NaN
        e, f = m // 8, (m % 8).double()
        pos = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2(e.double() - 7))
        grid = torch.cat([-pos.flip(0)[:-1], pos])
        odd = torch.cat([(m % 2 != 0).flip(0)[:-1], m % 2 != 0])
    hi = torch.searchsorted(grid, y.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    up, down = grid[hi] - y, y - grid[lo]
    take_hi = (up < down) | ((up == down) & odd[lo])
    return torch.where(take_hi, grid[hi], grid[lo])


def exact(case, seed):
    s = prepare(case, seed)
    lens, page, block, kv = _lens(case), case["page"], case["block"], case["H_kv"]
    dev = s["k"].device

    def slots(table, n, first=0):
        at = torch.arange(first, first + n, device=dev)
        return table[at // page].long() * page + at % page

    if case["op"] == "append":
        got = {}
        for name, new, codes, scales in (("k", s["k_new"], s["k"], s["ks"]), ("v", s["v_new"], s["v"], s["vs"])):
            flat, sc = codes.view(-1, kv, D).double(), scales.view(-1, kv).double()
            cu = s["cu_new"].tolist()
            for i, begin in enumerate(lens):
                n = cu[i + 1] - cu[i]
                slot = slots(s["table"][i], n, begin)
                x = new[cu[i]:cu[i + 1]].double()
                left = begin % block                                   # rows of the first block that are there already
                lead = (slot[0] // block * block + torch.arange(left, device=dev)).long()
                groups = (torch.arange(n, device=dev) + left) // block
                top = torch.zeros((int(groups[-1]) + 1, kv), dtype=torch.float64, device=dev)
                top = top.index_reduce_(0, groups, x.abs().amax(-1), "amax")
                blk = slot[torch.arange(top.shape[0], device=dev) * block - left * (torch.arange(top.shape[0], device=dev) > 0)] // block
                need = (top / QMAX[case["cache"]]).float().double()    # a scale is a float32 number
                if left:
                    before = sc[blk[0]].clone()
                    need[0] = torch.maximum(need[0], before)
                    grew = need[0] > before
                    y = flat[lead] * before[:, None] / need[0][:, None]
                    flat[lead] = torch.where(grew[:, None], _nearest(y, case["cache"]), flat[lead])
                need = need.clamp(min=TINY)
                sc[blk] = need
                flat[slot] = _nearest(x / need[groups][..., None], case["cache"])
            per = sc.repeat_interleave(block, 0)
            got[name], got[name + "s"] = (flat * per[..., None]).view(codes.shape), sc.view(scales.shape)
        return got

    if case["op"] == "evict":
        w = s["weights"].double()
        T = s["max_len"]
        first = s["src_pages"] * page
        kept_all, got = None, {}
        keep_lists = []
        w_out = torch.zeros_like(w)
        for i, n in enumerate(lens):
            m = min(n, case["budget"])
            old = max(0, n - case["recent"])
            pick = max(0, m - min(case["recent"], n))
            # heaviest first, equal ones in the order of their index
            order = torch.sort(-w[i, :, :old], dim=-1, stable=True).indices[:, :pick]
            tail = torch.arange(n - (m - pick), n, device=dev).expand(kv, -1)
            kept = torch.cat([order.sort(-1).values, tail], 1)
            keep_lists.append(kept)
            w_out[i, :, :m] = w[i].gather(1, kept)
        for name, codes, scales in (("k", s["k"], s["ks"]), ("v", s["v"], s["vs"])):
            out = codes.view(-1, kv, D).double()
            if scales is not None:
                sc = scales.view(-1, kv).double()
            for i, kept in enumerate(keep_lists):
                m = kept.shape[1]
                src = slots(s["table"][i], lens[i])[kept]              # [kv, m]
                dst = slots(s["dst"][i], m)
                h = torch.arange(kv, device=dev)[:, None]
                x = out[src, h]
                if scales is not None:
                    was = sc[src // block, h]                          # [kv, m]
                    pad = torch.nn.functional.pad(was, (0, -m % block)).view(kv, -1, block).amax(-1)
                    now = pad.repeat_interleave(block, 1)[:, :m]
                    sc[dst.expand(kv, -1) // block, h] = now
                    x = _nearest(x * was[..., None] / now[..., None], case["cache"])
                out[dst.expand(kv, -1), h] = x
            if scales is not None:
                out = out * sc.repeat_interleave(block, 0)[..., None]
            got[name] = out[first:].view(-1, page, kv, D)
        got.update(kept=None, lens=None, weights=w_out)
        return got

    # attention, one sequence and kv head at a time
    q, ql, G = s["q"].double(), case["q_len"], case["H"] // kv
    out = torch.empty(q.shape, dtype=torch.float64, device=dev)
    w = s["weights"].double() if case["op"] == "weights" else None
    for i, n in enumerate(lens):
        slot = slots(s["table"][i], n)
        for h in range(kv):
            k = _head(s["k"], s["ks"], slot, h, block)
            v = _head(s["v"], s["vs"], slot, h, block)
            x = q[i, h * G:(h + 1) * G].reshape(G * ql, D) @ k.T * s["scale"]
            x = x.view(G, ql, n)
            see = torch.arange(n, device=dev)[None] <= torch.arange(ql, device=dev)[:, None] + (n - ql)
            p = torch.softmax(x.masked_fill(~see, -math.inf), -1)
            out[i, h * G:(h + 1) * G] = (p.view(G * ql, n) @ v).view(G, ql, D)
            if w is not None:
                w[i, h, :n] += p.sum((0, 1))
    return out if w is None else (out, w)


def _head(codes, scales, slot, h, block):
    """Float64 [n, d]: one kv head's rows."""
    page = codes.shape[1]
    x = _raw(codes)[slot // page, slot % page, h].view(codes.dtype).double()
    return x if scales is None else x * scales[slot // page, slot % page // block, h].double()[:, None]
