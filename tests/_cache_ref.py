"""Plain float64 forms of the 8-bit cache, attention weights and eviction, one
sequence, head and block at a time (test infrastructure; no code of the library)."""

import math

import torch

D = 128
QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
TINY = 2.0 ** -126
POISON = {torch.int8: 127, torch.float8_e4m3fn: float("nan"), torch.bfloat16: float("nan"),
          torch.float32: float("nan")}


def nearest(y, dtype):
    """Float64 quotients -> values of the nearest codes, ties to even, by a table of all codes."""
    if dtype == torch.int8:
        grid = torch.arange(-127, 128, dtype=torch.float64)
        even = torch.arange(-127, 128) % 2 == 0
    else:
        pos = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        grid = torch.cat([-pos.flip(0)[:-1], pos])
        even = torch.cat([torch.arange(126, 0, -1), torch.arange(0, 127)]) % 2 == 0
    y = y.cpu()
    hi = torch.searchsorted(grid, y.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - y, y - grid[lo]
    return torch.where((up < down) | ((up == down) & even[hi]), grid[hi], grid[lo])


def scale_of(amax: float, qmax: float) -> float:
    """The float32 nearest to amax / qmax."""
    return float(torch.tensor(amax / qmax, dtype=torch.float64).float())


def append(new, lens, cu, table, codes, scales):
    """codes [P, ps, H, d] and scales [P, ps/bt, H] after appending `new` [n, H, d] (all on the CPU).

    Returns (code values float64, scales float32)."""
    P, ps, H, _ = codes.shape
    bt = ps // scales.shape[1]
    val, sc = codes.double().clone(), scales.clone()
    for s, start in enumerate(lens):
        rows = new[cu[s]:cu[s + 1]].double()
        pos = start
        while pos < start + rows.shape[0]:
            end = min(start + rows.shape[0], (pos // bt + 1) * bt)
            page, blk, off = int(table[s, pos // ps]), pos % ps // bt, pos % bt
            if not 0 <= page < P:
                pos = end
                continue
            for h in range(H):
                x = rows[pos - start:end - start, h]
                old = float(sc[page, blk, h]) if off else 0.0
                o = pos % ps
                if not torch.isfinite(x).all() or math.isnan(old):
                    sc[page, blk, h] = float("nan")
                    val[page, o:o + end - pos, h] = 0
                    continue
                new_s = max(old, scale_of(float(x.abs().max()), QMAX[codes.dtype]), TINY)
                if off and new_s > old:
                    b0 = blk * bt
                    val[page, b0:b0 + off, h] = nearest(val[page, b0:b0 + off, h] * old / new_s, codes.dtype)
                val[page, o:o + end - pos, h] = nearest(x / new_s, codes.dtype)
                sc[page, blk, h] = new_s
            pos = end
    return val, sc


def values(codes, scales, table_row, n, h):
    """Float64 [n, d]: head h of a sequence's first n tokens, NaN rows where the table has no page."""
    P, ps = codes.shape[:2]
    t = torch.arange(n, device=codes.device)
    page = table_row.to(codes.device).long()[t // ps]
    ok = (page >= 0) & (page < P)
    page = torch.where(ok, page, 0)
    raw = codes.view(torch.uint8) if codes.dtype == torch.float8_e4m3fn else codes
    x = raw[page, t % ps, h].view(codes.dtype).double()
    if scales is not None:
        x = x * scales[page, t % ps // (ps // scales.shape[1]), h].double()[:, None]
    return x, ok


def attend(q, k_pages, v_pages, ks, vs, table, lens, causal, scale):
    """(out, weights, spread, size): out [S, H, q_len, d]; weights list of [H_kv, n]; spread = sum_j p |v| and
    size = the largest sum of |q| |k| * scale, which rounding bounds are made of.  Float64."""
    S, H, ql, d = q.shape
    H_kv = k_pages.shape[2]
    G = H // H_kv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(out)
    weights, size = [], 0.0
    for s in range(S):
        n = int(lens[s])
        w = torch.zeros((H_kv, n), dtype=torch.float64, device=q.device)
        for h in range(H_kv):
            k, ok = values(k_pages, ks, table[s], n, h)
            v, _ = values(v_pages, vs, table[s], n, h)
            k, v = k[ok], v[ok]
            qq = q[s, h * G:(h + 1) * G].double()
            x = qq @ k.T * scale
            size = max(size, float((qq.abs() @ k.abs().T).max()) * scale) if k.numel() else size
            if causal:
                see = torch.arange(n, device=q.device)[None] <= torch.arange(ql, device=q.device)[:, None] + (n - ql)
                x = x.masked_fill(~see[:, ok], -math.inf)
            p = torch.softmax(x, -1)
            p = torch.where(torch.isneginf(x).all(-1, keepdim=True), 0.0, p)
            out[s, h * G:(h + 1) * G] = p @ v
            spread[s, h * G:(h + 1) * G] = p @ v.abs()
            w[h, ok] = p.sum((0, 1))
        weights.append(w)
    return out, weights, spread, size


def evict(weights, lens, budget, recent):
    """kept[s][h]: ascending list of the tokens that stay (weights on the CPU, float32)."""
    kept = []
    for s, L in enumerate(lens):
        heads = []
        for h in range(weights.shape[1]):
            if L <= budget:
                heads.append(list(range(L)))
                continue
            old = L - recent
            w = [float(x) for x in weights[s, h, :old]]
            order = sorted(range(old), key=lambda t: (1 if math.isnan(w[t]) else 0, -w[t] if not math.isnan(w[t]) else 0, t))
            heads.append(sorted(order[:budget - recent]) + list(range(old, L)))
        kept.append(heads)
    return kept
